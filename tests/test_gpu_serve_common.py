"""examples/serve_layers.py: the prompt that its requests have in common."""

import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_serve_layers import serve_layers, server, step, tokens  # noqa: E402


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


def test_nothing_in_common(monkeypatch, capsys):
    """A common prompt of no tokens is none, from the command line too."""
    say("serve_layers common of 0")
    s, other = server(2), server(2)
    assert s.common(tokens(0, 0)).shape == (0, s.hidden)
    assert s.shared_pages == 0 and s.lens.tolist() == [0, 0] and int(s.count) == s.pages
    x = tokens(21, 1)
    assert torch.equal(step(s, x, [20, 1])[0], step(other, x, [20, 1])[0])
    monkeypatch.setattr(sys, "argv", ["serve_layers.py", "--batch", "3", "--layers", "1",
                                      "--common", "0", "--prompt", "20", "--steps", "2"])
    serve_layers.main()
    assert "2 steps of 3 requests through 1 layers" in capsys.readouterr().out


def unchanged(s, before):
    return all(torch.equal(a, b) for a, b in zip((s.lens, s.table, s.free, s.count), before))


@pytest.mark.parametrize("pages,room", [(2, 200), (40, 30)])
def test_a_common_prompt_that_there_is_no_room_for(pages, room):
    """Too few pages, or too few entries in the requests' tables: nothing is common, and what is
    served afterwards is served as if nothing had been asked."""
    say("serve_layers common without room", pages, room)
    s, other = (server(2, pages=pages, tokens=room) for _ in range(2))
    before = [t.clone() for t in (s.lens, s.table, s.free, s.count)]
    with pytest.raises(ValueError, match="common prompt"):
        s.common(tokens(48, 0))
    assert s.shared_pages == 0 and unchanged(s, before)
    x = tokens(21, 1)
    assert torch.equal(step(s, x, [16, 5])[0], step(other, x, [16, 5])[0])


@pytest.mark.parametrize("common", [0, 32])
def test_a_common_prompt_while_requests_are_served(common):
    """It would take the place of what they have cached, or of the common prompt before it."""
    say("serve_layers common of running requests", common)
    s, other = server(2), server(2)
    for x in (s, other):
        x.common(tokens(common, 2))
        if not common:
            step(x, tokens(5, 3), [0, 5])
    before = [t.clone() for t in (s.lens, s.table, s.free, s.count)]
    with pytest.raises(ValueError, match="common prompt"):
        s.common(tokens(16, 4))
    assert s.shared_pages == common // 16 and unchanged(s, before)
    x = tokens(21, 1)
    assert torch.equal(step(s, x, [20, 1])[0], step(other, x, [20, 1])[0])
