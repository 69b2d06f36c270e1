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
