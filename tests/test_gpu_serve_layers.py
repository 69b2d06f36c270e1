"""The packed step's operators together, as examples/serve_layers.py uses them."""

import importlib.util
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SPEC = importlib.util.spec_from_file_location(
    "serve_layers", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                 "examples", "serve_layers.py"))
serve_layers = importlib.util.module_from_spec(SPEC)
SPEC.loader.exec_module(serve_layers)

LAYERS, HIDDEN = 2, 256


def say(*a):
    print("[gpu-case]", *a, file=sys.stderr, flush=True)


def server(batch, pages=40, tokens=200):
    return serve_layers.Server(batch, pages, tokens, layers=LAYERS, hidden=HIDDEN, heads=4,
                               kv_heads=2, dim=64, inner=320, page=16)


def step(s, x, new, release=None, T=None):
    """One step of the tokens x; their hidden states."""
    t = serve_layers.Step(s, T or len(x), max(new))
    t.x[:len(x)] = x
    t.new.copy_(torch.tensor(new))
    if release is not None:
        t.release.copy_(torch.tensor(release))
    return s.run(t)[:len(x)].clone(), t


def near(a, b):
    """Two ways to the same hidden states.  Attention may sum in another order, so that values round
    to the fp16 next to them, and so may what is rounded to 8 bits afterwards, by a step of a row's
    largest / 127 for values beside a border: a step for all of them is sqrt(HIDDEN) largest / 127,
    with largest at most 5 root mean squares in rows like these 4% of the row's norm, in each of two
    sublayers that a layer adds."""
    a, b = a.double(), b.double()
    return ((a - b).norm(dim=1) <= 0.04 * 2 * LAYERS * b.norm(dim=1)).all()


def tokens(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((n, HIDDEN), generator=g, device="cuda").half()


def test_requests_together_and_alone():
    """Prompts and single tokens packed, behind a common prompt, against each request alone on a
    server of its own that reads the common prompt as its own tokens."""
    say("serve_layers together and alone")
    common, B = tokens(48, 0), 4
    s = server(B)
    s.common(common)
    assert s.shared_pages == 3 and s.lens.tolist() == [48] * B
    prompts = [tokens(n, n) for n in (5, 40, 1, 17)]
    first, t = step(s, torch.cat(prompts), [len(p) for p in prompts], T=70)
    assert t.starts.tolist() == [0, 5, 45, 46, 63]
    assert t.positions.tolist() == [48 + i for p in prompts for i in range(len(p))] + [-1] * 7
    nexts = tokens(B, 9)
    second, _ = step(s, nexts, [1] * B)
    at = 0
    for b, p in enumerate(prompts):
        alone = server(1)
        want, _ = step(alone, torch.cat([common, p]), [48 + len(p)])
        assert near(first[at:at + len(p)], want[48:])
        want, _ = step(alone, nexts[b:b + 1], [1])
        assert near(second[b:b + 1], want)
        at += len(p)
    # all pages that are not free are the common ones and the requests' own, each once
    pages = -(-(s.lens - 48) // 16)
    assert int(s.count) == s.pages - 3 - int(pages.sum())
    own = torch.cat([s.table[b, 3:3 + int(n)] for b, n in enumerate(pages)])
    held = torch.cat([own, s.table[0, :3], s.free[:int(s.count)]]).tolist()
    assert sorted(held) == list(range(s.pages))


def test_a_request_ends_and_another_takes_its_place():
    say("serve_layers release")
    common = tokens(32, 1)
    s, fresh = server(2, pages=12), server(2, pages=12)
    for x in (s, fresh):
        x.common(common)
    step(s, tokens(90, 2), [50, 40])
    new = tokens(61, 3)
    # the second request ends; its place is taken while the first goes on
    got, _ = step(s, new, [1, 60], release=[0, 1])
    assert s.lens.tolist() == [83, 92]
    want, _ = step(fresh, new[1:], [0, 60])
    assert near(got[1:], want)
    # a step that there are no pages for leaves the request out
    _, t = step(s, tokens(100, 4), [99, 1])
    assert t.starts.tolist() == [0, 0, 1] and s.lens.tolist() == [83, 93]


def test_a_captured_step():
    """A graph of a single-token step, replayed with eager steps between, against eager ones."""
    say("serve_layers graph")
    B = 3
    s, eager = server(B), server(B)
    for x in (s, eager):
        x.common(tokens(16, 5))
        step(x, tokens(30, 6), [10, 15, 5])
    one = serve_layers.Step(s, B, 1)
    one.new.fill_(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run(one)
    for i in range(6):
        x = tokens(B, 10 + i)
        one.x.copy_(x)
        one.release.copy_(torch.tensor([0, int(i == 3), 0]))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = step(eager, x, [1] * B, release=[0, int(i == 3), 0])
        assert torch.equal(one.x, want)
        assert torch.equal(s.lens, eager.lens) and torch.equal(s.table, eager.table)
        if i == 2:  # an eager step of another shape between the replays
            y = tokens(7, 30)
            assert torch.equal(step(s, y, [3, 0, 4])[0], step(eager, y, [3, 0, 4])[0])


def test_the_example_runs(monkeypatch, capsys):
    say("serve_layers main")
    monkeypatch.setattr(sys, "argv", ["serve_layers.py", "--batch", "5", "--layers", "1",
                                      "--common", "128", "--prompt", "50", "--steps", "6"])
    serve_layers.main()
    assert "6 steps of 5 requests through 1 layers" in capsys.readouterr().out


def test_a_common_prompt_of_part_of_a_page_is_refused():
    with pytest.raises(ValueError, match="common prompt"):
        server(1).common(tokens(17, 0))
