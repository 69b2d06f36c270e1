"""That what a packed step's attention is held to tells the right tokens from their neighbours (no
GPU): mistakes planted in the definition, for the requests of test_gpu_serve_stages."""

import numpy as np
import pytest

from oracle import lowbit as lb
from test_lowbit_accuracy import definition, filled, outputs_hold

H, D, PAGE = 2, 64, 16


def outputs(c, q, length, table=None):
    one = lb.Cache(1, H, PAGE, D, c.table if table is None else table, [length])
    one.k, one.v, one.s = c.k, c.v, c.s
    return definition(one, q, D ** -0.5)[0]


MISTAKES = {
    "none": lambda c, q, n: outputs(c, q, n),
    "a token does not see itself": lambda c, q, n: outputs(c, q, n - 1),
    "a token sees the one behind it": lambda c, q, n: outputs(c, q, n + 1),
    # the last page for the first: as if a request had been given another's
    "a page that is not its own": lambda c, q, n: outputs(
        c, q, n, np.concatenate([c.table[:, -1:], c.table[:, 1:]], axis=1)),
}


@pytest.mark.parametrize("what", MISTAKES)
@pytest.mark.parametrize("length,n", [(53, 5), (88, 40), (49, 1), (65, 17), (32, 1), (92, 60)])
def test_mistakes_are_told(length, n, what):
    c = filled([length + 1 + PAGE], H, D, PAGE, -(-(length + 1) // PAGE) + 1, seed=length)
    q = np.random.default_rng(n).normal(size=(1, n, 4, D)).astype(np.float16)
    got = MISTAKES[what](c, q, length).astype(np.float16)
    assert outputs_hold(got, outputs(c, q, length)) == (what == "none")
