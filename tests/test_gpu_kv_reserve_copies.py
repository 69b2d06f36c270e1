"""bcq_kv_reserve into other arrays, with tables and stacks of a size that decides between one launch
and two."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_kv_slots import Server, say  # noqa: E402


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,width,spare,T", [
    (64, 257, 300, 100), (64, 512, 64, 64),  # long tables
    (1, 3000, 5, 3), (8, 1025, 40, 500),
    (64, 4, 24000, 64), (64, 4, 25000, 64),  # either side of what one workgroup copies
    (3, 20, 300, 6069), (3, 20, 300, 6070),
    (65, 21, 40, 65), (100, 17, 100, 100), (200, 3, 20, 200), (256, 2, 3, 256),
])
def test_full_tables(B, width, spare, T, in_place):
    """Sequences whose tables are full but for a page, some of which end."""
    say("kv_reserve copies", B, width, spare, T, in_place)
    rng = np.random.default_rng(B + width)
    page = 16
    lens = (width - 1) * page - rng.integers(0, page, B)
    s = Server(lens, page, 0, B * (width - 1) + spare, width, seed=T)
    ends = (rng.random(B) < 0.1).astype(np.int32)
    new = np.where(ends, rng.integers(1, T // B + 2, B), T // B)
    s.step(new, ends, T, in_place)
    s.step(np.ones(B), None, T, in_place)
