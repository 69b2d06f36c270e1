"""examples/decode_layer.py with a prompt that its cache has no room for."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_decode_layer import block  # noqa: E402


def test_a_prompt_without_room_is_refused():
    """The cache would hold its last tokens only, and attention see those as all there are."""
    b = block()  # room for 70 tokens in pages of 16
    assert b.prompt(torch.randn((2, 80, 256), device="cuda").half()).shape == (2, 80, 256)
    with pytest.raises(ValueError, match="room for 80"):
        b.prompt(torch.randn((2, 81, 256), device="cuda").half())
    assert b.cache.lens.tolist() == [40, 40]
