"""Arguments of the key/value cache's calls at the ends of their ranges (CPU only)."""
import pytest

pytest.importorskip("torch")

from hadamard_rotated_w4a4_amd import ops  # noqa: E402
from hadamard_rotated_w4a4_amd._lib import W4A4Error  # noqa: E402


@pytest.mark.parametrize("sizes", [(512, 1, 24, 4, 256, 32768), (1, 1, 24, 4, 256, 131072), (300, 3, 8, 8, 64, 5000)])
def test_windows_of_any_length_leave_the_plan(sizes):
    """A window past every token is as none."""
    whole = ops.attention_kv_plan(*sizes)
    for window in (sizes[-1], 1 << 31, (1 << 63) - 97, (1 << 63) - 96, (1 << 63) - 1):
        assert ops.attention_kv_plan(*sizes, window) == whole, window


def test_an_empty_pool_has_a_geometry_too():
    """A pool of no pages is refused for the sizes that any pool is refused for."""
    assert [tuple(x.shape) for x in ops.new_kv_cache(0, 64, 2, 64, "cpu")] == [(0, 2, 2, 2, 2048), (0, 2, 2, 2)]
    for page, heads, dim in ((40, 2, 64), (0, 2, 64), (-32, 2, 64), (64, 0, 64), (64, 2, 100), (64, 8193, 64)):
        for pages in (0, 1):
            with pytest.raises(W4A4Error, match="no cache"):
                ops.new_kv_cache(pages, page, heads, dim, "cpu")
    with pytest.raises(W4A4Error, match="no cache"):
        ops.new_kv_cache(-1, 64, 2, 64, "cpu")
