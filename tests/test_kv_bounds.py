"""Arguments of the key/value cache's calls at the ends of their ranges (CPU only)."""
import pytest

pytest.importorskip("torch")

from hadamard_rotated_w4a4_amd import ops  # noqa: E402


@pytest.mark.parametrize("sizes", [(512, 1, 24, 4, 256, 32768), (1, 1, 24, 4, 256, 131072), (300, 3, 8, 8, 64, 5000)])
def test_windows_of_any_length_leave_the_plan(sizes):
    """A window past every token is as none."""
    whole = ops.attention_kv_plan(*sizes)
    for window in (sizes[-1], 1 << 31, (1 << 63) - 97, (1 << 63) - 96, (1 << 63) - 1):
        assert ops.attention_kv_plan(*sizes, window) == whole, window
