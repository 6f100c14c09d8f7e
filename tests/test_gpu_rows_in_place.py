"""One row normalised in place, where its row stride means nothing: a token's row
of a wider buffer, given as two views with different strides."""
import numpy as np
import pytest

import rows_twin as twin

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("target", ["x", "residual"])
def test_one_row_in_place_through_views_of_other_strides(target):
    from hadamard_rotated_w4a4_amd import _lib as ops
    k = 1056
    rng = np.random.default_rng(1)
    buf = torch.from_numpy(rng.standard_normal((7, 2 * k)).astype(np.float32)).cuda().half()
    other = torch.from_numpy(rng.standard_normal((1, k)).astype(np.float32)).cuda().half()
    want, v = twin.norm(buf[5:6, :k].float().cpu().numpy(), other.float().cpu().numpy(), torch.float16, None, 1e-6)
    kept = buf.clone()
    wide, narrow = buf[5:6, :k], buf[5, :k][None]
    assert wide.data_ptr() == narrow.data_ptr() and wide.stride(0) != narrow.stride(0)
    print(f"[gpu rows] one row in place, h is {target}", flush=True)
    x, residual = (wide, other) if target == "x" else (other, wide)
    codes, scales, h = ops.rms_norm_quantize(x, None, 1e-6, ops.ACT_MX4, residual=residual, h=narrow)
    torch.cuda.synchronize()
    c, s = twin.mx4_rows(v, False)
    assert h is narrow and np.array_equal(h.float().cpu().numpy(), want)
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    kept[5, :k] = h[0]
    assert torch.equal(buf, kept)
