"""The plain implementations that the GPU tests of the quantised-row producers
and the MXFP4 product compare with, pinned to closed forms and to the oracle."""
import numpy as np
import pytest

import oracle
import rows_twin as twin


def test_int4_rows_equal_the_oracle():
    v = np.random.default_rng(1).standard_normal((5, 160)).astype(np.float32)
    v[:, 7] *= 20
    v[3, 32:64] = 0
    codes, scales = oracle.rotate_quantize_act(v)
    q, s = twin.int_rows(v, 7)
    assert np.array_equal(twin.int4_bytes(q), codes) and np.array_equal(s, scales)
    q8, s8 = oracle.rotate_quantize_act8(v)
    q, s = twin.int_rows(v, 127)
    assert np.array_equal(q, q8) and np.array_equal(s, s8)


@pytest.mark.parametrize("value,code", [(0.0, 0), (0.25, 0), (0.2500001, 1), (0.7499999, 1), (0.75, 2), (1.25, 2), (1.75, 4),
                                        (2.5, 4), (2.5000002, 5), (3.5, 6), (5.0, 6), (5.0000005, 7), (6.0, 7), (7.9999995, 7)])
def test_mx4_rounds_to_nearest_even_and_saturates(value, code):
    v = np.zeros((1, 32), np.float32)
    v[0, 0] = 4.0  # scale 2^0
    v[0, 5], v[0, 6] = value, -value
    codes, scales = twin.mx4_rows(v, False)
    assert scales.tolist() == [[127] * 8]
    assert codes[0, 2] >> 4 == code and codes[0, 3] & 15 == code | 8


@pytest.mark.parametrize("top,byte", [(0.0, 0), (1e-45, 0), (2.0 ** -125, 0), (2.0 ** -124, 1), (1.0, 125), (3.9999998, 126),
                                      (4.0, 127), (3.4028235e38, 252), (np.inf, 255), (np.nan, 255)])
def test_mx4_scale_byte(top, byte):
    v = np.zeros((1, 64), np.float32)
    v[0, 33] = top
    _, scales = twin.mx4_rows(v, False)
    assert scales[0, :2].tolist() == [0, byte] and (scales[0, 2:] == 127).all()


def test_read_back_inverts_the_codes():
    v = np.random.default_rng(2).standard_normal((3, 96)).astype(np.float32)
    q, s = twin.int_rows(v, 7)
    assert np.array_equal(twin.read_back("int4", twin.int4_bytes(q), s, 96), q.astype(np.float32) * np.repeat(s, 32, 1))
    c, b = twin.mx4_rows(v, False)
    x = twin.read_back("mx4", c, b, 96)
    step = 2.0 ** (b[:, :3].astype(int) - 127.0)  # half the widest gap of the grid, and the saturated end
    assert (np.abs(x - v).reshape(3, 3, 32) <= 2 * step[..., None]).all()


def test_norm_and_gate_closed_forms():
    h, v = twin.norm(np.full((1, 64), 3.0, np.float32), np.full((1, 64), 1.0, np.float32), twin.TORCH["bf16"], None, 1e-9)
    assert (h == 4.0).all() and np.allclose(v, 1.0, rtol=1e-6)
    g = np.array([-40.0, -1.0, 0.0, 1.0, 40.0])
    assert np.allclose(twin.silu(g), [-40 * np.exp(-40.0), -0.2689414213699951, 0, 0.7310585786300049, 40], rtol=1e-14)
    assert np.allclose(twin.gelu_tanh(np.array([1.0])), 0.841191990608306, rtol=1e-12)
