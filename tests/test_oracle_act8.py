"""Pins of the checkpoint and SwiGLU-backward oracle: the format's printed numbers, its
error bound, and the gradient against differences of the forward formula."""
import numpy as np
import pytest

from oracle import act8 as A8
from oracle import glue as GL
from oracle import gnf4_oracle as O


def bits(v):
    return O.bf16_bits(np.asarray(v, np.float64))


def test_printed_values():
    # amax 1.0: exponent 0, so s = 127 and a step is 2^-6
    x = np.zeros(32)
    x[:5] = [1.0, -0.5, 2.0 ** -6, 2.0 ** -7, 3 * 2.0 ** -7]
    c, s = A8.quantize_act8(bits(x))
    assert s.tolist() == [127]
    assert c[:5].tolist() == [64, -32, 1, 0, 2]         # half a step and one and a half: to the even code
    assert A8.values_act8(c, s)[:3].tolist() == [1.0, -0.5, 2.0 ** -6]


@pytest.mark.parametrize("v,s", [(0.0, 0), (2.0 ** -133, 0), (2.0 ** -126, 1), (1.9921875, 127), (3.3895e38, 254)])
def test_scale_is_the_exponent_field(v, s):
    x = np.zeros(32)
    x[7] = v
    c, sc = A8.quantize_act8(bits(x))
    assert sc[0] == s
    back = A8.values_act8(c, sc)
    assert np.all(np.abs(back - O.bf16_to_f64(bits(x))) <= 2.0 ** (s - 134.0))
    assert np.array_equal(O.round_to_bf16(back), back)


def test_error_is_half_a_step_over_every_bf16_block_maximum():
    rng = np.random.default_rng(0)
    x = rng.integers(0, 1 << 16, (4000, 32), dtype=np.uint16)
    x[(x & 0x7F80) == 0x7F80] &= 0xBFFF                 # finite values of any exponent
    c, s = A8.quantize_act8(x)
    v, back = O.bf16_to_f64(x), A8.values_act8(c, s)
    assert np.all(np.abs(v - back) <= 2.0 ** (s.astype(np.float64) - 134.0)[..., None].reshape(4000, 1))
    assert np.abs(c).max() == 127


@pytest.mark.parametrize("bad", [0x7F80, 0xFF80, 0x7FC1])
def test_non_finite_block_reads_back_as_nan(bad):
    x = bits(np.ones(64))
    x[40] = bad
    c, s = A8.quantize_act8(x)
    assert s.tolist() == [127, 255] and not c[32:].any()
    back = A8.values_act8(c, s)
    assert np.all(back[:32] == 1.0) and np.isnan(back[32:]).all()


def test_swiglu_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(1)
    h, d, step = rng.normal(size=(3, 16)) * 3, rng.normal(size=(3, 8)), 1e-5
    want = np.zeros_like(h)
    for j in range(16):
        for sgn in (1, -1):
            p = h.copy()
            p[:, j] += sgn * step
            act = GL.silu_f64(p[:, :8]) * p[:, 8:]
            want[:, j] += sgn * (d * act).sum(axis=1) / (2 * step)
    # the quotient of a smooth function of size 10 is off by step^2 and by 1e-15 / step
    np.testing.assert_allclose(A8.swiglu_backward_f64(d, h), want, atol=1e-8)
