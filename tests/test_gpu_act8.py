"""Parity of the 8-bit checkpoints (bit for bit) and of the SwiGLU's backward pass with the oracle.

A gradient's tolerance: one bf16 rounding (2^-8 of the value, 2^-134 where bf16 is subnormal),
and of the fp32 arithmetic 2^-15.9 of the oracle's bound: the exponential is off by 2^-17.5
(ex2.approx and the rounded argument, |gate| <= 88), which enters sig and 1 - sig, each used
once; two divisions of 2 ulp and six roundings of 2^-24 add less than 2^-20. Below |gate| = 88
the exponential is a subnormal, off by 2^-149 absolutely.
"""
import numpy as np
import pytest
import torch

from oracle import act8 as A8
from oracle import gnf4_oracle as O
from synth import generators as G

from gpu_support import bf16_dev, bf16_host_bits

pytestmark = pytest.mark.gpu


def lib():
    import bit_grouped_moe_gnf4_b200 as g
    return g


def any_bits(shape, seed=0, finite=True):
    """bf16 patterns of every exponent: each block of 32 within a few binades of its own."""
    rng = np.random.default_rng(seed)
    x = rng.integers(0, 1 << 16, shape, dtype=np.uint16)
    top = rng.integers(0, 255, shape[:-1] + (shape[-1] // 32, 1))
    e = np.clip(top - rng.integers(0, 10, shape[:-1] + (shape[-1] // 32, 32)), 0, 254).reshape(shape)
    x = (x & 0x807F) | (e.astype(np.uint16) << 7)
    if not finite:
        flat = x.reshape(-1)
        flat[:: 97] = rng.choice(np.array([0x7F80, 0xFF80, 0x7FC0, 0xFFFF], np.uint16), flat[:: 97].size)
    return x


@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (17, 2048), (1000, 96), (2, 5, 160), (1, 32 * 32771)])
@pytest.mark.parametrize("finite", [True, False])
def test_checkpoint_bits(shape, finite):
    x = any_bits(shape, seed=shape[-1], finite=finite)
    codes, scales = lib().quantize_act8(bf16_dev(x))
    want_c, want_s = A8.quantize_act8(x)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    back = O.bf16_to_f64(bf16_host_bits(lib().dequantize_act8(codes, scales)))
    assert np.array_equal(back, A8.values_act8(want_c, want_s), equal_nan=True)


def test_checkpoint_of_more_rows_than_one_pass():
    # past the grid's single pass, against the same rows in pieces
    x = torch.randn(6001, 2048, device="cuda").to(torch.bfloat16)
    codes, scales = lib().quantize_act8(x)
    c2 = torch.cat([lib().quantize_act8(p)[0] for p in x.split(997)])
    assert torch.equal(codes, c2)
    back = lib().dequantize_act8(codes, scales)
    b2 = torch.cat([lib().dequantize_act8(c, s) for c, s in zip(codes.split(997), scales.split(997))])
    assert torch.equal(back, b2)
    want_c, want_s = A8.quantize_act8(bf16_host_bits(x[-5:]))
    assert np.array_equal(codes[-5:].cpu().numpy(), want_c) and np.array_equal(scales[-5:].cpu().numpy(), want_s)


def test_elements_past_32_bits():
    # more than 2^32 elements in one call; the last rows, the middle and the first against calls of their own
    g = lib()
    R, I = (1 << 21) + 37, 1024
    h = torch.empty(R, 2 * I, dtype=torch.bfloat16, device="cuda").normal_()
    parts = [slice(0, 40), slice(R // 2 - 20, R // 2 + 20), slice(R - 41, R)]
    codes, scales = g.quantize_act8(h)
    back = g.dequantize_act8(codes, scales)
    for p in parts:
        want = g.quantize_act8(h[p].clone())
        assert torch.equal(codes[p], want[0]) and torch.equal(scales[p], want[1])
        assert torch.equal(back[p], g.dequantize_act8(*want))
    del back
    out, c2, s2 = g.swiglu_act8(h)
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
    del c2, s2
    d = out * 0.5
    for p in parts:
        assert torch.equal(out[p], g.swiglu(h[p].clone()))
    dh = g.swiglu_backward(d, act8=(codes, scales), act=out)[0]
    for p in parts:
        want = g.swiglu_backward(d[p].clone(), act8=(codes[p].clone(), scales[p].clone()), rebuild=True)
        assert torch.equal(dh[p], want[0]) and torch.equal(out[p], want[1])
    g.swiglu_backward(d, gate_up=h, out=dh)
    for p in parts:
        assert torch.equal(dh[p], g.swiglu_backward(d[p].clone(), gate_up=h[p].clone()))


def test_nothing_is_written_behind_the_rows():
    g = lib()
    codes = torch.full((5 * 96 + 64,), 77, dtype=torch.int8, device="cuda")
    scales = torch.full((5 * 3 + 7,), 77, dtype=torch.uint8, device="cuda")
    out = torch.full((5 * 96 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    x = bf16_dev(any_bits((5, 96)))
    c, s = codes[:480].view(5, 96), scales[:15].view(5, 3)
    g.quantize_act8(x, codes=c, scales=s)
    g.dequantize_act8(c, s, out=out[:480].view(5, 96))
    assert (codes[480:] == 77).all() and (scales[15:] == 77).all() and (out[480:] == 7).all()


@pytest.mark.parametrize("R,I", [(1, 32), (5, 96), (999, 2880), (130, 1024)])
def test_swiglu_act8_is_swiglu_and_quantize(R, I):
    g = lib()
    h = bf16_dev(G.activations_bf16(R, R, 2 * I, tag="h"))
    out, codes, scales = g.swiglu_act8(h)
    assert torch.equal(out, g.swiglu(h))
    want = g.quantize_act8(h)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


def grads_ok(got_bits, d, h, what):
    want, bound = A8.swiglu_backward_f64(d, h), A8.swiglu_backward_bound(d, h)
    I = d.shape[-1]
    g, u = np.abs(h[..., :I]), np.abs(h[..., I:])
    under = 2.0 ** -149 * np.concatenate([np.abs(d) * u * (1 + g), np.abs(d) * g], axis=-1)
    tol = 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * (2.0 ** -15.9 * bound + under) + 2.0 ** -134
    err = np.abs(O.bf16_to_f64(got_bits) - want)
    assert np.all(err <= tol), f"{what}: {int((err > tol).sum())} elements off, worst {float((err / tol).max()):.2f} of the bound"


@pytest.mark.parametrize("R,I", [(1, 32), (1, 8), (7, 72), (64, 768), (999, 2880), (128, 1024)])
@pytest.mark.parametrize("wide", [False, True])
def test_swiglu_backward(R, I, wide):
    g = lib()
    rng = np.random.default_rng(I)
    h = rng.normal(size=(R, 2 * I)) * 3
    if wide:                                            # both exponential regimes, gradual underflow
        h[:, :I] = np.linspace(-110, 110, R * I).reshape(R, I)
    h = O.bf16_to_f64(O.bf16_bits(h))
    d = O.bf16_to_f64(O.bf16_bits(rng.normal(size=(R, I))))
    dh, act = g.swiglu_backward(bf16_dev(O.bf16_bits(d)), gate_up=bf16_dev(O.bf16_bits(h)), rebuild=True)
    grads_ok(bf16_host_bits(dh), d, h, "bf16 rows")
    assert torch.equal(act, g.swiglu(bf16_dev(O.bf16_bits(h))))
    alone = g.swiglu_backward(bf16_dev(O.bf16_bits(d)), gate_up=bf16_dev(O.bf16_bits(h)))
    assert torch.equal(alone, dh)
    if I % 32 == 0:
        codes, scales = A8.quantize_act8(O.bf16_bits(h))
        q = (torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
        dh8, act8 = g.swiglu_backward(bf16_dev(O.bf16_bits(d)), act8=q, rebuild=True)
        h8 = A8.values_act8(codes, scales)
        grads_ok(bf16_host_bits(dh8), d, h8, "checkpoint")
        assert torch.equal(act8, g.swiglu(bf16_dev(O.bf16_bits(h8))))


def test_empty_calls():
    g = lib()
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert g.quantize_act8(e)[1].shape == (0, 2)
    assert g.dequantize_act8(*g.quantize_act8(e)).shape == (0, 64)
    assert g.swiglu_act8(e)[0].shape == (0, 32)
    assert g.swiglu_backward(e, gate_up=torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")).shape == (0, 128)


def test_captured_pass_replays_on_new_values():
    g = lib()
    h = torch.randn(64, 256, device="cuda").to(torch.bfloat16)
    d = torch.randn(64, 128, device="cuda").to(torch.bfloat16)

    def step():
        act, codes, scales = g.swiglu_act8(h)
        return act, g.swiglu_backward(d, act8=(codes, scales), rebuild=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (1, 2):
        torch.manual_seed(seed)
        h.copy_(torch.randn(64, 256, device="cuda"))
        d.copy_(torch.randn(64, 128, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1][0], want[1][0]) and torch.equal(got[1][1], want[1][1])


def test_other_stream():
    g = lib()
    x = torch.randn(512, 2048, device="cuda").to(torch.bfloat16)
    want = g.dequantize_act8(*g.quantize_act8(x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        codes, scales = g.quantize_act8(x)
    out = torch.empty_like(x)
    g.dequantize_act8(codes, scales, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
