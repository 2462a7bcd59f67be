"""Refusals of the adapter, checkpoint and SwiGLU-backward calls (no GPU, no launch): the C
ABI's status codes, then the binding's own checks of types and shapes."""
import ctypes

import pytest
import torch

import bit_grouped_moe_gnf4_b200 as g
from bit_grouped_moe_gnf4_b200 import _lib
from bit_grouped_moe_gnf4_b200._lib import lib

FAKE = 0x7f0000001000          # 16-byte aligned, never dereferenced: validation fails first
FAKE2 = FAKE + 4096
INVALID, SHAPE, MISALIGNED, OK = (_lib.GNF4_ERR_INVALID_ARG, _lib.GNF4_ERR_UNSUPPORTED_SHAPE,
                                  _lib.GNF4_ERR_MISALIGNED, _lib.GNF4_OK)


def apply(**kw):
    a = dict(base=FAKE, x=FAKE, dtype=0, A=FAKE, B=FAKE, off=FAKE, tok=None, wt=None, dst=None, scal=None, L=4, r=16,
             N=128, K=256, R=8, T_in=8, T_out=8, out=FAKE2, h=None, flags=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.gnf4_lora_apply(*a.values(), None)


def backward(**kw):
    a = dict(g=FAKE, x=FAKE, xc=None, xs=None, h=FAKE, A=FAKE, B=FAKE, off=FAKE, tok=None, wt=None, src=None, scal=None,
             L=4, r=16, N=128, K=256, R=8, T_in=8, T_g=8, dxb=FAKE, dx=FAKE2, gh=FAKE2, dA=FAKE, dB=FAKE, gdt=0, flags=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.gnf4_lora_backward(*a.values(), None)


COMMON = [
    (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(off=None), INVALID), (dict(x=None), INVALID),
    (dict(L=0), INVALID), (dict(r=0), INVALID), (dict(N=0), INVALID), (dict(K=-8), INVALID), (dict(R=-1), INVALID),
    (dict(T_in=7), INVALID), (dict(flags=_lib.GNF4_FORCE_DECODE), INVALID),
    (dict(r=12), SHAPE), (dict(r=136), SHAPE), (dict(K=252), SHAPE), (dict(N=132), SHAPE), (dict(L=2049), SHAPE),
    (dict(K=(1 << 24) + 8), SHAPE), (dict(R=1 << 31, T_in=1 << 31), SHAPE),
    (dict(x=FAKE + 8), MISALIGNED), (dict(A=FAKE + 2), MISALIGNED), (dict(B=FAKE + 8), MISALIGNED),
    (dict(off=FAKE + 4), MISALIGNED), (dict(tok=FAKE + 2), MISALIGNED), (dict(wt=FAKE + 1), MISALIGNED),
    (dict(scal=FAKE + 2), MISALIGNED), (dict(h=FAKE + 8), MISALIGNED),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(dtype=2), INVALID), (dict(out=None), INVALID), (dict(T_out=7), INVALID), (dict(base=FAKE + 8), MISALIGNED),
    (dict(out=FAKE + 4), MISALIGNED), (dict(out=FAKE), INVALID),         # x itself
    (dict(dst=FAKE + 2), MISALIGNED),
    (dict(), INVALID),                                   # not device memory
    (dict(R=0, x=None, base=None, out=None, A=None, B=None, off=None), OK),
])
def test_apply_refusals(kw, status):
    assert apply(**kw) == status
    assert status == OK or lib.gnf4_last_error()


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(gdt=1), INVALID), (dict(g=None), INVALID), (dict(h=None), INVALID), (dict(gh=None), INVALID),
    (dict(dA=None), INVALID), (dict(dB=None), INVALID),      # dA NULL: x must be as well
    (dict(dx=None), INVALID),                                # dx_base without dx
    (dict(gh=FAKE), INVALID), (dict(dx=FAKE, dxb=None), INVALID),        # h and grad_out themselves
    (dict(T_g=7), INVALID), (dict(xc=FAKE, xs=FAKE), INVALID), (dict(x=None, xc=FAKE), INVALID),
    (dict(x=None, xs=FAKE), INVALID), (dict(x=None, xc=FAKE, xs=FAKE, K=264), SHAPE),
    (dict(x=None, xc=FAKE + 8, xs=FAKE), MISALIGNED), (dict(g=FAKE + 2), MISALIGNED), (dict(dx=FAKE + 8), MISALIGNED),
    (dict(dA=FAKE + 2), MISALIGNED), (dict(dB=FAKE + 8), MISALIGNED), (dict(gh=FAKE + 8), MISALIGNED),
    (dict(src=FAKE + 2), MISALIGNED), (dict(), INVALID), (dict(R=0, off=None), INVALID),
])
def test_backward_refusals(kw, status):
    assert backward(**kw) == status
    assert status == OK or lib.gnf4_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(gh=None), INVALID), (dict(x=None), INVALID), (dict(x=None, xc=FAKE), INVALID), (dict(xc=FAKE), INVALID),
    (dict(off=None), INVALID), (dict(dA=None), INVALID), (dict(T_in=7), INVALID), (dict(L=0), INVALID),
    (dict(flags=2), INVALID), (dict(gdt=1), INVALID), (dict(r=12), SHAPE), (dict(K=252), SHAPE),
    (dict(x=None, xc=FAKE, xs=FAKE, K=264), SHAPE), (dict(gh=FAKE + 8), MISALIGNED), (dict(x=FAKE + 8), MISALIGNED),
    (dict(dA=FAKE + 8), MISALIGNED), (dict(off=FAKE + 4), MISALIGNED), (dict(tok=FAKE + 2), MISALIGNED),
    (dict(), INVALID),
])
def test_grad_a_refusals(kw, status):
    a = dict(gh=FAKE, x=FAKE, xc=None, xs=None, off=FAKE, tok=None, L=4, r=16, K=256, R=8, T_in=8, dA=FAKE, gdt=0, flags=0)
    assert set(kw) <= set(a)
    a.update(kw)
    assert lib.gnf4_lora_grad_a(*a.values(), None) == status
    assert lib.gnf4_last_error()


def test_rows_of_an_empty_tensor_are_refused():
    # every row's index is then out of range, and an address to read in its place is missing
    assert apply(T_in=0, tok=FAKE) == INVALID and b"must have a row" in lib.gnf4_last_error()
    assert backward(T_g=0, src=FAKE) == INVALID and b"must have a row" in lib.gnf4_last_error()
    assert apply(T_in=0, tok=FAKE, R=0) == OK


def test_act8_refusals():
    q, d = lib.gnf4_quantize_act8, lib.gnf4_dequantize_act8
    for f in (lambda a, r, K, b, c: q(a, r, K, b, c, None), lambda a, r, K, b, c: d(b, c, r, K, a, None)):
        assert f(None, 4, 64, FAKE, FAKE) == INVALID
        assert f(FAKE, 4, 64, None, FAKE) == INVALID
        assert f(FAKE, 4, 64, FAKE, None) == INVALID
        assert f(FAKE, -1, 64, FAKE, FAKE) == INVALID
        assert f(FAKE, 4, 0, FAKE, FAKE) == INVALID
        assert f(FAKE, 4, 48, FAKE, FAKE) == SHAPE
        assert f(FAKE, 1 << 60, 1 << 10, FAKE, FAKE) == SHAPE
        assert f(FAKE + 8, 4, 64, FAKE, FAKE) == MISALIGNED
        assert f(FAKE, 4, 64, FAKE + 8, FAKE) == MISALIGNED
        assert f(FAKE, 4, 64, FAKE, FAKE + 1) == INVALID         # any alignment, but not device memory
        assert f(None, 0, 64, None, None) == OK
    buf = (ctypes.c_uint16 * 1024)()
    addr = (ctypes.addressof(buf) + 15) & ~15
    assert q(addr, 1, 32, addr + 64, addr + 128, None) == INVALID
    assert b"device memory" in lib.gnf4_last_error()


def test_stall_is_refused_where_no_kernel_waits():
    stall = _lib.GNF4_TEST_STALL
    assert apply(r=72, flags=stall) == INVALID and b"nothing waits" in lib.gnf4_last_error()
    assert lib.gnf4_lora_grad_a(FAKE, FAKE, None, None, FAKE, None, 4, 32, 256, 8, 8, FAKE, 0, stall, None) == INVALID
    assert b"nothing waits" in lib.gnf4_last_error()
    for call in (lambda: apply(flags=stall), lambda: backward(flags=stall),        # let in, but no device memory
                 lambda: lib.gnf4_lora_grad_a(FAKE, FAKE, None, None, FAKE, None, 4, 40, 256, 8, 8, FAKE, 0, stall, None)):
        assert call() == INVALID and b"device memory" in lib.gnf4_last_error()


def test_sizes_past_one_pass_of_a_grid_are_refused():
    # 2^41 elements are let in (and then refused as no device memory); there is no second pass beyond
    most = 1 << 41
    for rows, K in ((1, most), (1 << 20, 1 << 21), (1 << 36, 32)):
        assert lib.gnf4_quantize_act8(FAKE, rows, K, FAKE, FAKE, None) == INVALID
        assert lib.gnf4_quantize_act8(FAKE, rows + 1, K, FAKE, FAKE, None) == SHAPE
        assert lib.gnf4_dequantize_act8(FAKE, FAKE, rows + 1, K, FAKE, None) == SHAPE
        assert b"2^41" in lib.gnf4_last_error()
    for R, I in ((1 << 20, 1 << 21), (1 << 36, 32), (1 << 11, 1 << 30)):
        assert lib.gnf4_swiglu_act8(FAKE, R, I, FAKE, FAKE, FAKE, None) == INVALID
        assert lib.gnf4_swiglu_act8(FAKE, R + 1, I, FAKE, FAKE, FAKE, None) == SHAPE
        assert lib.gnf4_swiglu_backward(FAKE, FAKE, None, None, R + 1, I, FAKE, None, None) == SHAPE
    assert lib.gnf4_swiglu_backward(FAKE, FAKE, None, None, 1 << 39, 8, FAKE, None, None) == SHAPE


def test_swiglu_refusals():
    f = lib.gnf4_swiglu_act8
    assert f(FAKE, 4, 40, FAKE, FAKE, FAKE, None) == SHAPE
    assert f(FAKE, 4, 64, None, FAKE, FAKE, None) == INVALID
    assert f(FAKE, 4, 64, FAKE + 8, FAKE, FAKE, None) == MISALIGNED
    assert f(None, 0, 64, None, None, None, None) == OK
    b = lib.gnf4_swiglu_backward
    assert b(FAKE, FAKE, None, None, 4, 60, FAKE, None, None) == SHAPE
    assert b(FAKE, None, FAKE, FAKE, 4, 40, FAKE, None, None) == SHAPE       # a checkpoint wants I % 32
    assert b(FAKE, FAKE, FAKE, FAKE, 4, 64, FAKE, None, None) == INVALID     # both
    assert b(FAKE, None, FAKE, None, 4, 64, FAKE, None, None) == INVALID
    assert b(FAKE, None, None, None, 4, 64, FAKE, None, None) == INVALID     # neither
    assert b(None, FAKE, None, None, 4, 64, FAKE, None, None) == INVALID
    assert b(FAKE, FAKE, None, None, 4, 64, None, None, None) == INVALID
    assert b(FAKE, FAKE, None, None, -4, 64, FAKE, None, None) == INVALID
    assert b(FAKE, FAKE, None, None, 4, 64, FAKE, FAKE + 8, None) == MISALIGNED
    assert b(FAKE, FAKE + 2, None, None, 4, 64, FAKE, None, None) == MISALIGNED
    assert b(None, None, None, None, 0, 64, None, None, None) == OK


# ---- the binding (CPU tensors: refused before the library is reached, or by it)
def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def parts(**kw):
    p = dict(base=t(8, 128), x=t(8, 256), A=t(4, 16, 256), B=t(4, 128, 16), adapter_offsets=t(5, dtype=torch.int64))
    p.update(kw)
    return p


@pytest.mark.parametrize("kw,err", [
    (dict(x=t(8, 256, dtype=torch.float32)), TypeError), (dict(A=t(4, 16, 256, dtype=torch.float16)), TypeError),
    (dict(x=t(8, 264)), ValueError), (dict(B=t(4, 128, 8)), ValueError), (dict(B=t(3, 128, 16)), ValueError),
    (dict(base=t(8, 120)), ValueError), (dict(base=None), ValueError), (dict(out=t(9, 128)), ValueError),
    (dict(adapter_offsets=t(4, dtype=torch.int64)), ValueError), (dict(adapter_offsets=t(5, dtype=torch.int32)), TypeError),
    (dict(scaling=t(3, dtype=torch.float32)), ValueError), (dict(row_token=t(8, dtype=torch.int64)), TypeError),
    (dict(row_token=t(8, dtype=torch.int32), row_dest=t(7, dtype=torch.int32)), ValueError),
    (dict(h=t(8, 8, dtype=torch.float32)), ValueError), (dict(A=t(4, 256, 16).mT), ValueError),
])
def test_binding_apply(kw, err):
    with pytest.raises(err):
        g.lora_apply(**parts(**kw))


@pytest.mark.parametrize("kw,err", [
    (dict(x=None), ValueError),                              # no dA then, and grad_h is missing
    (dict(x=None, grad_h=t(8, 16, dtype=torch.float32), dA=t(4, 16, 256)), ValueError),
    (dict(act8=(t(8, 256, dtype=torch.int8), t(8, 8, dtype=torch.uint8))), ValueError),
    (dict(x=None, act8=(t(8, 256, dtype=torch.int8), t(8, 4, dtype=torch.uint8))), ValueError),
    (dict(grad_dtype=torch.float16), TypeError), (dict(h=t(7, 16, dtype=torch.float32), R=8), ValueError),
    (dict(dx_base=t(8, 128)), ValueError), (dict(dA=t(4, 16, 256, dtype=torch.float32)), TypeError),
    (dict(stream=0), ValueError), (dict(grad_out=t(8, 120)), ValueError),
    (dict(grad_out=t(8, 128, dtype=torch.float16)), TypeError),
])
def test_binding_backward(kw, err):
    p = parts(h=t(8, 16, dtype=torch.float32))
    p["grad_out"] = p.pop("base")
    p.update(kw)
    with pytest.raises(err):
        g.lora_backward(**p)


def test_binding_grad_a():
    gh, off, x = t(8, 16, dtype=torch.float32), t(5, dtype=torch.int64), t(8, 256)
    for kw, err in ((dict(), ValueError), (dict(x=x, act8=(t(8, 256, dtype=torch.int8), t(8, 8, dtype=torch.uint8))), ValueError),
                    (dict(x=x.float()), TypeError), (dict(x=x, row_token=t(7, dtype=torch.int32)), ValueError),
                    (dict(x=x, dA=t(4, 8, 256)), ValueError), (dict(x=x, grad_dtype=torch.float16), TypeError)):
        with pytest.raises(err):
            g.lora_grad_a(gh, off, **kw)


def test_binding_act8():
    with pytest.raises(TypeError):
        g.quantize_act8(t(4, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        g.quantize_act8(t(64, 4).mT)
    with pytest.raises(ValueError):
        g.quantize_act8(t(4, 64), codes=t(4, 32, dtype=torch.int8))
    with pytest.raises(ValueError):
        g.dequantize_act8(t(4, 64, dtype=torch.int8), t(4, 1, dtype=torch.uint8))
    with pytest.raises(ValueError):
        g.swiglu_backward(t(4, 64))
    with pytest.raises(ValueError):
        g.swiglu_backward(t(4, 64), gate_up=t(4, 64))
    with pytest.raises(ValueError):
        g.swiglu_backward(t(4, 64), act8=(t(3, 128, dtype=torch.int8), t(3, 4, dtype=torch.uint8)))
