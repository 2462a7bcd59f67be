"""Thin torch-facing wrappers over the C ABI (argument marshalling only).

Every step of the computation runs in the CUDA kernels of libgnf4.so; these
functions only pass device pointers, sizes and the current stream.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from ._lib import lib, check


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    """A torch.cuda.Stream, a raw cudaStream_t handle as an int (0 = the legacy default
    stream), or None for torch's current stream."""
    if stream is None:
        # the handle itself: torch.cuda.current_stream() first makes a Stream object (3 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _need(t: torch.Tensor, dtype: torch.dtype, name: str) -> None:
    if type(t) is torch.Tensor and t.dtype is dtype and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def quantize_nf4(w: torch.Tensor, packed: Optional[torch.Tensor] = None,
                 absmax: Optional[torch.Tensor] = None, stream=None):
    """fp32 ``[..., K]`` device tensor -> (packed uint8 ``[..., K//2]``, absmax fp32 ``[..., K//64]``)."""
    _need(w, torch.float32, "w")
    K = w.shape[-1]
    rows = w.numel() // K if K else 0
    lead = tuple(w.shape[:-1])
    if packed is None:
        packed = torch.empty(lead + (K // 2,), dtype=torch.uint8, device=w.device)
    if absmax is None:
        absmax = torch.empty(lead + (K // 64,), dtype=torch.float32, device=w.device)
    check(lib.gnf4_quantize_nf4(_ptr(w), rows, K, _ptr(packed), _ptr(absmax), _stream(stream)),
          "gnf4_quantize_nf4")
    return packed, absmax


def quantize_mxfp4(w: torch.Tensor, blocks: Optional[torch.Tensor] = None,
                   scales: Optional[torch.Tensor] = None, stream=None):
    """fp32 ``[..., K]`` device tensor -> (blocks uint8 ``[..., K//2]``, scales uint8 ``[..., K//32]``)."""
    _need(w, torch.float32, "w")
    K = w.shape[-1]
    rows = w.numel() // K if K else 0
    lead = tuple(w.shape[:-1])
    if blocks is None:
        blocks = torch.empty(lead + (K // 2,), dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty(lead + (K // 32,), dtype=torch.uint8, device=w.device)
    check(lib.gnf4_quantize_mxfp4(_ptr(w), rows, K, _ptr(blocks), _ptr(scales), _stream(stream)),
          "gnf4_quantize_mxfp4")
    return blocks, scales


def grouped_gemm(fmt: str, x: torch.Tensor, W: torch.Tensor, scales: torch.Tensor,
                 expert_offsets: torch.Tensor, row_token: Optional[torch.Tensor] = None,
                 row_weight: Optional[torch.Tensor] = None, row_dest: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, T_out: Optional[int] = None, flags: int = 0,
                 R: Optional[int] = None, stream=None) -> torch.Tensor:
    """One grouped GEMM call (see include/gnf4.h). ``R`` (the routed row count) is
    taken from ``row_token``/``row_weight``/``row_dest`` when one is given, else it
    must be passed (it is never read back from the device). ``x`` is bf16 or fp16 (the
    output has its type); NF4 ``scales`` (absmax) are fp32 or bf16 (the bf16-absmax
    storage, see ``absmax_to_bf16``)."""
    if fmt not in ("nf4", "mxfp4"):
        raise ValueError("fmt must be 'nf4' or 'mxfp4'")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"x must be torch.bfloat16 or torch.float16, got {x.dtype}")
    _need(x, x.dtype, "x")
    _need(W, torch.uint8, "W")
    if fmt == "nf4":
        if scales.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"NF4 absmax must be torch.float32 or torch.bfloat16, got {scales.dtype}")
        _need(scales, scales.dtype, "scales")
    else:
        _need(scales, torch.uint8, "scales")
    _need(expert_offsets, torch.int64, "expert_offsets")
    for name, t, dt in (("row_token", row_token, torch.int32), ("row_weight", row_weight, torch.float32),
                        ("row_dest", row_dest, torch.int32)):
        if t is not None:
            _need(t, dt, name)
    E, N, K2 = W.shape
    K = x.shape[1]
    if K2 * 2 != K:
        raise ValueError(f"W is [E, N, K/2] = {tuple(W.shape)} but x has K = {K}")
    if R is None:
        for t in (row_token, row_weight, row_dest):
            if t is not None:
                R = t.numel()
                break
    if R is None:
        raise ValueError("pass R (routed rows) when row_token, row_weight and row_dest are all None")
    if out is None:
        T_out = R if T_out is None else T_out
        out = torch.empty((T_out, N), dtype=x.dtype, device=x.device)
    else:
        _need(out, x.dtype, "out")
        T_out = out.shape[0]
    xdt = _lib.GNF4_DTYPE_F16 if x.dtype == torch.float16 else _lib.GNF4_DTYPE_BF16
    if fmt == "nf4":
        sdt = _lib.GNF4_DTYPE_BF16 if scales.dtype == torch.bfloat16 else _lib.GNF4_DTYPE_F32
        st = lib.gnf4_grouped_gemm_nf4_ex(_ptr(x), xdt, _ptr(W), _ptr(scales), sdt, _ptr(expert_offsets),
                                          _ptr(row_token), _ptr(row_weight), _ptr(row_dest), E, N, K, R,
                                          x.shape[0], T_out, _ptr(out), flags, _stream(stream))
    else:
        st = lib.gnf4_grouped_gemm_mxfp4_ex(_ptr(x), xdt, _ptr(W), _ptr(scales), _ptr(expert_offsets),
                                            _ptr(row_token), _ptr(row_weight), _ptr(row_dest), E, N, K, R,
                                            x.shape[0], T_out, _ptr(out), flags, _stream(stream))
    check(st, f"gnf4_grouped_gemm_{fmt}_ex")
    return out


def grouped_gemm_swiglu(fmt: str, x: torch.Tensor, W: torch.Tensor, scales: torch.Tensor,
                        expert_offsets: torch.Tensor, row_token: Optional[torch.Tensor] = None,
                        row_weight: Optional[torch.Tensor] = None, row_dest: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, T_out: Optional[int] = None, flags: int = 0,
                        R: Optional[int] = None, stream=None) -> torch.Tensor:
    """gate_up grouped GEMM with the SwiGLU fused into its epilogue (include/gnf4.h,
    gnf4_grouped_gemm_swiglu_*): ``W`` is the fused gate_up stack ``[E, 2I, K/2]``, the
    result ``[T_out, I]`` holds silu(gate) * up in the activations' type."""
    if fmt not in ("nf4", "mxfp4"):
        raise ValueError("fmt must be 'nf4' or 'mxfp4'")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"x must be torch.bfloat16 or torch.float16, got {x.dtype}")
    _need(x, x.dtype, "x")
    _need(W, torch.uint8, "W")
    if fmt == "nf4":
        if scales.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"NF4 absmax must be torch.float32 or torch.bfloat16, got {scales.dtype}")
        _need(scales, scales.dtype, "scales")
    else:
        _need(scales, torch.uint8, "scales")
    _need(expert_offsets, torch.int64, "expert_offsets")
    for name, t, dt in (("row_token", row_token, torch.int32), ("row_weight", row_weight, torch.float32),
                        ("row_dest", row_dest, torch.int32)):
        if t is not None:
            _need(t, dt, name)
    E, N, K2 = W.shape
    K = x.shape[1]
    if K2 * 2 != K:
        raise ValueError(f"W is [E, N, K/2] = {tuple(W.shape)} but x has K = {K}")
    if R is None:
        for t in (row_token, row_weight, row_dest):
            if t is not None:
                R = t.numel()
                break
    if R is None:
        raise ValueError("pass R (routed rows) when row_token, row_weight and row_dest are all None")
    if out is None:
        T_out = R if T_out is None else T_out
        out = torch.empty((T_out, N // 2), dtype=x.dtype, device=x.device)
    else:
        _need(out, x.dtype, "out")
        T_out = out.shape[0]
    xdt = _lib.GNF4_DTYPE_F16 if x.dtype == torch.float16 else _lib.GNF4_DTYPE_BF16
    if fmt == "nf4":
        sdt = _lib.GNF4_DTYPE_BF16 if scales.dtype == torch.bfloat16 else _lib.GNF4_DTYPE_F32
        st = lib.gnf4_grouped_gemm_swiglu_nf4(_ptr(x), xdt, _ptr(W), _ptr(scales), sdt, _ptr(expert_offsets),
                                              _ptr(row_token), _ptr(row_weight), _ptr(row_dest), E, N, K, R,
                                              x.shape[0], T_out, _ptr(out), flags, _stream(stream))
    else:
        st = lib.gnf4_grouped_gemm_swiglu_mxfp4(_ptr(x), xdt, _ptr(W), _ptr(scales), _ptr(expert_offsets),
                                                _ptr(row_token), _ptr(row_weight), _ptr(row_dest), E, N, K, R,
                                                x.shape[0], T_out, _ptr(out), flags, _stream(stream))
    check(st, f"gnf4_grouped_gemm_swiglu_{fmt}")
    return out


def absmax_to_bf16(absmax: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The lossless fp32 -> bf16 NF4 absmax cast (include/gnf4.h, gnf4_absmax_to_bf16):
    raises Gnf4Error if any value has no bf16 equal (an fp32 source)."""
    _need(absmax, torch.float32, "absmax")
    if out is None:
        out = torch.empty(absmax.shape, dtype=torch.bfloat16, device=absmax.device)
    else:
        _need(out, torch.bfloat16, "out")
    check(lib.gnf4_absmax_to_bf16(_ptr(absmax), absmax.numel(), _ptr(out), _stream(stream)),
          "gnf4_absmax_to_bf16")
    return out


def grouped_gemm_nf4(x, W, absmax, expert_offsets, **kw):
    return grouped_gemm("nf4", x, W, absmax, expert_offsets, **kw)


def grouped_gemm_mxfp4(x, W, scales, expert_offsets, **kw):
    return grouped_gemm("mxfp4", x, W, scales, expert_offsets, **kw)


def dgrad(fmt: str, grad_out: torch.Tensor, W: torch.Tensor, scales: torch.Tensor,
          expert_offsets: torch.Tensor, row_src: Optional[torch.Tensor] = None,
          row_weight: Optional[torch.Tensor] = None, R: Optional[int] = None,
          out: Optional[torch.Tensor] = None, flags: int = 0, stream=None) -> torch.Tensor:
    """Input gradient of a grouped GEMM call (include/gnf4.h): bf16 ``[R, K]`` with
    ``out[r] = w(r) * grad_out[src(r)] @ dequant(W[e(r)])``. ``R`` is taken from
    ``row_src`` / ``row_weight`` when given, else from ``grad_out`` (rows in routed order)."""
    if fmt not in ("nf4", "mxfp4"):
        raise ValueError("fmt must be 'nf4' or 'mxfp4'")
    _need(grad_out, torch.bfloat16, "grad_out")
    _need(W, torch.uint8, "W")
    _need(scales, torch.float32 if fmt == "nf4" else torch.uint8, "scales")
    _need(expert_offsets, torch.int64, "expert_offsets")
    for name, t, dt in (("row_src", row_src, torch.int32), ("row_weight", row_weight, torch.float32)):
        if t is not None:
            _need(t, dt, name)
    E, N, K2 = W.shape
    if grad_out.dim() != 2 or grad_out.shape[1] != N:
        raise ValueError(f"grad_out must be [T_in, N = {N}], got {tuple(grad_out.shape)}")
    if R is None:
        for t in (row_src, row_weight):
            if t is not None:
                R = t.numel()
                break
    if R is None:
        R = grad_out.shape[0]
    K = 2 * K2
    if out is None:
        out = torch.empty((R, K), dtype=torch.bfloat16, device=grad_out.device)
    else:
        _need(out, torch.bfloat16, "out")
        if tuple(out.shape) != (R, K):
            raise ValueError(f"out must be [{R}, {K}], got {tuple(out.shape)}")
    fn = lib.gnf4_dgrad_nf4 if fmt == "nf4" else lib.gnf4_dgrad_mxfp4
    check(fn(_ptr(grad_out), _ptr(W), _ptr(scales), _ptr(expert_offsets), _ptr(row_src), _ptr(row_weight),
             E, N, K, R, grad_out.shape[0], _ptr(out), flags, _stream(stream)), f"gnf4_dgrad_{fmt}")
    return out


def routing_metadata(topk_ids: torch.Tensor, topk_weights: Optional[torch.Tensor], E: int,
                     stream=None):
    """Router top-k ``[T, k]`` (int32 ids, fp32 weights or None) -> (expert_offsets int64 [E+1],
    row_token int32 [T*k], row_weight fp32 [T*k] or None, row_dest int32 [T*k]) on the device,
    rows sorted by (expert, token, slot) (include/gnf4.h)."""
    _need(topk_ids, torch.int32, "topk_ids")
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids must be [T, k]")
    T, k = topk_ids.shape
    if topk_weights is not None:
        _need(topk_weights, torch.float32, "topk_weights")
        if tuple(topk_weights.shape) != (T, k):
            raise ValueError("topk_weights must match topk_ids")
    dev = topk_ids.device
    offsets = torch.empty(E + 1, dtype=torch.int64, device=dev)
    row_token = torch.empty(T * k, dtype=torch.int32, device=dev)
    row_weight = None if topk_weights is None else torch.empty(T * k, dtype=torch.float32, device=dev)
    row_dest = torch.empty(T * k, dtype=torch.int32, device=dev)
    check(lib.gnf4_routing_metadata(_ptr(topk_ids), _ptr(topk_weights), T, k, E, _ptr(offsets), _ptr(row_token),
                                    _ptr(row_weight), _ptr(row_dest), _stream(stream)), "gnf4_routing_metadata")
    return offsets, row_token, row_weight, row_dest


def swiglu(gate_up: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """bf16 ``[R, 2I]`` gate_up rows -> bf16 ``[R, I]``: ``silu(gate) * up`` (include/gnf4.h)."""
    _need(gate_up, torch.bfloat16, "gate_up")
    if gate_up.dim() != 2 or gate_up.shape[1] % 2:
        raise ValueError(f"gate_up must be [R, 2I], got {tuple(gate_up.shape)}")
    R, I = gate_up.shape[0], gate_up.shape[1] // 2
    if out is None:
        out = torch.empty((R, I), dtype=torch.bfloat16, device=gate_up.device)
    else:
        _need(out, torch.bfloat16, "out")
        if tuple(out.shape) != (R, I):
            raise ValueError(f"out must be [{R}, {I}], got {tuple(out.shape)}")
    check(lib.gnf4_swiglu(_ptr(gate_up), R, I, _ptr(out), _stream(stream)), "gnf4_swiglu")
    return out


def combine_topk(y: torch.Tensor, T: int, k: int, row_of_slot: Optional[torch.Tensor] = None,
                 slot_weight: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """bf16 ``[R, N]`` down rows -> bf16 ``[T, N]``: the fp32 slot-order sum over each
    token's k slots (include/gnf4.h)."""
    _need(y, torch.bfloat16, "y")
    if y.dim() != 2:
        raise ValueError("y must be [R, N]")
    for name, t, dt in (("row_of_slot", row_of_slot, torch.int32), ("slot_weight", slot_weight, torch.float32)):
        if t is not None:
            _need(t, dt, name)
            if t.numel() != T * k:
                raise ValueError(f"{name} must hold T*k = {T * k} entries, got {t.numel()}")
    R, N = y.shape
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=y.device)
    else:
        _need(out, torch.bfloat16, "out")
        if tuple(out.shape) != (T, N):
            raise ValueError(f"out must be [{T}, {N}], got {tuple(out.shape)}")
    check(lib.gnf4_combine_topk(_ptr(y), R, N, _ptr(row_of_slot), _ptr(slot_weight), T, k, _ptr(out),
                                _stream(stream)), "gnf4_combine_topk")
    return out


def _shaped(t: Optional[torch.Tensor], shape, dtype: torch.dtype, name: str, like: torch.Tensor) -> torch.Tensor:
    """``t`` checked against a type and shape, or a new tensor beside ``like`` if it is None."""
    if t is None:
        # beside one of its own shape a tensor is made faster
        return torch.empty_like(like, dtype=dtype) if like.shape == shape else like.new_empty(shape, dtype=dtype)
    _need(t, dtype, name)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


def _act8(act8, K: int, name: str):
    """A checkpoint (codes int8 ``[rows, K]``, scales uint8 ``[rows, K/32]``), checked."""
    codes, scales = act8
    _need(codes, torch.int8, f"{name} codes")
    _need(scales, torch.uint8, f"{name} scales")
    if codes.dim() != 2 or codes.shape[1] != K or scales.shape != (codes.shape[0], K // 32):
        raise ValueError(f"{name} must be codes [rows, {K}] and scales [rows, {K // 32}], got "
                         f"{list(codes.shape)} and {list(scales.shape)}")
    return codes, scales


def quantize_act8(x: torch.Tensor, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                  stream=None):
    """8-bit checkpoint of bf16 ``[..., K]`` rows: (codes int8 ``[..., K]``, scales uint8
    ``[..., K//32]``), one e8m0 scale per 32 elements (include/gnf4.h)."""
    _need(x, torch.bfloat16, "x")
    K = x.shape[-1]
    codes = _shaped(codes, x.shape, torch.int8, "codes", x)
    scales = _shaped(scales, (*x.shape[:-1], K // 32), torch.uint8, "scales", x)
    check(lib.gnf4_quantize_act8(_ptr(x), x.numel() // K if K else 0, K, _ptr(codes), _ptr(scales), _stream(stream)),
          "gnf4_quantize_act8")
    return codes, scales


def dequantize_act8(codes: torch.Tensor, scales: torch.Tensor, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """The bf16 values an 8-bit checkpoint stands for (include/gnf4.h)."""
    _need(codes, torch.int8, "codes")
    K = codes.shape[-1]
    _need(scales, torch.uint8, "scales")
    if scales.shape != (*codes.shape[:-1], K // 32):
        raise ValueError(f"scales must be [..., {K // 32}] beside codes {list(codes.shape)}, got {list(scales.shape)}")
    out = _shaped(out, codes.shape, torch.bfloat16, "out", codes)
    check(lib.gnf4_dequantize_act8(_ptr(codes), _ptr(scales), codes.numel() // K if K else 0, K, _ptr(out),
                                   _stream(stream)), "gnf4_dequantize_act8")
    return out


def swiglu_act8(gate_up: torch.Tensor, out: Optional[torch.Tensor] = None, codes: Optional[torch.Tensor] = None,
                scales: Optional[torch.Tensor] = None, stream=None):
    """``swiglu`` and the 8-bit checkpoint of its ``[R, 2I]`` input in one pass: (out ``[R, I]``,
    codes ``[R, 2I]``, scales ``[R, 2I/32]``) (include/gnf4.h)."""
    _need(gate_up, torch.bfloat16, "gate_up")
    if gate_up.dim() != 2 or gate_up.shape[1] % 2:
        raise ValueError(f"gate_up must be [R, 2I], got {tuple(gate_up.shape)}")
    R, I = gate_up.shape[0], gate_up.shape[1] // 2
    out = _shaped(out, (R, I), torch.bfloat16, "out", gate_up)
    codes = _shaped(codes, (R, 2 * I), torch.int8, "codes", gate_up)
    scales = _shaped(scales, (R, 2 * I // 32), torch.uint8, "scales", gate_up)
    check(lib.gnf4_swiglu_act8(_ptr(gate_up), R, I, _ptr(out), _ptr(codes), _ptr(scales), _stream(stream)),
          "gnf4_swiglu_act8")
    return out, codes, scales


def swiglu_backward(grad_out: torch.Tensor, gate_up: Optional[torch.Tensor] = None, act8=None,
                    out: Optional[torch.Tensor] = None, rebuild: bool = False, act: Optional[torch.Tensor] = None,
                    stream=None):
    """Gradient of ``swiglu``'s input, bf16 ``[R, 2I]``, from ``grad_out`` ``[R, I]`` and either the
    ``gate_up`` rows or their checkpoint ``act8 = (codes, scales)``. With ``rebuild`` (or ``act``
    given) returns (gradient, the activations ``[R, I]`` once more), else the gradient alone
    (include/gnf4.h)."""
    _need(grad_out, torch.bfloat16, "grad_out")
    if grad_out.dim() != 2:
        raise ValueError("grad_out must be [R, I]")
    R, I = grad_out.shape
    if (gate_up is None) == (act8 is None):
        raise ValueError("give either gate_up or act8")
    codes = scales = None
    if gate_up is not None:
        gate_up = _shaped(gate_up, (R, 2 * I), torch.bfloat16, "gate_up", grad_out)
    else:
        codes, scales = _act8(act8, 2 * I, "act8")
        if codes.shape[0] != R:
            raise ValueError(f"act8 must hold {R} rows, got {codes.shape[0]}")
    out = _shaped(out, (R, 2 * I), torch.bfloat16, "out", grad_out)
    if rebuild or act is not None:
        act = _shaped(act, (R, I), torch.bfloat16, "act", grad_out)
    check(lib.gnf4_swiglu_backward(_ptr(grad_out), _ptr(gate_up), _ptr(codes), _ptr(scales), R, I, _ptr(out),
                                   _ptr(act), _stream(stream)), "gnf4_swiglu_backward")
    return out if act is None else (out, act)


def _lora_common(A, B, adapter_offsets, row_token, row_weight, name, rows, scaling, R, dtype):
    _need(A, dtype, "A")
    _need(B, dtype, "B")
    try:
        (L, r, K), (L2, N, r2) = A.shape, B.shape
    except ValueError:
        L2 = None
    if L2 is None or L != L2 or r != r2:
        raise ValueError(f"A must be [L, r, K] and B [L, N, r], got {list(A.shape)} and {list(B.shape)}")
    _need(adapter_offsets, torch.int64, "adapter_offsets")
    if adapter_offsets.numel() != L + 1:
        raise ValueError(f"adapter_offsets must hold L + 1 = {L + 1} entries, got {adapter_offsets.numel()}")
    if row_token is not None:
        R = _row_array(row_token, torch.int32, "row_token", R)
    if row_weight is not None:
        R = _row_array(row_weight, torch.float32, "row_weight", R)
    if rows is not None:
        R = _row_array(rows, torch.int32, name, R)
    if scaling is not None:
        _need(scaling, torch.float32, "scaling")
        if scaling.numel() != L:
            raise ValueError(f"scaling must hold L = {L} entries, got {scaling.numel()}")
    return L, r, K, N, R


def _row_array(t, dtype, name, R):
    _need(t, dtype, name)
    n = t.numel()
    if R is None:
        return n
    if n < R:
        raise ValueError(f"{name} must hold R = {R} entries, got {n}")
    return R


def _lora_x(x, act8, K: int):
    """The adapters' input as bf16 rows or as a checkpoint: (codes, scales, rows)."""
    if (x is None) == (act8 is None):
        raise ValueError("give either x or act8")
    if x is None:
        codes, scales = _act8(act8, K, "act8")
        return codes, scales, codes.shape[0]
    _need(x, torch.bfloat16, "x")
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be [T_in, K = {K}], got {list(x.shape)}")
    return None, None, x.shape[0]


def lora_apply(base: Optional[torch.Tensor], x: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
               adapter_offsets: torch.Tensor, row_token: Optional[torch.Tensor] = None,
               row_weight: Optional[torch.Tensor] = None, row_dest: Optional[torch.Tensor] = None,
               scaling: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               h: Optional[torch.Tensor] = None, R: Optional[int] = None, flags: int = 0, stream=None) -> torch.Tensor:
    """Low-rank adapters on top of a projection's output, all adapters in one launch
    (include/gnf4.h, gnf4_lora_apply): ``out[dest r] = base[dest r] + scaling[e] w(r) B[e] (A[e]
    x[tok r])`` for the rows r of adapter e, sorted as ``adapter_offsets`` says. ``A`` ``[L, r, K]``,
    ``B`` ``[L, N, r]``, all of ``x``'s type (bf16 or fp16). ``out`` defaults to ``base`` (in place).
    ``h`` (fp32 ``[R, r]``) receives what ``lora_backward`` needs. ``R``: the rows' number or an
    upper bound of it, taken from the row arrays when it is not given, else from ``x``."""
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"x must be torch.bfloat16 or torch.float16, got {x.dtype}")
    _need(x, x.dtype, "x")
    L, r, K, N, R = _lora_common(A, B, adapter_offsets, row_token, row_weight, "row_dest", row_dest, scaling, R, x.dtype)
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be [T_in, K = {K}], got {list(x.shape)}")
    T_in = x.shape[0]
    if R is None:
        R = T_in
    if base is None and out is None:
        raise ValueError("give base, or out (then the adapters' product alone is written there)")
    if out is None:
        out = base
    _need(out, x.dtype, "out")
    if out.dim() != 2 or out.shape[1] != N:
        raise ValueError(f"out must be [T_out, N = {N}], got {list(out.shape)}")
    if base is not None and base is not out:
        _need(base, x.dtype, "base")
        if base.shape != out.shape:
            raise ValueError(f"base and out must be alike, got {list(base.shape)} and {list(out.shape)}")
    if h is not None:
        h = _shaped(h, (R, r), torch.float32, "h", x)
    xdt = _lib.GNF4_DTYPE_F16 if x.dtype == torch.float16 else _lib.GNF4_DTYPE_BF16
    check(lib.gnf4_lora_apply(_ptr(base), _ptr(x), xdt, _ptr(A), _ptr(B), _ptr(adapter_offsets), _ptr(row_token),
                              _ptr(row_weight), _ptr(row_dest), _ptr(scaling), L, r, N, K, R, T_in, out.shape[0],
                              _ptr(out), _ptr(h), flags, _stream(stream)), "gnf4_lora_apply")
    return out


def lora_backward(grad_out: torch.Tensor, h: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                  adapter_offsets: torch.Tensor, x: Optional[torch.Tensor] = None, act8=None,
                  row_token: Optional[torch.Tensor] = None, row_weight: Optional[torch.Tensor] = None,
                  row_src: Optional[torch.Tensor] = None, scaling: Optional[torch.Tensor] = None,
                  dx_base: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None, want_dx: bool = True,
                  grad_dtype: torch.dtype = torch.bfloat16, dA: Optional[torch.Tensor] = None,
                  dB: Optional[torch.Tensor] = None, grad_h: Optional[torch.Tensor] = None, R: Optional[int] = None,
                  flags: int = 0, stream=None):
    """Gradients of ``lora_apply`` (bf16; include/gnf4.h, gnf4_lora_backward): (dx bf16 ``[R, K]`` in
    routed order on top of ``dx_base``, or None without ``want_dx``; dA ``[L, r, K]``; dB ``[L, N, r]``),
    the last two in ``grad_dtype`` (bf16 or fp32). ``x`` is the forward's input or ``act8 = (codes,
    scales)`` its checkpoint; with neither dA is None, and ``lora_grad_a`` gives it from ``grad_h``; ``h`` what the forward wrote; ``row_src`` its ``row_dest``. ``grad_h``
    (fp32 ``[R, r]``) is the call's own buffer; it has to be given together with ``stream``."""
    _need(grad_out, torch.bfloat16, "grad_out")
    L, r, K, N, R = _lora_common(A, B, adapter_offsets, row_token, row_weight, "row_src", row_src, scaling, R,
                                 torch.bfloat16)
    if grad_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"grad_dtype must be torch.bfloat16 or torch.float32, got {grad_dtype}")
    if grad_out.dim() != 2 or grad_out.shape[1] != N:
        raise ValueError(f"grad_out must be [T_g, N = {N}], got {list(grad_out.shape)}")
    if R is None:
        R = h.shape[0]
    if x is None and act8 is None:
        codes = scales = None
        T_in = R if row_token is None else 2 ** 31 - 1     # no row of x is read
        if grad_h is None:
            raise ValueError("without x and act8 there is no dA: pass grad_h, which lora_grad_a takes")
        if dA is not None:
            raise ValueError("dA needs x or act8")
    else:
        codes, scales, T_in = _lora_x(x, act8, K)
    _shaped(h, (R, r), torch.float32, "h", grad_out)
    if stream is not None and grad_h is None:
        raise ValueError("pass grad_h with a stream of its own (a buffer made here would be reused too early)")
    if dx_base is not None:
        want_dx = True
        _shaped(dx_base, (R, K), torch.bfloat16, "dx_base", grad_out)
    if want_dx or dx is not None:
        dx = _shaped(dx, (R, K), torch.bfloat16, "dx", grad_out if dx_base is None else dx_base)
    if x is not None or act8 is not None:
        dA = _shaped(dA, (L, r, K), grad_dtype, "dA", A)
    dB = _shaped(dB, (L, N, r), grad_dtype, "dB", B)
    grad_h = _shaped(grad_h, (R, r), torch.float32, "grad_h", h)
    gdt = _lib.GNF4_DTYPE_F32 if grad_dtype == torch.float32 else _lib.GNF4_DTYPE_BF16
    check(lib.gnf4_lora_backward(_ptr(grad_out), _ptr(x), _ptr(codes), _ptr(scales), _ptr(h), _ptr(A), _ptr(B),
                                 _ptr(adapter_offsets), _ptr(row_token), _ptr(row_weight), _ptr(row_src),
                                 _ptr(scaling), L, r, N, K, R, T_in, grad_out.shape[0], _ptr(dx_base), _ptr(dx),
                                 _ptr(grad_h), _ptr(dA), _ptr(dB), gdt, flags, _stream(stream)),
          "gnf4_lora_backward")
    return dx, dA, dB


def lora_grad_a(grad_h: torch.Tensor, adapter_offsets: torch.Tensor, x: Optional[torch.Tensor] = None, act8=None,
                row_token: Optional[torch.Tensor] = None, grad_dtype: torch.dtype = torch.bfloat16,
                dA: Optional[torch.Tensor] = None, flags: int = 0, stream=None) -> torch.Tensor:
    """dA ``[L, r, K]`` alone, from the ``grad_h`` ``[R, r]`` of a ``lora_backward`` without x
    (include/gnf4.h, gnf4_lora_grad_a)."""
    _need(grad_h, torch.float32, "grad_h")
    _need(adapter_offsets, torch.int64, "adapter_offsets")
    if grad_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"grad_dtype must be torch.bfloat16 or torch.float32, got {grad_dtype}")
    if grad_h.dim() != 2:
        raise ValueError(f"grad_h must be [R, r], got {list(grad_h.shape)}")
    (R, r), L = grad_h.shape, adapter_offsets.numel() - 1
    rows = x if act8 is None else act8[0]
    if rows is None or rows.dim() != 2:
        raise ValueError("give either x or act8, with rows [T_in, K]")
    K = rows.shape[1]
    codes, scales, T_in = _lora_x(x, act8, K)
    if row_token is not None:
        _need(row_token, torch.int32, "row_token")
        if row_token.numel() < R:
            raise ValueError(f"row_token must hold R = {R} entries, got {row_token.numel()}")
    dA = _shaped(dA, (L, r, K), grad_dtype, "dA", grad_h)
    gdt = _lib.GNF4_DTYPE_F32 if grad_dtype == torch.float32 else _lib.GNF4_DTYPE_BF16
    check(lib.gnf4_lora_grad_a(_ptr(grad_h), _ptr(x), _ptr(codes), _ptr(scales), _ptr(adapter_offsets),
                               _ptr(row_token), L, r, K, R, T_in, _ptr(dA), gdt, flags, _stream(stream)),
          "gnf4_lora_grad_a")
    return dA


def device_status(stream=None) -> None:
    """Synchronise the stream; raise if a kernel gave up waiting on a barrier."""
    check(lib.gnf4_device_status(_stream(stream)), "gnf4_device_status")


def launches_per_call(R: int, flags: int = 0) -> int:
    return lib.gnf4_grouped_gemm_launches(R, flags)


version = lib.gnf4_version
