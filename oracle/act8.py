"""Plain CPU oracle for the 8-bit activation checkpoints and the SwiGLU's backward pass.

TEST INFRASTRUCTURE ONLY, like ``gnf4_oracle``; shares no code with the CUDA path.

The format is OCP MXINT8 (Open Compute Project, Microscaling Formats specification 1.0:
int8 elements with an implied 2^-6, one e8m0 scale per 32 elements, the scale's exponent
floor(log2 amax)), on bf16 input. An element counts steps of 2^(s - 133).
"""
from __future__ import annotations

import numpy as np

from .gnf4_oracle import bf16_to_f64

BLOCK = 32


def quantize_act8(x_bits: np.ndarray):
    """bf16 bits [..., K] -> (codes int8 [..., K], scales uint8 [..., K/32])."""
    x_bits = np.asarray(x_bits, np.uint16)
    shape = x_bits.shape
    blocks = x_bits.reshape(shape[:-1] + (shape[-1] // BLOCK, BLOCK))
    v = bf16_to_f64(blocks)
    s = np.zeros(blocks.shape[:-1], np.int64)
    finite = np.isfinite(v).all(axis=-1)
    amax = np.abs(np.where(np.isfinite(v), v, 0.0)).max(axis=-1)
    normal = amax >= 2.0 ** -126
    s[normal] = np.floor(np.log2(amax[normal])).astype(np.int64) + 127
    s[~finite] = 255
    with np.errstate(invalid="ignore"):
        c = np.clip(np.rint(v * 2.0 ** (133.0 - s[..., None])), -127, 127)
    c[~finite] = 0
    return c.astype(np.int8).reshape(shape), s.astype(np.uint8)


def values_act8(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The fp64 values of a checkpoint."""
    codes = np.asarray(codes, np.int8)
    c = codes.reshape(codes.shape[:-1] + (codes.shape[-1] // BLOCK, BLOCK)).astype(np.float64)
    s = np.asarray(scales, np.uint8).astype(np.float64)[..., None]
    return np.where(s == 255, np.nan, c * 2.0 ** (s - 133.0)).reshape(codes.shape)


def swiglu_backward_f64(grad_out: np.ndarray, gate_up: np.ndarray) -> np.ndarray:
    """d(silu(gate) up) by its inputs, times ``grad_out``: fp64 [R, I], [R, 2I] -> [R, 2I]."""
    I = grad_out.shape[-1]
    g, u = gate_up[..., :I], gate_up[..., I:]
    e = np.exp(-np.abs(g))
    sig = np.where(g >= 0, 1.0, e) / (1.0 + e)
    rest = np.where(g >= 0, e, 1.0) / (1.0 + e)
    return np.concatenate([grad_out * u * sig * (1.0 + g * rest), grad_out * g * sig], axis=-1)


def swiglu_backward_bound(grad_out: np.ndarray, gate_up: np.ndarray) -> np.ndarray:
    """What the fp32 error of a gradient is relative to: |d u sig| (1 + |g|) and |d g sig|."""
    I = grad_out.shape[-1]
    g, u = gate_up[..., :I], gate_up[..., I:]
    sig = np.where(g >= 0, 1.0, np.exp(-np.abs(g))) / (1.0 + np.exp(-np.abs(g)))
    return np.abs(np.concatenate([grad_out * u * sig * (1.0 + np.abs(g)), grad_out * g * sig], axis=-1))
