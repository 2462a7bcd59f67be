"""Plain CPU oracle for the low-rank adapters beside a projection and their gradients.

TEST INFRASTRUCTURE ONLY, like ``gnf4_oracle``; shares no code with the CUDA path. All
arrays fp64 (the values of the 16-bit inputs), one adapter after the other. The ``bound``
results are the same sums over magnitudes, which rounding errors are relative to.
"""
from __future__ import annotations

import numpy as np


def _rows(offsets, row, R):
    row = np.arange(R) if row is None else np.asarray(row)
    return [(e, slice(int(offsets[e]), int(offsets[e + 1]))) for e in range(len(offsets) - 1)], row


def _factor(offsets, weight, scaling, R):
    c = np.ones(R)
    if weight is not None:
        c = c * np.asarray(weight, np.float64)[:R]
    if scaling is not None:
        for e in range(len(offsets) - 1):
            c[int(offsets[e]):int(offsets[e + 1])] *= float(scaling[e])
    return c


def lora_apply_f64(base, x, A, B, offsets, row_token=None, row_weight=None, row_dest=None, scaling=None):
    """(out like base, h [R, r], bound like base)."""
    R = int(offsets[-1])
    segs, tok = _rows(offsets, row_token, R)
    dest = np.arange(R) if row_dest is None else np.asarray(row_dest)
    c = _factor(offsets, row_weight, scaling, R)
    out, bound, h = base.copy(), np.zeros_like(base), np.zeros((R, A.shape[1]))
    for e, s in segs:
        if s.start == s.stop:
            continue
        xs = x[tok[s]]
        h[s] = xs @ A[e].T
        out[dest[s]] = base[dest[s]] + c[s, None] * (h[s] @ B[e].T)
        top = (np.abs(xs) @ np.abs(A[e]).T).max(axis=1, keepdims=True)
        bound[dest[s]] = np.abs(c[s, None]) * top * np.abs(B[e]).sum(axis=1)[None, :]
    return out, h, bound


def lora_backward_f64(grad_out, x, h, A, B, offsets, row_token=None, row_weight=None, row_src=None, scaling=None,
                      dx_base=None):
    """dict of dx, dA, dB, grad_h and their bounds (``*_bound``)."""
    R = int(offsets[-1])
    segs, tok = _rows(offsets, row_token, R)
    src = np.arange(R) if row_src is None else np.asarray(row_src)
    c = _factor(offsets, row_weight, scaling, R)
    K = A.shape[2]
    o = dict(dx=np.zeros((R, K)) if dx_base is None else dx_base[:R].copy(), dA=np.zeros(A.shape), dB=np.zeros(B.shape),
             grad_h=np.zeros((R, A.shape[1])))
    b = {k + "_bound": np.zeros(v.shape) for k, v in o.items()}
    for e, s in segs:
        if s.start == s.stop:
            continue
        t = c[s, None] * grad_out[src[s]]
        o["grad_h"][s] = t @ B[e]
        o["dx"][s] += o["grad_h"][s] @ A[e]
        o["dA"][e] = o["grad_h"][s].T @ x[tok[s]]
        o["dB"][e] = t.T @ h[s]
        gb = np.abs(t) @ np.abs(B[e])
        b["grad_h_bound"][s] = gb
        b["dx_bound"][s] = gb @ np.abs(A[e])
        b["dA_bound"][e] = gb.T @ np.abs(x[tok[s]])
        b["dB_bound"][e] = np.abs(t).T @ np.abs(h[s])
    o.update(b)
    return o
