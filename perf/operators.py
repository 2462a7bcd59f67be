"""Cases for the operators that train and serve on top of frozen 4-bit experts: low-rank
adapters beside a projection (forward and gradients) and 8-bit activation checkpoints
(written, read back, and used by the SwiGLU's and the adapters' backward passes).

``run`` computes a case in plain torch (``own`` false) or through the library (``own`` true).
Shapes are those of ``synth/workloads.py`` (hidden 2048, fused gate_up 2 x 1024 or 2 x 768,
2880 / 5760), ranks 8 to 64 are generic.

Operators:
 act8    x [R, K] -> 8-bit checkpoint -> the values it stands for (bf16, all exact)
 swiglu  a SwiGLU's training pass: the activations, and from the output's gradient the
         gate_up rows' gradient and the rebuilt activations, through a checkpoint or bf16 rows
 lora    out[dest r] = base[dest r] + s_e w_r B_e (A_e x[tok r]) for the routed rows r of adapter e
 lora_bwd its gradients: dx on top of the projection's own, dA and dB of every adapter
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------- the cases
def listed():
    return [
        # a decode step's hidden rows to a checkpoint and back: a launch-bound call
        dict(name="act8_rows16", op="act8", R=16, K=2048),
        # the routed rows of a 4096-token batch, top-8, hidden 2048
        dict(name="act8_routed", op="act8", R=32768, K=2048),
        # 16 tokens, top-8, intermediate 1024, through the 8-bit checkpoint
        dict(name="swiglu_128_ckpt", op="swiglu", R=128, I=1024, ckpt=True),
        # 4096 tokens, top-8, intermediate 768, through the 8-bit checkpoint
        dict(name="swiglu_routed_ckpt", op="swiglu", R=32768, I=768, ckpt=True),
        # 999 rows of intermediate 2880 kept as bf16 rows
        dict(name="swiglu_999_bf16", op="swiglu", R=999, I=2880, ckpt=False),
        # one request's token beside a shared projection, one of 16 resident adapters
        dict(name="lora_token", op="lora", L=16, T=1, k=1, r=16, K=2048, N=2048, zipf=False, f16=False,
             gather=True, scatter=True, weights=False, bare=0.0),
        # 61 decoding requests over 128 adapters, some without one, fp16
        dict(name="lora_requests_f16", op="lora", L=128, T=61, k=1, r=16, K=2048, N=2048, zipf=True, f16=True,
             gather=True, scatter=True, weights=False, bare=0.1),
        # prompts of a few tenants, wide projection with sizes that are no power of two, rank 64
        dict(name="lora_prompts", op="lora", L=6, T=4096, k=1, r=64, K=2880, N=5760, zipf=False, f16=False,
             gather=True, scatter=True, weights=False, bare=0.0),
        # adapters of 128 experts beside gate_up, rows in routed order
        dict(name="lora_experts", op="lora", L=128, T=4096, k=8, r=16, K=2048, N=1536, zipf=False, f16=False,
             gather=False, scatter=False, weights=False, bare=0.0),
        # a small training call: 16 tokens, top-8 of 64 experts, the down projection (weighted, scattered)
        dict(name="lora_bwd_16tok", op="lora_bwd", L=64, T=16, k=8, r=16, K=1024, N=2048, zipf=False, ckpt=False,
             gather=False, scatter=True, weights=True, grads="bf16"),
        # one adapter on a shared projection, ragged rows, rank 32, fp32 gradients
        dict(name="lora_bwd_shared", op="lora_bwd", L=1, T=4001, k=1, r=32, K=2048, N=2048, zipf=False, ckpt=False,
             gather=False, scatter=False, weights=False, grads="f32"),
        # gate_up adapters of 128 experts, 4096 tokens, top-8, the token rows checkpointed in 8 bits
        dict(name="lora_bwd_experts_ckpt", op="lora_bwd", L=128, T=4096, k=8, r=16, K=2048, N=1536, zipf=False,
             ckpt=True, gather=True, scatter=False, weights=False, grads="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["act8", "swiglu", "lora", "lora", "lora_bwd", "lora_bwd"])
    if op == "act8":
        K = 32 * _log_int(rng, 8, 128)
        return dict(op=op, R=min(_log_int(rng, 1, 30000), 32768 * 2048 // K), K=K)
    if op == "swiglu":
        I = 32 * _log_int(rng, 8, 90)
        return dict(op=op, R=min(_log_int(rng, 1, 30000), 32768 * 768 // I), I=I, ckpt=rng.random() < 0.6)
    c = dict(op=op, r=8 * _log_int(rng, 1, 8), K=8 * _log_int(rng, 32, 360), N=8 * _log_int(rng, 32, 360),
             zipf=rng.random() < 0.4)
    if rng.random() < 0.5:                      # adapters of requests beside a shared projection
        c.update(L=_log_int(rng, 1, 200), k=1, T=_log_int(rng, 1, 4096), gather=True, scatter=True, weights=False)
    else:                                       # adapters of experts: gate_up (gathered) or down (scattered)
        down = rng.random() < 0.5
        c.update(L=rng.choice([16, 40, 64, 128]), k=rng.choice([2, 4, 8]), T=_log_int(rng, 1, 2048),
                 gather=not down, scatter=down, weights=down)
    if op == "lora":
        c.update(f16=rng.random() < 0.4, bare=rng.choice([0.0, 0.2]) if c["k"] == 1 else 0.0)
    else:
        c.update(ckpt=rng.random() < 0.5, grads=rng.choice(["bf16", "bf16", "f32"]))
        if c["ckpt"]:
            c["K"] = (c["K"] + 31) // 32 * 32
    return c


# --------------------------------------------------------------------------- inputs
def _routing(case, gen):
    """Rows sorted by adapter: what the routing step hands to every grouped call."""
    L, T, k = case["L"], case["T"], case["k"]
    logits = -torch.log(-torch.log(torch.rand(T, L, generator=gen, device=DEV).clamp(1e-9, 1 - 1e-7)))
    if case["zipf"]:
        logits = logits - 1.2 * torch.log(torch.arange(1, L + 1, device=DEV, dtype=torch.float32))
    top, ids = logits.topk(min(k, L), dim=1)
    k = ids.shape[1]
    w = torch.softmax(top, dim=1)
    ids = ids.reshape(-1)
    if case.get("bare", 0.0) > 0.0:             # requests without an adapter have no row
        gone = torch.rand(T * k, generator=gen, device=DEV) < case["bare"]
        gone[0] = False
        ids = torch.where(gone, torch.full_like(ids, L), ids)
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=L + 1)[:L]
    offsets = torch.zeros(L + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = counts.cumsum(0)
    R = int(offsets[-1])
    order = order[:R]
    # the same rows as a rectangle: one line per adapter, padded with R (a row of zeros)
    M = max(1, int(counts.max()))
    seg = torch.repeat_interleave(torch.arange(L, device=DEV), counts)
    pos = torch.arange(R, device=DEV) - offsets[:-1][seg]
    pad = torch.full((L, M), R, dtype=torch.int64, device=DEV)
    pad[seg, pos] = torch.arange(R, device=DEV)
    return dict(R=R, k=k, offsets=offsets, seg=seg, pad=pad, flat=seg * M + pos,
                tok=(order // k).to(torch.int32), dest=order.to(torch.int32), w=w.reshape(-1)[order].contiguous())


def _quantize(x):
    """MXINT8 (int8 elements, one e8m0 scale per 32): the scale is the exponent field of the
    block's largest magnitude, a code counts steps of 2^(s - 133)."""
    R, K = x.shape
    e = (x.view(torch.int16).to(torch.int32) >> 7) & 255
    s = e.view(R, K // 32, 32).amax(-1)
    low = s.clamp(min=6)                        # 2^(133 - s) in two factors that 32 bits hold
    up, more = ((260 - low) << 23).view(torch.float32), ((127 + low - s) << 23).view(torch.float32)
    c = torch.round(x.view(R, K // 32, 32).float() * more[..., None] * up[..., None]).clamp(-127, 127)
    return c.to(torch.int8).view(R, K), s.to(torch.uint8)


def _dequantize(codes, scales):
    R, K = codes.shape
    s = scales.to(torch.int32)
    step = torch.where(s >= 7, (s - 6) << 23, 1 << (s.clamp(max=6) + 16)).view(torch.float32)
    return (codes.view(R, K // 32, 32).float() * step[..., None]).view(R, K)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(dtype)

    st = dict(case=dict(case))
    op = case["op"]
    if op == "act8":
        # hidden states: a few channels are much larger than the rest
        x = torch.randn(case["R"], case["K"], generator=gen, device=DEV)
        x *= torch.exp(1.0 * torch.randn(case["K"], generator=gen, device=DEV))
        st["x"] = x.to(torch.bfloat16)
        return st
    if op == "swiglu":
        st["h"] = normal(case["R"], 2 * case["I"], scale=1.5)
        st["d"] = normal(case["R"], case["I"], scale=1e-2)
        return st
    K, N, L, r = case["K"], case["N"], case["L"], case["r"]
    dt = torch.float16 if case.get("f16") else torch.bfloat16
    st.update(_routing(case, gen))
    R, k = st["R"], st["k"]
    st["A"] = normal(L, r, K, scale=K ** -0.5, dtype=dt)
    st["B"] = normal(L, N, r, scale=0.5 * r ** -0.5, dtype=dt)
    st["scaling"] = 0.5 + 1.5 * torch.rand(L, generator=gen, device=DEV)
    x = normal(case["T"] if case["gather"] else R, K, dtype=dt)
    rows = case["T"] * k if case["scatter"] else R
    if op == "lora":
        st["x"] = x
        st["base"] = normal(rows, N, dtype=dt)
        st["out"] = st["base"].clone()          # rows without an adapter keep the projection's
        return st
    st["dy"] = normal(rows, N, scale=1e-2)
    st["dx_base"] = normal(R, K, scale=1e-2)
    if case["ckpt"]:
        st["codes"], st["scales"] = _quantize(x)
    else:
        st["x"] = x
    # what the forward pass kept: h = A x
    st["h"] = _products(x.float()[st["tok"].long()] if case["gather"] else x.float(), st["A"].float().mT, st)
    return st


# --------------------------------------------------------------------------- the plain forms
def _rect(rows, st):
    """[R, C] rows -> [L, M, C], zeros in the padding."""
    return torch.cat([rows, rows.new_zeros(1, rows.shape[1])])[st["pad"]]


def _products(rows, weights, st):
    """rows[r] @ weights[adapter of r], in 32 bits."""
    out = torch.bmm(_rect(rows, st), weights)
    return out.view(-1, out.shape[-1])[st["flat"]]


def _factor(st):
    f = st["scaling"][st["seg"]]
    return (f * st["w"] if st["case"]["weights"] else f)[:, None]


def _silu_parts(h):
    g, u = h.chunk(2, dim=1)
    s = 1.0 / (1.0 + torch.exp(-g))
    return g, u, s


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "act8":
        return _dequantize(*_quantize(st["x"])).to(torch.bfloat16)
    if op == "swiglu":
        g, u, s = _silu_parts(st["h"].float())
        act = (g * s * u).to(torch.bfloat16)
        if case["ckpt"]:
            g, u, s = _silu_parts(_dequantize(*_quantize(st["h"])))
        d = st["d"].float()
        dh = torch.cat([d * u * (s * (1.0 + g * (1.0 - s))), d * (g * s)], dim=1)
        return {"act": act, "dh": dh.to(torch.bfloat16), "again": (g * s * u).to(torch.bfloat16)}
    A, B = st["A"].float(), st["B"].float()
    dest = st["dest"].long() if case["scatter"] else None
    if op == "lora":
        x = st["x"].float()
        x = x[st["tok"].long()] if case["gather"] else x
        delta = _products(_products(x, A.mT, st), B.mT, st) * _factor(st)
        if dest is None:
            st["out"].copy_(st["base"].float() + delta)
        else:
            st["out"][dest] = (st["base"].float()[dest] + delta).to(st["out"].dtype)
        return st["out"]
    x = _dequantize(st["codes"], st["scales"]) if case["ckpt"] else st["x"].float()
    x = x[st["tok"].long()] if case["gather"] else x
    dy = st["dy"].float()
    dy = (dy if dest is None else dy[dest]) * _factor(st)
    g = _products(dy, B, st)
    dx = (st["dx_base"].float() + _products(g, A, st)).to(torch.bfloat16)
    gt = torch.float32 if case["grads"] == "f32" else torch.bfloat16
    dA = torch.bmm(_rect(g, st).mT, _rect(x, st)).to(gt)
    dB = torch.bmm(_rect(dy, st).mT, _rect(st["h"], st)).to(gt)
    return {"dx": dx, "dA": dA, "dB": dB}


def run(state):
    if not own:
        return _plain(state)
    import bit_grouped_moe_gnf4_b200 as lib
    st, case = state, state["case"]
    if case["op"] == "act8":
        return lib.dequantize_act8(*lib.quantize_act8(st["x"]))
    if case["op"] == "swiglu":
        if case["ckpt"]:
            act, codes, scales = lib.swiglu_act8(st["h"])
            dh, again = lib.swiglu_backward(st["d"], act8=(codes, scales), rebuild=True)
        else:
            act = lib.swiglu(st["h"])
            dh, again = lib.swiglu_backward(st["d"], gate_up=st["h"], rebuild=True)
        return {"act": act, "dh": dh, "again": again}
    rows = dict(row_token=st["tok"] if case["gather"] else None, row_weight=st["w"] if case["weights"] else None,
                scaling=st["scaling"], R=st["R"])
    dest = st["dest"] if case["scatter"] else None
    if case["op"] == "lora":
        return lib.lora_apply(st["base"], st["x"], st["A"], st["B"], st["offsets"], row_dest=dest, out=st["out"],
                              **rows)
    x = dict(act8=(st["codes"], st["scales"])) if case["ckpt"] else dict(x=st["x"])
    dx, dA, dB = lib.lora_backward(st["dy"], st["h"], st["A"], st["B"], st["offsets"], row_src=dest,
                                   dx_base=st["dx_base"], grad_dtype=torch.float32 if case["grads"] == "f32"
                                   else torch.bfloat16, **x, **rows)
    return {"dx": dx, "dA": dA, "dB": dB}


# --------------------------------------------------------------------------- what a pass cannot do without
def _active(case):
    """Adapters that are expected to have a row."""
    L, n = case["L"], case["T"]
    k = min(case["k"], L)
    if not case["zipf"]:
        return L * (1.0 - (1.0 - k / L) ** n)
    p = [(i + 1) ** -1.2 for i in range(L)]
    z = sum(p)
    return sum(1.0 - (1.0 - min(1.0, k * v / z)) ** n for v in p)


def work(case):
    op = case["op"]
    if op == "act8":
        n = case["R"] * case["K"]
        return {"bytes": n * (2 + 2 * 33 / 32 + 2), "flops": 4 * n}
    if op == "swiglu":
        n = case["R"] * case["I"]
        keep = 2 * 33 / 32
        ahead = 4 + 2 + (keep if case["ckpt"] else 0)
        back = 2 + (keep if case["ckpt"] else 4) + 4 + 2
        return {"bytes": n * (ahead + back), "flops": 30 * n}
    K, N, r, L = case["K"], case["N"], case["r"], case["L"]
    rows = case["T"] * min(case["k"], L) * (1.0 - case.get("bare", 0.0))
    xs = min(case["T"], rows) if case["gather"] else rows
    active = _active(case)
    if op == "lora":
        return {"bytes": 2 * (xs * K + 2 * rows * N + active * r * (K + N)), "flops": 2 * rows * r * (K + N)}
    gb = 4 if case["grads"] == "f32" else 2
    return {"bytes": xs * K * (33 / 32 if case["ckpt"] else 2) + 2 * rows * (N + 2 * K) + 4 * rows * r
            + 2 * active * r * (K + N) + gb * L * r * (K + N),
            "flops": 4 * rows * r * (K + N)}


# --------------------------------------------------------------------------- in 64 bits, from the definitions
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64

    def values8(x):
        """Each value to the nearest of c steps, |c| <= 127, the step 2^-6 of the power of two that the
        block's largest magnitude starts with."""
        v = x.to(f64).unflatten(1, (-1, 32))
        m = v.abs().amax(-1, keepdim=True)
        step = torch.where(m >= 2.0 ** -126, m / torch.frexp(m).mantissa / 128, torch.full_like(m, 2.0 ** -133))
        return (torch.round(v / step).clamp(-127, 127) * step).flatten(1)

    if op == "act8":
        return values8(st["x"])
    if op == "swiglu":
        d, h = st["d"].to(f64), st["h"].to(f64)
        I = case["I"]
        act = h[:, I:] * h[:, :I] * torch.sigmoid(h[:, :I])
        if case["ckpt"]:
            h = values8(st["h"])
        sg = torch.sigmoid(h[:, :I])
        silu = h[:, :I] * sg
        return {"act": act, "dh": torch.cat([d * h[:, I:] * (sg + silu * (1 - sg)), d * silu], 1),
                "again": silu * h[:, I:]}
    off = st["offsets"].tolist()
    tok = st["tok"].long() if case["gather"] else torch.arange(st["R"], device=DEV)
    dest = st["dest"].long() if case["scatter"] else torch.arange(st["R"], device=DEV)
    w = st["w"].to(f64) if case["weights"] else torch.ones(st["R"], dtype=f64, device=DEV)
    parts = [(e, slice(off[e], off[e + 1])) for e in range(case["L"])]
    if op == "lora":
        out = st["base"].to(f64)
        for e, s in parts:
            if s.start < s.stop:
                h = st["x"][tok[s]].to(f64) @ st["A"][e].to(f64).T
                out[dest[s]] += float(st["scaling"][e]) * w[s, None] * (h @ st["B"][e].to(f64).T)
        return out
    x = st["codes"].to(f64) * torch.ldexp(torch.ones((), dtype=f64, device=DEV), st["scales"].to(f64) - 133
                                          ).repeat_interleave(32, 1) if case["ckpt"] else st["x"].to(f64)
    dx = st["dx_base"].to(f64)
    dA = torch.zeros(st["A"].shape, dtype=f64, device=DEV)
    dB = torch.zeros(st["B"].shape, dtype=f64, device=DEV)
    for e, s in parts:
        if s.start < s.stop:
            t = float(st["scaling"][e]) * w[s, None] * st["dy"][dest[s]].to(f64)
            g = t @ st["B"][e].to(f64)
            dx[s] += g @ st["A"][e].to(f64)
            dA[e] = g.T @ x[tok[s]]
            dB[e] = t.T @ st["h"][s].to(f64)
    return {"dx": dx, "dA": dA, "dB": dB}
