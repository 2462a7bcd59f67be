"""Parity of the low-rank adapters and their gradients with the fp64 oracle, through the binding.

Tolerances. u is the output type's half step (bf16 2^-8, fp16 2^-11, fp32 2^-24), relative to
the value. What comes before that rounding is relative to the oracle's bound (the same sums
over magnitudes): an fp32 accumulation of n terms is off by at most n 2^-23 of it in any order,
also when an addition truncates instead of rounding, and every operand that is split into two
16-bit terms adds 2^-16 (bf16: 2^-9 of the remainder, itself 2^-9; fp16 less), three terms
2^-24. So with n = K + r (forward), N + r (dx), N + rows (dA), rows (dB), plus 32 for the
handful of products and joins on the way:
    |out - want| <= u |want| + (1 + u) (n 2^-23 + 2^-16) bound, and half a step of the type's subnormals
A base on top may be where the fp32 accumulation of the second product starts: r/8 additions
(two terms, 16 ranks each) of 2^-23 of it.
"""
import numpy as np
import pytest
import torch

from oracle import act8 as A8
from oracle import glue as GL
from oracle import gnf4_oracle as O
from oracle import lora as LO

from gpu_support import build_stack

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}    # half a subnormal step


def lib():
    import bit_grouped_moe_gnf4_b200 as g
    return g


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def near(got, want, bound, n, terms, what, base=0.0, r=0):
    u = HALF[got.dtype]
    e = n * 2.0 ** -23 + (2.0 ** -16 if terms == 2 else 2.0 ** -24)
    tol = u * np.abs(want) + (1 + u) * (e * bound + (r / 8 + 2) * 2.0 ** -23 * np.abs(base)) + TINY[got.dtype]
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), f"{what}: {int((err > tol).sum())} of {err.size} off, worst {float((err / tol).max()):.3g} of the bound"


class Problem:
    """Rows of `counts[e]` per adapter; options as in the call."""

    def __init__(self, counts, r, K, N, dtype=torch.bfloat16, gather=True, scatter=True, weights=True, scaling=True,
                 spare=0, seed=0, far=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        L, R = len(counts), int(sum(counts))
        self.R, self.L, self.spare = R, L, spare
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
        rand = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).to(dtype)  # noqa: E731
        T_in = max(1, R // 2 + 3) if gather else R + spare
        T_out = R + 5 + far if scatter else R + spare
        self.x, self.base = rand(T_in, K), rand(T_out, N)
        self.A, self.B = rand(L, r, K, scale=K ** -0.5), rand(L, N, r, scale=r ** -0.5)
        self.offsets = torch.from_numpy(off).cuda()
        # the entries behind the last row are never read: out of range on purpose
        pad = lambda a: torch.from_numpy(np.concatenate([a, np.full(spare, -7, a.dtype)])).cuda()  # noqa: E731
        self.tok = pad(rng.integers(0, T_in, R).astype(np.int32)) if gather else None
        self.dest = pad(rng.permutation(T_out)[:R].astype(np.int32)) if scatter else None
        self.w = torch.cat([torch.rand(R, generator=gen, device="cuda") + 0.1, torch.full((spare,), float("nan"), device="cuda")]) if weights else None
        self.s = torch.rand(L, generator=gen, device="cuda") * 2 - 1 if scaling else None

    def rows(self):
        return dict(row_token=self.tok, row_weight=self.w, scaling=self.s, R=self.R + self.spare)

    def host(self):
        cut = lambda t: None if t is None else t[:self.R].cpu().numpy()  # noqa: E731
        return dict(row_token=cut(self.tok), row_weight=cut(self.w), scaling=f64(self.s))

    def forward(self, **kw):
        g = lib()
        h = torch.full((self.R + self.spare, self.A.shape[1]), 5.0, device="cuda")
        out = self.base.clone()
        g.lora_apply(self.base, self.x, self.A, self.B, self.offsets, row_dest=self.dest, out=out, h=h, **self.rows(), **kw)
        torch.cuda.synchronize()
        return out, h

    def check_forward(self):
        out, h = self.forward()
        want, wh, bound = LO.lora_apply_f64(f64(self.base), f64(self.x), f64(self.A), f64(self.B),
                                            self.offsets.cpu().numpy(), row_dest=None if self.dest is None else
                                            self.dest[:self.R].cpu().numpy(), **self.host())
        K, r = self.A.shape[2], self.A.shape[1]
        near(out, want, bound, K + r + 32, 2, "out", f64(self.base), r)
        hb = np.abs(f64(self.x))[self.host()["row_token"] if self.tok is not None else slice(0, self.R)].max() * \
            np.abs(f64(self.A)).sum(axis=2).max()
        near(h[:self.R], wh, np.full_like(wh, hb), K + 32, 3, "h")
        assert (h[self.R:] == 5).all()
        free = np.ones(len(out), bool)
        free[np.arange(self.R) if self.dest is None else self.dest[:self.R].cpu().numpy()] = False
        assert torch.equal(out[torch.from_numpy(free).cuda()], self.base[torch.from_numpy(free).cuda()])
        return out, h

    def check_backward(self, grads=torch.bfloat16, act8=False, base=True):
        g = lib()
        gen = torch.Generator(device="cuda").manual_seed(99)
        r, K, N = self.A.shape[1], self.A.shape[2], self.B.shape[1]
        dy = (torch.randn(self.base.shape, generator=gen, device="cuda") * 0.1).to(torch.bfloat16)
        Rp = self.R + self.spare
        h = torch.randn(Rp, r, generator=gen, device="cuda")
        dxb = torch.randn(Rp, K, generator=gen, device="cuda").to(torch.bfloat16) if base else None
        x, xv = dict(x=self.x), f64(self.x)
        if act8:
            q = g.quantize_act8(self.x)
            x, xv = dict(act8=q), A8.values_act8(q[0].cpu().numpy(), q[1].cpu().numpy())
        gh = torch.full((Rp, r), 5.0, device="cuda")
        dx = torch.full((Rp, K), 3.0, device="cuda").to(torch.bfloat16)
        out = g.lora_backward(dy, h, self.A, self.B, self.offsets, row_src=self.dest, dx_base=dxb, dx=dx, grad_h=gh,
                              grad_dtype=grads, **x, **self.rows())
        torch.cuda.synchronize()
        assert out[0] is dx and (dx[self.R:] == 3).all() and (gh[self.R:] == 5).all()
        w = LO.lora_backward_f64(f64(dy), xv, f64(h), f64(self.A), f64(self.B), self.offsets.cpu().numpy(),
                                 row_src=None if self.dest is None else self.dest[:self.R].cpu().numpy(),
                                 dx_base=f64(dxb), **self.host())
        m = int(np.diff(self.offsets.cpu().numpy()).max())
        terms = 3 if grads == torch.float32 else 2
        near(gh[:self.R], w["grad_h"], w["grad_h_bound"], N + 32, 3, "grad_h")
        near(dx[:self.R], w["dx"], w["dx_bound"], N + r + 32, 2, "dx", 0.0 if dxb is None else f64(dxb)[:self.R], r)
        near(out[1], w["dA"], w["dA_bound"], N + m + 32, terms, "dA")
        near(out[2], w["dB"], w["dB_bound"], m + 32, terms, "dB")
        return out


ROWS = {
    "one": [1],
    "few": [0, 3, 0, 17, 1, 0],
    "ragged": [33, 0, 64, 100, 16, 15, 1],
    "long": [700],
    "skewed": [1500, 0, 2, 1, 40],
    "many": [i % 3 for i in range(300)],
    "limit": [1 if i % 17 == 0 else 0 for i in range(2048)],
}


@pytest.mark.parametrize("counts", list(ROWS))
@pytest.mark.parametrize("r,K,N", [(16, 256, 192), (8, 72, 40), (32, 520, 136)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_apply_over_row_counts(counts, r, K, N, dtype):
    Problem(ROWS[counts], r, K, N, dtype=dtype, seed=r).check_forward()


@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 104, 128])
@pytest.mark.parametrize("K,N", [(8, 8), (2048, 1536), (2888, 5768), (32, 2048)])
def test_apply_over_sizes(r, K, N):
    for counts in ([2, 0, 5], [40, 90]):
        Problem(counts, r, K, N, dtype=torch.float16 if r % 16 else torch.bfloat16, seed=K).check_forward()


@pytest.mark.parametrize("kw", [dict(gather=False), dict(scatter=False), dict(weights=False), dict(scaling=False),
                                dict(gather=False, scatter=False, weights=False, scaling=False), dict(spare=9),
                                dict(spare=40, gather=False, scatter=False)])
def test_apply_without_each_array(kw):
    for counts in ([3, 0, 20], [60, 1]):
        Problem(counts, 16, 264, 200, **kw).check_forward()


@pytest.mark.parametrize("counts", list(ROWS))
@pytest.mark.parametrize("r,K,N", [(16, 256, 192), (8, 96, 40), (40, 544, 136)])
@pytest.mark.parametrize("grads", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act8", [False, True])
def test_backward_over_row_counts(counts, r, K, N, grads, act8):
    Problem(ROWS[counts], r, K, N, seed=r).check_backward(grads, act8)


@pytest.mark.parametrize("r", [8, 24, 32, 64, 72, 128])
@pytest.mark.parametrize("K,N", [(8, 8), (32, 8), (2048, 1536), (1032, 2888)])
def test_backward_over_sizes(r, K, N):
    for counts, grads in (([2, 0, 5], torch.float32), ([40, 300], torch.bfloat16)):
        Problem(counts, r, K, N, seed=K).check_backward(grads, act8=K % 32 == 0)


@pytest.mark.parametrize("kw", [dict(gather=False), dict(scatter=False), dict(weights=False), dict(scaling=False),
                                dict(gather=False, scatter=False, weights=False, scaling=False), dict(spare=9),
                                dict(spare=40, gather=False, scatter=False)])
def test_backward_without_each_array(kw):
    for counts in ([3, 0, 20], [60, 1]):
        Problem(counts, 16, 264, 200, **kw).check_backward()
        Problem(counts, 16, 264, 200, **kw).check_backward(base=False)


LARGE = {"one": [2500], "several": [900, 0, 1, 700, 1000, 0], "many": [25] * 100, "more": [61] * 170,
         "skewed": [9000] + [i % 4 for i in range(200)]}


@pytest.mark.parametrize("counts", list(LARGE))
@pytest.mark.parametrize("r,K,N", [(16, 256, 192), (8, 72, 40), (24, 520, 136), (64, 264, 776), (40, 1032, 512), (128, 200, 264)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_many_rows(counts, r, K, N, dtype):
    p = Problem(LARGE[counts], r, K, N, dtype=dtype, seed=r, spare=3)
    p.check_forward()
    if dtype == torch.bfloat16:
        p.check_backward(torch.float32, act8=K % 32 == 0)


@pytest.mark.parametrize("r", [16, 24])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_for_several_rounds(r, dtype):
    # tiles of 64 rows, several to an SM, the last of most adapters partial
    p = Problem([100 + (37 * i) % 101 for i in range(140)] + [0, 1], r, 264, 288, dtype=dtype, seed=r, spare=5)
    assert p.R > 64 * 2 * 148
    p.check_forward()
    if dtype == torch.bfloat16:
        p.check_backward()


@pytest.mark.parametrize("r,K,N", [(8, 8, 8), (16, 40, 24), (32, 8, 16), (64, 16, 8)])
def test_many_rows_of_narrow_axes_and_many_adapters(r, K, N):
    p = Problem([2] * 2048, r, K, N, seed=r)
    p.check_forward()
    p.check_backward()
    Problem([13] * 2000, r, K, N, dtype=torch.float16, seed=r).check_forward()      # a table that leaves no room for 64 rows
    Problem([3000], r, K, N, seed=r).check_backward(torch.float32)


def test_many_rows_without_arrays_and_with_bad_ones():
    p = Problem([2600, 0, 77], 16, 264, 200, gather=False, scatter=False, weights=False, scaling=False)
    p.check_forward()
    p.check_backward(base=False)
    p = Problem([2600, 0, 77], 32, 96, 72)
    ok, _ = p.forward()
    dest = p.dest.clone()
    p.tok[2], p.dest[2677 - 1] = len(p.x), -1
    p.x[5] = float("nan")                                # one token's rows
    out, _ = p.forward()
    hit = (p.tok == 5)
    want = ok.clone()
    want[dest[-1].long()] = p.base[dest[-1].long()]
    want[dest[2].long()] = p.base[dest[2].long()]
    rest = torch.ones(len(out), dtype=torch.bool, device="cuda")
    rest[dest[hit].long()] = False
    assert torch.equal(out[rest], want[rest])
    hit[-1] = False
    assert out[dest[hit].long()].isnan().all()


def test_long_segments_split_over_a_cluster():
    # enough rows of one adapter for every cluster size of the gradient sums
    for m in (1100, 2300, 5000, 9001):
        Problem([m], 16, 136, 72, seed=m).check_backward(torch.float32)


@pytest.mark.parametrize("r,K,N", [(16, 608, 576), (8, 72, 40), (32, 520, 1032), (64, 264, 776), (128, 200, 264)])
@pytest.mark.parametrize("heavy", [(0,), (99,), (3, 4, 50), tuple(range(7))])
def test_a_few_adapters_have_most_rows(heavy, r, K, N):
    # a hundred adapters and more; those of many rows are shared by CTAs, alone or in a row, the first or the last
    counts = [1400 if i in heavy else i % 41 for i in range(100)]
    p = Problem(counts, r, K, N, seed=r, spare=1700)
    p.check_backward(torch.float32 if len(heavy) > 1 else torch.bfloat16, act8=K % 32 == 0)


@pytest.mark.parametrize("many", [300, 1300])
def test_a_few_of_many_adapters_have_most_rows(many):
    # runs of adapters to a thread
    counts = [2500 if i in (1, 299, 600, 1299) else 30 + i % 5 for i in range(many)]
    p = Problem(counts, 16, 96, 64, seed=many)
    p.check_backward()
    a = p.check_backward()
    assert all(torch.equal(u, v) for u, v in zip(a, p.check_backward()))


def test_half_of_the_adapters_have_most_rows():
    # as many of more than four times the average as there can be, and an average that spare rows raise
    Problem([257, 0, 0, 0, 0] * 30, 16, 520, 264, seed=1).check_backward()
    Problem([300, 1] * 60, 24, 520, 264, seed=2, spare=90).check_backward(torch.float32)


@pytest.mark.parametrize("r", [16, 64])
@pytest.mark.parametrize("counts", [[4096 if i == 66 else 0 for i in range(200)], [0] * 199 + [2000],
                                    [1500 if i in (0, 7, 8, 1023) else 20 * (i % 2) for i in range(1024)]])
def test_most_rows_in_one_of_many_adapters(counts, r):
    # an average of few rows
    p = Problem(counts, r, 96, 72, seed=r)
    p.check_backward(torch.float32)
    p.check_backward(act8=True)


def test_one_adapter_of_many_does_not_wait_for_its_rows_one_after_the_other():
    """The rows of one adapter are shared out also where 200 adapters have 20 rows on average: the
    backward pass then takes about a quarter longer than over even rows, and 3.8 times as long if
    one CTA walks them all. 2.4 lies between the two."""
    g = lib()
    L, R, r, K, N = 200, 4096, 16, 2048, 1536
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    A, B, x, dy, h = rand(L, r, K), rand(L, N, r), rand(R, K), rand(R, N), torch.randn(R, r, generator=gen, device="cuda")
    took = []
    for counts in ([R // L + (i < R % L) for i in range(L)], [R if i == 66 else 0 for i in range(L)]):
        off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)])).cuda()
        call = lambda: g.lora_backward(dy, h, A, B, off, x=x)  # noqa: E731
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(8):
                call()
        times = []
        for _ in range(12):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        took.append(min(times))
    assert took[1] < 2.4 * took[0], took


def bf16_terms(v, n):
    """The sum of n bf16 numbers, each the rounding of what the ones before it leave (fp64 arrays)."""
    total = np.zeros_like(v)
    for _ in range(n):
        total += O.bf16_to_f64(O.bf16_bits(v - total))
    return total


@pytest.mark.parametrize("r", [8, 32, 40, 128])
@pytest.mark.parametrize("act8", [False, True])
def test_fp32_gradients_of_single_rows_have_all_bits(r, act8):
    """One row an adapter: a gradient is one product of a 24-bit and an 8-bit number. Three bf16 terms
    leave 2^-27 of the first; the three products are exact and added up with 2^-23 each, and the
    result is fp32. With the first two terms alone the oracle's own products are past the tolerance."""
    g = lib()
    L, K, N = 5, 96, 72
    gen = torch.Generator(device="cuda").manual_seed(r)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, dy, h = rand(L, K).to(torch.bfloat16), rand(L, N).to(torch.bfloat16), rand(L, r)
    A, B = rand(L, r, K).to(torch.bfloat16), rand(L, N, r).to(torch.bfloat16)
    off = torch.arange(L + 1, device="cuda")
    gh = torch.empty(L, r, device="cuda")
    q = g.quantize_act8(x)
    src, xv = (dict(act8=q), A8.values_act8(q[0].cpu().numpy(), q[1].cpu().numpy())) if act8 else (dict(x=x), f64(x))
    _, dA, dB = g.lora_backward(dy, h, A, B, off, grad_h=gh, grad_dtype=torch.float32, **src)
    tol = 2.0 ** -27 + 3 * 2.0 ** -23 + 2.0 ** -24
    for got, left, outer in ((dA, f64(gh), lambda v: v[:, :, None] * xv[:, None, :]),
                             (dB, f64(h), lambda v: f64(dy)[:, :, None] * v[:, None, :])):
        want = outer(left)
        err = np.abs(f64(got) - want)
        assert np.all(err <= tol * np.abs(want)), float((err / np.abs(want).clip(1e-300)).max())
        assert np.any(np.abs(outer(bf16_terms(left, 2)) - want) > 2 * tol * np.abs(want))
        assert np.all(np.abs(outer(bf16_terms(left, 3)) - want) <= 2.0 ** -26 * np.abs(want))


@pytest.mark.parametrize("r,counts", [(16, [2, 1]), (16, [8] * 150), (32, [8] * 150), (64, [8] * 150), (128, [8] * 150),
                                      (8, [2400]), (24, [1300, 1200]), (64, [2500])])
def test_long_axes_lose_nothing(r, counts):
    """h and grad_h over 2^16 columns, all products positive. At most 32 matrix instructions follow one
    another, each off by 2^-23 of its own short sum; the sums of those chains (16 a warp, of eight
    warps) are added up with 2^-24 of the total each. In one chain of 512 the error was 9e-6."""
    g = lib()
    long_ = 1 << 16
    gen = torch.Generator(device="cuda").manual_seed(r)
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    L, R = len(counts), sum(counts)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)])).cuda()
    adapter = torch.repeat_interleave(torch.arange(L, device="cuda"), torch.tensor(counts, device="cuda"))
    tok = (torch.arange(R, device="cuda") % 8).to(torch.int32)
    x, short, A, B = rand(8, long_), rand(8, 8), rand(L, r, long_), rand(L, 8, r)
    tol = 32 * 2.0 ** -23 + (16 + 16) * 2.0 ** -24

    def off_by(got, weights):                            # weights [L, r, long]: every product of a token and an adapter
        worst = 0.0
        for e in range(L):
            want = x.double() @ weights[e].double().T
            mine = adapter == e
            worst = max(worst, float(((got[mine].double() - want[tok[mine].long()]) / want[tok[mine].long()]).abs().max()))
        return worst

    h, gh = torch.empty(R, r, device="cuda"), torch.empty(R, r, device="cuda")
    g.lora_apply(None, x, A, B, off, row_token=tok, out=torch.empty(R, 8, device="cuda").bfloat16(), h=h)
    assert off_by(h, A) <= tol
    Bt = A.mT.contiguous()
    g.lora_backward(x, h, B.mT.contiguous(), Bt, off, x=short, row_token=tok, row_src=tok, want_dx=False, grad_h=gh)
    assert off_by(gh, A) <= tol


@pytest.mark.parametrize("r", [16, 24, 64, 128])
@pytest.mark.parametrize("counts", [[(1 << 20) + 5000], [0, 1 << 18] + [4] * 198])
def test_long_sums_lose_nothing(counts, r):
    """fp32 gradients of an adapter of very many rows, all products positive or of either sign. At most
    48 matrix instructions follow one another (eight stages, two steps of 16 rows, three terms),
    each off by 2^-23 of its own short sum; those sums are added up, rounded to nearest (2^-24 of
    the total each), 256 rows at a time along the eighth (here a quarter with 200 adapters) of the
    rows that a CTA has. 16 for the three terms' remainders and the joins. In one unbroken chain of
    truncated sums the error was 2^-26 of the total for every instruction. A bf16 result's chains
    have 4096 instructions; of its own it has the rounding and 2^-17 for the terms."""
    g = lib()
    m, parts = max(counts), 8 if len(counts) == 1 else 4
    R, K, N = sum(counts), 32, 24
    gen = torch.Generator(device="cuda").manual_seed(r)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)])).cuda()
    e = int(np.argmax(counts))
    lo = int(off[e])
    A, B = torch.zeros(len(counts), r, K, device="cuda").bfloat16(), torch.zeros(len(counts), N, r, device="cuda").bfloat16()
    tol = (48 + 16) * 2.0 ** -23 + m / parts / 256 * 2.0 ** -24
    for positive in (True, False):
        rand = (lambda *s: torch.rand(*s, generator=gen, device="cuda")) if positive else \
               (lambda *s: torch.randn(*s, generator=gen, device="cuda"))  # noqa: E731
        x, dy, h = rand(R, K).to(torch.bfloat16), rand(R, N).to(torch.bfloat16), rand(R, r)
        dA = g.lora_grad_a(h, off, x=x, grad_dtype=torch.float32)
        q = g.quantize_act8(x)
        dA8 = g.lora_grad_a(h, off, act8=q, grad_dtype=torch.float32)
        dB = g.lora_backward(dy, h, A, B, off, x=x, want_dx=False, grad_dtype=torch.float32)[2]
        half = g.lora_grad_a(h, off, x=x)
        for got, left, right, what in ((dA, h, x, "dA"), (dA8, h, g.dequantize_act8(*q), "dA from codes"), (dB, dy, h, "dB"),
                                       (half, h, x, "bf16 dA")):
            want = torch.zeros(got[e].shape, dtype=torch.float64, device="cuda")
            bound = want.clone()
            for a, b in zip(left[lo:lo + m].split(1 << 17), right[lo:lo + m].split(1 << 17)):
                want += a.double().T @ b.double()
                bound += a.double().abs().T @ b.double().abs()
            err = (got[e].double() - want).abs()
            if got is half:
                allowed = tol + (4096 - 48) * 2.0 ** -23 + 2.0 ** -16
                assert (err <= 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * allowed * bound).all(), what
            else:
                worst = float((err / bound).max())
                assert worst <= tol, f"{what}, positive {positive}: {worst:.3g} of the magnitudes, {tol:.3g} allowed"


def test_in_place_and_deterministic():
    p = Problem([7, 0, 50, 1], 16, 256, 320)
    out, _ = p.forward()
    y = p.base.clone()
    assert lib().lora_apply(y, p.x, p.A, p.B, p.offsets, row_dest=p.dest, **p.rows()) is y
    assert torch.equal(y, out)
    assert torch.equal(p.forward()[0], out)
    a, b = p.check_backward(), p.check_backward()
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    # dx continues dx_base in place
    g = lib()
    dy, h = torch.randn_like(p.base), torch.randn(p.R, 16, device="cuda")
    dxb = torch.randn(p.R, 256, device="cuda").to(torch.bfloat16)
    kw = dict(x=p.x, row_src=p.dest, **p.rows())
    want = g.lora_backward(dy, h, p.A, p.B, p.offsets, dx_base=dxb, **kw)[0]
    got = g.lora_backward(dy, h, p.A, p.B, p.offsets, dx_base=dxb, dx=dxb, **kw)[0]
    assert got is dxb and torch.equal(got, want)


@pytest.mark.parametrize("r", [16, 32, 64, 128])
@pytest.mark.parametrize("counts", [[3, 0, 1], [40] * 30, [900, 0, 1600, 33], [2100] + [9] * 100])
@pytest.mark.parametrize("grads", [torch.bfloat16, torch.float32])
def test_a_call_repeats_itself_behind_others(counts, r, grads):
    # the same inputs, at first alone, then with other calls before and after and nothing waited for
    g = lib()
    one, two = (Problem(counts, r, 264, 200, seed=s) for s in (1, 2))
    for p in (one, two):
        p.dy, p.hh = torch.randn_like(p.base), torch.randn(p.R, r, device="cuda")

    def step(p):
        h = torch.empty(p.R, r, device="cuda")
        out = g.lora_apply(p.base, p.x, p.A, p.B, p.offsets, row_dest=p.dest, out=p.base.clone(), h=h, **p.rows())
        return (out, h, *g.lora_backward(p.dy, p.hh, p.A, p.B, p.offsets, x=p.x, row_src=p.dest, grad_dtype=grads, **p.rows()))

    torch.cuda.synchronize()
    want = step(one)
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        step(two)
        got.append(step(one))
        step(two)
    torch.cuda.synchronize()
    for again in got:
        assert all(torch.equal(a, b) for a, b in zip(again, want))


@pytest.mark.parametrize("r", [16, 24, 64, 128])
@pytest.mark.parametrize("R", [40, 300, 2600, 21000])
def test_a_rows_bits_do_not_depend_on_the_others(r, R):
    # one token of adapter 3, alone and among others, in the same R and L: every split that the calls choose
    g = lib()
    L, K, N = 5, 392, 328
    gen = torch.Generator(device="cuda").manual_seed(R)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    A, B, scal = rand(L, r, K), rand(L, N, r), torch.rand(L, generator=gen, device="cuda")
    token, above, behind, under = rand(1, K), rand(1, N), rand(1, N), rand(1, K)
    seen = []
    for before, after in (([0, 0, 0], [0, 0]), ([7, 0, 3], [9, 0]), ([0, R // 3, 1], [R // 4, 5])):
        at = sum(before)
        counts = before + [1 + after[0], after[1]]
        off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)])).cuda()
        x, base, dy, dxb = rand(R, K), rand(R, N), rand(R, N), rand(R, K)
        for t, row in ((x, token), (base, above), (dy, behind), (dxb, under)):
            t[at] = row
        h, gh = torch.zeros(R, r, device="cuda"), torch.zeros(R, r, device="cuda")
        out = g.lora_apply(base, x, A, B, off, scaling=scal, h=h, R=R)
        dx, _, _ = g.lora_backward(dy, h, A, B, off, x=x, scaling=scal, dx_base=dxb, grad_h=gh, R=R)
        seen.append([t[at].clone() for t in (out, h, dx, gh)])
    for again in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(again, seen[0]))


def test_base_none_is_zeros():
    g = lib()
    p = Problem([5, 40], 16, 128, 64, scatter=False)
    out = torch.full_like(p.base, 9.0)
    g.lora_apply(None, p.x, p.A, p.B, p.offsets, out=out, **p.rows())
    want = g.lora_apply(torch.zeros_like(p.base), p.x, p.A, p.B, p.offsets, out=p.base.clone(), **p.rows())
    assert torch.equal(out, want)


def test_parts_of_the_backward():
    g = lib()
    p = Problem([30, 0, 3], 24, 160, 72)
    dy, h = torch.randn_like(p.base), torch.randn(p.R, 24, device="cuda")
    kw = dict(row_src=p.dest, **p.rows())
    dx, dA, dB = g.lora_backward(dy, h, p.A, p.B, p.offsets, x=p.x, **kw)
    gh = torch.empty(p.R, 24, device="cuda")
    dx2, none, dB2 = g.lora_backward(dy, h, p.A, p.B, p.offsets, grad_h=gh, **kw)
    assert none is None and torch.equal(dx2, dx) and torch.equal(dB2, dB)
    assert torch.equal(g.lora_grad_a(gh, p.offsets, x=p.x, row_token=p.tok), dA)
    q = g.quantize_act8(p.x)
    want = g.lora_backward(dy, h, p.A, p.B, p.offsets, act8=q, **kw)
    assert torch.equal(g.lora_grad_a(gh, p.offsets, act8=q, row_token=p.tok), want[1])
    none, dA3, dB3 = g.lora_backward(dy, h, p.A, p.B, p.offsets, x=p.x, want_dx=False, **kw)
    assert none is None and torch.equal(dA3, dA) and torch.equal(dB3, dB)


@pytest.mark.parametrize("r", [16, 72])
def test_checkpoint_of_any_size_reads_as_its_values(r):
    # every exponent bf16 has: the gradient from the codes is the gradient from their values, bit for bit
    g = lib()
    rng = np.random.default_rng(r)
    T, K = 50, 288
    x = rng.integers(0, 1 << 16, (T, K), dtype=np.uint16)
    e = np.clip(rng.integers(0, 250, (T, K // 32, 1)) - rng.integers(0, 9, (T, K // 32, 32)), 0, 249).reshape(T, K)
    x = torch.from_numpy(((x & 0x807F) | (e << 7).astype(np.uint16)).view(np.int16)).cuda().view(torch.bfloat16)
    q = g.quantize_act8(x)
    off = torch.tensor([0, 20, 20, T], device="cuda")
    gh = torch.randn(T, r, device="cuda") * 1e-3
    for dt in (torch.bfloat16, torch.float32):
        assert torch.equal(g.lora_grad_a(gh, off, act8=q, grad_dtype=dt),
                           g.lora_grad_a(gh, off, x=g.dequantize_act8(*q), grad_dtype=dt))


def test_no_rows():
    g = lib()
    p = Problem([0, 0, 0], 16, 64, 32)
    out = p.base.clone()
    g.lora_apply(p.base, p.x, p.A, p.B, p.offsets, row_dest=p.dest, out=out, **p.rows())
    assert torch.equal(out, p.base)
    h = torch.empty(0, 16, device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        dx, dA, dB = g.lora_backward(p.base, h, p.A, p.B, p.offsets, x=p.x, grad_dtype=dt, row_src=p.dest, **p.rows())
        assert dx.shape == (0, 64) and not dA.any() and not dB.any() and dA.dtype == dt
    # an upper bound with no row behind it
    p = Problem([0, 0, 0], 16, 64, 32, spare=20)
    out, hh = p.forward()
    assert torch.equal(out, p.base) and (hh == 5).all()
    p.check_backward()


def test_a_row_that_is_not_finite_stays_alone():
    for bad in (float("inf"), float("nan")):
        p = Problem([40, 3], 24, 128, 64, gather=False, scatter=False)
        clean, _ = p.forward()
        p.x[17, 5] = bad
        out, _ = p.forward()
        keep = torch.arange(43, device="cuda") != 17
        assert torch.equal(out[keep], clean[keep]) and not torch.isfinite(out[17]).any()
    # tokens that no row names, and adapters without rows, may hold anything
    p = Problem([3, 0, 4], 16, 64, 64)
    clean, _ = p.forward()
    named = torch.zeros(len(p.x), dtype=torch.bool, device="cuda")
    named[p.tok.long()] = True
    p.x[~named] = float("nan")
    p.A[1] = float("nan")
    p.B[1] = float("inf")
    assert torch.equal(p.forward()[0], clean)


def test_an_infinite_product_is_infinite():
    # h overflows to infinity in one rank: B's sign decides, nothing turns into NaN
    g = lib()
    x = torch.full((1, 64), 3e38, device="cuda").to(torch.bfloat16)
    A, B = torch.zeros(1, 16, 64, device="cuda"), torch.zeros(1, 8, 16, device="cuda")
    A[0, 0] = 2.0
    B[0, :, 0] = torch.tensor([1.0, -1.0] * 4)
    off = torch.tensor([0, 1], device="cuda")
    out = g.lora_apply(torch.zeros(1, 8, device="cuda").to(torch.bfloat16), x, A.bfloat16(), B.bfloat16(), off)
    assert out[0].tolist() == [float("inf"), float("-inf")] * 4


def test_fp16_product_past_the_types_range():
    # h = 256 * 300 does not fit in fp16; the output does
    x = torch.full((3, 256), 300.0, device="cuda").half()
    A = torch.ones(1, 8, 256, device="cuda").half()
    B = torch.full((1, 16, 8), 2.0 ** -6, device="cuda").half()
    off = torch.tensor([0, 3], device="cuda")
    out = lib().lora_apply(torch.zeros(3, 16, device="cuda").half(), x, A, B, off)
    assert (out == 9600.0).all()                        # 8 * 76800 / 64


def test_row_indices_out_of_range_are_left_out():
    p = Problem([6, 5], 16, 64, 48)
    ok, _ = p.forward()
    tok, dest = p.tok.clone(), p.dest.clone()
    p.tok[2], p.dest[7] = len(p.x), -1
    out, _ = p.forward()
    want = ok.clone()
    want[dest[7].long()] = p.base[dest[7].long()]
    want[dest[2].long()] = p.base[dest[2].long()]       # zeros on top
    assert torch.equal(out, want)


@pytest.mark.parametrize("what", ["decrease", "past", "first", "token", "dest", "weight"])
def test_checked_calls_refuse_bad_rows(what):
    g = lib()
    p = Problem([4, 3, 5], 16, 64, 48)
    if what == "decrease":
        p.offsets[1] = 9
    elif what == "past":
        p.offsets[3] = 13
    elif what == "first":
        p.offsets[0] = 1
    elif what == "token":
        p.tok[11] = len(p.x)
    elif what == "dest":
        p.dest[0] = -1
    else:
        p.w[3] = float("inf")
    out = p.base.clone()
    with pytest.raises(g.Gnf4Error) as e:
        g.lora_apply(p.base, p.x, p.A, p.B, p.offsets, row_dest=p.dest, out=out, flags=g.GNF4_CHECK, **p.rows())
    assert e.value.status == 5
    h = torch.zeros(12, 16, device="cuda")
    with pytest.raises(g.Gnf4Error):
        g.lora_backward(p.base, h, p.A, p.B, p.offsets, x=p.x, row_src=p.dest, flags=g.GNF4_CHECK, **p.rows())
    torch.cuda.synchronize()
    assert torch.equal(out, p.base)


def test_checked_calls_pass_good_rows():
    p = Problem([4, 0, 5], 16, 64, 48, spare=3)
    a, b = p.forward()[0], p.forward(flags=lib().GNF4_CHECK)[0]
    assert torch.equal(a, b)


def test_far_rows_and_adapters():
    # element offsets past 2^31 in base, out, A and dA
    g = lib()
    p = Problem([2, 3], 16, 64, 2048, far=1_050_000)
    p.dest[:5] = torch.tensor([1_050_000, 1_050_006, 3, 1_049_999, 1_050_009], dtype=torch.int32, device="cuda")
    rows = p.dest.long()
    near_base = p.base[rows].clone()
    small = g.lora_apply(near_base, p.x, p.A, p.B, p.offsets, **p.rows())
    y = g.lora_apply(p.base, p.x, p.A, p.B, p.offsets, row_dest=p.dest, **p.rows())
    assert torch.equal(y[rows], small)
    del p, y
    L, r, K = 2048, 128, 8200
    A = torch.zeros(L, r, K, dtype=torch.bfloat16, device="cuda")
    B = torch.zeros(L, 8, r, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    A[-1] = torch.randn(r, K, generator=gen, device="cuda") * K ** -0.5
    B[-1] = torch.randn(8, r, generator=gen, device="cuda")
    x = torch.randn(3, K, generator=gen, device="cuda").to(torch.bfloat16)
    off = torch.zeros(L + 1, dtype=torch.int64, device="cuda")
    off[-1] = 3
    base = torch.zeros(3, 8, dtype=torch.bfloat16, device="cuda")
    h = torch.empty(3, r, device="cuda")
    out = g.lora_apply(base.clone(), x, A, B, off, h=h)
    off1 = torch.tensor([0, 3], device="cuda")
    assert torch.equal(out, g.lora_apply(base.clone(), x, A[-1:].contiguous(), B[-1:].contiguous(), off1))
    dy = torch.randn(3, 8, generator=gen, device="cuda").to(torch.bfloat16)
    dx, dA, dB = g.lora_backward(dy, h, A, B, off, x=x)
    dx1, dA1, dB1 = g.lora_backward(dy, h, A[-1:].contiguous(), B[-1:].contiguous(), off1, x=x)
    assert torch.equal(dx, dx1) and torch.equal(dA[-1:], dA1) and torch.equal(dB[-1:], dB1)
    assert not dA[:-1].any() and not dB[:-1].any()


def test_far_rows_of_the_backward():
    # element offsets past 2^31 in x, its codes, grad_out and what follows from them
    g = lib()
    T, K, N, r, n = 1_048_600, 2080, 2056, 40, 300
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    A, B, h = rand(2, r, K), rand(2, N, r), torch.randn(n, r, generator=gen, device="cuda")
    off = torch.tensor([0, 130, n], device="cuda")
    rows = torch.randperm(n, generator=gen, device="cuda")
    far = torch.cat([torch.arange(4, device="cuda"), T - n + torch.arange(4, n, device="cuda")])[rows].to(torch.int32)
    x, dy = rand(n, K), rand(n, N)
    q = g.quantize_act8(x)
    big_x, big_dy = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    big_x[far.long()], big_dy[far.long()] = x, dy
    for dt in (torch.bfloat16, torch.float32):
        want = g.lora_backward(dy, h, A, B, off, x=x, grad_dtype=dt)
        got = g.lora_backward(big_dy, h, A, B, off, x=big_x, row_token=far, row_src=far, grad_dtype=dt)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    del big_x
    codes, scales = torch.zeros(T, K, dtype=torch.int8, device="cuda"), torch.zeros(T, K // 32, dtype=torch.uint8, device="cuda")
    codes[far.long()], scales[far.long()] = q
    for rank in (r, 16):
        a, b, hh = A[:, :rank].contiguous(), B[:, :, :rank].contiguous(), h[:, :rank].contiguous()
        want = g.lora_backward(dy, hh, a, b, off, act8=q)
        got = g.lora_backward(big_dy, hh, a, b, off, act8=(codes, scales), row_token=far, row_src=far)
        assert all(torch.equal(u, v) for u, v in zip(got, want))


def test_rows_far_into_h():
    # more than 2^31 elements of h and grad_h; the last rows belong to an adapter of their own
    g = lib()
    r, R, last = 72, (1 << 25) - 700, 50
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    A, B, x, dy = rand(2, r, 8), rand(2, 8, r), rand(R, 8), rand(R, 8)
    off = torch.tensor([0, R - last, R], device="cuda")
    h, gh = torch.empty(R, r, device="cuda"), torch.empty(R, r, device="cuda")
    out = g.lora_apply(torch.zeros_like(dy), x, A, B, off, h=h)
    dx, dA, dB = g.lora_backward(dy, h, A, B, off, x=x, grad_h=gh, grad_dtype=torch.float32)
    tail = slice(R - last, R)
    o = np.array([0, last])
    want, wh, bound = LO.lora_apply_f64(np.zeros((last, 8)), f64(x[tail]), f64(A[1:]), f64(B[1:]), o)
    near(h[tail], wh, np.abs(f64(x[tail])) @ np.abs(f64(A[1])).T, 8 + 32, 3, "h")
    near(out[tail], want, bound, 8 + r + 32, 2, "out", np.zeros((last, 8)), r)
    w = LO.lora_backward_f64(f64(dy[tail]), f64(x[tail]), f64(h[tail]), f64(A[1:]), f64(B[1:]), o)
    near(gh[tail], w["grad_h"], w["grad_h_bound"], 8 + 32, 3, "grad_h")
    near(dx[tail], w["dx"], w["dx_bound"], 8 + r + 32, 2, "dx", np.zeros((last, 8)), r)
    near(dA[1:], w["dA"], w["dA_bound"], 8 + last + 32, 3, "dA")
    near(dB[1:], w["dB"], w["dB_bound"], last + 32, 3, "dB")


@pytest.mark.parametrize("r", [8, 40])
@pytest.mark.parametrize("R", [3, 2400])
def test_largest_axes(r, R):
    # K or N at their limit; entries of -1, 0 and 1 whose sums fp32 holds exactly
    g = lib()
    big, gen = 1 << 24, torch.Generator(device="cuda").manual_seed(r)
    few = lambda *s: torch.randint(-1, 2, s, generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16)  # noqa: E731
    off = torch.tensor([0, R], device="cuda")
    tok = torch.arange(R, device="cuda", dtype=torch.int32) % 3
    long_, short = few(3, big), few(3, 8)
    # forward down the long axis, and the gradient of B along it
    A, B = few(1, r, big), few(1, 8, r)
    h = torch.empty(R, r, device="cuda")
    out = g.lora_apply(torch.zeros(R, 8, device="cuda").bfloat16(), long_, A, B, off, row_token=tok, h=h)
    want = sum(a.double() @ b.double().T for a, b in zip(long_.split(1 << 21, 1), A[0].split(1 << 21, 1)))
    assert torch.equal(h.double(), want[tok.long()])
    assert torch.equal(out, (want @ B[0].double().T)[tok.long()].to(torch.bfloat16))
    ones = torch.ones(R, r, device="cuda")
    dB = g.lora_backward(long_, ones, few(1, r, 8), few(1, big, r), off, x=short, row_token=tok, row_src=tok, want_dx=False)[2]
    times = torch.bincount(tok.long(), minlength=3).double()
    assert torch.equal(dB[0], (times @ long_.double())[:, None].expand(big, r).to(torch.bfloat16))
    del dB
    # out along the long axis
    if R == 3:
        A, B = few(1, r, 8), few(1, big, r)
        want = (long_.double() + (short.double() @ A[0].double().T) @ B[0].double().T).to(torch.bfloat16)
        assert torch.equal(g.lora_apply(long_, short, A, B, off, row_token=tok), want)


def test_totals_beside_other_tensor_memory_kernels():
    # gradient sums with totals in tensor memory, larger ranks and projections, on three streams and captured
    g = lib()
    Wd, Sd, _, _ = build_stack("nf4", 4, 256, 512)
    x = torch.randn(4096, 512, device="cuda").to(torch.bfloat16)
    off = torch.tensor([0, 1000, 1000, 3000, 4096], device="cuda")
    want_y = g.grouped_gemm("nf4", x, Wd, Sd, off, R=4096)
    calls = []
    for r, counts in ((16, [9000, 5, 700] + [30] * 60), (32, [20000]), (64, [9000, 40]), (128, [5000, 5000])):
        p = Problem(counts, r, 520, 776, seed=r)
        dy, h = torch.randn_like(p.base), torch.randn(p.R, r, device="cuda")
        calls.append(lambda p=p, dy=dy, h=h: g.lora_backward(dy, h, p.A, p.B, p.offsets, x=p.x, row_src=p.dest,
                                                             grad_dtype=torch.float32, **p.rows()))
    want = [call() for call in calls]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = [call() for call in calls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            ys = [g.grouped_gemm("nf4", x, Wd, Sd, off, R=4096) for _ in range(4)]
        with torch.cuda.stream(streams[1]):
            got = [call() for call in reversed(calls)][::-1]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want_y) for y in ys)
        for outs in (got, captured):
            assert all(torch.equal(u, v) for a, b in zip(outs, want) for u, v in zip(a, b))
    g.device_status()


def test_captured_calls_replay_and_share_nothing():
    g = lib()
    probs = [Problem([9, 0, 30], 16, 128, 96, seed=i) for i in range(2)]
    graphs, outs = [], []
    for p in probs:
        p.dy, p.h = torch.randn_like(p.base), torch.randn(p.R, 16, device="cuda")

        def step(p=p):
            y = g.lora_apply(p.base, p.x, p.A, p.B, p.offsets, row_dest=p.dest, out=p.base.clone(), **p.rows())
            return (y, *g.lora_backward(p.dy, p.h, p.A, p.B, p.offsets, x=p.x, row_src=p.dest, **p.rows()))

        p.step = step
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in probs]
    for turn in range(3):
        for p in probs:
            p.x.copy_(torch.randn_like(p.x))
            p.dy.copy_(torch.randn_like(p.dy))
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):             # both at once
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for p, out in zip(probs, outs):
            assert all(torch.equal(a, b) for a, b in zip(out, p.step()))


@pytest.mark.parametrize("r", [64, 128])
def test_large_ranks_captured_beside_projections_on_another_stream(r):
    # the gradient sums and the projections both keep accumulators in tensor memory
    g = lib()
    p = Problem([700, 0, 90, 1500], r, 520, 776, seed=r)
    many = Problem([1400 if i == 3 else i % 41 for i in range(100)], r, 264, 200, seed=r)
    Wd, Sd, _, _ = build_stack("nf4", 4, 256, 512)
    x = torch.randn(4096, 512, device="cuda").to(torch.bfloat16)
    off = torch.tensor([0, 1000, 1000, 3000, 4096], device="cuda")
    want_y = g.grouped_gemm("nf4", x, Wd, Sd, off, R=4096)
    steps = []
    for q in (p, many):
        dy, h = torch.randn_like(q.base), torch.randn(q.R, r, device="cuda")
        steps.append(lambda q=q, dy=dy, h=h: g.lora_backward(dy, h, q.A, q.B, q.offsets, x=q.x, row_src=q.dest, **q.rows()))
    want = [step() for step in steps]
    torch.cuda.synchronize()
    graph, outs = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        for step in steps:
            outs.append(step())
    side = torch.cuda.Stream()
    for turn in range(3):
        for out in outs:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            ys = [g.grouped_gemm("nf4", x, Wd, Sd, off, R=4096) for _ in range(4)]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want_y) for y in ys)
        for got, ref in zip(outs, want):
            assert all(torch.equal(u, v) for u, v in zip(got, ref))
    g.device_status()


@pytest.mark.parametrize("r", [40, 64, 128])
@pytest.mark.parametrize("act8", [False, True])
def test_large_ranks_of_few_and_many_columns_and_rows(r, act8):
    # stages of 32 rows: one row, a last one short, eight and more of them, a cluster's unequal shares
    for counts, K, N in (([1], 32, 8), ([32, 33, 31], 288, 264), ([257, 0, 300], 96, 520), ([1029], 544, 128), ([4100, 7], 64, 72)):
        p = Problem(counts, r, K, N, seed=r + len(counts), spare=2)
        p.check_backward(torch.float32, act8)
        p.check_backward(torch.bfloat16, act8)


def test_large_rank_rows_that_are_not_finite_stay_in_their_adapter():
    g = lib()
    for r in (48, 128):
        p = Problem([50, 40, 3], r, 96, 64, gather=False, scatter=False)
        dy, h = torch.randn_like(p.base), torch.randn(p.R, r, device="cuda")
        clean = g.lora_backward(dy, h, p.A, p.B, p.offsets, x=p.x, grad_dtype=torch.float32, **p.rows())
        h[60, 3], p.x[60, 7] = float("nan"), float("inf")
        p.s[1] = float("inf")
        got = g.lora_backward(dy, h, p.A, p.B, p.offsets, x=p.x, grad_dtype=torch.float32, **p.rows())
        for u, v in zip(got[1:], clean[1:]):
            assert torch.equal(u[[0, 2]], v[[0, 2]])
        assert not torch.isfinite(got[2][1, :, 3]).any() and not torch.isfinite(got[1][1, :, 7]).any()


def test_other_stream():
    g = lib()
    p = Problem([9, 0, 300], 32, 512, 640)
    want, h = p.forward()
    s = torch.cuda.Stream()
    out = p.base.clone()
    gh = torch.empty(p.R, 32, device="cuda")
    torch.cuda.synchronize()
    g.lora_apply(p.base, p.x, p.A, p.B, p.offsets, row_dest=p.dest, out=out, stream=s, **p.rows())
    got = g.lora_backward(p.base, h, p.A, p.B, p.offsets, x=p.x, row_src=p.dest, grad_h=gh, stream=s, **p.rows())
    s.synchronize()
    ref = g.lora_backward(p.base, h, p.A, p.B, p.offsets, x=p.x, row_src=p.dest, **p.rows())
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("r,counts", [(16, [9, 0, 30]), (32, [40] * 100), (64, [2600, 1]), (40, [3]), (128, [50, 0, 700])])
def test_waits_that_give_up_are_reported_and_the_next_call_is_right(r, counts):
    """GNF4_TEST_STALL: the streaming kernel issues no copy and the gradient sums of ranks above 32
    no matrix product, so every first wait gives up after a short limit with nothing in flight.
    gnf4_device_status reports it once, and rows that do not exist stay as they were."""
    g = lib()
    p = Problem(counts, r, 136, 200, seed=r, spare=4)
    h, gh = torch.randn(p.R + 4, r, device="cuda"), torch.full((p.R + 4, r), 5.0, device="cuda")
    dy, dx = torch.randn_like(p.base), torch.full((p.R + 4, 136), 3.0, device="cuda").to(torch.bfloat16)

    def given_up(call):
        call()
        with pytest.raises(g.Gnf4Error) as e:
            g.device_status()
        assert e.value.status == 5 and "adapters" in str(e.value)
        g.device_status()                                # the record was cleared

    if r <= 64:
        out = p.base.clone()
        given_up(lambda: g.lora_apply(p.base, p.x, p.A, p.B, p.offsets, row_dest=p.dest, out=out, flags=g.GNF4_TEST_STALL, **p.rows()))
        assert torch.equal(out, p.base)                  # the sums were skipped
    given_up(lambda: g.lora_backward(dy, h, p.A, p.B, p.offsets, x=p.x, row_src=p.dest, dx=dx, grad_h=gh,
                                     flags=g.GNF4_TEST_STALL, **p.rows()))
    assert (dx[p.R:] == 3).all() and (gh[p.R:] == 5).all()
    if r > 32:
        given_up(lambda: g.lora_grad_a(h, p.offsets, x=p.x, row_token=p.tok, flags=g.GNF4_TEST_STALL))
    p.check_forward()
    p.check_backward(torch.float32)
    g.device_status()


def test_requests_through_routing_metadata():
    """Adapter ids of a batch of tokens, some without one, on top of one shared 4-bit projection."""
    g = lib()
    T, K, N, L, r = 37, 256, 128, 5, 16
    Wd, Sd, Wh, Sh = build_stack("nf4", 1, N, K)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, K, generator=gen, device="cuda").to(torch.bfloat16)
    A = (torch.randn(L, r, K, generator=gen, device="cuda") / 16).to(torch.bfloat16)
    B = torch.randn(L, N, r, generator=gen, device="cuda").to(torch.bfloat16)
    ids = torch.randint(-1, L, (T, 1), generator=gen, device="cuda", dtype=torch.int32)
    y = g.grouped_gemm("nf4", x, Wd, Sd, torch.tensor([0, T], device="cuda"), R=T)
    base = y.clone()
    off, tok, _, dst = g.routing_metadata(ids, None, L)
    g.lora_apply(y, x, A, B, off, row_token=tok, row_dest=dst, R=T)
    torch.cuda.synchronize()
    want, bound = f64(base), np.zeros((T, N))
    for i, e in enumerate(ids[:, 0].tolist()):
        if e >= 0:
            h = f64(A[e]) @ f64(x[i])
            want[i] += f64(B[e]) @ h
            bound[i] = (np.abs(f64(A[e])) @ np.abs(f64(x[i]))).max() * np.abs(f64(B[e])).sum(axis=1)
    near(y, want, bound, K + r + 32, 2, "y", f64(base), r)
    gone = ids[:, 0] < 0
    assert gone.any() and torch.equal(y[gone], base[gone])


def test_expert_layer_trains_its_adapters():
    """One MoE layer, forward and backward, as a trainer runs it: routing, gate_up with adapters,
    SwiGLU with an 8-bit checkpoint, down with adapters, combine; then the gradients of both
    pairs of adapters and of the tokens, against the oracles' chain on the same rounded values."""
    from oracle import dgrad as D
    g = lib()
    T, k, E, H, I, r = 45, 2, 6, 192, 128, 16
    Wd, Sd, Wh, Sh = build_stack("nf4", E, 2 * I, H, seed=1)
    Vd, Ud, Vh, Uh = build_stack("mxfp4", E, H, I, seed=2)
    gen = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).to(torch.bfloat16)  # noqa: E731
    x, dout = rand(T, H), rand(T, H)
    A1, B1, A2, B2 = rand(E, r, H, scale=0.1), rand(E, 2 * I, r, scale=0.05), rand(E, r, I, scale=0.1), rand(E, H, r, scale=0.05)
    s1, s2 = torch.rand(E, generator=gen, device="cuda") + 0.5, torch.rand(E, generator=gen, device="cuda") + 0.5
    ids = torch.stack([torch.randperm(E, generator=gen, device="cuda")[:k] for _ in range(T)]).to(torch.int32)
    wts = torch.rand(T, k, generator=gen, device="cuda")
    R = T * k

    # forward
    off, tok, w, dst = g.routing_metadata(ids, wts, E)
    h1, h2 = torch.empty(R, r, device="cuda"), torch.empty(R, r, device="cuda")
    gu0 = g.grouped_gemm("nf4", x, Wd, Sd, off, row_token=tok)
    gu = g.lora_apply(gu0, x, A1, B1, off, row_token=tok, scaling=s1, h=h1, out=gu0.clone())
    act, codes, scales = g.swiglu_act8(gu)
    y0 = g.grouped_gemm("mxfp4", act, Vd, Ud, off, row_weight=w, row_dest=dst, T_out=R)
    y = g.lora_apply(y0, act, A2, B2, off, row_weight=w, row_dest=dst, scaling=s2, h=h2, out=y0.clone())
    out = g.combine_topk(y, T, k)
    # backward: a token's slots all get its gradient, so rows read it through their token
    d_act0 = g.dgrad("mxfp4", dout, Vd, Ud, off, row_src=tok, row_weight=w)
    gh2 = torch.empty(R, r, device="cuda")
    d_act, _, dB2 = g.lora_backward(dout, h2, A2, B2, off, row_src=tok, row_weight=w, scaling=s2, dx_base=d_act0,
                                    dx=torch.empty_like(d_act0), grad_h=gh2)
    d_gu, act_again = g.swiglu_backward(d_act, act8=(codes, scales), rebuild=True)
    dA2 = g.lora_grad_a(gh2, off, x=act_again)
    dx0 = g.dgrad("nf4", d_gu, Wd, Sd, off, R=R)
    xq = g.quantize_act8(x)
    dx, dA1, dB1 = g.lora_backward(d_gu, h1, A1, B1, off, act8=xq, row_token=tok, scaling=s1, dx_base=dx0,
                                   dx=torch.empty_like(dx0))
    slot_row = torch.empty(R, dtype=torch.int32, device="cuda")
    slot_row[dst.long()] = torch.arange(R, dtype=torch.int32, device="cuda")
    d_x = g.combine_topk(dx, T, k, row_of_slot=slot_row)
    g.device_status()

    o, tk, ds, ww = (v.cpu().numpy() for v in (off, tok, dst, w))
    want, wh, b = LO.lora_apply_f64(f64(gu0), f64(x), f64(A1), f64(B1), o, row_token=tk, scaling=f64(s1))
    near(gu, want, b, H + r + 32, 2, "gate_up", f64(gu0), r)
    want, _, b = LO.lora_apply_f64(f64(y0), f64(act), f64(A2), f64(B2), o, row_weight=ww, row_dest=ds, scaling=f64(s2))
    near(y, want, b, I + r + 32, 2, "down", f64(y0), r)
    xb, gb = x.view(torch.int16).cpu().numpy().view(np.uint16), dout.view(torch.int16).cpu().numpy().view(np.uint16)
    # against the exact layer the rounded intermediate rows leave a few bf16 steps of each row's largest value
    exact_gu = O.grouped_rows_f64("nf4", xb, Wh, Sh, o, tk, None, H, np.arange(R))
    exact_gu, _, _ = LO.lora_apply_f64(exact_gu, f64(x), f64(A1), f64(B1), o, row_token=tk, scaling=f64(s1))
    assert np.all(np.abs(f64(gu) - exact_gu).max(axis=1) <= 2e-2 * np.abs(exact_gu).max(axis=1))
    bw = LO.lora_backward_f64(f64(dout), f64(act_again), f64(h2), f64(A2), f64(B2), o, row_src=tk, row_weight=ww,
                              scaling=f64(s2), dx_base=f64(d_act0))
    m = int(np.diff(o).max())
    near(d_act, bw["dx"], bw["dx_bound"], H + r + 32, 2, "d_act", f64(d_act0), r)
    near(dA2, bw["dA"], bw["dA_bound"], H + m + 32, 2, "dA of down")
    near(dB2, bw["dB"], bw["dB_bound"], m + 32, 2, "dB of down")
    gu8 = A8.values_act8(codes.cpu().numpy(), scales.cpu().numpy())
    sw = A8.swiglu_backward_f64(f64(d_act), gu8)
    assert np.all(np.abs(f64(d_gu) - sw) <= 2.0 ** -8 * np.abs(sw) + 2.0 ** -15 * A8.swiglu_backward_bound(f64(d_act), gu8) + 2.0 ** -126)
    want = GL.swiglu_rows_f64(O.bf16_bits(gu8))
    assert np.all(np.abs(f64(act_again) - want) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(want) + 2.0 ** -118)
    bw = LO.lora_backward_f64(f64(d_gu), A8.values_act8(xq[0].cpu().numpy(), xq[1].cpu().numpy()), f64(h1), f64(A1),
                              f64(B1), o, row_token=tk, scaling=f64(s1), dx_base=f64(dx0))
    near(dx, bw["dx"], bw["dx_bound"], 2 * I + r + 32, 2, "dx", f64(dx0), r)
    near(dA1, bw["dA"], bw["dA_bound"], 2 * I + m + 32, 2, "dA of gate_up")
    near(dB1, bw["dB"], bw["dB_bound"], m + 32, 2, "dB of gate_up")
    ref = D.dgrad_rows_f64("mxfp4", gb, Vh, Uh, o, tk, ww, np.arange(R))
    assert np.all(np.abs(f64(d_act0) - ref).max(axis=1) <= 2e-2 * np.abs(ref).max(axis=1))
    sums = np.zeros((T, H))
    np.add.at(sums, tk, f64(dx))
    top = np.zeros((T, H))
    np.add.at(top, tk, np.abs(f64(dx)))
    assert np.all(np.abs(f64(d_x) - sums) <= 2.0 ** -8 * np.abs(sums) + 2.0 ** -21 * top)
    assert torch.isfinite(out).all()
