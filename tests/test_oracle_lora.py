"""Pins of the adapter oracle: hand-computed rows, and every gradient against differences."""
import numpy as np

from oracle import lora as LO


def problem(seed=0):
    rng = np.random.default_rng(seed)
    L, r, K, N, T = 3, 2, 5, 4, 6
    offsets = np.array([0, 2, 2, 5])                    # adapter 1 has no row
    return dict(base=rng.normal(size=(7, N)), x=rng.normal(size=(T, K)), A=rng.normal(size=(L, r, K)),
                B=rng.normal(size=(L, N, r)), offsets=offsets, row_token=np.array([3, 0, 5, 3, 1]),
                row_weight=rng.normal(size=5), row_dest=np.array([6, 1, 0, 4, 2]), scaling=rng.normal(size=L))


def test_rows_by_hand():
    p = problem()
    out, h, _ = LO.lora_apply_f64(**p)
    for r, e in ((0, 0), (1, 0), (2, 2), (3, 2), (4, 2)):
        x = p["x"][p["row_token"][r]]
        hand = [sum(p["A"][e, j, k] * x[k] for k in range(5)) for j in range(2)]
        np.testing.assert_allclose(h[r], hand, rtol=1e-12)
        d = p["row_dest"][r]
        for n in range(4):
            v = sum(p["B"][e, n, j] * hand[j] for j in range(2)) * p["scaling"][e] * p["row_weight"][r]
            np.testing.assert_allclose(out[d, n], p["base"][d, n] + v, rtol=1e-12)
    assert np.array_equal(out[[3, 5]], p["base"][[3, 5]])       # rows that nothing names


def test_gradients_are_difference_quotients():
    p = problem(1)
    rng = np.random.default_rng(2)
    dy = rng.normal(size=p["base"].shape)

    def loss(**kw):
        return float((dy * LO.lora_apply_f64(**{**p, **kw})[0]).sum())

    _, h, _ = LO.lora_apply_f64(**p)
    g = LO.lora_backward_f64(dy, p["x"], h, p["A"], p["B"], p["offsets"], p["row_token"], p["row_weight"],
                             p["row_dest"], p["scaling"])
    # the gradient of a token is the sum of its routed rows'
    dx = np.zeros_like(p["x"])
    np.add.at(dx, p["row_token"], g["dx"])
    for name, got in (("x", dx), ("A", g["dA"]), ("B", g["dB"])):
        for i in np.ndindex(got.shape):
            plus, minus = p[name].copy(), p[name].copy()
            plus[i] += 0.5
            minus[i] -= 0.5
            # the loss is linear in each of the three, so the quotient is exact at any step
            np.testing.assert_allclose(got[i], loss(**{name: plus}) - loss(**{name: minus}), atol=1e-12)
    assert not g["dA"][1].any() and not g["dB"][1].any()
