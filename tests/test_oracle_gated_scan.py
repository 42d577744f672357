"""Pins of the gated-recurrence oracle (oracle/gated_scan.py) against things other than itself: a closed form, finite
differences of its forward, and the defining properties of the 8-bit checkpoint's values; planted mistakes are caught."""
import numpy as np
import pytest

import oracle as O
from oracle import gated_scan as M


def _inputs(n, E, seed):
    rng = np.random.default_rng(seed)
    d = {k: rng.standard_normal((n, E)) for k in ("x", "r", "g")}
    d["lam"] = rng.uniform(-6.0, 1.0, E)
    d["h0"] = rng.standard_normal(E)
    return d, rng.standard_normal((n, E)), rng.standard_normal(E)


def test_closed_form():
    """h_k is the sum of every earlier input times the product of the decays after it."""
    d, _, _ = _inputs(9, 5, 0)
    h = O.gated_scan_forward(**d)
    sr, sg = 1 / (1 + np.exp(-d["r"])), 1 / (1 + np.exp(-d["g"]))
    a = (1 + np.exp(d["lam"])) ** (-8 * sr)                # exp(-8 softplus(lam) sr)
    b = np.sqrt(1 - a * a) * sg * d["x"]
    for k in range(9):
        want = np.prod(a[:k + 1], axis=0) * d["h0"] + sum(np.prod(a[j + 1:k + 1], axis=0) * b[j] for j in range(k + 1))
        np.testing.assert_allclose(h[k], want, rtol=1e-12, atol=1e-14)


def _grads(d, dy, dh):
    return dict(zip(("x", "r", "g", "lam", "h0"), O.gated_scan_backward(**d, dy=dy, dh_last=dh)))


def _worst(d, dy, dh):
    """Largest difference between the gradient and central differences of the forward."""
    got, worst, eps = _grads(d, dy, dh), 0.0, 1e-6

    def loss():
        h = O.gated_scan_forward(**d)
        return float(np.sum(dy * h) + np.sum(dh * h[-1]))

    for name, t in d.items():
        for at in np.ndindex(t.shape):
            old = t[at]
            t[at] = old + eps
            up = loss()
            t[at] = old - eps
            down = loss()
            t[at] = old
            worst = max(worst, abs((up - down) / (2 * eps) - got[name][at]))
    return worst


def test_gradient_against_differences():
    # eps^2 times a third derivative of order one, and 1e-15 / eps of rounding
    assert _worst(*_inputs(7, 3, 1)) < 1e-7


@pytest.mark.parametrize("mistake", ["beta", "saturation", "carry"])
def test_differences_catch_mistakes(monkeypatch, mistake):
    real = O.gated_scan_backward

    def wrong(x, r, g, lam, h0, dy, dh_last, starts=None):
        dx, dr, dg, dlam, dh0 = real(x, r, g, lam, h0, dy, dh_last, starts)
        a, beta, sr, sg, la = M.gated_coefficients(r, g, lam)
        if mistake == "beta":                               # the path through sqrt(1 - a^2) forgotten
            dr = dr + dx * x * a * a / beta / beta * la * (1 - sr)
        elif mistake == "saturation":
            dg = dg / (1 - sg)
        else:
            dh0 = dh0 / a[0]
        return dx, dr, dg, dlam, dh0

    monkeypatch.setattr(O, "gated_scan_backward", wrong)
    assert _worst(*_inputs(7, 3, 1)) > 1e-4


def test_tiles_from_their_own_starts():
    d, dy, dh = _inputs(150, 2, 2)
    h = O.gated_scan_forward(**d)
    starts = np.concatenate([d["h0"][None], h])[0:150:64]
    for u, v in zip(O.gated_scan_backward(**d, dy=dy, dh_last=dh), O.gated_scan_backward(**d, dy=dy, dh_last=dh, starts=starts)):
        np.testing.assert_array_equal(u, v)


def test_closed_gate_passes_the_state():
    d, dy, dh = _inputs(4, 3, 3)
    d["r"][:] = -np.inf
    assert np.array_equal(O.gated_scan_forward(**d), np.tile(d["h0"], (4, 1)))
    g = _grads(d, dy, dh)
    assert all(np.all(g[k] == 0) for k in ("x", "r", "g", "lam"))
    np.testing.assert_allclose(g["h0"], dh + dy.sum(0))


def test_act8_values():
    rng = np.random.default_rng(4)
    v = rng.standard_normal((50, 150)) * np.exp(rng.uniform(-30, 30, (50, 1)))
    v[0] = 0.0
    v[1, :64] = 448.0
    v[2, 3] = 448.0 * 2 ** 5 * (1 + 1e-9)
    q = O.act8_values(v)
    np.testing.assert_array_equal(O.act8_values(q), q)                        # idempotent
    for c in (0, 64, 128):
        p, u = v[:, c:c + 64], q[:, c:c + 64]
        top = np.abs(p).max(1, keepdims=True)
        # half a step of 4 significant bits, or half the smallest step of the group's scale (at most top / 224 * 2^-9)
        assert np.all(np.abs(u - p) <= np.maximum(np.abs(p) * 2.0 ** -4, top / 224 * 2.0 ** -10))
    np.testing.assert_array_equal(q[1, :64], 448.0)
    e = np.array([[1.0, -0.0625, 1.875, 448.0, np.inf, -np.inf, np.nan, 0.0, 17.0, 19.0]])
    np.testing.assert_array_equal(O.act8_values(e), [[1.0, -0.0625, 1.875, 448.0, np.nan, np.nan, np.nan, 0.0, 16.0, 20.0]])


def test_act8_values_of_the_largest_numbers():
    """Every finite fp32 number comes back as a finite one, and next to the border by e4m3's own steps."""
    unit = 2.0 ** 120
    v = np.array([[float(np.finfo(np.float32).max), -248 * unit, 248 * unit * (1 - 2.0 ** -24), 233 * unit, 232 * unit]])
    np.testing.assert_array_equal(O.act8_values(v) / unit, [[240, -240, 240, 240, 224]])
    assert np.all(np.isfinite(O.act8_values(v).astype(np.float32)))
