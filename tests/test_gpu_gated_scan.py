"""The gated linear recurrence (r2l_gated_scan, its training forward and its gradient) on the GPU against the float64
oracle.

Tolerances.  u = 2^-24.  One position multiplies the state by a rounded exp (3u, with its error in the argument below)
and adds (1u), so after n positions a state is off by at most 4nu of H, the largest state that inputs of one sign would
reach; a relative error of 16u in log a (sigmoid, softplus, their product) moves a product of decays e^-s by
16u s e^-s <= 16u, and an input beta sigmoid(g) x is off by at most 32u: (4n + 64)u H in all.  The same holds for the
adjoint with dy.  A product of the two is off by twice that and what its factors add, (8n + 256)u of the product of the
bounds.  A sum of N such terms adds Nu of the sum of their bounds.  A sigmoid(r) below 2^-126 may come out as 0: log a is
then off by up to 8 softplus(lam) 2^-126 and beta, sqrt(-2 log a) there, by the square root of twice that, under 2^-58 for
softplus(lam) <= 64; beta, and the sqrt(-log a / 2) that dr and dlam have of it, enter once, times x, G or both.
bf16 results add half a step, 2^-8 of the value (where an intermediate's error moves it over a rounding border, that error is in the bound already)."""
import numpy as np
import pytest
import torch

import oracle as O
from reverse_selective_ssm_b200 import binding as bd
from reverse_selective_ssm_b200 import synthetic as S

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FLUSH = 2.0 ** -58
TILE = bd.GATED_TILE
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bd.load()


def make(B, L, E, dtype, seed, lens=None, gate_std=1.0):
    """CPU tensors of one problem; memories of 10 to 1000 positions at an open gate."""
    gen = torch.Generator().manual_seed(seed)

    def n(*shape, std=1.0):
        return torch.randn(shape, generator=gen) * std

    sp = -torch.log(0.9 + 0.099 * torch.rand(E, generator=gen, dtype=torch.float64)) / 8
    d = {"x": n(B * L, E).to(dtype), "r": n(B * L, E, std=gate_std).to(dtype), "g": n(B * L, E, std=gate_std).to(dtype),
         "lam": (sp + torch.log(-torch.expm1(-sp))).float(), "h0": n(B, E, std=0.5), "dy": n(B * L, E).to(dtype),
         "dh_last": n(B, E)}
    d["lens"] = [L] * B if lens is None else lens
    return d


def poison(d, L):
    """NaN in every row past a sequence's length: those rows are not read."""
    for b, n in enumerate(d["lens"]):
        for k in ("x", "r", "g", "dy"):
            d[k][b * L + n:(b + 1) * L] = float("nan")


def rows(d, key, b, L, forward):
    """Sequence b's valid rows in scan order, float64."""
    v = S.to_f64(d[key][b * L: b * L + d["lens"][b]])
    return v if forward else v[::-1].copy()


def lengths_tensor(d, L):
    return None if all(n == L for n in d["lens"]) else torch.tensor(d["lens"], dtype=torch.int32, device="cuda")


def half_step(dtype, v):
    return np.abs(v) * 2.0 ** -8 if dtype == BF16 else 0.0


def bounded(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    bad = np.nan_to_num(np.abs(got - want) - tol, nan=-1.0)
    worst = float(bad.max()) if bad.size else -1.0
    assert worst <= 0, f"{what}: off by {worst:.3e} more than the bound at {np.unravel_index(bad.argmax(), bad.shape)}"


def top(v):
    return np.abs(v).max(axis=0, initial=0.0)


def oracle_forward(d, b, L, forward, keys=("x", "r", "g")):
    x, r, g = (rows(d, k, b, L, forward) for k in keys)
    lam, h0 = S.to_f64(d["lam"]), S.to_f64(d["h0"][b])
    h = O.gated_scan_forward(x, r, g, lam, h0)
    H = np.maximum(O.gated_scan_forward(np.abs(x), r, g, lam, np.abs(h0)).max(axis=0, initial=0.0), np.abs(h0))
    return h, H


def check_forward(d, y, h_last, B, L, forward, y_before=None):
    dtype = d["x"].dtype
    y = S.to_f64(y.cpu())
    for b in range(B):
        n = d["lens"][b]
        h, H = oracle_forward(d, b, L, forward)
        tol = (4 * n + 64) * U * H + n * FLUSH * top(rows(d, "x", b, L, forward)) + 1e-37
        got = y[b * L: b * L + n]
        bounded(got if forward else got[::-1], h, tol * 1.01 + half_step(dtype, h), f"y of sequence {b}")
        bounded(S.to_f64(h_last[b].cpu()), h[-1] if n else S.to_f64(d["h0"][b]), tol if n else 0.0, f"h_last of {b}")
        if y_before is not None:
            rest = S.to_f64(y_before[b * L + n:(b + 1) * L])
            assert np.array_equal(y[b * L + n:(b + 1) * L], rest), "rows past the length were written"


def dev(d):
    return {k: v.cuda() for k, v in d.items() if torch.is_tensor(v)}


def flags_of(forward, act8=False):
    return (bd.R2L_FLAG_FORWARD_SCAN if forward else 0) | (bd.R2L_FLAG_ACT8 if act8 else 0)


# lengths around the tile of 64 and the sub-tiles of a power of two, widths around a vector and a group of 64
SHAPES = [
    # B, L, E, lens
    (1, 1, 1, None), (3, 1, 64, [1, 0, 1]), (2, 2, 7, None), (2, 15, 130, None), (1, 16, 64, None), (1, 17, 65, None),
    (3, 63, 96, [63, 1, 0]), (2, 64, 128, None), (2, 65, 63, [64, 65]), (4, 130, 72, [0, 127, 128, 129]),
    (2, 257, 200, [200, 257]), (1, 777, 515, None), (9, 33, 24, [33, 32, 31, 17, 16, 15, 2, 1, 0]), (300, 5, 8, None),
    (2, 1300, 64, None), (1, 3000, 192, None),
    # sequences of all lengths shared by a cluster, blocks of 8 warps by themselves, and threads that walk
    (3, 1500, 64, [0, 1500, 700]), (4, 600, 40, [600, 513, 1, 64]), (3, 1100, 2100, [1100, 0, 1025]),
    (640, 12, 6, [b % 13 for b in range(640)]),
]


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("forward", [False, True], ids=["r2l", "l2r"])
@pytest.mark.parametrize("B,L,E,lens", SHAPES)
def test_forward(B, L, E, lens, forward, dtype):
    d = make(B, L, E, dtype, seed=B + 7 * L + E, lens=lens)
    poison(d, L)
    c = dev(d)
    y0 = torch.full((B * L, E), 3.0, dtype=dtype, device="cuda")
    y, h = bd.gated_scan(c["x"], c["r"], c["g"], c["lam"], bd.gated_dims(E, dtype, flags_of(forward)), B, L, h0=c["h0"],
                         lengths=lengths_tensor(d, L), y=y0.clone())
    check_forward(d, y, h, B, L, forward, y0.cpu())


def check_backward(d, out, B, L, forward, keys=("x", "r", "g")):
    """out against the oracle; keys other than x, r, g name what an 8-bit checkpoint stands for."""
    dtype = d["x"].dtype
    E = d["x"].shape[1]
    lam = S.to_f64(d["lam"])
    dlam, dlam_bound, dlam_flush, terms = np.zeros(E), np.zeros(E), np.zeros(E), 0
    for b in range(B):
        n = d["lens"][b]
        x, r, g = (rows(d, k, b, L, forward) for k in keys)
        dy, dh = rows(d, "dy", b, L, forward), S.to_f64(d["dh_last"][b])
        h, H = oracle_forward(d, b, L, forward)                       # the checkpoint's states are the exact inputs'
        h0 = S.to_f64(d["h0"][b])
        starts = np.concatenate([h0[None], h])[:max(n, 1):TILE]
        H = np.maximum(H, oracle_forward(d, b, L, forward, keys)[1])
        want = O.gated_scan_backward(x, r, g, lam, h0, dy, dh, starts)
        # the adjoint with every term's magnitude (dx / (beta sg) is it; the last value is dh0)
        a, beta, sr, sg, la = O.gated_coefficients(r, g, lam)
        D, G = np.abs(dh), np.zeros_like(x)
        for k in range(n - 1, -1, -1):
            G[k] = np.abs(dy[k]) + D
            D = a[k] * G[k]
        Gm = np.maximum(G.max(axis=0, initial=0.0), np.abs(dh))
        eps = (8 * n + 256) * U
        with np.errstate(divide="ignore", invalid="ignore"):
            dla = Gm * (a * H + np.where(la == 0, 0.0, sg * np.abs(x) * a * a / beta))
        bound = {"dx": eps * Gm * beta * sg, "dg": eps * Gm * beta * sg * np.abs(x), "dr": eps * dla * np.abs(la)}
        flush = FLUSH * Gm * (1 + top(x))
        for name, w in (("dx", want[0]), ("dr", want[1]), ("dg", want[2])):
            got = S.to_f64(out[name].cpu())
            assert np.all(got[b * L + n:(b + 1) * L] == 0), f"{name}: padding rows are zeros"
            got = got[b * L: b * L + n]
            bounded(got if forward else got[::-1], w, bound[name] * 1.01 + half_step(dtype, w) + flush + 1e-37,
                    f"{name} of {b}")
        dlam += want[3]
        dlam_bound += (dla * sr).sum(axis=0) * 8 / (1 + np.exp(-lam))
        dlam_flush += n * flush * 8
        terms += n
        bounded(S.to_f64(out["dh0"][b].cpu()), want[4], eps * Gm + 1e-37, f"dh0 of {b}")
    longest = max(d["lens"])
    bounded(S.to_f64(out["dlam"].cpu()), dlam, (8 * longest + 256 + terms) * U * dlam_bound + dlam_flush + 1e-37, "dlam")


def train(d, c, B, L, E, dtype, forward, act8, stream=None):
    dims = bd.gated_dims(E, dtype, flags_of(forward, act8))
    lt = lengths_tensor(d, L)
    y, h, ck = bd.gated_scan_train(c["x"], c["r"], c["g"], c["lam"], dims, B, L, h0=c["h0"], lengths=lt, stream=stream)
    kept = {} if act8 else {k: c[k] for k in ("x", "r", "g")}
    out = bd.gated_scan_backward(c["dy"], c["lam"], dims, B, L, ck, dh_last=c["dh_last"], lengths=lt, stream=stream, **kept)
    return y, h, ck, out


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("forward", [False, True], ids=["r2l", "l2r"])
@pytest.mark.parametrize("B,L,E,lens", SHAPES)
def test_gradient(B, L, E, lens, forward, dtype):
    d = make(B, L, E, dtype, seed=B + 7 * L + E + 1, lens=lens)
    poison(d, L)
    y, h, _, out = train(d, dev(d), B, L, E, dtype, forward, act8=False)
    check_forward(d, y, h, B, L, forward)
    check_backward(d, out, B, L, forward)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("forward", [False, True], ids=["r2l", "l2r"])
@pytest.mark.parametrize("B,L,E,lens", SHAPES)
def test_gradient_from_8_bits(B, L, E, lens, forward, dtype):
    """The forward is the exact one; the gradient is the formula at what the 8 bits stand for, and bit for bit the
    gradient of unpack(pack(x, r, g)) with the same states."""
    d = make(B, L, E, dtype, seed=B + 7 * L + E + 2, lens=lens)
    poison(d, L)
    c = dev(d)
    y, h, ck, out = train(d, c, B, L, E, dtype, forward, act8=True)
    check_forward(d, y, h, B, L, forward)
    for k in ("x", "r", "g"):
        v = O.act8_values(S.to_f64(d[k]))
        d[k + "8"] = torch.from_numpy(v)
    check_backward(d, out, B, L, forward, ("x8", "r8", "g8"))

    lt = lengths_tensor(d, L)
    full = bd.gated_dims(E, dtype, flags_of(forward))
    exact = ck[: bd.gated_scan_checkpoint_size(full, B, L)]      # a checkpoint begins with its states
    back = {}
    for k in ("x", "r", "g"):
        q, s = bd.act8_pack(c[k], B, L, lengths=lt)
        back[k] = bd.act8_unpack(q, s, B, L, dtype, lengths=lt)
    same = bd.gated_scan_backward(c["dy"], c["lam"], full, B, L, exact, dh_last=c["dh_last"], lengths=lt, **back)
    for k in out:
        assert torch.equal(out[k], same[k]), k


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("spread", ["all", "some", "border"])
def test_fast_and_slow_channels(spread, dtype):
    """Decays from none to all at once in every channel, in a few channels of a row, and around half the state kept."""
    B, L, E, lens = 3, 200, 200, [200, 77, 130]
    d = make(B, L, E, dtype, seed=4, lens=lens)
    gen = torch.Generator().manual_seed(44)
    if spread == "all":
        d["lam"] = torch.randn(E, generator=gen) * 4
    elif spread == "some":
        d["lam"][::70] = torch.randn(len(range(0, E, 70)), generator=gen) * 2
    else:                                          # 8 softplus(lam) log2 e from 0.2 to 1.2
        sp = torch.linspace(0.2, 1.2, E, dtype=torch.float64) / (8 * 1.4426950408889634)
        d["lam"] = torch.log(torch.expm1(sp)).float()
    c = dev(d)
    for forward in (False, True):
        y, h, _, out = train(d, c, B, L, E, dtype, forward, False)
        check_forward(d, y, h, B, L, forward)
        check_backward(d, out, B, L, forward)
    y, h = bd.gated_scan(c["x"], c["r"], c["g"], c["lam"], bd.gated_dims(E, dtype), B, L, h0=c["h0"],
                         lengths=lengths_tensor(d, L))
    check_forward(d, y, h, B, L, False)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_columns_of_wider_arrays(dtype):
    """x, r and g as columns of one projection's output, y and the gradients as columns too: once at offsets that keep
    rows on 16-byte boundaries, once at odd ones."""
    B, L, E = 2, 150, 70
    d = make(B, L, E, dtype, seed=5)
    c = dev(d)
    ref = train(d, c, B, L, E, dtype, False, False)
    for pad, ld in ((72, 4 * 72), (71, 4 * 71 + 1)):
        wide = torch.zeros(B * L, ld, dtype=dtype, device="cuda")
        at = {k: wide[:, i * pad: i * pad + E] for i, k in enumerate(("x", "r", "g", "dy"))}
        for k in at:
            at[k].copy_(c[k])
        outs = torch.full((B * L, ld), 7.0, dtype=dtype, device="cuda")
        cols = [outs[:, i * pad: i * pad + E] for i in range(4)]
        dims = bd.gated_dims(E, dtype)
        y, h, ck = bd.gated_scan_train(at["x"], at["r"], at["g"], c["lam"], dims, B, L, h0=c["h0"], y=cols[0])
        g = bd.gated_scan_backward(at["dy"], c["lam"], dims, B, L, ck, at["x"], at["r"], at["g"], dh_last=c["dh_last"],
                                   dx=cols[1], dr=cols[2], dg=cols[3])
        check_forward(d, y, h, B, L, False)
        check_backward(d, g, B, L, False)
        for k in ("dx", "dr", "dg", "dlam", "dh0"):
            assert torch.equal(g[k], ref[3][k]), k
        for i in range(4):
            assert torch.all(outs[:, i * pad + E:(i + 1) * pad] == 7.0), "columns between were written"
        assert torch.all(outs[:, 4 * pad:] == 7.0)


@pytest.mark.parametrize("E", [1, 3, 5, 31, 63, 129])
@pytest.mark.parametrize("forward", [False, True], ids=["r2l", "l2r"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_rows_that_start_anywhere_among_nan(dtype, forward, E):
    """Each array in a buffer of NaN, with its own start and its own distance from row to row, some without a gap, in
    both forms of the training forward."""
    B, L = 3, 150
    d = make(B, L, E, dtype, seed=31 + E, lens=[150, 0, 131])
    poison(d, L)
    c = dev(d)

    def among_nan(t, start, gap):
        buf = torch.full((start + B * L * (E + gap) + 9,), float("nan"), dtype=dtype, device="cuda")
        at = buf.as_strided((B * L, E), (E + gap, 1), start)
        at.copy_(t)
        return at

    dims, lens = bd.gated_dims(E, dtype, flags=flags_of(forward)), lengths_tensor(d, L)
    for start, gap in ((1, 0), (7, 2), (4, 5)):
        x, r, g = (among_nan(c[k], start + 3 * j, gap + j) for j, k in enumerate(("x", "r", "g")))
        y, h = bd.gated_scan(x, r, g, c["lam"], dims, B, L, lengths=lens, h0=c["h0"])
        check_forward(d, y, h, B, L, forward)
        for act8 in (False, True):
            dims_t = bd.gated_dims(E, dtype, flags=flags_of(forward, act8))
            y_t, h_t, _ = bd.gated_scan_train(x, r, g, c["lam"], dims_t, B, L, lengths=lens, h0=c["h0"])
            check_forward(d, y_t, h_t, B, L, forward)


@pytest.mark.parametrize("forward", [False, True], ids=["r2l", "l2r"])
def test_pieces_and_steps_give_the_whole(forward):
    """A sequence in pieces, the state handed on, down to single tokens: decoding after a prefill."""
    B, L, E, dtype = 2, 140, 96, FP32
    d = make(B, L, E, dtype, seed=6)
    c = dev(d)
    dims = bd.gated_dims(E, dtype, flags_of(forward))
    state = c["h0"].clone()
    pieces = [70, 1, 64, 2, 1, 1, 1]
    y = torch.zeros(B, L, E, dtype=dtype, device="cuda")
    v = {k: c[k].view(B, L, E) for k in ("x", "r", "g")}
    at = 0
    for n in pieces:
        lo, hi = (at, at + n) if forward else (L - at - n, L - at)
        part = [v[k][:, lo:hi].reshape(B * n, E).contiguous() for k in ("x", "r", "g")]
        if n == 1:
            out = bd.gated_step(*part, c["lam"], dims, state)
        else:
            out, state = bd.gated_scan(*part, c["lam"], dims, B, n, h0=state, h_last=state)
        y[:, lo:hi] = out.view(B, n, E)
        at += n
    assert at == L
    check_forward(d, y.view(B * L, E), state, B, L, forward)


def test_steps_leave_finished_sequences_alone():
    B, E = 5, 200
    d = make(B, 1, E, BF16, seed=7, lens=[1, 0, 1, 0, 1])
    poison(d, 1)
    c = dev(d)
    y = torch.full((B, E), 3.0, dtype=BF16, device="cuda")
    y0, state = y.clone(), c["h0"].clone()
    bd.gated_step(c["x"], c["r"], c["g"], c["lam"], bd.gated_dims(E, BF16), state, y=y, lengths=lengths_tensor(d, 1))
    check_forward(d, y, state, B, 1, True, y0.cpu())
    new = torch.empty_like(state)
    bd.gated_step(c["x"], c["r"], c["g"], c["lam"], bd.gated_dims(E, BF16), c["h0"], new_state=new,
                  lengths=lengths_tensor(d, 1))
    assert torch.equal(new, state) and torch.equal(c["h0"].cpu(), d["h0"])


@pytest.mark.parametrize("L", [1, 3, 200])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_extreme_gates(dtype, L):
    """Gates at ±inf and at the type's lowest and highest values, and far out: positions whose recurrence gate is
    closed leave the state bit for bit, an open one forgets at its fastest; gradients stay finite."""
    B, E = 2, 64
    d = make(B, L, E, dtype, seed=8)
    low = torch.finfo(dtype).min
    vals = [float("-inf"), low, -100.0, -60.0, 60.0, 100.0, -low, float("inf")]
    for i, v in enumerate(vals):
        d["r"][:, 4 * i] = v
        d["g"][:, 4 * i + 1] = v
        d["r"][:, 4 * i + 2] = v
        d["g"][:, 4 * i + 2] = vals[-1 - i]
    d["lam"][40], d["lam"][41], d["lam"][42] = -30.0, 30.0, -100.0     # no decay to speak of, and all at once
    y, h, _, out = train(d, dev(d), B, L, E, dtype, False, False)
    check_forward(d, y, h, B, L, False)
    assert torch.equal(h[:, 0].cpu(), d["h0"][:, 0]) and torch.equal(h[:, 4].cpu(), d["h0"][:, 4])
    for k, v in out.items():
        assert bool(torch.isfinite(v.float()).all()), k
    check_backward(d, out, B, L, False)
    dims = bd.gated_dims(E, dtype)
    c = dev(d)
    y2, h2 = bd.gated_scan(c["x"], c["r"], c["g"], c["lam"], dims, B, L, h0=c["h0"])
    check_forward(d, y2, h2, B, L, False)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("fast", [False, True], ids=["slow", "fast"])
def test_infinite_gates_in_8_bits(dtype, fast):
    """±inf in r and g closes and opens gates in the 8-bit checkpoint too: it stands for them by ±256, whose sigmoid is
    0 (2^-369 in float64, below the flush bound) or 1."""
    B, L, E = 2, 130, 96
    d = make(B, L, E, dtype, seed=20)
    if fast:
        d["lam"] += 6.0
    inf = float("inf")
    d["r"][3::17, ::5], d["r"][5::19, 1::7] = -inf, inf
    d["g"][4::13, ::3], d["g"][6::11, 1::4] = -inf, inf
    d["r"][:, 64:] = -inf                                       # a whole group of channels closed throughout
    y, h, _, out = train(d, dev(d), B, L, E, dtype, False, True)
    check_forward(d, y, h, B, L, False)
    for k in ("x", "r", "g"):
        v = S.to_f64(d[k])
        d[k + "8"] = torch.from_numpy(O.act8_values(np.where(np.isinf(v), np.copysign(256.0, v), v)))
    for k, v in out.items():
        assert bool(torch.isfinite(v.float()).all()), k
    check_backward(d, out, B, L, False, ("x8", "r8", "g8"))


def test_optional_results_left_out():
    """The C entry points without h_last, status and dh0 (the binding always asks for them)."""
    B, L, E, dtype = 2, 70, 96, BF16
    for L in (1, 70, 1300):
        d = make(B, L, E, dtype, seed=23)
        c = dev(d)
        lib, dims = bd.load(), bd.gated_dims(E, dtype)
        y0, _, ck0, out0 = train(d, c, B, L, E, dtype, False, False)
        gi = bd.GatedIn(*(c[k].data_ptr() for k in ("x", "r", "g")), E, E, E, c["lam"].data_ptr(), c["h0"].data_ptr())
        st = torch.cuda.current_stream().cuda_stream
        y = torch.empty_like(y0)
        assert lib.r2l_gated_scan(gi, y.data_ptr(), E, None, dims, B, L, None, None, st) == 0
        check_forward(d, y, bd.gated_scan(c["x"], c["r"], c["g"], c["lam"], dims, B, L, h0=c["h0"])[1], B, L, False)
        ck = torch.empty_like(ck0)
        assert lib.r2l_gated_scan_train(gi, y.data_ptr(), E, None, dims, B, L, None, ck.data_ptr(), ck.numel(), None, st) == 0
        assert torch.equal(y, y0)
        dx, dr, dg = (torch.empty_like(y0) for _ in range(3))
        dlam = torch.empty(E, device="cuda")
        ws = torch.empty(bd.gated_scan_backward_workspace_size(dims, B, L), dtype=torch.uint8, device="cuda")
        gr = bd.GatedGrads(dx.data_ptr(), dr.data_ptr(), dg.data_ptr(), E, E, E, dlam.data_ptr(), None)
        assert lib.r2l_gated_scan_backward(gi, c["dy"].data_ptr(), E, c["dh_last"].data_ptr(), gr, dims, B, L, None,
                                           ck.data_ptr(), ck.numel(), ws.data_ptr(), ws.numel(), st) == 0
        assert all(torch.equal(a, out0[k]) for a, k in ((dx, "dx"), (dr, "dr"), (dg, "dg"), (dlam, "dlam")))


def test_many_sequences():
    """More sequences than one launch sums dlam over."""
    B, L, E = 2500, 3, 10
    d = make(B, L, E, FP32, seed=21, lens=[b % 4 for b in range(B)])
    y, h, _, out = train(d, dev(d), B, L, E, FP32, False, False)
    check_forward(d, y, h, B, L, False)
    check_backward(d, out, B, L, False)


def test_final_state_over_the_initial_one():
    """h_last = h0 in whole scans and training forwards of both block shapes and of a cluster."""
    for B, L, E in ((2, 100, 64), (2, 700, 96), (1, 2100, 64)):
        d = make(B, L, E, FP32, seed=22)
        c = dev(d)
        dims = bd.gated_dims(E, FP32)
        for f in (bd.gated_scan, bd.gated_scan_train):
            state = c["h0"].clone()
            out = f(c["x"], c["r"], c["g"], c["lam"], dims, B, L, h0=state, h_last=state)
            check_forward(d, out[0], state, B, L, False)


def test_all_positions_closed():
    """Nothing enters: zeros stay zeros exactly, and the adjoint passes through."""
    B, L, E = 2, 100, 64
    d = make(B, L, E, BF16, seed=9)
    d["r"][:] = float("-inf")
    d["h0"][:] = 0
    y, h, _, out = train(d, dev(d), B, L, E, BF16, False, False)
    assert torch.all(y == 0) and torch.all(h == 0)
    for k in ("dx", "dr", "dg", "dlam"):
        assert torch.all(out[k] == 0), k
    check_backward(d, out, B, L, False)


def test_nan_stays_in_its_channel_and_after_its_position():
    B, L, E = 2, 100, 64
    d = make(B, L, E, FP32, seed=10)
    d["x"][40, 5] = float("nan")
    y, h, _, _ = train(d, dev(d), B, L, E, FP32, True, False)
    bad = torch.isnan(y).cpu()
    want = torch.zeros_like(bad)
    want[40:100, 5] = True
    assert torch.equal(bad, want)


def test_no_initial_state_and_no_final_gradient():
    B, L, E = 2, 90, 64
    d = make(B, L, E, FP32, seed=11)
    c = dev(d)
    dims = bd.gated_dims(E, FP32)
    z = torch.zeros(B, E, device="cuda")
    y, h, ck = bd.gated_scan_train(c["x"], c["r"], c["g"], c["lam"], dims, B, L)
    y2, h2, ck2 = bd.gated_scan_train(c["x"], c["r"], c["g"], c["lam"], dims, B, L, h0=z)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    a = bd.gated_scan_backward(c["dy"], c["lam"], dims, B, L, ck, c["x"], c["r"], c["g"])
    b = bd.gated_scan_backward(c["dy"], c["lam"], dims, B, L, ck2, c["x"], c["r"], c["g"], dh_last=z)
    assert all(torch.equal(a[k], b[k]) for k in a)
    s = bd.gated_scan(c["x"][:B], c["r"][:B], c["g"][:B], c["lam"], dims, B, 1)
    t = bd.gated_scan(c["x"][:B], c["r"][:B], c["g"][:B], c["lam"], dims, B, 1, h0=z)
    assert torch.equal(s[0], t[0]) and torch.equal(s[1], t[1])


def test_lengths_outside_are_clamped_and_flagged():
    B, L, E = 3, 70, 64
    for n in (L, 1):
        d = make(B, n, E, BF16, seed=12, lens=[0, n, n])
        c = dev(d)
        status = torch.full((4,), -1, dtype=torch.int32, device="cuda")
        dims = bd.gated_dims(E, BF16)
        lt = torch.tensor([-5, n + 9, n], dtype=torch.int32, device="cuda")
        y, h = bd.gated_scan(c["x"], c["r"], c["g"], c["lam"], dims, B, n, h0=c["h0"], lengths=lt, status=status)
        check_forward(d, y, h, B, n, False)
        assert bd.get_device_status(status) == (6, bd.R2L_DEVFLAG_LENGTH_CLAMPED)
        bd.gated_scan(c["x"], c["r"], c["g"], c["lam"], dims, B, n, h0=c["h0"], status=status)
        assert bd.get_device_status(status) == (0, 0)
        y, h, ck = bd.gated_scan_train(c["x"], c["r"], c["g"], c["lam"], dims, B, n, h0=c["h0"], lengths=lt, status=status)
        assert bd.get_device_status(status) == (6, bd.R2L_DEVFLAG_LENGTH_CLAMPED)
        ws = torch.empty(bd.gated_scan_backward_workspace_size(dims, B, n), dtype=torch.uint8, device="cuda")
        out = bd.gated_scan_backward(c["dy"], c["lam"], dims, B, n, ck, c["x"], c["r"], c["g"], dh_last=c["dh_last"],
                                     lengths=lt, workspace=ws)
        check_backward(d, out, B, n, False)
        assert bd.get_device_status(ws) == (6, bd.R2L_DEVFLAG_LENGTH_CLAMPED)


def test_reproducible_and_independent_of_other_sequences_lengths():
    B, L, E = 3, 300, 130
    d = make(B, L, E, BF16, seed=13)
    c = dev(d)
    one, two = (train(d, c, B, L, E, BF16, False, True) for _ in range(2))
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    assert all(torch.equal(one[3][k], two[3][k]) for k in one[3])
    d["lens"] = [L, 17, 250]
    three = train(d, c, B, L, E, BF16, False, True)
    assert torch.equal(one[0][:L], three[0][:L])
    for k in ("dx", "dr", "dg"):
        assert torch.equal(one[3][k][:L], three[3][k][:L])


@pytest.mark.parametrize("act8", [False, True], ids=["full", "act8"])
def test_in_a_graph(act8):
    """A step, a scan, a training forward and its gradient captured together, replayed on new inputs."""
    B, L, E, dtype = 2, 150, 128, BF16
    d, d2 = make(B, L, E, dtype, seed=14, lens=[150, 90]), make(B, L, E, dtype, seed=15, lens=[31, 150])
    c = dev(d)
    dims = bd.gated_dims(E, dtype, flags_of(False, act8))
    lt = lengths_tensor(d, L)
    ck = torch.empty(bd.gated_scan_checkpoint_size(dims, B, L), dtype=torch.uint8, device="cuda")
    ws = torch.empty(bd.gated_scan_backward_workspace_size(dims, B, L), dtype=torch.uint8, device="cuda")
    step_state = torch.empty(B, E, device="cuda")

    def work():
        y, h = bd.gated_scan(c["x"], c["r"], c["g"], c["lam"], dims, B, L, h0=c["h0"], lengths=lt)
        s = bd.gated_step(c["x"][:B], c["r"][:B], c["g"][:B], c["lam"], dims, c["h0"], new_state=step_state)
        yt, ht, _ = bd.gated_scan_train(c["x"], c["r"], c["g"], c["lam"], dims, B, L, h0=c["h0"], lengths=lt, checkpoint=ck)
        kept = {} if act8 else {k: c[k] for k in ("x", "r", "g")}
        g = bd.gated_scan_backward(c["dy"], c["lam"], dims, B, L, ck, dh_last=c["dh_last"], lengths=lt, workspace=ws, **kept)
        return [y, h, s, yt, ht, *g.values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for e in (d2, d):
        for k, v in dev(e).items():
            c[k].copy_(v)
        lt.copy_(lengths_tensor(e, L))
        graph.replay()
        got = [t.clone() for t in held]
        for i, (u, v) in enumerate(zip(got, work())):
            rows_valid = torch.cat([torch.arange(L) < n for n in e["lens"]]).cuda()
            if i in (0, 3):                          # y past a length is not written
                u, v = u[rows_valid], v[rows_valid]
            assert torch.equal(u, v), i


def test_two_streams_at_once():
    """Independent calls on two streams, each stream's own tensors, many in flight."""
    B, L, E, dtype = 2, 400, 256, FP32
    ds = [make(B, L, E, dtype, seed=s) for s in (16, 17)]
    cs = [dev(d) for d in ds]
    alone = [train(d, c, B, L, E, dtype, False, False) for d, c in zip(ds, cs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        got += [(i, train(ds[i], cs[i], B, L, E, dtype, False, False, stream=streams[i] if i else streams[i].cuda_stream))
                for i in (0, 1)]
    torch.cuda.synchronize()
    for i, (y, h, _, out) in got:
        assert torch.equal(y, alone[i][0]) and torch.equal(h, alone[i][1])
        assert all(torch.equal(out[k], alone[i][3][k]) for k in out)


def test_offsets_past_32_bits():
    """One long sequence whose rows lie in a wide array: the last element is more than 2^32 bytes and 2^31 elements
    from the first."""
    L, E, ld, dtype = 70001, 24, 32768, BF16
    d = make(1, L, E, dtype, seed=18)
    assert (L - 1) * ld > 2 ** 31
    wide = torch.empty(L, ld, dtype=dtype, device="cuda")
    at = {k: wide[:, 1000 + i * 64: 1000 + i * 64 + E] for i, k in enumerate(("x", "r", "g", "y", "dy", "dx", "dr", "dg"))}
    c = dev(d)
    for k in ("x", "r", "g", "dy"):
        at[k].copy_(c[k])
    dims = bd.gated_dims(E, dtype)
    y, h, ck = bd.gated_scan_train(at["x"], at["r"], at["g"], c["lam"], dims, 1, L, h0=c["h0"], y=at["y"])
    check_forward(d, y, h, 1, L, False)
    out = bd.gated_scan_backward(at["dy"], c["lam"], dims, 1, L, ck, at["x"], at["r"], at["g"], dh_last=c["dh_last"],
                                 dx=at["dx"], dr=at["dr"], dg=at["dg"])
    check_backward(d, out, 1, L, False)
    y, h = bd.gated_scan(at["x"], at["r"], at["g"], c["lam"], dims, 1, L, h0=c["h0"], y=at["y"])
    check_forward(d, y, h, 1, L, False)


def test_binding_refuses_what_it_cannot_pass_on():
    B, L, E = 2, 10, 64
    d = make(B, L, E, BF16, seed=19)
    c = dev(d)
    dims = bd.gated_dims(E, BF16)
    ok = (c["x"], c["r"], c["g"], c["lam"], dims, B, L)

    def call(i, v, **kw):
        a = list(ok)
        a[i] = v
        return bd.gated_scan(*a, **kw)

    for i, v in ((0, c["x"][:-1]), (1, c["r"].float()), (2, c["g"].cpu()), (0, c["x"].t().contiguous().t()),
                 (1, c["r"][:1].expand(B * L, E)), (3, c["lam"].double()), (3, c["lam"][:-1])):
        with pytest.raises(ValueError):
            call(i, v)
    for kw in ({"h0": c["h0"][:1]}, {"h0": c["h0"].to(BF16)}, {"lengths": torch.ones(B, dtype=torch.int64, device="cuda")},
               {"lengths": torch.ones(B, dtype=torch.int32)}, {"y": torch.empty(B * L, E, device="cuda")},
               {"h_last": torch.empty(B, E + 1, device="cuda")}):
        with pytest.raises(ValueError):
            bd.gated_scan(*ok, **kw)
    with pytest.raises(bd.R2LError):
        bd.gated_scan(*ok, y=c["x"])
    _, _, ck = bd.gated_scan_train(*ok)
    with pytest.raises(ValueError):
        bd.gated_scan_backward(c["dy"], c["lam"], dims, B, L, ck)                 # x, r, g are needed
    with pytest.raises(bd.R2LError):                                                # a full checkpoint read as 8 bits
        bd.gated_scan_backward(c["dy"], c["lam"], bd.gated_dims(E, BF16, bd.R2L_FLAG_ACT8), B, L, ck)
    with pytest.raises(bd.R2LError):
        bd.gated_scan_train(*ok, checkpoint=ck[:16])
