"""Calls at the edges of what the gated scan and the 8-bit checkpoints accept: parameters without bounds, gates far out,
values near a type's largest, the default stream by its handle; and a hook's gradient from 8 bits.  On the GPU against the
float64 oracle (tolerances as in test_gpu_gated_scan.py and test_gpu_hook_backward.py)."""
import numpy as np
import pytest
import torch

import oracle as O
from reverse_selective_ssm_b200 import binding as bd
from reverse_selective_ssm_b200 import synthetic as S

from . import test_gpu_hook_backward as HB
from .test_gpu_gated_scan import check_backward, check_forward, dev, flags_of, lengths_tensor, make, train

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bd.load()


@pytest.mark.parametrize("L", [1, 3, 200, 1300])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_decay_parameters_without_bounds(dtype, L):
    """lam at ±inf and out to fp32's largest: a channel that never forgets keeps its state bit for bit, one that forgets
    at once holds its input alone, and a closed gate keeps the state even there.  64 channels hold slow ones only, 64
    both kinds.  The oracle has the limits: at lam = -700 the decay is 1 to the last digit, at 1e30 it is 0."""
    B, E = 2, 128
    d = make(B, L, E, dtype, seed=40 + L)
    slow, fast = [-INF, torch.finfo(FP32).min, -3e38, -2e38, -200.0], [INF, torch.finfo(FP32).max, 3e38, 2e38, 1e30]
    d["lam"][:5] = d["lam"][64:69] = torch.tensor(slow)
    d["lam"][70:75] = torch.tensor(fast)
    d["lam"][75] = INF
    d["r"][:, 75] = d["r"][:, 3] = -INF
    c = dev(d)
    for forward in (False, True):
        dims = bd.gated_dims(E, dtype, flags_of(forward))
        y, h, _, out = train(d, c, B, L, E, dtype, forward, False)
        y2, h2 = bd.gated_scan(c["x"], c["r"], c["g"], c["lam"], dims, B, L, h0=c["h0"])
        for k in [*range(5), *range(64, 69), 75]:
            assert torch.equal(h[:, k], c["h0"][:, k]) and torch.equal(h2[:, k], c["h0"][:, k]), k
        want = dict(d, lam=d["lam"].double().clamp(-700, 1e30))
        check_forward(want, y, h, B, L, forward)
        check_forward(want, y2, h2, B, L, forward)
        for k, v in out.items():
            assert bool(torch.isfinite(v.float()).all()), k
        check_backward(want, out, B, L, forward)


def test_a_decay_parameter_that_is_nan_shows():
    B, L, E = 2, 70, 64
    d = make(B, L, E, FP32, seed=41)
    d["lam"][7] = float("nan")
    for n in (1, L):
        e = {k: v[: B * n] if torch.is_tensor(v) and v.shape[0] == B * L else v for k, v in d.items()}
        y, h, _, out = train(e, dev(e), B, n, E, FP32, True, False)
        for t in (y, h, *out.values()):
            bad = torch.isnan(t).cpu().view(-1, E)
            assert bool(bad[:, 7].all()) and not bool(bad[:, :7].any()) and not bool(bad[:, 8:].any())


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("fast", [False, True], ids=["slow", "fast"])
@pytest.mark.parametrize("E", [96, 70])
def test_gates_far_out_in_8_bits(E, fast, dtype):
    """Masks of -1e9, of the type's lowest value and of -inf, alone and together among the channels of a scale: those
    gates are closed (or open) in the gradient from 8 bits as they are in the forward, and the other channels' gates
    come back as those of a row without masks that reaches 256."""
    B, L = 2, 130
    d = make(B, L, E, dtype, seed=43)
    if fast:
        d["lam"] += 6.0
    low = torch.finfo(dtype).min
    d["r"][2::17, ::5], d["r"][5::17, 1::7] = low, -1e9
    d["r"][5::17, ::9], d["r"][8::17, 3::8] = -INF, -low
    d["r"][11::17, 4::6], d["r"][11::17, 5::6], d["r"][11::17, 6::6] = -INF, low, 300.0
    d["r"][14::17, 2::3] = -257.0
    d["g"][3::13, ::3], d["g"][6::13, 1::4] = low, 1e9
    d["g"][6::13, ::4], d["g"][9::13, 2::5], d["g"][9::13, 1::5] = -INF, INF, low
    y, h, _, out = train(d, dev(d), B, L, E, dtype, False, True)
    check_forward(d, y, h, B, L, False)
    for k in ("x", "r", "g"):
        v = S.to_f64(d[k])
        held = O.act8_values(v if k == "x" else np.clip(v, -256.0, 256.0))
        d[k + "8"] = torch.from_numpy(held if k == "x" else np.where(np.abs(v) >= 256.0, np.copysign(np.inf, v), held))
    for k, v in out.items():
        assert bool(torch.isfinite(v.float()).all()), k
    check_backward(d, out, B, L, False, ("x8", "r8", "g8"))


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("cols", [128, 67])
def test_finite_values_stay_finite_in_8_bits(cols, dtype):
    """Values from 248 · 2^120 on would round to 256 · 2^120 = 2^128, which is no fp32 or bf16 number: they are held as
    240 · 2^120, the largest that is."""
    B, L, held = 1, 5, 240 * 2.0 ** 120
    x = torch.randn(L, cols, generator=torch.Generator().manual_seed(44)).to(dtype)
    big = torch.finfo(dtype).max
    x[0, 0], x[0, 1], x[0, 2] = big, -big, 3e38
    x[1, 3], x[1, 4] = 248 * 2.0 ** 120, -247 * 2.0 ** 120
    x[2, 5], x[2, 6], x[2, 7] = -big, INF, float("nan")
    x[3, 66] = big
    q, s = bd.act8_pack(x.cuda(), B, L)
    out = bd.act8_unpack(q, s, B, L, dtype).cpu()
    assert out[0, 0] == held and out[0, 1] == -held and out[1, 3] == held and out[1, 4] == -held
    assert out[2, 5] == -held and bool(torch.isnan(out[2, 6:8]).all()) and out[3, 66] == held
    want = torch.from_numpy(O.act8_values(S.to_f64(x))).to(dtype)
    nan = torch.isnan(want)
    assert int(nan.sum()) == 2 and torch.equal(nan, torch.isnan(out)) and torch.equal(out[~nan], want[~nan])
    q2, s2 = bd.act8_pack(out.cuda(), B, L)                 # packing what was unpacked changes nothing
    again = bd.act8_unpack(q2, s2, B, L, dtype).cpu()
    assert torch.equal(again[~nan], out[~nan]) and torch.equal(s, s2)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("E", [64, 67])
def test_finite_inputs_stay_finite_in_a_scan_of_8_bits(E, dtype):
    """The training forward packs as r2l_act8_pack does: its gradient is bit for bit that of the unpacked inputs.  dr and
    dlam hold σ(g) x a σ(r) / β before G multiplies it, here up to 240 · 2^120 · 0.99 / 0.05 > 2^128, so an infinity
    may stand there (in the same places of both); nothing else passes fp32's range."""
    B, L = 2, 90
    d = make(B, L, E, dtype, seed=45)
    d["dy"], d["dh_last"] = (d["dy"] * 1e-6).to(dtype), d["dh_last"] * 1e-6
    big = torch.finfo(dtype).max
    d["x"][3::20, ::5], d["x"][7::20, 2::9] = big, -248 * 2.0 ** 120
    c = dev(d)
    _, _, ck, out = train(d, c, B, L, E, dtype, False, True)
    full = bd.gated_dims(E, dtype)
    back = {k: bd.act8_unpack(*bd.act8_pack(c[k], B, L), B, L, dtype) for k in ("x", "r", "g")}
    assert all(bool(torch.isfinite(v).all()) for v in back.values())
    same = bd.gated_scan_backward(c["dy"], c["lam"], full, B, L, ck[: bd.gated_scan_checkpoint_size(full, B, L)],
                                  dh_last=c["dh_last"], **back)
    for k, v in out.items():
        assert torch.equal(v.nan_to_num(nan=7.0), same[k].nan_to_num(nan=7.0)), k
        if k in ("dx", "dg", "dh0"):
            assert bool(torch.isfinite(v).all()), k
        else:                                               # channels without such an x
            plain = ~(d["x"].abs() > 1e30).any(0).cuda()
            assert bool(torch.isfinite(v[..., plain]).all()), k


def test_the_default_stream_by_its_raw_handle():
    """stream=0 is the device's default stream, as cudaStream_t has it, not another one."""
    assert torch.cuda.default_stream().cuda_stream == 0
    device = torch.device("cuda", torch.cuda.current_device())
    with bd._elsewhere(device, 0) as raw:
        assert raw == 0 and torch.cuda.current_stream().cuda_stream == 0
    B, L, E = 2, 40, 64
    d = make(B, L, E, FP32, seed=46)
    c = dev(d)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                           # another stream being the current one
        torch.cuda.synchronize()
        y, h, _, out = train(d, c, B, L, E, FP32, False, False, stream=0)
        torch.cuda.synchronize()
    check_forward(d, y, h, B, L, False)
    check_backward(d, out, B, L, False)


def test_hook_gradient_from_8_bits_is_the_formula_at_what_they_hold():
    """A hook's whole gradient from a hidden state kept in 8 bits, against the oracle's gradient at the values that the
    8 bits stand for (bf16 holds them exactly), within the bf16 path's 2e-2; rows of 136 channels end in a short group.
    It is that gradient and not the exact hidden state's: bf16 is off by 2^-8 of a value, e4m3 by 2^-4, so the kernels'
    is nearer to the oracle's at the held values than half of what lies between the oracle's two."""
    dims = S.Dims(d_model=136, d_inner=192, d_state=16, dt_rank=8, d_conv=4)
    lengths = torch.tensor([75, 38], dtype=torch.int32)
    dims, h, w, dh_out = HB.make(2, 75, seed=47, lengths=lengths, dims=dims)
    B, L, E = h.shape
    flat, lt = h.cuda().view(B * L, E), lengths.cuda()
    q, s = bd.act8_pack(flat, B, L, lengths=lt)
    held = torch.full_like(flat, float("nan"))              # padding rows are not read
    bd.act8_unpack(q, s, B, L, lengths=lt, out=held)
    got = HB.run_gpu(dims, held.view(B, L, E).cpu(), w, 0.7, dh_out, lengths)
    exact = torch.from_numpy(O.act8_values(S.to_f64(h.view(B * L, E)))).to(h.dtype).view(B, L, E)
    want = HB.run_oracle(exact, w, 0.7, dh_out, lengths)
    HB.compare(got, want, h, dh_out, lengths)
    other = HB.run_oracle(h, w, 0.7, dh_out, lengths)
    for k in ("W_in", "W_x", "W_out"):
        between = np.linalg.norm(want["d" + k] - other["d" + k])
        assert np.linalg.norm(S.to_f64(got[2][k]) - want["d" + k]) < between / 2, k


@pytest.mark.parametrize("E", [1, 3, 31, 67, 129])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_long_rows_that_start_anywhere_among_nan_in_8_bits(dtype, E):
    """The training forward with 8-bit copies, and its gradient, on long sequences whose rows lie in buffers of NaN, each
    with its own start and distance: what lies beside a row counts neither for the states nor for a scale."""
    B, L = 2, 700
    d = make(B, L, E, dtype, seed=48 + E, lens=[700, 333])
    c = dev(d)

    def among_nan(t, start, gap):
        buf = torch.full((start + B * L * (E + gap) + 9,), float("nan"), dtype=dtype, device="cuda")
        at = buf.as_strided((B * L, E), (E + gap, 1), start)
        at.copy_(t)
        return at

    for forward in (False, True):
        y0, h0, ck0, out0 = train(d, c, B, L, E, dtype, forward, True)
        check_forward(d, y0, h0, B, L, forward)
        for start, gap in ((1, 1), (7, 4)):
            e = dict(c, **{k: among_nan(c[k], start + j, gap + j) for j, k in enumerate(("x", "r", "g", "dy"))})
            y, h, _, out = train(d, e, B, L, E, dtype, forward, True)
            check_forward(d, y, h, B, L, forward)
            assert torch.equal(h, h0) and all(torch.equal(out[k], out0[k]) for k in out)


@pytest.mark.parametrize("act8", [False, True], ids=["full", "act8"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,L,E,lens", [(1, 1100, 500, None), (1, 1100, 1000, None), (2, 1100, 1030, [1100, 514]),
                                        (1, 1100, 3040, None), (5, 777, 515, [777, 0, 388, 583, 194]), (2, 600, 512, [0, 600])])
def test_every_choice_of_clusters(B, L, E, lens, dtype, act8):
    """Few channels and long sequences: single blocks and clusters of every size, of full length and ragged."""
    d = make(B, L, E, dtype, seed=50, lens=lens)
    c = dev(d)
    y, h, _, out = train(d, c, B, L, E, dtype, False, act8)
    check_forward(d, y, h, B, L, False)
    if act8:
        for k in ("x", "r", "g"):
            d[k + "8"] = torch.from_numpy(O.act8_values(S.to_f64(d[k])))
    check_backward(d, out, B, L, False, ("x8", "r8", "g8") if act8 else ("x", "r", "g"))
    y, h = bd.gated_scan(c["x"], c["r"], c["g"], c["lam"], bd.gated_dims(E, dtype), B, L, h0=c["h0"],
                         lengths=lengths_tensor(d, L))
    check_forward(d, y, h, B, L, False)


@pytest.mark.parametrize("B,L,E", [(2, 1, 64), (2, 100, 70), (2, 700, 96), (1, 2100, 64), (3, 3, 40)])
def test_state_gradient_over_the_final_one(B, L, E):
    """dh0 = dh_last in blocks of both shapes, in a cluster and with a sequence of no positions (the C interface; the
    binding allocates dh0)."""
    for lens in (None, [0] + [L] * (B - 1)):
        d = make(B, L, E, FP32, seed=49, lens=lens)
        c = dev(d)
        lib, dims, lt = bd.load(), bd.gated_dims(E, FP32), lengths_tensor(d, L)
        _, _, ck, want = train(d, c, B, L, E, FP32, False, False)
        dh = c["dh_last"].clone()
        gi = bd.GatedIn(*(c[k].data_ptr() for k in ("x", "r", "g")), E, E, E, c["lam"].data_ptr(), None)
        got = {k: torch.empty_like(want[k]) for k in ("dx", "dr", "dg", "dlam")}
        gr = bd.GatedGrads(*(got[k].data_ptr() for k in ("dx", "dr", "dg")), E, E, E, got["dlam"].data_ptr(), dh.data_ptr())
        ws = torch.empty(bd.gated_scan_backward_workspace_size(dims, B, L), dtype=torch.uint8, device="cuda")
        assert lib.r2l_gated_scan_backward(gi, c["dy"].data_ptr(), E, dh.data_ptr(), gr, dims, B, L,
                                           None if lt is None else lt.data_ptr(), ck.data_ptr(), ck.numel(), ws.data_ptr(),
                                           ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(dh, want["dh0"]) and all(torch.equal(got[k], want[k]) for k in got)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("E", [64, 67])
def test_nan_beside_gates_far_out_in_8_bits(E, dtype):
    """A NaN in x, r or g among masked gates and far values of the same scales stays in its channel."""
    B, L = 1, 100
    d = make(B, L, E, dtype, seed=51)
    low, nan = torch.finfo(dtype).min, float("nan")
    d["x"][40, 5] = d["r"][41, 9] = d["g"][42, 13] = nan
    d["r"][41, 10], d["r"][41, 11], d["g"][42, 14], d["g"][42, 15] = low, INF, -1e9, -INF
    d["r"][43, 20], d["x"][44, 21] = -INF, 1e30
    _, _, _, out = train(d, dev(d), B, L, E, dtype, True, True)
    clean = dict(d)
    for k in ("x", "r", "g"):
        clean[k] = d[k].clone().nan_to_num(nan=0.0, posinf=INF, neginf=-INF)
    keep = torch.ones(E, dtype=torch.bool)
    keep[[5, 9, 13]] = False
    for k, v in out.items():
        v = v.cpu()
        assert bool(torch.isnan(v[..., ~keep]).any()) and not bool(torch.isnan(v[..., keep]).any()), k
    for k in ("x", "r", "g"):
        v = S.to_f64(clean[k])
        held = O.act8_values(v if k == "x" else np.clip(v, -256.0, 256.0))
        clean[k + "8"] = torch.from_numpy(held if k == "x" else np.where(np.abs(v) >= 256.0, np.copysign(np.inf, v), held))
    # the NaN channels aside, all is as if they held zeros there (a zero does not count for a scale either)
    want = {k: v.cpu().clone() for k, v in out.items()}
    _, _, _, zeros = train(clean, dev(clean), B, L, E, dtype, True, True)
    for k in want:
        assert torch.equal(want[k][..., keep], zeros[k].cpu()[..., keep]), k
    check_backward(clean, zeros, B, L, True, ("x8", "r8", "g8"))
