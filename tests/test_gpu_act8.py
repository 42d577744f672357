"""8-bit activation checkpoints on the GPU: the oracle's values exactly (the only rounding is e4m3's own), and a hook's
gradient from a hidden state that was kept in 8 bits."""
import numpy as np
import pytest
import torch

import oracle as O
from reverse_selective_ssm_b200 import binding as bd
from reverse_selective_ssm_b200 import synthetic as S

from . import gpu_util as G

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bd.load()


def _rounded(v, dtype):
    """float64 values in dtype (bf16 holds every e4m3 value times a power of two, unless it is tiny)."""
    return torch.from_numpy(v).to(dtype)


def _same(a, b):
    a, b = a.cpu(), b.cpu()
    nan = torch.isnan(a)
    assert torch.equal(nan, torch.isnan(b))
    assert torch.equal(a[~nan], b[~nan])


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,L,cols,lens", [(1, 1, 1, None), (2, 3, 64, [3, 0]), (3, 5, 63, [5, 1, 0]), (1, 7, 65, None),
                                           (2, 40, 200, [17, 40]), (1, 33, 2048, None), (4, 9, 1037, [9, 8, 0, 1])])
def test_pack_and_unpack(B, L, cols, lens, dtype):
    gen = torch.Generator().manual_seed(cols + L)
    # rows of very different sizes, values spread over many powers of two, exact ties, zeros
    x = torch.randn(B * L, cols, generator=gen) * torch.exp(torch.randn(B * L, cols, generator=gen) * 3)
    x *= torch.exp(torch.rand(B * L, 1, generator=gen) * 100 - 50)
    x[:, ::5] = torch.randint(-64, 65, x[:, ::5].shape, generator=gen).float()
    x[0, : cols // 2] = 0
    x = x.to(dtype)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    xd = x.cuda()
    valid = torch.cat([torch.arange(L) < n for n in (lens or [L] * B)])
    xd[~valid.cuda()] = float("nan")
    q = torch.full((B * L, cols), 99, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.full((B * L, -(-cols // 64)), 99, dtype=torch.uint8, device="cuda")
    bd.act8_pack(xd, B, L, lengths=lt, q=q, scales=s)
    assert torch.all(q.view(torch.uint8)[~valid] == 99) and torch.all(s[~valid] == 99)
    out = torch.full((B * L, cols), 5.0, dtype=dtype, device="cuda")
    bd.act8_unpack(q, s, B, L, lengths=lt, out=out)
    want = _rounded(O.act8_values(S.to_f64(x)), dtype)
    want[~valid] = 5.0
    _same(out, want)
    # the bytes are e4m3 values of the scaled rows: torch's own reading of them gives the same
    up = (s.cpu().int() << 23).view(FP32).double()
    read = q.cpu().float().double() * up.repeat_interleave(64, 1)[:, :cols]
    _same(read[valid].to(dtype), want[valid])
    # packing what was unpacked changes nothing
    q2, s2 = bd.act8_pack(out, B, L, lengths=lt)
    _same(bd.act8_unpack(q2, s2, B, L, dtype, lengths=lt)[valid.cuda()], want[valid])


def test_borders_and_special_values():
    x = torch.zeros(8, 128)
    x[0, 0] = 448.0
    x[1, 0] = 448.0000305                                   # the next scale
    x[2, :3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    x[2, 3:6] = torch.tensor([17.0, 19.0, -448.0])          # ties to even at the group's finite scale
    x[3, 0] = torch.finfo(FP32).max
    x[4, 0] = 1e-38
    x[5, 0], x[5, 1] = 1e-45, -1e-45                        # subnormal: below the least scale's smallest value
    x[6, 64:66] = torch.tensor([3.0, -2.0 ** -20])
    x[7, :3] = torch.tensor([448.0, 2.0 ** -10, 3 * 2.0 ** -10])   # half the smallest step goes to zero, three halves to two
    q, s = bd.act8_pack(x.cuda(), 1, 8)
    out = bd.act8_unpack(q, s, 1, 8, FP32)
    _same(out, torch.from_numpy(O.act8_values(x.double().numpy())).float())
    assert s[0, 0] == 127 and s[1, 0] == 128 and s[0, 1] == 1


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_columns_of_wider_arrays(dtype):
    B, L, cols = 2, 21, 200
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(B * L, cols, generator=gen).to(dtype)
    want = _rounded(O.act8_values(S.to_f64(x)), dtype)
    for off, ld in ((16, 256), (3, 331)):
        wide = torch.zeros(B * L, ld, dtype=dtype, device="cuda")
        wide[:, off: off + cols] = x.cuda()
        qw = torch.zeros(B * L, ld, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        q, s = bd.act8_pack(wide[:, off: off + cols], B, L, q=qw[:, off: off + cols])
        ow = torch.full((B * L, ld), 7.0, dtype=dtype, device="cuda")
        out = bd.act8_unpack(q, s, B, L, out=ow[:, off: off + cols])
        _same(out, want)
        assert torch.all(ow[:, :off] == 7) and torch.all(ow[:, off + cols:] == 7)
        rest = qw.view(torch.uint8)
        assert torch.all(rest[:, :off] == 0) and torch.all(rest[:, off + cols:] == 0)


def test_offsets_past_32_bits():
    M, cols, ld = 66001, 70, 32768
    wide = torch.empty(M, ld, dtype=BF16, device="cuda")
    x = torch.randn(M, cols, generator=torch.Generator().manual_seed(4)).to(BF16)
    wide[:, 5: 5 + cols] = x.cuda()
    q, s = bd.act8_pack(wide[:, 5: 5 + cols], 1, M)
    out = bd.act8_unpack(q, s, 1, M, out=wide[:, 100: 100 + cols])
    _same(out, _rounded(O.act8_values(S.to_f64(x)), BF16))


def test_hook_gradient_from_a_checkpoint_in_8_bits():
    """A hook's training step with its hidden state kept in 8 bits: the forward runs on the exact hidden state; the
    gradient, which recomputes the forward, runs on the checkpoint's values and is the gradient at those, bit for bit."""
    B, L, lens = 2, 64, [64, 37]
    case = S.make_case(1, B=B, L=L)
    dims = bd.dims_of(case.dims, case.dtype)
    d = case.dims.d_model
    w = G.device_weights(case)[0]
    h = case.h.cuda()
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, s = bd.act8_pack(h.view(B * L, d), B, L, lengths=lt)
    out, _ = bd.sidecar_forward_train(h, w, dims, case.s[0], lt)
    assert out.shape == h.shape
    del out
    back = torch.full_like(h, float("nan"))                 # padding rows are not read
    bd.act8_unpack(q, s, B, L, lengths=lt, out=back.view(B * L, d))
    dh_out = torch.randn(B, L, d, generator=torch.Generator().manual_seed(5)).cuda()
    grads = bd.alloc_grads(w)
    dh, ds = bd.sidecar_backward(back, w, dims, case.s[0], dh_out, grads, lt)
    want_h = _rounded(O.act8_values(S.to_f64(case.h.view(B * L, d))), case.dtype).view(B, L, d).cuda()
    want_grads = bd.alloc_grads(w)
    want_dh, want_ds = bd.sidecar_backward(want_h, w, dims, case.s[0], dh_out, want_grads, lt)
    assert torch.equal(dh, want_dh) and torch.equal(ds, want_ds)
    for k, v in grads.items():
        assert v is None or torch.equal(v, want_grads[k]), k
    # e4m3 moves a value by at most 2^-4 of it, so the hidden state is near, and so are the gradients' sizes
    exact = bd.alloc_grads(w)
    bd.sidecar_backward(h, w, dims, case.s[0], dh_out, exact, lt)
    assert np.isfinite(float(exact["W_in"].norm())) and float(grads["W_in"].norm()) > 0
