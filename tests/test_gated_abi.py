"""Refusals of the gated scan and the 8-bit checkpoints, on the host before a device is touched (no GPU needed)."""
import ctypes

import pytest
import torch

from reverse_selective_ssm_b200 import binding as bd
from reverse_selective_ssm_b200 import build as bld

FAKE = 0x10000      # aligned non-null values; never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    bld.build()
    return bd.load()


def _dims(E=128, dtype=torch.bfloat16, flags=0):
    return bd.gated_dims(E, dtype, flags)


def _in(**kw):
    d = dict(x=FAKE, r=FAKE + 64, g=FAKE + 128, ldx=128, ldr=128, ldg=128, lam=FAKE, h0=None)
    d.update(kw)
    return bd.GatedIn(**d)


def _fwd(lib, dims=None, B=2, L=100, y=FAKE + 192, ldy=128, h_last=None, lengths=None, status=None, **kw):
    dims = dims or _dims()
    return lib.r2l_gated_scan(ctypes.byref(_in(**kw)), y, ldy, h_last, ctypes.byref(dims), B, L, lengths, status, None)


def test_forward_refusals(lib):
    assert lib.r2l_gated_scan(None, FAKE, 128, None, ctypes.byref(_dims()), 1, 1, None, None, None) == 1
    assert lib.r2l_gated_scan(ctypes.byref(_in()), FAKE + 192, 128, None, None, 1, 1, None, None, None) == 1
    assert _fwd(lib, B=0) == 1
    assert _fwd(lib, L=0) == 1
    assert _fwd(lib, L=-1) == 1
    assert _fwd(lib, dims=_dims(E=0)) == 1
    bad = _dims()
    bad.dtype = 7
    assert _fwd(lib, dims=bad) == 1
    for name in ("x", "r", "g", "lam"):
        assert _fwd(lib, **{name: None}) == 1
    assert _fwd(lib, y=None) == 1
    for name in ("ldx", "ldr", "ldg", "ldy"):
        assert _fwd(lib, **{name: 127}) == 1                       # shorter than a row
    assert _fwd(lib, y=FAKE) == 1                                    # y on x
    assert _fwd(lib, y=FAKE + 64) == 1                               # y on r
    assert _fwd(lib, x=FAKE + 1) == 3
    assert _fwd(lib, y=FAKE + 193) == 3
    assert _fwd(lib, dims=_dims(dtype=torch.float32), g=FAKE + 130) == 3
    for name in ("lam", "h0", "h_last", "lengths", "status"):
        assert _fwd(lib, **{name: FAKE + 2}) == 3
    assert _fwd(lib, L=2 ** 30 + 1) == 2
    assert _fwd(lib, dims=_dims(E=2 ** 31 - 1), B=65536, L=65536, **{n: 2 ** 31 - 1 for n in ("ldx", "ldr", "ldg", "ldy")}) == 2


def test_checkpoint_sizes(lib):
    d, d8 = _dims(E=100), _dims(E=100, flags=bd.R2L_FLAG_ACT8)
    n = bd.gated_scan_checkpoint_size(d, 3, 129)
    assert 3 * 3 * 128 * 4 <= n < 3 * 3 * 128 * 4 + 256              # three tiles a sequence, whole groups of channels
    n8 = bd.gated_scan_checkpoint_size(d8, 3, 129)
    assert n + 3 * 3 * 129 * (128 + 2) <= n8 <= n + 3 * 3 * (129 * 128 + 144 * 2) + 6 * 256
    assert bd.gated_scan_checkpoint_size(d, 0, 1) == 0
    assert bd.gated_scan_checkpoint_size(_dims(E=2 ** 31 - 1, flags=bd.R2L_FLAG_ACT8), 1, 1) == 0
    assert bd.gated_scan_checkpoint_size(_dims(E=2 ** 20), 2 ** 31 - 1, 2 ** 31 - 1) == 0
    assert bd.gated_scan_checkpoint_size(d, 1, 0) == 0
    assert bd.gated_scan_checkpoint_size(_dims(E=-1), 1, 1) == 0
    assert bd.gated_scan_checkpoint_size(_dims(E=2), 1, 2 ** 30 + 1) == 0
    assert bd.gated_scan_backward_workspace_size(d, 3, 129) >= 3 * 100 * 4
    n = bd.gated_scan_backward_workspace_size(d, 2000, 1)           # sums of more than 1024 rows lie behind them
    assert n >= (2000 + 2) * 128 * 4
    assert bd.gated_scan_backward_workspace_size(d, 3, 0) == 0
    # serving setup: half the bytes of x, r and g in bf16, and the states
    big = bd.gated_scan_checkpoint_size(_dims(E=4096, flags=bd.R2L_FLAG_ACT8), 8, 4096)
    assert big < 0.53 * 3 * 2 * 8 * 4096 * 4096


def test_checkpoint_sizes_past_32_bits(lib):
    """B times the tiles of a sequence passes 2^31, and 2^32, long before B · L · E passes 2^50."""
    for B, L in ((65536, 2 ** 22), (2 ** 30, 65), (2 ** 31 - 1, 129), (2 ** 20, 2 ** 30)):
        states = B * -(-L // 64) * 64 * 4
        assert states <= bd.gated_scan_checkpoint_size(_dims(E=1), B, L) < states + 256
        got = bd.gated_scan_checkpoint_size(_dims(E=1, flags=bd.R2L_FLAG_ACT8), B, L)
        least = states + 3 * B * (64 * L + -(-L // 16) * 16)
        assert least <= got < least + 7 * 256
        # a buffer of a byte less is refused
        assert lib.r2l_gated_scan_train(ctypes.byref(_in()), FAKE + 192, 128, None, ctypes.byref(_dims(E=1)), B, L, None, FAKE,
                                        states - 1, None, None) == 4


def test_train_refusals(lib):
    def call(ck=FAKE, nbytes=1 << 40, dims=None, **kw):
        dims = dims or _dims()
        return lib.r2l_gated_scan_train(ctypes.byref(_in(**kw)), FAKE + 192, 128, None, ctypes.byref(dims), 2, 100, None, ck,
                                        nbytes, None, None)

    assert call(ck=None) == 4
    assert call(nbytes=bd.gated_scan_checkpoint_size(_dims(), 2, 100) - 1) == 4
    d8 = _dims(flags=bd.R2L_FLAG_ACT8)
    assert call(dims=d8, nbytes=bd.gated_scan_checkpoint_size(_dims(), 2, 100)) == 4
    assert call(ck=FAKE + 8) == 3
    assert call(x=None) == 1


def _bwd(lib, dims=None, B=2, L=100, dy=FAKE + 192, ld_dy=128, dh_last=None, lengths=None, ck=FAKE, ck_bytes=1 << 40,
         ws=FAKE, ws_bytes=1 << 40, grads=None, **kw):
    dims = dims or _dims()
    g = dict(dx=FAKE + 256, dr=FAKE + 320, dg=FAKE + 384, ld_dx=128, ld_dr=128, ld_dg=128, dlam=FAKE, dh0=None)
    g.update(grads or {})
    return lib.r2l_gated_scan_backward(ctypes.byref(_in(**kw)), dy, ld_dy, dh_last, ctypes.byref(bd.GatedGrads(**g)),
                                       ctypes.byref(dims), B, L, lengths, ck, ck_bytes, ws, ws_bytes, None)


def test_backward_refusals(lib):
    assert _bwd(lib, B=0) == 1
    assert _bwd(lib, L=0) == 1
    assert _bwd(lib, dy=None) == 1
    assert _bwd(lib, lam=None) == 1
    for name in ("x", "r", "g"):
        assert _bwd(lib, **{name: None}) == 1
    for name in ("dx", "dr", "dg", "dlam"):
        assert _bwd(lib, grads={name: None}) == 1
    for name in ("ld_dx", "ld_dr", "ld_dg"):
        assert _bwd(lib, grads={name: 127}) == 1
    assert _bwd(lib, ld_dy=127) == 1
    assert _bwd(lib, ldx=127) == 1
    assert _bwd(lib, grads={"dx": FAKE + 192}) == 1                    # dx on dy
    assert _bwd(lib, grads={"dr": FAKE + 256}) == 1                    # dr on dx
    assert _bwd(lib, grads={"dg": FAKE}) == 1                          # dg on x
    assert _bwd(lib, dy=FAKE + 1) == 3
    assert _bwd(lib, dh_last=FAKE + 2) == 3
    assert _bwd(lib, lengths=FAKE + 2) == 3
    assert _bwd(lib, grads={"dh0": FAKE + 2}) == 3
    assert _bwd(lib, ck=None) == 4
    assert _bwd(lib, ck_bytes=16) == 4
    assert _bwd(lib, ck=FAKE + 8) == 3
    assert _bwd(lib, ws=None) == 4
    assert _bwd(lib, ws_bytes=16) == 4
    assert _bwd(lib, ws=FAKE + 8) == 3
    # the 8-bit checkpoint holds x, r and g; their pointers are not read, and its size is asked for
    d8 = _dims(flags=bd.R2L_FLAG_ACT8)
    n = bd.gated_scan_checkpoint_size(d8, 2, 100)
    assert _bwd(lib, dims=d8, x=None, r=None, g=None, ck_bytes=n - 1) == 4


def test_act8_refusals(lib):
    Q, SC = FAKE + 4096, FAKE + 8192

    def pack(x=FAKE, ldx=100, dtype=0, B=2, L=10, cols=100, lengths=None, q=Q, ldq=100, scales=SC):
        return lib.r2l_act8_pack(x, ldx, dtype, B, L, cols, lengths, q, ldq, scales, None)

    def unpack(q=Q, ldq=100, scales=SC, dtype=0, B=2, L=10, cols=100, lengths=None, out=FAKE, ldo=100):
        return lib.r2l_act8_unpack(q, ldq, scales, dtype, B, L, cols, lengths, out, ldo, None)

    for f, rows, ld in ((pack, "x", "ldx"), (unpack, "out", "ldo")):
        for name in (rows, "q", "scales"):
            assert f(**{name: None}) == 1
        for name in ("B", "L", "cols"):
            assert f(**{name: 0}) == 1
        assert f(dtype=2) == 1
        assert f(**{ld: 99}) == 1
        assert f(ldq=99) == 1
        assert f(**{rows: FAKE + 1}) == 3
        assert f(dtype=1, **{rows: FAKE + 2}) == 3
        assert f(lengths=FAKE + 2) == 3
        assert f(q=FAKE) == 1 and f(scales=FAKE) == 1 and f(scales=Q) == 1      # one buffer for two
        assert f(L=2 ** 30 + 1) == 2


def test_binding_takes_device_tensors_only(lib):
    t, v = torch.zeros(4, 8), torch.zeros(8)
    d = _dims(E=8, dtype=torch.float32)
    for call in (lambda: bd.gated_scan(t, t, t, v, d, 2, 2), lambda: bd.gated_scan_backward(t, v, d, 2, 2, v),
                 lambda: bd.gated_step(t, t, t, v, d, t), lambda: bd.act8_pack(t, 2, 2), lambda: bd.act8_unpack(t, v, 2, 2)):
        with pytest.raises(ValueError, match="device tensors"):
            call()


def _strided(shape, strides, dtype=torch.bfloat16):
    """A tensor of this layout without memory."""
    return torch.empty_strided(shape, strides, dtype=dtype, device="meta")


def test_binding_refuses_row_strides_past_31_bits():
    """The C interface takes row strides as int: one of 2^32 + 64 elements must not arrive as 64."""
    dev = torch.device("meta")
    for stride in (2 ** 31, 2 ** 32 + 64, 2 ** 33 + 1):
        with pytest.raises(ValueError, match="x: .*stride"):
            bd._rows(_strided((2, 64), (stride, 1)), 2, 64, torch.bfloat16, dev, "x")
    assert bd._rows(_strided((2, 64), (2 ** 31 - 1, 1)), 2, 64, torch.bfloat16, dev, "x")[1] == 2 ** 31 - 1
    # one row has no distance to a next one
    for stride in (0, 64, 100, 2 ** 32 + 64):
        assert bd._rows(_strided((1, 64), (stride, 1)), 1, 64, torch.bfloat16, dev, "x")[1] == 64


def test_binding_refuses_sizes_past_31_bits(lib):
    """B and L are int in the C interface too: 2^32 + 1 positions must not arrive as one."""
    d = _dims(E=1)
    for B, L in ((2 ** 32 + 1, 1), (1, 2 ** 32 + 1), (2 ** 31, 1), (1, 2 ** 31)):
        with pytest.raises(ValueError, match="2\\^31"):
            bd._positions(B, L)
        for size in (bd.gated_scan_checkpoint_size, bd.gated_scan_backward_workspace_size):
            with pytest.raises(ValueError, match="2\\^31"):
                size(d, B, L)
    assert bd._positions(2 ** 31 - 1, 3) == 3 * (2 ** 31 - 1)
    with pytest.raises(ValueError, match="2\\^31"):
        bd.gated_dims(2 ** 32 + 64, torch.bfloat16)


def test_binding_refuses_a_status_without_room_for_a_word():
    dev = torch.device("meta")
    for n, dtype in ((0, torch.int32), (3, torch.uint8), (1, torch.int16)):
        with pytest.raises(ValueError, match="status"):
            bd._status(torch.empty(n, dtype=dtype, device=dev), dev)
    for n, dtype in ((1, torch.int32), (4, torch.uint8)):
        bd._status(torch.empty(n, dtype=dtype, device=dev), dev)
    assert bd._status(None, dev) is None


def test_binding_refuses_a_stream_of_another_device():
    class Elsewhere:
        device, cuda_stream = torch.device("cuda", 1), 0x40

    def never(raw):
        raise AssertionError("called")

    with pytest.raises(ValueError, match="stream"):
        bd._call_on(torch.device("cuda", 0), Elsewhere(), never)
