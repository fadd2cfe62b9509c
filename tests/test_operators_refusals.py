"""What the row writer, the rotary turn, the attention and the entry copies refuse on
the host, before any device call: runs without a GPU."""

import ctypes
import math

import pytest
import torch

from serving_pb_lru_amd import head_rows, latent_rows, pack_rows, rotate, ula

EINVAL = -1
P = 1 << 20                  # a plausible device address: refused calls never read it


def test_row_formats():
    size = lambda *a: ula.lib().ula_row_format_bytes(ctypes.byref(ula.RowFormat(*a)))
    assert latent_rows().row_bytes == 656 and size(0, 0, 0, 0) == size(0, 5, -1, 7) == 656   # the rest is not read
    for kv, dim, block in [(1, 64, 1), (8, 128, 1), (2, 64, 8), (1, 64, 16), (1, 128, 8), (3, 64, 2)]:
        want = -(-(2 * kv * dim * block + 8 * kv + 4) // 16) * 16
        assert head_rows(kv, dim, block).row_bytes == size(1, kv, dim, block) == want
    assert ula.lib().ula_row_format_bytes(None) == 0
    for bad in [(2, 0, 0, 0), (-1, 0, 0, 0), (1, 0, 64, 1), (1, -1, 64, 1),
                (1, 1, 63, 1), (1, 1, 96, 1), (1, 1, 64, 0), (1, 1, 64, 3), (1, 1, 64, 32), (1, 1, 128, 16), (1, 16, 128, 1),
                (1, 1 << 30, 128, 16)]:
        assert size(*bad) == 0, bad
    with pytest.raises(ula.UlaError):
        head_rows(16, 128, 1)


def test_attend_bytes():
    L = ula.lib()
    f, h = latent_rows(), head_rows(8, 128)
    need = lambda fmt, *a: L.ula_attend_bytes(ctypes.byref(fmt), *a)
    assert L.ula_attend_bytes(None, 1, 1, 1) == 0
    assert need(f, 0, 2048, 16) == 0 and need(f, 1, 0, 16) == 0 and need(f, 1, 1, 1) == 0
    assert need(f, -1, 1, 1) == need(f, 1, -1, 1) == need(f, 1, 1, 0) == need(f, 1, 1, 1 << 17) == 0
    assert need(h, 1, 4096, 12) == 0                   # query heads are a multiple of the KV heads
    # one long set: split, each part a 32-bit row and its log-sum
    for fmt, width in ((f, 512), (h, 128)):
        n = need(fmt, 1, 4096, 16)
        assert n > 0 and n % (4 * 16 * (width + 1)) < 512
    assert need(f, 1, 2048 * 1024, 16) > 0 and need(f, 1, 2048 * 1024 + 1, 16) == 0
    assert need(h, 1, 1 << 29, 8) > 0 and need(h, 1, 1 << 30, 8) == 0


def test_context_functions_refuse_null():
    L = ula.lib()
    a = ula.UlaAttendArgs()
    assert L.ula_attend(None, 0, 0, 1, 1, P, ctypes.byref(a), 0) == EINVAL
    assert L.ula_fork(None, 0, 0, 1, 1, 0) == EINVAL
    assert L.ula_rename(None, 0, 0, 1, 1, 0) == EINVAL


def pack_args(fmt=None, **kw):
    a = ula.UlaPackArgs()
    a.rows = fmt or latent_rows()
    a.type, a.n, a.layers, a.a, a.b = ula.BF16, 1, 1, P, P
    rot = kw.pop("rotary", None)
    for k, v in kw.items():
        setattr(a, k, v)
    if rot is not None:
        set_rotary(a.rotary, *rot)
    return a


def set_rotary(r, axes, sections, interleaved=0, theta=10000.0):
    r.axes, r.interleaved, r.theta = axes, interleaved, theta
    for i, s in enumerate(sections):
        r.sections[i] = s


BAD_ROTARY = [(0, (32,)), (4, (32, 0, 0)), (1, (31,)), (1, (33,)), (2, (16, 15)), (2, (33, -1)), (3, (16, 16, 1)),
              (1, (32,), 2), (1, (32,), -1), (1, (32,), 0, 0.0), (1, (32,), 0, -1.0), (1, (32,), 0, math.inf),
              (1, (32,), 0, math.nan)]


def test_pack_refuses():
    L = ula.lib()
    call = lambda a, out=P: L.ula_pack_rows(ctypes.byref(a), out, 0)
    assert L.ula_pack_rows(None, P, 0) == EINVAL
    for kw in [dict(type=3), dict(type=-1), dict(n=-1), dict(layers=-1), dict(a=None), dict(b=None), dict(a=P + 1),
               dict(type=ula.FP32, a=P + 2), dict(type=ula.FP32, b=P + 2), dict(count=P),
               dict(n=1 << 13, layers=1 << 13), dict(fmt=ula.RowFormat(1, 1, 65, 1)),
               dict(positions=P + 2, rotary=(1, (32,))), dict(fmt=head_rows(1, 64), count=P + 1),
               dict(fmt=head_rows(8, 128), n=1 << 25, layers=1)]:
        assert call(pack_args(**kw)) == EINVAL, kw
    assert call(pack_args(), None) == EINVAL and call(pack_args(), P + 8) == EINVAL
    for rot in BAD_ROTARY:
        assert call(pack_args(positions=P, rotary=rot)) == EINVAL, rot
    for kw in [dict(n=0), dict(layers=0), dict(n=0, positions=P, rotary=(2, (20, 12), 1))]:
        assert call(pack_args(a=None, b=None, **kw), None) == 0, kw


def rotate_args(**kw):
    a = ula.UlaRotateArgs()
    a.type, a.n, a.heads, a.dim, a.x, a.out, a.positions = ula.BF16, 1, 1, 64, P, P, P
    rot = kw.pop("rotary", (1, (kw.get("dim", 64) // 2,)))
    for k, v in kw.items():
        setattr(a, k, v)
    set_rotary(a.rotary, *rot)
    return a


def test_rotate_refuses():
    L = ula.lib()
    call = lambda a: L.ula_rotate(ctypes.byref(a), 0)
    assert L.ula_rotate(None, 0) == EINVAL
    for kw in [dict(type=3), dict(n=-1), dict(heads=-1), dict(dim=0), dict(dim=63), dict(dim=258), dict(dim=-2),
               dict(inverse=2), dict(inverse=-1), dict(x=None), dict(out=None), dict(positions=None), dict(x=P + 1),
               dict(out=P + 1), dict(type=ula.FP32, x=P + 2), dict(positions=P + 1), dict(n=1 << 30, heads=32)]:
        assert call(rotate_args(**kw)) == EINVAL, kw
    for strides in [(0, 64), (64, 0), (63, 128), (64, -63), (32, 64)]:      # rows of out that share elements
        a = rotate_args(n=2, heads=2)
        a.out_stride[:] = strides
        assert call(a) == EINVAL, strides
    for rot in BAD_ROTARY:
        assert call(rotate_args(rotary=rot)) == EINVAL, rot
    assert call(rotate_args(n=0, x=None, out=None, positions=None)) == 0
    assert call(rotate_args(heads=0, x=None, out=None)) == 0


def test_binding_takes_device_tensors_alone():
    lat, rope = torch.zeros(1, 1, 512), torch.zeros(1, 1, 64)
    with pytest.raises(ValueError, match="CUDA"):
        pack_rows(latent_rows(), lat, rope)
    with pytest.raises(ValueError):
        pack_rows(latent_rows(), lat[0], rope)
    with pytest.raises(ValueError, match="CUDA"):
        rotate(torch.zeros(1, 1, 64), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ula.UlaError):
        pack_rows(ula.RowFormat(1, 1, 65, 1), lat, rope)
