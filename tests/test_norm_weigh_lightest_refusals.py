"""What the norms, the entries' weights and the choice of the lightest entries refuse on the host, before any device
call: runs without a GPU."""

import ctypes
import math

import numpy as np
import pytest
import torch

from serving_pb_lru_amd import Engine, latent_rows, lightest, norm_rotate, ula
from test_operators_refusals import BAD_ROTARY, set_rotary

EINVAL, ERANGE = -1, -2
P = 1 << 20                  # a plausible device address: refused calls never read it


def norm_args(rotary=(1, (32,)), **kw):
    a = ula.UlaNormArgs()
    a.type, a.n, a.dim, a.q_heads, a.k_heads, a.rotary_dim, a.weight_type, a.eps = ula.BF16, 1, 64, 1, 1, 64, ula.BF16, 1e-6
    a.q, a.k, a.q_out, a.k_out, a.positions = P, P, 2 * P, 2 * P, P
    for name, v in kw.items():
        if name.endswith("stride"):
            getattr(a, name)[:] = v
        else:
            setattr(a, name, v)
    set_rotary(a.rotary, *rotary)
    return a


def test_norm_refuses():
    L = ula.lib()
    call = lambda a: L.ula_norm_rotate(ctypes.byref(a), 0)
    assert L.ula_norm_rotate(None, 0) == EINVAL
    for kw in [dict(type=3), dict(type=-1), dict(n=-1), dict(q_heads=-1), dict(k_heads=-1), dict(q_heads=1 << 24), dict(dim=0),
               dict(dim=63), dict(dim=258), dict(rotary_dim=-2), dict(rotary_dim=63), dict(rotary_dim=66), dict(weight_type=ula.FP16),
               dict(weight_type=5), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan), dict(q=None), dict(k=None),
               dict(q_out=None), dict(k_out=None), dict(q=P + 1), dict(k_out=P + 1), dict(q_weight=P + 1), dict(k_weight=P + 1),
               dict(weight_type=ula.FP32, q_weight=P + 2), dict(positions=None), dict(positions=P + 2),
               dict(n=1 << 30, q_heads=64, q_out_stride=(4096, 64))]:
        assert call(norm_args(**kw)) == EINVAL, kw
    for strides in [(0, 64), (64, 0), (63, 128), (64, -63)]:      # rows of a result that share elements
        for name in ("q_out_stride", "k_out_stride"):
            fine = dict(q_out_stride=(128, 64), k_out_stride=(128, 64))
            assert call(norm_args(n=2, q_heads=2, k_heads=2, **{**fine, name: strides})) == EINVAL, (name, strides)
    for rot in BAD_ROTARY:
        assert call(norm_args(rotary=rot)) == EINVAL, rot
    for kw in [dict(n=0), dict(q_heads=0, k_heads=0)]:
        assert call(norm_args(q=None, k=None, q_out=None, k_out=None, positions=None, **kw)) == 0, kw


def test_norm_binding():
    x, w = torch.zeros(2, 1, 64), torch.zeros(64)
    for grad in (dict(q=x.clone().requires_grad_()), dict(k=x.clone().requires_grad_()), dict(q_weight=w.clone().requires_grad_()),
                 dict(k=x, k_weight=w.clone().requires_grad_()), dict(out=(x.clone().requires_grad_(), None))):
        with pytest.raises(ValueError, match="gradient"):
            norm_rotate(**{"q": x, **grad})
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        norm_rotate(x.clone().requires_grad_())


def test_weigh_refuses():
    a = ula.UlaWeighArgs()
    assert ula.lib().ula_weigh(None, 0, 0, 1, 1, P, ctypes.byref(a), 0) == EINVAL
    sel, q = torch.zeros((1, 1), dtype=torch.int32), torch.zeros((1, 1, 576), dtype=torch.bfloat16)
    for kw in (dict(q=q.clone().requires_grad_()), dict(lse=torch.zeros(1, 1).requires_grad_()),
               dict(out=torch.zeros(1, 1).requires_grad_())):
        with pytest.raises(ValueError, match="gradient"):
            Engine.weigh(None, 0, 0, sel, **{"q": q, "lse": None, "fmt": latent_rows(), **kw})
    with pytest.raises(ValueError, match="shape"):
        Engine.weigh(None, 0, 0, sel, q[0], None, latent_rows())
    with pytest.raises(ValueError, match="CUDA"):
        Engine.weigh(None, 0, 0, sel, q, None, latent_rows())


def light_args(from_, to, n, **kw):
    a = ula.UlaLightestArgs()
    a.keep = [np.array(x, np.int32) for x in (from_, to, n)]
    a.first, a.last, a.count = (x.ctypes.data for x in a.keep)
    a.scores, a.capacity, a.ranges, a.most, a.out = P, 100000, len(from_), max(n, default=0), P
    for name, v in kw.items():
        setattr(a, name, v)
    return a


def test_lightest_refuses():
    L = ula.lib()
    call = lambda a: L.ula_lightest(ctypes.byref(a), 0)
    assert L.ula_lightest(None, 0) == EINVAL and L.ula_lightest_bytes(None) == 0
    one = ([3], [9], [2])
    for kw in [dict(ranges=-1), dict(most=-1), dict(capacity=-1), dict(mark=2), dict(mark=-1), dict(first=None), dict(last=None),
               dict(count=None), dict(most=1), dict(scores=None), dict(out=None), dict(scores=P + 4), dict(out=P + 2),
               dict(most=(1 << 31) - 1, ranges=1, count=None)]:
        assert call(light_args(*one, **kw)) == EINVAL, kw
    for bad, code in [(([3], [2], [0]), EINVAL), (([3], [9], [-1]), EINVAL), (([-1], [9], [1]), ERANGE),
                      (([3], [100001], [1]), ERANGE)]:
        a = light_args(*bad, most=4)
        assert call(a) == code and L.ula_lightest_bytes(ctypes.byref(a)) == 0, bad
    for ranges in [([0, 5], [6, 9], [1, 1]), ([5, 0], [9, 6], [1, 1]), ([0, 3, 2], [9, 4, 3], [1, 1, 1])]:
        assert call(light_args(*ranges, mark=1)) == EINVAL, ranges
    assert L.ula_lightest_bytes(ctypes.byref(light_args([0, 6, 6], [6, 6, 9], [1, 1, 1], mark=1))) == 0
    assert call(light_args([], [], [])) == 0 and call(light_args([3], [9], [0], out=None, scores=None)) == 0
    long = light_args([0, 0], [8192, 8193], [1, 1])
    need = L.ula_lightest_bytes(ctypes.byref(long))
    assert need == 2 * 2048 * 4 + 256 + -(-8193 * 8 // 256) * 256
    for kw in [dict(), dict(workspace=P, workspace_bytes=need - 1), dict(workspace=P + 16, workspace_bytes=need)]:
        for name, v in kw.items():
            setattr(long, name, v)
        assert call(long) == EINVAL, kw


def test_lightest_binding():
    scores = torch.zeros(100, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        lightest(scores, [0], [10], 2)
    for first, last, n in [([0, 1], [10], 2), ([0], [10], [1, 2]), ([0.5], [10], 1), ([1 << 40], [10], 1), ([[0]], [[10]], 1)]:
        with pytest.raises(ValueError, match="lightest"):
            lightest(scores, first, last, n)
