"""ula_norm_rotate against its formula in 64 bits.

Tolerance, from the arithmetic, with u = 2^-24: the sum of at most 256 squares runs in
chains of 8 fused steps and a tree of at most 6 (16 u of it), the mean's factor, its
product and eps's own rounding 3 u more, halved by the root; root and quotient
2 u each: the reciprocal is off by 14 u, and two products make 16 u of y (20 u are
taken). A turned value, p cos - q sin, is off by that of both, and by what
test_rows_gpu.py derives for the turn, on top. Then one rounding to the type: half a step."""

import numpy as np
import pytest

from test_rows_gpu import HALF, LEAST, assert_within, f64, on_gpu, positions_of, torch_type, turned, u

pytestmark = pytest.mark.gpu


def wanted(x, weight, eps, pos, sections, rotary, theta, interleaved, kind):
    """(exact, tolerance) of x [n][heads][dim]"""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
    if weight is not None:
        y = y * weight
    off = 20 * u * np.abs(y)
    if rotary:
        t, d = turned(y[..., :rotary], pos, sections, theta, interleaved)
        half = rotary // 2
        i0, i1 = (slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else (slice(0, half), slice(half, rotary))
        both = 20 * u * (np.abs(y[..., i0]) + np.abs(y[..., i1]))
        y, off = y.copy(), off.copy()
        off[..., :rotary] = d
        off[..., i0] += both
        off[..., i1] += both
        y[..., :rotary] = t
    return y, off + HALF[kind] * (np.abs(y) + off) + LEAST[kind]


# n, heads, kv heads, dim, rotary, axes, interleaved, type, weights, far positions: vectors and any even sizes,
# one token and many, no keys, no turn, every lane count
CASES = [
    (1, 1, 1, 128, 128, 1, False, "bf16", "same", False), (16, 32, 8, 128, 128, 1, False, "bf16", "same", False),
    (16, 40, 0, 64, 64, 1, True, "fp16", "fp32", True), (3, 5, 2, 256, 256, 2, False, "fp32", "none", False),
    (7, 3, 3, 192, 96, 3, True, "bf16", "fp32", True), (70, 12, 4, 96, 96, 1, False, "fp16", "same", False),
    (5, 2, 1, 2, 2, 1, False, "fp32", "same", False), (9, 3, 1, 6, 4, 1, True, "bf16", "same", False),
    (33, 4, 2, 100, 50, 2, False, "fp32", "fp32", True), (20, 1, 0, 254, 254, 1, True, "fp16", "none", False),
    (11, 6, 2, 8, 0, 1, False, "bf16", "fp32", False), (2100, 9, 3, 128, 64, 1, True, "bf16", "same", False),
    (4, 300, 20, 72, 24, 1, False, "fp16", "same", False), (1030, 1, 1, 40, 40, 3, False, "fp32", "same", False)]


@pytest.mark.parametrize("n,heads,kv,dim,rotary,axes,interleaved,kind,weights,far", CASES)
def test_against_the_formula(n, heads, kv, dim, rotary, axes, interleaved, kind, weights, far):
    import torch
    from serving_pb_lru_amd import norm_rotate
    print(f"norm n={n} heads={heads}/{kv} dim={dim} rotary={rotary} axes={axes} {kind} {weights}", flush=True)
    rng = np.random.default_rng([n, heads, dim, rotary])
    q = on_gpu(rng.standard_normal((n, heads, dim)) * 2.0 ** rng.integers(-4, 5, (n, heads, 1)), kind)
    k = on_gpu(rng.standard_normal((n, kv, dim)) * 2.0 ** rng.integers(-4, 5, (n, kv, 1)), kind) if kv else None
    wk = "fp32" if weights == "fp32" else kind
    w = [on_gpu(1 + 0.3 * rng.standard_normal(dim), wk) if weights != "none" else None for _ in range(2)]
    if not kv:
        w[1] = None
    pos = positions_of(rng, n, axes, far)
    half = rotary // 2
    sections = (half,) if axes == 1 else ((half // 4, half - half // 4) if axes == 2 else (half // 4, half // 3, half - half // 4 - half // 3))
    eps = 1e-5
    qo, ko = norm_rotate(q, k, *w, positions=torch.from_numpy(pos).cuda() if rotary else None, sections=sections if rotary else None,
                         theta=5000.0, interleaved=interleaved, rotary=rotary, eps=eps)
    assert (ko is None) == (kv == 0)
    for x, got, weight in ((q, qo, w[0]), (k, ko, w[1])):
        if x is not None:
            assert got.dtype == x.dtype and got.shape == x.shape and got.is_contiguous()
            y, tol = wanted(f64(x), None if weight is None else f64(weight), eps, pos, sections, rotary, 5000.0, interleaved, kind)
            assert_within(f64(got), y, tol)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary", [(64, 64), (128, 64), (192, 192)])
def test_strides_views_and_in_place_do_not_change_bits(dim, rotary, interleaved, kind):
    import torch
    from serving_pb_lru_amd import norm_rotate
    rng = np.random.default_rng([dim, rotary])
    n, heads, kv = 37, 6, 2
    whole = on_gpu(rng.standard_normal((n, heads + 2 * kv, dim)), kind)          # one projection's queries, keys and values
    q, k = whole[:, :heads], whole[:, heads:heads + kv]
    w = [on_gpu(1 + 0.3 * rng.standard_normal(dim), kind) for _ in range(2)]
    pos = torch.from_numpy(positions_of(rng, n, 1, False)).cuda()
    kw = dict(positions=pos, rotary=rotary, interleaved=interleaved)
    plain = norm_rotate(q.contiguous(), k.contiguous(), *w, **kw)
    view = norm_rotate(q, k, *w, **kw)
    apart = torch.zeros((heads, n, dim + 3), dtype=q.dtype, device="cuda")       # heads outermost, odd rows
    apart[..., 1:dim + 1] = q.transpose(0, 1)
    room = torch.full((n, kv, dim + 5), 3.0, dtype=q.dtype, device="cuda")
    odd = norm_rotate(apart[..., 1:dim + 1].transpose(0, 1), k, *w, out=(torch.empty_like(plain[0]), room[..., 3:dim + 3]), **kw)
    assert (room[..., :3] == 3).all() and (room[..., dim + 3:] == 3).all()
    alone = norm_rotate(q, None, w[0], **kw)[0]
    keys = norm_rotate(k, None, w[1], **kw)[0]
    rest = whole[:, heads + kv:].clone()
    here = norm_rotate(q, k, *w, out=(q, k), **kw)
    assert here[0] is q and here[1] is k and torch.equal(whole[:, heads + kv:], rest)
    for got in (view, odd, (alone, keys), here):
        assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])


@pytest.mark.parametrize("dim", [64, 6])
def test_rows_of_extreme_values(dim):
    """Zeros, values whose squares overflow or vanish, infinities and NaN: each row by itself."""
    import torch
    from serving_pb_lru_amd import norm_rotate
    rng = np.random.default_rng(3)
    x = rng.standard_normal((1, 8, dim)).astype(np.float32)
    x[0, 1] = 0
    x[0, 2] *= np.float32(2.0 ** 120)
    x[0, 3] *= np.float32(2.0 ** -120)
    x[0, 4, 3] = np.inf
    x[0, 5, 1] = np.nan
    x[0, 6] = np.float32(3e38)
    got = f64(norm_rotate(torch.from_numpy(x).cuda(), eps=1e-6)[0])
    with np.errstate(invalid="ignore", over="ignore"):
        want, tol = wanted(x.astype(np.float64), None, 1e-6, None, None, 0, 1.0, False, "fp32")
    want[0, 4] = 0
    want[0, 4, 3] = np.nan
    fine = ~np.isnan(want)
    assert np.array_equal(np.isnan(got), ~fine) and np.isnan(got[0, 5]).all()
    assert_within(got[fine], want[fine], np.where(np.isfinite(tol), tol, 0)[fine] + 2.0 ** -140)


def test_empty_calls_streams_and_graphs():
    import torch
    from serving_pb_lru_amd import norm_rotate
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    x = torch.randn((5, 3, 64), device="cuda").bfloat16()
    a, b = norm_rotate(x[:0], x[:0], positions=pos[:0])
    assert a.shape == b.shape == (0, 3, 64)
    assert norm_rotate(x[:, :0], x, positions=pos)[0].shape == (5, 0, 64)
    want = norm_rotate(x, positions=pos)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = norm_rotate(x, positions=pos, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm_rotate(x, positions=pos, out=(out, None))
    for i in range(3):
        x.normal_()
        pos += 1
        out.zero_()
        g.replay()
        assert torch.equal(out, norm_rotate(x, positions=pos)[0])
