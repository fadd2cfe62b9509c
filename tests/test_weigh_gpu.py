"""ula_weigh on both row formats against the 64-bit form of the formula.

Tolerance, with u = 2^-24. The exponent of a row's share, in the products' sums, is off
by what test_attend_gpu.py derives for a logit, 650 u R (R the largest sum of |q k|
|scale|) + 2^-22, and by the six fused steps from -lse to it, each at most u of
(|lse| + R) log2(e), twice more for lse times log2(e): 12 u (|lse| + R). That is the
share's relative error; the sum over rows adds rows u of it. Shares below 2^-126
vanish."""

import numpy as np
import pytest

import rows_ref as ref
from test_attend_gpu import engine_of, heads_rows_of, latent_rows_of, selection, torch_type
from test_tree_gpu import tokens_of

pytestmark = pytest.mark.gpu

u = 2.0 ** -24


def expected(fmt, rows, layer, sel, q, lse, scale):
    """64-bit (shares, their bounds); q [sets][rows per set][w] with heads innermost, lse [sets][rows]"""
    sets, k = sel.shape
    share, off = np.zeros((sets, k)), np.zeros((sets, k))
    block = 1 if fmt.kind == 0 else fmt.block_tokens
    for s in range(sets):
        live = sel[s] >= 0
        parts, used = tokens_of(fmt, rows[sel[s][live], layer])
        heads = q.shape[2]
        g = heads // len(parts)
        total, err = np.zeros(len(used)), np.zeros(len(used))
        for h, (keys, _) in enumerate(parts):
            x = q[s, :, h * g:(h + 1) * g].reshape(-1, q.shape[-1])
            l = lse[s, :, h * g:(h + 1) * g].reshape(-1)
            x, l = x[np.isfinite(l)], l[np.isfinite(l)]
            if len(l) == 0 or len(keys) == 0:
                continue
            w = np.exp(x @ keys.T * scale - l[:, None])
            reach = (np.abs(x) @ np.abs(keys[used]).T).max(-1, initial=0) * abs(scale)
            e = 650 * u * reach + 2.0 ** -22 + 12 * u * (np.abs(l) + reach) + q.shape[1] * heads * u
            total += w.sum(0)
            err += (w * e[:, None] + 2.0 ** -126).sum(0)
        total, err = np.where(used, total, 0).reshape(-1, block).sum(1), np.where(used, err, 0).reshape(-1, block).sum(1)
        share[s, live], off[s, live] = total, err + 16 * u * total
    return share, off


def units(share):
    return np.rint(np.clip(np.nan_to_num(share.astype(np.float64)), 0, 2.0 ** 22) * 2.0 ** 32).astype(np.int64)


def run(fmt, rows, layer, sel, shape, kind, rng, scale=None, off=()):
    """One attention and its weights; `off`: rows (node, head) left out by their lse."""
    import torch
    nodes, heads = shape
    eng = engine_of(rows, *sel.shape)
    try:
        dsel = torch.from_numpy(sel).cuda()
        width = 576 if fmt.kind == 0 else fmt.head_dim
        q = torch.from_numpy(rng.standard_normal((len(sel), nodes, heads, width))).to(torch_type(kind)).cuda()
        eng.step(0, dsel)
        lse = torch.cat([eng.attend(0, layer, dsel, q[:, t], fmt, scale=scale)[1][:, None] for t in range(nodes)], 1)
        for i, (t, h) in enumerate(off):
            lse[:, t, h] = (-np.inf, np.nan, np.inf)[i % 3]
            q[:, t, h] = np.nan
        n = len(rows)
        scores = torch.from_numpy(rng.integers(0, 1 << 40, n)).cuda()
        before = scores.cpu().numpy()
        got = eng.weigh(0, layer, dsel, q if nodes > 1 else q[:, 0], lse if nodes > 1 else lse[:, 0].contiguous(), fmt,
                        scores=scores, scale=scale)
        alone = eng.weigh(0, layer, dsel, q, lse, fmt, scale=scale)
        eng.sync()
        assert torch.equal(alone, got)
        share = got.cpu().numpy()
        want, tol = expected(fmt, rows, layer, sel, q.double().cpu().numpy(), lse.double().cpu().numpy(),
                             width ** -0.5 if scale is None else scale)
        over = np.abs(share - want) / np.maximum(tol, 1e-300)
        assert np.all((np.abs(share - want) <= tol)), f"worst {over.max():.3g} of the tolerance at {np.argwhere(over > 1)[:4].tolist()}"
        add = np.zeros(n, np.int64)
        np.add.at(add, sel[sel >= 0], units(share)[sel >= 0])
        assert np.array_equal(scores.cpu().numpy(), before + add)
        return share
    finally:
        eng.close()


# sets, k, nodes, heads, layers, layer, type, padding: rows at the edges of 32 and 64 and several chunks of them,
# keys at a group's edge (256), several groups of a workgroup, more than one takes (2048)
LATENT = [
    (1, 1, 1, 1, 1, 0, "bf16", 0), (2, 31, 1, 31, 1, 0, "bf16", 0), (2, 33, 1, 32, 3, 2, "fp16", 5),
    (1, 255, 1, 33, 1, 0, "bf16", 0), (1, 256, 1, 64, 2, 1, "fp16", 9), (2, 257, 1, 65, 1, 0, "bf16", 0),
    (3, 100, 1, 128, 1, 0, "fp16", 100), (1, 2300, 1, 16, 1, 0, "bf16", 0), (300, 600, 1, 20, 1, 0, "bf16", 31),
    (2, 70, 9, 16, 1, 0, "bf16", 3), (1, 300, 64, 5, 1, 0, "fp16", 0)]


@pytest.mark.parametrize("sets,k,nodes,heads,layers,layer,kind,pad", LATENT)
def test_latent_against_the_formula(sets, k, nodes, heads, layers, layer, kind, pad):
    from serving_pb_lru_amd import latent_rows
    print(f"weigh latent sets={sets} k={k} nodes={nodes} heads={heads} {kind} pad={pad}", flush=True)
    rng = np.random.default_rng([sets, k, nodes, heads])
    n = k + 40
    run(latent_rows(), latent_rows_of(rng, n, layers), layer, selection(rng, n, sets, k, pad), (nodes, heads), kind, rng,
        off=[(nodes - 1, 0)] if heads > 2 else ())


# sets, k, nodes, heads, kv heads, dim, block, type, padding, partly filled; rows per KV head either side of 16
HEADS = [
    (1, 1, 1, 1, 1, 64, 1, "bf16", 0, False), (2, 33, 1, 32, 8, 128, 1, "fp16", 4, False),
    (3, 31, 1, 24, 2, 64, 8, "bf16", 3, True), (1, 70, 1, 17, 1, 128, 8, "fp16", 0, True),
    (2, 64, 1, 40, 1, 64, 16, "bf16", 9, True), (1, 2100, 1, 6, 3, 64, 2, "fp16", 0, True),
    (5, 77, 11, 6, 2, 128, 2, "bf16", 77, False), (2, 130, 64, 4, 4, 64, 4, "fp16", 0, True),
    (40, 100, 1, 16, 1, 128, 1, "bf16", 17, False)]


@pytest.mark.parametrize("sets,k,nodes,heads,kv,dim,block,kind,pad,part", HEADS)
def test_heads_against_the_formula(sets, k, nodes, heads, kv, dim, block, kind, pad, part):
    from serving_pb_lru_amd import head_rows
    print(f"weigh heads sets={sets} k={k} nodes={nodes} heads={heads}/{kv} dim={dim} block={block} {kind}", flush=True)
    rng = np.random.default_rng([sets, k, nodes, heads, kv])
    n = k + 20
    counts = rng.integers(0, block + 1, n) if part else None
    rows = heads_rows_of(rng, n, 2, kv, dim, block, counts)
    if part:                                   # whatever lies behind the tokens in use
        for e in range(n):
            rows[e, :, :2 * kv * dim * block].reshape(2, 2, kv, block, dim)[:, :, :, counts[e]:] = 0x7F
    run(head_rows(kv, dim, block), rows, 1, selection(rng, n, sets, k, pad), (nodes, heads), kind, rng,
        off=[(0, 0), (nodes - 1, heads - 1)] if heads > 3 else ())


@pytest.mark.parametrize("name", ["latent", "heads"])
def test_shares_of_an_attention_add_up(name):
    """Over everything that a set attended to, each row's weights sum to 1; an address listed twice gets both."""
    import torch
    from serving_pb_lru_amd import head_rows, latent_rows
    fmt = latent_rows() if name == "latent" else head_rows(2, 64, 1)
    rng = np.random.default_rng(4)
    rows = latent_rows_of(rng, 300, 1) if name == "latent" else heads_rows_of(rng, 300, 1, 2, 64, 1)
    sel = selection(rng, 300, 4, 200, 11)
    sel[1] = sel[0]                            # two sets with the same addresses
    sel[2, 100:150] = sel[2, 20:70]            # a set with repeated ones
    share = run(fmt, rows, 0, sel, (1, 12), "bf16", rng)
    assert np.allclose(share.sum(1), 12, rtol=1e-4)
    assert np.array_equal(share[2, 100:150], share[2, 20:70])


@pytest.mark.parametrize("name", ["latent", "heads"])
def test_entries_that_hold_a_nan_add_nothing(name):
    import torch
    from serving_pb_lru_amd import head_rows, latent_rows
    fmt = latent_rows() if name == "latent" else head_rows(1, 64, 1)
    rng = np.random.default_rng(5)
    rows = latent_rows_of(rng, 40, 1) if name == "latent" else heads_rows_of(rng, 40, 1, 1, 64, 1)
    rows[7, 0, 5] = 0x7F
    sel = np.arange(40, dtype=np.int32)[None]
    eng = engine_of(rows, 1, 40)
    try:
        dsel = torch.from_numpy(sel).cuda()
        q = torch.from_numpy(rng.standard_normal((1, 5, 576 if fmt.kind == 0 else 64))).bfloat16().cuda()
        eng.step(0, dsel)
        scores = torch.zeros(40, dtype=torch.int64, device="cuda")
        share = eng.weigh(0, 0, dsel, q, torch.full((1, 5), 3.0, device="cuda"), fmt, scores=scores).cpu().numpy()[0]
        eng.sync()
        assert np.isnan(share[7]) and np.isfinite(np.delete(share, 7)).all()
        assert scores[7] == 0 and np.array_equal(scores.cpu().numpy(), units(share))
        # weights far above 1, from log-sums that are not these rows': the most that one call adds
        eng.weigh(0, 0, dsel, q, torch.full((1, 5), -80.0, device="cuda"), fmt, scores=scores.zero_())
        eng.sync()
        assert int(scores.max()) == 1 << 54 and int(scores.min()) == 0
    finally:
        eng.close()


def test_strides_streams_and_order():
    import torch
    from serving_pb_lru_amd import UlaError, latent_rows
    fmt = latent_rows()
    rng = np.random.default_rng(6)
    rows = latent_rows_of(rng, 600, 2)
    sel = torch.from_numpy(selection(rng, 600, 3, 400, 5)).cuda()
    q = torch.from_numpy(rng.standard_normal((3, 4, 10, 576))).to(torch.float16).cuda()
    eng = engine_of(rows, 3, 400)
    try:
        lse = torch.full((3, 4, 10), 6.5, device="cuda")
        with pytest.raises(UlaError) as e:
            eng.weigh(0, 0, sel, q, lse, fmt)
        assert e.value.name == "ENOTRESIDENT"
        eng.step(0, sel)
        first = eng.weigh(0, 1, sel, q, lse, fmt)
        wide = torch.zeros((10, 4, 3, 579), dtype=q.dtype, device="cuda")
        wide[..., 1:577] = q.permute(2, 1, 0, 3)
        out = torch.empty((3, 400), device="cuda")
        assert eng.weigh(0, 1, sel, wide[..., 1:577].permute(2, 1, 0, 3), lse, fmt, out=out) is out
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        scores = [torch.zeros(600, dtype=torch.int64, device="cuda") for _ in range(2)]
        side.wait_stream(torch.cuda.current_stream())
        other = eng.weigh(0, 1, sel, q, lse, fmt, scores=scores[0], stream=side)
        again = eng.weigh(0, 1, sel, q, lse, fmt, scores=scores[1])
        torch.cuda.current_stream().wait_stream(side)
        for x in (out, other, again):
            assert torch.equal(x, first)
        assert torch.equal(scores[0], scores[1])
        eng.sync()
    finally:
        eng.close()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("name", ["latent", "heads"])
def test_entries_of_infinite_logits(name, kind):
    """-infinity for every row that counts: no share. +infinity or NaN (0 x infinity) for one of them: infinite or NaN,
    of which the score takes 2^22 or nothing."""
    import torch
    from serving_pb_lru_amd import head_rows, latent_rows
    rng = np.random.default_rng(13)
    n, k, heads = 40, 33, 3
    rows = latent_rows_of(rng, n, 1) if name == "latent" else heads_rows_of(rng, n, 1, 1, 64, 1)
    fmt = latent_rows() if name == "latent" else head_rows(1, 64)
    sel = np.arange(k, dtype=np.int32)[None]
    if name == "latent":
        rows[5, 0, 512:514] = np.array([0x7F80], "<u2").view(np.uint8)
    else:
        rows[5, 0, :64] = 0
        rows[5, 0, 0] = 0x38
        rows[5, 0, 128:132] = np.array([np.inf], "<f4").view(np.uint8)
    for first, share in (((-1.0, -0.3, -2.0), 0.0), ((-1.0, 0.3, -2.0), np.inf), ((-1.0, 0.0, -2.0), np.nan)):
        q = torch.from_numpy(rng.standard_normal((1, heads, 576 if name == "latent" else 64))).to(torch_type(kind)).cuda()
        if name == "heads":
            q[..., 1:] = 0
        q[0, :, 512 if name == "latent" else 0] = torch.tensor(first).to(q.dtype).cuda()
        lse = torch.full((1, heads), 9.0, device="cuda")
        scores = torch.zeros(n, dtype=torch.int64, device="cuda")
        eng = engine_of(rows, 1, k)
        try:
            dsel = torch.from_numpy(sel).cuda()
            eng.step(0, dsel)
            got = eng.weigh(0, 0, dsel, q, lse, fmt, scores=scores).cpu().numpy()
            eng.sync()
        finally:
            eng.close()
        assert np.isfinite(np.delete(got, 5)).all()
        assert np.array_equal(got[0, 5], share, equal_nan=True)
        assert int(scores[5]) == {0.0: 0, np.inf: 1 << 54}.get(share, 0)


@pytest.mark.parametrize("name", ["latent", "heads"])
def test_rows_that_count_for_nothing_stay_out_whatever_an_entry_holds(name):
    """Entries with NaN codes and infinite scales in a call with no row of finite lse: shares of 0."""
    import torch
    from serving_pb_lru_amd import head_rows, latent_rows
    rng = np.random.default_rng(14)
    rows = latent_rows_of(rng, 40, 1) if name == "latent" else heads_rows_of(rng, 40, 1, 1, 64, 1)
    fmt = latent_rows() if name == "latent" else head_rows(1, 64)
    rows[5, 0, 3] = 0x7F
    at = 640 if name == "latent" else 128
    rows[9, 0, at:at + 4] = np.array([-np.inf], "<f4").view(np.uint8)
    eng = engine_of(rows, 1, 40)
    try:
        sel = torch.arange(40, dtype=torch.int32, device="cuda")[None]
        eng.step(0, sel)
        q = torch.from_numpy(rng.standard_normal((1, 40, 576 if name == "latent" else 64))).bfloat16().cuda()
        lse = torch.full((1, 40), float("nan"), device="cuda")
        assert not eng.weigh(0, 0, sel, q, lse, fmt).any()
        lse[0, 33] = 3.0
        some = eng.weigh(0, 0, sel, q, lse, fmt)
        lone = eng.weigh(0, 0, sel, q[:, 33:34], lse[:, 33:34].contiguous(), fmt)
        assert torch.allclose(some, lone, rtol=1e-5, atol=0, equal_nan=True) and bool(some[0, 5].isnan())
        eng.sync()
    finally:
        eng.close()
