"""ula_attend_tree on both row formats against the 64-bit form of the formulas.

Each node's result is the attention over the set's selected entries and the drafted
tokens that the node sees, so the tolerances are those of test_attend_gpu.py, derived
there, with the node's own number of tokens and the drafted rows' scales among the
others."""

import numpy as np
import pytest

import rows_ref as ref
from test_attend_gpu import (U, engine_of, heads_rows_of, latent_rows_of, selection, torch_type, value_scale)

pytestmark = pytest.mark.gpu


def trees(rng, sets, nodes):
    """Random trees: half of the nodes go on from the one before them."""
    from serving_pb_lru_amd import tree_masks
    parents = np.stack([[-1 if t == 0 or rng.random() < 0.1 else (t - 1 if rng.random() < 0.5 else int(rng.integers(0, t)))
                         for t in range(nodes)] for _ in range(sets)])
    return tree_masks(parents)


def tokens_of(fmt, rows, use=None):
    """[(heads part of kv, keys [tokens][w], values)] and which tokens of rows [n][bytes] are in use, [tokens]."""
    if fmt.kind == 0:
        keys, values = ref.latent_kv(rows)
        return [(keys, values)], np.ones(len(rows), bool)
    kk, vv, count = ref.heads_kv(rows, fmt.kv_heads, fmt.head_dim, fmt.block_tokens)
    used = (np.arange(fmt.block_tokens)[None] < count[:, None]).reshape(-1)
    flat = lambda x, h: x[:, h].reshape(-1, fmt.head_dim)
    return [(flat(kk, h), flat(vv, h)) for h in range(fmt.kv_heads)], used


def expected(fmt, rows, drafts, layer, sel, visible, q, scale):
    """64-bit (out, lse, bound of out, bound of lse), without the rounding to the type."""
    sets, nodes, heads = q.shape[:3]
    back = 512 if fmt.kind == 0 else fmt.head_dim
    per_set = len(drafts) // sets
    out, lse = np.zeros((sets, nodes, heads, back)), np.zeros((sets, nodes, heads))
    bo, bl = np.zeros_like(out), np.zeros_like(lse)
    big = max(value_scale(fmt, rows[:, layer]), value_scale(fmt, drafts[:, layer]))
    for s in range(sets):
        past, used = tokens_of(fmt, rows[sel[s][sel[s] >= 0], layer])
        new, fresh = tokens_of(fmt, drafts[s * per_set:(s + 1) * per_set, layer])
        for t in range(nodes):
            see = np.array([(int(visible[s, t]) >> j) & 1 == 1 and j < nodes for j in range(len(fresh))]) & fresh
            g = heads // len(past)
            for h, ((k0, v0), (k1, v1)) in enumerate(zip(past, new)):
                at = slice(h * g, (h + 1) * g)
                keys, values = np.concatenate([k0[used], k1[see]]), np.concatenate([v0[used], v1[see]])
                n = len(keys)
                o, l, mag, reach = ref.attention(q[s, t, at], keys, values, scale)
                d = 650 * U["fp32"] * reach + 2.0 ** -22
                out[s, t, at], lse[s, t, at] = o, l
                bo[s, t, at] = mag * (U["fp16"] + 2 * d[:, None] + (2 * (n + 64) + 8) * U["fp32"]) + n * 448 * big * 2.0 ** -31
                bl[s, t, at] = d + (n + 70) * U["fp32"] + 4 * U["fp32"] * np.abs(np.where(np.isinf(l), 0, l))
    return out, lse, bo, bl


def check(want, out, lse, kind):
    o, l, bo, bl = want
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    tol = bo + U[kind] * (np.abs(o) + bo) + 2.0 ** -25
    over = np.abs(got - o) / tol
    assert not (over > 1).any() and not np.isnan(got).any(), (
        f"{(over > 1).sum()} of {over.size} off, worst {np.nanmax(over):.3g}, first {np.argwhere(~(over <= 1))[:4].tolist()}")
    empty = np.isinf(l)
    assert np.array_equal(np.isneginf(glse), empty) and np.all(got[empty] == 0)
    assert np.all(np.abs(glse[~empty] - l[~empty]) <= bl[~empty]), np.max(np.abs(glse[~empty] - l[~empty]) - bl[~empty])


def run(fmt, rows, drafts, layer, sel, visible, heads, kind, rng, scale=None, shape=None):
    import torch
    eng = engine_of(rows, *sel.shape)
    try:
        dsel = torch.from_numpy(sel).cuda()
        width = 576 if fmt.kind == 0 else fmt.head_dim
        q = torch.from_numpy(rng.standard_normal((*visible.shape, heads, width))).to(torch_type(kind)).cuda()
        eng.step(0, dsel)
        out, lse = eng.attend_tree(0, layer, dsel, q, fmt, torch.from_numpy(drafts).cuda(),
                                   torch.from_numpy(visible).cuda(), scale=scale)
        eng.sync()
        check(expected(fmt, rows, drafts, layer, sel, visible, q.double().cpu().numpy(),
                       width ** -0.5 if scale is None else scale), out, lse, kind)
    finally:
        eng.close()


# sets, k, nodes, heads, layers, layer, type, padding: one node, whole trees (64), rows at the workgroups' edges
# (nodes x heads of 31..33, 63..65), history that ends inside a tile, none at all, several splits, all padding
LATENT_CASES = [
    (1, 1, 1, 1, 1, 0, "bf16", 0), (2, 31, 3, 11, 1, 0, "bf16", 0), (1, 32, 8, 4, 3, 2, "fp16", 0),
    (3, 33, 64, 1, 2, 1, "bf16", 5), (1, 0, 33, 2, 1, 0, "bf16", 0), (2, 100, 32, 3, 1, 0, "fp16", 0),
    (1, 257, 9, 7, 1, 0, "bf16", 200), (2, 64, 64, 5, 1, 0, "bf16", 64), (1, 2048, 5, 13, 1, 0, "bf16", 3),
    (1, 2048, 64, 2, 1, 0, "fp16", 0), (1, 4100, 13, 5, 1, 0, "bf16", 0), (40, 70, 4, 16, 1, 0, "bf16", 9),
    (6, 300, 16, 24, 1, 0, "fp16", 0)]


@pytest.mark.parametrize("sets,k,nodes,heads,layers,layer,kind,pad", LATENT_CASES)
def test_latent_against_the_formula(sets, k, nodes, heads, layers, layer, kind, pad):
    from serving_pb_lru_amd import latent_rows
    print(f"tree latent sets={sets} k={k} nodes={nodes} heads={heads} layers={layers} {kind} pad={pad}", flush=True)
    rng = np.random.default_rng([sets, k, nodes, heads])
    n = k + 50
    run(latent_rows(), latent_rows_of(rng, n, layers), latent_rows_of(rng, sets * nodes, layers), layer,
        selection(rng, n, sets, k, pad), trees(rng, sets, nodes), heads, kind, rng)


# sets, k, nodes, heads, kv heads, dim, block, type, padding, partly filled blocks; rows per KV head either side of
# 16, 32 and 64
HEADS_CASES = [
    (1, 1, 1, 1, 1, 64, 1, "bf16", 0, False), (2, 33, 5, 24, 8, 128, 1, "bf16", 4, False),
    (3, 31, 11, 6, 2, 64, 8, "fp16", 3, True), (1, 200, 17, 2, 1, 128, 8, "bf16", 0, True),
    (2, 64, 33, 2, 1, 64, 16, "bf16", 9, True), (1, 2100, 7, 6, 3, 64, 2, "fp16", 0, True),
    (2, 0, 64, 3, 3, 128, 2, "bf16", 0, True), (8, 300, 16, 8, 4, 128, 1, "bf16", 17, False),
    (1, 4000, 64, 4, 1, 128, 1, "fp16", 1, False), (5, 77, 61, 12, 2, 64, 4, "fp16", 77, False)]


@pytest.mark.parametrize("sets,k,nodes,heads,kv,dim,block,kind,pad,part", HEADS_CASES)
def test_heads_against_the_formula(sets, k, nodes, heads, kv, dim, block, kind, pad, part):
    from serving_pb_lru_amd import head_rows
    print(f"tree heads sets={sets} k={k} nodes={nodes} heads={heads}/{kv} dim={dim} block={block} {kind} pad={pad}", flush=True)
    rng = np.random.default_rng([sets, k, nodes, heads, kv])
    n, per_set = k + 20, -(-nodes // block)
    counts = rng.integers(0, block + 1, n) if part else None
    left = np.tile(np.minimum(nodes - np.arange(per_set) * block, block), sets)
    if part:                                  # a tree's block may be partly filled anywhere
        left = np.where(rng.random(len(left)) < 0.3, rng.integers(0, block + 1, len(left)), left)
    run(head_rows(kv, dim, block), heads_rows_of(rng, n, 2, kv, dim, block, counts),
        heads_rows_of(rng, sets * per_set, 2, kv, dim, block, left), 1, selection(rng, n, sets, k, pad),
        trees(rng, sets, nodes), heads, kind, rng)


# sets that fill the compute units stay whole and the others are split: the last ones of many, strided results
@pytest.mark.parametrize("sets,k,nodes,heads,kind,pad", [(257, 1500, 1, 20, "bf16", 0), (260, 300, 2, 16, "fp16", 40),
                                                         (17, 400, 64, 16, "bf16", 0)])
def test_whole_sets_beside_split_ones(sets, k, nodes, heads, kind, pad):
    import ctypes
    import torch
    from serving_pb_lru_amd import latent_rows, ula
    fmt, rng = latent_rows(), np.random.default_rng([sets, k, nodes])
    need = ula.lib().ula_attend_tree_bytes(ctypes.byref(fmt), sets, k, nodes, heads)
    assert 0 < need < sets * nodes * heads * 2 * 513 * 4          # less than two parts of every row
    rows, drafts = latent_rows_of(rng, k + 50, 1), latent_rows_of(rng, sets * nodes, 1)
    sel, visible = selection(rng, k + 50, sets, k, pad), trees(rng, sets, nodes)
    q = torch.from_numpy(rng.standard_normal((sets, nodes, heads, 576))).to(torch_type(kind)).cuda()
    room = torch.full((heads, sets, nodes, 520), 7.0, dtype=q.dtype, device="cuda")
    out, lse = call(fmt, rows, drafts, sel, visible, q, out=room[..., :512].permute(1, 2, 0, 3))
    check(expected(fmt, rows, drafts, 0, sel, visible, q.double().cpu().numpy(), 576 ** -0.5), out, lse, kind)
    assert (room[..., 512:] == 7).all()


def formats():
    from serving_pb_lru_amd import head_rows, latent_rows
    return {"latent": latent_rows(), "heads": head_rows(2, 64, 4), "heads128": head_rows(1, 128, 1)}


def some(fmt, rng, n, layers=1):
    if fmt.kind == 0:
        return latent_rows_of(rng, n, layers)
    return heads_rows_of(rng, n, layers, fmt.kv_heads, fmt.head_dim, fmt.block_tokens)


def call(fmt, rows, drafts, sel, visible, q, **kw):
    import torch
    eng = engine_of(rows, *sel.shape)
    try:
        dsel = torch.from_numpy(sel).cuda()
        eng.step(0, dsel)
        out, lse = eng.attend_tree(0, 0, dsel, q, fmt, torch.from_numpy(drafts).cuda(), torch.from_numpy(visible).cuda(), **kw)
        eng.sync()
        return out, lse
    finally:
        eng.close()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("name", ["latent", "heads", "heads128"])
def test_nodes_that_see_nothing(name, kind):
    """Empty masks, in sets with a history and in a set of padding; bits behind the last node are not looked at."""
    fmt = formats()[name]
    rng = np.random.default_rng(5)
    sets, k, nodes, heads = 3, 40, 7, 4
    rows = some(fmt, rng, 60)
    per_set = -(-nodes // (1 if fmt.kind == 0 else fmt.block_tokens))
    drafts = some(fmt, rng, sets * per_set)
    sel = selection(rng, 60, sets, k)
    sel[1] = -1
    visible = trees(rng, sets, nodes)
    visible[:, 3] = 0
    visible[1, 5] = 0
    visible |= np.int64(-1) << np.int64(nodes)                # all the bits that name no node
    import torch
    width = 576 if fmt.kind == 0 else fmt.head_dim
    q = torch.from_numpy(rng.standard_normal((sets, nodes, heads, width))).to(torch_type(kind)).cuda()
    out, lse = call(fmt, rows, drafts, sel, visible, q)
    check(expected(fmt, rows, drafts, 0, sel, visible, q.double().cpu().numpy(), width ** -0.5), out, lse, kind)
    empty = torch.zeros((sets, nodes), dtype=torch.bool)
    empty[1, 3] = empty[1, 5] = True
    assert torch.equal(torch.isneginf(lse).all(-1).cpu(), empty) and (out[empty.cuda()] == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("name", ["latent", "heads", "heads128"])
def test_what_a_drafted_row_holds_reaches_those_who_see_it(name, kind):
    """NaN codes, scales and keys that are not finite in drafted rows: nodes that do not see them keep
    their bits, the others' heads are NaN."""
    import torch
    fmt = formats()[name]
    rng = np.random.default_rng(6)
    sets, k, nodes, heads = 2, 50, 40, 4
    rows = some(fmt, rng, 60)
    block = 1 if fmt.kind == 0 else fmt.block_tokens
    per_set = -(-nodes // block)
    drafts = some(fmt, rng, sets * per_set)
    sel = selection(rng, 60, sets, k)
    visible = trees(rng, sets, nodes)
    visible[:, 0] = 1                                         # one node that sees itself alone
    bad = [3, 17, 33] if block == 1 else [12, 36]             # the first token of a block
    for j in bad:
        for t in range(nodes):
            if t >= 1 and t % 3 == 0:
                visible[:, t] |= np.int64(1) << np.int64(j)
            elif t not in bad:
                visible[:, t] &= ~(np.int64((1 << block) - 1) << np.int64(j))
    width = 576 if fmt.kind == 0 else fmt.head_dim
    q = torch.from_numpy(rng.standard_normal((sets, nodes, heads, width))).to(torch_type(kind)).cuda()
    clean, lclean = call(fmt, rows, drafts, sel, visible, q)
    part = 0 if fmt.kind == 0 else fmt.kv_heads * fmt.block_tokens * fmt.head_dim
    nan, inf = np.array([np.nan], "<f4").view(np.uint8), np.array([-np.inf], "<f4").view(np.uint8)

    def spoil_code(r):
        if fmt.kind == 0:
            r[77] = 0x7F
        else:
            for h in range(fmt.kv_heads):                     # a value of the block's first token, every KV head
                r[part + h * fmt.block_tokens * fmt.head_dim + 9] = 0xFF

    def spoil_scale(r):
        if fmt.kind == 0:
            r[644:648] = inf
        else:
            for h in range(fmt.kv_heads):
                r[2 * part + 4 * (fmt.kv_heads + h):][:4] = nan

    def spoil_key(r):
        if fmt.kind == 0:
            r[512:514] = np.array([0x7FC0], "<u2").view(np.uint8)
        else:
            for h in range(fmt.kv_heads):
                r[h * fmt.block_tokens * fmt.head_dim + 5] = 0x7F

    for spoil in (spoil_code, spoil_scale, spoil_key):
        rough = drafts.copy()
        for s in range(sets):
            for j in bad:
                spoil(rough[s * per_set + j // block, 0])
        out, lse = call(fmt, rows, rough, sel, visible, q)
        whole = spoil is spoil_scale and block > 1            # a scale belongs to the whole block
        hit = np.zeros((sets, nodes), bool)
        for j in bad:
            m = (1 << (block if whole else 1)) - 1
            hit |= (visible >> j & m) != 0
        assert hit.any() and not hit.all()
        hit = torch.from_numpy(hit).cuda()
        assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all(), spoil.__name__
        assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], lclean[~hit]), spoil.__name__


@pytest.mark.parametrize("name", ["latent", "heads", "heads128"])
def test_strides_and_alignment_do_not_change_bits(name):
    import torch
    fmt = formats()[name]
    rng = np.random.default_rng(7)
    sets, k, nodes, heads = 2, 300, 9, 6
    rows = some(fmt, rng, 320)
    per_set = -(-nodes // (1 if fmt.kind == 0 else fmt.block_tokens))
    drafts = some(fmt, rng, sets * per_set)
    sel, visible = selection(rng, 320, sets, k, 4), trees(rng, sets, nodes)
    width, back = (576, 512) if fmt.kind == 0 else (fmt.head_dim,) * 2
    q = torch.from_numpy(rng.standard_normal((sets, nodes, heads, width))).bfloat16().cuda()
    plain, lse = call(fmt, rows, drafts, sel, visible, q)
    wide = torch.zeros((heads, sets, nodes, width + 3), dtype=q.dtype, device="cuda")      # heads outermost, rows apart
    wide[..., 1:width + 1] = q.permute(2, 0, 1, 3)
    view = wide[..., 1:width + 1].permute(1, 2, 0, 3)
    room = torch.full((nodes, heads, sets, back + 5), 7.0, dtype=q.dtype, device="cuda")
    out = room[..., 2:back + 2].permute(2, 0, 1, 3)
    got, l2 = call(fmt, rows, drafts, sel, visible, view, out=out)
    assert got is out and torch.equal(out, plain) and torch.equal(l2, lse)
    assert (room[..., :2] == 7).all() and (room[..., back + 2:] == 7).all()


@pytest.mark.parametrize("name", ["latent", "heads128"])
def test_a_chain_is_an_attention_over_its_appended_tokens(name):
    """What verifying a drafted chain gives is, to rounding, what a plain attention gives once the tokens are appended."""
    import torch
    fmt = formats()[name]
    rng = np.random.default_rng(8)
    k, nodes, heads = 90, 6, 8
    rows, drafts = some(fmt, rng, 90), some(fmt, rng, nodes)
    width = 576 if fmt.kind == 0 else fmt.head_dim
    q = torch.from_numpy(rng.standard_normal((1, nodes, heads, width))).to(torch.float16).cuda()
    sel = np.arange(k, dtype=np.int32)[None]
    visible = np.array([[(1 << (t + 1)) - 1 for t in range(nodes)]], np.int64)
    out, lse = call(fmt, rows, drafts, sel, visible, q)
    want = expected(fmt, rows, drafts, 0, sel, visible, q.double().cpu().numpy(), width ** -0.5)
    both = np.concatenate([rows, drafts])
    eng = engine_of(both, nodes, k + nodes)
    try:
        each = np.full((nodes, k + nodes), -1, np.int32)
        for t in range(nodes):
            each[t, :k + t + 1] = np.arange(k + t + 1)
        dsel = torch.from_numpy(each).cuda()
        eng.step(0, dsel)
        o2, l2 = eng.attend(0, 0, dsel, q[0], fmt)
        eng.sync()
    finally:
        eng.close()
    check(want, out, lse, "fp16")
    check(want, o2[None], l2[None], "fp16")


def test_same_call_same_bits_and_other_streams():
    import torch
    from serving_pb_lru_amd import UlaError, latent_rows
    fmt = latent_rows()
    rng = np.random.default_rng(9)
    rows, drafts = latent_rows_of(rng, 500, 1), torch.from_numpy(latent_rows_of(rng, 2 * 12, 1)).cuda()
    sel = torch.from_numpy(selection(rng, 500, 2, 400)).cuda()
    visible = torch.from_numpy(trees(rng, 2, 12)).cuda()
    q = torch.from_numpy(rng.standard_normal((2, 12, 10, 576))).bfloat16().cuda()
    eng = engine_of(rows, 2, 400)
    try:
        with pytest.raises(UlaError) as e:
            eng.attend_tree(0, 0, sel, q, fmt, drafts, visible)
        assert e.value.name == "ENOTRESIDENT"
        eng.step(0, sel)
        first = eng.attend_tree(0, 0, sel, q, fmt, drafts, visible)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = eng.attend_tree(0, 0, sel, q, fmt, drafts, visible, stream=side)
        again = eng.attend_tree(0, 0, sel, q, fmt, drafts, visible)
        torch.cuda.current_stream().wait_stream(side)
        for a, b in ((first, other), (first, again)):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        eng.sync()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            g.capture_begin()
            try:
                with pytest.raises(UlaError) as e:
                    eng.attend_tree(0, 0, sel, q, fmt, drafts, visible)
                assert e.value.name == "EINVAL"
            finally:
                g.capture_end()
        torch.cuda.synchronize()
        eng.sync()
    finally:
        eng.close()
