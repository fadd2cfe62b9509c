"""ula_attend and ula_attend_tree where value scales rise or fall from tile to tile by many powers of two and every
token counts: the reference that follows weight times scale moves by more than 32 bits' range of exponents, and the
weights summed before the move must still be there after it.

Tolerances are those of test_attend_scales_gpu.py and test_tree_scales_gpu.py, of the same sums. Scales span
2^-60 .. 2^80 (2^-80 .. 2^80 for a tree over heads rows), the documented range; results are bf16, which holds them."""

import numpy as np
import pytest

import rows_ref as ref
from test_attend_gpu import U, engine_of, f32_bytes, heads_rows_of
from test_attend_scales_gpu import BITS, HEADS, check as attend_check, heads_case, latent_case
from test_tree_gpu import trees
from tree_plan import FORMS, heads_plan

pytestmark = pytest.mark.gpu

TILE, N = 32, 13 * 32 + 9                      # three tiles and more for each of a tree's four waves


def levels(order, low, high, n):
    """A power of two for each token: whole tiles of one scale, in `order`."""
    tiles = np.arange(n) // TILE
    count = tiles[-1] + 1
    if order == "rising":
        step = tiles / (count - 1)
    elif order == "falling":
        step = 1 - tiles / (count - 1)
    elif order == "up":                        # one step for every wave: its first tile low, the others high
        step = (tiles >= 4).astype(float)
    else:                                      # down and up again
        step = (tiles % 8 >= 4).astype(float)
    return low + np.rint(step * (high - low))


ORDERS = ["rising", "falling", "up", "waves"]


@pytest.mark.parametrize("name", ["latent", "heads"])
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("low,high", [(-30, 30), (-50, 50), (-60, 80)])
@pytest.mark.parametrize("against", [0.0, 0.1])
def test_attention(name, order, low, high, against):
    """Latent rows: sets enough to leave each its tiles in one workgroup; heads rows: three waves a set."""
    import torch
    from serving_pb_lru_amd import head_rows, latent_rows
    rng = np.random.default_rng([high, len(order), int(10 * against)])
    e = levels(order, low, high, N)
    rows = (latent_case if name == "latent" else heads_case)(
        rng, (-against * (e - (low + high) / 2) * BITS).astype(np.float32), np.repeat(2.0 ** e[:, None], 4, 1))
    sets = 300 if name == "latent" else 2
    fmt = latent_rows() if name == "latent" else head_rows(1, 64)
    sel = np.tile(np.arange(N, dtype=np.int32), (sets, 1))
    q = torch.zeros((sets, len(HEADS), 576 if name == "latent" else 64), dtype=torch.bfloat16, device="cuda")
    q[..., 512 if name == "latent" else 0] = torch.from_numpy(HEADS).to(q.dtype).cuda()
    eng = engine_of(rows, *sel.shape)
    try:
        d = torch.from_numpy(sel).cuda()
        eng.step(0, d)
        out, lse = eng.attend(0, 0, d, q, fmt, scale=1.0)
        eng.sync()
    finally:
        eng.close()
    assert (out == out[:1]).all() and (lse == lse[:1]).all()
    attend_check(fmt, rows, sel[:1], q[:1], out[:1], lse[:1], "bf16")


def tree_rows(dim, rng, logit, scales):
    """latent_case (dim None), or heads_case with a KV head of `dim`."""
    if dim is None:
        return latent_case(rng, logit, scales)
    rows = heads_rows_of(rng, len(logit), 1, 1, dim, 1)
    rows[:, 0, :dim] = 0
    rows[:, 0, 0] = 0x38
    rows[:, 0, 2 * dim:2 * dim + 4] = f32_bytes(logit[:, None])
    rows[:, 0, 2 * dim + 4:2 * dim + 8] = f32_bytes(scales[:, :1])
    return rows


# latent rows (whose scales count from 2^-60 on), and heads rows of both widths in every number of row groups
STEPS = [(-30, 30, 0.1), (-50, 50, 0.0), (-60, 80, 0.0), (-60, 80, 0.1)]
TREES = [(None, 0, 300, 4, *s) for s in STEPS] + [(*f, *s) for f in FORMS for s in STEPS + [(-80, 80, 0.0)]]


@pytest.mark.parametrize("dim,groups,sets,nodes,low,high,against", TREES)
@pytest.mark.parametrize("order", ORDERS)
def test_trees(dim, groups, sets, nodes, order, low, high, against):
    """A history in that order and drafted tokens of either end, the same in every set."""
    import torch
    from serving_pb_lru_amd import head_rows, latent_rows
    if dim:
        plan = heads_plan(sets, N, nodes, len(HEADS), 1, dim)
        assert plan.groups == groups and plan.splits == 1
    print(f"tree of {nodes} nodes, dim {dim}, {groups} groups, scales 2^{low}..2^{high} {order}", flush=True)
    rng = np.random.default_rng([high - low, len(order), int(10 * against), nodes])
    e = np.concatenate([levels(order, low, high, N), rng.choice([low, high], nodes)])
    all_rows = tree_rows(dim, rng, (-against * (e - (low + high) / 2) * BITS).astype(np.float32), np.repeat(2.0 ** e[:, None], 4, 1))
    rows, drafts = all_rows[:N], all_rows[N:]
    visible = trees(rng, 1, nodes)
    visible[:, 0] = 0
    fmt = head_rows(1, dim) if dim else latent_rows()
    q = torch.zeros((sets, nodes, len(HEADS), dim or 576), dtype=torch.bfloat16, device="cuda")
    q[..., 0 if dim else 512] = torch.from_numpy(HEADS).to(q.dtype).cuda()
    eng = engine_of(rows, sets, N)
    try:
        sel = torch.arange(N, dtype=torch.int32, device="cuda").repeat(sets, 1)
        eng.step(0, sel)
        out, lse = eng.attend_tree(0, 0, sel, q, fmt, torch.from_numpy(drafts).cuda().repeat(sets, 1, 1),
                                   torch.from_numpy(visible).cuda().repeat(sets, 1), scale=1.0)
        eng.sync()
    finally:
        eng.close()
    if dim:                                    # latent rows: the last sets are split, the others are not
        assert (out == out[:1]).all() and (lse == lse[:1]).all()
    x, u = q[0, 0].double().cpu().numpy(), U["fp32"]
    for t in range(nodes):
        r = np.concatenate([rows[:, 0], drafts[[j for j in range(nodes) if int(visible[0, t]) >> j & 1], 0]])
        n = len(r)
        if dim:
            kk, vv, _ = ref.heads_kv(r, 1, dim, 1)
            keys, values, scale = kk[:, 0, 0], vv[:, 0, 0], np.abs(ref.f32_at(r, 2 * dim + 4, 1))[:, 0]
        else:
            keys, values = ref.latent_kv(r)
            scale = np.abs(ref.f32_at(r, 640, 4)).max(-1)
        o, l, mag, reach = ref.attention(x, keys, values, 1.0)
        w = np.exp(x @ keys.T - l[:, None])
        d = 6 * u * reach + 2.0 ** -22
        least = n * 448 * 2.0 ** -32 * (w * scale).max(-1)
        if dim:
            d = d + np.log(2) * (2.0 ** -17 + 4 * u * (reach / np.log(2) + 80))
            least = least + 448 * 2.0 ** -80
        tol = mag * (2.0 ** -22 + 2 * d[:, None] + (2 * (n + 64) + 8) * u) + least[:, None]
        tol = tol + U["bf16"] * (np.abs(o) + tol) + 2.0 ** -133
        for s in (0, sets - 1):
            worst = (np.abs(out[s, t].double().cpu().numpy() - o) / tol).max(-1)
            assert np.all(worst <= 1), f"set {s} node {t}: off by {worst} of the tolerance, per head"
            off = np.abs(lse[s, t].double().cpu().numpy() - l)
            assert np.all(off <= d + (n + 74) * u + 4 * u * np.abs(l)), (s, t, off)
