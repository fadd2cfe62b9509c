"""ula_attend_tree where value scales and logits pull apart, a third of a tree's tokens drafted: the cases of
test_attend_scales_gpu.py, and over heads rows scales of either sign over the whole range, 0 and not finite.

Tolerance. As there; over heads rows log2 |scale| is a term of the exponent: a logarithm of at most 80 in 32 bits,
off by a step of 2^-17, and four sums with it (to the logit, from the reference, and both again where l is added up
from them), each rounding (R log2(e) + 80) once: d gains ln 2 (2^-17 + 4 u (R log2(e) + 80)), R the largest |logit|. A
scale below 2^-80 counts as 0: 448 2^-80 of a weight."""

import numpy as np
import pytest

import rows_ref as ref
from test_attend_gpu import U, engine_of, f32_bytes, heads_rows_of, torch_type
from test_attend_scales_gpu import BITS, HEADS, heads_case, latent_case, orders_of
from test_tree_gpu import trees

pytestmark = pytest.mark.gpu


def check(name, rows, drafts, sel, visible, q, out, lse, kind):
    for s in range(len(sel)):
        for t in range(visible.shape[1]):
            see = [j for j in range(len(drafts) // len(sel)) if int(visible[s, t]) >> j & 1]
            r = np.concatenate([rows[sel[s][sel[s] >= 0], 0], drafts[s * len(drafts) // len(sel):][see, 0]])
            n, x = len(r), q[s, t].double().cpu().numpy()
            if name == "latent":
                keys, values = ref.latent_kv(r)
                scale = np.abs(ref.f32_at(r, 640, 4)).max(-1)
            else:
                kk, vv, _ = ref.heads_kv(r, 1, 64, 1)
                keys, values = kk[:, 0, 0], vv[:, 0, 0]
                scale = np.abs(ref.f32_at(r, 132, 1))[:, 0]
            o, l, mag, reach = ref.attention(x, keys, values, 1.0)
            w = np.exp(x @ keys.T - l[:, None])
            least = n * 448 * 2.0 ** -32 * (w * np.maximum(scale, 2.0 ** -60)).max(-1)
            d = 6 * U["fp32"] * reach + 2.0 ** -22
            if name == "heads":
                d = d + np.log(2) * (2.0 ** -17 + 4 * U["fp32"] * (reach / np.log(2) + 80))
                least = n * 448 * 2.0 ** -32 * (w * scale).max(-1) + 448 * 2.0 ** -80
            tol = mag * (U["fp16"] + 2 * d[:, None] + (2 * (n + 64) + 8) * U["fp32"]) + least[:, None]
            tol = tol + U[kind] * (np.abs(o) + tol) + (2.0 ** -25 if kind == "fp16" else 2.0 ** -133)
            worst = (np.abs(out[s, t].double().cpu().numpy() - o) / tol).max(-1)
            assert np.all(worst <= 1), f"set {s} node {t}: off by {worst} of the tolerance, per head"
            off = np.abs(lse[s, t].double().cpu().numpy() - l)
            assert np.all(off <= d + (n + 74) * U["fp32"] + 4 * U["fp32"] * np.abs(l)), (s, t, off)


def call(name, rows, drafts, sel, visible, q):
    import torch
    from serving_pb_lru_amd import head_rows, latent_rows
    eng = engine_of(rows, *sel.shape)
    try:
        d = torch.from_numpy(sel).cuda()
        eng.step(0, d)
        out, lse = eng.attend_tree(0, 0, d, q, latent_rows() if name == "latent" else head_rows(1, 64),
                                   torch.from_numpy(drafts).cuda(), torch.from_numpy(visible).cuda(), scale=1.0)
        eng.sync()
        return out, lse
    finally:
        eng.close()


def queries(name, sets, nodes, kind):
    import torch
    q = torch.zeros((sets, nodes, len(HEADS), 576 if name == "latent" else 64), dtype=torch_type(kind), device="cuda")
    q[..., 512 if name == "latent" else 0] = torch.from_numpy(HEADS).to(q.dtype).cuda()
    return q


def run(name, logit, scales, kind, rng, blank=()):
    """Every order's first two thirds are selected, the rest drafted."""
    all_rows = (latent_case if name == "latent" else heads_case)(rng, logit, scales)
    all_rows[list(blank), 0, :512 if name == "latent" else 0] = 0
    if name == "heads":
        all_rows[list(blank), 0, 64:128] = 0
    orders = np.stack(orders_of(rng, len(logit)))
    k = 2 * len(logit) // 3
    sel, nodes = orders[:, :k].astype(np.int32), orders.shape[1] - k
    drafts = all_rows[orders[:, k:].reshape(-1)]
    visible = trees(rng, len(orders), nodes)
    visible[:, -1] = (1 << nodes) - 1
    visible[:, 0] = 0
    q = queries(name, len(orders), nodes, kind)
    out, lse = call(name, all_rows, drafts, sel, visible, q)
    check(name, all_rows, drafts, sel, visible, q, out, lse, kind)


@pytest.mark.parametrize("name", ["latent", "heads"])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("spread", [0, 25, 60])
@pytest.mark.parametrize("against", [0.5, 1.0, 2.0])
def test_scales_against_logits(name, kind, spread, against):
    rng = np.random.default_rng([spread, int(2 * against)])
    n = 97
    e = rng.uniform(-spread, 0, n)
    e[:8] = [0, -spread] * 4
    run(name, (-against * (e + spread / 2) * BITS).astype(np.float32), 2.0 ** np.repeat(e[:, None], 4, 1) / 512, kind, rng)


@pytest.mark.parametrize("name", ["latent", "heads"])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("ahead", [0, 25, 50])
def test_rows_of_zeros_with_most_of_the_weight(name, kind, ahead):
    rng = np.random.default_rng(ahead)
    scales = 2.0 ** rng.standard_normal((70, 4)) / 8
    logit = (rng.standard_normal(70) * 0.5).astype(np.float32)
    blank = [0, 9, 33, 34, 69]
    scales[blank] = 2.0 ** -126
    logit[blank] = ahead * BITS
    run(name, logit, scales, kind, rng, blank)


@pytest.mark.parametrize("against", [-0.5, 0.0, 1.0])
@pytest.mark.parametrize("low,high", [(-80, 80), (-3, 3), (-79, -61), (41, 80)])
def test_scales_of_either_sign_over_the_whole_range(low, high, against):
    """With a few that are 0 or too small to count."""
    rng = np.random.default_rng([100 + low, high % 1000, int(4 + 2 * against)])
    n = 97
    e = rng.uniform(low, high, n)
    scales = np.repeat((np.where(rng.random(n) < 0.4, -1, 1) * 2.0 ** e)[:, None], 4, 1)
    scales[[5, 50]] = 0
    scales[[6, 70]] = 2.0 ** -90
    scales[[7, 90]] = -2.0 ** -126
    run("heads", (-against * (e - (low + high) / 2) * BITS).astype(np.float32), scales, "bf16", rng)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_scales_that_are_not_finite(bad):
    """Of tokens out of use they reach nothing; of a selected entry, its own set alone."""
    import torch
    rng = np.random.default_rng(11)
    sets, k, nodes = 3, 70, 9
    rows, drafts = heads_rows_of(rng, 80, 1, 1, 64, 1), heads_rows_of(rng, sets * nodes, 1, 1, 64, 1)
    sel = np.stack([rng.permutation(79)[:k] for _ in range(sets)]).astype(np.int32)
    visible = trees(rng, sets, nodes)
    q = queries("heads", sets, nodes, "bf16")
    none = np.zeros(1, "<i4").view(np.uint8)
    unused, spare = sel[0, 12], drafts.copy()
    rows[unused, 0, 136:140] = none
    spare[4, 0, 136:140] = none
    clean, lclean = call("heads", rows, spare, sel, visible, q)
    for r in (rows[unused, 0], spare[4, 0]):
        r[128:136] = f32_bytes(np.full(2, bad))
        r[:128] = 0x7F
    out, lse = call("heads", rows, spare, sel, visible, q)
    assert not torch.isnan(out).any() and torch.equal(out, clean) and torch.equal(lse, lclean)
    sel[1, 33], sel[[0, 2]] = 79, np.where(sel[[0, 2]] == 79, 78, sel[[0, 2]])
    sel[1, 34:] = -1
    rows[79, 0, 132:136] = f32_bytes(np.full(1, bad))
    out, lse = call("heads", rows, spare, sel, visible, q)
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert torch.equal(out[[0, 2]], clean[[0, 2]]) and torch.equal(lse[[0, 2]], lclean[[0, 2]])


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("name", ["latent", "heads"])
@pytest.mark.parametrize("drafted", [False, True])
def test_logits_of_infinity(name, kind, drafted):
    """+infinity (heads 0 and 1) and NaN (head 3, of 0 x infinity) make a head NaN for the nodes that see the token;
    -infinity (head 2) has no weight: that head is as if the token were not there."""
    import torch
    rng = np.random.default_rng(12)
    sets, k, nodes = 2, 300, 20
    case = latent_case if name == "latent" else heads_case
    rows = case(rng, rng.standard_normal(320).astype(np.float32), 2.0 ** rng.standard_normal((320, 4)) / 8)
    drafts = case(rng, rng.standard_normal(sets * nodes).astype(np.float32), 2.0 ** rng.standard_normal((sets * nodes, 4)) / 8)
    sel = np.stack([rng.permutation(319)[:k] for _ in range(sets)]).astype(np.int32)
    visible = trees(rng, sets, nodes)
    without, at = sel.copy(), visible.copy()
    if drafted:
        at[0] &= ~np.int64(1 << 7)
    else:
        sel[0, 150], without[0, 150] = 319, -1
    q = queries(name, sets, nodes, kind)
    clean, lclean = call(name, rows, drafts, without, at, q)
    for r in ([drafts[7, 0]] if drafted else [rows[319, 0]]):
        if name == "latent":
            r[512:514] = np.array([0x7F80], "<u2").view(np.uint8)
        else:
            r[128:132] = f32_bytes(np.full(1, np.inf))
    out, lse = call(name, rows, drafts, sel, visible, q)
    hit = torch.zeros((sets, nodes), dtype=torch.bool)
    hit[0] = torch.from_numpy((visible[0] >> 7 & 1) == 1) if drafted else True
    assert hit.any() and not hit.all()
    for h in (0, 1, 3):
        assert torch.isnan(out[:, :, h]).all(-1).cpu().equal(hit) and torch.isnan(lse[:, :, h]).cpu().equal(hit)
    rest = (~hit).cuda()
    assert torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], lclean[rest])
    assert torch.equal(out[:, :, 2], clean[:, :, 2]) and torch.equal(lse[:, :, 2], lclean[:, :, 2])
