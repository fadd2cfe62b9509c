"""ula_attend on both row formats against the 64-bit form of the formulas.

Tolerance, from the arithmetic (no slack for anything else). With w the exact
softmax weights, A = sum_j w_j |v_j| and u(t) half a step of type t (bf16 2^-8,
fp16 2^-11, fp32 2^-24):
  - each weight times value scale is rounded to fp16 once: u(fp16) A, and 2^-25 at
    the bottom of its range. There the reference is such that the largest weight
    times the largest value scale S is 2^6 or more in the units of the sums, so
    n tokens' codes of at most 448 are off by n 448 S 2^-25 / 2^6;
  - logits are sums of at most 512 + 2 x 64 products (one rounding each in 32 bits,
    and a few for the scales; fp16's rotary channels are two bf16 values each):
    off by d = 650 u(fp32) R, R the largest sum of |q k| |scale| of any logit, plus
    2^-22 for the base-2 exponent and its function; a logit's error changes every
    weight and their sum: 2 (d + 2^-22) A;
  - the sums over n tokens in 32 bits, numerator and denominator: 2 n u(fp32) A
    (n grows by 64 for the joins), and a handful of products: 8 u(fp32) A;
  - the result is rounded to its type once: u(type) |o| (2^-25 at the bottom of
    fp16's range, where steps no longer shrink).
lse: d + 2^-22 + (n + 70) u(fp32) and its own rounding, u(fp32) |lse| x 4.
"""

import numpy as np
import pytest

import rows_ref as ref

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


def torch_type(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def random_codes(rng, shape, spread=120.0):
    return ref.e4m3_nearest(np.clip(rng.standard_normal(shape) * spread, -448, 448))


def f32_bytes(x):
    return np.ascontiguousarray(x, dtype="<f4").view(np.uint8)


def latent_rows_of(rng, n, layers):
    rows = np.empty((n, layers, ref.LATENT_ROW), np.uint8)
    rows[..., :512] = random_codes(rng, (n, layers, 512))
    rope = rng.standard_normal((n, layers, 64)).astype(np.float32)
    rows[..., 512:640] = np.ascontiguousarray((rope.view(np.uint32) >> 16).astype("<u2")).view(np.uint8)
    rows[..., 640:] = f32_bytes(2.0 ** rng.standard_normal((n, layers, 4)) / 120)
    return rows


def heads_rows_of(rng, n, layers, kv, dim, block, counts=None):
    from serving_pb_lru_amd import head_rows
    rows = np.zeros((n, layers, head_rows(kv, dim, block).row_bytes), np.uint8)
    part = kv * dim * block
    rows[..., :2 * part] = random_codes(rng, (n, layers, 2 * part))
    rows[..., 2 * part:2 * part + 8 * kv] = f32_bytes(2.0 ** rng.standard_normal((n, layers, 2 * kv)) / 120)
    counts = np.full(n, block, "<i4") if counts is None else counts.astype("<i4")
    rows[..., 2 * part + 8 * kv:2 * part + 8 * kv + 4] = np.repeat(counts[:, None], layers, 1).view(np.uint8).reshape(n, layers, 4)
    return rows


def engine_of(rows, sets, k, **kw):
    from serving_pb_lru_amd import Engine
    n, layers, rb = rows.shape
    kw = {"gpu_slots": n, "host_slots": 0, **kw}
    eng = Engine(num_groups=1, layers=layers, row_bytes=rb, ring=4, logical_capacity=n, max_sets=sets,
                 max_k=max(k, 1), **kw)
    eng.append(0, np.arange(n, dtype=np.int32), rows)
    return eng


def value_scale(fmt, rows):
    """The largest finite value scale of any row."""
    at, n = (640, 4) if fmt.kind == 0 else (2 * fmt.kv_heads * fmt.head_dim * fmt.block_tokens + 4 * fmt.kv_heads, fmt.kv_heads)
    x = np.abs(ref.f32_at(rows, at, n))
    return np.where(np.isfinite(x), x, 0).max()


def expected(fmt, rows, layer, sel, q, scale):
    """64-bit (out, lse, bound of out, bound of lse), without the rounding to the type."""
    outs = []
    for s in range(sel.shape[0]):
        r = rows[sel[s][sel[s] >= 0], layer]
        if fmt.kind == 0:
            keys, values = ref.latent_kv(r)
            parts = [(slice(None), keys, values)]
            heads = q.shape[1]
        else:
            kk, vv, count = ref.heads_kv(r, fmt.kv_heads, fmt.head_dim, fmt.block_tokens)
            use = np.arange(fmt.block_tokens)[None] < count[:, None]
            g = q.shape[1] // fmt.kv_heads
            parts = [(slice(h * g, (h + 1) * g), kk[:, h][use], vv[:, h][use]) for h in range(fmt.kv_heads)]
        o = np.empty((q.shape[1], 512 if fmt.kind == 0 else fmt.head_dim))
        mag, lse, dl = np.empty_like(o), np.empty(q.shape[1]), np.empty(q.shape[1])
        n = 0
        for at, keys, values in parts:
            o[at], lse[at], mag[at], reach = ref.attention(q[s, at], keys, values, scale)
            dl[at] = 650 * U["fp32"] * reach + 2.0 ** -22
            n = max(n, len(keys))
        least = n * 448 * value_scale(fmt, rows[:, layer]) * 2.0 ** -31
        bound = mag * (U["fp16"] + 2 * dl[:, None] + (2 * (n + 64) + 8) * U["fp32"]) + least
        outs.append((o, lse, bound, dl + (n + 70) * U["fp32"] + 4 * U["fp32"] * np.abs(np.where(np.isinf(lse), 0, lse))))
    return [np.stack(x) for x in zip(*outs)]


def check(fmt, rows, layer, sel, q, scale, out, lse, kind):
    o, l, bo, bl = expected(fmt, rows, layer, sel, q.double().cpu().numpy(), scale)
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    tol = bo + (U[kind] * (np.abs(o) + bo)) + 2.0 ** -25
    bad = np.abs(got - o) > tol
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outputs off, worst by {np.max(np.abs(got - o) / tol):.3g} of the "
                           f"tolerance, first at {np.argwhere(bad)[:4].tolist()}")
    empty = np.isinf(l)
    assert np.array_equal(np.isneginf(glse), empty) and np.all(got[empty] == 0)
    assert np.all(np.abs(glse[~empty] - l[~empty]) <= bl[~empty]), np.max(np.abs(glse[~empty] - l[~empty]) - bl[~empty])


def run(fmt, rows, layer, sel, heads, kind, rng, scale=None, **kw):
    import torch
    eng = engine_of(rows, *sel.shape, **kw)
    try:
        dsel = torch.from_numpy(sel).cuda()
        width = 576 if fmt.kind == 0 else fmt.head_dim
        q = torch.from_numpy(rng.standard_normal((sel.shape[0], heads, width))).to(torch_type(kind)).cuda()
        eng.step(0, dsel)
        out, lse = eng.attend(0, layer, dsel, q, fmt, scale=scale)
        eng.sync()
        check(fmt, rows, layer, sel, q, width ** -0.5 if scale is None else scale, out, lse, kind)
    finally:
        eng.close()


def selection(rng, n, sets, k, pad=0):
    sel = np.stack([rng.choice(n, size=k, replace=k > n) for _ in range(sets)]).astype(np.int32).reshape(sets, k)
    if pad and k:
        for s in range(sets):
            sel[s, rng.choice(k, size=min(pad, k), replace=False)] = -1
    return sel


# sets, k, heads, layers, layer, type, padding: one token to several splits of one set (k > 2048),
# tile edges (31, 32, 33, 64, 65), head blocks (1, 16, 17, 32, 33, 64, 65, 128, 130)
LATENT_CASES = [
    (1, 1, 1, 1, 0, "bf16", 0), (1, 1, 128, 1, 0, "fp16", 0), (2, 31, 16, 1, 0, "bf16", 0),
    (2, 32, 17, 3, 1, "bf16", 0), (3, 33, 32, 3, 2, "fp16", 5), (1, 64, 33, 1, 0, "bf16", 0),
    (2, 65, 64, 2, 0, "fp16", 1), (1, 257, 65, 1, 0, "bf16", 100), (4, 256, 16, 1, 0, "bf16", 0),
    (1, 1000, 128, 1, 0, "fp16", 0), (1, 2048, 130, 1, 0, "bf16", 7), (1, 4100, 8, 1, 0, "bf16", 0),
    (300, 40, 20, 1, 0, "bf16", 3), (3, 129, 2, 1, 0, "fp16", 129), (70, 700, 40, 1, 0, "bf16", 11)]


@pytest.mark.parametrize("sets,k,heads,layers,layer,kind,pad", LATENT_CASES)
def test_latent_against_the_formula(sets, k, heads, layers, layer, kind, pad):
    from serving_pb_lru_amd import latent_rows
    print(f"latent sets={sets} k={k} heads={heads} layers={layers} layer={layer} {kind} pad={pad}", flush=True)
    rng = np.random.default_rng([sets, k, heads])
    n = max(600, min(k, 4500) + 100) if sets < 100 else 2000
    run(latent_rows(), latent_rows_of(rng, n, layers), layer, selection(rng, n, sets, k, pad), heads, kind, rng)


# sets, k, heads, kv heads, dim, block, type, padding, partly filled blocks
HEADS_CASES = [
    (1, 1, 1, 1, 64, 1, "bf16", 0, False), (1, 1, 8, 8, 128, 1, "fp16", 0, False),
    (2, 33, 32, 8, 128, 1, "bf16", 4, False), (3, 31, 24, 2, 64, 8, "fp16", 3, True),
    (1, 200, 17, 1, 128, 8, "bf16", 0, True), (2, 64, 20, 1, 64, 16, "bf16", 9, True),
    (1, 2100, 6, 3, 64, 2, "fp16", 0, True), (5, 77, 33, 3, 128, 2, "bf16", 77, True),
    (64, 300, 8, 4, 128, 1, "bf16", 17, False), (1, 4000, 4, 1, 128, 1, "fp16", 1, False)]


@pytest.mark.parametrize("sets,k,heads,kv,dim,block,kind,pad,part", HEADS_CASES)
def test_heads_against_the_formula(sets, k, heads, kv, dim, block, kind, pad, part):
    from serving_pb_lru_amd import head_rows
    print(f"heads sets={sets} k={k} heads={heads}/{kv} dim={dim} block={block} {kind} pad={pad} part={part}", flush=True)
    rng = np.random.default_rng([sets, k, heads, kv])
    n = k + 50 if k < 4500 else 4500
    counts = rng.integers(0, block + 1, n) if part else None
    rows = heads_rows_of(rng, n, 2, kv, dim, block, counts)
    if part:   # counts outside [0, block] count as the nearest end; codes and scales behind them may be anything
        used = head_rows(kv, dim, block)
        at = 2 * kv * dim * block + 8 * kv
        rows[0, :, at:at + 4] = np.array([block + 3], "<i4").view(np.uint8)
        rows[1, :, at:at + 4] = np.array([-2], "<i4").view(np.uint8)
        rows[1, :, :at] = 0xFF          # all NaN, scales too: nothing of it is in use
        assert used.row_bytes == rows.shape[2]
        for e in range(2, min(n, 40)):
            c = int(counts[e])
            kvv = rows[e, :, :2 * kv * dim * block].reshape(2, 2, kv, block, dim)
            kvv[:, :, :, c:] = 0x7F     # NaN codes behind the tokens in use
    run(head_rows(kv, dim, block), rows, 1, selection(rng, n, sets, k, pad), heads, kind, rng)
