"""ula_attend where value scales and logits pull apart: a key of large weight and small scale beside
keys of small weight and large scale, in several orders inside a tile.

Tolerance. Weight times value scale is rounded to fp16 in units in which the set's largest product of
the two is 2^7 or more, a scale below 2^-60 counting as that. So it is off by 2^-11 of itself, and at
the bottom of fp16's range by 2^-25, which is 2^-32 of the largest: n tokens' codes of at most 448 add
n 448 2^-32 max_j(w_j max(s_j, 2^-60)). Nothing is allowed for rows that have no weight.
A logit here is one product of two 16-bit values (every other channel of q is 0), exact in 32 bits. The
factor scale log2(e), its product and the difference from the reference round once each, the
key scale (heads rows) twice: off by d = 6 u(fp32) R, R the largest |logit|, + 2^-22 for the function.
The rest is as in the formula's tests.
"""

import numpy as np
import pytest

import rows_ref as ref
from test_attend_gpu import U, engine_of, f32_bytes, heads_rows_of, latent_rows_of, torch_type

pytestmark = pytest.mark.gpu

ONE = 0x38                                             # e4m3 code of 1
BITS = np.log(2.0)
HEADS = np.array([1.0, 0.5, -1.0, 0.0])                # channel 0 of the heads' queries


def bf16(x):
    return (np.asarray(x, np.float32).view(np.uint32) + 0x8000 >> 16 << 16).view(np.float32)


def latent_case(rng, logit, scales):
    """Rows whose logit is `logit` times the query's first rotary channel, with value scales [n][4]."""
    rows = latent_rows_of(rng, len(logit), 1)
    rows[:, 0, 640:] = f32_bytes(scales)
    rope = np.zeros((len(logit), 64), np.float32)
    rope[:, 0] = bf16(logit)
    rows[:, 0, 512:640] = np.ascontiguousarray((rope.view(np.uint32) >> 16).astype("<u2")).view(np.uint8)
    return rows


def heads_case(rng, logit, scales):
    """The same with one KV head of 64: the first key channel is 1 and the key scale the logit."""
    rows = heads_rows_of(rng, len(logit), 1, 1, 64, 1)
    rows[:, 0, :64] = 0
    rows[:, 0, 0] = ONE
    rows[:, 0, 128:132] = f32_bytes(logit[:, None])
    rows[:, 0, 132:136] = f32_bytes(scales[:, :1])
    return rows


def check(fmt, rows, sel, q, out, lse, kind):
    for s in range(len(sel)):
        r = rows[sel[s][sel[s] >= 0], 0]
        n = len(r)
        if fmt.kind == 0:
            keys, values = ref.latent_kv(r)
            scale = np.abs(ref.f32_at(r, 640, 4)).max(-1)
        else:
            kk, vv, _ = ref.heads_kv(r, 1, 64, 1)
            keys, values = kk[:, 0, 0], vv[:, 0, 0]
            scale = np.abs(ref.f32_at(r, 132, 1))[:, 0]
        o, l, mag, reach = ref.attention(q[s].double().cpu().numpy(), keys, values, 1.0)
        w = np.exp(q[s].double().cpu().numpy() @ keys.T - l[:, None])
        least = n * 448 * 2.0 ** -32 * (w * np.maximum(scale, 2.0 ** -60)).max(-1)
        d = 6 * U["fp32"] * reach + 2.0 ** -22
        tol = mag * (U["fp16"] + 2 * d[:, None] + (2 * (n + 64) + 8) * U["fp32"]) + least[:, None]
        tol = tol + U[kind] * (np.abs(o) + tol) + (2.0 ** -25 if kind == "fp16" else 2.0 ** -133)
        got = out[s].double().cpu().numpy()
        worst = (np.abs(got - o) / tol).max(-1)
        assert np.all(worst <= 1), f"set {s}: off by {worst} of the tolerance, per head"
        off = np.abs(lse[s].double().cpu().numpy() - l)
        assert np.all(off <= d + (n + 74) * U["fp32"] + 4 * U["fp32"] * np.abs(l)), off


def run(name, logit, scales, orders, kind, rng, blank=()):
    import torch
    from serving_pb_lru_amd import head_rows, latent_rows
    fmt = latent_rows() if name == "latent" else head_rows(1, 64)
    rows = (latent_case if name == "latent" else heads_case)(rng, logit, scales)
    rows[list(blank), 0, :512 if name == "latent" else 0] = 0
    if name == "heads":
        rows[list(blank), 0, 64:128] = 0
    sel = np.stack(orders).astype(np.int32)
    q = torch.zeros((len(sel), len(HEADS), 576 if name == "latent" else 64), dtype=torch_type(kind), device="cuda")
    q[..., 512 if name == "latent" else 0] = torch.from_numpy(HEADS).to(q.dtype).cuda()
    eng = engine_of(rows, *sel.shape)
    try:
        d = torch.from_numpy(sel).cuda()
        eng.step(0, d)
        out, lse = eng.attend(0, 0, d, q, fmt, scale=1.0)
        eng.sync()
        check(fmt, rows, sel, q, out, lse, kind)
    finally:
        eng.close()


def orders_of(rng, n):
    """As they are, reversed, every distance of neighbours, shuffled."""
    a = np.arange(n)
    return [a, a[::-1]] + [np.argsort(a % m, kind="stable") for m in (2, 4, 8, 16)] + [rng.permutation(n) for _ in range(2)]


@pytest.mark.parametrize("name", ["latent", "heads"])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("spread", [0, 10, 25, 33, 60])
@pytest.mark.parametrize("against", [0.5, 1.0, 2.0])
def test_scales_against_logits(name, kind, spread, against):
    """Scales over `spread` powers of two, up to 2^-1 for fp16's sake, and logits (in powers of two)
    that fall by `against` as a scale rises by 1: by 2, the key of the least scale has most of the product."""
    rng = np.random.default_rng([spread, int(2 * against)])
    n = 97
    e = rng.uniform(-spread, 0, n)
    e[:8] = [0, -spread] * 4                           # the ends as neighbours
    scales = 2.0 ** np.repeat(e[:, None], 4, 1) / 512
    logit = (-against * (e + spread / 2) * BITS).astype(np.float32)
    run(name, logit, scales, orders_of(rng, n), kind, rng)


@pytest.mark.parametrize("name", ["latent", "heads"])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("ahead", [0, 17, 25, 30, 34, 50])
def test_a_key_of_zeros_with_most_of_the_weight(name, kind, ahead):
    """Rows whose latent channels (values) are all 0 have the writer's least scale, 2^-126, and here a
    logit 2^ahead above that of the ordinary rows beside them: those rows make the result."""
    rng = np.random.default_rng(ahead)
    n = 70
    scales = 2.0 ** rng.standard_normal((n, 4)) / 8
    logit = (rng.standard_normal(n) * 0.5).astype(np.float32)
    blank = [0, 9, 33, 34, 69]
    scales[blank] = 2.0 ** -126
    logit[blank] = ahead * BITS
    run(name, logit, scales, orders_of(rng, n), kind, rng, blank)
