"""ula_attend's fp16 results: weights times value scales keep 22 bits on their way into the second product.

Few keys, whose values cancel in some channels, so that the rounding of a single weight shows. Tolerance: the
product's two parts are off by 2^-22 of it (2^-25 in the units of test_attend_scales_gpu at the bottom of
fp16's range); a logit is one product and off by d as there; the sums of n keys in 32 bits, numerator,
denominator and joins, 2 (n + 64) u(fp32), and a handful of products 8 u(fp32), all of the sum of weight x
|value|; the result is rounded once, 2^-11 |o|.
"""

import numpy as np
import pytest

import rows_ref as ref
from test_attend_gpu import U, engine_of, torch_type
from test_attend_scales_gpu import BITS, heads_case, latent_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,sets,heads", [("latent", 5, 9), ("latent", 130, 64), ("heads", 5, 16)])
@pytest.mark.parametrize("k", [2, 3, 7])
def test_weights_keep_their_bits(name, sets, heads, k):
    import torch
    from serving_pb_lru_amd import head_rows, latent_rows
    fmt = latent_rows() if name == "latent" else head_rows(1, 64)
    rng = np.random.default_rng([sets, k])
    n = 300
    logit = (rng.standard_normal(n) * BITS).astype(np.float32)
    rows = (latent_case if name == "latent" else heads_case)(rng, logit, 2.0 ** rng.standard_normal((n, 4)) / 128)
    sel = np.stack([rng.choice(n, k, replace=False) for _ in range(sets)]).astype(np.int32)
    first = 512 if name == "latent" else 0
    q = torch.zeros((sets, heads, 576 if name == "latent" else 64), dtype=torch_type("fp16"), device="cuda")
    q[..., first] = torch.from_numpy(rng.uniform(-1, 1, (sets, heads))).to(q.dtype).cuda()
    eng = engine_of(rows, sets, k)
    try:
        d = torch.from_numpy(sel).cuda()
        eng.step(0, d)
        out, _ = eng.attend(0, 0, d, q, fmt, scale=1.0)
        eng.sync()
    finally:
        eng.close()
    q, out = q.double().cpu().numpy(), out.double().cpu().numpy()
    for s in range(sets):
        r = rows[sel[s], 0]
        if name == "latent":
            keys, values = ref.latent_kv(r)
            scale = ref.f32_at(r, 640, 4).max(-1)
        else:
            kk, vv, _ = ref.heads_kv(r, 1, 64, 1)
            keys, values, scale = kk[:, 0, 0], vv[:, 0, 0], ref.f32_at(r, 132, 1)[:, 0]
        o, lse, mag, reach = ref.attention(q[s], keys, values, 1.0)
        w = np.exp(q[s] @ keys.T - lse[:, None])
        least = k * 448 * 2.0 ** -32 * (w * scale).max(-1)
        off = 2.0 ** -22 + 2 * (6 * U["fp32"] * reach + 2.0 ** -22)[:, None] + (2 * (k + 64) + 8) * U["fp32"]
        tol = mag * off + least[:, None]
        tol = tol + U["fp16"] * (np.abs(o) + tol) + 2.0 ** -25
        worst = (np.abs(out[s] - o) / tol).max()
        assert worst <= 1, f"set {s}: off by {worst:.3g} of the tolerance"
