"""ula_attend_tree's softmax weights for bf16 results: products with value scales go through the second product in
two fp16 parts, as for fp16 results, so what they leave is 2^-22 of each and not 2^-11.

Few tokens of ordinary scales and one nonzero channel of q, so that logits and sums are off by little and a single
rounding to fp16 would show: values of either sign leave results far smaller than the sum of their magnitudes,
which their own rounding to bf16 cannot hide. Tolerance as in test_tree_scales_gpu.py with 2^-22 for the weights; over
heads rows log2 |scale| is at most 16 here, off by a step of 2^-20, and its four sums round (R log2(e) + 16) each."""

import numpy as np
import pytest

import rows_ref as ref
from test_attend_gpu import U
from test_attend_scales_gpu import HEADS, heads_case, latent_case
from test_tree_gpu import trees
from test_tree_scales_gpu import call, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["latent", "heads"])
@pytest.mark.parametrize("sets,k,nodes", [(24, 5, 3), (3, 3, 12)])
def test_weights_are_not_rounded_to_one_fp16_number(name, sets, k, nodes):
    rng = np.random.default_rng([sets, k, nodes])
    case = latent_case if name == "latent" else heads_case
    make = lambda n: case(rng, rng.standard_normal(n).astype(np.float32), 2.0 ** rng.standard_normal((n, 4)) / 120)
    rows, drafts = make(80), make(sets * nodes)
    sel = np.stack([rng.permutation(80)[:k] for _ in range(sets)]).astype(np.int32)
    visible = trees(rng, sets, nodes)
    q = queries(name, sets, nodes, "bf16")
    out, lse = call(name, rows, drafts, sel, visible, q)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    u, worst = U["fp32"], 0.0
    for s in range(sets):
        for t in range(nodes):
            see = [j for j in range(nodes) if int(visible[s, t]) >> j & 1]
            r = np.concatenate([rows[sel[s], 0], drafts[s * nodes:][see, 0]])
            n, x = len(r), q[s, t].double().cpu().numpy()
            if name == "latent":
                keys, values = ref.latent_kv(r)
                scale = np.abs(ref.f32_at(r, 640, 4)).max(-1)
            else:
                kk, vv, _ = ref.heads_kv(r, 1, 64, 1)
                keys, values, scale = kk[:, 0, 0], vv[:, 0, 0], np.abs(ref.f32_at(r, 132, 1))[:, 0]
            o, l, mag, reach = ref.attention(x, keys, values, 1.0)
            w = np.exp(x @ keys.T - l[:, None])
            d = 6 * u * reach + 2.0 ** -22
            if name == "heads":
                d = d + np.log(2) * (2.0 ** -20 + 4 * u * (reach / np.log(2) + 16))
            tol = mag * (2.0 ** -22 + 2 * d[:, None] + (2 * (n + 64) + 8) * u) + n * 448 * 2.0 ** -32 * (w * scale).max(-1)[:, None]
            tol = tol + U["bf16"] * (np.abs(o) + tol) + 2.0 ** -133
            worst = max(worst, (np.abs(got[s, t] - o) / tol).max())
            assert np.all(np.abs(got_lse[s, t] - l) <= d + (n + 74) * u + 4 * u * np.abs(l))
    assert worst <= 1, f"off by {worst:.3g} of the tolerance"
