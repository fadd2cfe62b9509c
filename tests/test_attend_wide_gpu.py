"""Latent attention in workgroups of 64 heads, which the plan takes where sets and heads fill the card:
whole and partly filled blocks of heads, one tile to several splits, both types, against the formulas."""

import numpy as np
import pytest

import test_attend_scales_gpu as scales
from test_attend_gpu import latent_rows_of, run, selection

pytestmark = pytest.mark.gpu


# sets, k, heads, layers, layer, type, padding
CASES = [(130, 33, 64, 1, 0, "fp16", 0), (130, 1, 64, 1, 0, "bf16", 0), (260, 31, 63, 1, 0, "fp16", 4), (200, 65, 100, 2, 1, "fp16", 7),
         (200, 64, 97, 1, 0, "bf16", 64), (150, 100, 64, 1, 0, "bf16", 3), (33, 2048, 100, 1, 0, "fp16", 50),
         (33, 2500, 64, 1, 0, "bf16", 9), (20, 4100, 128, 1, 0, "fp16", 0)]


@pytest.mark.parametrize("sets,k,heads,layers,layer,kind,pad", CASES)
def test_against_the_formula(sets, k, heads, layers, layer, kind, pad):
    from serving_pb_lru_amd import latent_rows
    print(f"latent sets={sets} k={k} heads={heads} layers={layers} layer={layer} {kind} pad={pad}", flush=True)
    rng = np.random.default_rng([sets, k, heads])
    n = max(600, k + 100)
    run(latent_rows(), latent_rows_of(rng, n, layers), layer, selection(rng, n, sets, k, pad), heads, kind, rng)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("spread,against", [(25, 2.0), (33, 1.0), (60, 2.0)])
def test_scales_against_logits(monkeypatch, kind, spread, against):
    """test_attend_scales_gpu's rows, with as many sets and heads as such workgroups need."""
    rng = np.random.default_rng([spread, 7])
    monkeypatch.setattr(scales, "HEADS", np.resize(scales.HEADS, 64))
    n = 97
    e = rng.uniform(-spread, 0, n)
    e[:8] = [0, -spread] * 4
    logit = (-against * (e + spread / 2) * scales.BITS).astype(np.float32)
    orders = sum((scales.orders_of(rng, n) for _ in range(17)), [])
    scales.run("latent", logit, 2.0 ** np.repeat(e[:, None], 4, 1) / 512, orders, kind, rng)
