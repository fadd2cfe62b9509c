"""ula_norm_rotate of one head a token, as a latent or a single KV head is, against its formula in 64 bits: token
counts at which a workgroup's step is nearly empty, with and without a turn. Tolerance as in test_norm_gpu.py."""

import numpy as np
import pytest

from test_norm_gpu import wanted
from test_rows_gpu import assert_within, f64, on_gpu, positions_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 1023, 1024, 2047, 2500, 8191])
@pytest.mark.parametrize("dim,rotary,kind", [(8, 0, "bf16"), (64, 0, "bf16"), (64, 64, "fp16"), (128, 0, "fp32"), (256, 0, "bf16")])
def test_one_head(n, dim, rotary, kind):
    import torch
    from serving_pb_lru_amd import norm_rotate
    print(f"norm of one head n={n} dim={dim} rotary={rotary} {kind}", flush=True)
    rng = np.random.default_rng([n, dim, rotary])
    x, w = on_gpu(rng.standard_normal((n, 1, dim)), kind), on_gpu(1 + 0.3 * rng.standard_normal(dim), kind)
    pos = positions_of(rng, n, 1, False)
    got = norm_rotate(x, None, w, positions=torch.from_numpy(pos).cuda() if rotary else None, rotary=rotary, eps=1e-5)[0]
    assert_within(f64(got), *wanted(f64(x), f64(w), 1e-5, pos, (rotary // 2,), rotary, 10000.0, False, kind))
