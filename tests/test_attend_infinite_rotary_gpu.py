"""ula_attend of rows whose rotary channels hold infinities: a logit of -infinity has no weight, one of +infinity makes
the head NaN, for fp16 queries (whose rotary channels are taken apart into two bf16 values) as for bf16 ones. Bits are
those of the same call without the entry."""

import numpy as np
import pytest

from test_attend_gpu import engine_of, latent_rows_of, torch_type

pytestmark = pytest.mark.gpu

# values of q at the infinite channel: both bf16 parts of one sign or of two as rounding goes, one part alone, the
# least ones of fp16
QUERIES = [1.0, 0.3330078125, 0.33349609375, 1.00390625, 1.0048828125, 6.103515625e-05, 5.9604644775390625e-08, 1000.5]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("k,where", [(33, 5), (300, 290)])
def test_infinite_rotary_channels(kind, k, where):
    import torch
    from serving_pb_lru_amd import latent_rows
    rng = np.random.default_rng([k, where])
    rows = latent_rows_of(rng, k, 1)
    heads = 2 * len(QUERIES) + 1
    q = torch.from_numpy(rng.standard_normal((3, heads, 576))).to(torch_type(kind)).cuda()
    at = torch.tensor(QUERIES + [-x for x in QUERIES] + [0.0]).to(q.dtype).cuda()
    q[..., 530] = at
    sel = np.tile(np.arange(k, dtype=np.int32), (3, 1))
    without = sel.copy()
    without[1:, where] = -1

    def call(selection):
        eng = engine_of(rows, 3, k)
        try:
            d = torch.from_numpy(selection).cuda()
            eng.step(0, d)
            out = eng.attend(0, 0, d, q, latent_rows())
            eng.sync()
            return out
        finally:
            eng.close()

    for value in (0x7F80, 0xFF80):
        rows[where, 0, 512 + 2 * 18:512 + 2 * 19] = np.array([value], "<u2").view(np.uint8)
        rows[0, 0, 512 + 2 * 18:512 + 2 * 19] = np.array([0x3F80], "<u2").view(np.uint8)
        out, lse = call(sel)
        clean, lclean = call(without)
        none = (at < 0) if value == 0x7F80 else (at > 0)
        assert int(none.sum()) == len(QUERIES)
        assert torch.isnan(out[:, ~none]).all() and torch.isnan(lse[:, ~none]).all()
        assert torch.equal(out[1:, none], clean[1:, none]) and torch.equal(lse[1:, none], lclean[1:, none])
        assert torch.isfinite(out[:, none]).all() and torch.isfinite(lse[:, none]).all()
