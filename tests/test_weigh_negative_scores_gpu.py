"""What ula_weigh does with negative scores, as documented: it adds to them as to others, so a loop that weighs its
layers before the choice that marks gives every address up once."""

import numpy as np
import pytest

from test_attend_gpu import engine_of, latent_rows_of
from test_weigh_gpu import units

pytestmark = pytest.mark.gpu


def test_layers_weighed_before_the_choice():
    import torch
    from serving_pb_lru_amd import latent_rows, lightest
    rng = np.random.default_rng(31)
    n, layers, fmt = 60, 3, latent_rows()
    rows = latent_rows_of(rng, n, layers)
    eng = engine_of(rows, 1, n)
    try:
        sel = torch.arange(n, dtype=torch.int32, device="cuda")[None]
        q = torch.from_numpy(rng.standard_normal((1, 5, 576))).bfloat16().cuda()
        lse = torch.full((1, 5), 6.0, device="cuda")
        eng.step(0, sel)
        scores, given_up = torch.zeros(n, dtype=torch.int64, device="cuda"), []
        total = np.zeros(n, np.int64)
        for _ in range(4):
            for layer in range(layers):
                share = eng.weigh(0, layer, sel, q, lse, fmt, scores=scores)
                total += units(share.cpu().numpy())[0]
                assert np.array_equal(scores.cpu().numpy(), total)
            for at in given_up:                # still selected: their marks once more
                scores[at], total[at] = -1, -1
            marked = lightest(scores, [0], [n], 7, mark=True).cpu().numpy()[0]
            total[marked] = -1
            given_up += marked.tolist()
        assert len(set(given_up)) == 28 and (total[given_up] == -1).all()
        share = eng.weigh(0, 0, sel, q, lse, fmt, scores=scores)
        assert np.array_equal(scores.cpu().numpy(), total + units(share.cpu().numpy())[0])
        eng.sync()
    finally:
        eng.close()
