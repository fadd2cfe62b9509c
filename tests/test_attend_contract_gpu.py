"""What ula_attend's description promises at its borders: factors of the logits, infinite logits."""

import numpy as np
import pytest

from test_attend_edges_gpu import Opened, formats, queries, rows_for, selection

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["latent", "heads"])
def test_factors_of_the_logits_near_the_range(name):
    """A factor that is finite, but not in powers of two, is refused; the largest that is taken gives zero
    logits for a query of zeros, so the mean of the values."""
    from serving_pb_lru_amd import UlaError
    rng = np.random.default_rng(21)
    fmt = formats()[name]
    with Opened(fmt, rows_for(name, rng, 100), selection(rng, 100, 2, 40)) as o:
        q = queries(rng, fmt, 2, 4) * 0
        want, wlse = o.attend(q, scale=0.0)
        for scale in (2.4e38, -2.4e38, 3.4e38, float("inf"), float("-inf"), float("nan")):
            assert pytest.raises(UlaError, o.attend, q, scale=scale).value.name == "EINVAL", scale
        for scale in (2.3e38, -2.3e38):
            out, lse = o.attend(q, scale=scale)
            assert bool((out == want).all()) and bool((lse == wlse).all())
        o.eng.sync()


@pytest.mark.parametrize("name", ["latent", "heads"])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_infinite_logits(name, kind):
    """Logits that overflow: those of -inf drop out, as if their entries were padding; sets of them alone are
    empty; one of +inf makes the heads that read it NaN."""
    import torch
    from test_attend_gpu import f32_bytes
    rng = np.random.default_rng(22)
    fmt = formats()[name]
    rows = rows_for(name, rng, 100)
    low, high = np.arange(0, 60, 3), 99                   # -inf for heads 0 and 1 (2 and 3 read KV head 1)
    code, scale = (0, 640) if fmt.kind == 0 else (0, 2 * 2 * 2 * 64)
    wide = 128 if fmt.kind == 0 else 2 * 64
    for r, c in [(low, 0xF8), (np.array([high]), 0x78)]:  # -256 and 256 in the first block's channel 0, else 0
        rows[r, 0, code:code + wide] = 0
        rows[r, 0, code] = c
        if fmt.kind == 1:
            rows[r, 0, code + 64] = c                     # the entry's second token
        rows[r, 0, scale:scale + 4] = f32_bytes([2.0 ** 118])
    sel = selection(rng, 60, 4, 40)
    sel[0, :20] = low
    sel[1] = np.resize(low, 40)
    sel[2, 7] = high
    sel[3] = np.setdiff1d(np.arange(60), low)
    with Opened(fmt, rows, sel) as o:
        q = queries(rng, fmt, 4, 4, kind)
        q[..., 0] = 8
        out, lse = o.attend(q, scale=1.0)
        without = sel.copy()
        without[np.isin(sel, low)] = -1
        want, wlse = o.attend(q, without, scale=1.0)
        o.eng.sync()
        heads = range(4) if fmt.kind == 0 else range(2)
        for h in heads:
            assert torch.equal(out[[0, 1, 3], h], want[[0, 1, 3], h]) and torch.equal(lse[[0, 1, 3], h], wlse[[0, 1, 3], h])
            assert not bool(out[1, h].any()) and bool(torch.isneginf(lse[1, h]))
            assert bool(out[2, h].isnan().all()) and bool(lse[2, h].isnan())
        for h in range(len(heads), 4):
            assert bool(out[:, h].isfinite().all()) and bool(lse[:, h].isfinite().all())
