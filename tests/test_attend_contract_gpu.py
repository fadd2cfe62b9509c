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
