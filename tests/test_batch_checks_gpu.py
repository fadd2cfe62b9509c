"""The host's checks of append and release batches, for batches of a few runs of addresses and of scattered
ones (which are checked one by one), and either side of the border between the two."""

import numpy as np
import pytest

from test_entries_gpu import Model

pytestmark = pytest.mark.gpu


def batches(first, n):
    """n distinct addresses from `first` on in as many runs as the key says."""
    at = lambda runs: np.concatenate([x + 2 * i for i, x in enumerate(np.array_split(np.arange(n), runs))]) + first
    return {runs: at(runs) for runs in (1, 2, n // 4, n // 4 + 1, n // 2, n)}


@pytest.mark.parametrize("policy", [0, 1])
def test_refusals_and_state(policy):
    from serving_pb_lru_amd import UlaError
    n = 40
    m = Model(29, N=4000, P=700, H=900, max_append=16, policy=policy)
    code = lambda f, *a: pytest.raises(UlaError, f, *a).value.name
    rows = np.zeros((n + 1, 2, 48), np.uint8)
    try:
        m.append(np.arange(3000, 3300))
        for runs, las in batches(100, n).items():
            assert len(np.unique(las)) == n and 1 + (np.diff(las) != 1).sum() == runs
            for extra, want in [(4000, "ERANGE"), (-1, "ERANGE"), (2 ** 31 - 1, "ERANGE"), (int(las[7]), "EDUP"),
                                (int(las[-1]), "EDUP"), (3100, "EDUP")]:
                for bad in (np.append(las, extra), np.insert(las, 0, extra), np.insert(las, n // 2, extra)):
                    bad = bad.astype(np.int32)
                    assert code(m.eng.append, 0, bad, rows) == want, (runs, extra)
            m.same("after the refused appends")
            for order in (las, las[::-1], m.rng.permutation(las)):
                m.append(order)
                m.same(f"append of {runs} runs")
                for extra, want in [(4000, "ERANGE"), (-5, "ERANGE"), (int(las[7]), "EDUP"), (99, "ERANGE")]:
                    for bad in (np.append(order, extra), np.insert(order, 0, extra)):
                        assert code(m.eng.release, 0, bad.astype(np.int32)) == want, (runs, extra)
                m.same("after the refused releases")
                m.release(order)
                m.same(f"release of {runs} runs")
        m.same("end", True)
        m.eng.sync()
    finally:
        m.close()
