"""Forks, renames and releases under the exact-LRU policy: the state against the oracle's, timestamps among
it (a fork is an append, a rename moves addresses alone)."""

import numpy as np
import pytest

from oracle.exact_lru import ExactLRUGroup
from test_entries_gpu import Model
from test_lru_gpu import _compare, _lru_state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", [1, 2])
@pytest.mark.parametrize("static", [False, True])
def test_a_mix_against_the_oracle(seed, static):
    m = Model(seed, policy=1, static_workspace=static)
    lru = ExactLRUGroup(m.N, m.P, m.H)
    rng = m.rng
    try:
        m.append(np.arange(80))
        lru.append(np.arange(80))
        for i in range(80):
            what = rng.choice(["step", "step", "fork", "rename", "release"])
            if what == "step":
                sel = rng.choice(sorted(m.rows), (2, 6))
                sel[rng.random((2, 6)) < 0.1] = -1
                m.step(sel)
                lru.step(sel)
            elif what == "fork":
                (src, ns), (dst, nd) = m.runs(True), m.runs(False)
                n = min(ns, nd, m.P + m.H - len(m.rows), int(rng.integers(1, 20)))
                if n:
                    m.fork(src, dst, n)
                    lru.append(range(dst, dst + n))
            elif what == "rename":
                (src, ns), (dst, nd) = m.runs(True), m.runs(False)
                n = min(ns, nd, int(rng.integers(1, 20)))
                m.rename(src, dst, n)
                places = [lru.where.pop(src + j) for j in range(n)]
                for j, (kind, s) in enumerate(places):
                    lru.where[dst + j] = (kind, s)
                    (lru.gown if kind == "gpu" else lru.hown)[s] = dst + j
            elif len(m.rows) > 40:
                at, n = m.runs(True)
                las = at + rng.permutation(min(n, int(rng.integers(1, 15))))
                m.release(las)
                lru.release(las)
            _compare(m.eng.export_state(0), _lru_state(lru, m.P), f"seed {seed}, operation {i}, {what}")
        m.same("end", True)
        m.eng.sync()
    finally:
        m.close()
