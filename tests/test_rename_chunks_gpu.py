"""ula_rename of more entries than one chunk takes, in chunks of the two-launch form."""

import pytest

from test_entries_gpu import Model

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_append", [4500, 4097, 5000])
def test_overlapping_chunks(max_append):
    """Two full chunks of more than one workgroup's entries and a short one, whose scratch places follow one
    another: up and down by a few addresses, by less than a chunk, by more than one, and to a range apart."""
    import numpy as np
    n = 10000
    m = Model(23, N=33000, P=7000, H=3500, max_append=max_append)
    try:
        m.append(np.arange(100, 100 + n))
        at = 100
        for dst in (103, 102, 4102, 0, 4600, 9400, 1, 20000, 20001, 15000):
            m.rename(at, dst, n)
            at = dst
            m.same(f"{n} entries to {dst} in chunks of {max_append}")
        m.fork(at, 0, 400)
        m.release(np.arange(at, at + n))
        m.same("end", True)
        m.eng.sync()
    finally:
        m.close()
