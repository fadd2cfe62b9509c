"""ula_lightest against a sort: whole numbers, so equal."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def wanted(scores, first, last, n, most):
    out = np.full((len(first), most), -1, np.int32)
    for i, (a, b, c) in enumerate(zip(first, last, n)):
        at = np.arange(a, b)[scores[a:b] >= 0]
        pick = np.sort(at[np.argsort(scores[at], kind="stable")[:c]])
        out[i, :len(pick)] = pick
    return out


def check(scores, first, last, n, most=None, mark=False, **kw):
    import torch
    from serving_pb_lru_amd import lightest
    t = torch.from_numpy(scores).cuda()
    got = lightest(t, first, last, n, most=most, mark=mark, **kw).cpu().numpy()
    n = np.full(len(first), n) if np.ndim(n) == 0 else np.asarray(n)
    want = wanted(scores, first, last, n, int(n.max(initial=0)) if most is None else most)
    assert got.shape == want.shape and np.array_equal(got, want), np.argwhere(got != want)[:5]
    after = scores.copy()
    if mark:
        after[want[want >= 0]] = -1
    assert np.array_equal(t.cpu().numpy(), after)


def heavy(rng, n):
    """Scores over many powers of two, some of no weight yet, some gone."""
    s = np.exp(3 * rng.standard_normal(n) + 18).astype(np.int64)
    s[rng.random(n) < 0.1] = 0
    s[rng.random(n) < 0.1] = -1
    return s


KINDS = {
    "heavy": heavy,
    "equal": lambda rng, n: np.full(n, 1 << 33, np.int64),
    "small": lambda rng, n: rng.integers(0, 70, n),
    "near": lambda rng, n: (1 << 45) + rng.integers(0, 1 << 25, n),          # one bin of magnitudes
    "twins": lambda rng, n: np.where(rng.random(n) < 0.5, (1 << 62) + 5, (1 << 62) + 4),
    "ends": lambda rng, n: rng.choice(np.array([0, 1, 63, 64, (1 << 63) - 1, (1 << 63) - 2, -(1 << 63), -1]), n),
    "gone": lambda rng, n: np.full(n, -7, np.int64),
}


# lengths either side of a wave, of a workgroup's threads, of what one workgroup takes (8192) and of 64 chunks
@pytest.mark.parametrize("length", [1, 2, 63, 64, 65, 1023, 1025, 8191, 8192, 8193, 20000, 65537, 600000])
@pytest.mark.parametrize("kind", list(KINDS))
def test_one_range(kind, length):
    rng = np.random.default_rng([length, len(kind)])
    scores = KINDS[kind](rng, length + 30).astype(np.int64)
    for n in sorted({1, length // 3, length}):
        check(scores, [13], [13 + length], n, mark=n == length // 3)


@pytest.mark.parametrize("mark", [False, True])
def test_ragged_ranges(mark):
    """More ranges than one launch takes, long ones among them, empty ones, counts of none and more than there is."""
    rng = np.random.default_rng(8)
    lengths = rng.integers(0, 300, 600)
    lengths[[3, 255, 256, 590]] = [9000, 30000, 8193, 17000]
    lengths[[0, 100, 599]] = 0
    gaps = rng.integers(0, 5, 600)
    first = np.cumsum(lengths + gaps) - lengths
    scores = heavy(rng, int(first[-1] + lengths[-1] + 9))
    n = rng.integers(0, 64, 600)
    n[[3, 255, 256, 590]] = [64, 0, 64, 63]
    order = rng.permutation(600)                       # ranges in any order
    check(scores, first[order], (first + lengths)[order], n[order], most=64, mark=mark)


def test_overlapping_ranges_and_columns():
    rng = np.random.default_rng(9)
    scores = heavy(rng, 40000)
    check(scores, [0, 0, 100, 20000], [40000, 100, 9000, 40000], [5, 100, 7, 4000], most=4001)
    check(scores, [0, 5], [10, 5], [0, 0])
    check(scores, [], [], [])
    check(scores, np.array([7], np.int64), np.array([40000], np.uint16), 12)


def test_streams_graphs_and_given_results():
    import torch
    from serving_pb_lru_amd import lightest
    rng = np.random.default_rng(10)
    scores = torch.from_numpy(heavy(rng, 50000)).cuda()
    first, last, n = [0, 30000], [30000, 33000], [500, 20]
    want = lightest(scores, first, last, n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lightest(scores, first, last, n, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.empty((2, 500), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lightest(scores, first, last, n, out=out, mark=True)
    for i in range(4):                                # each replay takes the next ones
        want = lightest(scores, first, last, n)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert (scores[out[out >= 0].long()] == -1).all()
