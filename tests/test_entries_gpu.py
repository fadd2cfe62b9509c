"""ula_fork, ula_rename and releases in batches: the state against the oracle (a fork is an append of
the copied rows, a rename moves mapping table and owner entries alone), and every row's bytes
against a model that only knows addresses."""

import numpy as np
import pytest

from gpu_harness import assert_same_state
from oracle.pblru import ABSENT, HOST_BIT, PBLRUGroup

pytestmark = pytest.mark.gpu

LAYERS, ROW = 2, 48


class Model:
    """Engine, oracle (policy PB-LRU) and the bytes of every address."""

    def __init__(self, seed, N=220, P=64, H=90, ring=3, placement="lowest", policy=0, max_append=7, **kw):
        from serving_pb_lru_amd import Engine
        self.rng = np.random.default_rng(seed)
        self.N, self.P, self.H = N, P, H
        self.eng = Engine(num_groups=1, layers=LAYERS, row_bytes=ROW, ring=ring, logical_capacity=N, gpu_slots=P,
                          host_slots=H, max_sets=2, max_k=8, max_append=max_append, policy=policy,
                          placement=int(placement == "ring"), **kw)
        self.ora = PBLRUGroup(N, P, H, ring, LAYERS, ROW, placement=placement) if policy == 0 else None
        self.chunk = max_append
        self.rows = {}

    def close(self):
        self.eng.close()

    def same(self, where, bytes_too=False):
        if self.ora is not None:
            assert_same_state(self.eng.export_state(0), self.ora.export_state(), where)
        if bytes_too and self.rows:
            las = np.array(sorted(self.rows), np.int32)
            got = self.eng.read_rows(0, las)
            want = np.stack([self.rows[a] for a in las])
            assert np.array_equal(got, want), f"{where}: rows differ, first {las[(got != want).any((1, 2))][:5]}"

    def chunks(self, n):
        return [(i, min(i + self.chunk, n)) for i in range(0, n, self.chunk)]

    def append(self, las):
        las = np.asarray(las, np.int32)
        rows = self.rng.integers(0, 256, (las.size, LAYERS, ROW), dtype=np.uint8)
        for a, b in self.chunks(las.size):
            self.eng.append(0, las[a:b], rows[a:b])
            if self.ora is not None:
                self.ora.append(las[a:b], rows[a:b])
        self.rows.update(zip(las.tolist(), rows))

    def step(self, sel):
        import torch
        sel = np.asarray(sel, np.int32)
        d = torch.from_numpy(sel).cuda()
        self.eng.step(0, d)
        if self.ora is not None:
            self.ora.step(sel)
        got = self.eng.gather_layers(0, 0, LAYERS, d).cpu().numpy()
        want = np.zeros((*sel.shape, LAYERS, ROW), np.uint8)
        for i in np.ndindex(sel.shape):
            if sel[i] >= 0:
                want[i] = self.rows[int(sel[i])]
        assert np.array_equal(got.transpose(1, 2, 0, 3), want), "gathered rows differ"

    def fork(self, src, dst, n):
        rows = np.stack([self.rows[a] for a in range(src, src + n)])
        self.eng.fork(0, src, dst, n)
        if self.ora is not None:
            for a, b in self.chunks(n):
                self.ora.append(np.arange(dst + a, dst + b), rows[a:b])
        self.rows.update((dst + i, rows[i]) for i in range(n))

    def rename(self, src, dst, n):
        self.eng.rename(0, src, dst, n)
        if self.ora is not None:
            o, loc = self.ora, self.ora.map[src:src + n].copy()
            o.map[src:src + n] = ABSENT
            o.map[dst:dst + n] = loc
            for i, l in enumerate(loc):
                if l & HOST_BIT:
                    o.hown[int(l & ~HOST_BIT)] = dst + i
                else:
                    o.gown[int(l)] = dst + i
        moved = [self.rows.pop(src + i) for i in range(n)]
        self.rows.update((dst + i, r) for i, r in enumerate(moved))

    def release(self, las):
        las = np.asarray(las, np.int32)
        self.eng.release(0, las)
        if self.ora is not None:
            self.ora.release(las)
        for a in las.tolist():
            del self.rows[a]

    def runs(self, present):
        """A run of addresses that are all present (or all absent): (first, length)."""
        have = np.zeros(self.N, bool)
        have[list(self.rows)] = True
        at = int(self.rng.choice(np.flatnonzero(have == present)))
        end = at
        while end < self.N and have[end] == present:
            end += 1
        return at, end - at


@pytest.mark.parametrize("placement", ["lowest", "ring"])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_a_long_mix_against_the_oracle(placement, seed):
    """Steps, appends, forks, renames (also onto overlapping ranges) and releases in any order; sources on
    the GPU, on the host and in the staging buffer of the last step; forks and renames of several chunks."""
    m = Model(seed, placement=placement)
    rng = m.rng
    try:
        m.append(np.arange(70))
        for i in range(120):
            what = rng.choice(["step", "step", "fork", "fork", "rename", "rename", "release", "append"])
            where = f"{placement} seed {seed}, operation {i}, {what}"
            room = m.P + m.H - len(m.rows)
            if what == "step":
                have = np.array(sorted(m.rows))
                sel = rng.choice(have, (2, 6), replace=True)
                sel[rng.random((2, 6)) < 0.1] = -1
                m.step(sel)
            elif what == "append":
                at, n = m.runs(False)
                n = min(n, int(rng.integers(1, 10)), room)
                if n:
                    m.append(at + rng.permutation(n))
            elif what == "fork":
                (src, ns), (dst, nd) = m.runs(True), m.runs(False)
                n = min(ns, nd, room, int(rng.integers(1, 25)))
                if n:
                    m.fork(src, dst, n)
            elif what == "rename":
                src, n = m.runs(True)
                n = min(n, int(rng.integers(1, 25)))
                have = set(m.rows) - set(range(src, src + n))
                fits = [d for d in range(m.N - n + 1) if not have & set(range(d, d + n))]
                near = [d for d in fits if abs(d - src) <= n]
                m.rename(src, int(rng.choice(near if rng.random() < 0.6 else fits)), n)
            elif len(m.rows) > 40:
                at, n = m.runs(True)
                n = min(n, int(rng.integers(1, 20)))
                m.release(at + rng.permutation(n))
            m.same(where, bytes_too=rng.random() < 0.15)
        m.same("end", True)
        m.eng.sync()
    finally:
        m.close()


@pytest.mark.parametrize("policy,static", [(1, False), (0, True), (1, True)])
def test_exact_lru_and_the_static_workspace(policy, static):
    m = Model(7, policy=policy, static_workspace=static)
    try:
        m.append(np.arange(60))
        for i in range(6):
            m.step(m.rng.choice(sorted(m.rows), (2, 8)))
            m.fork(3 * i, 60 + 10 * i, 9)
            m.rename(60 + 10 * i, 200 - 10 * i, 9)
            m.step(np.stack([np.arange(200 - 10 * i, 208 - 10 * i), np.arange(8)]))
            m.same(f"round {i}", True)
        m.release(np.arange(60))
        m.same("end", True)
        m.eng.sync()
    finally:
        m.close()


def test_sources_on_the_host_and_in_the_staging_buffer():
    """A step evicts entries whose rows are still staged: a fork of them copies those, a rename keeps
    track of them, and the next step writes them out under their new names."""
    m = Model(9, P=16, H=100)
    try:
        m.append(np.arange(60))                        # 0..15 on the GPU, the rest on the host
        m.step(np.arange(40, 56).reshape(2, 8))        # evicts all of 0..15, staged
        staged = m.eng.export_state(0)["map"][:16]
        assert np.all(staged & np.uint32(HOST_BIT))
        m.fork(0, 100, 16)
        m.rename(0, 80, 16)
        m.step(np.arange(16, 32).reshape(2, 8))
        m.same("after the write-back", True)
        m.step(np.arange(80, 96).reshape(2, 8))
        m.step(np.arange(100, 116).reshape(2, 8))
        m.same("end", True)
        m.eng.sync()
    finally:
        m.close()


def test_refusals_change_nothing():
    from serving_pb_lru_amd import UlaError
    import torch
    m = Model(11, N=100, P=16, H=24)
    try:
        m.append(np.arange(30))
        code = lambda f, *a: pytest.raises(UlaError, f, *a).value.name
        fork, rename = m.eng.fork, m.eng.rename
        for f in (fork, rename):
            assert code(f, 1, 0, 40, 1) == code(f, -1, 0, 40, 1) == code(f, 0, 0, 40, -1) == "EINVAL"
            for src, dst, n in [(-1, 40, 1), (0, -1, 1), (99, 40, 2), (0, 99, 2), (100, 40, 1), (25, 40, 6), (30, 40, 1),
                                (0, 40, 2 ** 31 - 1), (2 ** 31 - 1, 40, 2)]:
                assert code(f, 0, src, dst, n) == "ERANGE", (f, src, dst, n)
            f(0, 0, 40, 0)                             # nothing
        assert code(fork, 0, 0, 29, 5) == code(fork, 0, 0, 0, 1) == code(fork, 0, 5, 6, 3) == "EDUP"
        assert code(fork, 0, 0, 40, 11) == "EHOSTFULL"
        assert code(rename, 0, 0, 5, 3) == code(rename, 0, 10, 28, 3) == code(rename, 0, 3, 2, 4) == "EDUP"
        rename(0, 7, 7, 5)                             # onto itself
        m.same("after the refusals", True)
        m.fork(0, 40, 10)                              # exactly full
        m.same("full", True)
        # neither may be captured: both read and change the state of their moment
        x = torch.zeros(4, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            assert code(rename, 0, 40, 60, 3) == "EINVAL"
            x.add_(1)
        m.same("after the capture", True)
        m.release(np.arange(40, 45))
        torch.cuda.synchronize()
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            assert code(fork, 0, 0, 70, 3) == "EINVAL"
            x.add_(1)
        m.same("end", True)
        m.eng.sync()
    finally:
        m.close()


@pytest.mark.parametrize("n", [1, 1023, 1024, 1025, 4095, 4096, 4097, 6000])
def test_renames_of_many_sizes(n):
    """Either side of a workgroup's entries, to a range of its own and up and down by a few addresses."""
    m = Model(17, N=13000, P=5000, H=1200, max_append=6100)
    try:
        m.append(np.arange(50, 50 + n))
        for src, dst in [(50, 6500), (6500, 6507), (6507, 6400), (6400, 0), (0, 1), (1, 12999 - n)]:
            m.rename(src, dst, n)
            m.same(f"{n} entries from {src} to {dst}")
        m.release(np.arange(12999 - n, 12999))
        m.same("end", True)
        m.eng.sync()
    finally:
        m.close()


@pytest.mark.parametrize("policy", [0, 1])
def test_releases_of_many_orders(policy):
    """Batches that share words and spans of the bitmaps in every way: in order, reversed, scattered, one
    by one, over more than one span of 2048 slots; on the GPU and on the host; repeated or absent
    addresses refuse the whole batch."""
    from serving_pb_lru_amd import UlaError
    m = Model(13, N=9000, P=5000, H=3900, max_append=4096, policy=policy)
    try:
        m.append(np.arange(8500))
        m.step(m.rng.choice(8500, (2, 8)))
        for las in (np.arange(100, 400), np.arange(4999, 4500, -1), m.rng.permutation(np.arange(500, 4400))[:1500],
                    np.arange(5000, 8400, 3), np.array([8499]), np.arange(4400, 4500)):
            m.release(las)
            m.same(f"release of {las.size}")
        for las, name in [([0, 5, 0], "EDUP"), ([100, 0], "ERANGE"), ([9000, 1], "ERANGE"), ([-1], "ERANGE"),
                          ([3, 4, 5, 4], "EDUP"), ([5, 4, 3, 101], "ERANGE"), ([100, 100], "EDUP")]:
            assert pytest.raises(UlaError, m.eng.release, 0, np.array(las, np.int32)).value.name == name, las
        m.append(m.rng.permutation(np.concatenate([np.arange(100, 400), np.arange(4400, 4500), np.arange(4501, 5000)])))
        m.same("end", True)
        m.eng.sync()
    finally:
        m.close()


def test_a_decode_loop_of_all_operators():
    """A request is packed, appended and attended to; a second one forks its history and goes on by
    itself; the first is released and the second renamed to the front. After every step the
    attention equals the formula over the rows that were packed."""
    import torch
    import rows_ref as ref
    from serving_pb_lru_amd import Engine, latent_rows, pack_rows, rotate
    from test_attend_gpu import check
    fmt, layers, heads = latent_rows(), 2, 5
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, device="cuda", generator=gen).to(torch.bfloat16)
    eng = Engine(num_groups=1, layers=layers, row_bytes=656, ring=4, logical_capacity=400, gpu_slots=96, host_slots=200,
                 max_sets=2, max_k=40, max_append=64)
    rows = np.zeros((400, layers, 656), np.uint8)
    rng = np.random.default_rng(3)

    def packed(first, n):
        pos = torch.arange(first, first + n, dtype=torch.int32, device="cuda")
        return pack_rows(fmt, rand(n, layers, 512), rand(n, layers, 64), pos, interleaved=True)

    def turn(sets, at):
        q = rand(sets, heads, 576)
        pos = torch.tensor(at, dtype=torch.int32, device="cuda")
        return rotate(q[..., 512:], pos, interleaved=True, out=q[..., 512:]) is not None and q

    def look(sel):
        d = torch.from_numpy(sel).cuda()
        for layer in range(layers):
            q = turn(sel.shape[0], sel.max(1).tolist())
            out, lse = eng.attend(0, layer, d, q, fmt)
            check(fmt, rows, layer, sel, q, 1 / 24, out, lse, "bf16")

    try:
        prompt = packed(0, 60)
        eng.append(0, np.arange(60, dtype=np.int32), prompt)
        rows[:60] = prompt.cpu().numpy()
        first, second = 60, 0
        for t in range(12):
            if t == 4:                                  # a second request with the same history
                eng.fork(0, 0, 200, first)
                rows[200:200 + first] = rows[:first]
                second = 200 + first
            new = [first] + ([second] if second else [])
            r = torch.cat([packed(a % 200, 1) for a in new])
            sel = np.stack([np.sort(rng.choice(a - (a // 200) * 200 + 1, 40, replace=False)) + (a // 200) * 200 for a in new])
            sel[:, -1] = new                            # the token itself
            sel = sel.astype(np.int32)
            sel[0, rng.choice(39, 3, replace=False)] = -1
            eng.append_step(0, np.array(new, np.int32), r, torch.from_numpy(sel).cuda())
            rows[new] = r.cpu().numpy()
            look(sel)
            first += 1
            second += bool(second)
        eng.release(0, np.arange(first, dtype=np.int32))
        n = second - 200
        eng.rename(0, 200, 100, n)                      # ranges that overlap or not, in two moves
        eng.rename(0, 100, 0, n)
        rows[:n] = rows[200:200 + n].copy()
        sel = np.sort(rng.choice(n, (1, 40), replace=False)).astype(np.int32)
        eng.step(0, torch.from_numpy(sel).cuda())
        look(sel)
        eng.sync()
        las = np.arange(n, dtype=np.int32)
        assert np.array_equal(eng.read_rows(0, las), rows[:n])
    finally:
        eng.close()
