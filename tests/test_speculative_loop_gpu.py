"""A decode loop with drafted tokens and a bounded history: norms and turns, rows of a
tree of drafts, their attention, accepted drafts appended, the selected entries' weights
added up, and the lightest entries released. Every call's result is checked against its
64-bit form or, where it is a choice, against the same choice on the host."""

import numpy as np
import pytest

from test_attend_gpu import latent_rows_of, heads_rows_of, torch_type
from test_lightest_gpu import wanted as lightest_wanted
from test_norm_gpu import wanted as norm_wanted
from test_rows_gpu import assert_within, f64, on_gpu
from test_tree_gpu import check as tree_check, expected as tree_expected
from test_weigh_gpu import expected as weigh_expected, units

pytestmark = pytest.mark.gpu

SETS, SPAN, BUDGET, K, NODES, HEADS, LAYERS, STEPS = 3, 160, 70, 48, 7, 4, 2, 12


def path(parents, rng):
    """The accepted drafts: a random node and those on its way to the root, first to last; or none."""
    t, way = int(rng.integers(-1, len(parents))), []
    while t >= 0:
        way.append(t)
        t = int(parents[t])
    return way[::-1]


@pytest.mark.parametrize("name,kind,other_stream", [("latent", "bf16", False), ("heads", "fp16", False), ("heads", "bf16", True)])
def test_a_decode_loop(name, kind, other_stream):
    import torch
    from serving_pb_lru_amd import Engine, head_rows, latent_rows, lightest, norm_rotate, pack_rows, rotate, tree_masks
    rng = np.random.default_rng([len(name), len(kind), other_stream])
    kv, dim = 2, 64
    fmt = latent_rows() if name == "latent" else head_rows(kv, dim, 1)
    width, n = (576 if name == "latent" else dim), SETS * SPAN
    start = latent_rows_of(rng, n, LAYERS) if name == "latent" else heads_rows_of(rng, n, LAYERS, kv, dim, 1)
    rows = np.zeros_like(start)
    eng = Engine(num_groups=1, layers=LAYERS, row_bytes=fmt.row_bytes, ring=4, logical_capacity=n, gpu_slots=n,
                 host_slots=0, max_sets=SETS, max_k=K)
    stream = torch.cuda.Stream() if other_stream else torch.cuda.current_stream()
    try:
        with torch.cuda.stream(stream):
            held = [list(range(s * SPAN, s * SPAN + BUDGET - 9 * s)) for s in range(SETS)]
            free = [list(range(s * SPAN + BUDGET - 9 * s, (s + 1) * SPAN)) for s in range(SETS)]
            length = [len(h) for h in held]
            las = np.concatenate(held).astype(np.int32)
            rows[las] = start[las]
            eng.append(0, las, rows[las])
            scores = torch.full((n,), -1, dtype=torch.int64, device="cuda")
            scores[torch.from_numpy(las).long().cuda()] = 0
            total = np.full(n, -1, np.int64)
            total[las] = 0
            weight = [on_gpu(1 + 0.2 * rng.standard_normal(dim), kind) for _ in range(2)]
            layer = LAYERS - 1
            for step in range(STEPS):
                print(f"{name} {kind} step {step}: {[len(h) for h in held]} entries", flush=True)
                parents = np.stack([[-1 if t == 0 else int(rng.integers(-1, t)) for t in range(NODES)] for _ in range(SETS)])
                visible = tree_masks(parents)
                depth = np.array([[bin(int(v) & (1 << 64) - 1).count("1") - 1 for v in row] for row in visible])
                pos = torch.from_numpy((np.array(length)[:, None] + depth).reshape(-1).astype(np.int32)).cuda()
                tokens = SETS * NODES
                q = on_gpu(rng.standard_normal((tokens, HEADS, width)), kind)
                if name == "latent":
                    rotate(q[..., 512:], pos, out=q[..., 512:])
                    latent = on_gpu(rng.standard_normal((tokens, LAYERS, 512)), kind)
                    drafts = pack_rows(fmt, latent, on_gpu(rng.standard_normal((tokens, LAYERS, 64)), kind), pos)
                else:
                    k = on_gpu(rng.standard_normal((tokens, kv, dim)), kind)
                    before = f64(q), f64(k)
                    norm_rotate(q, k, *weight, positions=pos, out=(q, k))
                    for x, got, w in zip(before, (q, k), weight):
                        assert_within(f64(got), *norm_wanted(x, f64(w), 1e-6, pos.cpu().numpy()[:, None], (dim // 2,), dim,
                                                             10000.0, False, kind))
                    v = on_gpu(rng.standard_normal((tokens, LAYERS, 1, kv, dim)), kind)
                    drafts = pack_rows(fmt, k[:, None, None].expand(-1, LAYERS, -1, -1, -1), v)
                q = q.view(SETS, NODES, HEADS, width)
                sel = np.full((SETS, K), -1, np.int32)
                for s in range(SETS):
                    sel[s, rng.permutation(K)[:K - s]] = rng.choice(held[s], K - s, replace=False)
                dsel = torch.from_numpy(sel).cuda()
                eng.step(0, dsel)
                out, lse = eng.attend_tree(0, layer, dsel, q, fmt, drafts, torch.from_numpy(visible).cuda())
                share = eng.weigh(0, layer, dsel, q, lse, fmt, scores=scores)
                q64, drafted = f64(q), drafts.cpu().numpy().reshape(tokens, LAYERS, -1)
                tree_check(tree_expected(fmt, rows, drafted, layer, sel, visible, q64, width ** -0.5), out, lse, kind)
                want, off = weigh_expected(fmt, rows, layer, sel, q64, f64(lse), width ** -0.5)
                assert np.all(np.abs(f64(share) - want) <= off)
                added = np.zeros(n, np.int64)
                np.add.at(added, sel[sel >= 0], units(share.cpu().numpy())[sel >= 0])
                total += added
                assert np.array_equal(scores.cpu().numpy(), total)
                # accepted drafts become entries, with the bytes that the tree was attended to with
                taken, at = [], []
                for s in range(SETS):
                    way = path(parents[s], rng)[:len(free[s])]
                    new = [free[s].pop(0) for _ in way]
                    held[s] += new
                    length[s] += len(new)
                    taken += [s * NODES + t for t in way]
                    at += new
                la = np.array(at, np.int32)
                eng.append(0, la, drafts.view(tokens, LAYERS, -1)[torch.tensor(taken, dtype=torch.long, device="cuda")].contiguous())
                rows[la] = drafted[taken]
                if at:
                    scores[torch.from_numpy(la).long().cuda()] = 0
                # what is over the budget goes, lightest first
                first = [s * SPAN for s in range(SETS)]
                last, over = [f + SPAN for f in first], [max(0, len(h) - BUDGET) for h in held]
                total[la] = 0
                known = scores.cpu().numpy()
                assert np.array_equal(known, total)
                gone = lightest(scores, first, last, over, most=NODES, mark=True).cpu().numpy()
                assert np.array_equal(gone, lightest_wanted(known, first, last, over, NODES))
                known[gone[gone >= 0]] = total[gone[gone >= 0]] = -1
                assert np.array_equal(scores.cpu().numpy(), known)
                eng.release(0, gone[gone >= 0])
                for s in range(SETS):
                    held[s] = [a for a in held[s] if a not in set(gone[s].tolist())]
                    free[s] += [a for a in gone[s].tolist() if a >= 0]
                assert np.array_equal(np.flatnonzero(known >= 0), np.sort(np.concatenate(held)))
            eng.sync()
            las = np.sort(np.concatenate(held)).astype(np.int32)
            assert np.array_equal(eng.read_rows(0, las).reshape(len(las), LAYERS, -1), rows[las])
    finally:
        eng.close()
