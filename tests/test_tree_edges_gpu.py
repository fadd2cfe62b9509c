"""ula_attend_tree and ula_weigh at their borders: factors of the logits, queries that are not finite, the most rows
of a set, entries listed twice, selections that are not the last step's, calls on two streams at once. Tolerances are
those of the formula's tests."""

import numpy as np
import pytest

from test_attend_gpu import engine_of, selection, torch_type
from test_tree_gpu import call, check, expected, formats, some, trees
from test_weigh_gpu import expected as weigh_expected

pytestmark = pytest.mark.gpu


def width_of(fmt):
    return 576 if fmt.kind == 0 else fmt.head_dim


def case(name, rng, sets, k, nodes, heads, kind="bf16", pad=0):
    import torch
    fmt = formats()[name]
    block = 1 if fmt.kind == 0 else fmt.block_tokens
    rows, drafts = some(fmt, rng, k + 20), some(fmt, rng, sets * -(-nodes // block))
    q = torch.from_numpy(rng.standard_normal((sets, nodes, heads, width_of(fmt)))).to(torch_type(kind)).cuda()
    return fmt, rows, drafts, selection(rng, k + 20, sets, k, pad), trees(rng, sets, nodes), q


@pytest.mark.parametrize("name", ["latent", "heads", "heads128"])
@pytest.mark.parametrize("scale", [0.0, -0.04, 1.5, 1e-30])
def test_factors_of_the_logits(name, scale):
    rng = np.random.default_rng(21)
    fmt, rows, drafts, sel, visible, q = case(name, rng, 2, 130, 11, 6, "fp16", 3)
    out, lse = call(fmt, rows, drafts, sel, visible, q, scale=scale)
    check(expected(fmt, rows, drafts, 0, sel, visible, q.double().cpu().numpy(), scale), out, lse, "fp16")


@pytest.mark.parametrize("name", ["latent", "heads", "heads128"])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_queries_that_are_not_finite(name, kind):
    """A NaN or an infinity in one row of q makes that row's result NaN; the others keep their bits."""
    import torch
    rng = np.random.default_rng(22)
    fmt, rows, drafts, sel, visible, q = case(name, rng, 2, 200, 9, 4, kind, 2)
    clean, lclean = call(fmt, rows, drafts, sel, visible, q)
    q[0, 3, 1, 7] = float("nan")
    q[1, 8, 2, 9] = float("inf")
    q[1, 0, 0, -1] = -float("inf")
    out, lse = call(fmt, rows, drafts, sel, visible, q)
    hit = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    hit[0, 3, 1] = hit[1, 8, 2] = hit[1, 0, 0] = True
    assert torch.isnan(out[hit]).all()
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], lclean[~hit])


@pytest.mark.parametrize("name,nodes,heads", [("latent", 64, 130), ("heads", 64, 1024), ("heads128", 61, 1000)])
def test_many_rows(name, nodes, heads):
    rng = np.random.default_rng(23)
    fmt, rows, drafts, sel, visible, q = case(name, rng, 1, 37, nodes, heads)
    out, lse = call(fmt, rows, drafts, sel, visible, q)
    check(expected(fmt, rows, drafts, 0, sel, visible, q.double().cpu().numpy(), width_of(fmt) ** -0.5), out, lse, "bf16")


@pytest.mark.parametrize("name", ["latent", "heads"])
def test_an_entry_listed_more_than_once_counts_as_often(name):
    import torch
    rng = np.random.default_rng(24)
    fmt, rows, drafts, sel, visible, q = case(name, rng, 3, 70, 5, 4)
    sel[:, 40:60] = sel[:, :20]
    sel[2] = sel[1]                                   # and in another set
    eng = engine_of(rows, *sel.shape)
    try:
        dsel = torch.from_numpy(sel).cuda()
        eng.step(0, dsel)
        out, lse = eng.attend_tree(0, 0, dsel, q, fmt, torch.from_numpy(drafts).cuda(), torch.from_numpy(visible).cuda())
        scale = width_of(fmt) ** -0.5
        q64 = q.double().cpu().numpy()
        check(expected(fmt, rows, drafts, 0, sel, visible, q64, scale), out, lse, "bf16")
        scores = torch.zeros(len(rows), dtype=torch.int64, device="cuda")
        share = eng.weigh(0, 0, dsel, q, lse, fmt, scores=scores).double().cpu().numpy()
        want, off = weigh_expected(fmt, rows, 0, sel, q64, lse.double().cpu().numpy(), scale)
        assert np.all(np.abs(share - want) <= off)
        assert np.array_equal(share[:, 40:60], share[:, :20])
        total = np.zeros(len(rows))
        np.add.at(total, sel, share)
        assert np.all(np.abs(scores.cpu().numpy() * 2.0 ** -32 - total) <= sel.size * 2.0 ** -33 + total * 2.0 ** -40)
        eng.sync()
    finally:
        eng.close()


@pytest.mark.parametrize("name", ["latent", "heads128"])
def test_selections_other_than_the_steps(name):
    """Entries of an earlier step that are still on the GPU, and one that is not: it counts as padding and is reported."""
    import torch
    from serving_pb_lru_amd import Engine, UlaError
    rng = np.random.default_rng(25)
    fmt, rows, drafts, sel, visible, q = case(name, rng, 2, 60, 6, 4)
    other = sel[:, ::-1].copy()
    want, lwant = call(fmt, rows, drafts, other, visible, q)
    n = len(rows)
    eng = Engine(num_groups=1, layers=1, row_bytes=rows.shape[2], ring=4, logical_capacity=n + 1, gpu_slots=n, host_slots=8,
                 max_sets=2, max_k=60)
    try:
        eng.append(0, np.arange(n, dtype=np.int32), rows)
        eng.append(0, np.array([n], np.int32), rows[:1])                # the pool is full: to the host
        dsel, dother = torch.from_numpy(sel).cuda(), torch.from_numpy(other).cuda()
        eng.step(0, dsel)
        args = (fmt, torch.from_numpy(drafts).cuda(), torch.from_numpy(visible).cuda())
        out, lse = eng.attend_tree(0, 0, dother, q, *args)
        assert torch.equal(out, want) and torch.equal(lse, lwant)
        share = eng.weigh(0, 0, dother, q, lse, fmt)
        eng.sync()
        dother[1, 3] = n
        eng.attend_tree(0, 0, dother, q, *args)
        again = eng.weigh(0, 0, dother, q, lse, fmt)
        assert float(again[1, 3]) == 0 and torch.equal(again[0], share[0])
        with pytest.raises(UlaError) as e:
            eng.sync()
        assert e.value.name == "ENOTRESIDENT"
    finally:
        eng.close()


@pytest.mark.parametrize("name", ["latent", "heads"])
def test_calls_on_two_streams_at_once(name):
    import torch
    rng = np.random.default_rng(26)
    fmt, rows, drafts, sel, visible, q = case(name, rng, 8, 900, 12, 8)
    eng = engine_of(rows, *sel.shape)
    try:
        dsel = torch.from_numpy(sel).cuda()
        eng.step(0, dsel)
        args = (fmt, torch.from_numpy(drafts).cuda(), torch.from_numpy(visible).cuda())
        first = eng.attend_tree(0, 0, dsel, q, *args)
        shares = eng.weigh(0, 0, dsel, q, first[1], fmt)
        streams = [torch.cuda.Stream() for _ in range(2)]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        scores = torch.zeros(len(rows), dtype=torch.int64, device="cuda")
        torch.cuda.synchronize()
        got = []
        for _ in range(6):
            for s in streams:
                with torch.cuda.stream(s):
                    r = eng.attend_tree(0, 0, dsel, q, *args)
                    got.append((*r, eng.weigh(0, 0, dsel, q, r[1], fmt, scores=scores)))
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for o, l, w in got:
            assert torch.equal(o, first[0]) and torch.equal(l, first[1]) and torch.equal(w, shares)
        once = torch.zeros_like(scores)
        eng.weigh(0, 0, dsel, q, first[1], fmt, scores=once)
        assert torch.equal(scores, 12 * once)
        eng.sync()
    finally:
        eng.close()
