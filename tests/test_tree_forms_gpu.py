"""ula_attend_tree over heads rows in every form of its kernel (16 to 64 rows a workgroup, heads of 64 and 128, bf16 and
fp16), with several tiles for each of a workgroup's waves and drafted tokens in two tiles where the form has room for
them: the formula, nodes that see nothing, and drafted rows that hold anything. Many sets are what makes the library
take the larger forms: two sets' data are repeated, and the repeated results have the same bits. Tolerances as in
test_tree_gpu.py."""

import numpy as np
import pytest

from test_attend_gpu import engine_of, heads_rows_of, torch_type
from test_tree_gpu import check, expected, trees
from tree_plan import heads_plan

pytestmark = pytest.mark.gpu

# KV head width, groups of 16 rows, sets, nodes, query heads (of one KV head), tokens a block
CASES = [(64, 1, 2, 40, 1, 4), (64, 2, 256, 64, 1, 1), (64, 3, 256, 45, 2, 8), (64, 4, 256, 61, 2, 2),
         (128, 1, 2, 16, 1, 2), (128, 2, 2, 47, 1, 4), (128, 3, 128, 47, 2, 1), (128, 4, 128, 64, 2, 8)]
TOKENS = 13 * 32 + 20


class Call:
    """Two sets' data, and the same attention of them repeated."""

    def __init__(self, dim, groups, sets, nodes, heads, block, kind, seed):
        import torch
        from serving_pb_lru_amd import head_rows
        self.rng = rng = np.random.default_rng([dim, groups, nodes, seed])
        self.sets, self.nodes, self.heads, self.block, self.kind = sets, nodes, heads, block, kind
        self.fmt, self.k, self.per_set = head_rows(1, dim, block), TOKENS // block, -(-nodes // block)
        plan = heads_plan(sets, self.k * block, nodes, heads, 1, dim)
        assert plan.groups == groups and plan.splits == 1, (plan.groups, plan.splits)
        print(f"tree dim={dim} groups={groups} sets={sets} nodes={nodes} heads={heads} block={block} {kind}", flush=True)
        n = self.k + 30
        self.rows = heads_rows_of(rng, n, 1, 1, dim, block, rng.integers(1, block + 1, n))
        left = np.tile(np.minimum(nodes - np.arange(self.per_set) * block, block), 2)
        self.drafts = heads_rows_of(rng, 2 * self.per_set, 1, 1, dim, block, left)
        self.sel = np.stack([rng.permutation(n)[:self.k] for _ in range(2)]).astype(np.int32)
        self.sel[:, rng.permutation(self.k)[:self.k // 9]] = -1
        self.visible = trees(rng, 2, nodes)
        self.q = torch.from_numpy(rng.standard_normal((2, nodes, heads, dim))).to(torch_type(kind)).cuda()

    def __call__(self, drafts=None):
        import torch
        eng = engine_of(self.rows, self.sets, self.k)
        try:
            many = lambda x: x.repeat(self.sets // 2, *(1,) * (x.dim() - 1))
            sel = many(torch.from_numpy(self.sel).cuda())
            eng.step(0, sel)
            out, lse = eng.attend_tree(0, 0, sel, many(self.q), self.fmt,
                                       many(torch.from_numpy(self.drafts if drafts is None else drafts).cuda()),
                                       many(torch.from_numpy(self.visible).cuda()))
            eng.sync()
        finally:
            eng.close()
        bits = lambda x: x.contiguous().view(torch.uint8)
        for x in (out, lse):
            for s in range(2):
                assert (bits(x[s::2]) == bits(x[s:s + 1])).all()
        return out[:2], lse[:2]

    def check(self, out, lse):
        dim = self.fmt.head_dim
        check(expected(self.fmt, self.rows, self.drafts, 0, self.sel, self.visible, self.q.double().cpu().numpy(), dim ** -0.5),
              out, lse, self.kind)


@pytest.mark.parametrize("dim,groups,sets,nodes,heads,block", CASES)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_the_formula(dim, groups, sets, nodes, heads, block, kind):
    """With nodes that see no drafted token, in a set with a history and in one of padding alone."""
    import torch
    call = Call(dim, groups, sets, nodes, heads, block, kind, 1)
    call.visible[:, [1, nodes - 1]] = 0
    call.check(*call())
    call.sel[1] = -1
    out, lse = call()
    call.check(out, lse)
    empty = torch.from_numpy(call.visible[1] == 0)
    assert int(empty.sum()) == 2 and torch.equal(torch.isneginf(lse[1]).all(-1).cpu(), empty) and (out[1][empty.cuda()] == 0).all()


@pytest.mark.parametrize("dim,groups,sets,nodes,heads,block", CASES)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_what_a_drafted_row_holds(dim, groups, sets, nodes, heads, block, kind):
    """NaN codes in a key or a value and scales that are not finite reach the nodes that see the token (a scale: its
    block), and nobody else's bits."""
    import torch
    call = Call(dim, groups, sets, nodes, heads, block, kind, 2)
    part = block * dim
    bad = sorted({block * (j // block) for j in (3, nodes // 2, nodes - 4)})       # the first tokens of blocks
    for j in bad:
        for t in range(nodes):
            if t % 3 == 0:
                call.visible[:, t] |= np.int64(1) << np.int64(j)
            else:
                call.visible[:, t] &= ~(np.int64((1 << block) - 1) << np.int64(j))
    call.visible &= np.int64(-1) if nodes == 64 else np.int64((1 << nodes) - 1)
    clean, lclean = call()
    spoils = dict(value=(part + dim - 3, [0xFF], False), key=(5, [0x7F], False),
                  inf=(2 * part + 4, np.array([-np.inf], "<f4").view(np.uint8), True),
                  nan=(2 * part + 4, np.array([np.nan], "<f4").view(np.uint8), True))
    for name, (at, what, whole) in spoils.items():
        rough = call.drafts.copy()
        for s in range(2):
            for j in bad:
                rough[s * call.per_set + j // block, 0, at:at + len(what)] = what
        hit = np.zeros((2, nodes), bool)
        for j in bad:
            hit |= (call.visible >> j & ((1 << (block if whole else 1)) - 1)) != 0
        assert hit.any() and not hit.all()
        hit = torch.from_numpy(hit).cuda()
        out, lse = call(rough)
        assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all(), name
        assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], lclean[~hit]), name
