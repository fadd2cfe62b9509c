"""Tensors of another shape than documented, with enough elements: refused by name instead of read as something else.
Runs without a GPU: the tensors say that they are on one, and every call here ends before the device is asked for."""

import pytest
import torch

from serving_pb_lru_amd import Engine, head_rows, latent_rows, lightest


class Claimed:
    """A CPU tensor that says it is a CUDA tensor."""
    is_cuda, requires_grad = True, False

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


class Rows:
    """What the checks look at of an engine."""
    def __init__(self, fmt, layers, n):
        self.row_bytes, self.layers, self.N = fmt.row_bytes, layers, n


def of(shape, dtype=torch.float32):
    return Claimed(torch.zeros(shape, dtype=dtype))


SETS, K, NODES, HEADS, LAYERS = 2, 7, 5, 4, 3


@pytest.mark.parametrize("fmt,per_set", [(latent_rows(), NODES), (head_rows(2, 64, 4), 2)])
def test_attend_tree(fmt, per_set):
    eng, sel = Rows(fmt, LAYERS, 50), of((SETS, K), torch.int32)
    q = of((SETS, NODES, HEADS, 576 if fmt.kind == 0 else 64), torch.bfloat16)
    good = dict(drafts=of((SETS * per_set, LAYERS, fmt.row_bytes), torch.uint8), visible=of((SETS, NODES), torch.int64),
                lse=of((SETS, NODES, HEADS)))
    bad = dict(drafts=[(SETS * per_set + 1, LAYERS, fmt.row_bytes), (LAYERS, SETS * per_set, fmt.row_bytes),
                       (SETS * per_set * LAYERS, fmt.row_bytes), (SETS * per_set, LAYERS, fmt.row_bytes + 16)],
               visible=[(SETS, NODES + 1), (NODES, SETS), (SETS * NODES,), (SETS + 1, NODES)],
               lse=[(SETS, HEADS, NODES), (SETS, NODES + 1, HEADS), (SETS * NODES, HEADS), (SETS, NODES, HEADS + 1)])
    for name, shapes in bad.items():
        for shape in shapes:
            with pytest.raises(ValueError, match=f"{name}: shape"):
                Engine.attend_tree(eng, 0, 0, sel, q, fmt, **{**good, name: of(shape, good[name].dtype)})


@pytest.mark.parametrize("nodes", [(), (NODES,)])
def test_weigh(nodes):
    fmt = latent_rows()
    eng, sel, q = Rows(fmt, LAYERS, 50), of((SETS, K), torch.int32), of((SETS, *nodes, HEADS, 576), torch.float16)
    good = dict(lse=of((SETS, *nodes, HEADS)), out=of((SETS, K)))
    bad = dict(lse=[(SETS, *nodes, HEADS + 1), (SETS, NODES + 1, HEADS), (SETS * NODES * HEADS,), (SETS, HEADS, *nodes, 1)],
               out=[(K, SETS), (SETS, K + 1), (SETS * K,)])
    for name, shapes in bad.items():
        for shape in shapes:
            with pytest.raises(ValueError, match=f"{name}: shape"):
                Engine.weigh(eng, 0, 0, sel, q, fmt=fmt, **{**good, name: of(shape)})


def test_lightest():
    for shape in [(3, 5), (2, 6), (10,), (5, 2)]:
        with pytest.raises(ValueError, match="out: shape"):
            lightest(of(100, torch.int64), [0, 50], [50, 100], [5, 3], out=of(shape, torch.int32))
