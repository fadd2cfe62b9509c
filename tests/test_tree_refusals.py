"""What the attention of drafted trees refuses on the host, and the masks of trees: runs without a GPU."""

import ctypes

import numpy as np
import pytest
import torch

from serving_pb_lru_amd import Engine, head_rows, latent_rows, tree_masks, ula

EINVAL = -1
P = 1 << 20


def test_masks():
    assert tree_masks([-1, 0, 0, 1]).tolist() == [1, 3, 5, 11]
    chain = tree_masks(np.arange(64, dtype=np.int32)[None] - 1)
    assert chain.dtype == np.int64 and chain.shape == (1, 64)
    assert chain.view(np.uint64)[0].tolist() == [(1 << (t + 1)) - 1 for t in range(64)]
    two = tree_masks(np.array([[-1, 0, 1], [-1, -1, -1]]))
    assert two.tolist() == [[1, 3, 7], [1, 2, 4]]
    assert tree_masks(np.zeros((0, 3), np.int64)).shape == (0, 3) and tree_masks(np.zeros((2, 0), np.int64)).shape == (2, 0)
    for bad in ([0], [-2], [-1, 1], [-1, 2, 0], np.zeros((2, 65), int) - 1, np.zeros((1, 1, 1), int) - 1, [-1.0]):
        with pytest.raises(ValueError):
            tree_masks(bad)


def test_workspace():
    L = ula.lib()
    f, h = latent_rows(), head_rows(8, 128)
    need = lambda fmt, *a: L.ula_attend_tree_bytes(ctypes.byref(fmt), *a)
    assert L.ula_attend_tree_bytes(None, 1, 1, 1, 1) == 0
    assert need(f, 1, 0, 1, 1) == 0 and need(f, 0, 2048, 8, 16) == 0
    for bad in [(-1, 1, 1, 1), (1, -1, 1, 1), (1, 1, 0, 1), (1, 1, 65, 1), (1, 1, 1, 0), (1, 1, 64, 1025), (1 << 18, 1, 64, 1),
                (1, 2048 * 1024 + 1, 1, 1)]:
        assert need(f, *bad) == 0, bad
    assert need(h, 1, 4096, 4, 12) == 0               # query heads are a multiple of the KV heads
    for fmt, width in ((f, 512), (h, 128)):
        n = need(fmt, 1, 4096, 3, 16)
        assert n > 0 and n % (4 * 48 * (width + 1)) < 512


def test_refused():
    L = ula.lib()
    a = ula.UlaTreeArgs()
    assert L.ula_attend_tree(None, 0, 0, 1, 1, P, ctypes.byref(a), 0) == EINVAL
    sel = torch.zeros((1, 1), dtype=torch.int32)
    q = torch.zeros((1, 1, 1, 576), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="gradient"):
        Engine.attend_tree(None, 0, 0, sel, q.clone().requires_grad_(), latent_rows(), None, None)
    for kw in (dict(out=q.float().requires_grad_()), dict(lse=torch.zeros((1, 1, 1)).requires_grad_())):
        with pytest.raises(ValueError, match="gradient"):
            Engine.attend_tree(None, 0, 0, sel, q, latent_rows(), None, None, **kw)
    with pytest.raises(ValueError, match="shape"):
        Engine.attend_tree(None, 0, 0, sel, q[0], latent_rows(), None, None)
    with pytest.raises(ValueError, match="CUDA"):
        Engine.attend_tree(None, 0, 0, sel, q, latent_rows(), None, None)
