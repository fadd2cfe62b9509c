"""How ula_norm_rotate splits its rows into workgroups, from the library's host planner by its C++ name: every call has a
plan, whose workgroups hold all rows. Runs without a GPU."""

import ctypes

import pytest

from serving_pb_lru_amd import ula


class NormDev(ctypes.Structure):
    """NormDev of csrc/row_format.h"""
    _fields_ = ([(x, ctypes.c_void_p) for x in ("q", "k", "q_out", "k_out", "q_weight", "k_weight", "positions")] +
                [(x, ctypes.c_int64 * 2) for x in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")] +
                [("eps", ctypes.c_float)] +
                [(x, ctypes.c_int32) for x in ("n", "q_heads", "k_heads", "dim", "rotary", "wide_weights", "aligned",
                                               "tokens_per_block", "heads_per_block")])


@pytest.mark.parametrize("heads,kv", [(1, 0), (0, 1), (1, 1), (2, 1), (7, 0), (40, 8), (300, 20)])
def test_every_size_has_a_plan(heads, kv):
    """Few heads among them, whose rows leave a workgroup's step nearly empty, with and without a turn."""
    plan = ula.lib()._ZN3ula9plan_normEPNS_7NormDevE
    plan.restype = ctypes.c_longlong
    for n in (1, 2, 31, 1023, 1024, 1500, 2047, 2048, 3000, 4096, 8191, 100000, (1 << 24) - 1):
        for dim, rotaries in ((2, (0, 2)), (64, (0, 32, 64)), (100, (0, 50)), (128, (0, 128)), (256, (0, 256))):
            for rotary in rotaries:
                a = NormDev(n=n, q_heads=heads, k_heads=kv, dim=dim, rotary=rotary)
                blocks = plan(ctypes.byref(a))
                what = (n, dim, rotary, a.tokens_per_block, a.heads_per_block)
                assert 1 <= a.tokens_per_block <= 32 and 1 <= a.heads_per_block <= heads + kv, what
                assert blocks == -(-n // a.tokens_per_block) * -(-(heads + kv) // a.heads_per_block), what
