"""How the library splits a tree's attention over heads rows into workgroups: its host planner, by its C++ name, so
that a test can say which of the kernel's forms its sizes reach. Test infrastructure only."""

import ctypes

from serving_pb_lru_amd import ula


class Plan(ctypes.Structure):
    """AttendPlan of csrc/row_format.h"""
    _fields_ = [(x, ctypes.c_int32) for x in ("splits", "split_keys", "head_blocks", "groups", "whole")]


def heads_plan(sets, tokens, nodes, heads, kv_heads, head_dim) -> Plan:
    plan = ula.lib()._ZN3ula15plan_tree_headsEiiiii
    plan.restype = Plan
    return plan(sets, -(-tokens // 32) + -(-nodes // 32), nodes * heads, kv_heads, head_dim)


# KV head width, groups of 16 rows a workgroup, sets, nodes: with four query heads to one KV head and a history of
# 13 tiles and more, every form of the kernel over heads rows, all of a set's tokens in one workgroup
FORMS = [(64, 1, 2, 5), (64, 2, 256, 16), (64, 3, 256, 20), (64, 4, 256, 32),
         (128, 1, 2, 4), (128, 2, 2, 12), (128, 3, 128, 20), (128, 4, 128, 32)]
