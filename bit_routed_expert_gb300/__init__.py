"""GB300-native routed-expert MoE layer and Engram gather-decode (libbre, sm_103a).

The compute path is the C-ABI library built from ``csrc/`` (see ``include/bre.h``);
this package holds its Python binding (``api``), the build step (``build``) and the
seeded synthetic-input generator (``synth``).
"""
from .api import (FfnWeights, KvCache, MoeLayer, MoeStack, StepGraph, bre_dequant, engram_gather_decode, engram_inject, engram_inject_workspace,
                  kv_append, kv_attend, kv_attend_tree, kv_attend_tree_workspace, kv_attend_workspace, kv_compact, kv_fork, kv_read,
                  kv_resize, kv_resize_workspace, kv_rotate, kv_select, kv_select_workspace, rope_turns,
                  moe_combine, moe_expert_ffn, moe_expert_ffn_workspace, moe_permute, moe_residual_norm, moe_route, moe_route_ex, moe_route_permute,
                  moe_route_workspace)
from ._lib import BRE_FMT_Q2_K, BRE_FMT_Q8_0, BreError, load

__all__ = ["FfnWeights", "KvCache", "kv_append", "kv_attend", "kv_attend_tree", "kv_attend_tree_workspace",
           "kv_attend_workspace", "kv_compact", "kv_fork", "kv_read", "kv_resize", "kv_resize_workspace", "kv_rotate",
           "kv_select", "kv_select_workspace", "rope_turns", "MoeLayer", "MoeStack", "StepGraph", "bre_dequant", "engram_gather_decode", "engram_inject", "engram_inject_workspace", "moe_combine", "moe_expert_ffn",
           "moe_expert_ffn_workspace", "moe_permute", "moe_residual_norm", "moe_route", "moe_route_ex", "moe_route_permute",
           "moe_route_workspace",
           "BRE_FMT_Q2_K", "BRE_FMT_Q8_0", "BreError", "load"]
