"""GB300-native MoE speculative-verify hot path (router, reuse bias, expert
union, grouped SwiGLU expert FFN, EcoSpec draft selection, S2-MoE expansion,
expert residency with on-demand staging from host memory), and the 4-bit paged
KV cache of its attention half (write, read, tree attention, attention weights,
eviction).

The computation lives in ``libmoeverify.so`` (hand-written CUDA for sm_103a,
C ABI in ``include/moe_verify.h``); this package only marshals arguments.
Importing it loads the library and raises if it has not been built.
"""
from . import _lib
from .kv4 import Kv4Cache, kv4_append, kv4_attend, kv4_attend_workspace_bytes, kv4_evict, kv4_read, kv4_weigh  # noqa: F401
from .api import (ExpertLayer, ExpertPool, MoEError, StepSpec, VerifyPlan, VerifyStep, depth_policy,  # noqa: F401
                  eco_select,
                  expert_bytes, ffn_workspace_bytes, hot_list, HostExperts, launch_count, new_dev_err, pack_tiled,
                  profile_begin, profile_end, route, router_logits, s2_expand, set_nvtx, stage_experts,
                  step_workspace_bytes, union_permute, verify_ffn)

_lib.load()
