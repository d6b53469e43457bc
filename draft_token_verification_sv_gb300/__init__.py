"""GB300-native verify step of speculative decoding, and the 8-bit cache and
attention of the scoring pass before it, from a request's pages, positions and
prompt on.

The compute lives in ``libspec_verify.so`` (CUDA kernels for sm_103a behind
the C-ABI in include/spec_verify.h).  This package only loads it and
marshals PyTorch tensors into its calls.
"""
from . import _native
from ._native import SVError, lib
from .kvcache import kv_append, kv_assign, kv_attention, kv_cache, kv_commit, kv_pool, kv_read
from .prompt import prompt_attention, rope
from .verify import (build_t2d, d2t_scatter, sample, softmax_topp, topk, verify_chain, verify_tree,
                     verify_tree_sample, workspace)

__all__ = ["SVError", "lib", "build_t2d", "d2t_scatter", "kv_append", "kv_assign", "kv_attention",
           "kv_cache", "kv_commit", "kv_pool", "kv_read", "prompt_attention", "rope", "sample",
           "softmax_topp", "topk", "verify_chain", "verify_tree", "verify_tree_sample", "workspace",
           "_native"]
