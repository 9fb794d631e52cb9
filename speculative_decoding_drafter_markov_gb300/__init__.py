"""DSpark per-cycle hot path on one GB300 (sm_103a).

Semi-autoregressive Markov / RNN draft with confidences, the hardware-aware
prefix scheduler and lossless verification, and the operators of the target's
pass between them (paged-cache maps and writes, attention of drafted rows,
logit rules), as hand-written CUDA kernels behind the C ABI in include/dspark.h.
This package is the thin Python binding.
"""
from ._lib import (  # noqa: F401
    BF16, F32, SCHED_ASYNC, SCHED_SYNC, DSparkError, build_tags, cache_store, draft_markov,
    draft_markov_step, draft_markov_workspace_size, draft_rnn, load, logit_rules, page_map, philox, schedule,
    tree_attention, tree_attention_workspace_size, verify,
)

__all__ = ["draft_markov", "draft_rnn", "schedule", "build_tags", "verify", "page_map", "cache_store",
           "tree_attention", "logit_rules", "philox", "load", "DSparkError"]
