"""GB300-native forward pass of the gated delta rule (KDA / Gated DeltaNet / DeltaNet).

The computation lives in libkda.so (hand-written CUDA for sm_103a, C ABI in
include/kda.h).  This package only builds it and marshals torch tensors into
it:

    prefill(q, k, v, beta, log_decay, input_row_offsets, slot_idx, state_pool, chunk=64)
    decode_step(q, k, v, beta, log_decay, slot_idx, state_pool)
    gdp_prefill / gdp_decode_step   (Gated DeltaProduct: n_h transitions per token)
    prefill_bwd(...)                (the backward pass of prefill)
    conv_gates(...)                 (the front end: short conv + SiLU, gate activations)
    linear / linear_bwd             (the projections: bias, activation, residual in the epilogue)
    residual_norm / residual_norm_bwd (the norms around a block, its gate and residual scale)
    gated_norm / gated_norm_bwd     (the output norm of the recurrence with its gate)
    rotary / rotary_bwd             (rotary positions of queries and keys; rotary_frequencies)
    cache_append                    (new keys and values into the pages of a key-value cache)
    cache_attention                 (attention of new tokens over the pages)
    cache_update / cache_compact    (the page tables: continue, fork, grow, cut back, free; compact)
    cache_copy                      (pages or state slots copied within their pools)

There is no CPU or eager fallback: if the library is missing, calls raise.
"""
from .kda import (decode_step, get_device_error, make_params, prefill,  # noqa: F401
                  prefill_no_alloc, no_alloc_form, set_stage_events, uses_tensor_cores,
                  workspace_size, verify_window, fold_accepted, ring_record_elems,
                  gdp_prefill, gdp_decode_step, prefill_bwd, conv_gates)
from .layer import (linear, linear_bwd, residual_norm, residual_norm_bwd,  # noqa: F401
                    gated_norm, gated_norm_bwd)
from .cache import (CacheMoves, CacheRows, cache_append, cache_attention, cache_compact,  # noqa: F401
                    cache_copy, cache_update, rotary, rotary_bwd, rotary_frequencies)
from ._lib import KdaError, KdaParams, load  # noqa: F401

__all__ = ["prefill", "decode_step", "workspace_size", "get_device_error", "make_params",
           "set_stage_events", "prefill_no_alloc", "no_alloc_form", "uses_tensor_cores", "verify_window", "fold_accepted", "ring_record_elems", "gdp_prefill", "gdp_decode_step", "prefill_bwd", "conv_gates", "linear", "linear_bwd", "residual_norm", "residual_norm_bwd", "gated_norm", "gated_norm_bwd", "rotary", "rotary_bwd", "rotary_frequencies", "cache_append", "cache_attention", "cache_update", "cache_compact", "cache_copy", "CacheRows", "CacheMoves", "KdaError", "KdaParams", "load"]
