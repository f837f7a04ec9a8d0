"""B200-native chunkwise DeltaNet forward pass (with Gated DeltaNet, Gated Delta
Product and Kimi Delta Attention), the single-token form of these recurrences on a
cache of states, the gated linear recurrence with its backward pass, and the norms
around a block with theirs.

The computation lives in a CUDA library for sm_100a (``csrc/``, C ABI in
``include/deltanet.h``); this package only builds it, marshals arguments and
draws synthetic inputs (``workloads``).
"""
from ._lib import (DeltaNetError, chunk_state_rows, deltanet_fwd,  # noqa: F401
                   deltanet_fwd_noalloc, deltanet_fwd_states, gated_deltanet_fwd, gated_deltaproduct_fwd, get_error, last_launches,
                   last_schedule, load, release_workspace, set_kernel_events, status_string,
                   test_set_wait, kda_fwd, deltanet_step, deltanet_scan_fwd, deltanet_scan_bwd,
                   deltanet_scan_step, deltanet_norm_fwd, deltanet_norm_bwd, NormGrads)

__all__ = ["deltanet_fwd", "gated_deltanet_fwd", "gated_deltaproduct_fwd", "kda_fwd",
           "deltanet_fwd_states", "chunk_state_rows",
           "deltanet_step", "deltanet_scan_fwd", "deltanet_scan_bwd", "deltanet_scan_step",
           "deltanet_norm_fwd", "deltanet_norm_bwd", "NormGrads",
           "deltanet_fwd_noalloc", "get_error", "release_workspace", "last_schedule",
           "last_launches", "set_kernel_events", "status_string", "test_set_wait",
           "DeltaNetError", "load"]
