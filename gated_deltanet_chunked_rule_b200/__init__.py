"""Gated DeltaNet (gated delta rule) chunked prefill for B200 (sm_100a), with the
operators around it: the short causal convolution, the selective state space scan
and the gated layer norm.

The computation lives in libgdn.so (hand-written CUDA, C ABI in
include/gdn.h); this package is its thin Python binding.
"""
from .api import (  # noqa: F401
    Problem,
    chunk_gated_delta_rule,
    chunk_gated_delta_rule_bwd,
    chunk_gated_delta_rule_fwd,
    device_status,
    recurrent_gated_delta_rule,
)
from .layer_ops import (  # noqa: F401
    causal_conv1d,
    causal_conv1d_bwd,
    causal_conv1d_fwd,
    causal_conv1d_update,
    chunk_selective_scan,
    chunk_selective_scan_bwd,
    chunk_selective_scan_fwd,
    layer_norm,
    layer_norm_bwd,
    layer_norm_fwd,
    recurrent_selective_scan,
)
from ._binding import GdnError, lib  # noqa: F401
