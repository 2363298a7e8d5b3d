"""Falcon fast-weight attention on MI355X (gfx950): chunked forward pass and
single-token recurrent step, and the backward pass of the chunked form, behind a
C ABI (include/falcon.h), with the operators that stand next to it in a layer
stack: a gated linear recurrence, the query / key norm with rotary positions,
and causal attention."""

from .falcon import (VARIANTS, FalconError, ForwardCall, chunk_fwd, chunk_fwd_varlen, recurrent_step, new_state, lib,  # noqa: F401
                     make_shape, status_string, chunk_bwd, bwd_workspace_bytes, chunk_fwd_segmented,
                     segmented_workspace_bytes)
from .layer import (SCAN_CHUNK, attention_bwd, attention_fwd, gated_scan, gated_scan_bwd, gated_scan_step,  # noqa: F401
                    qk_norm_rope, qk_norm_rope_bwd, rope_frequencies)
