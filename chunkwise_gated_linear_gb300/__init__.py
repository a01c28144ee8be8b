"""Chunkwise forward pass of the gated delta rule with a per-channel gate (Kimi Delta
Attention) for GB300 (sm_103a): a C-ABI CUDA library (``include/kda.h``,
``lib/libkda.so``) and its thin Python binding (:mod:`.kda`). The operators around the recurrence in
a model's block (``include/kda_mixer.h``: short causal convolution, selective state space scan,
gated output norm, residual update with norms) are bound in :mod:`.mixer`, those of a softmax-attention
layer between recurrent ones (``include/kda_attention.h``: norms of queries and keys with the position
rotation, paged key-value cache, attention of the next tokens over it) in :mod:`.attention`."""

from .attention import (  # noqa: F401
    KVCache,
    kv_cache_read,
    kv_cache_write,
    paged_attn_step,
    qk_norm_bwd,
    qk_norm_fwd,
    qk_norm_step,
    rope_frequencies,
)
from .kda import (  # noqa: F401
    KdaError,
    chunk_kda_bwd,
    chunk_kda_fwd,
    kda_bwd_params,
    kda_chunk_bwd,
    kda_chunk_fwd,
    kda_chunk_fwd_ex,
    kda_chunk_fwd_f32,
    kda_chunk_fwd_fused,
    kda_chunk_fwd_noalloc,
    kda_frontend,
    kda_fwd_params,
    kda_get_device_error,
    kda_recurrent_fwd,
    kda_recurrent_fwd_ex,
    kda_recurrent_fwd_fused,
    lib,
    status_string,
)
from .mixer import (  # noqa: F401
    block_norm_bwd,
    block_norm_fwd,
    causal_conv_bwd,
    causal_conv_fwd,
    causal_conv_step,
    gated_norm_bwd,
    gated_norm_fwd,
    selective_scan_bwd,
    selective_scan_fwd,
    selective_scan_step,
)
