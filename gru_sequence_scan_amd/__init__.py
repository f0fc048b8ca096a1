"""MI355X (gfx950) multi-timestep LSTM / GRU / LSTMP / RSSM-prior forward.

A thin ctypes binding over the C ABI in include/rnn.h. Every step of the
computation runs in the library's HIP kernels; this module only marshals
PyTorch tensors (device memory) and the current HIP stream into the C
structs. There is no CPU fallback: if the native library is missing the
calls raise.

Low level (same names as the C ABI): rnn_abi_version, rnn_strerror,
rnn_workspace_bytes, rnn_forward_raw (= C rnn_forward), rnn_read_status,
rnn_device_check, rnn_plan_info, rnn_exchange_roundtrip_ns. High level: rnn_forward (LSTM / GRU / LSTMP, padded or
packed, multi-layer, bidirectional), rssm_prior_unroll and rssm_actor_unroll; training:
rnn_forward_train and rnn_backward (fp32 LSTM / LSTMP / GRU).

Operators of a decoder block: layer_norm (with the residual add), gated_scan (a gated linear recurrence) and
cross_attention (over an encoder's states), each with a _train form that also returns a context and a _backward that takes it.
"""

from .binding import (  # noqa: F401
    RNN_ABI_VERSION, RnnDesc, RnnWeights, RnnIO, RnnError, lib, lib_path,
    rnn_abi_version, rnn_strerror, rnn_workspace_bytes, rnn_forward_raw, rnn_read_status,
    rnn_device_check, rnn_exchange_roundtrip_ns, rnn_forward, rssm_prior_unroll, rssm_actor_unroll, rnn_plan_info,
    MODES, PIPE_MODES, STATUS, CLIP_CELL, CLIP_PROJ, RnnGrads, rnn_forward_train, rnn_backward, TrainContext,
)
from .block_ops import (  # noqa: F401
    RnnNormDesc, RnnGatedScanDesc, RnnGatedScanIO, RnnGatedScanGrads, BlockContext,
    layer_norm, layer_norm_train, layer_norm_backward, gated_scan, gated_scan_train, gated_scan_backward,
    RnnAttentionDesc, RnnAttentionIO, RnnAttentionGrads, cross_attention, cross_attention_train, cross_attention_backward,
)
