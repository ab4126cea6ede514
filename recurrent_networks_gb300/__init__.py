"""GB300-native head-wise recurrent scan (LSTM, GRU, Elman, sLSTM): forward and
backward through time in hand-written sm_103a CUDA kernels behind a C ABI
(include/rnn.h, librnn_gb300.so); beside it the operators of a recurrent
language model around the scan: the gated linear scan and its single-token
step, the gated delta rule (a matrix for a state) and its step, the group norm
of a scan's heads, 8-bit activation checkpoints and the token embedding."""
from .functional import (checkpoint_pack, checkpoint_unpack, embedding, flashrnn, gated_delta,  # noqa: F401
                         gated_delta_step, gated_scan, gated_scan_step, group_norm, input_projection)

__all__ = ["flashrnn", "input_projection", "gated_scan", "gated_scan_step", "checkpoint_pack", "checkpoint_unpack",
           "embedding", "gated_delta", "gated_delta_step", "group_norm"]
