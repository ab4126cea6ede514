"""GB300-native head-wise recurrent scan (LSTM, GRU, Elman, sLSTM): forward and
backward through time in hand-written sm_103a CUDA kernels behind a C ABI
(include/rnn.h, librnn_gb300.so); beside it the operators of a recurrent
language model around the scan: the gated linear scan and its single-token
step, 8-bit activation checkpoints and the token embedding."""
from .functional import (checkpoint_pack, checkpoint_unpack, embedding, flashrnn, gated_scan,  # noqa: F401
                         gated_scan_step, input_projection)

__all__ = ["flashrnn", "input_projection", "gated_scan", "gated_scan_step", "checkpoint_pack", "checkpoint_unpack",
           "embedding"]
