"""Kimi Delta Attention gated delta-rule scan for GB300 (sm_103a), the gated linear
recurrence beside it, the norms around both, and the pool of states that a serving
loop keeps, in fp32 or parked in 8 bits.

The compute lives in libkda.so (C ABI: include/kda.h); this package is its thin
Python binding plus the seeded synthetic-input generator. Importing the package
does not load the library; the first call does, and raises if it is missing.
"""
from .kda import (DecodeGraph, chunk_fwd, chunk_fwd_host, decode_host,  # noqa: F401
                  decode_step, decode_tokens, host_workspace_size, output_gate_rmsnorm,
                  status_string, workspace_size)
from .norm import (output_gate_rmsnorm_bwd, rmsnorm_bwd, rmsnorm_fwd, rmsnorm_quant)  # noqa: F401
from .pool import state_compact, state_copy, state_dequantize, state_quantize  # noqa: F401
from .scan import gated_scan_bwd, gated_scan_fwd, gated_scan_step  # noqa: F401

__all__ = ["DecodeGraph", "chunk_fwd", "chunk_fwd_host", "decode_host", "decode_step", "decode_tokens",
           "gated_scan_bwd", "gated_scan_fwd", "gated_scan_step", "host_workspace_size",
           "output_gate_rmsnorm", "output_gate_rmsnorm_bwd", "rmsnorm_bwd", "rmsnorm_fwd", "rmsnorm_quant",
           "state_compact", "state_copy", "state_dequantize", "state_quantize", "status_string",
           "workspace_size"]
