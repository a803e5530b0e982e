"""Kimi Delta Attention gated delta-rule scan for GB300 (sm_103a), the gated linear
recurrence beside it, and the pool of states that a serving loop keeps.

The compute lives in libkda.so (C ABI: include/kda.h); this package is its thin
Python binding plus the seeded synthetic-input generator. Importing the package
does not load the library; the first call does, and raises if it is missing.
"""
from .kda import (DecodeGraph, chunk_fwd, chunk_fwd_host, decode_host,  # noqa: F401
                  decode_step, host_workspace_size, output_gate_rmsnorm, status_string,
                  workspace_size)
from .pool import state_compact, state_copy  # noqa: F401
from .scan import gated_scan_bwd, gated_scan_fwd, gated_scan_step  # noqa: F401

__all__ = ["DecodeGraph", "chunk_fwd", "chunk_fwd_host", "decode_host", "decode_step",
           "gated_scan_bwd", "gated_scan_fwd", "gated_scan_step", "host_workspace_size",
           "output_gate_rmsnorm", "state_compact", "state_copy", "status_string", "workspace_size"]
