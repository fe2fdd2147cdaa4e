"""MATE token-mix core of LinGen on NVIDIA B200 (sm_100a).

The computation lives in libmate.so (C ABI: include/mate.h); this package
only loads it and marshals torch tensors into its calls.
"""
from .api import (Codes, bissd, bissd_workspace, block, block_norm, compose, frontend, frontend_i8, gate_norm,
                  gate_norm_i8, linear, linear_i8, mate_bissd_fwd, mate_bissd_workspace_bytes, mate_block_norm_fwd,
                  mate_compose_fwd, mate_debug_rms_map, mate_debug_tesa_map, mate_frontend_fwd, mate_frontend_i8_fwd,
                  mate_frontend_workspace_bytes, mate_gate_norm_fwd, mate_gate_norm_i8_fwd, mate_last_error,
                  mate_linear_i8_fwd, mate_quant_rows_fwd, mate_version, modulation, quantize_block, quantize_rows,
                  rms_map, stack, tesa, tesa_fwd, tesa_map)
from ._lib import MateError, load

__all__ = ["Codes", "bissd", "bissd_workspace", "block", "block_norm", "compose", "frontend", "frontend_i8", "gate_norm",
           "gate_norm_i8", "linear", "linear_i8", "mate_bissd_fwd", "mate_bissd_workspace_bytes", "mate_block_norm_fwd",
           "mate_compose_fwd", "mate_frontend_fwd", "mate_frontend_i8_fwd", "mate_gate_norm_fwd", "mate_gate_norm_i8_fwd",
           "mate_frontend_workspace_bytes", "mate_debug_rms_map", "mate_debug_tesa_map", "mate_last_error",
           "mate_linear_i8_fwd", "mate_quant_rows_fwd", "mate_version", "modulation", "quantize_block", "quantize_rows",
           "rms_map", "stack", "tesa", "tesa_fwd", "tesa_map", "MateError", "load"]
