"""B200-native Mamba-2 SSD scan: chunked forward and decode step (sm_100a),
and the operators around it.

The compute lives in libssd.so (C ABI in include/ssd.h); ``ssd`` is its
Python binding.  ``inputs`` holds the seeded synthetic workloads.
"""
from . import inputs  # noqa: F401
from .ssd import (  # noqa: F401
    SSDError,
    alloc_workspace,
    bc_norm_rotate_bwd,
    bc_norm_rotate_fwd,
    chunk_scan_fwd,
    gated_scan_bwd,
    gated_scan_fwd,
    gated_scan_fwd_states,
    gated_step,
    linear_bwd,
    linear_fwd,
    linear_fwd_preact,
    load_library,
    read_device_status,
    step,
    workspace_size,
)
