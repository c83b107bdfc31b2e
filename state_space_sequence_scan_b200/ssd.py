"""Python binding of libssd.so (argument marshalling only).

Every step of the scan and of the decode update runs in the CUDA library; this
module checks tensor shapes/dtypes/devices, allocates outputs and workspace
through PyTorch (device memory is the only thing PyTorch provides here), and
passes raw pointers plus the current CUDA stream across the C ABI declared in
include/ssd.h.  There is no CPU fallback: without the built library, or
without a CUDA device, every compute call raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libssd.so")

SSD_OK = 0
STATUS_NAMES = {
    0: "SSD_OK", 1: "SSD_ERR_INVALID_ARG", 2: "SSD_ERR_UNSUPPORTED", 3: "SSD_ERR_ALIGNMENT",
    4: "SSD_ERR_WORKSPACE", 5: "SSD_ERR_CUDA", 6: "SSD_ERR_DEVICE_TIMEOUT", 7: "SSD_ERR_PRECONDITION",
}
DTYPES = {torch.float32: 0, torch.bfloat16: 1}
PATHS = {"auto": 0, "simt": 1, "tensor": 2}
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2}
DZ_WIDE = 0x100
GATED_CHUNK = 64     # tokens between the gated recurrence's chunk states

EXPORTED = ("ssd_chunk_scan_workspace_size", "ssd_chunk_scan_fwd", "ssd_chunk_scan_fwd_states", "ssd_step",
            "ssd_read_device_status", "ssd_status_string", "ssd_last_cuda_error", "ssd_version",
            "ssd_trace_enable", "ssd_trace_read", "ssd_trace_kernel_name", "ssd_trace_kernel_count",
            "ssd_conv1d_silu_split", "ssd_gated_rmsnorm", "ssd_chunk_scan_fwd_varlen",
            "ssd_chunk_scan_bwd_workspace_size", "ssd_chunk_scan_bwd", "ssd_chunk_scan_bwd_varlen",
            "ssd_set_test_fault", "ssd_conv_scan_fwd", "ssd_gated_scan_workspace_size", "ssd_gated_scan_fwd",
            "ssd_gated_scan_bwd", "ssd_gated_step", "ssd_bc_norm_rotate_fwd", "ssd_bc_norm_rotate_bwd_workspace_size",
            "ssd_bc_norm_rotate_bwd", "ssd_linear_workspace_size", "ssd_linear_fwd", "ssd_linear_bwd")

_lib = None


class SSDError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str = ""):
        self.status = status
        name = STATUS_NAMES.get(status, str(status))
        super().__init__("%s failed: %s%s" % (fn, name, (" (" + detail + ")") if detail else ""))


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libssd.so and declares the C signatures.  Raises if it is missing:
    there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libssd.so is not built (%s); run python -m state_space_sequence_scan_b200.build"
                           % path)
    lib = ctypes.CDLL(path)
    vp, i64, f32, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int, ctypes.c_size_t
    lib.ssd_chunk_scan_workspace_size.restype = i32
    lib.ssd_chunk_scan_workspace_size.argtypes = [i64] * 7 + [i32, i32, ctypes.POINTER(sz)]
    lib.ssd_chunk_scan_fwd.restype = i32
    lib.ssd_chunk_scan_fwd.argtypes = [vp] * 10 + [i64] * 7 + [f32, f32, i32, i32, vp, sz, vp]
    lib.ssd_chunk_scan_fwd_varlen.restype = i32
    lib.ssd_chunk_scan_fwd_varlen.argtypes = [vp] * 12 + [i64] * 7 + [f32, f32, i32, i32, vp, sz, vp]
    lib.ssd_chunk_scan_fwd_states.restype = i32
    lib.ssd_chunk_scan_fwd_states.argtypes = [vp] * 11 + [i64] * 7 + [f32, f32, i32, i32, vp, sz, vp]
    lib.ssd_chunk_scan_bwd_workspace_size.restype = i32
    lib.ssd_chunk_scan_bwd_workspace_size.argtypes = [i64] * 7 + [i32, ctypes.POINTER(sz)]
    lib.ssd_chunk_scan_bwd.restype = i32
    lib.ssd_chunk_scan_bwd.argtypes = [vp] * 18 + [i64] * 7 + [f32, f32, i32, vp, sz, vp]
    lib.ssd_chunk_scan_bwd_varlen.restype = i32
    lib.ssd_chunk_scan_bwd_varlen.argtypes = [vp] * 19 + [i64] * 7 + [f32, f32, i32, i32, vp, sz, vp]
    lib.ssd_step.restype = i32
    lib.ssd_step.argtypes = [vp] * 9 + [i64] * 5 + [f32, f32, i32, vp]
    lib.ssd_read_device_status.restype = i32
    lib.ssd_read_device_status.argtypes = [vp, vp]
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_status_string.argtypes = [i32]
    lib.ssd_last_cuda_error.restype = i32
    lib.ssd_last_cuda_error.argtypes = []
    lib.ssd_version.restype = i32
    lib.ssd_version.argtypes = []
    lib.ssd_trace_enable.restype = i32
    lib.ssd_trace_enable.argtypes = [i32]
    lib.ssd_trace_read.restype = i32
    lib.ssd_trace_read.argtypes = [i32, ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_double)]
    lib.ssd_trace_kernel_name.restype = ctypes.c_char_p
    lib.ssd_trace_kernel_name.argtypes = [i32]
    lib.ssd_trace_kernel_count.restype = i32
    lib.ssd_trace_kernel_count.argtypes = []
    lib.ssd_set_test_fault.restype = i32
    lib.ssd_set_test_fault.argtypes = [i32]
    lib.ssd_conv1d_silu_split.restype = i32
    lib.ssd_conv1d_silu_split.argtypes = [vp] * 6 + [i64] * 7 + [i32, vp]
    lib.ssd_gated_rmsnorm.restype = i32
    lib.ssd_gated_rmsnorm.argtypes = [vp] * 4 + [i64] * 3 + [f32, i32, vp]
    lib.ssd_conv_scan_fwd.restype = i32
    lib.ssd_conv_scan_fwd.argtypes = [vp] * 3 + [i64] + [vp] * 7 + [i64] * 7 + [f32, f32, i32, vp, sz, vp]
    lib.ssd_gated_scan_workspace_size.restype = i32
    lib.ssd_gated_scan_workspace_size.argtypes = [i64] * 3 + [i32, i32, ctypes.POINTER(sz)]
    lib.ssd_gated_scan_fwd.restype = i32
    lib.ssd_gated_scan_fwd.argtypes = [vp] * 9 + [i64] * 5 + [f32, i32, vp, sz, vp]
    lib.ssd_gated_scan_bwd.restype = i32
    lib.ssd_gated_scan_bwd.argtypes = [vp] * 14 + [i64] * 6 + [f32, i32, vp, sz, vp]
    lib.ssd_gated_step.restype = i32
    lib.ssd_gated_step.argtypes = [vp] * 6 + [i64] * 4 + [f32, i32, vp]
    lib.ssd_bc_norm_rotate_fwd.restype = i32
    lib.ssd_bc_norm_rotate_fwd.argtypes = [vp] * 8 + [i64] * 5 + [f32, i32, i32, vp]
    lib.ssd_bc_norm_rotate_bwd_workspace_size.restype = i32
    lib.ssd_bc_norm_rotate_bwd_workspace_size.argtypes = [i64] * 4 + [ctypes.POINTER(sz)]
    lib.ssd_bc_norm_rotate_bwd.restype = i32
    lib.ssd_bc_norm_rotate_bwd.argtypes = [vp] * 12 + [i64] * 5 + [f32, i32, i32, vp, sz, vp]
    lib.ssd_linear_workspace_size.restype = i32
    lib.ssd_linear_workspace_size.argtypes = [i64] * 3 + [i32, i32, ctypes.POINTER(sz)]
    lib.ssd_linear_fwd.restype = i32
    lib.ssd_linear_fwd.argtypes = [vp] * 6 + [i64] * 3 + [i32, i32, i32, vp, sz, vp]
    lib.ssd_linear_bwd.restype = i32
    lib.ssd_linear_bwd.argtypes = [vp] * 7 + [i64] * 3 + [i32, i32, vp, sz, vp]
    _lib = lib
    return lib


def set_test_fault(kind: int) -> None:
    """TEST ONLY (ssd_set_test_fault): makes the waits of one kind of call run
    out, so that its device-side timeout path runs: kind 1 the tensor-path
    scan's, 2 the gated recurrence's, 3 the projections' on tcgen05; kind 0
    restores normal operation."""
    _check("ssd_set_test_fault", load_library().ssd_set_test_fault(int(kind)))


def _check(fn: str, st: int):
    if st != SSD_OK:
        detail = ""
        if st == 5:
            detail = "cudaError %d" % load_library().ssd_last_cuda_error()
        raise SSDError(fn, st, detail)


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(dev: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need_cuda(name: str, t: torch.Tensor, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def workspace_size(batch: int, seqlen: int, nheads: int, head_dim: int, state_dim: int, ngroups: int,
                   chunk_size: int, dtype: torch.dtype = torch.bfloat16, path: str = "auto") -> int:
    lib = load_library()
    out = ctypes.c_size_t(0)
    _check("ssd_chunk_scan_workspace_size", lib.ssd_chunk_scan_workspace_size(
        batch, seqlen, nheads, head_dim, state_dim, ngroups, chunk_size, DTYPES[dtype], PATHS[path],
        ctypes.byref(out)))
    return int(out.value)


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    """Workspace as a uint8 CUDA tensor (PyTorch allocations are 256-byte aligned)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def chunk_scan_fwd(x: torch.Tensor, dt_raw: torch.Tensor, dt_bias: torch.Tensor, A: torch.Tensor,
                   B: torch.Tensor, C: torch.Tensor, D: torch.Tensor,
                   init_state: Optional[torch.Tensor] = None, chunk_size: int = 256,
                   dt_limit: Tuple[float, float] = (0.0, math.inf), path: str = "auto",
                   workspace: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                   final_state: Optional[torch.Tensor] = None,
                   want_final_state: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunked forward scan.  Shapes as in include/ssd.h:
    x [b,L,H,P], dt_raw [b,L,H] f32, dt_bias/A/D [H] f32, B/C [b,L,G,N] (same
    dtype as x, f32 or bf16), init_state [b,H,N,P] f32 or None.
    Returns (y [b,L,H,P] f32, final_state [b,H,N,P] f32 or None)."""
    lib = load_library()
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [b,L,H,P] and B, C [b,L,G,N]")
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev = x.device
    _need_cuda("x", x)
    if x.dtype not in DTYPES:
        raise ValueError("x/B/C must be float32 or bfloat16")
    _need_cuda("B", B, x.dtype, (b, L, G, N))
    _need_cuda("C", C, x.dtype, (b, L, G, N))
    _need_cuda("dt_raw", dt_raw, torch.float32, (b, L, H))
    for nm, t in (("dt_bias", dt_bias), ("A", A), ("D", D)):
        _need_cuda(nm, t, torch.float32, (H,))
    if init_state is not None:
        _need_cuda("init_state", init_state, torch.float32, (b, H, N, P))
    if y is None:
        y = torch.empty((b, L, H, P), dtype=torch.float32, device=dev)
    else:
        _need_cuda("y", y, torch.float32, (b, L, H, P))
    if want_final_state and final_state is None:
        final_state = torch.empty((b, H, N, P), dtype=torch.float32, device=dev)
    elif final_state is not None:
        _need_cuda("final_state", final_state, torch.float32, (b, H, N, P))
    need = workspace_size(b, L, H, P, N, G, chunk_size, x.dtype, path)
    if workspace is None:
        workspace = alloc_workspace(need, dev)
    st = lib.ssd_chunk_scan_fwd(
        _ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(init_state),
        _ptr(y), _ptr(final_state), b, L, H, P, N, G, int(chunk_size),
        float(dt_limit[0]), float(dt_limit[1]), DTYPES[x.dtype], PATHS[path],
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(dev))
    _check("ssd_chunk_scan_fwd", st)
    return y, final_state


def chunk_scan_fwd_states(x: torch.Tensor, dt_raw: torch.Tensor, dt_bias: torch.Tensor, A: torch.Tensor,
                          B: torch.Tensor, C: torch.Tensor, D: torch.Tensor,
                          init_state: Optional[torch.Tensor] = None, chunk_size: int = 256,
                          dt_limit: Tuple[float, float] = (0.0, math.inf), path: str = "auto",
                          workspace: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                          final_state: Optional[torch.Tensor] = None,
                          chunk_states: Optional[torch.Tensor] = None
                          ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """chunk_scan_fwd that also returns the chunk-boundary states
    [b, ceil(L/chunk_size), H, N, P] f32 (ssd_chunk_scan_fwd_states): chunk c
    holds the state after token min((c+1) chunk_size, L) - 1.  Under
    path="auto" a chunk size that is not a multiple of 128 runs on the SIMT
    path, the one that has the state at any token."""
    lib = load_library()
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [b,L,H,P] and B, C [b,L,G,N]")
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev = x.device
    _need_cuda("x", x)
    if x.dtype not in DTYPES:
        raise ValueError("x/B/C must be float32 or bfloat16")
    _need_cuda("B", B, x.dtype, (b, L, G, N))
    _need_cuda("C", C, x.dtype, (b, L, G, N))
    _need_cuda("dt_raw", dt_raw, torch.float32, (b, L, H))
    for nm, t in (("dt_bias", dt_bias), ("A", A), ("D", D)):
        _need_cuda(nm, t, torch.float32, (H,))
    if init_state is not None:
        _need_cuda("init_state", init_state, torch.float32, (b, H, N, P))
    if path == "auto" and int(chunk_size) % 128 != 0:
        path = "simt"
    nc = (L + int(chunk_size) - 1) // int(chunk_size)
    if y is None:
        y = torch.empty((b, L, H, P), dtype=torch.float32, device=dev)
    else:
        _need_cuda("y", y, torch.float32, (b, L, H, P))
    if final_state is None:
        final_state = torch.empty((b, H, N, P), dtype=torch.float32, device=dev)
    else:
        _need_cuda("final_state", final_state, torch.float32, (b, H, N, P))
    if chunk_states is None:
        chunk_states = torch.empty((b, nc, H, N, P), dtype=torch.float32, device=dev)
    else:
        _need_cuda("chunk_states", chunk_states, torch.float32, (b, nc, H, N, P))
    need = workspace_size(b, L, H, P, N, G, chunk_size, x.dtype, path)
    if workspace is None:
        workspace = alloc_workspace(need, dev)
    st = lib.ssd_chunk_scan_fwd_states(
        _ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(init_state),
        _ptr(y), _ptr(final_state), _ptr(chunk_states), b, L, H, P, N, G, int(chunk_size),
        float(dt_limit[0]), float(dt_limit[1]), DTYPES[x.dtype], PATHS[path],
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(dev))
    _check("ssd_chunk_scan_fwd_states", st)
    return y, final_state, chunk_states


def bwd_workspace_size(b: int, L: int, H: int, P: int, N: int, G: int, Q: int, in_dtype=torch.bfloat16) -> int:
    """Bytes of workspace ssd_chunk_scan_bwd needs for these sizes."""
    lib = load_library()
    out = ctypes.c_size_t(0)
    _check("ssd_chunk_scan_bwd_workspace_size",
           lib.ssd_chunk_scan_bwd_workspace_size(b, L, H, P, N, G, Q, DTYPES[in_dtype], ctypes.byref(out)))
    return int(out.value)


def chunk_scan_bwd(x: torch.Tensor, dt_raw: torch.Tensor, dt_bias: torch.Tensor, A: torch.Tensor,
                   B: torch.Tensor, C: torch.Tensor, D: torch.Tensor, dy: torch.Tensor,
                   dfinal_state: Optional[torch.Tensor] = None, init_state: Optional[torch.Tensor] = None,
                   chunk_size: int = 256, dt_limit: Tuple[float, float] = (0.0, math.inf),
                   workspace: Optional[torch.Tensor] = None, want_dinit: bool = True,
                   out: Optional[dict] = None, seq_idx: Optional[torch.Tensor] = None,
                   path: str = "simt") -> dict:
    """Deterministic backward of chunk_scan_fwd (ssd_chunk_scan_bwd), or of
    chunk_scan_fwd_varlen with the same seq_idx [b, L] int32 (packed rows,
    ssd_chunk_scan_bwd_varlen): the gradients of <dy, y> + <dfinal_state,
    final_state> with respect to every input, float32, keyed by input name
    ("x", "dt_raw", "dt_bias", "A", "B", "C", "D", "init_state"; the last None
    unless want_dinit).  `out` may hold preallocated outputs under the same
    keys.  path "simt" (fp32 CUDA cores), "tensor" (the block products on the
    tensor cores, bf16 inputs: the forward tensor path's precision) or
    "auto" (tensor where it applies)."""
    lib = load_library()
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [b,L,H,P] and B, C [b,L,G,N]")
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev = x.device
    _need_cuda("x", x)
    if x.dtype not in DTYPES:
        raise ValueError("x/B/C must be float32 or bfloat16")
    _need_cuda("B", B, x.dtype, (b, L, G, N))
    _need_cuda("C", C, x.dtype, (b, L, G, N))
    _need_cuda("dt_raw", dt_raw, torch.float32, (b, L, H))
    _need_cuda("dy", dy, torch.float32, (b, L, H, P))
    for nm, t in (("dt_bias", dt_bias), ("A", A), ("D", D)):
        _need_cuda(nm, t, torch.float32, (H,))
    for nm, t in (("init_state", init_state), ("dfinal_state", dfinal_state)):
        if t is not None:
            _need_cuda(nm, t, torch.float32, (b, H, N, P))
    f = torch.float32
    shapes = {"x": (b, L, H, P), "dt_raw": (b, L, H), "dt_bias": (H,), "A": (H,), "B": (b, L, G, N),
              "C": (b, L, G, N), "D": (H,), "init_state": (b, H, N, P)}
    g = dict(out or {})
    for k, shp in shapes.items():
        if k == "init_state" and not want_dinit:
            g[k] = None
            continue
        if g.get(k) is None:
            g[k] = torch.empty(shp, dtype=f, device=dev)
        else:
            _need_cuda("out[%s]" % k, g[k], f, shp)
    Q = int(chunk_size)
    need = bwd_workspace_size(b, L, H, P, N, G, Q, x.dtype)
    if workspace is None:
        workspace = alloc_workspace(need, dev)
    if seq_idx is not None:
        _need_cuda("seq_idx", seq_idx, torch.int32, (b, L))
    st = lib.ssd_chunk_scan_bwd_varlen(
        _ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(init_state), _ptr(seq_idx),
        _ptr(dy),
        _ptr(dfinal_state), _ptr(g["x"]), _ptr(g["dt_raw"]), _ptr(g["dt_bias"]), _ptr(g["A"]), _ptr(g["B"]),
        _ptr(g["C"]), _ptr(g["D"]), _ptr(g["init_state"]), b, L, H, P, N, G, Q, float(dt_limit[0]),
        float(dt_limit[1]), DTYPES[x.dtype], PATHS[path], _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(dev))
    _check("ssd_chunk_scan_bwd_varlen", st)
    return g


def chunk_scan_fwd_varlen(x: torch.Tensor, dt_raw: torch.Tensor, dt_bias: torch.Tensor, A: torch.Tensor,
                          B: torch.Tensor, C: torch.Tensor, D: torch.Tensor, seq_idx: torch.Tensor,
                          init_state: Optional[torch.Tensor] = None, chunk_size: int = 256,
                          dt_limit: Tuple[float, float] = (0.0, math.inf), path: str = "auto",
                          workspace: Optional[torch.Tensor] = None, want_chunk_states: bool = False
                          ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Packed rows (ssd_chunk_scan_fwd_varlen): seq_idx [b, L] int32 document
    ids; the state restarts from zero at every document start (a row's first
    document from init_state).  Returns (y, final state, chunk-boundary
    states or None); with the states, path="auto" and a chunk size that is
    not a multiple of 128 runs on the SIMT path."""
    lib = load_library()
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [b,L,H,P] and B, C [b,L,G,N]")
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev = x.device
    _need_cuda("x", x)
    if x.dtype not in DTYPES:
        raise ValueError("x/B/C must be float32 or bfloat16")
    _need_cuda("B", B, x.dtype, (b, L, G, N))
    _need_cuda("C", C, x.dtype, (b, L, G, N))
    _need_cuda("dt_raw", dt_raw, torch.float32, (b, L, H))
    _need_cuda("seq_idx", seq_idx, torch.int32, (b, L))
    for nm, t in (("dt_bias", dt_bias), ("A", A), ("D", D)):
        _need_cuda(nm, t, torch.float32, (H,))
    if init_state is not None:
        _need_cuda("init_state", init_state, torch.float32, (b, H, N, P))
    Q = int(chunk_size)
    y = torch.empty((b, L, H, P), dtype=torch.float32, device=dev)
    fs = torch.empty((b, H, N, P), dtype=torch.float32, device=dev)
    cs = torch.empty((b, (L + Q - 1) // Q, H, N, P), dtype=torch.float32, device=dev) if want_chunk_states else None
    if want_chunk_states and path == "auto" and Q % 128 != 0:
        path = "simt"
    need = workspace_size(b, L, H, P, N, G, Q, x.dtype, path)
    if workspace is None:
        workspace = alloc_workspace(need, dev)
    st = lib.ssd_chunk_scan_fwd_varlen(
        _ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(init_state), _ptr(seq_idx),
        _ptr(y), _ptr(fs), _ptr(cs), b, L, H, P, N, G, Q, float(dt_limit[0]), float(dt_limit[1]),
        DTYPES[x.dtype], PATHS[path], _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(dev))
    _check("ssd_chunk_scan_fwd_varlen", st)
    return y, fs, cs


def conv1d_silu_split(xbc: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor, nheads: int, head_dim: int,
                      ngroups: int, state_dim: int) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Causal depthwise conv1d + SiLU over xbc [b, L, H*P + 2*G*N] (channels
    x | B | C), split into the scan's x [b,L,H,P], B and C [b,L,G,N] (same
    dtype as xbc).  weight [Cd, K] f32, bias [Cd] f32 (ssd_conv1d_silu_split)."""
    lib = load_library()
    if xbc.dim() != 3 or weight.dim() != 2:
        raise ValueError("xbc must be [b, L, Cd] and weight [Cd, K]")
    b, L, Cd = xbc.shape
    if Cd != nheads * head_dim + 2 * ngroups * state_dim:
        raise ValueError("xbc has %d channels, not H*P + 2*G*N" % Cd)
    _need_cuda("xbc", xbc)
    if xbc.dtype not in DTYPES:
        raise ValueError("xbc must be float32 or bfloat16")
    _need_cuda("weight", weight, torch.float32, (Cd, weight.shape[1]))
    _need_cuda("bias", bias, torch.float32, (Cd,))
    dev = xbc.device
    x = torch.empty((b, L, nheads, head_dim), dtype=xbc.dtype, device=dev)
    B = torch.empty((b, L, ngroups, state_dim), dtype=xbc.dtype, device=dev)
    C = torch.empty_like(B)
    st = lib.ssd_conv1d_silu_split(_ptr(xbc), _ptr(weight), _ptr(bias), _ptr(x), _ptr(B), _ptr(C), b, L, nheads,
                                   head_dim, ngroups, state_dim, weight.shape[1], DTYPES[xbc.dtype], _stream(dev))
    _check("ssd_conv1d_silu_split", st)
    return x, B, C


def conv_scan_fwd(xbc: torch.Tensor, conv_weight: torch.Tensor, conv_bias: torch.Tensor, dt_raw: torch.Tensor,
                  dt_bias: torch.Tensor, A: torch.Tensor, D: torch.Tensor, nheads: int, head_dim: int,
                  ngroups: int, state_dim: int, init_state: Optional[torch.Tensor] = None, chunk_size: int = 256,
                  dt_limit: Tuple[float, float] = (0.0, math.inf), workspace: Optional[torch.Tensor] = None,
                  y: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
                  want_final_state: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The conv1d and the scan in the combined arrangement (ssd_conv_scan_fwd):
    y and final_state of chunk_scan_fwd(*conv1d_silu_split(xbc, ...)) without
    writing x, B, C.  xbc [b, L, H*P + 2*G*N] bf16, conv_weight [Cd, 4] f32,
    conv_bias [Cd] f32; the rest as for chunk_scan_fwd (tensor-core shapes)."""
    lib = load_library()
    if xbc.dim() != 3:
        raise ValueError("xbc must be [b, L, Cd]")
    b, L, Cd = xbc.shape
    H, P, G, N = int(nheads), int(head_dim), int(ngroups), int(state_dim)
    if Cd != H * P + 2 * G * N:
        raise ValueError("xbc has %d channels, not H*P + 2*G*N" % Cd)
    dev = xbc.device
    _need_cuda("xbc", xbc, torch.bfloat16)
    _need_cuda("conv_weight", conv_weight, torch.float32, (Cd, conv_weight.shape[-1]))
    _need_cuda("conv_bias", conv_bias, torch.float32, (Cd,))
    _need_cuda("dt_raw", dt_raw, torch.float32, (b, L, H))
    for nm, t in (("dt_bias", dt_bias), ("A", A), ("D", D)):
        _need_cuda(nm, t, torch.float32, (H,))
    if init_state is not None:
        _need_cuda("init_state", init_state, torch.float32, (b, H, N, P))
    if y is None:
        y = torch.empty((b, L, H, P), dtype=torch.float32, device=dev)
    else:
        _need_cuda("y", y, torch.float32, (b, L, H, P))
    if want_final_state and final_state is None:
        final_state = torch.empty((b, H, N, P), dtype=torch.float32, device=dev)
    elif final_state is not None:
        _need_cuda("final_state", final_state, torch.float32, (b, H, N, P))
    need = workspace_size(b, L, H, P, N, G, chunk_size, torch.bfloat16, "tensor")
    if workspace is None:
        workspace = alloc_workspace(need, dev)
    st = lib.ssd_conv_scan_fwd(
        _ptr(xbc), _ptr(conv_weight), _ptr(conv_bias), conv_weight.shape[-1], _ptr(dt_raw), _ptr(dt_bias), _ptr(A),
        _ptr(D), _ptr(init_state), _ptr(y), _ptr(final_state), b, L, H, P, N, G, int(chunk_size),
        float(dt_limit[0]), float(dt_limit[1]), DTYPES[xbc.dtype], _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(dev))
    _check("ssd_conv_scan_fwd", st)
    return y, final_state


def gated_rmsnorm(y: torch.Tensor, z: torch.Tensor, weight: torch.Tensor, group_size: int,
                  eps: float = 1e-5) -> torch.Tensor:
    """out = rmsnorm_over_groups(y * silu(z)) * weight, f32 (ssd_gated_rmsnorm).
    y f32 [..., D], z [..., D] f32 or bf16, weight [D] f32."""
    lib = load_library()
    D = y.shape[-1]
    _need_cuda("y", y, torch.float32)
    _need_cuda("z", z, None, tuple(y.shape))
    if z.dtype not in DTYPES:
        raise ValueError("z must be float32 or bfloat16")
    _need_cuda("weight", weight, torch.float32, (D,))
    out = torch.empty(y.shape, dtype=torch.float32, device=y.device)
    st = lib.ssd_gated_rmsnorm(_ptr(y), _ptr(z), _ptr(weight), _ptr(out), y.numel() // D, D, int(group_size),
                               float(eps), DTYPES[z.dtype], _stream(y.device))
    _check("ssd_gated_rmsnorm", st)
    return out


# ---- the operators around the scan: gated recurrence, norm and rotation of
# B and C, projections.  Their tensors may live on a device that is not the
# current one; the call switches for its launches.  Small calls are bound by
# this side, so a check that holds costs one expression, sizes of workspaces
# are remembered by their arguments, and the stream is asked for as a handle.


def _tensor(name: str, t, shape, dtype: torch.dtype, dev: torch.device) -> int:
    """Checks a contiguous tensor; its address."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev.index and \
            t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != dev:
        raise ValueError("%s must be on %s, got %s" % (name, dev, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _optional(name: str, t, shape, dtype: torch.dtype, dev: torch.device) -> Optional[int]:
    return None if t is None else _tensor(name, t, shape, dtype, dev)


def _rows(name: str, t, shape, dtype: torch.dtype, dev: torch.device) -> Tuple[int, int]:
    """Checks a tensor whose last axis is contiguous and whose rows (all other
    axes, in order) are evenly spaced; its address and the spacing."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev.index:
        if t.is_contiguous():
            return t.data_ptr(), shape[-1]
        if len(shape) == 2 and shape[0] > 1:   # halves of a step's projection
            ld, one = t.stride()
            if one == 1 and ld >= shape[1]:
                return t.data_ptr(), ld
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != dev:
        raise ValueError("%s must be on %s, got %s" % (name, dev, t.device))
    width = shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), width
    st = t.stride()
    ld = None
    span = 1                                   # rows spanned by the axes seen so far
    for n, s in zip(reversed(shape[:-1]), reversed(st[:-1])):
        if n == 1:
            continue
        if ld is None:
            ld = s
        elif s != ld * span:
            raise ValueError("%s must have evenly spaced rows" % name)
        span *= n
    ld = width if ld is None else ld
    if (st[-1] != 1 and width != 1) or ld < width:
        raise ValueError("%s must have contiguous rows that do not overlap" % name)
    return t.data_ptr(), ld


def _rows_share(p: int, q: int, rows: int, width: int, ld: int, size: int) -> bool:
    """Whether two tensors of equally spaced rows at these addresses share an
    element: their rows lie side by side, or apart."""
    if rows * width == 0:
        return False
    off = abs(q - p)
    span = ((rows - 1) * ld + width) * size
    off_row = off % (ld * size)
    return off < span and (off_row < width * size or (ld * size - off_row < width * size and off + ld * size - off_row < span))


def _like(t: torch.Tensor) -> torch.Tensor:
    """An output of t's shape and type, contiguous."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty_like(t, memory_format=torch.contiguous_format)


def _cuda_input(name: str, t) -> torch.device:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype not in DTYPES:
        raise ValueError("%s must be float32 or bfloat16" % name)
    return t.device


def _enqueue(name: str, fn, dev: torch.device, *args) -> None:
    """Calls a compute entry point on the device's current stream."""
    index = dev.index
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != SSD_OK:
        _check(name, st)


def _workspace(ws: Optional[torch.Tensor], need: int, dev: torch.device) -> Tuple[int, int, torch.Tensor]:
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not ws.is_cuda or ws.device != dev or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on %s" % dev)
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


@functools.lru_cache(maxsize=1024)
def gated_scan_workspace_size(batch: int, seqlen: int, dim: int, dtype: torch.dtype = torch.bfloat16,
                              backward: bool = False) -> int:
    """Bytes of workspace gated_scan_fwd (or gated_scan_bwd) needs."""
    out = ctypes.c_size_t(0)
    _check("ssd_gated_scan_workspace_size", load_library().ssd_gated_scan_workspace_size(
        batch, seqlen, dim, DTYPES[dtype], int(bool(backward)), ctypes.byref(out)))
    return out.value


def _gated_scan(x, r_raw, g_raw, lam, init_state, seq_idx, decay_scale, want_states, workspace):
    lib = load_library()
    dev = _cuda_input("x", x)
    if x.dim() != 3:
        raise ValueError("x must be [b, L, D]")
    b, L, D = x.shape
    f = torch.float32
    px, ldx = _rows("x", x, x.shape, x.dtype, dev)
    pr, ldr = _rows("r_raw", r_raw, x.shape, x.dtype, dev)
    pg, ldg = _rows("g_raw", g_raw, x.shape, x.dtype, dev)
    if ldr != ldg:
        raise ValueError("r_raw and g_raw must have the same row spacing")
    pl = _tensor("lam", lam, (D,), f, dev)
    pi = _optional("init_state", init_state, (b, D), f, dev)
    ps = _optional("seq_idx", seq_idx, (b, L), torch.int32, dev)
    y = _like(x)
    final = lam.new_empty((b, D))
    states = lam.new_empty((b, (L + GATED_CHUNK - 1) // GATED_CHUNK, D)) if want_states else None
    wp, wn, workspace = _workspace(workspace, gated_scan_workspace_size(b, L, D, x.dtype) if workspace is None else 0, dev)
    _enqueue("ssd_gated_scan_fwd", lib.ssd_gated_scan_fwd, dev, px, pr, pg, pl, pi, ps, y.data_ptr(), final.data_ptr(),
             None if states is None else states.data_ptr(), b, L, D, ldx, ldg, float(decay_scale), DTYPES[x.dtype], wp, wn)
    return y, final, states


def gated_scan_fwd(x: torch.Tensor, r_raw: torch.Tensor, g_raw: torch.Tensor, lam: torch.Tensor,
                   init_state: Optional[torch.Tensor] = None, seq_idx: Optional[torch.Tensor] = None,
                   decay_scale: float = 8.0, workspace: Optional[torch.Tensor] = None
                   ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gated linear recurrence (ssd_gated_scan_fwd), one decay per channel:
        h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(g_raw_t) x_t,
        a_t = exp(-decay_scale softplus(lam) sigmoid(r_raw_t)).
    x, r_raw, g_raw [b, L, D] f32 or bf16 with evenly spaced rows (r_raw and
    g_raw may be the halves of one [b, L, 2D] projection), lam [D] f32,
    init_state [b, D] f32 or None, seq_idx [b, L] int32 document ids of packed
    rows or None.  Returns (y [b, L, D] in x's type, final_state [b, D] f32)."""
    return _gated_scan(x, r_raw, g_raw, lam, init_state, seq_idx, decay_scale, False, workspace)[:2]


def gated_scan_fwd_states(x: torch.Tensor, r_raw: torch.Tensor, g_raw: torch.Tensor, lam: torch.Tensor,
                          init_state: Optional[torch.Tensor] = None, seq_idx: Optional[torch.Tensor] = None,
                          decay_scale: float = 8.0, workspace: Optional[torch.Tensor] = None
                          ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """gated_scan_fwd that also returns the chunk states [b, ceil(L / 64), D]
    f32 that gated_scan_bwd starts from: the state after token
    min(64 (c + 1), L) - 1."""
    return _gated_scan(x, r_raw, g_raw, lam, init_state, seq_idx, decay_scale, True, workspace)


def gated_scan_bwd(x: torch.Tensor, r_raw: torch.Tensor, g_raw: torch.Tensor, lam: torch.Tensor,
                   chunk_states: Optional[torch.Tensor], dy: torch.Tensor,
                   dfinal_state: Optional[torch.Tensor] = None, init_state: Optional[torch.Tensor] = None,
                   seq_idx: Optional[torch.Tensor] = None, decay_scale: float = 8.0, want_dinit: bool = True,
                   out: Optional[dict] = None, workspace: Optional[torch.Tensor] = None) -> dict:
    """Deterministic backward of gated_scan_fwd_states on the same inputs, from
    its chunk states: the gradients of <dy, y> + <dfinal_state, final_state>
    keyed by input name: "x", "r_raw", "g_raw" [b, L, D] in x's type, "lam" [D]
    f32, "init_state" [b, D] f32 (None unless want_dinit).  `out` may hold
    preallocated "r_raw" and "g_raw" with evenly spaced rows (the halves of
    one [b, L, 2D] gradient)."""
    lib = load_library()
    dev = _cuda_input("x", x)
    if x.dim() != 3:
        raise ValueError("x must be [b, L, D]")
    b, L, D = x.shape
    f, t = torch.float32, x.dtype
    px, ldx = _rows("x", x, x.shape, t, dev)
    pr, ldr = _rows("r_raw", r_raw, x.shape, t, dev)
    pg, ldg = _rows("g_raw", g_raw, x.shape, t, dev)
    if ldr != ldg:
        raise ValueError("r_raw and g_raw must have the same row spacing")
    pl = _tensor("lam", lam, (D,), f, dev)
    pi = _optional("init_state", init_state, (b, D), f, dev)
    ps = _optional("seq_idx", seq_idx, (b, L), torch.int32, dev)
    pc = _optional("chunk_states", chunk_states, (b, (L + GATED_CHUNK - 1) // GATED_CHUNK, D), f, dev)
    pdy = _tensor("dy", dy, x.shape, t, dev)
    pdf = _optional("dfinal_state", dfinal_state, (b, D), f, dev)
    dx = _like(x)
    dr, dg = (out or {}).get("r_raw"), (out or {}).get("g_raw")
    dr = _like(x) if dr is None else dr
    dg = _like(x) if dg is None else dg
    pdr, lddr = _rows("out[r_raw]", dr, x.shape, t, dev)
    pdg, lddg = _rows("out[g_raw]", dg, x.shape, t, dev)
    if lddr != lddg:
        raise ValueError("out[r_raw] and out[g_raw] must have the same row spacing")
    if out is not None and _rows_share(pdr, pdg, b * L, D, lddr, dr.element_size()):
        raise ValueError("out[r_raw] and out[g_raw] must not overlap")
    dlam = torch.empty_like(lam)
    dinit = lam.new_empty((b, D)) if want_dinit else None
    wp, wn, workspace = _workspace(
        workspace, gated_scan_workspace_size(b, L, D, t, True) if workspace is None else 0, dev)
    _enqueue("ssd_gated_scan_bwd", lib.ssd_gated_scan_bwd, dev, px, pr, pg, pl, pi, ps, pc, pdy, pdf, dx.data_ptr(), pdr,
             pdg, dlam.data_ptr(), None if dinit is None else dinit.data_ptr(), b, L, D, ldx, ldg, lddg,
             float(decay_scale), DTYPES[t], wp, wn)
    return {"x": dx, "r_raw": dr, "g_raw": dg, "lam": dlam, "init_state": dinit}


def gated_step(x: torch.Tensor, r_raw: torch.Tensor, g_raw: torch.Tensor, lam: torch.Tensor, state: torch.Tensor,
               decay_scale: float = 8.0) -> torch.Tensor:
    """One decode token of the gated recurrence: x, r_raw, g_raw [b, D], state
    [b, D] f32 updated in place.  Returns y [b, D] in x's type."""
    dev = _cuda_input("x", x)
    if x.dim() != 2:
        raise ValueError("x must be [b, D]")
    b, D = x.shape
    px, ldx = _rows("x", x, x.shape, x.dtype, dev)
    pr, ldr = _rows("r_raw", r_raw, x.shape, x.dtype, dev)
    pg, ldg = _rows("g_raw", g_raw, x.shape, x.dtype, dev)
    if ldr != ldg:
        raise ValueError("r_raw and g_raw must have the same row spacing")
    pl = _tensor("lam", lam, (D,), torch.float32, dev)
    ps = _tensor("state", state, (b, D), torch.float32, dev)
    y = _like(x)
    _enqueue("ssd_gated_step", load_library().ssd_gated_step, dev, px, pr, pg, pl, ps, y.data_ptr(), b, D, ldx, ldg,
             float(decay_scale), DTYPES[x.dtype])
    return y


def _norm_rotate_args(B, C, weight_B, weight_C, inv_freq, positions):
    dev = _cuda_input("B", B)
    if B.dim() != 4:
        raise ValueError("B and C must be [b, L, G, N]")
    b, L, G, N = B.shape
    f = torch.float32
    R = 0 if inv_freq is None else 2 * inv_freq.numel()
    if R > N:
        raise ValueError("inv_freq has %d pairs, more than state_dim / 2" % (R // 2))
    shape, t = B.shape, B.dtype
    return dev, (b, L, G, N, R), (
        _tensor("B", B, shape, t, dev), _tensor("C", C, shape, t, dev),
        _tensor("weight_B", weight_B, (N,), f, dev), _tensor("weight_C", weight_C, (N,), f, dev),
        _optional("inv_freq", inv_freq, (R // 2,), f, dev), _optional("positions", positions, (b, L), torch.int32, dev))


def bc_norm_rotate_fwd(B: torch.Tensor, C: torch.Tensor, weight_B: torch.Tensor, weight_C: torch.Tensor,
                       inv_freq: Optional[torch.Tensor], positions: Optional[torch.Tensor] = None, eps: float = 1e-5,
                       interleaved: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """RMS norm of B and C [b, L, G, N] (f32 or bf16) over N, times weight_B,
    weight_C [N] f32, then the rotation of the pairs of the first
    2 * len(inv_freq) elements by position * inv_freq (ssd_bc_norm_rotate_fwd).
    inv_freq f32, or None for the norm alone; positions [b, L] int32, or None
    for 0 .. L-1; pairs are (j, j + R/2), or (2j, 2j + 1) when interleaved.
    Returns (B_out, C_out) in B's type."""
    dev, (b, L, G, N, R), ptrs = _norm_rotate_args(B, C, weight_B, weight_C, inv_freq, positions)
    Bo, Co = torch.empty_like(B), torch.empty_like(B)
    _enqueue("ssd_bc_norm_rotate_fwd", load_library().ssd_bc_norm_rotate_fwd, dev, *ptrs, Bo.data_ptr(), Co.data_ptr(),
             b, L, G, N, R, float(eps), int(bool(interleaved)), DTYPES[B.dtype])
    return Bo, Co


@functools.lru_cache(maxsize=1024)
def bc_norm_rotate_bwd_workspace_size(batch: int, seqlen: int, ngroups: int, state_dim: int) -> int:
    out = ctypes.c_size_t(0)
    _check("ssd_bc_norm_rotate_bwd_workspace_size", load_library().ssd_bc_norm_rotate_bwd_workspace_size(
        batch, seqlen, ngroups, state_dim, ctypes.byref(out)))
    return out.value


def bc_norm_rotate_bwd(B: torch.Tensor, C: torch.Tensor, weight_B: torch.Tensor, weight_C: torch.Tensor,
                       inv_freq: Optional[torch.Tensor], dB_out: torch.Tensor, dC_out: torch.Tensor,
                       positions: Optional[torch.Tensor] = None, eps: float = 1e-5, interleaved: bool = False,
                       workspace: Optional[torch.Tensor] = None) -> dict:
    """Deterministic backward of bc_norm_rotate_fwd from its inputs and the
    gradients of its outputs: "B", "C" in B's type, "weight_B", "weight_C" [N]
    f32 (summed over tokens and groups)."""
    dev, (b, L, G, N, R), ptrs = _norm_rotate_args(B, C, weight_B, weight_C, inv_freq, positions)
    pdB = _tensor("dB_out", dB_out, B.shape, B.dtype, dev)
    pdC = _tensor("dC_out", dC_out, B.shape, B.dtype, dev)
    dB, dC = torch.empty_like(B), torch.empty_like(B)
    dwB = torch.empty_like(weight_B)
    dwC = torch.empty_like(weight_B)
    wp, wn, workspace = _workspace(
        workspace, bc_norm_rotate_bwd_workspace_size(b, L, G, N) if workspace is None else 0, dev)
    _enqueue("ssd_bc_norm_rotate_bwd", load_library().ssd_bc_norm_rotate_bwd, dev, *ptrs, pdB, pdC, dB.data_ptr(),
             dC.data_ptr(), dwB.data_ptr(), dwC.data_ptr(), b, L, G, N, R, float(eps), int(bool(interleaved)),
             DTYPES[B.dtype], wp, wn)
    return {"B": dB, "C": dC, "weight_B": dwB, "weight_C": dwC}


@functools.lru_cache(maxsize=1024)
def linear_workspace_size(rows: int, n_out: int, n_in: int, dtype: torch.dtype = torch.bfloat16,
                          backward: bool = False, wide_dz: bool = False) -> int:
    """Bytes of workspace linear_fwd (or linear_bwd) needs."""
    out = ctypes.c_size_t(0)
    _check("ssd_linear_workspace_size", load_library().ssd_linear_workspace_size(
        rows, n_out, n_in, DTYPES[dtype], (2 if wide_dz else 1) if backward else 0, ctypes.byref(out)))
    return out.value


def _linear(x, weight, bias, residual, activation, out_dtype, want_preact, workspace):
    dev = _cuda_input("x", x)
    if weight.dim() != 2 or x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError("x must be [..., n_in] and weight [n_out, n_in]")
    if activation not in ACTIVATIONS:
        raise ValueError("activation must be one of %s" % ", ".join(ACTIVATIONS))
    N, K = weight.shape
    lead = x.shape[:-1]
    M = lead.numel()
    out_dtype = x.dtype if out_dtype is None else out_dtype
    if out_dtype not in DTYPES:
        raise ValueError("out_dtype must be float32 or bfloat16")
    px = _tensor("x", x, x.shape, x.dtype, dev)
    pw = _tensor("weight", weight, (N, K), x.dtype, dev)
    pb = _optional("bias", bias, (N,), torch.float32, dev)
    pr = _optional("residual", residual, lead + (N,), out_dtype, dev)
    y = x.new_empty(lead + (N,)) if out_dtype is x.dtype else x.new_empty(lead + (N,), dtype=out_dtype)
    z = x.new_empty(lead + (N,)) if want_preact else None
    wp, wn, workspace = _workspace(workspace, linear_workspace_size(M, N, K, x.dtype) if workspace is None else 0, dev)
    _enqueue("ssd_linear_fwd", load_library().ssd_linear_fwd, dev, px, pw, pb, pr, y.data_ptr(),
             None if z is None else z.data_ptr(), M, N, K, ACTIVATIONS[activation], DTYPES[x.dtype], DTYPES[out_dtype],
             wp, wn)
    return y, z


def linear_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               residual: Optional[torch.Tensor] = None, activation: str = "none",
               out_dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A layer's projection, out = act(x W^T + bias) + residual, in one pass
    (ssd_linear_fwd).  x [..., n_in] and weight [n_out, n_in] f32 or bf16, bias
    [n_out] f32, residual [..., n_out] in the output's type; activation
    "none", "silu" or "gelu" (the erf form); out_dtype x's type (default) or
    float32."""
    return _linear(x, weight, bias, residual, activation, out_dtype, False, workspace)[0]


def linear_fwd_preact(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                      residual: Optional[torch.Tensor] = None, activation: str = "none",
                      out_dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None
                      ) -> Tuple[torch.Tensor, torch.Tensor]:
    """linear_fwd that also returns x W^T + bias in x's type, which linear_bwd
    of an activation reads: (out, preact)."""
    return _linear(x, weight, bias, residual, activation, out_dtype, True, workspace)


def linear_bwd(x: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor, preact: Optional[torch.Tensor] = None,
               activation: str = "none", want_dx: bool = True, want_dweight: bool = True, want_dbias: bool = True,
               workspace: Optional[torch.Tensor] = None, wide_dz: bool = False) -> dict:
    """Deterministic backward of linear_fwd: with dz = dy act'(preact), "x" =
    dz W and "weight" = dz^T x in x's type, "bias" = column sums of dz, f32
    (None where not wanted).  The residual's gradient is dy itself.  preact
    (linear_fwd_preact's) is needed for an activation.  With one, a bf16 call
    rounds dz to bf16 where it enters a product; wide_dz keeps 16 bits of it,
    for about twice the time (and a workspace of that size)."""
    dev = _cuda_input("x", x)
    if weight.dim() != 2 or x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError("x must be [..., n_in] and weight [n_out, n_in]")
    if activation not in ACTIVATIONS:
        raise ValueError("activation must be one of %s" % ", ".join(ACTIVATIONS))
    if activation != "none" and preact is None:
        raise ValueError("the backward of %s needs preact" % activation)
    N, K = weight.shape
    lead, t = x.shape[:-1], x.dtype
    M = lead.numel()
    px = _tensor("x", x, x.shape, t, dev)
    pw = _tensor("weight", weight, (N, K), t, dev)
    pdy = _tensor("dy", dy, lead + (N,), t, dev)
    pz = _optional("preact", preact, lead + (N,), t, dev)
    dx = _like(x) if want_dx else None
    dw = torch.empty_like(weight) if want_dweight else None
    db = torch.empty((N,), dtype=torch.float32, device=dev) if want_dbias else None
    wp, wn, workspace = _workspace(
        workspace, linear_workspace_size(M, N, K, t, True, bool(wide_dz)) if workspace is None else 0, dev)
    _enqueue("ssd_linear_bwd", load_library().ssd_linear_bwd, dev, px, pw, pdy, pz,
             None if dx is None else dx.data_ptr(), None if dw is None else dw.data_ptr(),
             None if db is None else db.data_ptr(), M, N, K, ACTIVATIONS[activation] | (DZ_WIDE if wide_dz else 0), DTYPES[t],
             wp, wn)
    return {"x": dx, "weight": dw, "bias": db}


def read_device_status(workspace: Optional[torch.Tensor]) -> int:
    """Synchronises the current stream and returns the device status code of
    the calls on `workspace`; with None, reads and clears the current
    device's status of the calls that take no workspace (conv1d)."""
    lib = load_library()
    if workspace is None:
        dev = torch.device("cuda", torch.cuda.current_device())
        return int(lib.ssd_read_device_status(None, _stream(dev)))
    return int(lib.ssd_read_device_status(_ptr(workspace), _stream(workspace.device)))


def step(x: torch.Tensor, dt_raw: torch.Tensor, dt_bias: torch.Tensor, A: torch.Tensor,
         B: torch.Tensor, C: torch.Tensor, D: torch.Tensor, state: torch.Tensor,
         dt_limit: Tuple[float, float] = (0.0, math.inf),
         y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One decode token: x [b,H,P], dt_raw [b,H] f32, B/C [b,G,N], state
    [b,H,N,P] f32 updated in place.  Returns y [b,H,P] f32."""
    lib = load_library()
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be [b,H,P] and B, C [b,G,N]")
    b, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    _need_cuda("x", x)
    if x.dtype not in DTYPES:
        raise ValueError("x/B/C must be float32 or bfloat16")
    _need_cuda("B", B, x.dtype, (b, G, N))
    _need_cuda("C", C, x.dtype, (b, G, N))
    _need_cuda("dt_raw", dt_raw, torch.float32, (b, H))
    for nm, t in (("dt_bias", dt_bias), ("A", A), ("D", D)):
        _need_cuda(nm, t, torch.float32, (H,))
    _need_cuda("state", state, torch.float32, (b, H, N, P))
    if y is None:
        y = torch.empty((b, H, P), dtype=torch.float32, device=x.device)
    else:
        _need_cuda("y", y, torch.float32, (b, H, P))
    st = lib.ssd_step(_ptr(x), _ptr(dt_raw), _ptr(dt_bias), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                      _ptr(state), _ptr(y), b, H, P, N, G, float(dt_limit[0]), float(dt_limit[1]),
                      DTYPES[x.dtype], _stream(x.device))
    _check("ssd_step", st)
    return y


def trace_enable(max_launches: int) -> None:
    """Start (max_launches > 0) or stop (0) per-kernel event tracing."""
    _check("ssd_trace_enable", load_library().ssd_trace_enable(int(max_launches)))


def trace_read() -> dict:
    """{kernel name: (launches, total device ms)} for every traced kernel."""
    lib = load_library()
    out = {}
    for k in range(lib.ssd_trace_kernel_count()):
        n = ctypes.c_int(0)
        ms = ctypes.c_double(0.0)
        _check("ssd_trace_read", lib.ssd_trace_read(k, ctypes.byref(n), ctypes.byref(ms)))
        if n.value:
            out[lib.ssd_trace_kernel_name(k).decode()] = (int(n.value), float(ms.value))
    return out
