"""ctypes binding of libssd_mi355x.so (the C ABI in include/ssd.h).

Argument marshalling only: every step of the forward pass and of the decode
step runs in the library's HIP kernels. torch provides device memory and the
current stream. The library is loaded on first use; a missing library raises
(there is no CPU fallback).
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional, Tuple

import torch

_LIB_NAME = "libssd_mi355x.so"
# SSD_MI355X_LIBRARY names another build of the same library (the sanitizer
# build the CPU checks load); by default the in-tree one.
_LIB_PATH = os.environ.get("SSD_MI355X_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)), _LIB_NAME)
_lib = None

SSD_OK = 0
STATUS = {0: "SSD_OK", 1: "SSD_ERR_INVALID_ARGUMENT", 2: "SSD_ERR_UNSUPPORTED",
          3: "SSD_ERR_WORKSPACE_TOO_SMALL", 4: "SSD_ERR_HIP"}
DTYPE_F32, DTYPE_BF16 = 0, 1

# Every symbol include/ssd.h declares.
EXPORTS = ("ssd_abi_version", "ssd_status_string", "ssd_default_state_block", "ssd_fwd_layout",
           "ssd_fwd_workspace_bytes", "ssd_fwd", "ssd_fwd_ex", "ssd_chunk_cumsum", "ssd_chunk_state",
           "ssd_state_passing", "ssd_chunk_scan", "ssd_step", "ssd_fwd_mamba2", "ssd_step_mamba2",
           "ssd_bwd_workspace_bytes", "ssd_bwd", "ssd_set_state_chain", "ssd_state_chain_cooperative",
           "ssd_chunk_scan_kernel", "ssd_bwd_mamba2_workspace_bytes", "ssd_bwd_mamba2", "ssd_fwd_noalloc",
           "ssd_lin_attn_workspace_bytes", "ssd_lin_attn_bwd_workspace_bytes", "ssd_lin_attn_fwd", "ssd_lin_attn_bwd",
           "ssd_lin_attn_step", "ssd_group_norm_workspace_bytes", "ssd_group_norm", "ssd_group_norm_bwd",
           "ssd_pages_copy", "ssd_pages_clear", "ssd_pages_compact_workspace_bytes", "ssd_pages_compact",
           "ssd_gated_delta_workspace_bytes", "ssd_gated_delta_bwd_workspace_bytes", "ssd_gated_delta_fwd",
           "ssd_gated_delta_bwd", "ssd_gated_delta_step", "ssd_rotary")


class SSDError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")


class Shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32), ("nheads", ctypes.c_int32),
                ("ngroups", ctypes.c_int32), ("headdim", ctypes.c_int32), ("dstate", ctypes.c_int32),
                ("num_seqs", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Layout(ctypes.Structure):
    _fields_ = [("slots_per_row", ctypes.c_int64), ("nslots", ctypes.c_int64), ("blocks_per_row", ctypes.c_int64),
                ("nblocks", ctypes.c_int64), ("table_offset", ctypes.c_size_t),
                ("block_table_offset", ctypes.c_size_t), ("cumsum_offset", ctypes.c_size_t),
                ("key_cumsum_offset", ctypes.c_size_t), ("block_decay_offset", ctypes.c_size_t), ("block_states_offset", ctypes.c_size_t),
                ("start_states_offset", ctypes.c_size_t), ("total_bytes", ctypes.c_size_t)]


class LinShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32), ("nheads", ctypes.c_int32),
                ("nkv_heads", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("num_seqs", ctypes.c_int32), ("dtype", ctypes.c_int32), ("q_row", ctypes.c_int64),
                ("k_row", ctypes.c_int64), ("v_row", ctypes.c_int64)]


class NormShape(ctypes.Structure):
    _fields_ = [("samples", ctypes.c_int32), ("positions", ctypes.c_int32), ("channels", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("x_row", ctypes.c_int64), ("z_row", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("gate", ctypes.c_int32), ("center", ctypes.c_int32)]


class PagesShape(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int32), ("slots", ctypes.c_int32), ("page_bytes", ctypes.c_int64)]


class DeltaShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32), ("nheads", ctypes.c_int32),
                ("nqk_heads", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("num_seqs", ctypes.c_int32), ("dtype", ctypes.c_int32), ("q_row", ctypes.c_int64),
                ("k_row", ctypes.c_int64), ("v_row", ctypes.c_int64)]


class RotaryShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("k_heads", ctypes.c_int32), ("dim", ctypes.c_int32), ("rot", ctypes.c_int32),
                ("num_seqs", ctypes.c_int32), ("dtype", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("q_row", ctypes.c_int64), ("k_row", ctypes.c_int64),
                ("q_out_row", ctypes.c_int64), ("k_out_row", ctypes.c_int64)]


def library_path() -> str:
    return _LIB_PATH


def lib():
    """The loaded library; raises when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_NAME} is not built (python -m ssd_chunked_scan_fwd_amd.build)")
        L = ctypes.CDLL(_LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        shp = ctypes.POINTER(Shape)
        L.ssd_abi_version.restype = i32
        L.ssd_abi_version.argtypes = []
        L.ssd_status_string.restype = ctypes.c_char_p
        L.ssd_status_string.argtypes = [ctypes.c_int]
        L.ssd_default_state_block.restype = i32
        L.ssd_default_state_block.argtypes = [shp, i32]
        L.ssd_fwd_layout.restype = ctypes.c_int
        L.ssd_fwd_layout.argtypes = [shp, i32, i32, ctypes.POINTER(Layout)]
        L.ssd_fwd_workspace_bytes.restype = ctypes.c_int
        L.ssd_fwd_workspace_bytes.argtypes = [shp, i32, i32, ctypes.POINTER(sz)]
        L.ssd_fwd.restype = ctypes.c_int
        L.ssd_fwd.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, shp, vp, sz, vp]
        L.ssd_fwd_noalloc.restype = ctypes.c_int
        L.ssd_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, shp, vp]
        L.ssd_fwd_ex.restype = ctypes.c_int
        L.ssd_fwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, vp, vp, shp, vp, sz, vp]
        L.ssd_chunk_cumsum.restype = ctypes.c_int
        L.ssd_chunk_cumsum.argtypes = [vp, vp, i32, i32, shp, vp, sz, vp]
        L.ssd_chunk_state.restype = ctypes.c_int
        L.ssd_chunk_state.argtypes = [vp, vp, vp, i32, i32, shp, vp, sz, vp]
        L.ssd_state_passing.restype = ctypes.c_int
        L.ssd_state_passing.argtypes = [vp, vp, i32, i32, vp, shp, vp, sz, vp]
        L.ssd_chunk_scan.restype = ctypes.c_int
        L.ssd_chunk_scan.argtypes = [vp, vp, vp, vp, i32, i32, vp, shp, vp, sz, vp]
        L.ssd_step.restype = ctypes.c_int
        L.ssd_step.argtypes = [vp, vp, vp, vp, vp, vp, shp, vp]
        L.ssd_fwd_mamba2.restype = ctypes.c_int
        L.ssd_fwd_mamba2.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, vp, vp, shp, vp, sz, vp]
        L.ssd_bwd_workspace_bytes.restype = ctypes.c_int
        L.ssd_bwd_workspace_bytes.argtypes = [shp, i32, i32, ctypes.POINTER(sz)]
        L.ssd_bwd.restype = ctypes.c_int
        L.ssd_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, shp, vp, sz, vp]
        L.ssd_step_mamba2.restype = ctypes.c_int
        L.ssd_step_mamba2.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, shp, vp]
        L.ssd_set_state_chain.restype = i32
        L.ssd_set_state_chain.argtypes = [i32]
        L.ssd_state_chain_cooperative.restype = ctypes.c_int
        L.ssd_state_chain_cooperative.argtypes = [shp, i32, i32, ctypes.POINTER(i32)]
        L.ssd_chunk_scan_kernel.restype = ctypes.c_int
        L.ssd_chunk_scan_kernel.argtypes = [shp, i32, i32, ctypes.POINTER(i32)]
        L.ssd_bwd_mamba2_workspace_bytes.restype = ctypes.c_int
        L.ssd_bwd_mamba2_workspace_bytes.argtypes = [shp, i32, i32, ctypes.POINTER(sz)]
        L.ssd_bwd_mamba2.restype = ctypes.c_int
        L.ssd_bwd_mamba2.argtypes = [vp] * 12 + [i32, i32] + [vp] * 9 + [shp, vp, sz, vp]
        f32, lin, norm, pages = ctypes.c_float, ctypes.POINTER(LinShape), ctypes.POINTER(NormShape), ctypes.POINTER(PagesShape)
        delta = ctypes.POINTER(DeltaShape)
        for name, args in (("ssd_lin_attn_workspace_bytes", [lin, ctypes.POINTER(sz)]),
                           ("ssd_lin_attn_bwd_workspace_bytes", [lin, ctypes.POINTER(sz)]),
                           ("ssd_lin_attn_fwd", [vp] * 5 + [f32] + [vp] * 3 + [lin, vp, sz, vp]),
                           ("ssd_lin_attn_bwd", [vp] * 5 + [f32] + [vp] * 7 + [lin, vp, sz, vp]),
                           ("ssd_lin_attn_step", [vp] * 6 + [i32, f32, vp, lin, vp]),
                           ("ssd_group_norm_workspace_bytes", [norm, i32, ctypes.POINTER(sz)]),
                           ("ssd_group_norm", [vp] * 4 + [f32] + [vp] * 2 + [norm, vp, sz, vp]),
                           ("ssd_group_norm_bwd", [vp] * 10 + [norm, vp, sz, vp]),
                           ("ssd_pages_copy", [vp, vp, vp, i32, pages, vp]),
                           ("ssd_pages_clear", [vp, vp, i32, pages, vp]),
                           ("ssd_pages_compact_workspace_bytes", [pages, ctypes.POINTER(sz)]),
                           ("ssd_pages_compact", [vp] * 4 + [pages, vp, sz, vp]),
                           ("ssd_gated_delta_workspace_bytes", [delta, ctypes.POINTER(sz)]),
                           ("ssd_gated_delta_bwd_workspace_bytes", [delta, ctypes.POINTER(sz)]),
                           ("ssd_gated_delta_fwd", [vp] * 6 + [f32] + [vp] * 3 + [delta, vp, sz, vp]),
                           ("ssd_gated_delta_bwd", [vp] * 6 + [f32] + [vp] * 9 + [delta, vp, sz, vp]),
                           ("ssd_gated_delta_step", [vp] * 7 + [i32, f32, vp, delta, vp]),
                           ("ssd_rotary", [vp] * 6 + [f32] + [vp] * 2 + [ctypes.POINTER(RotaryShape), vp])):
            getattr(L, name).restype = ctypes.c_int
            getattr(L, name).argtypes = args
        _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return DTYPE_BF16
    if dt == torch.float32:
        return DTYPE_F32
    raise TypeError(f"unsupported dtype {dt}")


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _call(fn: str, *args):
    st = getattr(lib(), fn)(*args)
    if st != SSD_OK:
        raise SSDError(fn, st)


def make_shape(X: torch.Tensor, B: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None) -> Shape:
    b, T, H, P = X.shape
    G, N = B.shape[2], B.shape[3]
    S = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    return Shape(b, T, H, G, P, N, S, _dtype_code(X.dtype))


def default_state_block(shape: Shape, chunk: int) -> int:
    return int(lib().ssd_default_state_block(ctypes.byref(shape), int(chunk)))


def layout(shape: Shape, chunk: int, state_block: int = 0) -> Layout:
    L = Layout()
    _call("ssd_fwd_layout", ctypes.byref(shape), int(chunk), int(state_block), ctypes.byref(L))
    return L


def workspace_bytes(shape: Shape, chunk: int, state_block: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _call("ssd_fwd_workspace_bytes", ctypes.byref(shape), int(chunk), int(state_block), ctypes.byref(n))
    return int(n.value)


class Workspace:
    """A caller-owned workspace for one shape, chunk length and state block, with
    typed views of the stages' intermediate results (for inspection and tests)."""

    def __init__(self, shape: Shape, chunk: int, device, state_block: int = 0):
        self.shape = shape
        self.chunk = int(chunk)
        self.state_block = int(state_block) if state_block > 0 else default_state_block(shape, chunk)
        self.layout = layout(shape, chunk, self.state_block)
        self.buffer = torch.empty(self.layout.total_bytes, dtype=torch.uint8, device=device)

    @property
    def nbytes(self) -> int:
        return self.buffer.numel()

    def _view(self, off: int, count: int, dtype: torch.dtype, shape):
        esz = torch.empty((), dtype=dtype).element_size()
        return self.buffer[off:off + count * esz].view(dtype).view(*shape)

    def table(self) -> torch.Tensor:
        n = self.layout.nslots
        return self._view(self.layout.table_offset, n * 4, torch.int32, (n, 4))

    def block_table(self) -> torch.Tensor:
        n = self.layout.nblocks
        return self._view(self.layout.block_table_offset, n * 4, torch.int32, (n, 4))

    def cumsum(self) -> torch.Tensor:
        s, n = self.shape, self.layout.nslots
        return self._view(self.layout.cumsum_offset, n * s.nheads * self.chunk, torch.float32,
                          (n, s.nheads, self.chunk))

    def key_cumsum(self) -> torch.Tensor:
        s, n = self.shape, self.layout.nslots
        return self._view(self.layout.key_cumsum_offset, n * s.nheads * self.chunk, torch.float32,
                          (n, s.nheads, self.chunk))

    def block_decay(self) -> torch.Tensor:
        s, n = self.shape, self.layout.nblocks
        return self._view(self.layout.block_decay_offset, n * s.nheads, torch.float32, (n, s.nheads))

    def block_states(self) -> torch.Tensor:
        s, n = self.shape, self.layout.nblocks
        return self._view(self.layout.block_states_offset, n * s.nheads * s.headdim * s.dstate, torch.float32,
                          (n, s.nheads, s.headdim, s.dstate))

    def start_states(self) -> torch.Tensor:
        s, n = self.shape, self.layout.nblocks
        dt = torch.bfloat16 if s.dtype == DTYPE_BF16 else torch.float32
        return self._view(self.layout.start_states_offset, n * s.nheads * s.headdim * s.dstate, dt,
                          (n, s.nheads, s.headdim, s.dstate))


def _expect(t: Optional[torch.Tensor], name: str, shape=None, dtype=None, device=None, align: int = 0):
    """Raise ValueError unless `t` (None passes) has the given shape, dtype,
    contiguity and device."""
    _expect_all([(t, name, shape, dtype, align)], device)


def _expect_all(specs, device=None):
    """Check every (tensor, name, shape, dtype, align) in `specs`: first the
    structure of all of them (shape, dtype, contiguity), then their device and
    alignment, so a mismatched tensor is reported as such wherever it lives."""
    specs = [sp for sp in specs if sp[0] is not None]
    for t, name, shape, dtype, _ in specs:
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a torch tensor")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    for t, name, _, _, align in specs:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        if device is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
        if align and t.data_ptr() % align:
            raise ValueError(f"{name} must be {align}-byte aligned")


def _check_inputs(X, log_a, B, C, cu_seqlens):
    """The forward inputs against one another: X [b, T, H, P], log_a [b, T, H]
    fp32, B and C [b, T, G, N] of X's dtype with H % G == 0, cu_seqlens int32
    [S + 1] with b == 1. Returns their specs for _expect_all."""
    if not isinstance(X, torch.Tensor) or X.dim() != 4:
        raise ValueError("X must be a 4-d tensor [batch, seqlen, nheads, headdim]")
    if X.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"X has dtype {X.dtype}; bfloat16 and float32 are supported")
    b, T, H, P = X.shape
    if not isinstance(B, torch.Tensor) or B.dim() != 4 or tuple(B.shape[:2]) != (b, T):
        raise ValueError(f"B must be a 4-d tensor [{b}, {T}, ngroups, dstate]")
    G, N = B.shape[2], B.shape[3]
    if G < 1 or H % G:
        raise ValueError(f"nheads {H} must be a multiple of ngroups {G}")
    if cu_seqlens is not None:
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be a 1-d tensor of num_seqs + 1 >= 2 entries")
        if b != 1:
            raise ValueError("packed sequences (cu_seqlens) need batch 1")
    return [(X, "X", None, None, 0), (B, "B", (b, T, G, N), X.dtype, 0), (C, "C", (b, T, G, N), X.dtype, 0),
            (log_a, "log_a", (b, T, H), torch.float32, 0), (cu_seqlens, "cu_seqlens", None, torch.int32, 0)]


def _nseq(shape: Shape) -> int:
    return shape.num_seqs if shape.num_seqs > 0 else shape.batch


def _state_spec(t: Optional[torch.Tensor], shape: Shape, name: str):
    """A state tensor: fp32 [rows or sequences, H, P, N], 16-byte aligned."""
    return (t, name, (_nseq(shape), shape.nheads, shape.headdim, shape.dstate), torch.float32, 16)


def _check_state(t: Optional[torch.Tensor], shape: Shape, name: str, device=None):
    _expect_all([_state_spec(t, shape, name)], device)


def _check_workspace(ws: "Workspace", shape: Shape, chunk: int):
    if not isinstance(ws, Workspace):
        raise ValueError("workspace must be a Workspace")
    mine = tuple(getattr(ws.shape, f) for f, _ in Shape._fields_)
    theirs = tuple(getattr(shape, f) for f, _ in Shape._fields_)
    if mine != theirs or ws.chunk != int(chunk):
        raise ValueError("the workspace was made for another shape or chunk length")


def fwd(X: torch.Tensor, log_a: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
        cu_seqlens: Optional[torch.Tensor] = None, chunk: int = 128, state_block: int = 0,
        Y: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None, want_final: bool = True,
        workspace: Optional[Workspace] = None,
        initial_state: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunked SSD forward pass (ssd_fwd_ex). Returns (Y, final_state or None).

    state_block <= 0 uses the library's default (the workspace's, when one is given).
    initial_state: fp32 [rows or sequences, H, P, N] the state each row (each
    packed sequence) starts from; None for zero states.
    """
    specs = _check_inputs(X, log_a, B, C, cu_seqlens)
    shape = make_shape(X, B, cu_seqlens)
    if workspace is not None:
        _check_workspace(workspace, shape, chunk)
        if state_block > 0 and state_block != workspace.state_block:
            raise ValueError("state_block differs from the workspace's")
    _expect_all(specs + [_state_spec(initial_state, shape, "initial_state"), (Y, "Y", tuple(X.shape), X.dtype, 0),
                         _state_spec(final_state, shape, "final_state")], X.device)
    if Y is None:
        Y = torch.empty_like(X)
    if final_state is None and want_final:
        final_state = torch.empty(_nseq(shape), X.shape[2], X.shape[3], B.shape[3], dtype=torch.float32,
                                  device=X.device)
    if workspace is None:
        workspace = Workspace(shape, chunk, X.device, state_block)
    _call("ssd_fwd_ex", _ptr(X), _ptr(log_a), _ptr(B), _ptr(C), _ptr(cu_seqlens), _ptr(initial_state), int(chunk),
          workspace.state_block,
          _ptr(Y), _ptr(final_state), ctypes.byref(shape), _ptr(workspace.buffer), workspace.nbytes,
          _stream(X.device))
    return Y, final_state


def _stage_check(shape: Shape, ws: Workspace, X=None, log_a=None, B=None, C=None, Y=None, cu_seqlens=None):
    """Tensors handed to a single stage against the shape its workspace was made for."""
    _check_workspace(ws, shape, ws.chunk)
    dt = torch.bfloat16 if shape.dtype == DTYPE_BF16 else torch.float32
    b, T, H, G, P, N = shape.batch, shape.seqlen, shape.nheads, shape.ngroups, shape.headdim, shape.dstate
    want_cu = shape.num_seqs + 1 if shape.num_seqs > 0 else None
    if (cu_seqlens is None) != (want_cu is None):
        raise ValueError("cu_seqlens must be given exactly when the shape is packed (num_seqs > 0)")
    _expect_all([(X, "X", (b, T, H, P), dt, 0), (Y, "Y", (b, T, H, P), dt, 0), (B, "B", (b, T, G, N), dt, 0),
                 (C, "C", (b, T, G, N), dt, 0), (log_a, "log_a", (b, T, H), torch.float32, 0),
                 (cu_seqlens, "cu_seqlens", (want_cu,) if want_cu else None, torch.int32, 0)], ws.buffer.device)


NOALLOC_SCRATCH_BYTES = 64 << 20   # SSD_NOALLOC_SCRATCH_BYTES


def fwd_noalloc(X: torch.Tensor, log_a: torch.Tensor, B: torch.Tensor, C: torch.Tensor, Y: torch.Tensor,
                final_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                chunk: int = 128) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """ssd_fwd_noalloc: the forward pass in the library's static per-GPU scratch (no
    workspace; nothing allocated here either, so Y, and final_state when wanted,
    are the caller's). Calls that overlap on one GPU race on that scratch."""
    specs = _check_inputs(X, log_a, B, C, cu_seqlens)
    shape = make_shape(X, B, cu_seqlens)
    if Y is None:
        raise ValueError("Y is required")
    _expect_all(specs + [(Y, "Y", tuple(X.shape), X.dtype, 0), _state_spec(final_state, shape, "final_state")],
                X.device)
    _call("ssd_fwd_noalloc", _ptr(X), _ptr(log_a), _ptr(B), _ptr(C), _ptr(cu_seqlens), int(chunk), _ptr(Y),
          _ptr(final_state), ctypes.byref(shape), _stream(X.device))
    return Y, final_state


def chunk_cumsum(log_a, cu_seqlens, shape: Shape, ws: Workspace):
    _stage_check(shape, ws, log_a=log_a, cu_seqlens=cu_seqlens)
    _call("ssd_chunk_cumsum", _ptr(log_a), _ptr(cu_seqlens), ws.chunk, ws.state_block, ctypes.byref(shape),
          _ptr(ws.buffer), ws.nbytes, _stream(ws.buffer.device))


def chunk_state(X, B, cu_seqlens, shape: Shape, ws: Workspace):
    _stage_check(shape, ws, X=X, B=B, cu_seqlens=cu_seqlens)
    _call("ssd_chunk_state", _ptr(X), _ptr(B), _ptr(cu_seqlens), ws.chunk, ws.state_block, ctypes.byref(shape),
          _ptr(ws.buffer), ws.nbytes, _stream(ws.buffer.device))


def state_passing(cu_seqlens, final_state, shape: Shape, ws: Workspace, initial_state=None):
    _stage_check(shape, ws, cu_seqlens=cu_seqlens)
    _expect_all([_state_spec(initial_state, shape, "initial_state"), _state_spec(final_state, shape, "final_state")],
                ws.buffer.device)
    _call("ssd_state_passing", _ptr(cu_seqlens), _ptr(initial_state), ws.chunk, ws.state_block, _ptr(final_state),
          ctypes.byref(shape), _ptr(ws.buffer), ws.nbytes, _stream(ws.buffer.device))


def chunk_scan(X, B, C, cu_seqlens, Y, shape: Shape, ws: Workspace):
    _stage_check(shape, ws, X=X, B=B, C=C, Y=Y, cu_seqlens=cu_seqlens)
    _call("ssd_chunk_scan", _ptr(X), _ptr(B), _ptr(C), _ptr(cu_seqlens), ws.chunk, ws.state_block, _ptr(Y),
          ctypes.byref(shape), _ptr(ws.buffer), ws.nbytes, _stream(ws.buffer.device))


def _check_step(state, x, B, C, y, log_a=None):
    """Decode-step tensors: x [b, H, P], state fp32 [b, H, P, N] (16-byte aligned),
    B and C [b, G, N] of x's dtype, log_a fp32 [b, H], y like x."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a 3-d tensor [batch, nheads, headdim]")
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"x has dtype {x.dtype}; bfloat16 and float32 are supported")
    b, H, P = x.shape
    if not isinstance(B, torch.Tensor) or B.dim() != 3 or B.shape[0] != b:
        raise ValueError(f"B must be a 3-d tensor [{b}, ngroups, dstate]")
    G, N = B.shape[1], B.shape[2]
    if G < 1 or H % G:
        raise ValueError(f"nheads {H} must be a multiple of ngroups {G}")
    if state is None:
        raise ValueError("state is required")
    specs = [(x, "x", None, None, 0), (B, "B", (b, G, N), x.dtype, 0), (C, "C", (b, G, N), x.dtype, 0),
             (state, "state", (b, H, P, N), torch.float32, 16), (log_a, "log_a", (b, H), torch.float32, 0),
             (y, "y", (b, H, P), x.dtype, 0)]
    return Shape(b, 1, H, G, P, N, 0, _dtype_code(x.dtype)), specs


def step(state: torch.Tensor, x: torch.Tensor, log_a: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
         y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One decode step (ssd_step): updates `state` in place and returns y."""
    if log_a is None:
        raise ValueError("log_a is required")
    shape, specs = _check_step(state, x, B, C, y, log_a)
    _expect_all(specs, x.device)
    if y is None:
        y = torch.empty_like(x)
    _call("ssd_step", _ptr(state), _ptr(x), _ptr(log_a), _ptr(B), _ptr(C), _ptr(y), ctypes.byref(shape),
          _stream(x.device))
    return y


def _check_mamba2(X, dt, dt_bias, A_log, D, z, H: int):
    """Specs of the Mamba-2 call's extra tensors: dt [*X.shape[:-1]] fp32, dt_bias,
    A_log, D [H] fp32, z like X."""
    if dt is None or A_log is None:
        raise ValueError("dt and A_log are required")
    return [(dt, "dt", tuple(X.shape[:-1]), torch.float32, 0), (dt_bias, "dt_bias", (H,), torch.float32, 0),
            (A_log, "A_log", (H,), torch.float32, 0), (D, "D", (H,), torch.float32, 0),
            (z, "z", tuple(X.shape), X.dtype, 0)]


def fwd_mamba2(X: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
               dt_bias: Optional[torch.Tensor] = None, D: Optional[torch.Tensor] = None,
               z: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, chunk: int = 128,
               state_block: int = 0, Y: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
               want_final: bool = True, workspace: Optional[Workspace] = None,
               initial_state: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The Mamba-2 block's SSD call (ssd_fwd_mamba2). Returns (Y, final_state or None).

    X is the block's x (unscaled), dt the raw step sizes [b, T, H] fp32; dt_bias,
    A_log and D are fp32 [H]; z (the gate) has X's shape and dtype. The other
    arguments are those of fwd().
    """
    specs = _check_inputs(X, None, B, C, cu_seqlens) + _check_mamba2(X, dt, dt_bias, A_log, D, z, X.shape[2])
    shape = make_shape(X, B, cu_seqlens)
    if workspace is not None:
        _check_workspace(workspace, shape, chunk)
        if state_block > 0 and state_block != workspace.state_block:
            raise ValueError("state_block differs from the workspace's")
    _expect_all(specs + [_state_spec(initial_state, shape, "initial_state"), (Y, "Y", tuple(X.shape), X.dtype, 0),
                         _state_spec(final_state, shape, "final_state")], X.device)
    if Y is None:
        Y = torch.empty_like(X)
    if final_state is None and want_final:
        final_state = torch.empty(_nseq(shape), X.shape[2], X.shape[3], B.shape[3], dtype=torch.float32,
                                  device=X.device)
    if workspace is None:
        workspace = Workspace(shape, chunk, X.device, state_block)
    _call("ssd_fwd_mamba2", _ptr(X), _ptr(dt), _ptr(dt_bias), _ptr(A_log), _ptr(D), _ptr(z), _ptr(B), _ptr(C),
          _ptr(cu_seqlens), _ptr(initial_state), int(chunk), workspace.state_block, _ptr(Y), _ptr(final_state),
          ctypes.byref(shape), _ptr(workspace.buffer), workspace.nbytes, _stream(X.device))
    return Y, final_state


def step_mamba2(state: torch.Tensor, x: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor,
                C: torch.Tensor, dt_bias: Optional[torch.Tensor] = None, D: Optional[torch.Tensor] = None,
                z: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One Mamba-2 decode step (ssd_step_mamba2): updates `state` in place and returns y."""
    shape, specs = _check_step(state, x, B, C, y)
    _expect_all(specs + _check_mamba2(x, dt, dt_bias, A_log, D, z, x.shape[1]), x.device)
    if y is None:
        y = torch.empty_like(x)
    _call("ssd_step_mamba2", _ptr(state), _ptr(x), _ptr(dt), _ptr(dt_bias), _ptr(A_log), _ptr(D), _ptr(z),
          _ptr(B), _ptr(C), _ptr(y), ctypes.byref(shape), _stream(x.device))
    return y


def set_state_chain(mode: int) -> int:
    """ssd_set_state_chain: 1 runs the state chain as one cooperative launch when
    it fits, 0 (the default) always as two launches. Returns the previous mode."""
    return int(lib().ssd_set_state_chain(int(mode)))


def state_chain_cooperative(shape: Shape, chunk: int, state_block: int = 0) -> bool:
    """ssd_state_chain_cooperative: whether mode 1 runs this shape's state chain as
    the cooperative launch on the current device (uncaptured stream)."""
    r = ctypes.c_int32(0)
    _call("ssd_state_chain_cooperative", ctypes.byref(shape), int(chunk), int(state_block), ctypes.byref(r))
    return bool(r.value)


SCAN_KERNELS = ("f32", "single", "pair", "half_pair", "half_pair_wide")


def chunk_scan_kernel(shape: Shape, chunk: int, state_block: int = 0) -> str:
    """ssd_chunk_scan_kernel: the chunk_scan kernel a forward call with this shape
    runs: "f32", "single" (one head per workgroup), "pair" (two heads, whole
    chunks, one workgroup per CU), "half_pair" (two heads, chunks in halves of
    64 tokens, two workgroups per CU) or "half_pair_wide" (the same walk at
    dstate 256, one workgroup per CU)."""
    r = ctypes.c_int32(-1)
    _call("ssd_chunk_scan_kernel", ctypes.byref(shape), int(chunk), int(state_block), ctypes.byref(r))
    return SCAN_KERNELS[r.value]


def bwd_workspace_bytes(shape: Shape, chunk: int, state_block: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _call("ssd_bwd_workspace_bytes", ctypes.byref(shape), int(chunk), int(state_block), ctypes.byref(n))
    return int(n.value)


def bwd(X: torch.Tensor, log_a: torch.Tensor, B: torch.Tensor, C: torch.Tensor, dY: torch.Tensor,
        cu_seqlens: Optional[torch.Tensor] = None, chunk: int = 128, state_block: int = 0,
        initial_state: Optional[torch.Tensor] = None, dfinal_state: Optional[torch.Tensor] = None,
        want_dinit: bool = False, workspace: Optional[torch.Tensor] = None):
    """Backward pass (ssd_bwd): gradients of <dY, Y> + <dfinal_state, final_state>
    for the forward pass with these inputs. Returns dict(dX, dlog_a, dB, dC, dinit or None)."""
    specs = _check_inputs(X, log_a, B, C, cu_seqlens)
    if dY is None:
        raise ValueError("dY is required")
    shape = make_shape(X, B, cu_seqlens)
    _expect_all(specs + [(dY, "dY", tuple(X.shape), X.dtype, 0), _state_spec(initial_state, shape, "initial_state"),
                         _state_spec(dfinal_state, shape, "dfinal_state")], X.device)
    nbytes = bwd_workspace_bytes(shape, chunk, state_block)
    _expect(workspace, "workspace", dtype=torch.uint8, device=X.device, align=256)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=X.device)
    dX = torch.empty_like(X)
    dla = torch.empty_like(log_a)
    dB = torch.empty_like(B)
    dC = torch.empty_like(C)
    dinit = None
    if want_dinit:
        nseq = X.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
        dinit = torch.empty(nseq, X.shape[2], X.shape[3], B.shape[3], dtype=torch.float32, device=X.device)
    _call("ssd_bwd", _ptr(X), _ptr(log_a), _ptr(B), _ptr(C), _ptr(cu_seqlens), _ptr(initial_state), _ptr(dY),
          _ptr(dfinal_state), int(chunk), int(state_block), _ptr(dX), _ptr(dla), _ptr(dB), _ptr(dC), _ptr(dinit),
          ctypes.byref(shape), _ptr(workspace), workspace.numel(), _stream(X.device))
    return dict(dX=dX, dlog_a=dla, dB=dB, dC=dC, dinit=dinit)


def bwd_mamba2_workspace_bytes(shape: Shape, chunk: int, state_block: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _call("ssd_bwd_mamba2_workspace_bytes", ctypes.byref(shape), int(chunk), int(state_block), ctypes.byref(n))
    return int(n.value)


def bwd_mamba2(X: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
               dY: torch.Tensor, dt_bias: Optional[torch.Tensor] = None, D: Optional[torch.Tensor] = None,
               z: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, chunk: int = 128,
               state_block: int = 0, initial_state: Optional[torch.Tensor] = None,
               dfinal_state: Optional[torch.Tensor] = None, want_dinit: bool = False,
               workspace: Optional[torch.Tensor] = None):
    """Backward pass of the Mamba-2 call (ssd_bwd_mamba2). Returns dict(dX, ddt, ddt_bias,
    dA_log, dD or None, dz or None, dB, dC, dinit or None)."""
    specs = _check_inputs(X, None, B, C, cu_seqlens) + _check_mamba2(X, dt, dt_bias, A_log, D, z, X.shape[2])
    if dY is None:
        raise ValueError("dY is required")
    shape = make_shape(X, B, cu_seqlens)
    _expect_all(specs + [(dY, "dY", tuple(X.shape), X.dtype, 0), _state_spec(initial_state, shape, "initial_state"),
                         _state_spec(dfinal_state, shape, "dfinal_state")], X.device)
    nbytes = bwd_mamba2_workspace_bytes(shape, chunk, state_block)
    _expect(workspace, "workspace", dtype=torch.uint8, device=X.device, align=256)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=X.device)
    H = X.shape[2]
    out = dict(dX=torch.empty_like(X), ddt=torch.empty_like(dt),
               ddt_bias=torch.empty(H, dtype=torch.float32, device=X.device),
               dA_log=torch.empty(H, dtype=torch.float32, device=X.device),
               dD=None if D is None else torch.empty(H, dtype=torch.float32, device=X.device),
               dz=None if z is None else torch.empty_like(z), dB=torch.empty_like(B), dC=torch.empty_like(C),
               dinit=None)
    if want_dinit:
        nseq = X.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
        out["dinit"] = torch.empty(nseq, H, X.shape[3], B.shape[3], dtype=torch.float32, device=X.device)
    _call("ssd_bwd_mamba2", _ptr(X), _ptr(dt), _ptr(dt_bias), _ptr(A_log), _ptr(D), _ptr(z), _ptr(B), _ptr(C),
          _ptr(cu_seqlens), _ptr(initial_state), _ptr(dY), _ptr(dfinal_state), int(chunk), int(state_block),
          _ptr(out["dX"]), _ptr(out["ddt"]), _ptr(out["ddt_bias"]), _ptr(out["dA_log"]), _ptr(out["dD"]),
          _ptr(out["dz"]), _ptr(out["dB"]), _ptr(out["dC"]), _ptr(out["dinit"]), ctypes.byref(shape),
          _ptr(workspace), workspace.numel(), _stream(X.device))
    return out


# ---------------------------------------------------------------------------
# Linear attention with one decay a head
# ---------------------------------------------------------------------------

def _call_on(device: torch.device, fn: str, *args):
    """_call on the device's current stream, with `device` current, whichever device the caller's is."""
    stream = torch._C._cuda_getCurrentRawStream(device.index)   # what current_stream(device) wraps, at a tenth of its time
    if device.index == torch._C._cuda_getDevice():
        _call(fn, *args, stream)
    else:
        with torch.cuda.device(device):
            _call(fn, *args, stream)


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check_dtype(t, name: str, dim: str, dims: int):
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError(f"{name} must be a {dims}-d tensor {dim}")
    if t.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{name} has dtype {t.dtype}; bfloat16 and float32 are supported")


def _int32(sizes: dict):
    """The sizes that the C ABI takes in 32 bits (ctypes would cut them off)."""
    for name, n in sizes.items():
        if n > 0x7FFFFFFF:
            raise ValueError(f"{name} {n} does not fit 32 bits")


def _token_row(t: torch.Tensor, name: str) -> int:
    """Elements from token to token of [batch, seqlen, heads, d]: heads and their
    elements lie together, tokens at one distance, rows of the batch follow on."""
    b, T, H, D = t.shape
    st = t.stride()
    if (D > 1 and st[3] != 1) or (H > 1 and st[2] != D):
        raise ValueError(f"{name} must have its heads contiguous (strides {st})")
    if t.numel() == 0:
        return H * D
    row = st[1] if T > 1 else (st[0] if b > 1 else H * D)
    if row < H * D or (b > 1 and st[0] != T * row):
        raise ValueError(f"{name} must have its tokens at one distance (strides {st})")
    return row


def _expect_device(specs, device, align: int = 16):
    """Device and alignment of every given (tensor, name)."""
    index = device.index if device.type == "cuda" else -1
    for t, name in specs:
        if t is None:
            continue
        at = t.get_device()
        if at < 0:
            raise ValueError(f"{name} must be a device tensor")
        if at != index:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
        if t.data_ptr() % align:
            raise ValueError(f"{name} must be {align}-byte aligned")


def _lin_shape(q, k, v, cu_seqlens):
    """The shape of a call over prompts, its tensors checked against one another
    (their devices and alignment come after, with the outputs')."""
    _check_dtype(q, "q", "[batch, seqlen, nheads, dk]", 4)
    b, T, H, Dk = q.shape
    if not isinstance(k, torch.Tensor) or k.dim() != 4 or k.shape[0] != b or k.shape[1] != T or k.shape[3] != Dk:
        raise ValueError(f"k must be a 4-d tensor [{b}, {T}, nkv_heads, {Dk}]")
    Hk = k.shape[2]
    if Hk < 1 or H % Hk:
        raise ValueError(f"nheads {H} must be a multiple of nkv_heads {Hk}")
    if not isinstance(v, torch.Tensor) or v.dim() != 4 or tuple(v.shape[:3]) != (b, T, Hk):
        raise ValueError(f"v must be a 4-d tensor [{b}, {T}, {Hk}, dv]")
    for t, name in ((k, "k"), (v, "v")):
        if t.dtype != q.dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {q.dtype}")
    S = 0
    if cu_seqlens is not None:
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be a 1-d tensor of num_seqs + 1 >= 2 entries")
        if b != 1:
            raise ValueError("packed sequences (cu_seqlens) need batch 1")
        S = cu_seqlens.numel() - 1
    _int32(dict(batch=b, seqlen=T, nheads=H, dk=Dk, dv=v.shape[3], num_seqs=S))
    # A batch without tokens runs nothing: its heads and sizes are checked as those of one token.
    return _lin_struct(max(b, 1), max(T, 1), H, Hk, Dk, v.shape[3], S, _dtype_code(q.dtype), _token_row(q, "q"), _token_row(k, "k"),
                       _token_row(v, "v"))


def _structure(specs):
    """Shape, dtype and contiguity of every given (tensor, name, shape, dtype)."""
    for t, name, shape, dtype in specs:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a torch tensor")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.dtype != dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _check(device, specs):
    """Structure, device and alignment of every given (tensor, name, shape, dtype, align);
    dtype None: its structure was checked before. One pass while all is well, as a
    small call's time is its host's; what is wrong is then found in order."""
    index = device.index if device.type == "cuda" else -1
    if index >= 0:
        for t, name, shape, dtype, align in specs:
            if t is not None and not (
                    (dtype is None or (isinstance(t, torch.Tensor) and t.dtype == dtype and
                                       (shape is None or t.shape == shape) and t.is_contiguous()))
                    and t.get_device() == index and t.data_ptr() % align == 0):
                break
        else:
            return
    _structure([(t, name, shape, dtype) for t, name, shape, dtype, _ in specs if dtype is not None])
    for t, name, _, _, align in specs:
        _expect_device([(t, name)], device, align)


@functools.lru_cache(maxsize=256)
def _lin_struct(*values) -> LinShape:
    """The C shape of these sizes (the library only reads it)."""
    return LinShape(*values)


@functools.lru_cache(maxsize=256)
def _size_of(fn: str, struct, values, *more) -> int:
    """A workspace size query: a function of the sizes alone, asked once for each."""
    n = ctypes.c_size_t(0)
    _call(fn, ctypes.byref(struct(*values)), *more, ctypes.byref(n))
    return int(n.value)


def _room(size: int, workspace, device):
    """The workspace of a call and its size: the caller's where it is large enough."""
    if workspace is not None and workspace.numel() >= size:
        return workspace, workspace.numel()
    return (torch.empty(size, dtype=torch.uint8, device=device) if size else None), size


def _share(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two contiguous tensors share memory."""
    return (a.data_ptr() < b.data_ptr() + b.numel() * b.element_size() and
            b.data_ptr() < a.data_ptr() + a.numel() * a.element_size())


def _check_scale(scale: float):
    """As the C ABI does, to which a batch without tokens does not get."""
    if not 2.0 ** -126 <= abs(scale) < 2.0 ** 128:
        raise ValueError(f"scale {scale} must be a normal fp32 number, not 0")


def _state_of_no_tokens(state: Optional[torch.Tensor], out: Optional[torch.Tensor], want: bool, shape, device):
    """What a batch without tokens makes of a state: the state itself, or zeros."""
    if out is None and want:
        out = torch.empty(shape, dtype=torch.float32, device=device)
    if out is not None:
        out.copy_(state) if state is not None else out.zero_()
    return out


def _lin_values(shape: LinShape):
    return (shape.batch, shape.seqlen, shape.nheads, shape.nkv_heads, shape.dk, shape.dv, shape.num_seqs, shape.dtype,
            shape.q_row, shape.k_row, shape.v_row)


def _lin_workspace(fn: str, shape: LinShape, workspace, device):
    return _room(_size_of(fn, LinShape, _lin_values(shape)), workspace, device)


def lin_attn_shape(q, k, v, cu_seqlens=None) -> LinShape:
    """The shape of a call with these tensors (for lin_attn_workspace_bytes)."""
    return LinShape(*_lin_values(_lin_shape(q, k, v, cu_seqlens)))   # the caller's own


def lin_attn_workspace_bytes(shape: LinShape) -> int:
    n = ctypes.c_size_t(0)
    _call("ssd_lin_attn_workspace_bytes", ctypes.byref(shape), ctypes.byref(n))
    return int(n.value)


def lin_attn_bwd_workspace_bytes(shape: LinShape) -> int:
    n = ctypes.c_size_t(0)
    _call("ssd_lin_attn_bwd_workspace_bytes", ctypes.byref(shape), ctypes.byref(n))
    return int(n.value)


def lin_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                 cu_seqlens: Optional[torch.Tensor] = None, scale: float = 1.0,
                 initial_state: Optional[torch.Tensor] = None, o: Optional[torch.Tensor] = None,
                 final_state: Optional[torch.Tensor] = None, want_final: bool = True,
                 workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Linear attention with one decay a head over prompts (ssd_lin_attn_fwd). Returns (o, final_state or None).

    q [b, T, H, dk], k [b, T, Hk, dk], v [b, T, Hk, dv] (bf16 or fp32; tokens may lie
    in wider rows, as slices of one projection do), log_decay [H] fp32 <= 0, states
    fp32 [rows or sequences, H, dv, dk]. cu_seqlens may hold empty sequences, and a
    batch no rows or tokens at all (its final states are the initial ones); rows
    of o that belong to no sequence are left as they were (undefined in an o made here).
    """
    shape = _lin_shape(q, k, v, cu_seqlens)
    b, T, H, Dk = q.shape
    Dv, nseq = v.shape[3], shape.num_seqs or b
    if log_decay is None:
        raise ValueError("log_decay is required")
    st = (nseq, H, Dv, Dk)
    _check(q.device, ((q, "q", None, None, 16), (k, "k", None, None, 16), (v, "v", None, None, 16),
                      (initial_state, "initial_state", st, torch.float32, 16), (o, "o", (b, T, H, Dv), q.dtype, 16),
                      (final_state, "final_state", st, torch.float32, 16),
                      (log_decay, "log_decay", (H,), torch.float32, 4), (cu_seqlens, "cu_seqlens", None, torch.int32, 4),
                      (workspace, "workspace", None, torch.uint8, 256)))
    if final_state is not None and initial_state is not None and _share(final_state, initial_state):
        raise ValueError("final_state must not overlap initial_state: blocks of a prompt read the one while others write the other")
    workspace, have = _lin_workspace("ssd_lin_attn_workspace_bytes", shape, workspace, q.device)
    if o is None:
        o = torch.empty(b, T, H, Dv, dtype=q.dtype, device=q.device)
    if b * T == 0:
        _check_scale(scale)
        return o, _state_of_no_tokens(initial_state, final_state, want_final, st, q.device)
    if final_state is None and want_final:
        final_state = torch.empty(st, dtype=torch.float32, device=q.device)
    _call_on(q.device, "ssd_lin_attn_fwd", _addr(q), _addr(k), _addr(v), _addr(log_decay), _addr(cu_seqlens), float(scale),
             _addr(initial_state), _addr(o), _addr(final_state), ctypes.byref(shape), _addr(workspace), have)
    return o, final_state


def lin_attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, do: torch.Tensor,
                 cu_seqlens: Optional[torch.Tensor] = None, scale: float = 1.0,
                 initial_state: Optional[torch.Tensor] = None, dfinal_state: Optional[torch.Tensor] = None,
                 want_dinit: bool = False, workspace: Optional[torch.Tensor] = None):
    """Gradients of <do, o> + <dfinal_state, final_state> of lin_attn_fwd with these
    inputs (ssd_lin_attn_bwd). Returns dict(dq, dk, dv, dinit or None); log_decay is
    a constant of the layer. Rows that belong to no sequence are undefined."""
    shape = _lin_shape(q, k, v, cu_seqlens)
    b, T, H, Dk = q.shape
    Dv, nseq = v.shape[3], shape.num_seqs or b
    if log_decay is None or do is None:
        raise ValueError("log_decay and do are required")
    st = (nseq, H, Dv, Dk)
    _check(q.device, ((q, "q", None, None, 16), (k, "k", None, None, 16), (v, "v", None, None, 16),
                      (do, "do", (b, T, H, Dv), q.dtype, 16), (initial_state, "initial_state", st, torch.float32, 16),
                      (dfinal_state, "dfinal_state", st, torch.float32, 16),
                      (log_decay, "log_decay", (H,), torch.float32, 4), (cu_seqlens, "cu_seqlens", None, torch.int32, 4),
                      (workspace, "workspace", None, torch.uint8, 256)))
    workspace, have = _lin_workspace("ssd_lin_attn_bwd_workspace_bytes", shape, workspace, q.device)
    out = dict(dq=torch.empty(q.shape, dtype=q.dtype, device=q.device), dk=torch.empty(k.shape, dtype=q.dtype, device=q.device),
               dv=torch.empty(v.shape, dtype=q.dtype, device=q.device),
               dinit=torch.empty(st, dtype=torch.float32, device=q.device) if want_dinit else None)
    if b * T == 0:
        _check_scale(scale)
        _state_of_no_tokens(dfinal_state, out["dinit"], want_dinit, st, q.device)
        return out
    _call_on(q.device, "ssd_lin_attn_bwd", _addr(q), _addr(k), _addr(v), _addr(log_decay), _addr(cu_seqlens), float(scale),
             _addr(initial_state), _addr(do), _addr(dfinal_state), _addr(out["dq"]), _addr(out["dk"]), _addr(out["dv"]),
             _addr(out["dinit"]), ctypes.byref(shape), _addr(workspace), have)
    return out


def lin_attn_step(state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                  slots: Optional[torch.Tensor] = None, scale: float = 1.0,
                  o: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token for each entry of a batch (ssd_lin_attn_step): updates `state`
    [num_slots, H, dv, dk] fp32 in place and returns o [b, H, dv].

    q [b, H, dk], k [b, Hk, dk], v [b, Hk, dv]; slots int32 [b]: the state each entry
    uses (None: entry i uses state i). Slots outside the pool are padding (o = 0);
    entries that name one slot are taken in the order of the batch; there may be none.
    """
    _check_dtype(q, "q", "[batch, nheads, dk]", 3)
    b, H, Dk = q.shape
    if not isinstance(k, torch.Tensor) or k.dim() != 3 or k.shape[0] != b or k.shape[2] != Dk:
        raise ValueError(f"k must be a 3-d tensor [{b}, nkv_heads, {Dk}]")
    Hk = k.shape[1]
    if Hk < 1 or H % Hk:
        raise ValueError(f"nheads {H} must be a multiple of nkv_heads {Hk}")
    if not isinstance(v, torch.Tensor) or v.dim() != 3 or tuple(v.shape[:2]) != (b, Hk):
        raise ValueError(f"v must be a 3-d tensor [{b}, {Hk}, dv]")
    Dv = v.shape[2]
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be a 4-d tensor [num_slots, nheads, dv, dk]")
    if log_decay is None:
        raise ValueError("log_decay is required")
    n = state.shape[0]
    _int32(dict(batch=b, nheads=H, dk=Dk, dv=Dv, num_slots=n))
    if slots is None and n < b:
        raise ValueError(f"state has {n} slots for {b} entries")
    dtype, device = q.dtype, q.device
    _check(device, ((q, "q", None, dtype, 16), (k, "k", None, dtype, 16), (v, "v", None, dtype, 16),
                    (state, "state", (n, H, Dv, Dk), torch.float32, 16), (o, "o", (b, H, Dv), dtype, 16),
                    (log_decay, "log_decay", (H,), torch.float32, 4), (slots, "slots", (b,), torch.int32, 4)))
    if o is None:
        o = torch.empty((b, H, Dv), dtype=dtype, device=device)
    if b == 0:
        _check_scale(scale)
        _size_of("ssd_lin_attn_workspace_bytes", LinShape, (1, 1, H, Hk, Dk, Dv, 0, _dtype_code(dtype), 0, 0, 0))   # its sizes
        return o
    shape = _lin_struct(b, 1, H, Hk, Dk, Dv, 0, _dtype_code(dtype), 0, 0, 0)
    _call_on(device, "ssd_lin_attn_step", _addr(state), _addr(q), _addr(k), _addr(v), _addr(log_decay), _addr(slots), n,
             float(scale), _addr(o), ctypes.byref(shape))
    return o


# ---------------------------------------------------------------------------
# Group norm over channels-last rows
# ---------------------------------------------------------------------------

_ACTS = {"none": 0, "silu": 1}
_GATES = {"after": 1, "before": 2}


def _row_pitch(t: torch.Tensor, name: str) -> int:
    """Elements from row to row of [samples, ..., channels]."""
    C = t.shape[-1]
    if C > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have its channels contiguous")
    pitch, rows = None, 1
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size > 1:
            if pitch is None:
                pitch = stride
            if stride != rows * pitch:
                raise ValueError(f"{name} must have its rows at one distance")
        rows *= size
    pitch = C if pitch is None else pitch
    if pitch < C:
        raise ValueError(f"{name} must have its rows at one distance of at least {C} channels")
    return pitch


def _norm_shape(x, groups, z, act, gate, center) -> NormShape:
    if not isinstance(x, torch.Tensor) or x.dim() < 2:
        raise ValueError("x must be a tensor [samples, ..., channels]")
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"x has dtype {x.dtype}; bfloat16 and float32 are supported")
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    if gate not in _GATES:
        raise ValueError(f"gate must be one of {sorted(_GATES)}")
    C = x.shape[-1]
    if groups < 1 or C % groups:
        raise ValueError(f"channels {C} must be a multiple of groups {groups}")
    if z is not None:
        if not isinstance(z, torch.Tensor) or z.shape != x.shape:
            raise ValueError(f"z must have x's shape {tuple(x.shape)}")
        if z.dtype != x.dtype:
            raise ValueError(f"z has dtype {z.dtype}, expected {x.dtype}")
    positions = 1
    for d in x.shape[1:-1]:
        positions *= d
    _int32(dict(samples=x.shape[0], positions=positions, channels=C))
    # No samples: nothing is run, and the rest is checked as for one.
    return NormShape(max(x.shape[0], 1), positions, C, int(groups), _row_pitch(x, "x"), 0 if z is None else _row_pitch(z, "z"),
                     _dtype_code(x.dtype), _ACTS[act], 0 if z is None else _GATES[gate], 1 if center else 0)


def _norm_workspace(shape: NormShape, backward: int, workspace, device):
    values = (shape.samples, shape.positions, shape.channels, shape.groups, shape.x_row, shape.z_row, shape.dtype, shape.act,
              shape.gate, shape.center)
    return _room(_size_of("ssd_group_norm_workspace_bytes", NormShape, values, backward), workspace, device)


def group_norm(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               z: Optional[torch.Tensor] = None, eps: float = 1e-5, act: str = "none", gate: str = "after",
               center: bool = True, y: Optional[torch.Tensor] = None, stats: Optional[torch.Tensor] = None,
               want_stats: bool = True, workspace: Optional[torch.Tensor] = None):
    """Group norm over channels-last x [samples, ..., channels] (ssd_group_norm). Returns (y, stats or None).

    A group is channels / groups channels over every position of a sample; for the
    norm of a token pass [tokens, channels]. act ("none", "silu") follows the norm;
    with z, gate "after" multiplies y by silu(z), "before" the input. weight and
    bias are fp32 [channels]; center=False takes the root mean square. x and z may
    have rows in wider rows. stats [samples, groups, 2] fp32 are the mean and
    1 / sqrt(var + eps) that group_norm_bwd takes. There may be no samples.
    """
    shape = _norm_shape(x, groups, z, act, gate, center)
    n, C = x.shape[0], shape.channels
    st = (n, shape.groups, 2)
    e = x.element_size()
    _check(x.device, ((x, "x", None, None, e), (z, "z", None, None, e), (weight, "weight", (C,), torch.float32, e),
                      (bias, "bias", (C,), torch.float32, e), (y, "y", x.shape, x.dtype, e),
                      (stats, "stats", st, torch.float32, e), (workspace, "workspace", None, torch.uint8, 256)))
    workspace, have = _norm_workspace(shape, 0, workspace, x.device)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if stats is None and want_stats:
        stats = torch.empty(st, dtype=torch.float32, device=x.device)
    if n == 0:
        if not 0.0 < eps < float("inf"):
            raise ValueError(f"eps {eps} must be above 0")
        return y, stats
    _call_on(x.device, "ssd_group_norm", _addr(x), _addr(z), _addr(weight), _addr(bias), float(eps), _addr(y), _addr(stats),
             ctypes.byref(shape), _addr(workspace), have)
    return y, stats


def group_norm_bwd(x: torch.Tensor, groups: int, stats: torch.Tensor, dy: torch.Tensor,
                   weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                   z: Optional[torch.Tensor] = None, act: str = "none", gate: str = "after", center: bool = True,
                   workspace: Optional[torch.Tensor] = None):
    """Gradients of <dy, y> of group_norm with these inputs and its stats
    (ssd_group_norm_bwd). Returns dict(dx, dz, dweight, dbias), dz, dweight and
    dbias None where z, weight or bias is."""
    shape = _norm_shape(x, groups, z, act, gate, center)
    n, C = x.shape[0], shape.channels
    st = (n, shape.groups, 2)
    if stats is None or dy is None:
        raise ValueError("stats and dy are required")
    e = x.element_size()
    _check(x.device, ((x, "x", None, None, e), (z, "z", None, None, e), (dy, "dy", x.shape, x.dtype, e),
                      (weight, "weight", (C,), torch.float32, e), (bias, "bias", (C,), torch.float32, e),
                      (stats, "stats", st, torch.float32, e), (workspace, "workspace", None, torch.uint8, 256)))
    workspace, have = _norm_workspace(shape, 1, workspace, x.device)
    out = dict(dx=torch.empty(x.shape, dtype=x.dtype, device=x.device),
               dz=None if z is None else torch.empty(x.shape, dtype=x.dtype, device=x.device),
               dweight=None if weight is None else torch.empty(C, dtype=torch.float32, device=x.device),
               dbias=None if bias is None else torch.empty(C, dtype=torch.float32, device=x.device))
    if n == 0:
        for name in ("dweight", "dbias"):
            if out[name] is not None:
                out[name].zero_()
        return out
    _call_on(x.device, "ssd_group_norm_bwd", _addr(x), _addr(z), _addr(weight), _addr(bias), _addr(stats), _addr(dy),
             _addr(out["dx"]), _addr(out["dz"]), _addr(out["dweight"]), _addr(out["dbias"]), ctypes.byref(shape),
             _addr(workspace), have)
    return out


# ---------------------------------------------------------------------------
# Pages of a pool of states
# ---------------------------------------------------------------------------

PAGES_MAX_PAIRS = 1024   # SSD_PAGES_MAX_PAIRS


def _pages_shape(pool) -> PagesShape:
    if not isinstance(pool, torch.Tensor) or pool.dim() < 3:
        raise ValueError("pool must be a tensor [layers, slots, ...]")
    if not pool.is_contiguous():
        raise ValueError("pool must be contiguous")
    if pool.numel() == 0:
        raise ValueError("pool is empty")
    _int32(dict(layers=pool.shape[0], slots=pool.shape[1]))
    return PagesShape(pool.shape[0], pool.shape[1], pool.numel() // (pool.shape[0] * pool.shape[1]) * pool.element_size())


def pages_copy(pool: torch.Tensor, src: torch.Tensor, dst: torch.Tensor) -> torch.Tensor:
    """pool[:, dst[i]] = pool[:, src[i]] for all pairs at once (ssd_pages_copy), in place:
    every source is read as it was before the call. pool [layers, slots, ...] of any
    type; src and dst int32 [n], n <= PAGES_MAX_PAIRS. A pair with an index outside the
    pool is left out; of pairs with one destination the last is kept."""
    shape = _pages_shape(pool)
    if not isinstance(src, torch.Tensor) or src.dim() != 1:
        raise ValueError("src must be a 1-d tensor")
    if dst is None:
        raise ValueError("dst is required")
    _int32(dict(pairs=src.numel()))
    _check(pool.device, ((pool, "pool", None, None, 1), (src, "src", None, torch.int32, 4),
                         (dst, "dst", src.shape, torch.int32, 4)))
    if src.numel():
        _call_on(pool.device, "ssd_pages_copy", _addr(pool), _addr(src), _addr(dst), src.numel(), ctypes.byref(shape))
    return pool


def pages_clear(pool: torch.Tensor, slots: torch.Tensor) -> torch.Tensor:
    """Zeroes pool[:, slots] in place (ssd_pages_clear); slots int32 [n], indices outside the pool are left out."""
    shape = _pages_shape(pool)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a 1-d tensor")
    _structure([(slots, "slots", None, torch.int32)])
    _int32({"number of slots": slots.numel()})
    _expect_device([(pool, "pool")], pool.device, 1)
    _expect_device([(slots, "slots")], pool.device, 4)
    if slots.numel():
        _call_on(pool.device, "ssd_pages_clear", _addr(pool), _addr(slots), slots.numel(), ctypes.byref(shape))
    return pool


def pages_compact(pool: torch.Tensor, live: torch.Tensor, where: Optional[torch.Tensor] = None,
                  count: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Moves the live pages of pool [layers, slots, ...] into its first `count` slots, in
    place (ssd_pages_compact). live: uint8 or bool [slots]. Returns (where, count): int32
    [slots], each old page's new index (-1: dead), and int32 [1]."""
    shape = _pages_shape(pool)
    if isinstance(live, torch.Tensor) and live.dtype == torch.bool:
        live = live.view(torch.uint8)
    if live is None:
        raise ValueError("live is required")
    _check(pool.device, ((pool, "pool", None, None, 1), (live, "live", (shape.slots,), torch.uint8, 1),
                         (where, "where", (shape.slots,), torch.int32, 4), (count, "count", (1,), torch.int32, 4),
                         (workspace, "workspace", None, torch.uint8, 256)))
    size = _size_of("ssd_pages_compact_workspace_bytes", PagesShape, (shape.layers, shape.slots, shape.page_bytes))
    workspace, have = _room(size, workspace, pool.device)
    if where is None:
        where = torch.empty(shape.slots, dtype=torch.int32, device=pool.device)
    if count is None:
        count = torch.empty(1, dtype=torch.int32, device=pool.device)
    _call_on(pool.device, "ssd_pages_compact", _addr(pool), _addr(live), _addr(where), _addr(count), ctypes.byref(shape),
             _addr(workspace), have)
    return where, count


# ---------------------------------------------------------------------------
# The gated delta rule
# ---------------------------------------------------------------------------

def _delta_shape(q, k, v, cu_seqlens):
    """The shape of a call over prompts, its tensors checked against one another."""
    _check_dtype(q, "q", "[batch, seqlen, nqk_heads, dk]", 4)
    b, T, Hk, Dk = q.shape
    if not isinstance(k, torch.Tensor) or tuple(k.shape) != (b, T, Hk, Dk):
        raise ValueError(f"k must be a 4-d tensor [{b}, {T}, {Hk}, {Dk}]")
    if not isinstance(v, torch.Tensor) or v.dim() != 4 or tuple(v.shape[:2]) != (b, T):
        raise ValueError(f"v must be a 4-d tensor [{b}, {T}, nheads, dv]")
    H = v.shape[2]
    if Hk < 1 or H < 1 or H % Hk:
        raise ValueError(f"nheads {H} must be a multiple of nqk_heads {Hk}")
    for t, name in ((k, "k"), (v, "v")):
        if t.dtype != q.dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {q.dtype}")
    S = 0
    if cu_seqlens is not None:
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be a 1-d tensor of num_seqs + 1 >= 2 entries")
        if b != 1:
            raise ValueError("packed sequences (cu_seqlens) need batch 1")
        S = cu_seqlens.numel() - 1
    _int32(dict(batch=b, seqlen=T, nheads=H, dk=Dk, dv=v.shape[3], num_seqs=S))
    # A batch without tokens runs nothing: its heads and sizes are checked as those of one token.
    return _delta_struct(max(b, 1), max(T, 1), H, Hk, Dk, v.shape[3], S, _dtype_code(q.dtype), _token_row(q, "q"),
                         _token_row(k, "k"), _token_row(v, "v"))


@functools.lru_cache(maxsize=256)
def _delta_struct(*values) -> DeltaShape:
    """The C shape of these sizes (the library only reads it)."""
    return DeltaShape(*values)


def _delta_values(shape: DeltaShape):
    return tuple(getattr(shape, name) for name, _ in DeltaShape._fields_)


def _delta_size(fn: str, shape: DeltaShape) -> int:
    """Workspace bytes; refuses sizes that the library does not take, of a batch without tokens too."""
    return _size_of(fn, DeltaShape, _delta_values(shape))


def gated_delta_shape(q, k, v, cu_seqlens=None) -> DeltaShape:
    """The shape of a call with these tensors (for gated_delta_workspace_bytes)."""
    return DeltaShape(*_delta_values(_delta_shape(q, k, v, cu_seqlens)))   # the caller's own


def gated_delta_workspace_bytes(shape: DeltaShape) -> int:
    n = ctypes.c_size_t(0)
    _call("ssd_gated_delta_workspace_bytes", ctypes.byref(shape), ctypes.byref(n))
    return int(n.value)


def gated_delta_bwd_workspace_bytes(shape: DeltaShape) -> int:
    n = ctypes.c_size_t(0)
    _call("ssd_gated_delta_bwd_workspace_bytes", ctypes.byref(shape), ctypes.byref(n))
    return int(n.value)


def gated_delta_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: Optional[torch.Tensor],
                    beta: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None, scale: float = 1.0,
                    initial_state: Optional[torch.Tensor] = None, o: Optional[torch.Tensor] = None,
                    final_state: Optional[torch.Tensor] = None, want_final: bool = True,
                    workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The gated delta rule over prompts (ssd_gated_delta_fwd). Returns (o, final_state or None).

    q, k [b, T, Hk, dk], v [b, T, H, dv] (bf16 or fp32; tokens may lie in wider rows,
    as slices of one projection do; value head h reads query and key head
    h / (H / Hk)), log_decay [b, T, H] fp32 <= 0 or None (no decay), beta [b, T, H]
    fp32, states fp32 [rows or sequences, H, dv, dk]. cu_seqlens may hold empty
    sequences, and a batch no rows or tokens at all (its final states are the initial
    ones); rows of o that belong to no sequence are left as they were (undefined in an
    o made here).
    """
    shape = _delta_shape(q, k, v, cu_seqlens)
    b, T, H, Dv = v.shape
    Dk, nseq = q.shape[3], shape.num_seqs or b
    if beta is None:
        raise ValueError("beta is required")
    st = (nseq, H, Dv, Dk)
    _check(q.device, ((q, "q", None, None, 16), (k, "k", None, None, 16), (v, "v", None, None, 16),
                      (initial_state, "initial_state", st, torch.float32, 16), (o, "o", (b, T, H, Dv), q.dtype, 16),
                      (final_state, "final_state", st, torch.float32, 16),
                      (log_decay, "log_decay", (b, T, H), torch.float32, 4), (beta, "beta", (b, T, H), torch.float32, 4),
                      (cu_seqlens, "cu_seqlens", None, torch.int32, 4), (workspace, "workspace", None, torch.uint8, 256)))
    if final_state is not None and initial_state is not None and _share(final_state, initial_state):
        raise ValueError("final_state must not overlap initial_state")
    size = _delta_size("ssd_gated_delta_workspace_bytes", shape)
    if o is None:
        o = torch.empty(b, T, H, Dv, dtype=q.dtype, device=q.device)
    if b * T == 0:
        _check_scale(scale)
        return o, _state_of_no_tokens(initial_state, final_state, want_final, st, q.device)
    workspace, have = _room(size, workspace, q.device)
    if final_state is None and want_final:
        final_state = torch.empty(st, dtype=torch.float32, device=q.device)
    _call_on(q.device, "ssd_gated_delta_fwd", _addr(q), _addr(k), _addr(v), _addr(log_decay), _addr(beta), _addr(cu_seqlens),
             float(scale), _addr(initial_state), _addr(o), _addr(final_state), ctypes.byref(shape), _addr(workspace), have)
    return o, final_state


def gated_delta_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: Optional[torch.Tensor],
                    beta: torch.Tensor, do: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None, scale: float = 1.0,
                    initial_state: Optional[torch.Tensor] = None, dfinal_state: Optional[torch.Tensor] = None,
                    want_dinit: bool = False, workspace: Optional[torch.Tensor] = None):
    """Gradients of <do, o> + <dfinal_state, final_state> of gated_delta_fwd with these
    inputs (ssd_gated_delta_bwd). Returns dict(dq, dk, dv, dlog_decay, dbeta, dinit),
    dlog_decay None without decays and dinit unless it is wanted. Rows that belong to
    no sequence are undefined."""
    shape = _delta_shape(q, k, v, cu_seqlens)
    b, T, H, Dv = v.shape
    Dk, nseq = q.shape[3], shape.num_seqs or b
    if beta is None or do is None:
        raise ValueError("beta and do are required")
    st = (nseq, H, Dv, Dk)
    _check(q.device, ((q, "q", None, None, 16), (k, "k", None, None, 16), (v, "v", None, None, 16),
                      (do, "do", (b, T, H, Dv), q.dtype, 16), (initial_state, "initial_state", st, torch.float32, 16),
                      (dfinal_state, "dfinal_state", st, torch.float32, 16),
                      (log_decay, "log_decay", (b, T, H), torch.float32, 4), (beta, "beta", (b, T, H), torch.float32, 4),
                      (cu_seqlens, "cu_seqlens", None, torch.int32, 4), (workspace, "workspace", None, torch.uint8, 256)))
    size = _delta_size("ssd_gated_delta_bwd_workspace_bytes", shape)
    new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=q.device)   # noqa: E731
    out = dict(dq=new(q.shape, q.dtype), dk=new(k.shape, q.dtype), dv=new(v.shape, q.dtype),
               dlog_decay=None if log_decay is None else new((b, T, H), torch.float32), dbeta=new((b, T, H), torch.float32),
               dinit=new(st, torch.float32) if want_dinit else None)
    if b * T == 0:
        _check_scale(scale)
        _state_of_no_tokens(dfinal_state, out["dinit"], want_dinit, st, q.device)
        return out
    workspace, have = _room(size, workspace, q.device)
    _call_on(q.device, "ssd_gated_delta_bwd", _addr(q), _addr(k), _addr(v), _addr(log_decay), _addr(beta), _addr(cu_seqlens),
             float(scale), _addr(initial_state), _addr(do), _addr(dfinal_state), _addr(out["dq"]), _addr(out["dk"]),
             _addr(out["dv"]), _addr(out["dlog_decay"]), _addr(out["dbeta"]), _addr(out["dinit"]), ctypes.byref(shape),
             _addr(workspace), have)
    return out


def gated_delta_step(state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     log_decay: Optional[torch.Tensor], beta: torch.Tensor, slots: Optional[torch.Tensor] = None,
                     scale: float = 1.0, o: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token for each entry of a batch (ssd_gated_delta_step): updates `state`
    [num_slots, H, dv, dk] fp32 in place and returns o [b, H, dv].

    q, k [b, Hk, dk], v [b, H, dv], log_decay (or None) and beta [b, H] fp32; slots
    int32 [b]: the state each entry uses (None: entry i uses state i). Slots outside
    the pool are padding (o = 0); entries that name one slot are taken in the order
    of the batch; there may be none.
    """
    _check_dtype(q, "q", "[batch, nqk_heads, dk]", 3)
    b, Hk, Dk = q.shape
    if not isinstance(k, torch.Tensor) or tuple(k.shape) != (b, Hk, Dk):
        raise ValueError(f"k must be a 3-d tensor [{b}, {Hk}, {Dk}]")
    if not isinstance(v, torch.Tensor) or v.dim() != 3 or v.shape[0] != b:
        raise ValueError(f"v must be a 3-d tensor [{b}, nheads, dv]")
    H, Dv = v.shape[1:]
    if Hk < 1 or H < 1 or H % Hk:
        raise ValueError(f"nheads {H} must be a multiple of nqk_heads {Hk}")
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be a 4-d tensor [num_slots, nheads, dv, dk]")
    if beta is None:
        raise ValueError("beta is required")
    n = state.shape[0]
    _int32(dict(batch=b, nheads=H, dk=Dk, dv=Dv, num_slots=n))
    if slots is None and n < b:
        raise ValueError(f"state has {n} slots for {b} entries")
    dtype, device = q.dtype, q.device
    _check(device, ((q, "q", None, dtype, 16), (k, "k", None, dtype, 16), (v, "v", None, dtype, 16),
                    (state, "state", (n, H, Dv, Dk), torch.float32, 16), (o, "o", (b, H, Dv), dtype, 16),
                    (log_decay, "log_decay", (b, H), torch.float32, 4), (beta, "beta", (b, H), torch.float32, 4),
                    (slots, "slots", (b,), torch.int32, 4)))
    if o is None:
        o = torch.empty((b, H, Dv), dtype=dtype, device=device)
    if b == 0:
        _check_scale(scale)
        _size_of("ssd_gated_delta_workspace_bytes", DeltaShape, (1, 1, H, Hk, Dk, Dv, 0, _dtype_code(dtype), 0, 0, 0))   # its sizes
        return o
    shape = _delta_struct(b, 1, H, Hk, Dk, Dv, 0, _dtype_code(dtype), 0, 0, 0)
    _call_on(device, "ssd_gated_delta_step", _addr(state), _addr(q), _addr(k), _addr(v), _addr(log_decay), _addr(beta),
             _addr(slots), n, float(scale), _addr(o), ctypes.byref(shape))
    return o


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

_ROTARY_LAYOUTS = {"half": 0, "interleaved": 1}
_ROTARY_MOST = 1024   # elements of a head, as the C ABI checks


def rotary_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       original_length: int = 0, slow: float = 1.0, fast: float = 32.0, device=None):
    """The frequencies base^(-2 i / rot), i < rot / 2, as rotary takes them (fp32), and the
    scale that goes with them: (freq, scale). For contexts `factor` times as long as
    the one that a model was trained on:

      "none"      as they are;
      "linear"    divided by factor;
      "ntk"       of the base times factor^(rot / (rot - 2)): the fastest stays, the slowest
                  is divided by factor;
      "by_parts"  divided by factor where they turn less than `slow` times over
                  original_length, kept where more than `fast` times, mixed in between;
                  scale 1 + 0.1 ln factor, of queries and of keys.
    """
    if rot < 2 or rot % 2:
        raise ValueError(f"rot {rot} must be even and at least 2")
    if scaling not in ("none", "linear", "ntk", "by_parts"):
        raise ValueError(f"scaling {scaling!r} must be none, linear, ntk or by_parts")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be above 0")
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    if scaling == "ntk":
        if rot < 4:
            raise ValueError("ntk scaling needs rot of at least 4")
        base = base * factor ** (rot / (rot - 2))
    freq, scale = base ** (-i / rot), 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "by_parts":
        if original_length < 1 or not fast > slow:
            raise ValueError("by_parts scaling needs original_length and fast > slow")
        turns = original_length * freq / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        freq = freq * keep + freq / factor * (1 - keep)
        scale = 1 + 0.1 * math.log(factor) if factor > 1 else 1.0
    return freq.float().to(device), scale


def _row_of(shape, stride, name: str) -> int:
    """Elements from token to token of [batch, seqlen, heads, d] or [batch, heads, d] (one row of tokens): heads and
    their elements lie together, tokens at one distance, rows of the batch follow on."""
    if len(shape) == 3:
        shape, stride = (1,) + tuple(shape), (0,) + tuple(stride)
    b, T, H, D = shape
    if (D > 1 and stride[3] != 1) or (H > 1 and stride[2] != D):
        raise ValueError(f"{name} must have its heads contiguous (strides {stride})")
    if b * T * H * D == 0:
        return H * D
    row = stride[1] if T > 1 else (stride[0] if b > 1 else H * D)
    if row < H * D or (b > 1 and stride[0] != T * row):
        raise ValueError(f"{name} must have its tokens at one distance (strides {stride})")
    return row


@functools.lru_cache(maxsize=256)
def _rotary_struct(dtype, layout, inverse, entries, starts, q, k, q_out, k_out) -> RotaryShape:
    """The C shape of tensors of these (shape, strides), checked against one another; once for each call's sizes, as a
    token's call is its host's time. entries: frequencies; starts: entries of cu_seqlens, 0 without."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"q has dtype {dtype}; bfloat16 and float32 are supported")
    if layout not in _ROTARY_LAYOUTS:
        raise ValueError(f"layout {layout!r} must be half or interleaved")
    shape = q[0]
    if len(shape) not in (3, 4):
        raise ValueError("q must be a tensor [batch, seqlen, heads, dim] or [batch, heads, dim]")
    if k is not None and (len(k[0]) != len(shape) or k[0][:-2] != shape[:-2] or k[0][-1] != shape[-1]):
        raise ValueError(f"k must be a tensor [..., heads, {shape[-1]}] of q's leading sizes {tuple(shape[:-2])}")
    for name, src, out in (("q_out", q, q_out), ("k_out", k, k_out)):
        if out is not None and (src is None or out[0] != src[0]):
            raise ValueError(f"{name} must have the shape of what is turned")
    b, T = (1, shape[0]) if len(shape) == 3 else shape[:2]
    H, dim, Hk = shape[-2], shape[-1], 0 if k is None else k[0][-2]
    if H < 1 or (k is not None and Hk < 1):
        raise ValueError("q and k must have at least one head")
    if starts == 1 or (starts and (len(shape) == 3 or b != 1)):
        raise ValueError("cu_seqlens must have num_seqs + 1 >= 2 entries, for q [1, seqlen, heads, dim]")
    if not 2 <= 2 * entries <= dim:
        raise ValueError(f"freq has {entries} entries for heads of {dim}")
    S = starts - 1 if starts else 0
    _int32(dict(batch=b, seqlen=T, q_heads=H, k_heads=Hk, dim=dim, num_seqs=S))
    row = lambda t, name: 0 if t is None else _row_of(*t, name)   # noqa: E731
    # A batch without tokens runs nothing: its heads and sizes are checked as those of one token.
    return RotaryShape(max(b, 1), max(T, 1), H, Hk, dim, 2 * entries, S, _dtype_code(dtype), _ROTARY_LAYOUTS[layout], inverse,
                       row(q, "q"), row(k, "k"), row(q_out, "q_out"), row(k_out, "k_out"))


def _rotary(q, k, freq, positions, cu_seqlens, offsets, layout, scale, q_out, k_out, inverse):
    for t, name, none in ((q, "q", False), (k, "k", True), (freq, "freq", False), (positions, "positions", True),
                          (cu_seqlens, "cu_seqlens", True), (offsets, "offsets", True), (q_out, "q_out", True),
                          (k_out, "k_out", True)):
        if not (isinstance(t, torch.Tensor) or (none and t is None)):
            raise ValueError(f"{name} must be a torch tensor")
    if freq.dim() != 1 or (cu_seqlens is not None and cu_seqlens.dim() != 1):
        raise ValueError("freq and cu_seqlens must be 1-d tensors")
    if positions is None:
        if q.dim() == 3:
            raise ValueError("positions are required for one token an entry")
    elif offsets is not None:
        raise ValueError("positions and offsets exclude each other")
    of = lambda t: None if t is None else (t.shape, t.stride())   # noqa: E731
    dtype, device, e = q.dtype, q.device, q.element_size()
    shape = _rotary_struct(dtype, layout, inverse, freq.numel(), 0 if cu_seqlens is None else cu_seqlens.numel(), of(q), of(k),
                           of(q_out), of(k_out))
    index = device.index if device.type == "cuda" else -1
    for t, name in ((q, "q"), (k, "k"), (q_out, "q_out"), (k_out, "k_out")):
        if t is not None and not (t.dtype == dtype and t.get_device() == index >= 0 and t.data_ptr() % e == 0):
            if t.dtype != dtype:
                raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
            _expect_device([(t, name)], device, e)
    _check(device, ((freq, "freq", None, torch.float32, 4), (positions, "positions", q.shape[:-2], torch.int32, 4),
                    (cu_seqlens, "cu_seqlens", None, torch.int32, 4),
                    (offsets, "offsets", None if offsets is None else (shape.num_seqs or q.shape[0],), torch.int32, 4)))
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=dtype, device=device)
    if k is not None and k_out is None:
        k_out = torch.empty(k.shape, dtype=dtype, device=device)
    if q.numel() == 0:
        _check_scale(scale)
        if shape.dim > _ROTARY_MOST:
            raise ValueError(f"heads of {shape.dim} elements; up to {_ROTARY_MOST} are supported")
        return q_out, k_out
    _call_on(device, "ssd_rotary", q.data_ptr(), _addr(k), freq.data_ptr(), _addr(positions), _addr(cu_seqlens), _addr(offsets),
             float(scale), q_out.data_ptr(), _addr(k_out), ctypes.byref(shape))
    return q_out, k_out


def rotary(q: torch.Tensor, k: Optional[torch.Tensor], freq: torch.Tensor, positions: Optional[torch.Tensor] = None,
           cu_seqlens: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None, layout: str = "half",
           scale: float = 1.0, q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """Rotary positions of queries and keys (ssd_rotary). Returns (q_out, k_out or None).

    q [b, T, H, dim] and k [b, T, Hk, dim] or None (bf16 or fp32; tokens may lie in wider
    rows), or one token an entry [b, H, dim] with its positions [b]. Of each head the
    first 2 * len(freq) elements are turned, in pairs (i, i + len(freq)) for layout
    "half" or (2 i, 2 i + 1) for "interleaved", by position * freq[i]; freq fp32, of
    rotary_frequencies or any other. positions int32 [b, T], or None: a token's place in
    its row or packed sequence, plus offsets [rows or sequences] int32. q_out and k_out
    may be q and k (in place).
    """
    return _rotary(q, k, freq, positions, cu_seqlens, offsets, layout, scale, q_out, k_out, 0)


def rotary_bwd(dq: torch.Tensor, dk: Optional[torch.Tensor], freq: torch.Tensor, positions: Optional[torch.Tensor] = None,
               cu_seqlens: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None, layout: str = "half",
               scale: float = 1.0, q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """Gradients of q and k from those of rotary's results with these arguments: turned
    back, the same scale. Returns (gradient of q, gradient of k or None)."""
    return _rotary(dq, dk, freq, positions, cu_seqlens, offsets, layout, scale, q_out, k_out, 1)
