"""Thin ctypes binding to libw4.so (include/w4.h).  Argument marshalling only:
every step of the computation runs in the library's CUDA kernels.

Tensors are torch CUDA tensors (torch is used for device memory and streams).
Each function enqueues on the given stream, or on torch's current stream of the
tensor's device when ``stream`` is None, and raises W4Error on a non-OK status.
Importing this module raises if the CUDA library has not been built.
"""
from __future__ import annotations

import contextlib
import ctypes
import enum
import math
import os
import struct
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4.so")
HEADER_BYTES = 128
GROUP = 128
MAX_TOKENS = 8
STATIC_SCRATCH_BYTES = 4 * 1024 * 1024   # W4_STATIC_SCRATCH_BYTES

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the CUDA library first "
        "(python -c 'import __graft_entry__ as g; g.build()'). There is no CPU fallback.")

_lib = ctypes.CDLL(LIB_PATH)
_P = ctypes.c_void_p
_I = ctypes.c_int
_ST = ctypes.c_int


def _decl(name, res, *args):
    fn = getattr(_lib, name)
    fn.restype = res
    fn.argtypes = list(args)
    return fn


_status_string = _decl("w4_status_string", ctypes.c_char_p, _ST)
_version = _decl("w4_version", _I)
_repacked_sizes = _decl("w4_repacked_sizes", _ST, _I, _I, ctypes.POINTER(ctypes.c_size_t),
                        ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t))
_repack = _decl("w4_repack", _ST, _P, _P, _P, _I, _I, _P, _P, _P, _P)
_check_header = _decl("w4_check_header", _ST, _P, _I, _I)
_dequant = _decl("w4_dequant", _ST, _P, _P, _P, _I, _I, _P, _P)
_gemv = _decl("w4_gemv", _ST, _P, _P, _P, _P, _P, _I, _I, _I, _P)
_gemv_f32 = _decl("w4_gemv_f32", _ST, _P, _P, _P, _P, _P, _I, _I, _I, _P)
_repacked_sizes_swiglu = _decl("w4_repacked_sizes_swiglu", _ST, _I, _I,
                               ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t),
                               ctypes.POINTER(ctypes.c_size_t))
_repack_swiglu = _decl("w4_repack_swiglu", _ST, _P, _P, _P, _I, _I, _P, _P, _P, _P)
_check_header_swiglu = _decl("w4_check_header_swiglu", _ST, _P, _I, _I)
_gemv_swiglu = _decl("w4_gemv_swiglu", _ST, _P, _P, _P, _P, _P, _I, _I, _I, _P)
_gemv_swiglu_f32 = _decl("w4_gemv_swiglu_f32", _ST, _P, _P, _P, _P, _P, _I, _I, _I, _P)
_quantize = _decl("w4_quantize", _ST, _P, _I, _I, _I, _P, _P, _P, _P)
_gemv_ws_static = _decl("w4_gemv_ws_static", _ST, _P, _P, _P, _P, _P, _I, _I, _I, _P)
_selftest_bounded_wait = _decl("w4_selftest_bounded_wait", _ST, _P, _P)
_stream_read = _decl("w4_stream_read", _ST, _P, ctypes.c_size_t, _I, _P, _P)
_gemm = _decl("w4_gemm", _ST, _P, _P, _P, _P, _P, _I, _I, _I, _P)
_gemm_f32 = _decl("w4_gemm_f32", _ST, _P, _P, _P, _P, _P, _I, _I, _I, _P)
_gemv_config = _decl("w4_gemv_config", _ST, _I, _I, ctypes.POINTER(_I), ctypes.POINTER(_I),
                     ctypes.POINTER(_I))


class _LaunchInfo(ctypes.Structure):
    _fields_ = [("k_splits", _I), ("zero_point_folded", _I), ("grid_x", _I), ("grid_y", _I),
                ("persistent", _I), ("overlap", _I), ("capped", _I), ("ring_stages", _I),
                ("wide_prologue", _I), ("blocks_per_sm_max", _I),
                ("smem_bytes", ctypes.c_size_t)]


_gemv_plan = _decl("w4_gemv_plan", _ST, _I, _I, _I, ctypes.POINTER(_LaunchInfo))
_gemv_workspace_bytes = _decl("w4_gemv_workspace_bytes", _ST, _I, _I,
                              ctypes.POINTER(ctypes.c_size_t))
_gemv_ws = _decl("w4_gemv_ws", _ST, _P, _P, _P, _P, _P, _I, _I, _I, _P, ctypes.c_size_t, _P)
_gemv_ws_f32 = _decl("w4_gemv_ws_f32", _ST, _P, _P, _P, _P, _P, _I, _I, _I, _P, ctypes.c_size_t,
                     _P)


class Status(enum.IntEnum):
    OK = 0
    INVALID_ARG = 1
    UNSUPPORTED = 2
    LAYOUT = 3
    CUDA = 4
    SCRATCH_LIMIT = 5


class W4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = Status(status) if status in Status._value2member_map_ else status
        super().__init__(f"{where}: {status_string(status)}")


def status_string(status: int) -> str:
    return _status_string(int(status)).decode()


def library_path() -> str:
    return LIB_PATH


def version() -> int:
    return _version()


def _ok(status: int, where: str) -> None:
    if status != 0:
        raise W4Error(status, where)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream, like: torch.Tensor):
    if stream is None:
        stream = torch.cuda.current_stream(like.device)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def repacked_sizes(K: int, N: int):
    """Byte sizes (qweight, scales, zeros) of the kernel layout for N x K."""
    q, s, z = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _ok(_repacked_sizes(K, N, ctypes.byref(q), ctypes.byref(s), ctypes.byref(z)),
        "w4_repacked_sizes")
    return q.value, s.value, z.value


def repack(qweight, scales, zeros, K: int, N: int, qweight_out, scales_out, zeros_out,
           stream=None) -> None:
    """w4_repack: canonical device tensors -> the three kernel-layout buffers."""
    _ok(_repack(_ptr(qweight), _ptr(scales), _ptr(zeros), K, N, _ptr(qweight_out),
                _ptr(scales_out), _ptr(zeros_out), _stream(stream, qweight)), "w4_repack")


def check_header(header_bytes: bytes, K: int, N: int) -> None:
    buf = ctypes.create_string_buffer(bytes(header_bytes), HEADER_BYTES)
    _ok(_check_header(ctypes.cast(buf, ctypes.c_void_p), K, N), "w4_check_header")


def dequant(qweight, scales, zeros, K: int, N: int, w_out, stream=None) -> None:
    """w4_dequant: canonical weights -> binary16 [N, K] (bit patterns in w_out)."""
    _ok(_dequant(_ptr(qweight), _ptr(scales), _ptr(zeros), K, N, _ptr(w_out),
                 _stream(stream, qweight)), "w4_dequant")


def gemv(qweight, scales, zeros, x, y, M: int, K: int, N: int, stream=None) -> None:
    """w4_gemv: y[M, N] (bfloat16) = W x with W in the kernel layout."""
    _ok(_gemv(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(x), _ptr(y), M, K, N,
              _stream(stream, x)), "w4_gemv")


def gemv_f32(qweight, scales, zeros, x, y, M: int, K: int, N: int, stream=None) -> None:
    """w4_gemv_f32: as gemv but y is float32 (before the bfloat16 cast)."""
    _ok(_gemv_f32(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(x), _ptr(y), M, K, N,
                  _stream(stream, x)), "w4_gemv_f32")


def gemm(qweight, scales, zeros, x, y, M: int, K: int, N: int, stream=None) -> None:
    """w4_gemm: y[M, N] (bfloat16) for any M >= 1 (M <= 16: w4_gemv in passes
    of 8; more: one tensor-core pass over the weight)."""
    _ok(_gemm(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(x), _ptr(y), M, K, N,
              _stream(stream, x)), "w4_gemm")


def gemm_f32(qweight, scales, zeros, x, y, M: int, K: int, N: int, stream=None) -> None:
    """w4_gemm_f32: as gemm, fp32 result."""
    _ok(_gemm_f32(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(x), _ptr(y), M, K, N,
                  _stream(stream, x)), "w4_gemm_f32")


def gemv_workspace_bytes(K: int, N: int) -> int:
    """Bytes of workspace gemv_ws needs for N x K on the current device."""
    n = ctypes.c_size_t()
    _ok(_gemv_workspace_bytes(K, N, ctypes.byref(n)), "w4_gemv_workspace_bytes")
    return n.value


def workspace_counter_bytes(N: int) -> int:
    """Bytes of the row-block counters at the start of a gemv_ws workspace."""
    return ((N + 127) // 128 * 4 + 255) // 256 * 256


def workspace(K: int, N: int, device=None) -> torch.Tensor:
    """A zero-filled workspace tensor for gemv_ws (allocated by torch)."""
    return torch.zeros(gemv_workspace_bytes(K, N), dtype=torch.uint8,
                       device=device if device is not None else "cuda")


def gemv_ws(qweight, scales, zeros, x, y, M: int, K: int, N: int, workspace,
            stream=None) -> None:
    """w4_gemv_ws: as gemv, split evenly over one wave, combining through
    `workspace` (zero-filled before first use; each call leaves its counters,
    the first workspace_counter_bytes(N) bytes, at zero)."""
    _ok(_gemv_ws(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(x), _ptr(y), M, K, N,
                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                 _stream(stream, x)), "w4_gemv_ws")


def gemv_ws_f32(qweight, scales, zeros, x, y, M: int, K: int, N: int, workspace,
                stream=None) -> None:
    """w4_gemv_ws_f32: gemv_ws writing the fp32 result."""
    _ok(_gemv_ws_f32(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(x), _ptr(y), M, K, N,
                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                     _stream(stream, x)), "w4_gemv_ws_f32")


def gemv_ws_static(qweight, scales, zeros, x, y, M: int, K: int, N: int, stream=None) -> None:
    """w4_gemv_ws_static: gemv_ws with the library's static device scratch
    (allocates nothing).  Calls on one device must not overlap on the GPU;
    the first call on a device should come before any stream capture."""
    _ok(_gemv_ws_static(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(x), _ptr(y), M, K, N,
                        _stream(stream, x)), "w4_gemv_ws_static")


def repacked_sizes_swiglu(K: int, I: int):
    """Byte sizes (qweight, scales, zeros) of the gate/up-interleaved layout."""
    q, s, z = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _ok(_repacked_sizes_swiglu(K, I, ctypes.byref(q), ctypes.byref(s), ctypes.byref(z)),
        "w4_repacked_sizes_swiglu")
    return q.value, s.value, z.value


def repack_swiglu(qweight, scales, zeros, K: int, I: int, qweight_out, scales_out, zeros_out,
                  stream=None) -> None:
    """w4_repack_swiglu: fused [2I, K] gate/up weight -> interleaved kernel layout."""
    _ok(_repack_swiglu(_ptr(qweight), _ptr(scales), _ptr(zeros), K, I, _ptr(qweight_out),
                       _ptr(scales_out), _ptr(zeros_out), _stream(stream, qweight)),
        "w4_repack_swiglu")


def check_header_swiglu(header_bytes: bytes, K: int, I: int) -> None:
    buf = ctypes.create_string_buffer(bytes(header_bytes), HEADER_BYTES)
    _ok(_check_header_swiglu(ctypes.cast(buf, ctypes.c_void_p), K, I), "w4_check_header_swiglu")


def gemv_swiglu(qweight, scales, zeros, x, y, M: int, K: int, I: int, stream=None) -> None:
    """w4_gemv_swiglu: y[M, I] (bfloat16) = silu(gate x) * (up x)."""
    _ok(_gemv_swiglu(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(x), _ptr(y), M, K, I,
                     _stream(stream, x)), "w4_gemv_swiglu")


def gemv_swiglu_f32(qweight, scales, zeros, x, y, M: int, K: int, I: int, stream=None) -> None:
    """w4_gemv_swiglu_f32: the fp32 result."""
    _ok(_gemv_swiglu_f32(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(x), _ptr(y), M, K, I,
                         _stream(stream, x)), "w4_gemv_swiglu_f32")


QUANT_ASYMMETRIC = 0      # W4_QUANT_ASYMMETRIC
QUANT_SYMMETRIC = 1       # W4_QUANT_SYMMETRIC


def quantize(w, K: int, N: int, mode: int, qweight, scales, zeros, stream=None) -> None:
    """w4_quantize: binary16 W [N, K] -> canonical qweight, scales, zeros."""
    _ok(_quantize(_ptr(w), K, N, int(mode), _ptr(qweight), _ptr(scales), _ptr(zeros),
                  _stream(stream, w)), "w4_quantize")


def selftest_bounded_wait(status, stream=None) -> None:
    """w4_selftest_bounded_wait: the GEMV kernels' bounded mbarrier wait on a
    barrier nothing completes; `status` (a one-element int32 CUDA tensor)
    becomes 1 when the wait gave up as it must.  About 2 s on the GPU."""
    _ok(_selftest_bounded_wait(_ptr(status), _stream(stream, status)),
        "w4_selftest_bounded_wait")


STREAM_READ_RING = 0      # W4_STREAM_READ_RING
STREAM_READ_LD128 = 1     # W4_STREAM_READ_LD128


def stream_read(src, mode: int, out, stream=None) -> None:
    """w4_stream_read: read all of `src` (a CUDA tensor) once, folding it
    into out[0] (out: two-element int32 CUDA tensor); for measuring the
    read-only bandwidth."""
    _ok(_stream_read(_ptr(src), src.numel() * src.element_size(), int(mode), _ptr(out),
                     _stream(stream, src)), "w4_stream_read")


def gemv_config(K: int, N: int):
    """(16-row tiles per block, K splits, zero point folded) that w4_gemv uses
    for N x K."""
    t, s, f = _I(), _I(), _I()
    _ok(_gemv_config(K, N, ctypes.byref(t), ctypes.byref(s), ctypes.byref(f)), "w4_gemv_config")
    return t.value, s.value, bool(f.value)


def gemv_plan(M: int, K: int, N: int) -> dict:
    """The launch w4_gemv makes for M tokens of an N x K weight on the current
    device (w4_gemv_plan): split, arithmetic, grid, residency, overlap."""
    info = _LaunchInfo()
    _ok(_gemv_plan(M, K, N, ctypes.byref(info)), "w4_gemv_plan")
    return {name: (bool(getattr(info, name)) if name in
                   ("zero_point_folded", "persistent", "overlap", "capped", "wide_prologue")
                   else int(getattr(info, name))) for name, _ in _LaunchInfo._fields_}


@dataclass
class PackedWeight:
    """An N x K weight in the kernel layout (three device buffers)."""
    K: int
    N: int
    qweight: torch.Tensor   # uint8 bytes, starts with the 128-byte header
    scales: torch.Tensor    # uint8 bytes
    zeros: torch.Tensor     # uint8 bytes

    def gemv(self, x: torch.Tensor, y: torch.Tensor | None = None, stream=None,
             workspace: torch.Tensor | None = None) -> torch.Tensor:
        """y = W x for x bfloat16 [M, K] on the device; returns y bfloat16 [M, N].
        With a workspace (see `workspace()`), uses gemv_ws."""
        M = x.shape[0]
        if y is None:
            y = torch.empty((M, self.N), dtype=torch.bfloat16, device=x.device)
        if workspace is None:
            gemv(self.qweight, self.scales, self.zeros, x, y, M, self.K, self.N, stream)
        else:
            gemv_ws(self.qweight, self.scales, self.zeros, x, y, M, self.K, self.N, workspace,
                    stream)
        return y

    def gemv_f32(self, x: torch.Tensor, y: torch.Tensor | None = None, stream=None,
                 workspace: torch.Tensor | None = None):
        M = x.shape[0]
        if y is None:
            y = torch.empty((M, self.N), dtype=torch.float32, device=x.device)
        if workspace is None:
            gemv_f32(self.qweight, self.scales, self.zeros, x, y, M, self.K, self.N, stream)
        else:
            gemv_ws_f32(self.qweight, self.scales, self.zeros, x, y, M, self.K, self.N,
                        workspace, stream)
        return y


def pack(qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, K: int, N: int,
         stream=None) -> PackedWeight:
    """Allocate the kernel-layout buffers (torch), repack into them and check
    the header once."""
    dev = qweight.device
    qb, sb, zb = repacked_sizes(K, N)
    qo = torch.empty(qb, dtype=torch.uint8, device=dev)
    so = torch.empty(sb, dtype=torch.uint8, device=dev)
    zo = torch.empty(zb, dtype=torch.uint8, device=dev)
    repack(qweight, scales, zeros, K, N, qo, so, zo, stream)
    check_header(qo[:HEADER_BYTES].cpu().numpy().tobytes(), K, N)
    return PackedWeight(K, N, qo, so, zo)


@dataclass
class PackedSwiGLU:
    """A fused [2I, K] gate/up weight in the interleaved kernel layout."""
    K: int
    I: int
    qweight: torch.Tensor
    scales: torch.Tensor
    zeros: torch.Tensor

    def gemv(self, x: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """y[M, I] = silu(gate x) * (up x), bfloat16."""
        M = x.shape[0]
        if y is None:
            y = torch.empty((M, self.I), dtype=torch.bfloat16, device=x.device)
        gemv_swiglu(self.qweight, self.scales, self.zeros, x, y, M, self.K, self.I, stream)
        return y

    def gemv_f32(self, x: torch.Tensor, y: torch.Tensor | None = None, stream=None):
        M = x.shape[0]
        if y is None:
            y = torch.empty((M, self.I), dtype=torch.float32, device=x.device)
        gemv_swiglu_f32(self.qweight, self.scales, self.zeros, x, y, M, self.K, self.I, stream)
        return y


def pack_swiglu(qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, K: int,
                I: int, stream=None) -> PackedSwiGLU:
    """Allocate the interleaved-layout buffers (torch), repack the fused
    [2I, K] gate/up weight into them and check the header once."""
    dev = qweight.device
    qb, sb, zb = repacked_sizes_swiglu(K, I)
    qo = torch.empty(qb, dtype=torch.uint8, device=dev)
    so = torch.empty(sb, dtype=torch.uint8, device=dev)
    zo = torch.empty(zb, dtype=torch.uint8, device=dev)
    repack_swiglu(qweight, scales, zeros, K, I, qo, so, zo, stream)
    check_header_swiglu(qo[:HEADER_BYTES].cpu().numpy().tobytes(), K, I)
    return PackedSwiGLU(K, I, qo, so, zo)


# ---- rotary positions, the paged key-value cache and attention over it ---------

ROPE_HALF = 0             # W4_ROPE_HALF
ROPE_INTERLEAVED = 1      # W4_ROPE_INTERLEAVED
ROPE_SCALE_NONE = 0       # W4_ROPE_SCALE_NONE
ROPE_SCALE_LINEAR = 1     # W4_ROPE_SCALE_LINEAR
ROPE_SCALE_BASE = 2       # W4_ROPE_SCALE_BASE
ROPE_SCALE_PARTS = 3      # W4_ROPE_SCALE_PARTS
KV_BF16 = 0               # W4_KV_BF16
KV_INT8 = 1               # W4_KV_INT8
KV_INT4 = 2               # W4_KV_INT4
KV_ERR_POSITION = 1       # W4_KV_ERR_POSITION
KV_ERR_PAGE = 2           # W4_KV_ERR_PAGE
KV_ERR_SEQUENCE = 4       # W4_KV_ERR_SEQUENCE
KV_ERR_LENGTH = 8         # W4_KV_ERR_LENGTH
KV_ERR_WAIT = 16          # W4_KV_ERR_WAIT
KV_ERR_BLOCK = 32         # W4_KV_ERR_BLOCK
RECORD_TOKENS = 16        # tokens of a cache record; page sizes are multiples of it

_I64 = ctypes.c_int64


# w4_heads, w4_rotation and w4_block_table as bytes: these calls are a few
# microseconds long, and ctypes structures would cost a good part of that.
_pack_heads = struct.Struct("=Qqq").pack
_pack_rotation = struct.Struct("=Qiii4x").pack
_pack_table = struct.Struct("=Qiiq").pack


class _RopeSpec(ctypes.Structure):
    _fields_ = [("rotary_dim", _I), ("scaling", _I), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("original_context", ctypes.c_double),
                ("low_turns", ctypes.c_double), ("high_turns", ctypes.c_double),
                ("amplitude", ctypes.c_double)]


class _KvCache(ctypes.Structure):
    _fields_ = [("pool", _P), ("format", _I), ("kv_heads", _I), ("head_dim", _I),
                ("page_tokens", _I), ("pages", _I), ("error", _P)]


_rope_table = _decl("w4_rope_table", _ST, _P, _I, _P, _P)
_rope = _decl("w4_rope", _ST, _P, _P, _I, _I, _I, _P, _P, _P, _P)
_kv_pool_bytes = _decl("w4_kv_pool_bytes", _ST, _P, ctypes.POINTER(ctypes.c_size_t))
_kv_append = _decl("w4_kv_append", _ST, _P, _P, _P, _P, _P, _I, _I, _P, _P, _P, _P, _P)
_kv_read = _decl("w4_kv_read", _ST, _P, _P, _P, _I, _P, _P, _P, _P)
_paged_attn_workspace_bytes = _decl("w4_paged_attn_workspace_bytes", _ST, _P,
                                    ctypes.POINTER(ctypes.c_size_t))
_ATTN_ARGS = (_P, _P, _P, _I, _I, _P, _P, ctypes.c_float, _I, _P, _P, ctypes.c_size_t, _P)
_paged_attn = _decl("w4_paged_attn", _ST, *_ATTN_ARGS)
_paged_attn_f32 = _decl("w4_paged_attn_f32", _ST, *_ATTN_ARGS)
_SPARSE_ARGS = (_P, _P, _P, _I, _I, _P, _P, _P, _P, _I, ctypes.c_float, _P, _P, ctypes.c_size_t,
                _P)
_sparse_attn = _decl("w4_sparse_attn", _ST, *_SPARSE_ARGS)
_sparse_attn_f32 = _decl("w4_sparse_attn_f32", _ST, *_SPARSE_ARGS)
_key_bounds = _decl("w4_key_bounds", _ST, _P, _P, _I, _P, _P, _P)
_block_scores = _decl("w4_block_scores", _ST, _P, _P, _P, _I, _I, _P, _P, _P, _I, _P)
_select = _decl("w4_select", _ST, _P, _I, _I, _I, _P, _I, _I, _I, _I, _P, _P, _P)
_attn_weights = _decl("w4_attn_weights", _ST, _P, _P, _P, _I, _I, _P, _P, ctypes.c_float, _I, _P,
                      ctypes.c_float, _P, _I, _P)
_kv_gather = _decl("w4_kv_gather", _ST, _P, _P, _P, _P, _P, _I, _P, _P, _I, _P, _I, _P)


def _heads(t, dtype=torch.bfloat16) -> bytes | None:
    """[tokens, heads, head_dim] with a contiguous last dimension, as w4_heads."""
    if t is None:
        return None
    if t.dtype is not dtype or t.dim() != 3 or not t.is_cuda:
        raise ValueError(f"expected a {dtype} CUDA tensor [tokens, heads, head_dim]")
    st, sh, sd = t.stride()
    if sd != 1 and t.shape[2] > 1:
        raise ValueError("the last dimension must be contiguous")
    return _pack_heads(t.data_ptr(), st, sh)


def _int32(t, n: int, what: str) -> int | None:
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.numel() != n or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what}: expected {n} contiguous int32 values on the device")
    return t.data_ptr()


def _block_table(t) -> bytes:
    if t.dtype is torch.int32 and t.dim() == 2 and t.is_cuda:
        seqs, width = t.shape
        row, column = t.stride()
        if row < width and seqs == 1:
            row = width                     # of one row: any stride will do
        if column == 1 and row >= width:
            return _pack_table(t.data_ptr(), seqs, width, row)
    raise ValueError("block table: expected a CUDA int32 tensor [seqs, pages] whose rows do not "
                     "overlap (an expanded one has to be made contiguous)")


_capturing = torch._C._cuda_isCurrentStreamCapturing


def _raw_stream(stream, like) -> int:
    """As _stream, without making a Stream object for the current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(like.get_device())
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


_no_stream = contextlib.nullcontext()


def _on(stream, device):
    """The context in which a call on `stream` makes what it makes by itself:
    torch hands out memory, and fills it, by the current stream's order."""
    if stream is None:
        return _no_stream
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else \
            torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def rope_table(spec: dict, rows: int, table, stream=None) -> None:
    """w4_rope_table: fill `table`, float32 [rows, rotary_dim/2, 2] on the
    device.  spec: the fields of w4_rope_spec (missing ones: no scaling,
    factor 1, amplitude 1)."""
    full = dict(scaling=ROPE_SCALE_NONE, factor=1.0, original_context=0.0, low_turns=0.0,
                high_turns=0.0, amplitude=1.0)
    full.update(spec)
    s = _RopeSpec(**full)
    if table.dtype != torch.float32 or table.numel() != rows * s.rotary_dim:
        raise ValueError("table: expected float32 [rows, rotary_dim/2, 2]")
    _ok(_rope_table(ctypes.byref(s), rows, _ptr(table), _stream(stream, table)),
        "w4_rope_table")


def rope(x, y, positions, rotation: "RopeTable", error=None, stream=None) -> None:
    """w4_rope: y[t, h] = x[t, h] rotated by row positions[t] of the table
    (y may be x; a negative position rotates back)."""
    T, H, D = x.shape
    if y.shape != x.shape:
        raise ValueError("y: expected the shape of x")
    _ok(_rope(_heads(x), _heads(y), T, H, D, _int32(positions, T, "positions"), rotation.packed,
              _ptr(error), _raw_stream(stream, x)), "w4_rope")


def kv_pool_bytes(fmt: int, kv_heads: int, head_dim: int, page_tokens: int, pages: int) -> int:
    """Bytes of a paged cache's pool."""
    c, n = _KvCache(None, fmt, kv_heads, head_dim, page_tokens, pages, None), ctypes.c_size_t()
    _ok(_kv_pool_bytes(ctypes.byref(c), ctypes.byref(n)), "w4_kv_pool_bytes")
    return n.value


def kv_append(cache: "PagedCache", k, v, positions, table, seq_ids=None, q=None, q_out=None,
              rotation: "RopeTable | None" = None, stream=None) -> None:
    """w4_kv_append: write tokens into the cache, rotating k and q (into q_out;
    without a rotation q is copied there)."""
    shape = k.shape
    if v.shape != shape or shape[1:] != cache.head_shape:
        raise ValueError(f"k, v: expected [tokens, {cache.kv_heads}, {cache.head_dim}]")
    T, q_heads = shape[0], 0
    if q is not None:
        q_shape = q.shape
        if len(q_shape) != 3 or q_shape[0] != T or q_shape[2] != cache.head_dim or \
                q_out is None or q_out.shape != q_shape:
            raise ValueError("q, q_out: expected [tokens, q_heads, head_dim]")
        q_heads = q_shape[1]
    _ok(_kv_append(cache.ref, _heads(k), _heads(v), _heads(q), _heads(q_out), q_heads, T,
                   _int32(positions, T, "positions"), _int32(seq_ids, T, "seq_ids"),
                   _block_table(table), rotation and rotation.packed, _raw_stream(stream, k)),
        "w4_kv_append")


def kv_read(cache: "PagedCache", k_out, v_out, positions, table, seq_ids=None,
            stream=None) -> None:
    """w4_kv_read: the cached keys and values of the listed tokens, bfloat16."""
    T = positions.numel()
    shape = (T, *cache.head_shape)
    for x in (k_out, v_out):
        if x is not None and x.shape != shape:
            raise ValueError("k_out, v_out: expected [tokens, kv_heads, head_dim]")
    _ok(_kv_read(cache.ref, _heads(k_out), _heads(v_out), T,
                 _int32(positions, T, "positions"), _int32(seq_ids, T, "seq_ids"),
                 _block_table(table), _raw_stream(stream, positions)), "w4_kv_read")


def paged_attn_workspace_bytes(cache: "PagedCache") -> int:
    """Bytes of workspace that paged_attn needs on the current device."""
    n = ctypes.c_size_t()
    _ok(_paged_attn_workspace_bytes(cache.ref, ctypes.byref(n)), "w4_paged_attn_workspace_bytes")
    return n.value


def _attn(fn, where, dtype, cache, q, out, lens, table, scale, window, lse, workspace, stream):
    # window: what the call has between scale and lse, or (blocks, counts) ahead of scale;
    # workspace: its address and bytes; stream: a raw one
    shape = q.shape
    T, H, D = shape
    B = table.shape[0]
    if not B or T % B or D != cache.head_dim or out.shape != shape:
        raise ValueError("q, out: expected [seqs * tokens, q_heads, head_dim]")
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.numel() != T * H:
            raise ValueError("lse: expected float32 [seqs * tokens, q_heads]")
        lse = _ptr(lse)
    scale = D ** -0.5 if scale is None else scale
    if type(window) is tuple:
        blocks, counts = window
        most = blocks.shape[-1]
        middle = (_filled(blocks, (B, cache.kv_heads, most), torch.int32, "blocks"),
                  _int32(counts, B, "counts"), most, scale)
    else:
        middle = (scale, window)
    _ok(fn(cache.ref, _heads(q), _heads(out, dtype), H, T // B, _int32(lens, B, "lens"),
           _block_table(table), *middle, lse, *workspace, stream), where)


def paged_attn(cache: "PagedCache", q, out, lens, table, workspace, scale=None, window: int = 0,
               lse=None, stream=None) -> None:
    """w4_paged_attn: out[b * tokens + i] (bfloat16) = attention of the new
    token i of sequence b over its cached tokens."""
    _attn(_paged_attn, "w4_paged_attn", torch.bfloat16, cache, q, out, lens, table, scale,
          window, lse, (_ptr(workspace), workspace.nbytes), _raw_stream(stream, q))


def paged_attn_f32(cache: "PagedCache", q, out, lens, table, workspace, scale=None,
                   window: int = 0, lse=None, stream=None) -> None:
    """w4_paged_attn_f32: as paged_attn, fp32 result."""
    _attn(_paged_attn_f32, "w4_paged_attn_f32", torch.float32, cache, q, out, lens, table, scale,
          window, lse, (_ptr(workspace), workspace.nbytes), _raw_stream(stream, q))


def sparse_attn(cache: "PagedCache", q, out, lens, table, blocks, counts, workspace, scale=None,
                lse=None, stream=None) -> None:
    """w4_sparse_attn: as paged_attn, over the blocks that blocks[b, h, :counts[b]]
    (int32 [seqs, kv_heads, most], ascending) lists for every key/value head."""
    _attn(_sparse_attn, "w4_sparse_attn", torch.bfloat16, cache, q, out, lens, table, scale,
          (blocks, counts), lse, (_ptr(workspace), workspace.nbytes), _raw_stream(stream, q))


def sparse_attn_f32(cache: "PagedCache", q, out, lens, table, blocks, counts, workspace,
                    scale=None, lse=None, stream=None) -> None:
    """w4_sparse_attn_f32: as sparse_attn, fp32 result."""
    _attn(_sparse_attn_f32, "w4_sparse_attn_f32", torch.float32, cache, q, out, lens, table,
          scale, (blocks, counts), lse, (_ptr(workspace), workspace.nbytes),
          _raw_stream(stream, q))


def _filled(t, shape, dtype, what: str) -> int:
    """Address of a contiguous CUDA tensor of this shape (a tuple) and type."""
    if t.shape != shape or t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous {dtype} CUDA tensor {list(shape)}")
    return t.data_ptr()


def _new_tokens(cache: "PagedCache", q, B: int) -> tuple:
    """(rows, q_heads, new tokens of a sequence) of the queries of a call."""
    T, H, D = q.shape
    if not B or T % B or D != cache.head_dim:
        raise ValueError("q: expected [seqs * tokens, q_heads, head_dim]")
    return T, H, T // B


def key_bounds(cache: "PagedCache", bounds, lens, table, tokens: int = 1, stream=None) -> None:
    """w4_key_bounds: the largest and the smallest key values, bfloat16 [pages,
    kv_heads, 2, head_dim], of the blocks that the last `tokens` tokens of every
    sequence lie in."""
    _ok(_key_bounds(cache.ref, _filled(bounds, cache.bounds_shape, torch.bfloat16, "bounds"),
                    tokens, _int32(lens, table.shape[0], "lens"), _block_table(table),
                    _raw_stream(stream, bounds)), "w4_key_bounds")


def block_scores(cache: "PagedCache", bounds, q, lens, table, scores, stream=None) -> None:
    """w4_block_scores: how large q . k can be in every block of a sequence,
    float32 [seqs, kv_heads, columns]."""
    B, columns = table.shape[0], scores.shape[-1]
    _, H, M = _new_tokens(cache, q, B)
    _ok(_block_scores(cache.ref, _filled(bounds, cache.bounds_shape, torch.bfloat16, "bounds"),
                      _heads(q), H, M, _int32(lens, B, "lens"), _block_table(table),
                      _filled(scores, (B, cache.kv_heads, columns), torch.float32, "scores"),
                      columns, _raw_stream(stream, q)), "w4_block_scores")


def select(scores, lens, index, counts, unit: int = 1, first: int = 0, last: int = 0,
           stream=None) -> None:
    """w4_select: of the ceil(lens[b] / unit) items of every row of scores, float32
    [seqs, heads, columns], the first `first`, the last `last` and the best others,
    as many as a row of index has (int32 [seqs, heads, count]), ascending; how many
    there are goes into counts, int32 [seqs]."""
    shape = scores.shape
    if len(shape) != 3:
        raise ValueError("scores: expected float32 [seqs, heads, columns]")
    B, H, columns = shape
    count = index.shape[-1]
    _ok(_select(_filled(scores, shape, torch.float32, "scores"), B, H, columns,
                _int32(lens, B, "lens"), unit, first, last, count,
                _filled(index, (B, H, count), torch.int32, "index"),
                _int32(counts, B, "counts"), _raw_stream(stream, scores)), "w4_select")


def attn_weights(cache: "PagedCache", q, lse, lens, table, weights, before=None,
                 decay: float = 1.0, scale=None, window: int = 0, stream=None) -> None:
    """w4_attn_weights: weights, float32 [seqs, kv_heads, columns], = decay * before (may
    be weights; None: 0) + what every cached token gets of the new tokens' attention,
    whose log-sum-exp is lse, float32 [seqs * tokens, q_heads]."""
    B, columns = table.shape[0], weights.shape[-1]
    T, H, M = _new_tokens(cache, q, B)
    expected = (B, cache.kv_heads, columns)
    _ok(_attn_weights(cache.ref, _heads(q), _filled(lse, (T, H), torch.float32, "lse"), H, M,
                      _int32(lens, B, "lens"), _block_table(table),
                      q.shape[2] ** -0.5 if scale is None else scale, window,
                      before if before is None else
                      _filled(before, expected, torch.float32, "before"), decay,
                      _filled(weights, expected, torch.float32, "weights"), columns,
                      _raw_stream(stream, q)), "w4_attn_weights")


def kv_gather(cache: "PagedCache", table, lens, index, counts, to, weights=None,
              weights_out=None, stream=None) -> None:
    """w4_kv_gather: place i of sequence b in the pages of `to` gets token index[b, h, i]
    of those of `table`, for i < counts[b] and every key/value head h (index int32
    [seqs, kv_heads, most]); weights_out[b, h, i] (float32 [seqs, kv_heads, most or more])
    its entry of weights (float32 [seqs, kv_heads, columns])."""
    B, H = table.shape[0], cache.kv_heads
    most, columns, columns_out = index.shape[-1], 0, 0
    if (weights is None) != (weights_out is None):
        raise ValueError("weights, weights_out: expected both or neither")
    if weights is not None:
        columns, columns_out = weights.shape[-1], weights_out.shape[-1]
        weights = _filled(weights, (B, H, columns), torch.float32, "weights")
        weights_out = _filled(weights_out, (B, H, columns_out), torch.float32, "weights_out")
    _ok(_kv_gather(cache.ref, _block_table(table), _int32(lens, B, "lens"),
                   _filled(index, (B, H, most), torch.int32, "index"),
                   _int32(counts, B, "counts"), most, _block_table(to), weights, columns,
                   weights_out, columns_out, _raw_stream(stream, index)), "w4_kv_gather")


class RopeTable:
    """A table of rotations: float32 [rows, rotary_dim/2, 2] (cos, sin) pairs
    on the device, and which values of a head form a pair."""

    def __init__(self, table: torch.Tensor, layout: int = ROPE_HALF):
        if table.dim() != 3 or table.shape[2] != 2 or table.dtype != torch.float32:
            raise ValueError("table: expected float32 [rows, rotary_dim/2, 2]")
        self.table, self.layout = table, layout
        self.packed = _pack_rotation(_ptr(table), table.shape[0], 2 * table.shape[1], layout)

    @classmethod
    def make(cls, rows: int, rotary_dim: int, base: float, layout: int = ROPE_HALF, device=None,
             stream=None, **scaling) -> "RopeTable":
        """A table filled by w4_rope_table; scaling: scaling, factor,
        original_context, low_turns, high_turns, amplitude of w4_rope_spec."""
        device = torch.device("cuda" if device is None else device)
        with _on(stream, device):
            t = torch.empty((rows, rotary_dim // 2, 2), dtype=torch.float32, device=device)
        rope_table(dict(rotary_dim=rotary_dim, base=base, **scaling), rows, t, stream)
        return cls(t, layout)

    def apply(self, x: torch.Tensor, positions: torch.Tensor, out: torch.Tensor | None = None,
              error: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """x [tokens, heads, head_dim] bfloat16, rotated; out may be x (default:
        a new tensor, made on `stream`)."""
        if out is None:
            with _on(stream, x.device):
                out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        rope(x, out, positions, self, error, stream)
        return out


class PagedCache:
    """A paged key-value cache over a caller's pool (a contiguous CUDA tensor
    of kv_pool_bytes() bytes).  Its calls record what is out of range in
    `error` (one int32 on the device; see check()).  The error word, and make()'s
    pool, are filled on torch's current stream; what a later call makes by itself
    is made on the stream of that call.  attend() uses a workspace that the cache
    keeps for the stream (see `workspace`), under graph capture one of the
    graph's own, unless it is given one: calls that overlap on the device need
    one each."""

    def __init__(self, pool: torch.Tensor, fmt: int, kv_heads: int, head_dim: int,
                 page_tokens: int = RECORD_TOKENS, error: torch.Tensor | None = None):
        per_page = kv_pool_bytes(fmt, kv_heads, head_dim, page_tokens, 1)
        nbytes = pool.numel() * pool.element_size()
        if nbytes == 0 or nbytes % per_page:
            raise ValueError(f"pool: expected a multiple of {per_page} bytes")
        self.pool, self.format = pool, fmt
        self.kv_heads, self.head_dim, self.page_tokens = kv_heads, head_dim, page_tokens
        self.head_shape = (kv_heads, head_dim)
        self.pages = nbytes // per_page
        self.bounds_shape = (self.pages, kv_heads, 2, head_dim)
        self.error = torch.zeros(1, dtype=torch.int32, device=pool.device) if error is None \
            else error
        self._struct = _KvCache(_ptr(pool), fmt, kv_heads, head_dim, page_tokens, self.pages,
                                _ptr(self.error))
        self.ref = ctypes.byref(self._struct)
        self._workspaces = {}              # by raw stream: (address, bytes), tensor

    @classmethod
    def make(cls, pages: int, fmt: int, kv_heads: int, head_dim: int,
             page_tokens: int = RECORD_TOKENS, device=None) -> "PagedCache":
        """A cache with a pool of its own (allocated by torch, zero-filled)."""
        n = kv_pool_bytes(fmt, kv_heads, head_dim, page_tokens, pages)
        return cls(torch.zeros(n, dtype=torch.uint8,
                               device=device if device is not None else "cuda"),
                   fmt, kv_heads, head_dim, page_tokens)

    def append(self, k, v, positions, table, seq_ids=None, q=None, q_out=None, rope=None,
               stream=None) -> None:
        """Write tokens into the cache: k, and q into q_out, rotated by `rope`
        (without one as they are), v as it is."""
        kv_append(self, k, v, positions, table, seq_ids, q, q_out, rope, stream)

    def read(self, positions, table, seq_ids=None, k=None, v=None, stream=None):
        """The cached keys and values of the listed tokens (default outputs: new
        tensors, made on `stream`, zero where a token is left out)."""
        shape = (positions.numel(), self.kv_heads, self.head_dim)
        if k is None or v is None:
            with _on(stream, self.pool.device):
                if k is None:
                    k = torch.zeros(shape, dtype=torch.bfloat16, device=self.pool.device)
                if v is None:
                    v = torch.zeros(shape, dtype=torch.bfloat16, device=self.pool.device)
        kv_read(self, k, v, positions, table, seq_ids, stream)
        return k, v

    def new_workspace(self) -> torch.Tensor:
        """A workspace for attend()."""
        return torch.empty(paged_attn_workspace_bytes(self), dtype=torch.uint8,
                           device=self.pool.device)

    @property
    def workspace(self) -> torch.Tensor | None:
        """The workspace of attend() on torch's current stream: the one that it
        has made, or that was set here."""
        kept = self._workspaces.get(_raw_stream(None, self.pool))
        return kept and kept[1]

    @workspace.setter
    def workspace(self, ws: torch.Tensor | None) -> None:
        if ws is None:
            self._workspaces.pop(_raw_stream(None, self.pool), None)
        else:
            self._workspaces[_raw_stream(None, self.pool)] = (_ptr(ws), ws.nbytes), ws

    def _workspace_on(self, stream):
        """A workspace that no call on another stream uses, as in _workspaces.  A
        captured call's is the graph's: an eager one may run beside a replay, and
        memory that was made under capture is not for others."""
        with _on(stream, self.pool.device):
            capturing = _capturing()
            raw = _raw_stream(stream, self.pool)
            kept = None if capturing else self._workspaces.get(raw)
            if kept is None:
                ws = self.new_workspace()
                kept = (_ptr(ws), ws.nbytes), ws
                if not capturing:
                    self._workspaces[raw] = kept
            return kept

    def attend(self, q, lens, table, scale=None, window: int = 0, out=None, lse=None,
               workspace=None, stream=None):
        """Attention of the new tokens; returns (out bfloat16, lse float32), by
        default new tensors, made on `stream`."""
        return self._attend(_paged_attn, "w4_paged_attn", q, lens, table, scale, window, out, lse,
                            workspace, stream)

    def attend_blocks(self, q, lens, table, blocks, counts, scale=None, out=None, lse=None,
                      workspace=None, stream=None):
        """Attention of the new tokens over the blocks blocks[b, h, :counts[b]] (ascending,
        int32 [seqs, kv_heads, most]) alone; as attend() otherwise."""
        return self._attend(_sparse_attn, "w4_sparse_attn", q, lens, table, scale,
                            (blocks, counts), out, lse, workspace, stream)

    def _attend(self, fn, where, q, lens, table, scale, window, out, lse, workspace, stream):
        raw, kept = _raw_stream(stream, q), None
        if workspace is not None:
            kept = (_ptr(workspace), workspace.nbytes), workspace
        elif stream is None and not _capturing():
            kept = self._workspaces.get(raw)
        if kept is None:
            kept = self._workspace_on(stream)
        if out is None or lse is None:
            with _on(stream, q.device):
                if out is None:
                    out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
                if lse is None:
                    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        _attn(fn, where, torch.bfloat16, self, q, out, lens, table, scale, window, lse, kept[0],
              raw)
        return out, lse

    def new_bounds(self) -> torch.Tensor:
        """Bounds of the keys of all pages, for key_bounds() to fill (made on torch's
        current stream)."""
        return torch.zeros(self.bounds_shape, dtype=torch.bfloat16, device=self.pool.device)

    def key_bounds(self, bounds, lens, table, tokens: int = 1, stream=None) -> torch.Tensor:
        """Bring `bounds` (see new_bounds) up to date for the blocks that the last
        `tokens` tokens of every sequence lie in."""
        key_bounds(self, bounds, lens, table, tokens, stream)
        return bounds

    def block_scores(self, bounds, q, lens, table, scores=None, stream=None) -> torch.Tensor:
        """How large q . k can be in every block; [seqs, kv_heads, width] (default: a
        new tensor, made on `stream`; -inf past a sequence's blocks)."""
        if scores is None:
            with _on(stream, q.device):
                scores = torch.full((table.shape[0], self.kv_heads, table.shape[1]), -math.inf,
                                    dtype=torch.float32, device=q.device)
        block_scores(self, bounds, q, lens, table, scores, stream)
        return scores

    def attn_weights(self, q, lse, lens, table, scale=None, window: int = 0, before=None,
                     decay: float = 1.0, weights=None, columns: int | None = None,
                     stream=None) -> torch.Tensor:
        """decay * before + what every cached token gets of the new tokens' attention, by
        key/value head; q, lens, table, scale and window as attend() had them, lse as it
        returned it.  before may be weights.  [seqs, kv_heads, columns] (default: a new
        tensor, made on `stream`, with before's columns, or room for all of a table's
        tokens; 0 past a sequence's tokens)."""
        if weights is None:
            if columns is None:
                columns = table.shape[1] * self.page_tokens if before is None else before.shape[2]
            with _on(stream, q.device):
                weights = torch.zeros((table.shape[0], self.kv_heads, columns),
                                      dtype=torch.float32, device=q.device)
        attn_weights(self, q, lse, lens, table, weights, before, decay, scale, window, stream)
        return weights

    def gather(self, table, lens, index, counts, to, weights=None, weights_out=None,
               stream=None):
        """Move listed tokens to other pages: place i of sequence b in `to` gets token
        index[b, h, i] in `table`, for i < counts[b] and every head; returns weights_out, the
        tokens' weights (default, where weights are given: a new tensor of their shape,
        or as wide as the list where that is wider, made on `stream`, 0 past the counts)."""
        if weights is not None and weights_out is None:
            columns = max(weights.shape[-1], index.shape[-1])
            with _on(stream, index.device):
                weights_out = torch.zeros((*index.shape[:2], columns), dtype=torch.float32,
                                          device=index.device)
        kv_gather(self, table, lens, index, counts, to, weights, weights_out, stream)
        return weights_out

    def check(self) -> None:
        """Raise W4Error if a call recorded an error, and clear it.  Waits for
        the device: the calls may have been on any stream."""
        torch.cuda.synchronize(self.error.device)
        bits = int(self.error.item())
        if bits:
            self.error.zero_()
            torch.cuda.synchronize(self.error.device)
            raise W4Error(Status.INVALID_ARG, f"paged cache (error word {bits})")
