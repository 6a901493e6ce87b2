"""GB300-native tensor-parallel row-parallel linear epilogue.

Thin Python binding of ``libare.so`` (C ABI in ``include/are.h``): argument
marshalling only.  Every step of the computation runs in the library's CUDA
kernels; PyTorch supplies device memory and streams.  There is no CPU path:
calling any operation without the built library raises ``AreLibraryMissing``.

Operations (the same names as the C ABI, without the ``are_`` prefix):

* ``gemm_rs(A, B, out, ws)``      R partial GEMMs, ring-order fp32 sum,
  reduce-scattered into R owner row segments (bf16).
* ``gemm_ar(A, B, out, ws)``      R partial GEMMs rounded to bf16, all-reduced
  into every rank view.
* ``allreduce_rmsnorm(partials, residual, gamma, eps, out, ws)``
  all-reduce + residual + RMSNorm in one Lamport-synchronised kernel.
* ``allreduce_rmsnorm_quant_groups(partials, residual, gamma, eps, out_q,
  out_scale, ws, group)``  the same with FP8 codes and a scale per group of
  columns.
* ``allreduce_rmsnorm_backward(dy, h, gamma, eps, dh, dgamma, ws)``  its
  backward pass.
* ``allreduce_layernorm(partials, residual, gamma, beta, eps, out, ws)`` and
  ``allreduce_layernorm_backward(dy, h, gamma, eps, dh, dgamma, dbeta, ws)``  the
  same pair with LayerNorm.
* ``embedding_ar(ids, tables, out, ws)`` and ``embedding_ar_backward(ids, dy,
  dtables, ws)``  lookup in a table split over the ranks, and its gradient by
  sorted tokens.
* ``gemm_cross_entropy(h, w, targets, loss, lse, ws)`` and
  ``gemm_cross_entropy_backward(h, w, targets, lse, dloss, dh, dw, ws)``  softmax
  cross entropy of an output layer split over the ranks, without its logits, and
  its gradients.
* ``gemm_ar_qweight(x, w, out, ws)``, ``gemm_ar_qweight_qx(xq, xscale, w, out,
  ws)``  the row-parallel linear of a few tokens with 4-bit weights
  (``QWeight``), all-reduced; tokens in bf16 or in FP8 codes with scales.
"""
from __future__ import annotations

import ctypes
import os
from array import array
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libare.so")

# status codes (are_status)
OK, EINVAL, ENOMEM, ECUDA, ETIMEOUT, EBUSY, ENODEV, ECAPACITY, ECAPTURE = range(9)
# ops
OP_GEMM_RS, OP_GEMM_AR, OP_ALLREDUCE_RMSNORM = 1, 2, 3
OP_ALLREDUCE_RMSNORM_BACKWARD, OP_GEMM_AR_QWEIGHT = 4, 5
OP_ALLREDUCE_LAYERNORM, OP_ALLREDUCE_LAYERNORM_BACKWARD = 6, 7
OP_GEMM_CROSS_ENTROPY, OP_EMBEDDING_AR, OP_EMBEDDING_AR_BACKWARD = 8, 9, 10
# index formats (are_index_format)
INDEX_I32, INDEX_I64 = 0, 1
# scale formats (are_scale_format)
SCALE_F32, SCALE_E8M0 = 0, 1
# debug flags
DEBUG_NO_REARM, DEBUG_LOG_PIECES, DEBUG_COUNT_CANON, DEBUG_SKIP_PUBLISH, DEBUG_SKIP_STAGE = 1, 2, 4, 8, 16
DEBUG_SINGLE_CTA, DEBUG_WAIT_PROFILE, DEBUG_AR_ONESHOT, DEBUG_AR_LAMPORT, DEBUG_PAIR_CTA = 32, 64, 128, 256, 512
DEBUG_RS_RING, DEBUG_RS_SPLIT, DEBUG_QWEIGHT_FEW, DEBUG_QWEIGHT_STAGED = 1024, 2048, 4096, 8192
# device status codes
DEV_OK, DEV_MASK_TIMEOUT, DEV_STAGE_TIMEOUT, DEV_PIPE_TIMEOUT = 0, 1, 2, 3
# snapshot kinds
SNAP_MASKS, SNAP_STAGING, SNAP_PIECES, SNAP_COUNTERS, SNAP_CHUNKS = 1, 2, 3, 4, 5
CHUNK_CAP = 64          # chunk counters per owner segment in the workspace
CHUNK_Q = 1 << 32       # counter advance per completed chunk
# kernels (are_kernel), as reported by Workspace.last_launch()
KERNEL_NAMES = {0: "none", 1: "memset", 2: "gemm_reduce_kernel", 3: "gemm_pair_kernel", 4: "ar_rmsnorm_kernel",
                5: "ar_oneshot_kernel", 6: "norm_quant_rows_kernel", 7: "norm_backward_rows_kernel",
                8: "qweight_kernel", 9: "layernorm_rows_kernel", 10: "layernorm_backward_rows_kernel",
                11: "xent_kernel<LogSum>", 12: "xent_kernel<DLogits>", 13: "embed_kernel", 14: "embed_sort_kernel",
                15: "embed_few_kernel", 16: "layernorm_narrow_kernel",
                17: "layernorm_backward_narrow_kernel"}
PIECE_WORDS = 64
TILE_M, TILE_N = 128, 256

# Every C-ABI symbol declared in include/are.h.
EXPORTS = [
    "are_version", "are_status_string", "are_supports", "are_workspace_create", "are_workspace_destroy",
    "are_workspace_reset", "are_workspace_set_debug", "are_workspace_set_oneshot_max_bytes",
    "are_workspace_set_gemm_order", "are_workspace_set_chunks", "are_chunk_generation", "are_chunk_wait",
    "are_workspace_set_vocab_piece", "are_workspace_set_logit_gradient",
    "are_get_device_status", "are_debug_snapshot", "are_debug_last_launch",
    "are_gemm_rs", "are_gemm_ar", "are_allreduce_rmsnorm", "are_allreduce_add_rmsnorm", "are_allreduce_rmsnorm_quant",
    "are_allreduce_rmsnorm_noalloc", "are_noalloc_device_status",
    "are_allreduce_rmsnorm_quant_groups", "are_allreduce_rmsnorm_backward", "are_gemm_ar_qweight",
    "are_gemm_ar_qweight_qx", "are_allreduce_layernorm", "are_allreduce_layernorm_backward",
    "are_gemm_cross_entropy", "are_gemm_cross_entropy_backward",
    "are_embedding_ar", "are_embedding_ar_backward",
]


class AreError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


class AreLibraryMissing(RuntimeError):
    pass


class _Caps(ctypes.Structure):
    _fields_ = [("R_max", ctypes.c_int32), ("M_max", ctypes.c_int64), ("N_max", ctypes.c_int64),
                ("K_max", ctypes.c_int64), ("timeout_ns", ctypes.c_uint64), ("debug_flags", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class _DevStatus(ctypes.Structure):
    _fields_ = [("code", ctypes.c_uint32), ("where", ctypes.c_uint32), ("a", ctypes.c_int32), ("b", ctypes.c_int32)]


class _LaunchInfo(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("grid", ctypes.c_int32), ("block", ctypes.c_int32),
                ("cluster", ctypes.c_int32), ("rank_block", ctypes.c_int32), ("variant", ctypes.c_int32),
                ("rank_group", ctypes.c_int32), ("group_m", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load ``libare.so`` (idempotent).  Raises AreLibraryMissing if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise AreLibraryMissing(
            f"{path} is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    vp, i32, i64, u32, u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint32, ctypes.c_uint64
    lib.are_version.restype = i32
    lib.are_status_string.restype = ctypes.c_char_p
    lib.are_status_string.argtypes = [i32]
    lib.are_supports.restype = i32
    lib.are_supports.argtypes = [i32, i32, i64, i64, i64]
    lib.are_workspace_create.restype = i32
    lib.are_workspace_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(_Caps)]
    lib.are_workspace_destroy.restype = i32
    lib.are_workspace_destroy.argtypes = [vp]
    lib.are_workspace_reset.restype = i32
    lib.are_workspace_reset.argtypes = [vp]
    lib.are_workspace_set_debug.restype = i32
    lib.are_workspace_set_debug.argtypes = [vp, u32, i64]
    lib.are_workspace_set_oneshot_max_bytes.restype = i32
    lib.are_workspace_set_oneshot_max_bytes.argtypes = [vp, u64]
    lib.are_workspace_set_gemm_order.restype = i32
    lib.are_workspace_set_gemm_order.argtypes = [vp, i32, i32, i32]
    lib.are_workspace_set_vocab_piece.restype = i32
    lib.are_workspace_set_vocab_piece.argtypes = [vp, i64]
    lib.are_workspace_set_logit_gradient.restype = i32
    lib.are_workspace_set_logit_gradient.argtypes = [vp, i32]
    lib.are_workspace_set_chunks.restype = i32
    lib.are_workspace_set_chunks.argtypes = [vp, i32, i32]
    lib.are_chunk_generation.restype = i32
    lib.are_chunk_generation.argtypes = [vp, ctypes.POINTER(u64)]
    lib.are_chunk_wait.restype = i32
    lib.are_chunk_wait.argtypes = [vp, i32, i32, u64, u64]
    lib.are_get_device_status.restype = i32
    lib.are_get_device_status.argtypes = [vp, ctypes.POINTER(_DevStatus)]
    lib.are_debug_snapshot.restype = i32
    lib.are_debug_snapshot.argtypes = [vp, i32, vp, ctypes.c_size_t]
    lib.are_debug_last_launch.restype = i32
    lib.are_debug_last_launch.argtypes = [vp, ctypes.POINTER(_LaunchInfo)]
    lib.are_noalloc_device_status.restype = i32
    lib.are_noalloc_device_status.argtypes = [ctypes.POINTER(_DevStatus)]
    for name in ("are_gemm_rs", "are_gemm_ar"):
        f = getattr(lib, name)
        f.restype = i32
        f.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp, vp]
    lib.are_allreduce_rmsnorm.restype = i32
    lib.are_allreduce_rmsnorm.argtypes = [vp, vp, vp, ctypes.c_float, vp, i32, i64, i64, vp, vp]
    lib.are_allreduce_add_rmsnorm.restype = i32
    lib.are_allreduce_add_rmsnorm.argtypes = [vp, vp, vp, ctypes.c_float, vp, vp, i32, i64, i64, vp, vp]
    lib.are_allreduce_rmsnorm_quant.restype = i32
    lib.are_allreduce_rmsnorm_quant.argtypes = [vp, vp, vp, ctypes.c_float, vp, vp, vp, i32, i64, i64, vp, vp]
    lib.are_allreduce_rmsnorm_noalloc.restype = i32
    lib.are_allreduce_rmsnorm_noalloc.argtypes = [vp, vp, vp, ctypes.c_float, vp, i32, i64, i64, vp]
    f32 = ctypes.c_float
    lib.are_allreduce_rmsnorm_quant_groups.restype = i32
    lib.are_allreduce_rmsnorm_quant_groups.argtypes = [vp, vp, vp, f32, i32, i32, vp, vp, vp, i32, i64, i64, vp, vp]
    lib.are_allreduce_rmsnorm_backward.restype = i32
    lib.are_allreduce_rmsnorm_backward.argtypes = [vp, vp, vp, f32, vp, vp, vp, i32, i64, i64, vp, vp]
    lib.are_gemm_ar_qweight.restype = i32
    lib.are_gemm_ar_qweight.argtypes = [vp, vp, i32, vp, i32, i64, i64, i64, vp, vp]
    lib.are_gemm_ar_qweight_qx.restype = i32
    lib.are_gemm_ar_qweight_qx.argtypes = [vp, vp, i32, i32, vp, i32, vp, i32, i64, i64, i64, vp, vp]
    lib.are_allreduce_layernorm.restype = i32
    lib.are_allreduce_layernorm.argtypes = [vp, vp, vp, vp, f32, vp, vp, i32, i64, i64, vp, vp]
    lib.are_allreduce_layernorm_backward.restype = i32
    lib.are_allreduce_layernorm_backward.argtypes = [vp, vp, vp, f32, vp, vp, vp, vp, i32, i64, i64, vp, vp]
    lib.are_gemm_cross_entropy.restype = i32
    lib.are_gemm_cross_entropy.argtypes = [vp, vp, vp, i32, i64, vp, vp, i32, i64, i64, i64, vp, vp]
    lib.are_gemm_cross_entropy_backward.restype = i32
    lib.are_gemm_cross_entropy_backward.argtypes = [vp, vp, vp, i32, i64, vp, vp, vp, vp, i32, i64, i64, i64, vp, vp]
    lib.are_embedding_ar.restype = i32
    lib.are_embedding_ar.argtypes = [vp, i32, vp, f32, vp, i32, i64, i64, i64, vp, vp]
    lib.are_embedding_ar_backward.restype = i32
    lib.are_embedding_ar_backward.argtypes = [vp, i32, vp, f32, i32, vp, i32, i64, i64, i64, vp, vp]
    _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load_library().are_status_string(status).decode()
    except AreLibraryMissing:
        return f"status {status}"


def version() -> int:
    return load_library().are_version()


def supports(op: int, R: int, M: int, N: int, K: int = 0) -> bool:
    return load_library().are_supports(op, R, M, N, K) == OK


def _check(status: int, what: str):
    if status != OK:
        raise AreError(status, what)


def _stream_handle(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _current_device() -> int:
    import torch
    return torch.cuda.current_device() if torch.cuda.is_available() else -1


def _ptrs(tensors) -> ctypes.Array:
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def _check_bf16(t, what: str):
    import torch
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA bfloat16 tensor")


class Workspace:
    """Device workspace (tile masks, partial buffer, armed staging, status word).

    Sized once from the capacities; use one workspace per stream.
    ``vocab_piece``: columns of the vocabulary whose gradient the cross entropy
    holds at a time (8192, say); 0 for a workspace without its buffers."""

    def __init__(self, R_max: int, M_max: int, N_max: int, K_max: int = 0, timeout_ns: int = 0,
                 debug_flags: int = 0, vocab_piece: int = 0):
        lib = load_library()
        caps = _Caps(R_max, M_max, N_max, K_max, timeout_ns, debug_flags, 0)
        h = ctypes.c_void_p()
        self.device_index = _current_device()
        _check(lib.are_workspace_create(ctypes.byref(h), ctypes.byref(caps)), "are_workspace_create")
        self._h = h
        self.caps = dict(R_max=R_max, M_max=M_max, N_max=N_max, K_max=K_max)
        if vocab_piece:
            try:
                self.set_vocab_piece(vocab_piece)
            except AreError:
                self.close()
                raise

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("workspace is closed")
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None:
            load_library().are_workspace_destroy(self._h)
            self._h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def reset(self):
        _check(load_library().are_workspace_reset(self.handle), "are_workspace_reset")

    def set_debug(self, flags: int, arg: int = -1):
        _check(load_library().are_workspace_set_debug(self.handle, flags, arg), "are_workspace_set_debug")

    def set_oneshot_max_bytes(self, nbytes: int):
        """Per-rank input size (M*N*2 bytes) up to which allreduce_rmsnorm uses
        its one-shot kernel (0: always the Lamport kernel)."""
        _check(load_library().are_workspace_set_oneshot_max_bytes(self.handle, nbytes),
               "are_workspace_set_oneshot_max_bytes")

    def device_status(self) -> dict:
        st = _DevStatus()
        rc = load_library().are_get_device_status(self.handle, ctypes.byref(st))
        if rc not in (OK, ETIMEOUT):
            raise AreError(rc, "are_get_device_status")
        return {"status": rc, "code": st.code, "where": st.where, "a": st.a, "b": st.b}

    def last_launch(self) -> dict:
        """Which kernel the last operation on this workspace launched, and its
        launch shape (host-side record; no device access)."""
        li = _LaunchInfo()
        _check(load_library().are_debug_last_launch(self.handle, ctypes.byref(li)), "are_debug_last_launch")
        return {"kernel": KERNEL_NAMES.get(li.kernel, str(li.kernel)), "grid": li.grid, "block": li.block,
                "cluster": li.cluster, "rank_block": li.rank_block, "variant": li.variant,
                "rank_group": li.rank_group, "group_m": li.group_m}

    def set_gemm_order(self, group_m: int = 0, block_pairs: int = 0, rank_group: int = 0):
        """Order of the CTA-pair GEMM kernel's work units (0 = the library's
        choice; block_pairs < 0 = a pair's R units consecutive).  Results do
        not depend on it."""
        _check(load_library().are_workspace_set_gemm_order(self.handle, group_m, block_pairs, rank_group),
               "are_workspace_set_gemm_order")

    def set_vocab_piece(self, columns: int):
        """Allocate the cross entropy's buffers, for a gradient of so many columns of
        the vocabulary at a time, in place of those that are there; 0 releases them.
        Synchronises."""
        _check(load_library().are_workspace_set_vocab_piece(self.handle, columns), "are_workspace_set_vocab_piece")

    def set_logit_gradient(self, parts: int):
        """bf16 parts of the logits' gradient in the cross entropy's backward
        products: 2 (the default), as near as fp32, or 1, rounded once to bf16, in
        half the products' time."""
        _check(load_library().are_workspace_set_logit_gradient(self.handle, parts), "are_workspace_set_logit_gradient")

    def set_chunks(self, chunks: int, stripe: int = 0):
        """GEMM+RS chunked owner-segment completion: `chunks` per segment (0 =
        off); `stripe` 0 = destination-rotated chunk-major order, > 0 = striped,
        -1 = the usual order."""
        _check(load_library().are_workspace_set_chunks(self.handle, chunks, stripe), "are_workspace_set_chunks")

    def chunk_generation(self) -> int:
        g = ctypes.c_uint64()
        _check(load_library().are_chunk_generation(self.handle, ctypes.byref(g)), "are_chunk_generation")
        return g.value

    def chunk_wait(self, segment: int, chunk: int, generation: int, timeout_ns: int = 1_000_000_000) -> bool:
        """Host-side wait for a chunk to reach `generation`; False on timeout."""
        rc = load_library().are_chunk_wait(self.handle, segment, chunk, generation, timeout_ns)
        if rc not in (OK, ETIMEOUT):
            raise AreError(rc, "are_chunk_wait")
        return rc == OK

    def chunk_counters(self):
        """[R_max, CHUNK_CAP] uint64 completion counters (synchronises)."""
        import numpy as np
        n = self.caps["R_max"] * CHUNK_CAP * 8
        return self.snapshot(SNAP_CHUNKS, n).view(np.uint64).reshape(self.caps["R_max"], CHUNK_CAP)

    def snapshot(self, kind: int, nbytes: int):
        import numpy as np
        buf = np.empty(nbytes, dtype=np.uint8)
        _check(load_library().are_debug_snapshot(self.handle, kind, buf.ctypes.data, nbytes), "are_debug_snapshot")
        return buf


def gemm_rs(A: Sequence, B: Sequence, out, ws: Workspace, stream=None):
    """out[s] = rows [s*M/R, (s+1)*M/R) of bf16(sum_r A[r] @ B[r]).

    ``out`` is either a list of R segment tensors [M/R, N] or one [M, N]
    tensor (segments are then its consecutive row bands)."""
    R = len(A)
    M, K = A[0].shape
    N = B[0].shape[1]
    for t in list(A) + list(B):
        _check_bf16(t, "A/B")
    if isinstance(out, (list, tuple)):
        segs = list(out)
        for t in segs:
            _check_bf16(t, "out")
        seg_ptrs = (ctypes.c_void_p * R)(*[t.data_ptr() for t in segs])
    else:
        _check_bf16(out, "out")
        S = M // R if R else 0
        seg_ptrs = (ctypes.c_void_p * R)(*[out.data_ptr() + s * S * N * 2 for s in range(R)])
    rc = load_library().are_gemm_rs(_ptrs(A), _ptrs(B), seg_ptrs, R, M, N, K, ws.handle, _stream_handle(stream))
    _check(rc, "are_gemm_rs")


def gemm_ar(A: Sequence, B: Sequence, out, ws: Workspace, stream=None):
    """Every view out[v] = bf16(sum_r f32(bf16(A[r] @ B[r]))).

    ``out`` is a list of R [M, N] views (they may alias) or one tensor used
    for every view."""
    R = len(A)
    M, K = A[0].shape
    N = B[0].shape[1]
    for t in list(A) + list(B):
        _check_bf16(t, "A/B")
    views = list(out) if isinstance(out, (list, tuple)) else [out] * R
    for t in views:
        _check_bf16(t, "out")
    rc = load_library().are_gemm_ar(_ptrs(A), _ptrs(B), _ptrs(views), R, M, N, K, ws.handle, _stream_handle(stream))
    _check(rc, "are_gemm_ar")


def allreduce_rmsnorm(partials: Sequence, residual, gamma, eps: float, out, ws: Workspace, stream=None):
    """out = bf16(rmsnorm(sum_r partials[r] + residual) * gamma)."""
    import torch
    R = len(partials)
    M, N = partials[0].shape
    for t in partials:
        _check_bf16(t, "partials")
    if residual is not None:
        _check_bf16(residual, "residual")
    _check_bf16(out, "out")
    if gamma.dtype != torch.float32 or not gamma.is_cuda or not gamma.is_contiguous():
        raise ValueError("gamma must be a contiguous CUDA float32 tensor")
    rc = load_library().are_allreduce_rmsnorm(
        _ptrs(partials), residual.data_ptr() if residual is not None else None, gamma.data_ptr(), float(eps),
        out.data_ptr(), R, M, N, ws.handle, _stream_handle(stream))
    _check(rc, "are_allreduce_rmsnorm")


def allreduce_add_rmsnorm(partials: Sequence, residual, gamma, eps: float, out, residual_out, ws: Workspace,
                          stream=None):
    """As ``allreduce_rmsnorm``, and residual_out = bf16(sum_r partials[r] +
    residual), the residual the next layer takes (may be ``residual`` itself)."""
    import torch
    R = len(partials)
    M, N = partials[0].shape
    for t in partials:
        _check_bf16(t, "partials")
    if residual is not None:
        _check_bf16(residual, "residual")
    _check_bf16(out, "out")
    if residual_out is not None:
        _check_bf16(residual_out, "residual_out")
    if gamma.dtype != torch.float32 or not gamma.is_cuda or not gamma.is_contiguous():
        raise ValueError("gamma must be a contiguous CUDA float32 tensor")
    rc = load_library().are_allreduce_add_rmsnorm(
        _ptrs(partials), residual.data_ptr() if residual is not None else None, gamma.data_ptr(), float(eps),
        out.data_ptr(), residual_out.data_ptr() if residual_out is not None else None, R, M, N, ws.handle,
        _stream_handle(stream))
    _check(rc, "are_allreduce_add_rmsnorm")


def allreduce_rmsnorm_quant(partials: Sequence, residual, gamma, eps: float, out_q, out_scale, ws: Workspace,
                            residual_out=None, stream=None):
    """Quantising variant: out_q (uint8 FP8 E4M3 codes [M, N]) and out_scale
    (fp32 [M]) with y ~= e4m3(out_q) * out_scale per row; residual_out optional."""
    import torch
    R = len(partials)
    M, N = partials[0].shape
    for t in partials:
        _check_bf16(t, "partials")
    if residual is not None:
        _check_bf16(residual, "residual")
    if residual_out is not None:
        _check_bf16(residual_out, "residual_out")
    if out_q.dtype != torch.uint8 or not out_q.is_cuda or not out_q.is_contiguous():
        raise ValueError("out_q must be a contiguous CUDA uint8 tensor")
    if out_scale.dtype != torch.float32 or not out_scale.is_cuda or not out_scale.is_contiguous():
        raise ValueError("out_scale must be a contiguous CUDA float32 tensor")
    if gamma.dtype != torch.float32 or not gamma.is_cuda or not gamma.is_contiguous():
        raise ValueError("gamma must be a contiguous CUDA float32 tensor")
    rc = load_library().are_allreduce_rmsnorm_quant(
        _ptrs(partials), residual.data_ptr() if residual is not None else None, gamma.data_ptr(), float(eps),
        out_q.data_ptr(), out_scale.data_ptr(), residual_out.data_ptr() if residual_out is not None else None,
        R, M, N, ws.handle, _stream_handle(stream))
    _check(rc, "are_allreduce_rmsnorm_quant")


def allreduce_rmsnorm_noalloc(partials: Sequence, residual, gamma, eps: float, out, stream=None):
    """As ``allreduce_rmsnorm`` but without a workspace and without any device
    allocation, for callers that cannot let a library allocate: the scratch is
    a fixed array inside the library (M * N <= 2,097,152).  Calls that can
    overlap on the GPU race on that array."""
    import torch
    R = len(partials)
    M, N = partials[0].shape
    for t in partials:
        _check_bf16(t, "partials")
    if residual is not None:
        _check_bf16(residual, "residual")
    _check_bf16(out, "out")
    if gamma.dtype != torch.float32 or not gamma.is_cuda or not gamma.is_contiguous():
        raise ValueError("gamma must be a contiguous CUDA float32 tensor")
    rc = load_library().are_allreduce_rmsnorm_noalloc(
        _ptrs(partials), residual.data_ptr() if residual is not None else None, gamma.data_ptr(), float(eps),
        out.data_ptr(), R, M, N, _stream_handle(stream))
    _check(rc, "are_allreduce_rmsnorm_noalloc")


def noalloc_device_status() -> dict:
    """Status word of the allocation-free entry point on the current device
    (synchronises the device; describes the last call only)."""
    st = _DevStatus()
    rc = load_library().are_noalloc_device_status(ctypes.byref(st))
    if rc not in (OK, ETIMEOUT):
        raise AreError(rc, "are_noalloc_device_status")
    return {"status": rc, "code": st.code, "where": st.where, "a": st.a, "b": st.b}


# Argument checks of the operations below: type, shape, contiguity, and the
# workspace's device.  The host's time is most of a one-token call's, so ranks
# are checked attribute by attribute through ``map`` (about half the time of a
# loop over the tensors).
def _need(t, dtype, shape, dev: int, what: str):
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on CUDA device {dev}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _need_one_of(t, dtypes, shape, dev: int, what: str):
    _need(t, t.dtype if t.dtype in dtypes else next(iter(dtypes)), shape, dev, what)


def _need_all(tensors, dtype, shape, dev: int, what: str):
    T = _tensor_type()
    n = len(tensors)
    if (list(map(T.get_device, tensors)) != [dev] * n or not all(map(T.is_contiguous, tensors))
            or [t.dtype for t in tensors] != [dtype] * n or [t.shape for t in tensors] != [shape] * n):
        for t in tensors:
            _need(t, dtype, shape, dev, what)


_T = None


def _tensor_type():
    global _T
    if _T is None:
        import torch
        _T = torch.Tensor
    return _T


def _addresses(tensors) -> array:
    """The tensors' addresses, as the C array of pointers that the ABI takes."""
    return array("Q", map(_tensor_type().data_ptr, tensors))


def _at(a: array) -> int:
    return a.buffer_info()[0]


def _address(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _ranks(tensors, what: str) -> int:
    if not 1 <= len(tensors) <= 8:
        raise ValueError(f"{what}: 1 to 8 ranks, got {len(tensors)}")
    return len(tensors)


def _matrix(t, what: str):
    if t.dim() != 2:
        raise ValueError(f"{what} must have two dimensions, got {tuple(t.shape)}")
    return t.shape


def _group_of(group: int, what: str) -> int:
    if group not in (32, 64, 128):
        raise ValueError(f"{what} must be 32, 64 or 128, got {group}")
    return group


def _on_stream(stream, dev: int) -> int:
    import torch
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)  # current_stream(dev).cuda_stream without its wrapper
    if stream.device_index != dev:
        raise ValueError(f"the stream is on CUDA device {stream.device_index}, the workspace on {dev}")
    return stream.cuda_stream


_kinds: dict = {}


def _scale_kinds() -> dict:
    """The scale format of each type that a scale tensor may have."""
    if not _kinds:
        import torch
        _kinds.update({torch.float32: SCALE_F32, torch.uint8: SCALE_E8M0, torch.float8_e8m0fnu: SCALE_E8M0})
    return _kinds


def allreduce_rmsnorm_quant_groups(partials: Sequence, residual, gamma, eps: float, out_q, out_scale, ws: Workspace,
                                   group: int = 128, residual_out=None, stream=None):
    """FP8 E4M3 codes of y = rmsnorm(sum_r partials[r] + residual) * gamma with
    one scale per ``group`` (32, 64, 128) columns: y ~= e4m3(out_q) * scale.

    ``out_q``: [M, N] uint8 or float8_e4m3fn.  ``out_scale``:
    [M, ceil(N / group)], float32 (max / 448) or uint8 / float8_e8m0fnu (the
    power of two above it).  ``residual_out`` (may be ``residual``): bf16 sum."""
    import torch
    dev, bf16 = ws.device_index, torch.bfloat16
    R = _ranks(partials, "partials")
    shape = _matrix(partials[0], "partials")
    M, N = shape
    _need_all(partials, bf16, shape, dev, "partials")
    if residual is not None:
        _need(residual, bf16, shape, dev, "residual")
    if residual_out is not None:
        _need(residual_out, bf16, shape, dev, "residual_out")
    _need(gamma, torch.float32, (N,), dev, "gamma")
    _need_one_of(out_q, (torch.uint8, torch.float8_e4m3fn), shape, dev, "out_q")
    kinds = _scale_kinds()
    _need_one_of(out_scale, kinds, (M, -(-N // _group_of(group, "group"))), dev, "out_scale")
    parts = _addresses(partials)
    rc = load_library().are_allreduce_rmsnorm_quant_groups(
        _at(parts), _address(residual), gamma.data_ptr(), eps, kinds[out_scale.dtype], group, out_q.data_ptr(),
        out_scale.data_ptr(), _address(residual_out), R, M, N, ws.handle, _on_stream(stream, dev))
    _check(rc, "are_allreduce_rmsnorm_quant_groups")


def allreduce_rmsnorm_backward(dy: Sequence, h, gamma, eps: float, dh, dgamma, ws: Workspace, dres=None, stream=None):
    """Backward pass of all-reduce + residual + RMSNorm.

    ``dy``: R bf16 [M, N] partials of the output's gradient, summed first;
    ``h``: the updated residual (``residual_out`` of the forward call);
    ``dres``: the gradient of that residual, or None.  Writes ``dh`` (bf16; may
    be ``dres``), the gradient of every partial and of the incoming residual,
    and ``dgamma`` (float32 [N], or None)."""
    import torch
    dev, bf16 = ws.device_index, torch.bfloat16
    R = _ranks(dy, "dy")
    shape = _matrix(dy[0], "dy")
    M, N = shape
    _need_all(dy, bf16, shape, dev, "dy")
    _need(h, bf16, shape, dev, "h")
    _need(dh, bf16, shape, dev, "dh")
    if dres is not None:
        _need(dres, bf16, shape, dev, "dres")
    _need(gamma, torch.float32, (N,), dev, "gamma")
    if dgamma is not None:
        _need(dgamma, torch.float32, (N,), dev, "dgamma")
    parts = _addresses(dy)
    rc = load_library().are_allreduce_rmsnorm_backward(
        _at(parts), h.data_ptr(), gamma.data_ptr(), eps, _address(dres), dh.data_ptr(), _address(dgamma), R, M, N,
        ws.handle, _on_stream(stream, dev))
    _check(rc, "are_allreduce_rmsnorm_backward")


def allreduce_layernorm(partials: Sequence, residual, gamma, beta, eps: float, out, ws: Workspace, residual_out=None,
                        stream=None):
    """out = bf16(layernorm(sum_r partials[r] + residual) * gamma + beta).

    ``gamma``, ``beta``: float32 [N], ``beta`` may be None.  ``residual_out``
    (may be ``residual``): the bf16 sum, the residual that the next layer takes."""
    import torch
    dev, bf16 = ws.device_index, torch.bfloat16
    R = _ranks(partials, "partials")
    shape = _matrix(partials[0], "partials")
    M, N = shape
    _need_all(partials, bf16, shape, dev, "partials")
    if residual is not None:
        _need(residual, bf16, shape, dev, "residual")
    if residual_out is not None:
        _need(residual_out, bf16, shape, dev, "residual_out")
    _need(gamma, torch.float32, (N,), dev, "gamma")
    if beta is not None:
        _need(beta, torch.float32, (N,), dev, "beta")
    _need(out, bf16, shape, dev, "out")
    parts = _addresses(partials)
    rc = load_library().are_allreduce_layernorm(
        _at(parts), _address(residual), gamma.data_ptr(), _address(beta), eps, out.data_ptr(), _address(residual_out), R, M,
        N, ws.handle, _on_stream(stream, dev))
    _check(rc, "are_allreduce_layernorm")


def allreduce_layernorm_backward(dy: Sequence, h, gamma, eps: float, dh, dgamma, dbeta, ws: Workspace, dres=None,
                                 stream=None):
    """Backward pass of all-reduce + residual + LayerNorm.

    As ``allreduce_rmsnorm_backward``; ``dgamma`` and ``dbeta``: float32 [N],
    either may be None."""
    import torch
    dev, bf16 = ws.device_index, torch.bfloat16
    R = _ranks(dy, "dy")
    shape = _matrix(dy[0], "dy")
    M, N = shape
    _need_all(dy, bf16, shape, dev, "dy")
    _need(h, bf16, shape, dev, "h")
    _need(dh, bf16, shape, dev, "dh")
    if dres is not None:
        _need(dres, bf16, shape, dev, "dres")
    _need(gamma, torch.float32, (N,), dev, "gamma")
    for t, what in ((dgamma, "dgamma"), (dbeta, "dbeta")):
        if t is not None:
            _need(t, torch.float32, (N,), dev, what)
    parts = _addresses(dy)
    rc = load_library().are_allreduce_layernorm_backward(
        _at(parts), h.data_ptr(), gamma.data_ptr(), eps, _address(dres), dh.data_ptr(), _address(dgamma), _address(dbeta),
        R, M, N, ws.handle, _on_stream(stream, dev))
    _check(rc, "are_allreduce_layernorm_backward")


def _index_format(t, M: int, dev: int, what: str) -> int:
    import torch
    _need_one_of(t, (torch.int64, torch.int32), (M,), dev, what)
    return INDEX_I64 if t.dtype is torch.int64 else INDEX_I32


def _tables(ids, rows, tables: Sequence, dev: int, what: str, rows_what: str):
    """Checks that both directions of the embedding share; (R, M, N, V, index format)."""
    import torch
    M, N = _matrix(rows, rows_what)
    _need(rows, torch.bfloat16, (M, N), dev, rows_what)
    R = _ranks(tables, what)
    V = _matrix(tables[0], what)[0]
    _need_all(tables, torch.bfloat16, (V, N), dev, what)
    return R, M, N, V, _index_format(ids, M, dev, "ids")


def embedding_ar(ids, tables: Sequence, out, ws: Workspace, scale: float = 1.0, stream=None):
    """out[i] = bf16(scale * row ids[i] of cat(tables)); zeros where ids[i] is
    outside the vocabulary.

    ``ids``: int64 or int32 [M]; ``tables``: R bf16 [V, N] tensors, rank r's
    holds the vocabulary from r * V on; ``out``: bf16 [M, N]."""
    dev = ws.device_index
    R, M, N, V, fmt = _tables(ids, out, tables, dev, "tables", "out")
    rows = _addresses(tables)
    rc = load_library().are_embedding_ar(ids.data_ptr(), fmt, _at(rows), scale, out.data_ptr(), R, M, N, V, ws.handle,
                                         _on_stream(stream, dev))
    _check(rc, "are_embedding_ar")


def embedding_ar_backward(ids, dy, dtables: Sequence, ws: Workspace, scale: float = 1.0, accumulate: bool = False,
                          stream=None):
    """The gradient of ``embedding_ar`` for every rank's table: row v of
    cat(dtables) = bf16(scale * the fp32 sum of the dy[i] with ids[i] = v).

    ``dy``: bf16 [M, N].  Every row is written, or, with ``accumulate``, the
    rows that tokens have are added to and the others left alone.  The
    workspace needs ``M_max`` >= M and ``N_max`` >= N."""
    dev = ws.device_index
    R, M, N, V, fmt = _tables(ids, dy, dtables, dev, "dtables", "dy")
    rows = _addresses(dtables)
    rc = load_library().are_embedding_ar_backward(ids.data_ptr(), fmt, dy.data_ptr(), scale, int(bool(accumulate)), _at(rows), R,
                                                  M, N, V, ws.handle, _on_stream(stream, dev))
    _check(rc, "are_embedding_ar_backward")


def _output_layer(h, w: Sequence, targets, vocab, dev: int):
    """Checks that both directions of the cross entropy share; (R, M, N, K, vocab, index format)."""
    import torch
    M, K = _matrix(h, "h")
    _need(h, torch.bfloat16, (M, K), dev, "h")
    R = _ranks(w, "w")
    N = _matrix(w[0], "w")[0]
    _need_all(w, torch.bfloat16, (N, K), dev, "w")
    vocab = R * N if vocab is None else vocab
    if not 1 <= vocab <= R * N:
        raise ValueError(f"vocab must be 1 to {R * N}, got {vocab}")
    return R, M, N, K, vocab, _index_format(targets, M, dev, "targets")


def gemm_cross_entropy(h, w: Sequence, targets, loss, lse, ws: Workspace, vocab: Optional[int] = None, stream=None):
    """loss[i] = lse[i] - z[i, targets[i]], lse[i] = log sum_v exp z[i, v], with
    the logits z = h @ cat(w).T never stored.

    ``h``: bf16 [M, K]; ``w``: R bf16 [N, K] tensors, rank r's holds the
    vocabulary from r * N on; ``targets``: int64 or int32 [M], outside the
    vocabulary (-100, say): loss 0; ``loss``, ``lse``: float32 [M]; ``vocab``:
    indices that count (R * N), the rows of ``w`` behind are padding.  The
    workspace needs ``vocab_piece`` > 0, ``M_max`` >= M and ``K_max`` >= K."""
    import torch
    dev = ws.device_index
    R, M, N, K, vocab, fmt = _output_layer(h, w, targets, vocab, dev)
    _need(loss, torch.float32, (M,), dev, "loss")
    _need(lse, torch.float32, (M,), dev, "lse")
    weights = _addresses(w)
    rc = load_library().are_gemm_cross_entropy(h.data_ptr(), _at(weights), targets.data_ptr(), fmt, vocab, loss.data_ptr(),
                                               lse.data_ptr(), R, M, N, K, ws.handle, _on_stream(stream, dev))
    _check(rc, "are_gemm_cross_entropy")


def gemm_cross_entropy_backward(h, w: Sequence, targets, lse, dloss, dh, dw, ws: Workspace, vocab: Optional[int] = None,
                                stream=None):
    """Gradients of ``gemm_cross_entropy``: ``dloss`` (float32 [M]) is the
    gradient of ``loss``, ``lse`` what the forward call wrote.

    Writes ``dh`` (bf16 [M, K], summed over the ranks, or None) and ``dw`` (R
    bf16 [N, K] tensors, or None)."""
    import torch
    dev = ws.device_index
    R, M, N, K, vocab, fmt = _output_layer(h, w, targets, vocab, dev)
    _need(lse, torch.float32, (M,), dev, "lse")
    _need(dloss, torch.float32, (M,), dev, "dloss")
    if dh is not None:
        _need(dh, torch.bfloat16, (M, K), dev, "dh")
    grads = None
    if dw is not None:
        if len(dw) != R:
            raise ValueError(f"{R} ranks of weights, {len(dw)} of gradients")
        _need_all(dw, torch.bfloat16, (N, K), dev, "dw")
        grads = _addresses(dw)
    weights = _addresses(w)
    rc = load_library().are_gemm_cross_entropy_backward(
        h.data_ptr(), _at(weights), targets.data_ptr(), fmt, vocab, lse.data_ptr(), dloss.data_ptr(), _address(dh),
        None if grads is None else _at(grads), R, M, N, K, ws.handle, _on_stream(stream, dev))
    _check(rc, "are_gemm_cross_entropy_backward")


class QWeight:
    """One rank's 4-bit weights: weight (n, k) = (u - zero[n, k // group]) *
    scale[n, k // group].

    ``codes``: uint8 [N, K / 2], byte i of a row holds k = 2i in its lower and
    2i + 1 in its upper four bits; ``scale``: bf16 [N, ceil(K / group)];
    ``zero``: uint8 of the same shape, values 0..15, or None (8 everywhere);
    ``group``: 32, 64 or 128.  The tensors are checked here, once; it holds
    tensors of its own over the same memory, none of which can be replaced, so
    what a call uses is what was checked.  Their contents may change, and a
    tensor given another memory (``t.data = ...``) needs another QWeight."""

    __slots__ = ("codes", "scale", "zero", "group", "N", "K", "_key")

    def __setattr__(self, name, value):
        raise AttributeError(f"QWeight.{name} cannot be replaced: make another QWeight")

    def __delattr__(self, name):
        raise AttributeError(f"QWeight.{name} cannot be removed")

    def __init__(self, codes, scale, zero=None, group: int = 128):
        import torch
        dev = codes.get_device()
        N, half = _matrix(codes, "codes")
        K = 2 * half
        _need(codes, torch.uint8, (N, half), dev, "codes")
        groups = (N, -(-K // _group_of(group, "group")))
        _need(scale, torch.bfloat16, groups, dev, "scale")
        if zero is not None:
            _need(zero, torch.uint8, groups, dev, "zero")
        own = dict(codes=codes.detach(), scale=scale.detach(), zero=None if zero is None else zero.detach(), group=group,
                   N=N, K=K, _key=(N, K, group, dev))
        for name, value in own.items():
            object.__setattr__(self, name, value)

    def __reduce__(self):  # copies and pickles are checked again
        return QWeight, (self.codes, self.scale, self.zero, self.group)


def _qweights(w: Sequence, R: int, M: int, K: int, out, dev: int):
    """The C arrays of the weights and of the output views, and the weights' N and group."""
    import torch
    if len(w) != R:
        raise ValueError(f"{R} ranks of tokens, {len(w)} of weights")
    N, group = w[0].N, w[0].group
    if [q._key for q in w] != [(N, K, group, dev)] * R:
        raise ValueError(f"every rank's weights must be [{N}, {K}] in groups of {group} on CUDA device {dev}")
    if w[0].zero is not None and all([q.zero is not None for q in w]):
        weights = _addresses([t for q in w for t in (q.codes, q.scale, q.zero)])
        missing = 0 in weights
    else:
        found = [_address(t) for q in w for t in (q.codes, q.scale, q.zero)]
        weights = array("Q", [v or 0 for v in found])  # no zero points: a null pointer
        missing = 0 in found
    if missing and N and K:
        raise ValueError("weights whose memory has been given back (a storage resized to nothing)")
    if isinstance(out, (list, tuple)):
        if len(out) != R:
            raise ValueError(f"{R} ranks, {len(out)} output views")
        _need_all(out, torch.bfloat16, (M, N), dev, "out")
        views = _addresses(out)
    else:
        _need(out, torch.bfloat16, (M, N), dev, "out")
        views = array("Q", [out.data_ptr()]) * R
    return weights, group, views, N


def gemm_ar_qweight(x: Sequence, w: Sequence, out, ws: Workspace, stream=None):
    """Every view out[v] = bf16(sum_r x[r] @ w[r].T) with 4-bit weights.

    ``x``: R bf16 [M, K] token tensors; ``w``: R ``QWeight``; ``out``: one
    bf16 [M, N] tensor, or a list of R views (they may alias)."""
    import torch
    dev = ws.device_index
    R = _ranks(x, "x")
    shape = _matrix(x[0], "x")
    M, K = shape
    _need_all(x, torch.bfloat16, shape, dev, "x")
    weights, group, views, N = _qweights(w, R, M, K, out, dev)
    tokens = _addresses(x)
    rc = load_library().are_gemm_ar_qweight(_at(tokens), _at(weights), group, _at(views), R, M, N, K, ws.handle,
                                            _on_stream(stream, dev))
    _check(rc, "are_gemm_ar_qweight")


def gemm_ar_qweight_qx(xq: Sequence, xscale: Sequence, w: Sequence, out, ws: Workspace, xgroup: int = 128,
                       stream=None):
    """As ``gemm_ar_qweight`` with tokens e4m3(xq[r]) * xscale[r], as
    ``allreduce_rmsnorm_quant_groups`` writes them.

    ``xq``: R [M, K] tensors, all uint8 or all float8_e4m3fn; ``xscale``: R tensors
    [M, ceil(K / xgroup)], float32 or uint8 / float8_e8m0fnu (all of one
    kind)."""
    import torch
    dev = ws.device_index
    R = _ranks(xq, "xq")
    shape = _matrix(xq[0], "xq")
    M, K = shape
    if len(xscale) != R:
        raise ValueError(f"{R} ranks of codes, {len(xscale)} of scales")
    kinds = _scale_kinds()
    sshape, sdt = (M, -(-K // _group_of(xgroup, "xgroup"))), xscale[0].dtype
    if sdt not in kinds:
        raise ValueError(f"xscale must be float32, uint8 or float8_e8m0fnu, got {sdt}")
    codes = xq[0].dtype
    _need_all(xq, codes if codes is torch.float8_e4m3fn else torch.uint8, shape, dev, "xq")
    _need_all(xscale, sdt, sshape, dev, "xscale")
    weights, group, views, N = _qweights(w, R, M, K, out, dev)
    tokens, scales = _addresses(xq), _addresses(xscale)
    rc = load_library().are_gemm_ar_qweight_qx(_at(tokens), _at(scales), kinds[sdt], xgroup, _at(weights), group,
                                               _at(views), R, M, N, K, ws.handle, _on_stream(stream, dev))
    _check(rc, "are_gemm_ar_qweight_qx")
