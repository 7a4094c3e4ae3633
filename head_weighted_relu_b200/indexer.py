"""Thin ctypes binding over libhwr_indexer.so (include/hwr_indexer.h).

The functions named like the C entry points marshal arguments only: torch
tensors become raw device pointers, torch streams become cudaStream_t.  Every
step of the indexer runs in the library's kernels; there is no fallback.  If the
library is missing, importing this module raises.

`topk(...)` is the convenience call most users want: it allocates outputs and
workspace with torch (plumbing) and calls indexer_topk.  Around it,
`rotate_quantise(...)` makes its FP8 rows, `cache_append(...)` keeps the keys and
values of new tokens in a paged 8-bit cache, and `cache_attend(...)` attends over
that cache, over what `topk` selected or over whole sequences.
"""

from __future__ import annotations

import ctypes
import math
import os
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# HWR_INDEXER_LIB may point at another build of the same library (same ABI)
LIB_PATH = os.environ.get("HWR_INDEXER_LIB") or os.path.join(_HERE, "libhwr_indexer.so")

TOKEN, COMPRESSED, POOLED = 0, 1, 2
BF16, FP8_E4M3 = 0, 1
FLAG_PRUNE = 1
FLAG_TEST_WAIT_TIMEOUT = 1 << 30   # test hook: the kernel's wait-timeout path (outputs not valid)

STATUS_NAMES = {0: "INDEXER_OK", 1: "INDEXER_EINVAL", 2: "INDEXER_EWORKSPACE",
                3: "INDEXER_EUNSUPPORTED", 4: "INDEXER_ECUDA", 5: "INDEXER_EDEVICE"}

# every symbol include/hwr_indexer.h declares
EXPORTS = ("indexer_out_width", "indexer_workspace_bytes", "indexer_partition_rows",
           "indexer_topk", "indexer_topk_noalloc", "indexer_noalloc_read_status",
           "indexer_host_workspace_bytes", "indexer_topk_host",
           "indexer_docs_workspace_bytes", "indexer_topk_docs",
           "indexer_padded_workspace_bytes", "indexer_topk_padded",
           "indexer_witness_workspace_bytes", "indexer_topk_witness",
           "indexer_pool_keys",
           "indexer_rotate_quantise", "indexer_cache_append",
           "indexer_cache_attend_workspace_bytes", "indexer_cache_attend",
           "indexer_pair_overlap", "indexer_pair_regions", "indexer_read_status", "indexer_read_prune_counters",
           "indexer_status_string",
           "indexer_abi_version", "indexer_build_info")


class IndexerError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        msg = _lib.indexer_status_string(status).decode()
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)} ({msg})")


class Problem(ctypes.Structure):
    """Mirror of indexer_problem."""
    _fields_ = [("S", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int32),
                ("D", ctypes.c_int32), ("q_pos0", ctypes.c_int64), ("visibility", ctypes.c_int32),
                ("ratio", ctypes.c_int32), ("K", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("reserved", ctypes.c_int32)]


ACT_BF16, ACT_FP16 = 0, 1
ATTEND_AUTO, ATTEND_STREAM, ATTEND_TILE = 0, 1, 2   # kernels of cache_attend
ATTEND_TEST_WAIT_TIMEOUT = 1 << 8   # with ATTEND_TILE: test hook of its failure path
STATUS_TOKEN = 8   # status bit of the cache calls: a token's page or position does not exist


class Rotation(ctypes.Structure):
    """Mirror of indexer_rotation."""
    _fields_ = [("table", ctypes.c_void_p), ("rows", ctypes.c_int64), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class CacheDesc(ctypes.Structure):
    """Mirror of indexer_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("block", ctypes.c_int32), ("heads", ctypes.c_int32), ("D", ctypes.c_int32)]


class Sequences(ctypes.Structure):
    """Mirror of indexer_sequences."""
    _fields_ = [("S", ctypes.c_int64), ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("table_pages", ctypes.c_int32), ("B", ctypes.c_int32)]


class Attention(ctypes.Structure):
    """Mirror of indexer_attention."""
    _fields_ = [("Hq", ctypes.c_int32), ("act", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("sel_width", ctypes.c_int32), ("max_q", ctypes.c_int32), ("scale", ctypes.c_float),
                ("kernel", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m head_weighted_relu_b200.build` "
            "(the indexer has no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    lib.indexer_build_info.argtypes = []
    lib.indexer_build_info.restype = ctypes.c_char_p
    if "HWR_INDEXER_LIB" not in os.environ:
        # the library must come from the sources beside it (a stale build would
        # otherwise pass unnoticed)
        from . import build as _build
        want = "source_sha256=" + _build.source_hash()
        got = lib.indexer_build_info().decode()
        if got != want:
            raise ImportError(f"{LIB_PATH} was built from other sources ({got[:30]}...); "
                              "rebuild it with `python -m head_weighted_relu_b200.build`")
    P = ctypes.POINTER(Problem)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.indexer_out_width.argtypes = [P, ctypes.POINTER(i32)]
    lib.indexer_workspace_bytes.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
    lib.indexer_partition_rows.argtypes = [P, i32, ctypes.POINTER(i64)]
    lib.indexer_topk.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.indexer_topk_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.indexer_noalloc_read_status.argtypes = [ctypes.POINTER(i32), vp]
    lib.indexer_host_workspace_bytes.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
    lib.indexer_topk_host.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.indexer_docs_workspace_bytes.argtypes = [P, vp, i32, ctypes.POINTER(ctypes.c_size_t)]
    lib.indexer_topk_docs.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.indexer_padded_workspace_bytes.argtypes = [P, vp, i32, i64, ctypes.POINTER(ctypes.c_size_t)]
    lib.indexer_topk_padded.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, i32, i64, vp, vp, vp, vp,
                                        ctypes.c_size_t, vp]
    lib.indexer_witness_workspace_bytes.argtypes = [P, i64, ctypes.POINTER(ctypes.c_size_t)]
    lib.indexer_topk_witness.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.indexer_pool_keys.argtypes = [vp, i64, i32, vp, i32, vp, vp]
    lib.indexer_rotate_quantise.argtypes = [vp, i64, i32, i32, i32, i64, vp, ctypes.POINTER(Rotation), vp, vp, vp, vp]
    CD, SQ, AT = ctypes.POINTER(CacheDesc), ctypes.POINTER(Sequences), ctypes.POINTER(Attention)
    lib.indexer_cache_append.argtypes = [CD, SQ, vp, vp, i64, i32, ctypes.POINTER(Rotation), vp, i32, i64, vp, vp, vp]
    lib.indexer_cache_attend_workspace_bytes.argtypes = [CD, SQ, AT, ctypes.POINTER(ctypes.c_size_t)]
    lib.indexer_cache_attend.argtypes = [CD, SQ, AT, vp, i64, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.indexer_pair_overlap.argtypes = [vp, vp, i64, i32, vp, vp]
    lib.indexer_pair_regions.argtypes = [vp, vp, i64, i32, vp, vp, vp, vp, vp]
    lib.indexer_read_status.argtypes = [vp, ctypes.POINTER(i32), vp]
    lib.indexer_read_prune_counters.argtypes = [vp, ctypes.POINTER(ctypes.c_uint64), vp]
    lib.indexer_status_string.argtypes = [ctypes.c_int]
    lib.indexer_status_string.restype = ctypes.c_char_p
    lib.indexer_abi_version.argtypes = []
    for name in EXPORTS:
        if name not in ("indexer_status_string", "indexer_build_info"):
            getattr(lib, name).restype = ctypes.c_int
    return lib


_lib = _load()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn, status):
    if status != 0:
        raise IndexerError(fn, status)


def make_problem(S, T, H, D, K, visibility=TOKEN, ratio=1, dtype=BF16, q_pos0=0,
                 prune=False, flags=0) -> Problem:
    if isinstance(dtype, str):
        dtype = {"bf16": BF16, "fp8": FP8_E4M3}[dtype]
    return Problem(S=S, T=T, H=H, D=D, q_pos0=q_pos0, visibility=visibility, ratio=ratio,
                   K=K, dtype=dtype, flags=(FLAG_PRUNE if prune else 0) | flags, reserved=0)


def indexer_out_width(problem: Problem) -> int:
    w = ctypes.c_int32()
    _check("indexer_out_width", _lib.indexer_out_width(ctypes.byref(problem), ctypes.byref(w)))
    return w.value


def indexer_workspace_bytes(problem: Problem) -> int:
    n = ctypes.c_size_t()
    _check("indexer_workspace_bytes",
           _lib.indexer_workspace_bytes(ctypes.byref(problem), ctypes.byref(n)))
    return n.value


def indexer_partition_rows(problem: Problem, n_parts: int) -> list:
    """Row bounds [0, ..., S] splitting the problem's query rows into n_parts
    parts of about equal visible-pair count (one part per GPU)."""
    b = (ctypes.c_int64 * (n_parts + 1))()
    _check("indexer_partition_rows", _lib.indexer_partition_rows(ctypes.byref(problem), n_parts, b))
    return [int(x) for x in b]


def indexer_topk(problem, q, k, w, q_scale, k_scale, pool_coef, out_idx, out_len, out_score,
                 workspace, stream=None):
    _check("indexer_topk", _lib.indexer_topk(
        ctypes.byref(problem), _ptr(q), _ptr(k), _ptr(w), _ptr(q_scale), _ptr(k_scale),
        _ptr(pool_coef), _ptr(out_idx), _ptr(out_len), _ptr(out_score), _ptr(workspace),
        ctypes.c_size_t(workspace.numel() * workspace.element_size()), _stream(stream)))


def indexer_witness_workspace_bytes(problem: Problem, n_seeds: int) -> int:
    n = ctypes.c_size_t()
    _check("indexer_witness_workspace_bytes",
           _lib.indexer_witness_workspace_bytes(ctypes.byref(problem), ctypes.c_int64(n_seeds), ctypes.byref(n)))
    return n.value


def indexer_topk_witness(problem, q, k, w, q_scale, k_scale, pool_coef, seeds, out_idx, out_len, out_score,
                         workspace, stream=None):
    """indexer_topk starting from a seed threshold: seeds is a [S, n] int32
    device tensor of key indices per query (e.g. the previous decode step's
    out_idx), -1 or invisible entries ignored.  Same result as indexer_topk."""
    if seeds.dtype != torch.int32 or seeds.dim() != 2 or not seeds.is_contiguous():
        raise ValueError("seeds must be a contiguous [S, n] int32 tensor")
    _check("indexer_topk_witness", _lib.indexer_topk_witness(
        ctypes.byref(problem), _ptr(q), _ptr(k), _ptr(w), _ptr(q_scale), _ptr(k_scale),
        _ptr(pool_coef), _ptr(seeds), ctypes.c_int64(seeds.shape[1]), _ptr(out_idx), _ptr(out_len),
        _ptr(out_score), _ptr(workspace),
        ctypes.c_size_t(workspace.numel() * workspace.element_size()), _stream(stream)))


def indexer_host_workspace_bytes(problem: Problem) -> int:
    n = ctypes.c_size_t()
    _check("indexer_host_workspace_bytes",
           _lib.indexer_host_workspace_bytes(ctypes.byref(problem), ctypes.byref(n)))
    return n.value


def indexer_topk_host(problem, q, k, w, q_scale, k_scale, pool_coef, out_idx, out_len, out_score,
                      workspace, stream=None):
    """indexer_topk on host tensors (pinned for the copies to overlap): inputs and
    outputs live in host memory, `workspace` is a device buffer of
    indexer_host_workspace_bytes bytes.  Ordered on `stream`; synchronise it
    before reading the outputs."""
    _check("indexer_topk_host", _lib.indexer_topk_host(
        ctypes.byref(problem), _ptr(q), _ptr(k), _ptr(w), _ptr(q_scale), _ptr(k_scale),
        _ptr(pool_coef), _ptr(out_idx), _ptr(out_len), _ptr(out_score), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def _bounds(doc_bounds):
    import numpy as np
    b = np.ascontiguousarray(np.asarray(doc_bounds, dtype=np.int64))
    return b, ctypes.c_void_p(b.ctypes.data), len(b) - 1


def indexer_docs_workspace_bytes(problem: Problem, doc_bounds) -> int:
    b, ptr, n = _bounds(doc_bounds)
    out = ctypes.c_size_t()
    _check("indexer_docs_workspace_bytes",
           _lib.indexer_docs_workspace_bytes(ctypes.byref(problem), ptr, n, ctypes.byref(out)))
    return out.value


def indexer_topk_docs(problem, q, k, w, q_scale, k_scale, pool_coef, doc_bounds, out_idx, out_len,
                      out_score, workspace, stream=None):
    """indexer_topk for a packed batch of documents: doc_bounds (host, n_docs + 1
    token positions) splits the tokens; a query sees only its own document."""
    b, ptr, n = _bounds(doc_bounds)
    _check("indexer_topk_docs", _lib.indexer_topk_docs(
        ctypes.byref(problem), _ptr(q), _ptr(k), _ptr(w), _ptr(q_scale), _ptr(k_scale), _ptr(pool_coef),
        ptr, n, _ptr(out_idx), _ptr(out_len), _ptr(out_score), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def indexer_padded_workspace_bytes(problem: Problem, seq_lens, stride: int) -> int:
    b, ptr, n = _bounds(seq_lens)
    out = ctypes.c_size_t()
    _check("indexer_padded_workspace_bytes",
           _lib.indexer_padded_workspace_bytes(ctypes.byref(problem), ptr, n + 1, stride, ctypes.byref(out)))
    return out.value


def indexer_topk_padded(problem, q, k, w, q_scale, k_scale, pool_coef, seq_lens, stride, out_idx, out_len,
                        out_score, workspace, stream=None):
    """indexer_topk for a padded batch: sequence b is rows b*stride ..
    b*stride + seq_lens[b] - 1 (seq_lens on the host); padding rows select
    nothing."""
    b, ptr, n = _bounds(seq_lens)
    _check("indexer_topk_padded", _lib.indexer_topk_padded(
        ctypes.byref(problem), _ptr(q), _ptr(k), _ptr(w), _ptr(q_scale), _ptr(k_scale), _ptr(pool_coef),
        ptr, n + 1, stride, _ptr(out_idx), _ptr(out_len), _ptr(out_score), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def indexer_topk_noalloc(problem, q, k, w, q_scale, k_scale, pool_coef, out_idx, out_len,
                         out_score, stream=None):
    """indexer_topk without a workspace: for callers that cannot allocate device
    memory.  Scratch is the library's fixed 64 MiB device array; larger problems
    raise IndexerError (INDEXER_EWORKSPACE).  Calls share that array, so calls
    that could overlap on the GPU must be serialised."""
    _check("indexer_topk_noalloc", _lib.indexer_topk_noalloc(
        ctypes.byref(problem), _ptr(q), _ptr(k), _ptr(w), _ptr(q_scale), _ptr(k_scale),
        _ptr(pool_coef), _ptr(out_idx), _ptr(out_len), _ptr(out_score), _stream(stream)))


def indexer_noalloc_read_status(stream=None) -> int:
    """Status word of the last indexer_topk_noalloc call (read and cleared)."""
    f = ctypes.c_int32()
    _check("indexer_noalloc_read_status", _lib.indexer_noalloc_read_status(ctypes.byref(f), _stream(stream)))
    return f.value


def indexer_pool_keys(k, T_tokens, D, pool_coef, ratio, out_kp, stream=None):
    _check("indexer_pool_keys", _lib.indexer_pool_keys(
        _ptr(k), T_tokens, D, _ptr(pool_coef), ratio, _ptr(out_kp), _stream(stream)))


def indexer_pair_overlap(idx, lens, S, width, out_shared, stream=None):
    _check("indexer_pair_overlap", _lib.indexer_pair_overlap(
        _ptr(idx), _ptr(lens), S, width, _ptr(out_shared), _stream(stream)))


def indexer_pair_regions(idx, lens, S, width, out_shared, out_left, out_right, out_counts, stream=None):
    _check("indexer_pair_regions", _lib.indexer_pair_regions(
        _ptr(idx), _ptr(lens), S, width, _ptr(out_shared), _ptr(out_left), _ptr(out_right), _ptr(out_counts),
        _stream(stream)))


def indexer_read_status(workspace, stream=None) -> int:
    f = ctypes.c_int32()
    _check("indexer_read_status",
           _lib.indexer_read_status(_ptr(workspace), ctypes.byref(f), _stream(stream)))
    return f.value


def indexer_read_prune_counters(workspace, stream=None):
    """(pairs screened, pairs bounded below the threshold, pairs skipped) of the
    last call that used `workspace`."""
    c = (ctypes.c_uint64 * 3)()
    _check("indexer_read_prune_counters", _lib.indexer_read_prune_counters(
        _ptr(workspace), c, _stream(stream)))
    return tuple(int(x) for x in c)


def indexer_abi_version() -> int:
    return _lib.indexer_abi_version()


def indexer_build_info() -> str:
    """The build's identity: "source_sha256=<hash of the sources and flags>"."""
    return _lib.indexer_build_info().decode()


# ---------------------------------------------------------------------------
# Convenience layer (allocation through torch; compute through the library).
# ---------------------------------------------------------------------------

def _as_storage(x):
    """q / k storage as the library expects it: bf16, or e4m3 codes as uint8."""
    if x.dtype == torch.float8_e4m3fn:
        return x.view(torch.uint8)
    return x


def allocate(problem: Problem, device, with_scores=False):
    """Outputs and workspace for `problem` on `device` (torch allocations)."""
    width = indexer_out_width(problem)
    out_idx = torch.empty((problem.S, width), dtype=torch.int32, device=device)
    out_len = torch.empty((problem.S,), dtype=torch.int32, device=device)
    out_score = (torch.empty((problem.S, width), dtype=torch.float32, device=device)
                 if with_scores else None)
    ws = torch.empty((max(indexer_workspace_bytes(problem), 256),), dtype=torch.uint8, device=device)
    return out_idx, out_len, out_score, ws


def topk(q, k, w, K, visibility=TOKEN, ratio=1, q_pos0=0, q_scale=None, k_scale=None,
         pool_coef=None, with_scores=False, stream=None, buffers=None, prune=False):
    """Indexer top-K of every query row (prune=True: the lossless pruning stage).

    q [S, H, D] bf16 (or e4m3 / uint8 codes with q_scale [S, H]), k [T, D] likewise
    (k_scale [T]), w [S, H] float32.  Returns (idx [S, W] int32, len [S] int32) and,
    with_scores=True, also score [S, W] float32.
    """
    q, k = _as_storage(q), _as_storage(k)
    S, H, D = q.shape
    fp8 = q.dtype == torch.uint8
    prob = make_problem(S=S, T=k.shape[0], H=H, D=D, K=K, visibility=visibility,
                        ratio=ratio if visibility != TOKEN else 1,
                        dtype=FP8_E4M3 if fp8 else BF16, q_pos0=q_pos0, prune=prune)
    if buffers is None:
        buffers = allocate(prob, q.device, with_scores)
    out_idx, out_len, out_score, ws = buffers
    indexer_topk(prob, q.contiguous(), k.contiguous(), w.contiguous().float(),
                 None if q_scale is None else q_scale.contiguous().float(),
                 None if k_scale is None else k_scale.contiguous().float(),
                 None if pool_coef is None else pool_coef.contiguous(),
                 out_idx, out_len, out_score, ws, stream)
    if with_scores:
        return out_idx, out_len, out_score
    return out_idx, out_len


def pair_overlap(idx, lens, stream=None):
    """Exact |A_2p ∩ A_2p+1| for each non-overlapping adjacent pair of rows."""
    S, width = idx.shape
    out = torch.empty((S // 2,), dtype=torch.int32, device=idx.device)
    indexer_pair_overlap(idx.contiguous(), lens.contiguous(), S, width, out, stream)
    return out


def pair_regions(idx, lens, stream=None):
    """Shared, left-only and right-only KV indices of each adjacent query pair,
    each [S/2, width] (ascending, -1 padded), and their lengths [S/2, 3]."""
    S, width = idx.shape
    outs = [torch.empty((S // 2, width), dtype=torch.int32, device=idx.device) for _ in range(3)]
    counts = torch.empty((S // 2, 3), dtype=torch.int32, device=idx.device)
    indexer_pair_regions(idx.contiguous(), lens.contiguous(), S, width, *outs, counts, stream)
    return outs[0], outs[1], outs[2], counts


def pool_keys(k, pool_coef, ratio, stream=None):
    """Pooled keys kp [T // ratio, D] bf16 from token keys k [T, D]."""
    T, D = k.shape
    out = torch.empty((T // ratio, D), dtype=torch.bfloat16, device=k.device)
    indexer_pool_keys(k.contiguous(), T, D, pool_coef.contiguous(), ratio, out, stream)
    return out


# ---------------------------------------------------------------------------
# Around the indexer: FP8 rows, the paged 8-bit cache, attention over it.
# ---------------------------------------------------------------------------

_ACT = {torch.bfloat16: ACT_BF16, torch.float16: ACT_FP16}
_CODES = (torch.uint8, torch.float8_e4m3fn)


# The checks run on every call of a decode step, so they read each attribute of a
# tensor once and build a message only where they fail.

def _act(x, what):
    a = _ACT.get(x.dtype)
    if a is None:
        raise ValueError(f"{what} must be bfloat16 or float16, not {x.dtype}")
    return a


def _tokens(x, what, device, shape, dtype):
    """Token stride of activations `shape` = (S, H, D) whose heads are packed (so a
    slice of a wider projection passes unchanged)."""
    if x.shape != shape or x.dtype != dtype or x.get_device() != device:
        raise ValueError(f"{what}: expected {tuple(shape)} {dtype} on cuda:{device}, "
                         f"got {tuple(x.shape)} {x.dtype} on {x.device}")
    S, H, D = shape
    st, sh, sd = x.stride()
    if (sd != 1 or (sh != D and H > 1)) and x.numel():
        raise ValueError(f"{what}: heads must be packed within a token (strides {x.stride()})")
    return st if S > 1 else H * D


def _ints(x, what, device, shape):
    if x.dtype != torch.int32 or x.shape != shape or not x.is_contiguous() or x.get_device() != device:
        raise ValueError(f"{what} must be a contiguous {tuple(shape)} int32 tensor on cuda:{device}")
    return x.data_ptr()


def _result(x, what, device, shape, dtype):
    if x.dtype != dtype or x.shape != shape or not x.is_contiguous() or x.get_device() != device:
        raise ValueError(f"{what} must be a contiguous {tuple(shape)} {dtype} tensor on cuda:{device}")
    return x


_NO_ROTATION = Rotation(None, 0, 0, 0)


def _rotation(table, interleaved, device):
    if table is None:
        return _NO_ROTATION
    if table.dim() != 2 or table.dtype != torch.float32 or not table.is_contiguous() or table.get_device() != device:
        raise ValueError(f"the rotation table must be a contiguous [positions, rot_dim] float32 tensor on cuda:{device}")
    rows, rot_dim = table.shape
    return Rotation(table.data_ptr(), rows, rot_dim, 1 if interleaved else 0)


def _device_of(x):
    i = x.get_device()
    if i < 0:
        raise ValueError(f"tensors must be on a CUDA device, not {x.device}")
    return i


# The current device and its stream's handle, without the objects around them
# (a few microseconds of a decode step's call).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _call(fn, device, stream, *args):
    """lib.fn(*args, stream) with `device` current, on the caller's stream or the
    device's current one."""
    if _current_device() == device:
        status = getattr(_lib, fn)(*args, _current_stream(device) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            status = getattr(_lib, fn)(*args, _current_stream(device) if stream is None else stream.cuda_stream)
    if status != 0:
        raise IndexerError(fn, status)


def _new(stream, like, shape, dtype):
    """An uninitialised tensor for the call, on the device of `like`: on the call's
    stream, so that its memory is not handed to other work while the call may
    still use it.  shape None: that of `like`."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _new(None, like, shape, dtype)
    if shape is None:
        return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)
    return like.new_empty(shape, dtype=dtype)


def rope_table(positions: int, rot_dim: int, base: float = 10000.0, device="cuda"):
    """Rotation table [positions, rot_dim] float32 (cosines, then sines) of the
    angles position * base^(-2i/rot_dim), computed in binary64."""
    inv = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def rotate_quantise(x, positions=None, table=None, interleaved=False, out=None, status=None, stream=None):
    """Rotated rows in the indexer's FP8 form: x [S, H, D] bf16 or fp16 ->
    (codes [S, H, D] uint8, scale [S, H] float32), to be passed to `topk` as q
    and q_scale (with H = 1, as k and k_scale rows).

    positions [S] int32 (None: 0, 1, ...), table as from `rope_table` (None: no
    rotation).  out = (codes, scale) writes into given contiguous tensors, e.g.
    the next rows of the indexer's key arrays.  status: a [1] int32 tensor that
    bits are ORed into.
    """
    device = _device_of(x)
    act = _act(x, "x")
    shape = x.shape
    if len(shape) != 3:
        raise ValueError(f"x must be [S, H, D], not {tuple(shape)}")
    S, H, D = shape
    stride = _tokens(x, "x", device, shape, x.dtype)
    rot = _rotation(table, interleaved, device)
    pos = None if positions is None else _ints(positions, "positions", device, (S,))
    if out is None:
        codes = _new(stream, x, None, torch.uint8)
        scale = _new(stream, x, (S, H), torch.float32)
    else:
        codes, scale = out
        if not (codes.dtype in _CODES and codes.is_contiguous() and codes.numel() == S * H * D
                and codes.get_device() == device and scale.dtype == torch.float32 and scale.is_contiguous()
                and scale.numel() == S * H and scale.get_device() == device):
            raise ValueError("out must be contiguous codes (S*H*D of them) and float32 scales (S*H) on x's device")
    _call("indexer_rotate_quantise", device, stream, x.data_ptr(), S, H, D, act, stride, pos, rot, codes.data_ptr(),
          scale.data_ptr(), None if status is None else _ints(status, "status", device, (1,)))
    return codes, scale


class KVCache(NamedTuple):
    """A paged 8-bit cache: k and v [pages, page_size, heads, D] e4m3 codes
    (uint8 or float8_e4m3fn; any strides that both share and that keep a head's D
    codes together, so [pages, heads, page_size, D] memory can be given
    transposed), k_scale and v_scale [pages, page_size // block, heads] float32."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    def descriptor(self) -> CacheDesc:
        k, v, ks, vs = self
        shape, strides = k.shape, k.stride()
        if (len(shape) != 4 or v.shape != shape or v.stride() != strides or strides[3] != 1 or k.dtype not in _CODES
                or v.dtype not in _CODES or v.get_device() != k.get_device()):
            raise ValueError("k and v must be alike: [pages, page_size, heads, D] e4m3 codes, the last dimension "
                             "contiguous")
        pages, page_size, heads, D = shape
        sshape = ks.shape
        blocks = sshape[1] if len(sshape) == 3 else 0
        if (sshape != (pages, blocks, heads) or vs.shape != sshape or not 0 < blocks <= page_size
                or page_size % blocks or ks.dtype != torch.float32 or vs.dtype != torch.float32
                or not (ks.is_contiguous() and vs.is_contiguous())
                or not ks.get_device() == vs.get_device() == k.get_device()):
            raise ValueError("k_scale and v_scale must be contiguous [pages, page_size // block, heads] float32 tensors "
                             "on the device of k")
        return CacheDesc(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), pages, strides[0], strides[1],
                         strides[2], page_size, page_size // blocks, heads, D)


def allocate_cache(pages, page_size, heads, D, block=16, device="cuda") -> KVCache:
    """A cache for pages * page_size tokens, uninitialised (what a sequence has
    not been given by `cache_append` is never read)."""
    if block < 1 or page_size % block:
        raise ValueError("page_size must be a multiple of block")
    k, v = (torch.empty((pages, page_size, heads, D), dtype=torch.uint8, device=device) for _ in range(2))
    ks, vs = (torch.empty((pages, page_size // block, heads), dtype=torch.float32, device=device) for _ in range(2))
    return KVCache(k, v, ks, vs)


def _sequences(S, cu_q, kv_len, page_table, device) -> Sequences:
    B = kv_len.numel()
    shape = page_table.shape
    if (len(shape) != 2 or shape[0] != B or page_table.dtype != torch.int32 or page_table.get_device() != device
            or (page_table.stride(1) != 1 and shape[1] > 1)):
        raise ValueError(f"page_table must be a [{B}, pages] int32 tensor on cuda:{device} with contiguous rows")
    return Sequences(S, _ints(cu_q, "cu_q", device, (B + 1,)), _ints(kv_len, "kv_len", device, (B,)),
                     page_table.data_ptr(), page_table.stride(0) if B > 1 else shape[1], shape[1], B)


def cache_append(cache: KVCache, k, v, cu_q, kv_len, page_table, table=None, interleaved=False, q=None, q_out=None,
                 status=None, stream=None):
    """Appends the rows of k and v [S, heads, D] (bf16 or fp16) to the cache, k
    rotated by its position on the way, quantised with a power-of-two scale per
    block of tokens and head.

    Rows cu_q[b] .. cu_q[b+1]-1 are the newest tokens of sequence b, whose
    length with them is kv_len[b]; its position p lies at offset p % page_size of
    page page_table[b, p // page_size].  With q [S, Hq, D] given, its rotated
    rows are returned (in q_out, if given); rows that belong to no sequence are
    left as they were.  status: a [1] int32 tensor that bits are ORed into.
    """
    device = _device_of(cache.k)
    desc = cache.descriptor()
    S, dtype = k.shape[0], k.dtype
    act = _act(k, "k")
    shape = (S, desc.heads, desc.D)
    stride = _tokens(k, "k", device, shape, dtype)
    if _tokens(v, "v", device, shape, dtype) != stride:
        raise ValueError("k and v must have the same strides")
    seqs = _sequences(S, cu_q, kv_len, page_table, device)
    rot = _rotation(table, interleaved, device)
    q_heads = q_stride = 0
    qp = qo = None
    if q is not None:
        shape = q.shape
        q_heads = shape[1] if len(shape) == 3 else 0
        q_stride = _tokens(q, "q", device, (S, q_heads, desc.D), dtype)
        if q_out is None:
            q_out = _new(stream, q, None, dtype)
        else:
            _result(q_out, "q_out", device, shape, dtype)
        qp, qo = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    _call("indexer_cache_append", device, stream, desc, seqs, k.data_ptr(), v.data_ptr(), stride, act, rot, qp, q_heads,
          q_stride, qo, None if status is None else _ints(status, "status", device, (1,)))
    return q_out


def cache_attend(cache: KVCache, q, cu_q, kv_len, page_table, scale=None, causal=True, selected=None, max_q=0,
                 with_lse=False, out=None, workspace=None, status=None, stream=None, kernel=ATTEND_AUTO):
    """Attention of q [S, Hq, D] (bf16 or fp16, already rotated) over the cache:
    out [S, Hq, D], and with_lse=True also the log-sum-exp [S, Hq] float32.

    Sequences as in `cache_append` (kv_len counts the newest rows, already
    appended).  A row sees its sequence's positions up to its own, or with
    causal=False all of them; selected = (idx [S, W], len [S]) int32, as `topk`
    returns them for positions counted from the sequence's start, narrows that to
    the positions named.  A row that sees nothing gives 0 and -inf.  scale
    defaults to D ** -0.5.  max_q: rows of the longest sequence, if known (it
    chooses the kernel: results may differ by roundings; or name it by `kernel`).
    Left at 0, all S rows count as one sequence's: give it for a batch.
    workspace: a uint8 tensor kept by the caller (its size from
    `cache_attend_workspace_bytes`); by default it is allocated for the call.
    """
    device = _device_of(cache.k)
    desc = cache.descriptor()
    act, dtype = _act(q, "q"), q.dtype
    shape = q.shape
    S, Hq = shape[0], shape[1] if len(shape) == 3 else 0
    stride = _tokens(q, "q", device, (S, Hq, desc.D), dtype)
    seqs = _sequences(S, cu_q, kv_len, page_table, device)
    si = sl = None
    width = 0
    if selected is not None:
        idx, lens = selected
        width = idx.shape[-1]
        if width < 1:
            raise ValueError("selected indices must be [S, W] with W > 0")
        si, sl = _ints(idx, "selected indices", device, (S, width)), _ints(lens, "selected lengths", device, (S,))
    att = Attention(Hq, act, 1 if causal else 0, width, max_q, scale if scale is not None else 1 / math.sqrt(desc.D),
                    kernel)
    if workspace is None:
        workspace = _new(stream, q, (_attend_workspace(device, desc, seqs, att),), torch.uint8)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on cuda:{device}")
    if out is None:
        out = _new(stream, q, None, dtype)
    else:
        _result(out, "out", device, shape, dtype)
    lse = _new(stream, q, (S, Hq), torch.float32) if with_lse else None
    _call("indexer_cache_attend", device, stream, desc, seqs, att, q.data_ptr(), stride, si, sl, out.data_ptr(),
          None if lse is None else lse.data_ptr(),
          None if status is None else _ints(status, "status", device, (1,)), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return (out, lse) if with_lse else out


_attend_sizes = {}   # workspace bytes by what they depend on: the device and the shapes


def _attend_workspace(device, desc, seqs, att) -> int:
    key = (device, desc.heads, desc.D, desc.page_size, desc.block, seqs.S, seqs.B, seqs.table_pages, att.Hq, att.act,
           att.sel_width, att.max_q, att.kernel)
    size = _attend_sizes.get(key)
    if size is not None:
        return size
    n = ctypes.c_size_t()
    with torch.cuda.device(device):
        status = _lib.indexer_cache_attend_workspace_bytes(desc, seqs, att, n)
    if status != 0:
        raise IndexerError("indexer_cache_attend_workspace_bytes", status)
    if len(_attend_sizes) >= 4096:
        _attend_sizes.clear()
    _attend_sizes[key] = n.value
    return n.value


def cache_attend_workspace_bytes(cache: KVCache, q, cu_q, kv_len, page_table, selected_width=0, max_q=0,
                                 kernel=ATTEND_AUTO) -> int:
    """Bytes of workspace for `cache_attend` on these tensors' shapes."""
    device = _device_of(cache.k)
    desc = cache.descriptor()
    return _attend_workspace(device, desc, _sequences(q.shape[0], cu_q, kv_len, page_table, device),
                             Attention(q.shape[1], _act(q, "q"), 1, selected_width, max_q, 1.0, kernel))
