"""Python binding of the HyLRA C-ABI library (argument marshalling only).

Every function here forwards to the entry point of the same name in
``libhylra.so`` (declared in ``include/hylra.h``).  Device buffers are torch
CUDA tensors (only their ``data_ptr()`` crosses the boundary); host buffers
for the policy functions are numpy arrays.  There is no fallback: if the
shared library is missing or a call fails, an exception is raised.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhylra.so")

BLOCK_TOKENS = 128
HEAD_DIM = 128
MAX_GROUP = 8
MAX_BATCH = 1024
MAX_TOPK = 1024
MAX_SEQLEN = 262144

BF16 = 0
FP32 = 1
FP16 = 2  # paged calls only

STATUS_BAD_SEQLEN = 0x1
STATUS_BAD_INDEX = 0x2
STATUS_DUP_INDEX = 0x4
STATUS_NONFINITE = 0x8
STATUS_TIMEOUT = 0x10
STATUS_NO_PAGES = 0x20

ERRORS = {0: "HYLRA_OK", -1: "HYLRA_ERR_INVALID", -2: "HYLRA_ERR_UNSUPPORTED",
          -3: "HYLRA_ERR_CUDA", -4: "HYLRA_ERR_WORKSPACE"}

EXPORTS = ("hylra_workspace_bytes", "hylra_workspace_init", "hylra_decode_full",
           "hylra_decode_reuse", "hylra_decode_step", "hylra_decode_step_host",
           "hylra_similarity", "hylra_dp_policy", "hylra_read_status", "hylra_strerror",
           "hylra_version", "hylra_decode_full_noalloc", "hylra_static_policy",
           "hylra_stage_bytes", "hylra_gather_blocks", "hylra_decode_reuse_staged",
           "hylra_decode_step_offload", "hylra_overlap_counts",
           "hylra_similarity_from_counts", "hylra_set_wait_limit", "hylra_token_scores",
           "hylra_token_topk", "hylra_paged_workspace_bytes", "hylra_paged_tables",
           "hylra_paged_append", "hylra_paged_decode", "hylra_paged_select",
           "hylra_paged_decode_topk")


class HylraError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {ERRORS.get(code, code)} ({code})")
        self.code = code


class Shape(ctypes.Structure):
    """Mirror of hylra_shape_t."""

    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("max_seqlen", ctypes.c_int32),
                ("kv_capacity", ctypes.c_int64), ("total_tokens", ctypes.c_int64),
                ("seq_offsets", ctypes.c_void_p)]


class PagedShape(ctypes.Structure):
    """Mirror of hylra_paged_t."""

    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("softmax_scale", ctypes.c_float)]


def make_shape(batch, num_q_heads, num_kv_heads, topk, max_seqlen, dtype=BF16, kv_capacity=0,
               total_tokens=0, seq_offsets=None, head_dim=HEAD_DIM,
               block_size=BLOCK_TOKENS) -> Shape:
    """Build a Shape; ``seq_offsets`` is a device int64 tensor (packed layout) or None."""
    ptr = None if seq_offsets is None else int(seq_offsets.data_ptr())
    return Shape(batch, num_q_heads, num_kv_heads, head_dim, block_size, topk, dtype,
                 max_seqlen, kv_capacity, total_tokens, ptr)


_lib: Optional[ctypes.CDLL] = None


def load() -> ctypes.CDLL:
    """Load libhylra.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m kv_cache_sparsity_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, S, I32, I64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
    SP, PP = ctypes.POINTER(Shape), ctypes.POINTER(PagedShape)
    sig = {
        "hylra_workspace_bytes": [SP, ctypes.POINTER(ctypes.c_size_t)],
        "hylra_workspace_init": [P, S, P],
        "hylra_decode_full": [SP, P, P, P, P, P, P, P, S, P],
        "hylra_decode_reuse": [SP, P, P, P, P, P, P, P, S, P],
        "hylra_decode_step": [SP, I32, P, P, P, P, P, P, P, P, S, P],
        "hylra_decode_step_host": [SP, I32, P, P, P, P, P, P, P, P, P, P, P, S, P],
        "hylra_similarity": [I32, I32, I32, P, P],
        "hylra_overlap_counts": [I32, I32, I32, P, P, P],
        "hylra_similarity_from_counts": [I32, P, P, P],
        "hylra_dp_policy": [I32, P, ctypes.c_double, P, ctypes.POINTER(I32),
                            ctypes.POINTER(ctypes.c_double)],
        "hylra_read_status": [P, ctypes.POINTER(ctypes.c_uint32), ctypes.c_int, P],
        "hylra_decode_full_noalloc": [SP, P, P, P, P, P, P, P, P],
        "hylra_static_policy": [I32, I32, P, ctypes.POINTER(I32)],
        "hylra_stage_bytes": [SP, ctypes.POINTER(ctypes.c_size_t)],
        "hylra_gather_blocks": [SP, P, P, P, P, P, P, P],
        "hylra_decode_reuse_staged": [SP, P, P, P, P, P, P, P, S, P],
        "hylra_decode_step_offload": [SP, I32, P, P, P, P, P, P, P, P, P, P, P, S, P],
        "hylra_set_wait_limit": [I64],
        "hylra_token_scores": [SP, P, P, P, P, P, P, P, P, S, P],
        "hylra_token_topk": [I32, I32, P, P, I32, P],
        "hylra_paged_workspace_bytes": [PP, ctypes.POINTER(ctypes.c_size_t)],
        "hylra_paged_tables": [PP, P, P, P, I32, P, P, P, P, P, I32, P, P, S, P],
        "hylra_paged_append": [PP, P, P, I64, P, I32, P, P, P, P, S, P],
        "hylra_paged_decode": [PP, P, P, P, P, P, P, P, P, S, P],
        "hylra_paged_select": [PP, P, P, P, P, I32, I32, I32, P, P, S, P],
        "hylra_paged_decode_topk": [PP, P, P, P, P, P, P, I32, P, P, P, S, P],
        "hylra_strerror": [ctypes.c_int],
        "hylra_version": [],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_char_p if name == "hylra_strerror" else ctypes.c_int
    _lib = lib
    return lib


def _check(rc: int, what: str):
    if rc != 0:
        raise HylraError(rc, what)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    return int(t.data_ptr())


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def version() -> int:
    return load().hylra_version()


def strerror(code: int) -> str:
    return load().hylra_strerror(code).decode()


def workspace_bytes(shape: Shape) -> int:
    n = ctypes.c_size_t(0)
    _check(load().hylra_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)),
           "hylra_workspace_bytes")
    return n.value


def _on_device_of(ws):
    """Context in which the workspace's device is the current one."""
    import torch
    dev = ws.get_device()
    if dev < 0 or dev == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def workspace_init(ws, stream=None):
    """Zero a workspace, on its device's current stream unless given another."""
    with _on_device_of(ws):
        _check(load().hylra_workspace_init(_ptr(ws), ws.numel() * ws.element_size(),
                                           _stream(stream)), "hylra_workspace_init")


def decode_full(shape: Shape, q, K, V, seqlens, out, topk_out, ws, stream=None):
    _check(load().hylra_decode_full(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(V),
                                    _ptr(seqlens), _ptr(out), _ptr(topk_out), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream)),
           "hylra_decode_full")


def decode_reuse(shape: Shape, q, K, V, seqlens, topk_in, out, ws, stream=None):
    _check(load().hylra_decode_reuse(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(V),
                                     _ptr(seqlens), _ptr(topk_in), _ptr(out), _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream)),
           "hylra_decode_reuse")


def _ptr_array(ts):
    arr = (ctypes.c_void_p * len(ts))(*[_ptr(t) for t in ts])
    return arr


def decode_step(shape: Shape, policy: Sequence[int], qs, Ks, Vs, seqlens, outs, topk, ws,
                stream=None):
    L = len(policy)
    pol = (ctypes.c_uint8 * L)(*[int(x) for x in policy])
    _check(load().hylra_decode_step(ctypes.byref(shape), L, pol, _ptr_array(qs), _ptr_array(Ks),
                                    _ptr_array(Vs), _ptr(seqlens), _ptr_array(outs), _ptr(topk),
                                    _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "hylra_decode_step")


def decode_step_host(shape: Shape, policy: Sequence[int], q_host, q_dev, Ks, Vs, seqlens,
                     out_dev, out_host, topk_dev, topk_host, ws, stream=None):
    """Step with per-step inputs/outputs in host memory (pinned torch CPU tensors)."""
    L = len(policy)
    pol = (ctypes.c_uint8 * L)(*[int(x) for x in policy])
    _check(load().hylra_decode_step_host(ctypes.byref(shape), L, pol, _ptr(q_host), _ptr(q_dev),
                                         _ptr_array(Ks), _ptr_array(Vs), _ptr(seqlens),
                                         _ptr(out_dev), _ptr(out_host), _ptr(topk_dev),
                                         _ptr(topk_host), _ptr(ws),
                                         ws.numel() * ws.element_size(), _stream(stream)),
           "hylra_decode_step_host")


def decode_full_noalloc(shape: Shape, q, K, V, seqlens, out, topk_out, status_out=None,
                        stream=None):
    """Reset layer on the library's built-in scratch (no workspace argument)."""
    _check(load().hylra_decode_full_noalloc(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(V),
                                            _ptr(seqlens), _ptr(out), _ptr(topk_out),
                                            _ptr(status_out), _stream(stream)),
           "hylra_decode_full_noalloc")


def set_wait_limit(cycles: int):
    """Limit (SM clocks) of the kernels' bounded waits for later launches;
    cycles <= 0 restores the default."""
    _check(load().hylra_set_wait_limit(int(cycles)), "hylra_set_wait_limit")


def read_status(ws, clear: bool = True, stream=None) -> int:
    """The workspace's status word, read on its device's current stream unless given another."""
    v = ctypes.c_uint32(0)
    with _on_device_of(ws):
        _check(load().hylra_read_status(_ptr(ws), ctypes.byref(v), int(clear), _stream(stream)),
               "hylra_read_status")
    return v.value


def token_scores(shape: Shape, q, K, V, seqlens, out, topk_out, scores, ws, stream=None):
    """Reset layer + per-token attention mass (scores: device fp32 [B][Hkv][max_seqlen])."""
    _check(load().hylra_token_scores(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(V),
                                     _ptr(seqlens), _ptr(out), _ptr(topk_out), _ptr(scores),
                                     _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "hylra_token_scores")


def token_topk(scores: np.ndarray, k: int, lengths=None) -> np.ndarray:
    """scores: fp32 [U, n] host array (lengths: int32 [U] valid entries or None)
    -> int32 [U, k] indices in rank order, -1 padded."""
    sc = np.ascontiguousarray(scores, dtype=np.float32)
    U, n = sc.shape
    ln = None if lengths is None else np.ascontiguousarray(lengths, dtype=np.int32)
    out = np.zeros((U, k), dtype=np.int32)
    _check(load().hylra_token_topk(U, n, sc.ctypes.data, None if ln is None else ln.ctypes.data,
                                   int(k), out.ctypes.data), "hylra_token_topk")
    return out


def similarity(topk: np.ndarray) -> np.ndarray:
    """topk: int32 [L, S, k] host array -> M [L, L] float64."""
    t = np.ascontiguousarray(topk, dtype=np.int32)
    L, S, k = t.shape
    M = np.zeros((L, L), dtype=np.float64)
    _check(load().hylra_similarity(L, S, k, t.ctypes.data, M.ctypes.data), "hylra_similarity")
    return M


def overlap_counts(topk: np.ndarray):
    """topk: int32 [L, S, k] host array -> (inter [L, L] int64, total [L] int64)."""
    t = np.ascontiguousarray(topk, dtype=np.int32)
    L, S, k = t.shape
    inter = np.zeros((L, L), dtype=np.int64)
    total = np.zeros(L, dtype=np.int64)
    _check(load().hylra_overlap_counts(L, S, k, t.ctypes.data, inter.ctypes.data,
                                       total.ctypes.data), "hylra_overlap_counts")
    return inter, total


def similarity_from_counts(inter: np.ndarray, total: np.ndarray) -> np.ndarray:
    """(inter [L, L], total [L]) int64 host arrays -> M [L, L] float64."""
    i = np.ascontiguousarray(inter, dtype=np.int64)
    t = np.ascontiguousarray(total, dtype=np.int64)
    L = t.shape[0]
    M = np.zeros((L, L), dtype=np.float64)
    _check(load().hylra_similarity_from_counts(L, i.ctypes.data, t.ctypes.data, M.ctypes.data),
           "hylra_similarity_from_counts")
    return M


def dp_policy(M: np.ndarray, theta: float):
    """-> (policy tuple, resets, cumulative similarity)."""
    m = np.ascontiguousarray(M, dtype=np.float64)
    L = m.shape[0]
    pol = np.zeros(L, dtype=np.uint8)
    R = ctypes.c_int32(0)
    S = ctypes.c_double(0.0)
    _check(load().hylra_dp_policy(L, m.ctypes.data, float(theta), pol.ctypes.data,
                                  ctypes.byref(R), ctypes.byref(S)), "hylra_dp_policy")
    return tuple(int(x) for x in pol), R.value, S.value


def static_policy(num_layers: int, period: int):
    """-> (policy tuple, resets): a reset every `period` layers (Jump3: 3)."""
    pol = np.zeros(num_layers, dtype=np.uint8)
    R = ctypes.c_int32(0)
    _check(load().hylra_static_policy(int(num_layers), int(period), pol.ctypes.data,
                                      ctypes.byref(R)), "hylra_static_policy")
    return tuple(int(x) for x in pol), R.value


def stage_bytes(shape: Shape) -> int:
    n = ctypes.c_size_t(0)
    _check(load().hylra_stage_bytes(ctypes.byref(shape), ctypes.byref(n)), "hylra_stage_bytes")
    return n.value


def gather_blocks(shape: Shape, K_host, V_host, seqlens, topk_in, K_stage, V_stage, stream=None):
    """K_host / V_host: pinned torch CPU tensors (the device reads them in place)."""
    _check(load().hylra_gather_blocks(ctypes.byref(shape), _ptr(K_host), _ptr(V_host),
                                      _ptr(seqlens), _ptr(topk_in), _ptr(K_stage), _ptr(V_stage),
                                      _stream(stream)), "hylra_gather_blocks")


def decode_reuse_staged(shape: Shape, q, K_stage, V_stage, seqlens, topk_in, out, ws,
                        stream=None):
    _check(load().hylra_decode_reuse_staged(ctypes.byref(shape), _ptr(q), _ptr(K_stage),
                                            _ptr(V_stage), _ptr(seqlens), _ptr(topk_in),
                                            _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
                                            _stream(stream)), "hylra_decode_reuse_staged")


def decode_step_offload(shape: Shape, policy: Sequence[int], qs, Ks, Vs, offloaded, seqlens,
                        outs, topk, K_stage, V_stage, ws, stream=None):
    """Ks[l] / Vs[l] of layers with offloaded[l] = 1 are pinned torch CPU tensors;
    K_stage / V_stage each hold two staging slots (2 x stage_bytes bytes)."""
    L = len(policy)
    pol = (ctypes.c_uint8 * L)(*[int(x) for x in policy])
    off = (ctypes.c_uint8 * L)(*[int(x) for x in offloaded])
    _check(load().hylra_decode_step_offload(ctypes.byref(shape), L, pol, _ptr_array(qs),
                                            _ptr_array(Ks), _ptr_array(Vs), off, _ptr(seqlens),
                                            _ptr_array(outs), _ptr(topk), _ptr(K_stage),
                                            _ptr(V_stage), _ptr(ws),
                                            ws.numel() * ws.element_size(), _stream(stream)),
           "hylra_decode_step_offload")


# ------------------------------------------------------------- paged cache
#
# Device buffers are torch CUDA tensors of one device; the calls run on that
# device's current stream unless given another.  A tensor of the wrong type,
# shape or layout raises ValueError before the library is called.


def make_paged_shape(batch, num_q_heads, num_kv_heads, page_size, num_pages, max_pages,
                     dtype=BF16, head_dim=HEAD_DIM, pool=None, scale=0.0) -> PagedShape:
    """Build a PagedShape.  ``pool``: the K pool as a [num_pages, num_kv_heads,
    page_size, head_dim] tensor of any strides (the V pool has the same), for
    example ``pages.transpose(1, 2)`` of a [page, row, head, d] array; without
    it the pools are contiguous in that order.  ``scale`` 0: 1/sqrt(head_dim)."""
    strides = (num_kv_heads * page_size * head_dim, page_size * head_dim, head_dim)
    if pool is not None:
        want = (num_pages, num_kv_heads, page_size, head_dim)
        if tuple(pool.shape) != want:
            raise ValueError(f"pool: shape {tuple(pool.shape)}, expected {want}")
        if pool.stride(3) != 1:
            raise ValueError("pool: the elements of a row must be adjacent")
        strides = pool.stride()[:3]
    return PagedShape(batch, num_q_heads, num_kv_heads, head_dim, page_size, dtype, num_pages,
                      max_pages, *strides, scale)


def paged_workspace_bytes(shape: PagedShape) -> int:
    n = ctypes.c_size_t(0)
    _check(load().hylra_paged_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)),
           "hylra_paged_workspace_bytes")
    return n.value


def _want(what, t, dtype, shape, dev, dense=True):
    """Raise unless t is a tensor of this type and shape on device index dev (contiguous if dense)."""
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{what}: {t.dtype} {tuple(t.shape)}, expected {dtype} {shape}")
    if t.get_device() != dev:
        raise ValueError(f"{what}: on {t.device}, expected cuda:{dev}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")


# A decode step makes a handful of these calls per layer, and a small one costs
# the GPU less than its checks cost the host: each call tests all its tensors in
# one expression, against tuples made once per shape, and looks for the one to
# name only when that fails.


class _Forms:
    """What the tensors of a PagedShape's calls must look like."""

    def __init__(self, s: PagedShape):
        import torch
        if s.dtype not in (BF16, FP16):  # as the library answers for such a shape
            raise HylraError(-2 if s.dtype == FP32 else -1, f"PagedShape.dtype {s.dtype}")
        self.torch = torch
        self.dtype = torch.bfloat16 if s.dtype == BF16 else torch.float16
        self.pool = (s.num_pages, s.num_kv_heads, s.page_size, s.head_dim)
        self.strides = (s.page_stride, s.head_stride, s.token_stride, 1)
        self.q = (s.batch, s.num_q_heads, s.head_dim)
        self.table = (s.batch, s.max_pages)
        self.lens = (s.batch,)
        self.lse = (s.batch, s.num_q_heads)
        self.heads = (s.batch, s.num_kv_heads)
        self.means = (s.num_pages, s.num_kv_heads, s.head_dim)


@functools.lru_cache(maxsize=256)
def _forms_of(fields: bytes) -> _Forms:
    return _Forms(PagedShape.from_buffer_copy(fields))


def _forms(s: PagedShape) -> _Forms:
    # by the fields' values: the shape may be changed, copied and pickled between calls
    return _forms_of(bytes(s))


def _want_pools(f: _Forms, K, V, dev):
    if (K.dtype is f.dtype and V.dtype is f.dtype and K.shape == f.pool and V.shape == f.pool
            and K.stride() == f.strides and V.stride() == f.strides and K.get_device() == dev
            and V.get_device() == dev):
        return
    for what, t in (("K_pages", K), ("V_pages", V)):
        _want(what, t, f.dtype, f.pool, dev, dense=False)
        # the stride of a dimension of one element has no meaning
        if any(n > 1 and a != b for n, a, b in zip(f.pool, t.stride(), f.strides)):
            raise ValueError(f"{what}: strides {t.stride()} differ from the shape's {f.strides}")


def _want_query(f: _Forms, q, block_table, seqlens, dev):
    i32 = f.torch.int32
    if (q.dtype is f.dtype and block_table.dtype is i32 and seqlens.dtype is i32
            and q.shape == f.q and block_table.shape == f.table and seqlens.shape == f.lens
            and q.is_contiguous() and block_table.is_contiguous() and seqlens.is_contiguous()
            and q.get_device() == dev and block_table.get_device() == dev
            and seqlens.get_device() == dev):
        return
    _want("q", q, f.dtype, f.q, dev)
    _want("block_table", block_table, i32, f.table, dev)
    _want("seqlens", seqlens, i32, f.lens, dev)


def _want_result(f: _Forms, out, lse, dev):
    f32 = f.torch.float32
    if not (out.dtype is f32 and out.shape == f.q and out.is_contiguous()
            and out.get_device() == dev):
        _want("out", out, f32, f.q, dev)
    if lse is not None and not (lse.dtype is f32 and lse.shape == f.lse and lse.is_contiguous()
                                and lse.get_device() == dev):
        _want("lse", lse, f32, f.lse, dev)


def _paged_call(torch, entry, ws, dev, stream, *args):
    """entry(*args, workspace, stream), on the workspace's device."""
    if dev < 0 or not ws.is_contiguous():
        raise ValueError("ws: must be a contiguous CUDA tensor")
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _paged_call(torch, entry, ws, dev, stream, *args)
    st = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
    rc = entry(*args, ws.data_ptr(), ws.nbytes, st)
    if rc:
        raise HylraError(rc, entry.__name__)


def paged_tables(shape: PagedShape, cached_lens, new_lens, free_pages, free_count, block_table,
                 seqlens_out, cu_new, slot_map, free_count_out, ws, stream=None):
    """Pages, slots and lengths of a step's new tokens (all int32)."""
    f = _forms(shape)
    dev, i32, B = ws.get_device(), f.torch.int32, f.lens[0]
    nfree, nslots = free_pages.numel(), slot_map.numel()
    if not (cached_lens.dtype is i32 and new_lens.dtype is i32 and free_pages.dtype is i32
            and free_count.dtype is i32 and block_table.dtype is i32 and seqlens_out.dtype is i32
            and cu_new.dtype is i32 and slot_map.dtype is i32 and free_count_out.dtype is i32
            and cached_lens.shape == f.lens and new_lens.shape == f.lens
            and free_pages.dim() == 1 and free_count.numel() == 1 and block_table.shape == f.table
            and seqlens_out.shape == f.lens and cu_new.numel() == B + 1 and slot_map.dim() == 1
            and free_count_out.numel() == 1 and cached_lens.is_contiguous()
            and new_lens.is_contiguous() and free_pages.is_contiguous()
            and block_table.is_contiguous() and seqlens_out.is_contiguous()
            and cu_new.is_contiguous() and slot_map.is_contiguous()
            and cached_lens.get_device() == dev and new_lens.get_device() == dev
            and free_pages.get_device() == dev and free_count.get_device() == dev
            and block_table.get_device() == dev and seqlens_out.get_device() == dev
            and cu_new.get_device() == dev and slot_map.get_device() == dev
            and free_count_out.get_device() == dev):
        for what, t, n in (("cached_lens", cached_lens, f.lens), ("new_lens", new_lens, f.lens),
                           ("free_pages", free_pages, (nfree,)), ("free_count", free_count, (1,)),
                           ("block_table", block_table, f.table),
                           ("seqlens_out", seqlens_out, f.lens), ("cu_new", cu_new, (B + 1,)),
                           ("slot_map", slot_map, (nslots,)),
                           ("free_count_out", free_count_out, (1,))):
            _want(what, t, i32, n, dev)
    _paged_call(f.torch, (_lib or load()).hylra_paged_tables, ws, dev, stream, ctypes.byref(shape),
                cached_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(), nfree,
                free_count.data_ptr(), block_table.data_ptr(), seqlens_out.data_ptr(),
                cu_new.data_ptr(), slot_map.data_ptr(), nslots, free_count_out.data_ptr())


def paged_append(shape: PagedShape, K_new, V_new, slot_map, K_pages, V_pages, key_means, ws,
                 stream=None):
    """K_new / V_new [T, Hkv, d] (each token's heads adjacent, tokens at any stride) into the
    pools; key_means [num_pages, Hkv, d] or None."""
    f = _forms(shape)
    dev, t, n = ws.get_device(), f.dtype, slot_map.numel()
    H, d = f.means[1], f.means[2]
    rows, ks, vs = (n, H, d), K_new.stride(), V_new.stride()
    if not (slot_map.dtype is f.torch.int32 and slot_map.dim() == 1 and slot_map.is_contiguous()
            and slot_map.get_device() == dev and K_new.dtype is t and V_new.dtype is t
            and K_new.shape == rows and V_new.shape == rows and K_new.get_device() == dev
            and V_new.get_device() == dev):
        _want("slot_map", slot_map, f.torch.int32, (n,), dev)
        _want("K_new", K_new, t, rows, dev, dense=False)
        _want("V_new", V_new, t, rows, dev, dense=False)
    if n and (ks[2] != 1 or vs[2] != 1 or (H > 1 and (ks[1] != d or vs[1] != d))):
        raise ValueError("K_new and V_new: a token's heads must be adjacent")
    if n > 1 and ks[0] != vs[0]:
        raise ValueError("K_new and V_new must have the same token stride")
    _want_pools(f, K_pages, V_pages, dev)
    if key_means is not None and not (key_means.dtype is t and key_means.shape == f.means
                                      and key_means.is_contiguous()
                                      and key_means.get_device() == dev):
        _want("key_means", key_means, t, f.means, dev)
    _paged_call(f.torch, (_lib or load()).hylra_paged_append, ws, dev, stream, ctypes.byref(shape),
                K_new.data_ptr(), V_new.data_ptr(), ks[0] if n > 1 else H * d,
                slot_map.data_ptr(), n, K_pages.data_ptr(), V_pages.data_ptr(),
                None if key_means is None else key_means.data_ptr())


def paged_decode(shape: PagedShape, q, K_pages, V_pages, block_table, seqlens, out, ws, lse=None,
                 stream=None):
    """Attention of one query token per sequence over its pages; lse: fp32 [B, Hq] or None."""
    f, dev = _forms(shape), ws.get_device()
    _want_query(f, q, block_table, seqlens, dev)
    _want_pools(f, K_pages, V_pages, dev)
    _want_result(f, out, lse, dev)
    _paged_call(f.torch, (_lib or load()).hylra_paged_decode, ws, dev, stream, ctypes.byref(shape),
                q.data_ptr(), K_pages.data_ptr(), V_pages.data_ptr(), block_table.data_ptr(),
                seqlens.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr())


def _want_list(f: _Forms, page_idx, dev):
    k = page_idx.shape[-1]
    if not (page_idx.dtype is f.torch.int32 and page_idx.shape == (*f.heads, k)
            and page_idx.is_contiguous() and page_idx.get_device() == dev):
        _want("page_idx", page_idx, f.torch.int32, (*f.heads, k), dev)
    return k


def paged_select(shape: PagedShape, q, key_means, block_table, seqlens, page_idx, ws, sink=1,
                 recent=1, stream=None):
    """The most promising pages of each (sequence, KV head) into page_idx int32 [B, Hkv, k]."""
    f, dev = _forms(shape), ws.get_device()
    _want_query(f, q, block_table, seqlens, dev)
    if not (key_means.dtype is f.dtype and key_means.shape == f.means
            and key_means.is_contiguous() and key_means.get_device() == dev):
        _want("key_means", key_means, f.dtype, f.means, dev)
    k = _want_list(f, page_idx, dev)
    _paged_call(f.torch, (_lib or load()).hylra_paged_select, ws, dev, stream, ctypes.byref(shape),
                q.data_ptr(), key_means.data_ptr(), block_table.data_ptr(), seqlens.data_ptr(),
                k, sink, recent, page_idx.data_ptr())


def paged_decode_topk(shape: PagedShape, q, K_pages, V_pages, block_table, seqlens, page_idx, out,
                      ws, lse=None, stream=None):
    """paged_decode over the pages listed in page_idx int32 [B, Hkv, k]."""
    f, dev = _forms(shape), ws.get_device()
    _want_query(f, q, block_table, seqlens, dev)
    _want_pools(f, K_pages, V_pages, dev)
    k = _want_list(f, page_idx, dev)
    _want_result(f, out, lse, dev)
    _paged_call(f.torch, (_lib or load()).hylra_paged_decode_topk, ws, dev, stream, ctypes.byref(shape),
                q.data_ptr(), K_pages.data_ptr(), V_pages.data_ptr(), block_table.data_ptr(),
                seqlens.data_ptr(), page_idx.data_ptr(), k, out.data_ptr(),
                None if lse is None else lse.data_ptr())
