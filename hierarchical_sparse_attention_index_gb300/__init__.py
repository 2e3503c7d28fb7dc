"""Python binding of libhsa, the GB300 (sm_103a) CSA2 hierarchical sparse indexer and sparse
attention (DeepSeek-V4.1-Flash decode hot path).

The functions keep the C ABI's names (``hsa_index_full`` and so on; see include/hsa.h). They
only marshal arguments. Tensors are passed as raw device pointers, and every step of the path
runs in the library's CUDA kernels. The library is built in-tree by ``build.py``. Loading it
when it is missing raises, because there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhsa.so")

HSA_D_LATENT, HSA_D_INDEX, HSA_H_INDEX, HSA_H_ATTN = 512, 128, 16, 64
HSA_TOPK, HSA_CAND_BLOCKS, HSA_BLOCK, HSA_POOL_SLOTS, HSA_SWA_W = 512, 2048, 8, 16384, 128
HSA_MAX_NQ, HSA_MAX_VIS = 8, 1 << 20
HSA_NOALLOC_SCRATCH_BYTES = 64 << 20
HSA_SCALE_E8M0, HSA_SCALE_E4M3 = 0, 1
HSA_MODE_FULL, HSA_MODE_REINDEX, HSA_MODE_REUSE = 0, 1, 2
HSA_FLAG_INDEX_RANGE, HSA_FLAG_WRITE_RANGE, HSA_FLAG_TIMEOUT = 1, 2, 4
HSA_CACHE_ROPE, HSA_CACHE_POOL_TAIL = 1, 2
HSA_POOL_TAIL_SLOTS = 160
HSA_ROPE_DIMS, HSA_ROPE_THETA = 64, 160000.0
HSA_BF16, HSA_F16, HSA_E4M3 = 0, 1, 2
HSA_MAX_GROUP = 128

STATUS = {0: "HSA_OK", 1: "HSA_ERR_INVALID_ARG", 2: "HSA_ERR_SHAPE", 3: "HSA_ERR_ALIGN",
          4: "HSA_ERR_WORKSPACE", 5: "HSA_ERR_CUDA", 6: "HSA_ERR_TIMEOUT", 7: "HSA_ERR_UNSUPPORTED"}
STATUS_CODES = {v: k for k, v in STATUS.items()}

EXPORTS = ("hsa_abi_version", "hsa_status_string", "hsa_workspace_bytes", "hsa_workspace_init",
           "hsa_cache_write_compress", "hsa_index_full", "hsa_index_reindex", "hsa_sparse_attn_decode",
           "hsa_schedule_step", "hsa_get_device_status", "hsa_index_full_noalloc", "hsa_set_wait_limit",
           "hsa_debug_stall_next_scan", "hsa_paged_cache_write", "hsa_paged_attn_workspace_bytes",
           "hsa_paged_attn_decode", "hsa_prompt_attn")


class HsaError(RuntimeError):
    def __init__(self, fn, code, text):
        super().__init__(f"{fn} failed: {text} ({code})")
        self.code = code


class hsa_cache(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("ratio", ctypes.c_int32), ("capacity", ctypes.c_int64),
                ("kv_scale_fmt", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("kv_q", ctypes.c_void_p), ("kv_s", ctypes.c_void_p), ("ik_q", ctypes.c_void_p),
                ("ik_s", ctypes.c_void_p)]


class hsa_step_args(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("nq", ctypes.c_int32),
                ("modes", ctypes.POINTER(ctypes.c_int32)), ("q_idx", ctypes.POINTER(ctypes.c_void_p)),
                ("w_idx", ctypes.POINTER(ctypes.c_void_p)), ("q_attn", ctypes.POINTER(ctypes.c_void_p)),
                ("swa", ctypes.POINTER(ctypes.c_void_p)), ("out", ctypes.POINTER(ctypes.c_void_p)),
                ("topk", ctypes.POINTER(ctypes.c_void_p)), ("pool", ctypes.c_void_p),
                ("vis", ctypes.c_void_p), ("max_vis", ctypes.c_int64), ("sm_scale", ctypes.c_float)]


class hsa_paged_cache(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("n_pages", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("table", ctypes.c_void_p), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


class hsa_prompt_args(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads_q", ctypes.c_int32), ("heads_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("window", ctypes.c_int32),
                ("n_q", ctypes.c_int64), ("n_k", ctypes.c_int64), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64), ("cu_q", ctypes.c_void_p),
                ("cu_k", ctypes.c_void_p), ("sm_scale", ctypes.c_float), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libhsa.so (build it first with build.build()); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libhsa.so not found at {path}: build it with "
                           "`python -m hierarchical_sparse_attention_index_gb300.build`")
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    C, G = ctypes.POINTER(hsa_cache), ctypes.POINTER(hsa_paged_cache)
    sig = {
        "hsa_abi_version": (I32, []),
        "hsa_status_string": (ctypes.c_char_p, [I32]),
        "hsa_workspace_bytes": (SZ, [I32, I32, I64]),
        "hsa_workspace_init": (I32, [P, SZ, P]),
        "hsa_cache_write_compress": (I32, [C, P, P, P, I64, P, P]),
        "hsa_index_full": (I32, [C, P, P, P, I32, I64, P, P, P, SZ, P]),
        "hsa_index_reindex": (I32, [C, P, P, P, I32, I64, P, P, P, SZ, P]),
        "hsa_sparse_attn_decode": (I32, [C, P, P, P, P, I32, I64, F, P, P, SZ, P]),
        "hsa_schedule_step": (I32, [C, ctypes.POINTER(hsa_step_args), P, SZ, P]),
        "hsa_get_device_status": (I32, [P, ctypes.POINTER(ctypes.c_uint32)]),
        "hsa_index_full_noalloc": (I32, [C, P, P, P, I32, I64, P, P, P]),
        "hsa_set_wait_limit": (I32, [ctypes.c_uint64]),
        "hsa_debug_stall_next_scan": (I32, []),
        "hsa_paged_cache_write": (I32, [G, P, P, I32, I64, I64, I64, P, P, P]),
        "hsa_paged_attn_workspace_bytes": (SZ, [G, I32, I32, I64]),
        "hsa_paged_attn_decode": (I32, [G, P, I32, I32, P, I32, I64, I32, F, P, P, P, SZ, P]),
        "hsa_prompt_attn": (I32, [ctypes.POINTER(hsa_prompt_args), P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(t):
    """Device (or host) address of a tensor, None stays NULL, ints pass through."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_current_device = _raw_stream = None


def _device_calls():
    """torch.cuda.current_device, and the address of a device's current stream. torch.cuda.current_stream()
    makes a Stream object first, which costs as much as a launch, so the address is asked for directly
    where torch offers it."""
    global _current_device, _raw_stream
    import torch
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda d: torch.cuda.current_stream(d).cuda_stream)
    _current_device = torch.cuda.current_device


def _stream(stream):
    if stream is None:
        if _current_device is None:
            _device_calls()
        return _raw_stream(_current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, code):
    if code != 0:
        text = load_library().hsa_status_string(code).decode()
        raise HsaError(fn, code, text)


class Cache:
    """Caller-owned FP4 cache of one KV-source layer: four uint8 device tensors
    (kv_q [B][cap][256], kv_s [B][cap][32], ik_q [B][cap][64], ik_s [B][cap][4]); `flags` holds
    HSA_CACHE_* bits (HSA_CACHE_ROPE: the writer applies RoPE to the main-KV latent)."""

    def __init__(self, batch, capacity, ratio=1, kv_scale_fmt=HSA_SCALE_E8M0, device="cuda", tensors=None, flags=0):
        import torch
        self.batch, self.capacity, self.ratio, self.kv_scale_fmt = batch, capacity, ratio, kv_scale_fmt
        self.flags = flags
        if tensors is None:
            z = dict(dtype=torch.uint8, device=device)
            tensors = (torch.zeros(batch, capacity, 256, **z), torch.zeros(batch, capacity, 32, **z),
                       torch.zeros(batch, capacity, 64, **z), torch.zeros(batch, capacity, 4, **z))
        self.kv_q, self.kv_s, self.ik_q, self.ik_s = tensors
        self.desc = hsa_cache(batch, ratio, capacity, kv_scale_fmt, flags, _ptr(self.kv_q), _ptr(self.kv_s),
                              _ptr(self.ik_q), _ptr(self.ik_s))

    @property
    def ref(self):
        return ctypes.byref(self.desc)


def hsa_abi_version():
    return load_library().hsa_abi_version()


def hsa_status_string(code):
    return load_library().hsa_status_string(code).decode()


def hsa_workspace_bytes(batch, nq, max_vis):
    return load_library().hsa_workspace_bytes(batch, nq, max_vis)


def hsa_workspace_init(ws, stream=None):
    _check("hsa_workspace_init", load_library().hsa_workspace_init(_ptr(ws), ws.numel() * ws.element_size(),
                                                                   _stream(stream)))


def new_workspace(batch, nq, max_vis, device="cuda", stream=None):
    """Allocate (torch) and zero-fill a workspace for the given sizes."""
    import torch
    n = hsa_workspace_bytes(batch, nq, max_vis)
    if n == 0:
        raise ValueError("invalid workspace sizes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    hsa_workspace_init(ws, stream)
    return ws


def hsa_cache_write_compress(cache: Cache, wkv, wgate, w_idx, n_tokens, start_entry=None, stream=None):
    _check("hsa_cache_write_compress", load_library().hsa_cache_write_compress(
        cache.ref, _ptr(wkv), _ptr(wgate), _ptr(w_idx), n_tokens, _ptr(start_entry), _stream(stream)))


def hsa_index_full(cache: Cache, q, w, vis, nq, max_vis, topk_out, pool_out, ws, stream=None):
    _check("hsa_index_full", load_library().hsa_index_full(
        cache.ref, _ptr(q), _ptr(w), _ptr(vis), nq, max_vis, _ptr(topk_out), _ptr(pool_out), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def hsa_index_reindex(cache: Cache, q, w, vis, nq, max_vis, pool, topk_out, ws, stream=None):
    _check("hsa_index_reindex", load_library().hsa_index_reindex(
        cache.ref, _ptr(q), _ptr(w), _ptr(vis), nq, max_vis, _ptr(pool), _ptr(topk_out), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def hsa_index_full_noalloc(cache: Cache, q, w, vis, nq, max_vis, topk_out, pool_out, stream=None):
    """hsa_index_full for callers that cannot allocate device memory: its scratch is a fixed
    array inside the library (HSA_NOALLOC_SCRATCH_BYTES), shared by every call, so calls that
    overlap on the GPU race. The first call on a device looks up the array's address there and
    should come before any stream capture."""
    _check("hsa_index_full_noalloc", load_library().hsa_index_full_noalloc(
        cache.ref, _ptr(q), _ptr(w), _ptr(vis), nq, max_vis, _ptr(topk_out), _ptr(pool_out), _stream(stream)))


def hsa_sparse_attn_decode(cache: Cache, q, topk, swa, vis, nq, max_vis, sm_scale, out, ws, stream=None):
    _check("hsa_sparse_attn_decode", load_library().hsa_sparse_attn_decode(
        cache.ref, _ptr(q), _ptr(topk), _ptr(swa), _ptr(vis), nq, max_vis, float(sm_scale), _ptr(out),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


class StepArgs:
    """Builds hsa_step_args from per-layer tensor lists (None for unused slots)."""

    def __init__(self, modes, q_idx, w_idx, q_attn, swa, out, topk, pool, vis, nq, max_vis, sm_scale):
        n = len(modes)
        arr = lambda xs: (ctypes.c_void_p * n)(*[_ptr(x) for x in xs])  # noqa: E731
        self._keep = [arr(q_idx), arr(w_idx), arr(q_attn), arr(swa), arr(out), arr(topk),
                      (ctypes.c_int32 * n)(*modes)]
        self.tensors = (q_idx, w_idx, q_attn, swa, out, topk, pool, vis)
        vp = ctypes.POINTER(ctypes.c_void_p)
        self.args = hsa_step_args(n, nq, ctypes.cast(self._keep[6], ctypes.POINTER(ctypes.c_int32)),
                                  ctypes.cast(self._keep[0], vp), ctypes.cast(self._keep[1], vp),
                                  ctypes.cast(self._keep[2], vp), ctypes.cast(self._keep[3], vp),
                                  ctypes.cast(self._keep[4], vp), ctypes.cast(self._keep[5], vp),
                                  _ptr(pool), _ptr(vis), max_vis, float(sm_scale))


def hsa_schedule_step(caches, step: StepArgs, ws, stream=None):
    """`caches`: one Cache per layer slot (a list), or one Cache that every slot uses."""
    n = step.args.n_layers
    if isinstance(caches, Cache):
        caches = [caches] * n
    if len(caches) != n:
        raise ValueError(f"{len(caches)} caches for {n} layer slots")
    descs = (hsa_cache * n)(*[c.desc for c in caches])
    _check("hsa_schedule_step", load_library().hsa_schedule_step(
        descs, ctypes.byref(step.args), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


# ---------------------------------------------------------------- dense attention
# The checks below run before every call, so they ask a tensor for as little as they can.
_DTYPES = {}


def _dtype(t):
    """The hsa_dtype of a tensor."""
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.bfloat16: HSA_BF16, torch.float16: HSA_F16, torch.float8_e4m3fn: HSA_E4M3,
                        "i32": torch.int32, "i64": torch.int64, "f32": torch.float32})
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"unsupported type {t.dtype}")
    return code


def _rows(name, t, heads, dim):
    """Row stride of [rows][heads][dim] values: rows may stand apart, a row is contiguous."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [rows][{heads}][{dim}]")
    if stride[2] != 1 or (heads > 1 and stride[1] != dim):
        raise ValueError(f"{name}: a row of [{heads}][{dim}] must be contiguous")
    return stride[0] if shape[0] > 1 else heads * dim


def _given(name, t, dtype, shape, device):
    """Address of a contiguous tensor argument (the library takes nothing else of it); None passes."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {list(shape)} on device {device}, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    return t.data_ptr()


def _stream_on(name, device, stream):
    """The stream to launch on. The library launches on the current device, so its tensors have to be
    there (-1: not on a GPU)."""
    if device < 0:
        raise ValueError(f"{name} is not on a CUDA device")
    if _current_device is None:
        _device_calls()
    if device != _current_device():
        raise ValueError(f"{name} is on device {device}: expected the current one, {_current_device()}")
    return _raw_stream(device) if stream is None else _stream(stream)


class PagedCache:
    """Caller-owned paged key-value cache of a dense attention layer: pools k and v
    [n_pages][heads][page_size][head_dim] (bfloat16, float16 or float8_e4m3fn) and an int32 table
    [batch][max_pages] of page ids, all contiguous. A value is its stored number times its scale."""

    def __init__(self, k, v, table, k_scale=1.0, v_scale=1.0):
        import torch
        if k.dim() != 4 or table.dim() != 2:
            raise ValueError("k and v are [n_pages][heads][page_size][head_dim], table is [batch][max_pages]")
        self.k, self.v, self.table = k, v, table
        self.dtype, self.device = _dtype(k), k.get_device()
        _given("k", k, k.dtype, k.shape, self.device)
        _given("v", v, k.dtype, k.shape, self.device)
        _given("table", table, torch.int32, table.shape, self.device)
        n_pages, self.heads, self.page_size, self.head_dim = k.shape
        self.batch, max_pages = table.shape
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.desc = hsa_paged_cache(self.batch, self.heads, self.head_dim, self.page_size, self.dtype, 0, n_pages, max_pages,
                                    _ptr(k), _ptr(v), _ptr(table), self.k_scale, self.v_scale)

    @property
    def ref(self):
        return ctypes.byref(self.desc)


def hsa_paged_cache_write(cache: PagedCache, k, v, cu=None, start=None, stream=None):
    """k, v: [n_tokens][heads][head_dim], rows at any stride; cu: int32 [batch + 1] or None (equal
    shares); start: int64 [batch] or None (0)."""
    device = cache.device
    stream = _stream_on("cache", device, stream)
    k_stride, v_stride = _rows("k", k, cache.heads, cache.head_dim), _rows("v", v, cache.heads, cache.head_dim)
    n = k.shape[0]
    if v.shape[0] != n or k.dtype is not v.dtype or k.get_device() != device or v.get_device() != device:
        raise ValueError("k and v differ in shape or type, or are not on the cache's device")
    dtype = _dtype(k)
    _check("hsa_paged_cache_write", load_library().hsa_paged_cache_write(
        cache.ref, k.data_ptr(), v.data_ptr(), dtype, k_stride, v_stride, n,
        _given("cu", cu, _DTYPES["i32"], (cache.batch + 1,), device),
        _given("start", start, _DTYPES["i64"], (cache.batch,), device), stream))


def hsa_paged_attn_workspace_bytes(cache: PagedCache, heads_q, nq, max_vis):
    return load_library().hsa_paged_attn_workspace_bytes(cache.ref, heads_q, nq, max_vis)


def new_paged_workspace(cache: PagedCache, heads_q, nq, max_vis):
    """Allocate (torch) a workspace of hsa_paged_attn_decode for the given sizes."""
    import torch
    n = hsa_paged_attn_workspace_bytes(cache, heads_q, nq, max_vis)
    if n == 0:
        raise ValueError("invalid workspace sizes")
    return torch.empty(n, dtype=torch.uint8, device=cache.k.device)


def hsa_paged_attn_decode(cache: PagedCache, q, vis, max_vis, sm_scale, out, ws, window=0, lse=None, stream=None):
    """q, out: [batch][nq][heads_q][head_dim]; vis: int32 [batch][nq]; lse: float32 [batch][nq][heads_q] or None."""
    device, shape = cache.device, q.shape
    stream = _stream_on("cache", device, stream)
    if len(shape) != 4 or shape[0] != cache.batch or shape[3] != cache.head_dim:
        raise ValueError(f"q: shape {tuple(shape)}, expected [{cache.batch}][nq][heads_q][{cache.head_dim}]")
    if ws is not None and (ws.get_device() != device or not ws.is_contiguous()):
        raise ValueError("ws: expected a contiguous tensor on the cache's device")
    _, nq, heads_q, _ = shape
    dtype = _dtype(q)
    _check("hsa_paged_attn_decode", load_library().hsa_paged_attn_decode(
        cache.ref, _given("q", q, q.dtype, shape, device), dtype, heads_q,
        _given("vis", vis, _DTYPES["i32"], (cache.batch, nq), device), nq, max_vis, window, sm_scale,
        _given("out", out, q.dtype, shape, device), _given("lse", lse, _DTYPES["f32"], shape[:3], device), _ptr(ws),
        ws.numel() * ws.element_size() if ws is not None else 0, stream))


def hsa_prompt_attn(q, k, v, cu_q, sm_scale, out, cu_k=None, window=0, lse=None, stream=None):
    """q, out: [n_q][heads_q][head_dim], k, v: [n_k][heads_kv][head_dim], rows at any stride; cu_q,
    cu_k: int32 [batch + 1] (cu_k None: cu_q); lse: float32 [n_q][heads_q] or None."""
    device = q.get_device()
    stream = _stream_on("q", device, stream)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k, v and out are [rows][heads][head_dim]")
    (n_q, heads_q, dim), (n_k, heads_kv, _) = q.shape, k.shape
    q_stride, out_stride = _rows("q", q, heads_q, dim), _rows("out", out, heads_q, dim)
    k_stride, v_stride = _rows("k", k, heads_kv, dim), _rows("v", v, heads_kv, dim)
    if out.shape[0] != n_q or v.shape[0] != n_k or not q.dtype is k.dtype is v.dtype is out.dtype or \
            not device == k.get_device() == v.get_device() == out.get_device():
        raise ValueError("q, k, v and out differ in type or device, q and out or k and v in shape")
    dtype, i32, cu_shape = _dtype(q), _DTYPES["i32"], cu_q.shape
    if len(cu_shape) != 1:
        raise ValueError("cu_q is [batch + 1]")
    a = hsa_prompt_args(cu_shape[0] - 1, heads_q, heads_kv, dim, dtype, window, n_q, n_k, q.data_ptr(), k.data_ptr(),
                        v.data_ptr(), q_stride, k_stride, v_stride, out_stride, _given("cu_q", cu_q, i32, cu_shape, device),
                        _given("cu_k", cu_k, i32, cu_shape, device), sm_scale, out.data_ptr(),
                        _given("lse", lse, _DTYPES["f32"], (n_q, heads_q), device))
    _check("hsa_prompt_attn", load_library().hsa_prompt_attn(ctypes.byref(a), stream))


def hsa_set_wait_limit(ns):
    """Limit of the kernels' bounded waits for later launches, in ns (0: the default, 2 s)."""
    _check("hsa_set_wait_limit", load_library().hsa_set_wait_limit(int(ns)))


def hsa_debug_stall_next_scan():
    """Test hook: the next hsa_index_full withholds one copy of its scan, so a bounded wait runs
    out (HSA_FLAG_TIMEOUT); that call's outputs are invalid, later calls are unaffected."""
    _check("hsa_debug_stall_next_scan", load_library().hsa_debug_stall_next_scan())


def hsa_get_device_status(stream=None):
    """Synchronise the stream and return (status code, flags); the flags are cleared."""
    flags = ctypes.c_uint32(0)
    code = load_library().hsa_get_device_status(_stream(stream), ctypes.byref(flags))
    return code, flags.value
