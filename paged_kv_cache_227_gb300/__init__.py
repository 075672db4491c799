"""Paged KV-cache decode attention for one GB300 (sm_103a).

A thin ctypes binding over the C ABI in ``include/pa.h``: the functions below
carry the same names as the C entry points and only marshal arguments (torch
tensors -> device pointers, the current torch stream -> cudaStream_t).  Every
step of the computation runs in the library's CUDA kernels; there is no CPU
fallback, and importing fails loudly when the library has not been built.
"""
import ctypes
import os

import torch


_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpagedattn.so")

PA_FP16, PA_BF16, PA_FP32, PA_E4M3, PA_INT8 = 0, 1, 2, 3, 4
PA_OK = 0
PA_ERR_INVALID, PA_ERR_UNSUPPORTED, PA_ERR_OOM = -1, -2, -3
PA_ERR_CUDA, PA_ERR_DEVICE_CHECK, PA_ERR_TIMEOUT = -4, -5, -6
PA_ERR_SCRATCH_LIMIT = -7
PA_STATIC_SCRATCH_BYTES = 12 << 20
BLOCK_SIZE, HEAD_DIM, MAX_GROUP = 16, 128, 8

_DTYPE_CODE = {torch.float16: PA_FP16, torch.bfloat16: PA_BF16, torch.float32: PA_FP32}
_CODE_DTYPE = {v: k for k, v in _DTYPE_CODE.items()}
_DTYPE8_CODE = {torch.float8_e4m3fn: PA_E4M3, torch.int8: PA_INT8}


class PagedAttentionError(RuntimeError):
    def __init__(self, code, what):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} ({code})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"the CUDA library {LIB_PATH} is not built; run paged_kv_cache_227_gb300.build.build() "
            "(or __graft_entry__.build()) first - there is no fallback")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sigs = {
        "pa_pool_bytes": (sz, [i32, i32, i32, i32, i32]),
        "pa_pool_create": (i32, [i32, i32, i32, i32, i32, ctypes.POINTER(vp)]),
        "pa_pool_destroy": (i32, [vp]),
        "pa_pool_info": (i32, [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(sz)]),
        "pa_pool_shape": (i32, [vp] + [ctypes.POINTER(i32)] * 4),
        "pa_cache_append": (i32, [vp, vp, vp, vp, i32, vp]),
        "pa_rope_append": (i32, [vp, vp, i64, i32, vp, i64, vp, i64, vp, i32, vp, vp, i32, i32, vp, i32, vp, i64, vp]),
        "pa_norm_rope_append": (i32, [vp, vp, i64, i32, vp, i64, vp, i64, vp, vp, f32, vp, i32, vp, vp, i32, i32, vp, i32,
                                      vp, i64, vp]),
        "pa_pool8_bytes": (sz, [i32, i32, i32, i32, i32]),
        "pa_pool8_create": (i32, [i32, i32, i32, i32, i32, ctypes.POINTER(vp)]),
        "pa_pool8_destroy": (i32, [vp]),
        "pa_pool8_info": (i32, [vp, ctypes.POINTER(vp), ctypes.POINTER(vp)]),
        "pa_check8": (i32, [vp, vp, ctypes.POINTER(i64)]),
        "pa_cache_append8": (i32, [vp, i32, vp, vp, vp, i32, vp]),
        "pa_norm_rope_append8": (i32, [vp, i32, vp, i64, i32, vp, i64, vp, i64, vp, vp, f32, vp, i32, vp, vp, i32, i32, vp,
                                       i32, vp, i64, vp]),
        "pa_decode8_workspace_bytes": (sz, [vp, i32, i32, i32]),
        "pa_decode8": (i32, [vp, vp, i32, vp, i32, vp, i32, i32, f32, vp, i32, vp, sz, vp]),
        "pa_selftest_decode8_timeout": (i32, [vp, vp, i32, vp, i32, vp, i32, i32, f32, vp, i32, vp, sz, i32,
                                              ctypes.c_longlong, vp]),
        "pa_copy_blocks8": (i32, [vp, vp, vp, i32, vp]),
        "pa_quantize_blocks": (i32, [vp, vp, vp, vp, vp, i32, vp]),
        "pa_dequantize_blocks": (i32, [vp, vp, vp, vp, i32, vp]),
        "pa_decode_weights_workspace_bytes": (sz, [vp, i32, i32, i32]),
        "pa_decode_weights": (i32, [vp, vp, vp, i32, vp, i32, i32, f32, vp, i32, vp, f32, vp, sz, vp]),
        "pa_decode_shared_workspace_bytes": (sz, [vp, i32, i32, i32, i32]),
        "pa_decode_shared": (i32, [vp, vp, vp, i32, vp, i32, i32, f32, vp, vp, i32, vp, i32, vp, i32, vp, sz, vp]),
        "pa_selftest_shared_timeout": (i32, [vp, vp, vp, i32, vp, i32, i32, f32, vp, vp, i32, vp, i32, vp, i32, vp, sz,
                                             ctypes.c_longlong, vp]),
        "pa_evict": (i32, [vp, vp, vp, vp, i32, vp, i32, vp, vp, i32, i32, i32, vp, vp, vp]),
        "pa_alloc_evict": (i32, [vp, vp, vp, i32]),
        "pa_decode": (i32, [vp, vp, vp, i32, vp, i32, i32, f32, vp, i32, vp]),
        "pa_decode_workspace_bytes": (sz, [vp, i32, i32, i32, i32]),
        "pa_decode_split": (i32, [vp, vp, vp, i32, vp, i32, i32, f32, vp, i32, i32, vp, sz, vp]),
        "pa_append_decode": (i32, [vp, vp, vp, vp, vp, i32, vp, i32, i32, f32, vp, i32, i32, vp, sz, vp]),
        "pa_decode_multi_workspace_bytes": (ctypes.c_size_t, [vp, i32, i32, i32, i32]),
        "pa_decode_multi": (i32, [vp, vp, vp, i32, vp, i32, vp, i32, i32, f32, vp, i32, vp, ctypes.c_size_t, vp]),
        "pa_decode_cascade_workspace_bytes": (ctypes.c_size_t, [vp, i32, i32, i32, i32]),
        "pa_decode_cascade": (i32, [vp, vp, vp, i32, vp, i32, i32, f32, vp, vp, vp, i32, vp, i32, vp,
                                    ctypes.c_size_t, vp]),
        "pa_cascade_groups": (i32, [vp, i32, i32, vp, i32, vp, vp, vp, ctypes.POINTER(i32)]),
        "pa_selftest_wait_timeout": (i32, [vp, ctypes.c_longlong, vp]),
        "pa_decode_split_static": (i32, [vp, vp, vp, i32, vp, i32, i32, f32, vp, i32, i32, vp]),
        "pa_copy_blocks": (i32, [vp, vp, vp, i32, vp]),
        "pa_check": (i32, [vp, vp, ctypes.POINTER(i64)]),
        "pa_profile_start": (i32, [i32]),
        "pa_profile_stop": (i32, [ctypes.POINTER(f32), i32]),
        "pa_strerror": (ctypes.c_char_p, [i32]),
        "pa_alloc_create": (i32, [i32, i32, vp, ctypes.POINTER(vp)]),
        "pa_alloc_destroy": (i32, [vp]),
        "pa_alloc_seq_add": (i32, [vp, i32]),
        "pa_alloc_fork": (i32, [vp, i32, i32]),
        "pa_alloc_append_slot": (i32, [vp, i32, ctypes.POINTER(i64), ctypes.POINTER(ctypes.c_int32),
                                       ctypes.POINTER(ctypes.c_int32)]),
        "pa_alloc_extend": (i32, [vp, i32, i32, vp, ctypes.POINTER(ctypes.c_int32),
                                  ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(i32)]),
        "pa_alloc_seq_free": (i32, [vp, i32]),
        "pa_alloc_table": (i32, [vp, i32, vp, i32, ctypes.POINTER(i32)]),
        "pa_alloc_seq_len": (i32, [vp, i32]),
        "pa_alloc_refcount": (i32, [vp, i32]),
        "pa_alloc_num_free": (i32, [vp]),
        "pa_alloc_seq_add_cached": (i32, [vp, i32, vp, i32, ctypes.POINTER(i32)]),
        "pa_alloc_append_token": (i32, [vp, i32, ctypes.c_int32, ctypes.POINTER(i64), ctypes.POINTER(ctypes.c_int32),
                                        ctypes.POINTER(ctypes.c_int32)]),
        "pa_alloc_block_hash": (i32, [vp, i32, ctypes.POINTER(ctypes.c_uint64)]),
        "pa_alloc_prefix_stats": (i32, [vp, ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(i64)]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def strerror(code):
    return lib.pa_strerror(int(code)).decode()


def _check(code, what):
    if code != PA_OK:
        raise PagedAttentionError(code, what)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, name, dtype=None, device=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if device and not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


class _PoolHandle:
    """Destroys its pa_pool_t (or pa_pool8_t) when nothing refers to it any more:
    the Pool, and every tensor that views its memory."""

    def __init__(self, destroy=lib.pa_pool_destroy):
        self.ptr = ctypes.c_void_p()
        self._destroy = destroy

    def destroy(self):
        if self.ptr:
            self._destroy(self.ptr)
            self.ptr = ctypes.c_void_p()

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


class _CudaArray:
    """Exposes a raw device buffer through __cuda_array_interface__ so torch can
    view it without copying; torch keeps this object, and with it the buffer's
    owner, as long as a view lives."""

    def __init__(self, ptr, shape, typestr, owner):
        self.owner = owner
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr,
                                         "data": (ptr, False), "version": 3, "strides": None}


class Pool:
    """Owns one pa_pool_t: K and V arrays [num_blocks][n_kv_heads][16][128].
    close() releases the memory at once (views of k and v must not be used
    after it); a pool that is only dropped lives on as long as its views."""

    def __init__(self, num_blocks, n_kv_heads, dtype=torch.bfloat16, block_size=BLOCK_SIZE,
                 d_head=HEAD_DIM):
        self._h = _PoolHandle()
        code = lib.pa_pool_create(num_blocks, block_size, n_kv_heads, d_head, _DTYPE_CODE[dtype],
                                  ctypes.byref(self._h.ptr))
        _check(code, "pa_pool_create")
        self.num_blocks, self.n_kv_heads, self.dtype = num_blocks, n_kv_heads, dtype
        self.device = torch.device("cuda", torch.cuda.current_device())
        k, v, nbytes = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_size_t()
        _check(lib.pa_pool_info(self._h.ptr, ctypes.byref(k), ctypes.byref(v), ctypes.byref(nbytes)), "pa_pool_info")
        self.bytes_per_pool = nbytes.value
        shape = (num_blocks, n_kv_heads, BLOCK_SIZE, HEAD_DIM)
        # views of the library-owned memory (int16 carrier, reinterpreted)
        self.k = torch.as_tensor(_CudaArray(k.value, shape, "<i2", self._h), device=self.device).view(dtype)
        self.v = torch.as_tensor(_CudaArray(v.value, shape, "<i2", self._h), device=self.device).view(dtype)

    @property
    def handle(self):
        return self._h.ptr

    def close(self):
        if self._h.ptr:
            self.k = self.v = None
            self._h.destroy()


class Pool8:
    """Owns one pa_pool8_t, a cache in 8 bits: codes k and v [num_blocks][n_kv_heads]
    [16][128] (torch.float8_e4m3fn or torch.int8; strided views, a tile's K and
    V lie on end) and their scales k_scale and v_scale [num_blocks][n_kv_heads]
    (torch.float8_e8m0fnu, powers of two): a code stands for code * scale.
    close() and dropping it: as for Pool."""

    def __init__(self, num_blocks, n_kv_heads, dtype=torch.float8_e4m3fn, block_size=BLOCK_SIZE, d_head=HEAD_DIM):
        self._h = _PoolHandle(lib.pa_pool8_destroy)
        code = lib.pa_pool8_create(num_blocks, block_size, n_kv_heads, d_head, _DTYPE8_CODE[dtype],
                                   ctypes.byref(self._h.ptr))
        _check(code, "pa_pool8_create")
        self.num_blocks, self.n_kv_heads, self.dtype = num_blocks, n_kv_heads, dtype
        self.device = torch.device("cuda", torch.cuda.current_device())
        codes, exps = ctypes.c_void_p(), ctypes.c_void_p()
        _check(lib.pa_pool8_info(self._h.ptr, ctypes.byref(codes), ctypes.byref(exps)), "pa_pool8_info")
        shape = (num_blocks, n_kv_heads, 2, BLOCK_SIZE, HEAD_DIM)
        kv = torch.as_tensor(_CudaArray(codes.value, shape, "|u1", self._h), device=self.device).view(dtype)
        scale = torch.as_tensor(_CudaArray(exps.value, shape[:3], "|u1", self._h), device=self.device)
        scale = scale.view(torch.float8_e8m0fnu)
        self.k, self.v = kv[:, :, 0], kv[:, :, 1]
        self.k_scale, self.v_scale = scale[:, :, 0], scale[:, :, 1]

    @property
    def handle(self):  # (a pa_pool8_t is no pa_pool_t: the calls of the one read past the other)
        raise TypeError("this call takes a Pool, got a Pool8")

    @property
    def handle8(self):
        return self._h.ptr

    def close(self):
        if self._h.ptr:
            self.k = self.v = self.k_scale = self.v_scale = None
            self._h.destroy()


def _handle8(pool):
    if not isinstance(pool, Pool8):
        raise TypeError(f"this call takes a Pool8, got {type(pool).__name__}")
    return pool.handle8


def pa_pool_bytes(num_blocks, n_kv_heads, dtype, block_size=BLOCK_SIZE, d_head=HEAD_DIM):
    return lib.pa_pool_bytes(num_blocks, block_size, n_kv_heads, d_head, _DTYPE_CODE[dtype])


def pa_pool_create(num_blocks, block_size, n_kv_heads, d_head, dtype):
    return Pool(num_blocks, n_kv_heads, dtype, block_size, d_head)


def pa_cache_append(pool, k_new, v_new, slot_mapping, stream=None):
    _need(k_new, "k_new", pool.dtype); _need(v_new, "v_new", pool.dtype)
    _need(slot_mapping, "slot_mapping", torch.int64)
    n_tok = slot_mapping.numel()
    if k_new.shape != (n_tok, pool.n_kv_heads, HEAD_DIM) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [n_tok][n_kv_heads][128]")
    _check(lib.pa_cache_append(pool.handle, _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), n_tok,
                               _stream(stream)), "pa_cache_append")


def _decode_args(pool, q, block_tables, seq_lens, out):
    _need(q, "q", pool.dtype); _need(block_tables, "block_tables", torch.int32)
    _need(seq_lens, "seq_lens", torch.int32); _need(out, "out")
    B, Hq, d = q.shape
    if d != HEAD_DIM or block_tables.dim() != 2 or block_tables.shape[0] != B or seq_lens.shape != (B,):
        raise ValueError("shapes: q [B][Hq][128], block_tables [B][W], seq_lens [B]")
    if out.shape != q.shape or out.dtype not in _DTYPE_CODE:
        raise ValueError("out must be [B][Hq][128] of fp16, bf16 or fp32")
    return B, Hq, block_tables.shape[1]


def pa_decode(pool, q, block_tables, seq_lens, scale, out, stream=None):
    B, Hq, W = _decode_args(pool, q, block_tables, seq_lens, out)
    _check(lib.pa_decode(pool.handle, _ptr(q), _ptr(block_tables), W, _ptr(seq_lens), B, Hq,
                         float(scale), _ptr(out), _DTYPE_CODE[out.dtype], _stream(stream)), "pa_decode")


def pa_decode_workspace_bytes(pool, num_seqs, n_q_heads, max_blocks_per_seq, partition_blocks=0):
    return lib.pa_decode_workspace_bytes(pool.handle, num_seqs, n_q_heads, max_blocks_per_seq,
                                         partition_blocks)


def workspace_for(pool, q, block_tables, partition_blocks=0):
    n = pa_decode_workspace_bytes(pool, q.shape[0], q.shape[1], block_tables.shape[1], partition_blocks)
    if n == 0:
        raise PagedAttentionError(PA_ERR_INVALID, "pa_decode_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def pa_decode_split(pool, q, block_tables, seq_lens, scale, out, partition_blocks=0,
                    workspace=None, stream=None):
    B, Hq, W = _decode_args(pool, q, block_tables, seq_lens, out)
    if workspace is None:
        workspace = workspace_for(pool, q, block_tables, partition_blocks)
    _check(lib.pa_decode_split(pool.handle, _ptr(q), _ptr(block_tables), W, _ptr(seq_lens), B, Hq,
                               float(scale), _ptr(out), _DTYPE_CODE[out.dtype], int(partition_blocks),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(stream)), "pa_decode_split")


def pa_decode_split_static(pool, q, block_tables, seq_lens, scale, out, partition_blocks=0, stream=None):
    """pa_decode_split without a caller workspace: uses the library's static
    device scratch (see include/pa.h); allocates nothing."""
    B, Hq, W = _decode_args(pool, q, block_tables, seq_lens, out)
    _check(lib.pa_decode_split_static(pool.handle, _ptr(q), _ptr(block_tables), W, _ptr(seq_lens), B, Hq,
                                      float(scale), _ptr(out), _DTYPE_CODE[out.dtype], int(partition_blocks),
                                      _stream(stream)), "pa_decode_split_static")


def pa_append_decode(pool, q, k_new, v_new, block_tables, seq_lens, scale, out, partition_blocks=0,
                     workspace=None, stream=None):
    B, Hq, W = _decode_args(pool, q, block_tables, seq_lens, out)
    _need(k_new, "k_new", pool.dtype); _need(v_new, "v_new", pool.dtype)
    if k_new.shape != (B, pool.n_kv_heads, HEAD_DIM) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [B][n_kv_heads][128]")
    if workspace is None:
        workspace = workspace_for(pool, q, block_tables, partition_blocks)
    _check(lib.pa_append_decode(pool.handle, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(block_tables), W,
                                _ptr(seq_lens), B, Hq, float(scale), _ptr(out), _DTYPE_CODE[out.dtype],
                                int(partition_blocks), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream)),
           "pa_append_decode")


def pa_decode_multi(pool, q, q_start, block_tables, seq_lens, scale, out, workspace=None, stream=None):
    """Several new query tokens per sequence (causal within them); q and out
    are [n_q][Hq][128], q_start int32 [B+1] on the device (see include/pa.h)."""
    _need(q, "q", pool.dtype); _need(q_start, "q_start", torch.int32)
    _need(block_tables, "block_tables", torch.int32); _need(seq_lens, "seq_lens", torch.int32); _need(out, "out")
    n_q, Hq, d = q.shape
    B = seq_lens.shape[0]
    if d != HEAD_DIM or q_start.shape != (B + 1,) or block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise ValueError("shapes: q [n_q][Hq][128], q_start [B+1], block_tables [B][W], seq_lens [B]")
    if out.shape != q.shape or out.dtype not in _DTYPE_CODE:
        raise ValueError("out must be [n_q][Hq][128] of fp16, bf16 or fp32")
    W = block_tables.shape[1]
    if workspace is None:
        n = lib.pa_decode_multi_workspace_bytes(pool.handle, n_q, B, Hq, W)
        if n == 0:
            raise PagedAttentionError(PA_ERR_INVALID, "pa_decode_multi_workspace_bytes")
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    _check(lib.pa_decode_multi(pool.handle, _ptr(q), _ptr(q_start), n_q, _ptr(block_tables), W, _ptr(seq_lens), B, Hq,
                               float(scale), _ptr(out), _DTYPE_CODE[out.dtype], _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream)), "pa_decode_multi")


def cascade_groups(block_tables, seq_lens, n_q_heads, n_kv_heads, max_members=None):
    """Host: (group_start, members, prefix_blocks) int32 numpy arrays for
    pa_decode_cascade from host tables [B][W] and lengths [B].  max_members: the
    largest group, by default what pa_decode_cascade takes (8 / G); the batch
    size for pa_decode_shared."""
    import numpy as np
    t = np.ascontiguousarray(block_tables, dtype=np.int32)
    lens = np.ascontiguousarray(seq_lens, dtype=np.int32)
    B, W = t.shape
    gs = np.zeros(B + 1, np.int32)
    mem = np.zeros(max(B, 1), np.int32)
    pre = np.zeros(max(B, 1), np.int32)
    ng = ctypes.c_int()
    _check(lib.pa_cascade_groups(t.ctypes.data_as(ctypes.c_void_p), B, W, lens.ctypes.data_as(ctypes.c_void_p),
                                 MAX_GROUP // (n_q_heads // n_kv_heads) if max_members is None else int(max_members), gs.ctypes.data_as(ctypes.c_void_p),
                                 mem.ctypes.data_as(ctypes.c_void_p), pre.ctypes.data_as(ctypes.c_void_p),
                                 ctypes.byref(ng)), "pa_cascade_groups")
    n = ng.value
    return gs[:n + 1].copy(), mem[:gs[n]].copy(), pre[:n].copy()


def pa_decode_cascade(pool, q, block_tables, seq_lens, scale, out, group_start, members, prefix_blocks,
                      workspace=None, stream=None):
    """pa_decode with each group's shared prefix read once (include/pa.h);
    the group arrays are int32 device tensors."""
    B, Hq, W = _decode_args(pool, q, block_tables, seq_lens, out)
    for t, n in ((group_start, "group_start"), (members, "members"), (prefix_blocks, "prefix_blocks")):
        _need(t, n, torch.int32)
    ng = prefix_blocks.shape[0]
    if workspace is None:
        n = lib.pa_decode_cascade_workspace_bytes(pool.handle, B, Hq, W, ng)
        if n == 0:
            raise PagedAttentionError(PA_ERR_INVALID, "pa_decode_cascade_workspace_bytes")
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    _check(lib.pa_decode_cascade(pool.handle, _ptr(q), _ptr(block_tables), W, _ptr(seq_lens), B, Hq, float(scale),
                                 _ptr(group_start) if ng else None, _ptr(members) if ng else None,
                                 _ptr(prefix_blocks) if ng else None, ng, _ptr(out), _DTYPE_CODE[out.dtype],
                                 _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)),
           "pa_decode_cascade")


# The cache operators' checks: one pass over each tensor that also yields its
# address, since at the smallest sizes a call is bound by the host (rotary append
# of 64 tokens: 2.3 us on the GPU).
def _at(pool, t, name, dtype):
    """Address of a contiguous `dtype` tensor on the pool's device."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == pool.device and t.is_contiguous():
        return t.data_ptr()
    _refuse(pool, t, name, dtype)
    raise ValueError(f"{name} must be contiguous")


def _refuse(pool, t, name, dtype):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != pool.device:
        raise ValueError(f"{name} must be on the GPU, on the pool's device {pool.device}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _int32(x):
    """A count for a C int: past its range it means the same as its ends."""
    return max(-1, min(int(x), 0x7fffffff))


def _raw_stream(pool, stream):
    """The given stream, or the pool's device's current one, as an address."""
    return torch._C._cuda_getCurrentRawStream(pool.device.index) if stream is None else stream.cuda_stream


def _decode_at(pool, q, block_tables, seq_lens, out, dtype=None):
    """Checks of a decode's tensors (as _decode_args), q of `dtype` or the pool's;
    their addresses and sizes."""
    qa = _at(pool, q, "q", pool.dtype if dtype is None else dtype)
    ta = _at(pool, block_tables, "block_tables", torch.int32)
    la = _at(pool, seq_lens, "seq_lens", torch.int32)
    code = _DTYPE_CODE.get(out.dtype) if isinstance(out, torch.Tensor) else 0
    if code is None:
        raise ValueError("out must be [B][Hq][128] of fp16, bf16 or fp32")
    oa = _at(pool, out, "out", getattr(out, "dtype", None))
    shape = q.shape
    if len(shape) != 3 or shape[2] != HEAD_DIM or block_tables.dim() != 2 or block_tables.shape[0] != shape[0] \
            or seq_lens.shape != shape[:1]:
        raise ValueError("shapes: q [B][Hq][128], block_tables [B][W], seq_lens [B]")
    if out.shape != shape:
        raise ValueError("out must be [B][Hq][128] of fp16, bf16 or fp32")
    return qa, ta, la, oa, code, shape[0], shape[1], block_tables.shape[1]


def _workspace(nbytes, what, device, stream):
    """A workspace for one call, from the memory of the stream it runs on (memory
    of another stream could still be in use there, or be handed out again)."""
    if nbytes == 0:
        raise PagedAttentionError(PA_ERR_INVALID, what)
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _heads(pool, dtype, t, name, shape):
    """Checks [n_tok][n_heads][128] rows of `dtype` with contiguous heads; their
    address and token stride in elements."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == pool.device):
        _refuse(pool, t, name, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    tok, head, dim = t.stride()
    if (dim != 1 or (head != HEAD_DIM and shape[1] > 1)) and shape[0]:
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), (tok if shape[0] > 1 else shape[1] * HEAD_DIM)


def _rope_at(pool, dtype, q, k_new, v_new, positions, inv_freq, axis_of_pair, slot_mapping, q_out):
    """Checks of the rotary appends' tensors, rows of `dtype`; the C calls' arguments
    up to the norms, and behind them."""
    sa = _at(pool, slot_mapping, "slot_mapping", torch.int64)
    pos = _at(pool, positions, "positions", torch.int32)
    fa = _at(pool, inv_freq, "inv_freq", torch.float32)
    n = slot_mapping.numel()
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if q.dim() != 3:
        raise ValueError("q must be [n_tok][Hq][128]")
    Hq = q.shape[1]
    q_rows, kv_rows = (n, Hq, HEAD_DIM), (n, pool.n_kv_heads, HEAD_DIM)
    qa, qs = _heads(pool, dtype, q, "q", q_rows)
    ka, ks = _heads(pool, dtype, k_new, "k_new", kv_rows)
    va, vs = _heads(pool, dtype, v_new, "v_new", kv_rows)
    oa, os_ = _heads(pool, dtype, q_out, "q_out", q_rows)
    # (ValueError outside 0 .. 255; an array's own bytes are not its numbers)
    axes = bytes(axis_of_pair if isinstance(axis_of_pair, (list, tuple, bytes, bytearray)) else list(axis_of_pair))
    if positions.dim() != 2 or positions.shape[1] != n:
        raise ValueError("positions must be [n_axes][n_tok]")
    if inv_freq.shape != (len(axes),):
        raise ValueError("inv_freq and axis_of_pair must have rot_dim / 2 entries each")
    return (qa, qs, Hq, ka, ks, va, vs), (pos, positions.shape[0], axes, fa, 2 * len(axes)), (sa, n, oa, os_)


def pa_rope_append(pool, q, k_new, v_new, positions, inv_freq, axis_of_pair, slot_mapping, q_out, interleaved=False,
                   stream=None):
    """Rotary positions of one or several axes on new tokens' q and k, with the
    cache write of k and v (see include/pa.h).  q and q_out [n][Hq][128], k_new
    and v_new [n][Hkv][128] with any token stride (slices of a fused projection
    work), positions int32 [n_axes][n], inv_freq fp32 [rot_dim/2],
    axis_of_pair: rot_dim/2 ints on the host (bytes are taken as they are),
    slot_mapping int64 [n].  q_out may be q."""
    rows, turn, to = _rope_at(pool, pool.dtype, q, k_new, v_new, positions, inv_freq, axis_of_pair, slot_mapping, q_out)
    _check(lib.pa_rope_append(pool.handle, *rows, *turn, 1 if interleaved else 0, *to, _raw_stream(pool, stream)),
           "pa_rope_append")


def _norm_at(pool, dtype, weight, name):
    if weight is None:
        return None
    a = _at(pool, weight, name, dtype)
    if weight.shape != (HEAD_DIM,):
        raise ValueError(f"{name} must be [128]")
    return a


def pa_norm_rope_append(pool, q, k_new, v_new, q_weight, k_weight, positions, inv_freq, axis_of_pair, slot_mapping, q_out,
                        eps=1e-6, interleaved=False, stream=None):
    """pa_rope_append with the RMS norm of each q and k head before the rotation
    (see include/pa.h): q_weight and k_weight [128] of the pool's dtype, or None:
    rows of that kind are not normed."""
    rows, turn, to = _rope_at(pool, pool.dtype, q, k_new, v_new, positions, inv_freq, axis_of_pair, slot_mapping, q_out)
    _check(lib.pa_norm_rope_append(pool.handle, *rows, _norm_at(pool, pool.dtype, q_weight, "q_weight"),
                                   _norm_at(pool, pool.dtype, k_weight, "k_weight"), float(eps), *turn,
                                   1 if interleaved else 0, *to, _raw_stream(pool, stream)), "pa_norm_rope_append")


def _row_dtype(t, name):
    """The type of 16-bit rows next to an 8-bit pool."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16 and t.dtype is not torch.float16:
        raise TypeError(f"{name} must be fp16 or bf16, got {t.dtype}")
    return t.dtype


def pa_norm_rope_append8(pool, q, k_new, v_new, q_weight, k_weight, positions, inv_freq, axis_of_pair, slot_mapping, q_out,
                         eps=1e-6, interleaved=False, stream=None):
    """pa_norm_rope_append into a Pool8 (see include/pa.h for how blocks get their
    scales): rows, weights and q_out all fp16 or all bf16.  The rows of one block
    are consecutive, in the order of their slots."""
    dtype = _row_dtype(q, "q")
    rows, turn, to = _rope_at(pool, dtype, q, k_new, v_new, positions, inv_freq, axis_of_pair, slot_mapping, q_out)
    _check(lib.pa_norm_rope_append8(_handle8(pool), _DTYPE_CODE[dtype], *rows, _norm_at(pool, dtype, q_weight, "q_weight"),
                                    _norm_at(pool, dtype, k_weight, "k_weight"), float(eps), *turn,
                                    1 if interleaved else 0, *to, _raw_stream(pool, stream)), "pa_norm_rope_append8")


def pa_cache_append8(pool, k_new, v_new, slot_mapping, stream=None):
    """Writes k_new and v_new [n][Hkv][128] (fp16 or bf16) into a Pool8 at
    slot_mapping int64 [n] (see include/pa.h)."""
    dtype = _row_dtype(k_new, "k_new")
    ka, va = _at(pool, k_new, "k_new", dtype), _at(pool, v_new, "v_new", dtype)
    sa = _at(pool, slot_mapping, "slot_mapping", torch.int64)
    n = slot_mapping.numel()
    if k_new.shape != (n, pool.n_kv_heads, HEAD_DIM) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new must be [n_tok][n_kv_heads][128]")
    _check(lib.pa_cache_append8(_handle8(pool), _DTYPE_CODE[dtype], ka, va, sa, n, _raw_stream(pool, stream)),
           "pa_cache_append8")


def decode8_workspace_for(pool, q, block_tables, stream=None):
    """Workspace of pa_decode8 for these sizes."""
    n = lib.pa_decode8_workspace_bytes(_handle8(pool), q.shape[0], q.shape[1], block_tables.shape[1])
    return _workspace(n, "pa_decode8_workspace_bytes", pool.device, stream)


def _decode8_args(pool, q, block_tables, seq_lens, scale, out, workspace, stream):
    """Checks of pa_decode8; the C call's arguments up to the stream."""
    dtype = _row_dtype(q, "q")
    qa, ta, la, oa, code, B, Hq, W = _decode_at(pool, q, block_tables, seq_lens, out, dtype)
    if workspace is None:
        workspace = decode8_workspace_for(pool, q, block_tables, stream)
    return (_handle8(pool), qa, _DTYPE_CODE[dtype], ta, W, la, B, Hq, float(scale), oa, code,
            _at(pool, workspace, "workspace", torch.uint8), workspace.numel()), workspace


def pa_decode8(pool, q, block_tables, seq_lens, scale, out, workspace=None, stream=None):
    """Decode attention over a Pool8: q [B][Hq][128] fp16 or bf16, out [B][Hq][128]
    of fp16, bf16 or fp32, tables and lengths as for pa_decode."""
    args, _own = _decode8_args(pool, q, block_tables, seq_lens, scale, out, workspace, stream)
    _check(lib.pa_decode8(*args, _raw_stream(pool, stream)), "pa_decode8")


def pa_selftest_decode8_timeout(pool, q, block_tables, seq_lens, scale, out, limit_ns, cta=-1, workspace=None, stream=None):
    """pa_decode8 some of whose loads do not come, in one CTA or (-1) all: their
    waits give up after limit_ns and PA_ERR_TIMEOUT is recorded (read it with
    pa_check8).  Returns the launch status."""
    args, _own = _decode8_args(pool, q, block_tables, seq_lens, scale, out, workspace, stream)
    return lib.pa_selftest_decode8_timeout(*args, int(cta), int(limit_ns), _raw_stream(pool, stream))


def _block_ids(pool, t, name, n=None):
    a = _at(pool, t, name, torch.int32)
    if t.dim() != 1 or (n is not None and t.numel() != n):
        raise ValueError(f"{name} must be [n], as long as src")
    return a


def _both_pools(pool, pool8):
    if not isinstance(pool8, Pool8) or isinstance(pool, Pool8):
        raise TypeError("one Pool and one Pool8 are needed")


def pa_copy_blocks8(pool, src, dst, stream=None):
    """pa_copy_blocks for a Pool8."""
    sa = _block_ids(pool, src, "src")
    _check(lib.pa_copy_blocks8(_handle8(pool), sa, _block_ids(pool, dst, "dst", src.numel()), src.numel(),
                               _raw_stream(pool, stream)), "pa_copy_blocks8")


def pa_quantize_blocks(pool, src, pool8, dst, rows=None, stream=None):
    """Blocks src of a Pool into blocks dst of a Pool8; rows int32 [n]: how many
    rows of each count (None: all 16; see include/pa.h)."""
    _both_pools(pool, pool8)
    sa = _block_ids(pool8, src, "src")
    da = _block_ids(pool8, dst, "dst", src.numel())
    ra = None if rows is None else _block_ids(pool8, rows, "rows", src.numel())
    _check(lib.pa_quantize_blocks(pool.handle, sa, _handle8(pool8), da, ra, src.numel(), _raw_stream(pool8, stream)),
           "pa_quantize_blocks")


def pa_dequantize_blocks(pool8, src, pool, dst, stream=None):
    """Blocks src of a Pool8 into blocks dst of a Pool."""
    _both_pools(pool, pool8)
    sa = _block_ids(pool8, src, "src")
    _check(lib.pa_dequantize_blocks(_handle8(pool8), sa, pool.handle, _block_ids(pool8, dst, "dst", src.numel()), src.numel(),
                                    _raw_stream(pool8, stream)), "pa_dequantize_blocks")


def pa_check8(pool, stream=None):
    """pa_check for a Pool8."""
    detail = ctypes.c_int64()
    code = lib.pa_check8(_handle8(pool), _stream(stream), ctypes.byref(detail))
    return code, detail.value


def shared_workspace_for(pool, q, block_tables, prefix_blocks, stream=None):
    """Workspace of pa_decode_shared for these sizes."""
    n = lib.pa_decode_shared_workspace_bytes(pool.handle, q.shape[0], q.shape[1], block_tables.shape[1],
                                             prefix_blocks.shape[0])
    return _workspace(n, "pa_decode_shared_workspace_bytes", pool.device, stream)


def _shared_args(pool, q, block_tables, seq_lens, scale, out, group_start, members, prefix_blocks, workspace, stream):
    """Checks of pa_decode_shared; the C call's arguments up to the stream."""
    qa, ta, la, oa, code, B, Hq, W = _decode_at(pool, q, block_tables, seq_lens, out)
    ga = _at(pool, group_start, "group_start", torch.int32)
    ma = _at(pool, members, "members", torch.int32)
    pa_ = _at(pool, prefix_blocks, "prefix_blocks", torch.int32)
    ng, nm = prefix_blocks.numel(), members.numel()
    if prefix_blocks.dim() != 1 or members.dim() != 1 or group_start.shape != (ng + 1,):
        raise ValueError("shapes: group_start [n_groups+1], members [n_members], prefix_blocks [n_groups]")
    if workspace is None:
        workspace = shared_workspace_for(pool, q, block_tables, prefix_blocks, stream)
    wa = _at(pool, workspace, "workspace", torch.uint8)
    return (pool.handle, qa, ta, W, la, B, Hq, float(scale), ga, ma, nm, pa_, ng, oa, code, wa, workspace.numel()), workspace


def pa_decode_shared(pool, q, block_tables, seq_lens, scale, out, group_start, members, prefix_blocks, workspace=None,
                     stream=None):
    """pa_decode with each group's shared prefix attended once for all of its
    members, groups of any size (see include/pa.h); the group arrays are int32
    device tensors (cascade_groups with max_members=B finds them)."""
    args, _own = _shared_args(pool, q, block_tables, seq_lens, scale, out, group_start, members, prefix_blocks, workspace,
                              stream)  # (_own: a workspace made for this call lives until it is launched)
    _check(lib.pa_decode_shared(*args, _raw_stream(pool, stream)), "pa_decode_shared")


def pa_selftest_shared_timeout(pool, q, block_tables, seq_lens, scale, out, group_start, members, prefix_blocks, limit_ns,
                               workspace=None, stream=None):
    """pa_decode_shared whose prefix product gets no loads: its waits give up
    after limit_ns and PA_ERR_TIMEOUT is recorded (read it with pa_check).
    Returns the launch status."""
    args, _own = _shared_args(pool, q, block_tables, seq_lens, scale, out, group_start, members, prefix_blocks, workspace,
                              stream)
    return lib.pa_selftest_shared_timeout(*args, int(limit_ns), _raw_stream(pool, stream))


def weights_workspace_for(pool, q, block_tables, stream=None):
    """Workspace of pa_decode_weights for these sizes."""
    n = lib.pa_decode_weights_workspace_bytes(pool.handle, q.shape[0], q.shape[1], block_tables.shape[1])
    return _workspace(n, "pa_decode_weights_workspace_bytes", pool.device, stream)


def _per_token_at(pool, t, name, B, W, dtype):
    a = _at(pool, t, name, dtype)
    if t.shape != (B, pool.n_kv_heads, W * BLOCK_SIZE):
        raise ValueError(f"{name} must be [B][n_kv_heads][16 * W]")
    return a


def pa_decode_weights(pool, q, block_tables, seq_lens, scale, out, weights, decay=1.0, workspace=None, stream=None):
    """pa_decode_split that also adds each cached token's attention weight to
    weights [B][Hkv][16*W] (fp32): weights = decay * weights + the weights of
    this step, summed over the query heads of a kv head (see include/pa.h)."""
    qa, ta, la, oa, code, B, Hq, W = _decode_at(pool, q, block_tables, seq_lens, out)
    wa = _per_token_at(pool, weights, "weights", B, W, torch.float32)
    if workspace is None:
        workspace = weights_workspace_for(pool, q, block_tables, stream)
    _check(lib.pa_decode_weights(pool.handle, qa, ta, W, la, B, Hq, float(scale), oa, code, wa, float(decay),
                                 _at(pool, workspace, "workspace", torch.uint8), workspace.numel(),
                                 _raw_stream(pool, stream)), "pa_decode_weights")


def pa_evict(pool, weights, block_tables, seq_lens, keep, seq_lens_out, kept, n_sink=0, n_recent=0, dst_tables=None,
             weights_out=None, stream=None):
    """Keeps the heaviest keep[i] tokens of each kv head of sequence i, with the
    first n_sink and the last n_recent always among them, and closes the cache
    up in order (see include/pa.h).  In place unless dst_tables [B][Wd] is given;
    weights_out defaults to weights.  seq_lens_out int32 [B] and kept int32
    [B][Hkv][16*W] are written."""
    ta = _at(pool, block_tables, "block_tables", torch.int32)
    la = _at(pool, seq_lens, "seq_lens", torch.int32)
    ka = _at(pool, keep, "keep", torch.int32)
    na = _at(pool, seq_lens_out, "seq_lens_out", torch.int32)
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [B][W]")
    B, W = block_tables.shape
    if seq_lens.shape != (B,) or keep.shape != (B,) or seq_lens_out.shape != (B,):
        raise ValueError("seq_lens, keep and seq_lens_out must be [B]")
    wa = _per_token_at(pool, weights, "weights", B, W, torch.float32)
    oa = wa if weights_out is None else _per_token_at(pool, weights_out, "weights_out", B, W, torch.float32)
    xa = _per_token_at(pool, kept, "kept", B, W, torch.int32)
    da, Wd = None, 0
    if dst_tables is not None:
        da = _at(pool, dst_tables, "dst_tables", torch.int32)
        if dst_tables.dim() != 2 or dst_tables.shape[0] != B:
            raise ValueError("dst_tables must be [B][Wd]")
        Wd = dst_tables.shape[1]
        if Wd == 0:  # (an empty tensor has a null address, which would mean in place)
            raise PagedAttentionError(PA_ERR_INVALID, "pa_evict")
    _check(lib.pa_evict(pool.handle, wa, oa, ta, W, da, Wd, la, ka, B, _int32(n_sink), _int32(n_recent), na, xa,
                        _raw_stream(pool, stream)), "pa_evict")


def pa_copy_blocks(pool, src, dst, stream=None):
    _need(src, "src", torch.int32); _need(dst, "dst", torch.int32)
    if src.numel() != dst.numel():
        raise ValueError("src and dst must have the same length")
    _check(lib.pa_copy_blocks(pool.handle, _ptr(src), _ptr(dst), src.numel(), _stream(stream)),
           "pa_copy_blocks")


def pa_profile_start(capacity):
    """Time the main decode kernel of the next `capacity` decode calls."""
    _check(lib.pa_profile_start(int(capacity)), "pa_profile_start")


def pa_profile_stop(cap=1 << 20):
    """Milliseconds of each recorded decode kernel (list of floats)."""
    import numpy as np
    buf = np.zeros(max(1, cap), dtype=np.float32)
    n = lib.pa_profile_stop(buf.ctypes.data_as(ctypes.POINTER(ctypes.c_float)), cap)
    if n < 0:
        _check(n, "pa_profile_stop")
    return buf[:min(n, cap)].tolist()


def pa_selftest_wait_timeout(pool, limit_ns, stream=None):
    """Runs the kernels' bounded wait on a barrier nothing arrives at; it gives
    up after limit_ns and records PA_ERR_TIMEOUT (read it with pa_check).
    Returns the launch status."""
    return lib.pa_selftest_wait_timeout(pool.handle, int(limit_ns), _stream(stream))


def pa_check(pool, stream=None):
    """Synchronises the stream and returns (status, detail) of the pool's device
    error word, clearing it."""
    detail = ctypes.c_int64()
    code = lib.pa_check(pool.handle, _stream(stream), ctypes.byref(detail))
    return code, detail.value


class BlockAllocator:
    """The library's host block allocator (pa_alloc_*)."""

    def __init__(self, num_blocks, block_size=BLOCK_SIZE, free_order=None):
        self._h = ctypes.c_void_p()
        arr = None
        if free_order is not None:
            arr = (ctypes.c_int32 * num_blocks)(*[int(b) for b in free_order])
        _check(lib.pa_alloc_create(num_blocks, block_size, arr, ctypes.byref(self._h)), "pa_alloc_create")
        self.num_blocks, self.block_size = num_blocks, block_size

    def __del__(self):
        try:
            if self._h:
                lib.pa_alloc_destroy(self._h)
                self._h = ctypes.c_void_p()
        except Exception:
            pass

    def seq_add(self, seq):
        _check(lib.pa_alloc_seq_add(self._h, seq), "pa_alloc_seq_add")

    def fork(self, parent, child):
        _check(lib.pa_alloc_fork(self._h, parent, child), "pa_alloc_fork")

    def append_slot(self, seq):
        slot, cs, cd = ctypes.c_int64(), ctypes.c_int32(), ctypes.c_int32()
        code = lib.pa_alloc_append_slot(self._h, seq, ctypes.byref(slot), ctypes.byref(cs), ctypes.byref(cd))
        if code == PA_ERR_OOM:
            raise MemoryError("no free block")
        _check(code, "pa_alloc_append_slot")
        return slot.value, cs.value, cd.value

    def extend(self, seq, n):
        """n appends; returns (slots int64 list, (cow_src, cow_dst))."""
        import numpy as np
        slots = np.zeros(max(n, 1), dtype=np.int64)
        cs, cd, done = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int()
        code = lib.pa_alloc_extend(self._h, seq, n, slots.ctypes.data_as(ctypes.c_void_p), ctypes.byref(cs),
                                   ctypes.byref(cd), ctypes.byref(done))
        if code == PA_ERR_OOM:
            raise MemoryError(f"no free block after {done.value} tokens")
        _check(code, "pa_alloc_extend")
        return slots[:n], (cs.value, cd.value)

    def seq_add_cached(self, seq, tokens):
        """New sequence sharing the cached full blocks of `tokens` (a prompt of
        token ids); returns the number of tokens it now holds."""
        import numpy as np
        arr = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
        n = ctypes.c_int()
        _check(lib.pa_alloc_seq_add_cached(self._h, seq, arr.ctypes.data_as(ctypes.c_void_p) if arr.size else None,
                                           int(arr.size), ctypes.byref(n)), "pa_alloc_seq_add_cached")
        return n.value

    def append_token(self, seq, token):
        slot, cs, cd = ctypes.c_int64(), ctypes.c_int32(), ctypes.c_int32()
        code = lib.pa_alloc_append_token(self._h, seq, int(token), ctypes.byref(slot), ctypes.byref(cs),
                                         ctypes.byref(cd))
        if code == PA_ERR_OOM:
            raise MemoryError("no free block")
        _check(code, "pa_alloc_append_token")
        return slot.value, cs.value, cd.value

    def block_hash(self, block):
        h = ctypes.c_uint64()
        r = lib.pa_alloc_block_hash(self._h, block, ctypes.byref(h))
        if r < 0:
            _check(r, "pa_alloc_block_hash")
        return h.value if r == 1 else None

    def prefix_stats(self):
        q, h, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(lib.pa_alloc_prefix_stats(self._h, ctypes.byref(q), ctypes.byref(h), ctypes.byref(c)),
               "pa_alloc_prefix_stats")
        return q.value, h.value, c.value

    def evict(self, seqs, keep):
        """Shrinks sequences for a pa_evict call (see pa_alloc_evict): read the
        old tables before and the new ones after."""
        n = len(seqs)
        if len(keep) != n:
            raise ValueError("seqs and keep must have the same length")
        code = lib.pa_alloc_evict(self._h, (ctypes.c_int * max(n, 1))(*[int(x) for x in seqs]),
                                  (ctypes.c_int * max(n, 1))(*[_int32(x) for x in keep]), n)
        if code == PA_ERR_OOM:
            raise MemoryError("no free block")
        _check(code, "pa_alloc_evict")

    def seq_free(self, seq):
        _check(lib.pa_alloc_seq_free(self._h, seq), "pa_alloc_seq_free")

    def table(self, seq):
        import numpy as np
        n = ctypes.c_int()
        _check(lib.pa_alloc_table(self._h, seq, None, 0, ctypes.byref(n)), "pa_alloc_table")
        out = np.zeros(max(n.value, 1), dtype=np.int32)
        _check(lib.pa_alloc_table(self._h, seq, out.ctypes.data_as(ctypes.c_void_p), n.value, ctypes.byref(n)),
               "pa_alloc_table")
        return out[:n.value].tolist()

    def seq_len(self, seq):
        r = lib.pa_alloc_seq_len(self._h, seq)
        if r < 0:
            _check(r, "pa_alloc_seq_len")
        return r

    def refcount(self, block):
        r = lib.pa_alloc_refcount(self._h, block)
        if r < 0:
            _check(r, "pa_alloc_refcount")
        return r

    def num_free(self):
        return lib.pa_alloc_num_free(self._h)
