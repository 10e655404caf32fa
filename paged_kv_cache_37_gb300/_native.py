"""ctypes binding of libpagedkv.so (the C ABI declared in include/pagedkv.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Functions keep the C names; device buffers are torch CUDA tensors
(their data pointers are passed through), block tables and lengths are int32
CUDA tensors, and the stream defaults to torch's current stream.  A failing
call raises PagedKVError carrying the library's status and message.  There is
no fallback: if the library is not built, or a device call fails, the call
raises.
"""
import ctypes
import os

from . import build as _build_mod

PF_OK = 0
PF_ERR_INVALID = 1
PF_ERR_OOM = 2
PF_ERR_DOUBLE_FREE = 3
PF_ERR_CUDA = 4
PF_ERR_UNSUPPORTED = 5

PF_F16 = 1
PF_F32 = 2
PF_E4M3 = 3

PF_DEV_BAD_BLOCK_ID = 1
PF_DEV_BAD_LENGTH = 2
PF_DEV_BAD_POSITION = 4
PF_DEV_WAIT_TIMEOUT = 8
PF_DEV_NONFINITE = 16
PF_STEP_OVERLAP_PREVIOUS = 1
PF_ROPE_INTERLEAVED = 1

_lib = None


class PagedKVError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"[status {status}] {message}")
        self.status = status


class OutOfBlocks(PagedKVError):
    pass


class DoubleFree(PagedKVError):
    pass


def build(force=False, verbose=False):
    """Compile the library in-tree for sm_103a (see build.py)."""
    return _build_mod.build(force=force, verbose=verbose)


def lib():
    """Load libpagedkv.so (it must have been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build_mod.LIB
    if not os.path.exists(path):
        raise PagedKVError(PF_ERR_UNSUPPORTED,
                           f"{path} is not built; call paged_kv_cache_37_gb300.build() first")
    L = ctypes.CDLL(path)
    P, I, Z, F, U64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_uint64
    I64 = ctypes.c_int64
    sigs = {
        "pf_last_error": (ctypes.c_char_p, []),
        "pf_abi_version": (I, []),
        "pf_pool_bytes": (Z, [I, I, I, I, I, I]),
        "pf_pool_create": (I, [ctypes.POINTER(P), P, P, I, I, I, I, I, I]),
        "pf_pool_create_e4m3": (I, [ctypes.POINTER(P), P, P, P, P, I, I, I, I, I]),
        "pf_scale_bytes": (Z, [I, I, I]),
        "pf_pool_destroy": (I, [P]),
        "pf_alloc_create": (I, [ctypes.POINTER(P), I, U64]),
        "pf_alloc_destroy": (I, [P]),
        "pf_alloc_blocks": (I, [P, I, P]),
        "pf_free_blocks": (I, [P, P, I]),
        "pf_alloc_free_count": (I, [P]),
        "pf_seq_reserve": (I, [P, I, P, I, I, I]),
        "pf_seq_release": (I, [P, I, P, I]),
        "pf_alloc_share": (I, [P, P, I]),
        "pf_alloc_refcount": (I, [P, ctypes.c_int32]),
        "pf_alloc_cow": (I, [P, P, P, P]),
        "pf_alloc_compact": (I, [P, P, P, P, ctypes.POINTER(I)]),
        "pf_seq_fork": (I, [P, I, P, I, P, I]),
        "pf_block_image_bytes": (Z, [P]),
        "pf_paged_prefill_attention": (I, [P, I, P, P, I, P, P, I, I, I, F, P, I, P, Z, P]),
        "pf_prefill_workspace_bytes": (Z, [P, I, I, I, I]),
        "pf_paged_cross_attention": (I, [P, I, P, P, I, P, P, I, I, I, F, P, I, P, Z, P]),
        "pf_cross_workspace_bytes": (Z, [P, I, I, I, I]),
        "pf_paged_window_attention": (I, [P, I, P, P, I, P, P, I, I, I, F, I, I, P, I, P, Z, P]),
        "pf_window_workspace_bytes": (Z, [P, I, I, I, I, I, I]),
        "pf_paged_tree_attention": (I, [P, I, P, P, I, P, P, I, I, I, F, P, I, P, I, P, Z, P]),
        "pf_tree_workspace_bytes": (Z, [P, I, I, I, I]),
        "pf_copy_blocks": (I, [P, P, P, I, P]),
        "pf_compact_blocks": (I, [P, P, P, I, P, P, I, I, P, P]),
        "pf_swap_out": (I, [P, P, I, P, P]),
        "pf_swap_in": (I, [P, P, P, I, P]),
        "pf_write_kv": (I, [P, I, P, P, P, I, I, P, P, I, P]),
        "pf_norm_rope_write": (I, [P, I, P, I64, P, I64, P, I64, I, I, P, P, F, P, I, I, I, P, P, I, I, P, P, P, I64, P,
                                   I64, P]),
        "pf_append_kv": (I, [P, I, P, P, P, I, P, P, I, I, P]),
        "pf_gather_kv": (I, [P, I, P, I, P, P, I, P, P, P]),
        "pf_decode_workspace_bytes": (Z, [P, I, I, I, I]),
        "pf_decode_workspace_init": (I, [P, Z, P]),
        "pf_paged_decode_attention": (I, [P, I, P, P, I, P, I, I, F, P, I, I, P, Z, P]),
        "pf_device_status": (I, [ctypes.POINTER(I), I, P]),
        "pf_test_inject_wait_timeout": (I, []),
        "pf_paged_decode_attention_noalloc": (I, [P, I, P, P, I, P, I, I, F, P, I, I, P]),
        "pf_decode_step": (I, [P, I, P, P, P, P, I, P, I, I, F, P, I, I, P, Z, I, P]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def _check(rc):
    if rc != PF_OK:
        msg = lib().pf_last_error().decode(errors="replace")
        cls = {PF_ERR_OOM: OutOfBlocks, PF_ERR_DOUBLE_FREE: DoubleFree}.get(rc, PagedKVError)
        raise cls(rc, msg)


# --------------------------------------------------------------- helpers

def _dev_ptr(t, name, dtype=None, dev=None):
    """Address of a contiguous CUDA tensor, on device dev if given (an int: what
    ctypes takes for a pointer argument without a wrapper object)."""
    try:
        on = t.get_device()
    except AttributeError:
        raise TypeError(f"{name} must be a torch tensor") from None
    if dev is None or on != dev:
        if not t.is_cuda:
            raise PagedKVError(PF_ERR_INVALID, f"{name} must be a CUDA tensor")
        if dev is not None:
            raise PagedKVError(PF_ERR_INVALID, f"{name} is on {t.device}, the current device is cuda:{dev}")
    if not t.is_contiguous():
        raise PagedKVError(PF_ERR_INVALID, f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise PagedKVError(PF_ERR_INVALID, f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _rows_ptr(t, name, shape, dev, float16):
    """Address and stride between tokens (in values) of fp16 rows [T, heads,
    head_dim] on device dev, heads contiguous and tokens any distance apart."""
    if t.shape != shape:
        raise PagedKVError(PF_ERR_INVALID, f"{name} must have {shape[0]} rows of [{shape[1]}, {shape[2]}]")
    if t.get_device() != dev:
        if not t.is_cuda:
            raise PagedKVError(PF_ERR_INVALID, f"{name} must be a CUDA tensor")
        raise PagedKVError(PF_ERR_INVALID, f"{name} is on {t.device}, the current device is cuda:{dev}")
    if t.dtype is not float16:
        raise PagedKVError(PF_ERR_INVALID, f"{name} must be {float16}, got {t.dtype}")
    if t.is_contiguous():
        return t.data_ptr(), shape[1] * shape[2]
    apart, head, one = t.stride()
    if one != 1 or (shape[1] > 1 and head != shape[2]):
        raise PagedKVError(PF_ERR_INVALID, f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), apart if shape[0] > 1 else shape[1] * shape[2]


def _need_tensors(**arguments):
    """TypeError for the first argument that is no tensor (after an attribute of one was missing)."""
    import torch
    for name, t in arguments.items():
        if t is not None and not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor") from None


def _stream_ptr(stream):
    import torch
    if stream is None:
        # the raw handle of torch's current stream; building the Stream object
        # around it takes 2.9 us of a call's 11 (GB300 host), this 0.1
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _pool_device(pool):
    """The device that a call's tensors have to lie on: torch's current one
    (whose current stream the call takes by default), and the pool's."""
    import torch
    dev = torch.cuda.current_device()
    if pool.device != dev:
        raise PagedKVError(PF_ERR_INVALID, f"the pool is on cuda:{pool.device}, the current device is cuda:{dev}")
    return dev


def _host_i32(a, name):
    import numpy as np
    if not isinstance(a, np.ndarray) or a.dtype != np.int32 or not a.flags.c_contiguous:
        raise TypeError(f"{name} must be a C-contiguous numpy int32 array")
    return a.ctypes.data_as(ctypes.c_void_p)


# ------------------------------------------------------------------ ABI

def pf_last_error():
    return lib().pf_last_error().decode(errors="replace")


def pf_abi_version():
    return lib().pf_abi_version()


def pf_pool_bytes(n_layers, n_blocks, block_size, n_kv_heads, head_dim, dtype=PF_F16):
    return lib().pf_pool_bytes(n_layers, n_blocks, block_size, n_kv_heads, head_dim, dtype)


class Pool:
    """Handle of a pf_pool over two caller-owned [L, N, B, Hkv, D] tensors, fp16
    or e4m3 with [L, N, Hkv] fp32 scales (kept referenced here so they outlive
    the handle)."""

    def __init__(self, handle, k_pool, v_pool, k_scale=None, v_scale=None):
        self.handle = handle
        self.k_pool = k_pool
        self.v_pool = v_pool
        self.k_scale = k_scale
        self.v_scale = v_scale
        self.device = k_pool.get_device()
        self.n_layers, self.n_blocks, self.block_size, self.n_kv_heads, self.head_dim = k_pool.shape

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.pf_pool_destroy(self.handle)
            self.handle = None


def pf_scale_bytes(n_layers, n_blocks, n_kv_heads):
    return lib().pf_scale_bytes(n_layers, n_blocks, n_kv_heads)


def pf_pool_create_e4m3(k_pool, v_pool, k_scale, v_scale):
    """8-bit pool: torch.float8_e4m3fn tensors [L, N, B, Hkv, D] and fp32
    scales [L, N, Hkv], filled by pf_append_kv."""
    import torch
    if k_pool.dim() != 5 or k_pool.shape != v_pool.shape:
        raise PagedKVError(PF_ERR_INVALID, "pools must both be [n_layers, n_blocks, block_size, n_kv_heads, head_dim]")
    L, N, B, H, D = k_pool.shape
    if k_scale is None or v_scale is None or tuple(k_scale.shape) != (L, N, H) or tuple(v_scale.shape) != (L, N, H):
        raise PagedKVError(PF_ERR_INVALID, "an e4m3 pool needs k_scale and v_scale [n_layers, n_blocks, n_kv_heads]")
    if len({t.get_device() for t in (k_pool, v_pool, k_scale, v_scale)}) != 1:
        raise PagedKVError(PF_ERR_INVALID, "pools and scales must lie on one device")
    h = ctypes.c_void_p()
    _check(lib().pf_pool_create_e4m3(ctypes.byref(h), _dev_ptr(k_pool, "k_pool", torch.float8_e4m3fn),
                                     _dev_ptr(v_pool, "v_pool", torch.float8_e4m3fn),
                                     _dev_ptr(k_scale, "k_scale", torch.float32),
                                     _dev_ptr(v_scale, "v_scale", torch.float32), L, N, B, H, D))
    return Pool(h, k_pool, v_pool, k_scale, v_scale)


def pf_pool_create(k_pool, v_pool, k_scale=None, v_scale=None):
    """Pool over fp16 tensors, or over torch.float8_e4m3fn tensors and their
    scales (pf_pool_create_e4m3)."""
    import torch
    if k_pool.dtype == torch.float8_e4m3fn:
        return pf_pool_create_e4m3(k_pool, v_pool, k_scale, v_scale)
    if k_scale is not None or v_scale is not None:
        raise PagedKVError(PF_ERR_INVALID, "an fp16 pool has no scales")
    if k_pool.dim() != 5 or k_pool.shape != v_pool.shape:
        raise PagedKVError(PF_ERR_INVALID, "pools must both be [n_layers, n_blocks, block_size, n_kv_heads, head_dim]")
    kp = _dev_ptr(k_pool, "k_pool", torch.float16)
    vp = _dev_ptr(v_pool, "v_pool", torch.float16)
    h = ctypes.c_void_p()
    L, N, B, H, D = k_pool.shape
    _check(lib().pf_pool_create(ctypes.byref(h), kp, vp, L, N, B, H, D, PF_F16))
    return Pool(h, k_pool, v_pool)


def pf_pool_destroy(pool):
    if pool.handle:
        _check(lib().pf_pool_destroy(pool.handle))
        pool.handle = None


class Allocator:
    """Handle of a pf_alloc (host free list)."""

    def __init__(self, handle, n_blocks):
        self.handle = handle
        self.n_blocks = n_blocks

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.pf_alloc_destroy(self.handle)
            self.handle = None


def pf_alloc_create(n_blocks, shuffle_seed=0):
    h = ctypes.c_void_p()
    _check(lib().pf_alloc_create(ctypes.byref(h), n_blocks, shuffle_seed))
    return Allocator(h, n_blocks)


def pf_alloc_destroy(alloc):
    if alloc.handle:
        _check(lib().pf_alloc_destroy(alloc.handle))
        alloc.handle = None


def pf_alloc_blocks(alloc, n):
    import numpy as np
    ids = np.zeros(max(n, 1), dtype=np.int32)
    _check(lib().pf_alloc_blocks(alloc.handle, n, ids.ctypes.data_as(ctypes.c_void_p)))
    return ids[:n]


def pf_free_blocks(alloc, ids):
    import numpy as np
    ids = np.ascontiguousarray(ids, dtype=np.int32)
    _check(lib().pf_free_blocks(alloc.handle, ids.ctypes.data_as(ctypes.c_void_p), ids.size))


def pf_alloc_compact(alloc):
    """Pack the referenced blocks into the lowest ids.  Returns (src, dst,
    block_map), host int32 arrays: move the contents and the device tables
    with pf_compact_blocks, host rows by block_map[row]."""
    import numpy as np
    src, dst, block_map = (np.zeros(alloc.n_blocks, dtype=np.int32) for _ in range(3))
    n = ctypes.c_int()
    _check(lib().pf_alloc_compact(alloc.handle, *(a.ctypes.data_as(ctypes.c_void_p) for a in (src, dst, block_map)),
                                  ctypes.byref(n)))
    return src[:n.value].copy(), dst[:n.value].copy(), block_map


def pf_alloc_free_count(alloc):
    return lib().pf_alloc_free_count(alloc.handle)


def pf_seq_reserve(alloc, block_size, table_row, cur_len, new_len):
    """Grow one sequence; table_row is a host int32 numpy row, updated in place."""
    _check(lib().pf_seq_reserve(alloc.handle, block_size, _host_i32(table_row, "table_row"),
                                table_row.size, cur_len, new_len))


def pf_seq_release(alloc, block_size, table_row, length):
    _check(lib().pf_seq_release(alloc.handle, block_size, _host_i32(table_row, "table_row"), length))


def pf_alloc_share(alloc, ids):
    """One more reference on each listed block (a fork's shared prefix)."""
    import numpy as np
    ids = np.ascontiguousarray(ids, dtype=np.int32)
    _check(lib().pf_alloc_share(alloc.handle, ids.ctypes.data_as(ctypes.c_void_p), ids.size))


def pf_alloc_refcount(alloc, block):
    return lib().pf_alloc_refcount(alloc.handle, int(block))


def pf_alloc_cow(alloc, table_row, j):
    """Copy-on-write of table_row[j] (host int32 numpy row, patched in place)
    before a write into that block.  Returns None when the block is the
    writer's own, else (old block, new block) for pf_copy_blocks."""
    import numpy as np
    if not isinstance(table_row, np.ndarray) or table_row.dtype != np.int32:
        raise TypeError("table_row must be a numpy int32 array")
    entry = table_row[j:j + 1]
    src, dst = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().pf_alloc_cow(alloc.handle, entry.ctypes.data_as(ctypes.c_void_p), ctypes.byref(src),
                              ctypes.byref(dst)))
    return None if dst.value < 0 else (src.value, dst.value)


def pf_seq_fork(alloc, block_size, parent_row, length, child_row):
    """child_row[:ceil(length/B)] = parent_row's blocks, shared (host int32 rows)."""
    _check(lib().pf_seq_fork(alloc.handle, block_size, _host_i32(parent_row, "parent_row"), length,
                             _host_i32(child_row, "child_row"), child_row.size))


def pf_block_image_bytes(pool):
    return lib().pf_block_image_bytes(pool.handle)


def pf_copy_blocks(pool, src_ids, dst_ids, stream=None):
    """Block dst_ids[i] := block src_ids[i], every layer, K and V (device int32)."""
    import torch
    n = src_ids.numel()
    if dst_ids.numel() != n:
        raise PagedKVError(PF_ERR_INVALID, "src_ids and dst_ids must have the same length")
    dev = None if pool.k_scale is None else _pool_device(pool)
    _check(lib().pf_copy_blocks(pool.handle, _dev_ptr(src_ids, "src_ids", torch.int32, dev),
                                _dev_ptr(dst_ids, "dst_ids", torch.int32, dev), n, _stream_ptr(stream)))


def pf_compact_blocks(pool, src_ids, dst_ids, block_map, block_tables, context_lens, stream=None):
    """Block dst_ids[i] := block src_ids[i] in every layer, and the used entries
    of block_tables (in place) through block_map, in one launch (device int32)."""
    import torch
    n = src_ids.numel()
    if dst_ids.numel() != n:
        raise PagedKVError(PF_ERR_INVALID, "src_ids and dst_ids must have the same length")
    if block_map.numel() != pool.n_blocks:
        raise PagedKVError(PF_ERR_INVALID, "block_map must have n_blocks entries")
    if block_tables.dim() != 2 or context_lens.numel() != block_tables.shape[0]:
        raise PagedKVError(PF_ERR_INVALID, "block_tables must be [n_rows, max_blocks]; context_lens [n_rows]")
    dev = _pool_device(pool)
    _check(lib().pf_compact_blocks(pool.handle, _dev_ptr(src_ids, "src_ids", torch.int32, dev),
                                   _dev_ptr(dst_ids, "dst_ids", torch.int32, dev), n,
                                   _dev_ptr(block_map, "block_map", torch.int32, dev),
                                   _dev_ptr(block_tables, "block_tables", torch.int32, dev), block_tables.shape[0],
                                   block_tables.shape[1], _dev_ptr(context_lens, "context_lens", torch.int32, dev),
                                   _stream_ptr(stream)))


def _pinned_ptr(t, name, nbytes):
    import torch
    if not isinstance(t, torch.Tensor) or t.is_cuda or not t.is_pinned() or not t.is_contiguous():
        raise PagedKVError(PF_ERR_INVALID, f"{name} must be a contiguous pinned host tensor")
    if t.numel() * t.element_size() < nbytes:
        raise PagedKVError(PF_ERR_INVALID, f"{name} holds {t.numel() * t.element_size()} bytes, needs {nbytes}")
    return ctypes.c_void_p(t.data_ptr())


def pf_swap_out(pool, ids, host_dst, stream=None):
    """Images of blocks ids (device int32) into the pinned host tensor host_dst."""
    import torch
    n = ids.numel()
    ptr = _pinned_ptr(host_dst, "host_dst", n * pf_block_image_bytes(pool))
    dev = None if pool.k_scale is None else _pool_device(pool)
    _check(lib().pf_swap_out(pool.handle, _dev_ptr(ids, "ids", torch.int32, dev), n, ptr, _stream_ptr(stream)))


def pf_swap_in(pool, host_src, ids, stream=None):
    """Blocks ids (device int32) take the images in the pinned host tensor host_src."""
    import torch
    n = ids.numel()
    ptr = _pinned_ptr(host_src, "host_src", n * pf_block_image_bytes(pool))
    dev = None if pool.k_scale is None else _pool_device(pool)
    _check(lib().pf_swap_in(pool.handle, ptr, _dev_ptr(ids, "ids", torch.int32, dev), n, _stream_ptr(stream)))


def pf_prefill_workspace_bytes(pool, n_seqs, n_q_heads, max_blocks_per_seq, max_new_tokens):
    """Workspace bytes of the decode-kernel path of pf_paged_prefill_attention
    (0: that path does not apply, no workspace needed)."""
    return lib().pf_prefill_workspace_bytes(pool.handle, n_seqs, n_q_heads, max_blocks_per_seq, max_new_tokens)


def pf_paged_prefill_attention(pool, layer, q, block_tables, context_lens, cu_q, max_new_tokens, scale, out,
                               workspace=None, stream=None):
    """Causal attention of each sequence's last n_s = cu_q[s+1] - cu_q[s]
    tokens (q rows cu_q[s]..cu_q[s+1]-1) over its context (device tensors).
    With a workspace, short appends run on the decode kernel."""
    import torch
    n = context_lens.numel()
    if block_tables.dim() != 2 or block_tables.shape[0] != n or cu_q.numel() != n + 1:
        raise PagedKVError(PF_ERR_INVALID, "block_tables must be [n_seqs, max_blocks]; cu_q [n_seqs + 1]")
    if q.dim() != 3 or q.shape[2] != pool.head_dim or tuple(out.shape) != tuple(q.shape):
        raise PagedKVError(PF_ERR_INVALID, "q must be [T_q, n_q_heads, head_dim], out must have the shape of q")
    dev = None if pool.k_scale is None else _pool_device(pool)
    out_dtype = {torch.float16: PF_F16, torch.float32: PF_F32}.get(out.dtype)
    if out_dtype is None:
        raise PagedKVError(PF_ERR_INVALID, "out must be float16 or float32")
    _check(lib().pf_paged_prefill_attention(
        pool.handle, layer, _dev_ptr(q, "q", torch.float16, dev),
        _dev_ptr(block_tables, "block_tables", torch.int32, dev), block_tables.shape[1],
        _dev_ptr(context_lens, "context_lens", torch.int32, dev),
        _dev_ptr(cu_q, "cu_q", torch.int32, dev), n, int(max_new_tokens), q.shape[1], float(scale),
        _dev_ptr(out, "out", None, dev), out_dtype,
        None if workspace is None else _dev_ptr(workspace, "workspace", None, dev),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream_ptr(stream)))


def pf_cross_workspace_bytes(pool, n_seqs, n_q_heads, max_blocks_per_seq, max_q_tokens):
    """Workspace bytes of pf_paged_cross_attention (0: it needs none)."""
    return lib().pf_cross_workspace_bytes(pool.handle, n_seqs, n_q_heads, max_blocks_per_seq, max_q_tokens)


def pf_paged_cross_attention(pool, layer, q, block_tables, context_lens, cu_q, max_q_tokens, scale, out,
                             workspace=None, stream=None):
    """Attention of each sequence's queries (q rows cu_q[s]..cu_q[s+1]-1) over
    all of its context, whose length is its own (device tensors).  With a
    workspace, calls of few rows are cut over the SMs."""
    import torch
    n = context_lens.numel()
    if block_tables.dim() != 2 or block_tables.shape[0] != n or cu_q.numel() != n + 1:
        raise PagedKVError(PF_ERR_INVALID, "block_tables must be [n_seqs, max_blocks]; cu_q [n_seqs + 1]")
    if q.dim() != 3 or q.shape[2] != pool.head_dim or tuple(out.shape) != tuple(q.shape):
        raise PagedKVError(PF_ERR_INVALID, "q must be [T_q, n_q_heads, head_dim], out of its shape")
    out_dtype = {torch.float16: PF_F16, torch.float32: PF_F32}.get(out.dtype)
    if out_dtype is None:
        raise PagedKVError(PF_ERR_INVALID, "out must be float16 or float32")
    dev = _pool_device(pool)
    if q.numel() == 0:
        return
    _check(lib().pf_paged_cross_attention(
        pool.handle, layer, _dev_ptr(q, "q", torch.float16, dev),
        _dev_ptr(block_tables, "block_tables", torch.int32, dev), block_tables.shape[1],
        _dev_ptr(context_lens, "context_lens", torch.int32, dev),
        _dev_ptr(cu_q, "cu_q", torch.int32, dev), n, int(max_q_tokens), q.shape[1], float(scale),
        _dev_ptr(out, "out", None, dev), out_dtype,
        None if workspace is None else _dev_ptr(workspace, "workspace", None, dev),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream_ptr(stream)))


def _masked_args(pool, q, block_tables, context_lens, cu_q, out, workspace):
    """Checked arguments that the masked attention calls share: addresses of q,
    tables, lengths, cu_q, out and workspace, and the sizes among the arguments."""
    import torch
    try:
        shape, table = q.shape, block_tables.shape
        n = context_lens.numel()
        if len(table) != 2 or table[0] != n or (cu_q is not None and cu_q.numel() != n + 1):
            raise PagedKVError(PF_ERR_INVALID, "block_tables must be [n_seqs, max_blocks]; cu_q [n_seqs + 1]")
        if len(shape) != 3 or shape[2] != pool.head_dim or out.shape != shape:
            raise PagedKVError(PF_ERR_INVALID, "q must be [T_q, n_q_heads, head_dim], out of its shape")
        if cu_q is None and shape[0] != n:
            raise PagedKVError(PF_ERR_INVALID, "without cu_q, q must have a row per sequence")
        out_dtype = PF_F16 if out.dtype is torch.float16 else PF_F32
        if out_dtype == PF_F32 and out.dtype is not torch.float32:
            _need_tensors(out=out)
            raise PagedKVError(PF_ERR_INVALID, "out must be float16 or float32")
        dev, i32 = _pool_device(pool), torch.int32
        return (dev, shape[0], n, shape[1], table[1], out_dtype, _dev_ptr(q, "q", torch.float16, dev),
                _dev_ptr(block_tables, "block_tables", i32, dev), _dev_ptr(context_lens, "context_lens", i32, dev),
                None if cu_q is None else _dev_ptr(cu_q, "cu_q", i32, dev), _dev_ptr(out, "out", None, dev),
                None if workspace is None else _dev_ptr(workspace, "workspace", None, dev),
                0 if workspace is None else workspace.nbytes)
    except AttributeError:
        _need_tensors(q=q, block_tables=block_tables, context_lens=context_lens, cu_q=cu_q, out=out, workspace=workspace)
        raise


def pf_window_workspace_bytes(pool, n_seqs, n_q_heads, max_blocks_per_seq, max_new_tokens, window, n_sinks=0):
    """Workspace bytes of pf_paged_window_attention (0: it needs none)."""
    return lib().pf_window_workspace_bytes(pool.handle, n_seqs, n_q_heads, max_blocks_per_seq, max_new_tokens,
                                           window, n_sinks)


def pf_paged_window_attention(pool, layer, q, block_tables, context_lens, cu_q, max_new_tokens, scale, window, n_sinks,
                              out, workspace=None, stream=None):
    """Causal attention of each sequence's last tokens (q rows
    cu_q[s]..cu_q[s+1]-1; cu_q None: one each, row s) over the last `window`
    tokens up to the query's own and the first n_sinks."""
    _, rows, n, hq, width, out_dtype, q_p, bt_p, len_p, cu_p, out_p, ws_p, ws_bytes = _masked_args(
        pool, q, block_tables, context_lens, cu_q, out, workspace)
    if rows == 0:
        return
    _check(lib().pf_paged_window_attention(pool.handle, layer, q_p, bt_p, width, len_p, cu_p, n, int(max_new_tokens), hq, float(scale),
                                           int(window), int(n_sinks), out_p, out_dtype, ws_p, ws_bytes, _stream_ptr(stream)))


def pf_tree_workspace_bytes(pool, n_seqs, n_q_heads, max_blocks_per_seq, max_draft_tokens):
    """Workspace bytes of pf_paged_tree_attention (0: it needs none)."""
    return lib().pf_tree_workspace_bytes(pool.handle, n_seqs, n_q_heads, max_blocks_per_seq, max_draft_tokens)


def pf_paged_tree_attention(pool, layer, q, block_tables, context_lens, cu_q, max_draft_tokens, scale, tree, out,
                            workspace=None, stream=None):
    """Attention of each sequence's last tokens, drafts that form a tree: all see
    the tokens before them, and draft j where bit j % 64 of the query's
    tree[row, j // 64] is set (tree: int64 [T_q, words])."""
    import torch
    if cu_q is None:
        raise PagedKVError(PF_ERR_INVALID, "cu_q must be given")
    dev, rows, n, hq, width, out_dtype, q_p, bt_p, len_p, cu_p, out_p, ws_p, ws_bytes = _masked_args(
        pool, q, block_tables, context_lens, cu_q, out, workspace)
    try:
        bits = tree.shape
    except AttributeError:
        raise TypeError("tree must be a torch tensor") from None
    if len(bits) != 2 or bits[0] != rows:
        raise PagedKVError(PF_ERR_INVALID, "tree must be [T_q, words], a row per query")
    if rows == 0:
        return
    _check(lib().pf_paged_tree_attention(pool.handle, layer, q_p, bt_p, width, len_p, cu_p, n, int(max_draft_tokens), hq, float(scale),
                                         _dev_ptr(tree, "tree", torch.int64, dev), bits[1], out_p, out_dtype, ws_p, ws_bytes,
                                         _stream_ptr(stream)))


def pf_append_kv(pool, layer, k_new, v_new, block_tables, context_lens, cu_new, max_new_tokens=1, stream=None):
    """Quantise new rows into an 8-bit pool: sequence s's last
    cu_new[s+1]-cu_new[s] tokens are rows cu_new[s].. of k_new / v_new; cu_new
    None: one token per sequence with a context, row s."""
    import torch
    n = context_lens.numel()
    if k_new.dim() != 3 or tuple(k_new.shape[1:]) != (pool.n_kv_heads, pool.head_dim) or v_new.shape != k_new.shape:
        raise PagedKVError(PF_ERR_INVALID, "k_new / v_new must be [n_tokens, n_kv_heads, head_dim]")
    if block_tables.dim() != 2 or block_tables.shape[0] != n:
        raise PagedKVError(PF_ERR_INVALID, "block_tables must be [n_seqs, max_blocks]")
    if k_new.shape[0] != n if cu_new is None else cu_new.numel() != n + 1:
        raise PagedKVError(PF_ERR_INVALID, "cu_new must have n_seqs + 1 entries, or be None with one row per sequence")
    dev = _pool_device(pool)
    if k_new.numel() == 0:
        return
    _check(lib().pf_append_kv(pool.handle, layer, _dev_ptr(k_new, "k_new", torch.float16, dev),
                              _dev_ptr(v_new, "v_new", torch.float16, dev),
                              _dev_ptr(block_tables, "block_tables", torch.int32, dev), block_tables.shape[1],
                              _dev_ptr(context_lens, "context_lens", torch.int32, dev),
                              None if cu_new is None else _dev_ptr(cu_new, "cu_new", torch.int32, dev), n,
                              int(max_new_tokens), _stream_ptr(stream)))


def pf_norm_rope_write(pool, layer, q, k, v, block_tables, seq_idx, pos, angles, q_out, k_out=None, q_weight=None,
                       k_weight=None, eps=1e-6, interleaved=False, rope_pos=None, stream=None):
    """Norm (with weights, fp32 [head_dim]) and rotate q and k rows, and write K
    and V into the pages of an fp16 pool, in one launch.  angles: fp32
    [n_positions, rot_dim] (make_rope_angles), or None for no rotation; token
    i's is row rope_pos[i], or pos[i].  q [T, n_q_heads, D], k, v [T, n_kv_heads,
    D] and the outputs may be slices of wider rows (heads contiguous).  Without
    block_tables nothing is cached and k_out takes the keys; q or k None: only the
    other."""
    import torch
    f16, f32, i32 = torch.float16, torch.float32, torch.int32
    dev = _pool_device(pool)
    try:
        first = k if q is None else q
        if first is None:
            raise PagedKVError(PF_ERR_INVALID, "neither queries nor keys")
        if first.dim() != 3:
            raise PagedKVError(PF_ERR_INVALID, "q and k must be [n_tokens, heads, head_dim]")
        n, hq, D = first.shape
        if D != pool.head_dim:
            raise PagedKVError(PF_ERR_INVALID, f"q and k must have head_dim {pool.head_dim}")
        if (q is None) != (q_out is None):
            raise PagedKVError(PF_ERR_INVALID, "q needs q_out, and q_out q")
        keys = (n, pool.n_kv_heads, D)
        q_ptr = k_ptr = v_ptr = q_to = k_to = w_q = w_k = ang = rp = bt = seq = at = None
        q_apart = k_apart = v_apart = q_to_apart = k_to_apart = n_positions = rot = rows = width = 0
        if q is None:
            hq = 0
        else:
            q_ptr, q_apart = _rows_ptr(q, "q", (n, hq, D), dev, f16)
            q_to, q_to_apart = _rows_ptr(q_out, "q_out", (n, hq, D), dev, f16)
        if k is not None:
            k_ptr, k_apart = _rows_ptr(k, "k", keys, dev, f16)
        if v is not None:
            v_ptr, v_apart = _rows_ptr(v, "v", keys, dev, f16)
        if k_out is not None:
            k_to, k_to_apart = _rows_ptr(k_out, "k_out", keys, dev, f16)
        if q_weight is not None:
            if q_weight.numel() != D:
                raise PagedKVError(PF_ERR_INVALID, "q_weight must be [head_dim]")
            w_q = _dev_ptr(q_weight, "q_weight", f32, dev)
        if k_weight is not None:
            if k_weight.numel() != D:
                raise PagedKVError(PF_ERR_INVALID, "k_weight must be [head_dim]")
            w_k = _dev_ptr(k_weight, "k_weight", f32, dev)
        if angles is not None:
            if angles.dim() != 2:
                raise PagedKVError(PF_ERR_INVALID, "angles must be [n_positions, rot_dim]")
            n_positions, rot = angles.shape
            ang = _dev_ptr(angles, "angles", f32, dev)
        if rope_pos is not None:
            if rope_pos.numel() != n:
                raise PagedKVError(PF_ERR_INVALID, "rope_pos must have n_tokens entries")
            rp = _dev_ptr(rope_pos, "rope_pos", i32, dev)
        if block_tables is not None:
            if block_tables.dim() != 2:
                raise PagedKVError(PF_ERR_INVALID, "block_tables must be [n_seqs, max_blocks]")
            rows, width = block_tables.shape
            bt = _dev_ptr(block_tables, "block_tables", i32, dev)
        if seq_idx is not None:
            if seq_idx.numel() != n:
                raise PagedKVError(PF_ERR_INVALID, "seq_idx must have n_tokens entries")
            seq = _dev_ptr(seq_idx, "seq_idx", i32, dev)
        if pos is not None:
            if pos.numel() != n:
                raise PagedKVError(PF_ERR_INVALID, "pos must have n_tokens entries")
            at = _dev_ptr(pos, "pos", i32, dev)
    except AttributeError:
        _need_tensors(q=q, k=k, v=v, block_tables=block_tables, seq_idx=seq_idx, pos=pos, angles=angles, q_out=q_out,
                      k_out=k_out, q_weight=q_weight, k_weight=k_weight, rope_pos=rope_pos)
        raise
    _check(lib().pf_norm_rope_write(
        pool.handle, layer, q_ptr, q_apart, k_ptr, k_apart, v_ptr, v_apart, n, hq, w_q, w_k, float(eps), ang, n_positions,
        rot, PF_ROPE_INTERLEAVED if interleaved else 0, rp, bt, rows, width, seq, at, q_to, q_to_apart, k_to,
        k_to_apart, _stream_ptr(stream)))


def pf_write_kv(pool, layer, k_new, v_new, block_tables, seq_idx, pos, stream=None):
    import torch
    n = k_new.shape[0]
    if tuple(k_new.shape) != (n, pool.n_kv_heads, pool.head_dim) or tuple(v_new.shape) != tuple(k_new.shape):
        raise PagedKVError(PF_ERR_INVALID, "k_new / v_new must be [n_tokens, n_kv_heads, head_dim]")
    if seq_idx.numel() != n or pos.numel() != n or block_tables.dim() != 2:
        raise PagedKVError(PF_ERR_INVALID, "seq_idx / pos must have n_tokens entries; block_tables is 2-D")
    _check(lib().pf_write_kv(pool.handle, layer, _dev_ptr(k_new, "k_new", torch.float16),
                             _dev_ptr(v_new, "v_new", torch.float16),
                             _dev_ptr(block_tables, "block_tables", torch.int32),
                             block_tables.shape[0], block_tables.shape[1],
                             _dev_ptr(seq_idx, "seq_idx", torch.int32), _dev_ptr(pos, "pos", torch.int32),
                             n, _stream_ptr(stream)))


def pf_gather_kv(pool, layer, block_tables, context_lens, cu_off, k_out, v_out, stream=None):
    import torch
    n = context_lens.numel()
    if block_tables.dim() != 2 or block_tables.shape[0] != n or cu_off.numel() < n:
        raise PagedKVError(PF_ERR_INVALID, "block_tables must be [n_seqs, max_blocks]; cu_off needs n_seqs entries")
    dev = None if pool.k_scale is None else _pool_device(pool)
    _check(lib().pf_gather_kv(pool.handle, layer, _dev_ptr(block_tables, "block_tables", torch.int32, dev),
                              block_tables.shape[1], _dev_ptr(context_lens, "context_lens", torch.int32, dev),
                              _dev_ptr(cu_off, "cu_off", torch.int64, dev), n,
                              _dev_ptr(k_out, "k_out", torch.float16, dev),
                              _dev_ptr(v_out, "v_out", torch.float16, dev),
                              _stream_ptr(stream)))


def pf_decode_workspace_bytes(pool, n_seqs, n_q_heads, max_blocks_per_seq, split_tokens=0):
    b = lib().pf_decode_workspace_bytes(pool.handle, n_seqs, n_q_heads, max_blocks_per_seq, split_tokens)
    if b == 0:
        raise PagedKVError(PF_ERR_INVALID, pf_last_error())
    return b


def pf_decode_workspace_init(workspace, stream=None):
    _check(lib().pf_decode_workspace_init(_dev_ptr(workspace, "workspace"),
                                          workspace.numel() * workspace.element_size(), _stream_ptr(stream)))


def pf_paged_decode_attention(pool, layer, q, block_tables, context_lens, scale, out, split_tokens,
                              workspace, stream=None):
    import torch
    n, hq, d = q.shape
    if block_tables.dim() != 2 or block_tables.shape[0] != n or context_lens.numel() != n:
        raise PagedKVError(PF_ERR_INVALID, "block_tables must be [n_seqs, max_blocks]; context_lens [n_seqs]")
    if tuple(out.shape) != (n, hq, d) or d != pool.head_dim:
        raise PagedKVError(PF_ERR_INVALID, "q must be [n_seqs, n_q_heads, head_dim], out must have the shape of q")
    dev = None if pool.k_scale is None else _pool_device(pool)
    if out.dtype == torch.float16:
        out_dtype = PF_F16
    elif out.dtype == torch.float32:
        out_dtype = PF_F32
    else:
        raise PagedKVError(PF_ERR_INVALID, "out must be float16 or float32")
    _check(lib().pf_paged_decode_attention(
        pool.handle, layer, _dev_ptr(q, "q", torch.float16, dev),
        _dev_ptr(block_tables, "block_tables", torch.int32, dev), block_tables.shape[1],
        _dev_ptr(context_lens, "context_lens", torch.int32, dev), n, hq, float(scale),
        _dev_ptr(out, "out", None, dev), out_dtype, split_tokens, _dev_ptr(workspace, "workspace", None, dev),
        workspace.numel() * workspace.element_size(), _stream_ptr(stream)))


def pf_decode_step(pool, layer, q, k_new, v_new, block_tables, context_lens, scale, out, split_tokens, workspace,
                   flags=0, stream=None):
    """Fused decode step: write each sequence's new K/V row at position
    context_lens[s] - 1, then decode attention over the grown context.
    flags=PF_STEP_OVERLAP_PREVIOUS overlaps the launch with the previous
    kernel on the stream, which must not write context_lens or block_tables."""
    import torch
    n, hq, d = q.shape
    if block_tables.dim() != 2 or block_tables.shape[0] != n or context_lens.numel() != n:
        raise PagedKVError(PF_ERR_INVALID, "block_tables must be [n_seqs, max_blocks]; context_lens [n_seqs]")
    if tuple(k_new.shape) != (n, pool.n_kv_heads, d) or tuple(v_new.shape) != tuple(k_new.shape):
        raise PagedKVError(PF_ERR_INVALID, "k_new / v_new must be [n_seqs, n_kv_heads, head_dim]")
    if tuple(out.shape) != (n, hq, d) or d != pool.head_dim:
        raise PagedKVError(PF_ERR_INVALID, "q must be [n_seqs, n_q_heads, head_dim], out must have the shape of q")
    dev = None if pool.k_scale is None else _pool_device(pool)
    out_dtype = {torch.float16: PF_F16, torch.float32: PF_F32}.get(out.dtype)
    if out_dtype is None:
        raise PagedKVError(PF_ERR_INVALID, "out must be float16 or float32")
    _check(lib().pf_decode_step(
        pool.handle, layer, _dev_ptr(q, "q", torch.float16, dev), _dev_ptr(k_new, "k_new", torch.float16, dev),
        _dev_ptr(v_new, "v_new", torch.float16, dev), _dev_ptr(block_tables, "block_tables", torch.int32, dev),
        block_tables.shape[1], _dev_ptr(context_lens, "context_lens", torch.int32, dev), n, hq, float(scale),
        _dev_ptr(out, "out", None, dev), out_dtype, split_tokens, _dev_ptr(workspace, "workspace", None, dev),
        workspace.numel() * workspace.element_size(), int(flags), _stream_ptr(stream)))


def pf_paged_decode_attention_noalloc(pool, layer, q, block_tables, context_lens, scale, out, split_tokens,
                                      stream=None):
    """pf_paged_decode_attention without a workspace argument: the scratch is
    a fixed array inside the library, for callers that cannot allocate."""
    import torch
    n, hq, d = q.shape
    if block_tables.dim() != 2 or block_tables.shape[0] != n or context_lens.numel() != n:
        raise PagedKVError(PF_ERR_INVALID, "block_tables must be [n_seqs, max_blocks]; context_lens [n_seqs]")
    if tuple(out.shape) != (n, hq, d) or d != pool.head_dim:
        raise PagedKVError(PF_ERR_INVALID, "q must be [n_seqs, n_q_heads, head_dim], out must have the shape of q")
    out_dtype = {torch.float16: PF_F16, torch.float32: PF_F32}.get(out.dtype)
    if out_dtype is None:
        raise PagedKVError(PF_ERR_INVALID, "out must be float16 or float32")
    dev = None if pool.k_scale is None else _pool_device(pool)
    _check(lib().pf_paged_decode_attention_noalloc(
        pool.handle, layer, _dev_ptr(q, "q", torch.float16, dev),
        _dev_ptr(block_tables, "block_tables", torch.int32, dev), block_tables.shape[1],
        _dev_ptr(context_lens, "context_lens", torch.int32, dev), n, hq, float(scale),
        _dev_ptr(out, "out", None, dev), out_dtype, split_tokens, _stream_ptr(stream)))


def pf_test_inject_wait_timeout():
    """Testing hook: block 0 of the next decode-attention launch leaves one
    stage of its copy ring unfilled; the waits for it give up after 1 s (see
    the C header)."""
    _check(lib().pf_test_inject_wait_timeout())


def pf_device_status(reset=False, stream=None):
    st = ctypes.c_int(0)
    _check(lib().pf_device_status(ctypes.byref(st), 1 if reset else 0, _stream_ptr(stream)))
    return st.value
