"""ctypes binding of the C ABI in include/attn_varlen.h.

Argument marshalling only: every step of the attention runs in the CUDA
library.  There is no fallback -- if the in-tree library cannot be built or
loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import threading

from . import build as _build

# Return codes (include/attn_varlen.h)
OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED_DIM = -2
ERR_MISALIGNED = -3
ERR_UNSUPPORTED_DEVICE = -4
ERR_CUDA = -5
ERR_OOM = -6
ERR_DEVICE_TIMEOUT = -7
ERR_WORKSPACE_SMALL = -8
ERR_DRIVER = -9
ERR_NOALLOC_LIMIT = -10
ERR_BAD_BLOCK_TABLE = -11
ERR_BAD_DRAFT = -12
ERR_NO_FREE_BLOCK = -13
ERR_BAD_ROW = -14
NOALLOC_MAX_SEQS = 1024

# Every symbol the header declares, with (restype, argtypes).
_P, _I, _SZ, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
SYMBOLS = {
    "attn_varlen_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "attn_varlen_workspace_size": (_SZ, [_I]),
    "attn_varlen_fwd_ws": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _SZ, _P]),
    "attn_varlen_check": (_I, [_P]),
    "attn_varlen_check_ws": (_I, [_P, _P]),
    "attn_varlen_check_noalloc": (_I, [_P]),
    "attn_varlen_strerror": (ctypes.c_char_p, [_I]),
    "attn_varlen_version": (_I, []),
    "attn_varlen_fwd_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "attn_varlen_last_cuda_error": (ctypes.c_char_p, []),
    "attn_varlen_fwd_causal": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "attn_varlen_fwd_heads": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]),
    "paged_attn_decode": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P]),
    "chunk_delta_rule_output": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I,
                                     ctypes.c_float, _P, _P]),
    "paged_attn_tree_workspace_size": (_SZ, [_I]),
    "paged_attn_tree": (_I, [_P] * 7 + [_I] * 8 + [ctypes.c_float, _I, _P, _P, _SZ, _P]),
    "paged_attn_cache_write": (_I, [_P] * 7 + [_I] * 7 + [_L] * 4 + [_P]),
    "paged_attn_cache_accept": (_I, [_P] * 7 + [_I] * 7 + [_P, _P]),
    "paged_attn_cache_free": (_I, [_P] * 4 + [_I] * 5 + [_P]),
    "paged_attn_cache_fork_workspace_size": (_SZ, [_I, _I]),
    "paged_attn_cache_fork": (_I, [_P] * 7 + [_I] * 7 + [_P, _SZ, _P]),
    "paged_attn_cache_compact_workspace_size": (_SZ, [_I]),
    "paged_attn_cache_compact": (_I, [_P] * 5 + [_I] * 6 + [_P, _P, _P, _SZ, _P]),
}

_LOCK = threading.Lock()
_LIB = None


class AttnVarlenError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = f"{where}: {strerror(code)} (code {code})"
        if code == ERR_CUDA:
            msg += f": {load().attn_varlen_last_cuda_error().decode()}"
        super().__init__(msg)


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load the in-tree CUDA library (building it first when absent)."""
    global _LIB
    with _LOCK:
        if _LIB is None:
            path = _build.lib_path()
            if build_if_missing:
                path = _build.build()
            lib = ctypes.CDLL(path)
            for name, (res, args) in SYMBOLS.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _LIB = lib
        return _LIB


def strerror(code: int) -> str:
    return load().attn_varlen_strerror(int(code)).decode()


def workspace_size(num_seqs: int) -> int:
    return int(load().attn_varlen_workspace_size(int(num_seqs)))


def _stream_handle(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(int(stream.cuda_stream))


def _check_inputs(q, k, v, cu_q, cu_k, out):
    import torch
    if q.dtype != torch.bfloat16 or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise TypeError("q, k, v must be bfloat16")
    if q.dim() != 3 or k.dim() != 3 or v.shape != k.shape:
        raise ValueError("q, k, v must be [total_tokens, num_heads, head_dim]; k and v alike")
    if q.shape[1:] != k.shape[1:]:
        raise ValueError("q and k must share num_heads and head_dim")
    for t in (q, k, v, out):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v and out must be contiguous CUDA tensors")
    if cu_q.dtype != torch.int32 or cu_k.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    if cu_q.dim() != 1 or cu_q.shape != cu_k.shape or cu_q.numel() < 1:
        raise ValueError("cu_seqlens_q/k must be 1-D, equal length, >= 1 entry")
    if not cu_q.is_cuda or not cu_k.is_cuda or not cu_q.is_contiguous() or not cu_k.is_contiguous():
        raise ValueError("cu_seqlens must be contiguous CUDA tensors")
    if out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must have q's shape and dtype")


def attn_varlen_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, out=None, stream=None,
                    workspace=None, causal=False, heads=None):
    """softmax(q k^T / sqrt(head_dim)) v per packed sequence and head.

    q: bf16 [total_q, H, D]; k, v: bf16 [total_k, H, D]; cu_seqlens_q/k:
    int32 [num_seqs + 1] on the same device.  Returns ``out`` (allocated with
    ``torch.empty_like(q)`` when not given; rows outside every query slice are
    left untouched).  ``workspace``: optional uint8 CUDA tensor of at least
    ``workspace_size(num_seqs)`` bytes, zero-filled before first use.
    ``causal``: row r of a sequence sees keys j <= r + L_k - L_q
    (attn_varlen_fwd_causal; library-owned workspace only).  ``heads``: a
    ``(head_begin, head_count)`` pair to compute only those heads of the
    same tensors in place (attn_varlen_fwd_heads; library-owned workspace).
    """
    import torch
    if out is None:
        out = torch.empty_like(q)
    _check_inputs(q, k, v, cu_seqlens_q, cu_seqlens_k, out)
    lib = load()
    num_seqs = cu_seqlens_q.numel() - 1
    H, D = q.shape[1], q.shape[2]
    s = _stream_handle(stream, q.device)
    if (causal or heads is not None) and workspace is not None:
        raise ValueError("the causal and head-range entry points use the library-owned workspace")
    with torch.cuda.device(q.device):
        if heads is not None:
            rc = lib.attn_varlen_fwd_heads(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                           cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
                                           num_seqs, H, int(heads[0]), int(heads[1]), D,
                                           1 if causal else 0, out.data_ptr(), s)
        elif causal:
            rc = lib.attn_varlen_fwd_causal(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                            cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
                                            num_seqs, H, D, out.data_ptr(), s)
        elif workspace is None:
            rc = lib.attn_varlen_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                     cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
                                     num_seqs, H, D, out.data_ptr(), s)
        else:
            rc = lib.attn_varlen_fwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                        cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
                                        num_seqs, H, D, out.data_ptr(), workspace.data_ptr(),
                                        workspace.numel() * workspace.element_size(), s)
    if rc != OK:
        raise AttnVarlenError(rc, "attn_varlen_fwd")
    return out


def check(stream=None, device=None, workspace=None, noalloc=False) -> int:
    """Synchronise and return (and clear) the device status; raises on error.

    ``workspace``: the caller-owned workspace to read; ``noalloc``: read the
    status of attn_varlen_fwd_noalloc's fixed scratch instead."""
    import torch
    dev = device if device is not None else torch.cuda.current_device()
    s = _stream_handle(stream, dev)
    with torch.cuda.device(dev):
        if noalloc:
            rc = load().attn_varlen_check_noalloc(s)
        elif workspace is None:
            rc = load().attn_varlen_check(s)
        else:
            rc = load().attn_varlen_check_ws(workspace.data_ptr(), s)
    if rc != OK:
        raise AttnVarlenError(rc, "attn_varlen_check")
    return rc


def attn_varlen_fwd_noalloc(q, k, v, cu_seqlens_q, cu_seqlens_k, out, stream=None):
    """attn_varlen_fwd through the entry point that allocates nothing.

    For callers that must not allocate device memory at call time; ``out``
    must be given.  Uses the library's fixed scratch (at most
    NOALLOC_MAX_SEQS sequences per call); calls on one device must not
    overlap on the GPU.
    """
    import torch
    _check_inputs(q, k, v, cu_seqlens_q, cu_seqlens_k, out)
    num_seqs = cu_seqlens_q.numel() - 1
    s = _stream_handle(stream, q.device)
    with torch.cuda.device(q.device):
        rc = load().attn_varlen_fwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                            cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
                                            num_seqs, q.shape[1], q.shape[2], out.data_ptr(), s)
    if rc != OK:
        raise AttnVarlenError(rc, "attn_varlen_fwd_noalloc")
    return out


def paged_attn_decode(query, k_cache, v_cache, block_tables, seq_lens, out=None, stream=None):
    """One decode step over a paged KV cache (include/paged_attn_decode.h).

    query [num_seqs, Hq, D]; k_cache [num_blocks, Hkv, D/8, 16, 8]; v_cache
    [num_blocks, Hkv, D, 16], all bf16 or all fp16 CUDA tensors;
    block_tables int32 [num_seqs, max_blocks]; seq_lens int32 [num_seqs].
    Returns ``out`` (allocated like ``query`` when not given).
    """
    import torch
    if out is None:
        out = torch.empty_like(query)
    if query.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("query must be bf16 or fp16")
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("out", out)):
        if t.dtype != query.dtype or not t.is_contiguous() or t.device != query.device:
            raise ValueError(f"{name} must be a contiguous {query.dtype} tensor on {query.device}")
    for name, t in (("block_tables", block_tables), ("seq_lens", seq_lens)):
        if t.dtype != torch.int32 or not t.is_contiguous() or t.device != query.device:
            raise ValueError(f"{name} must be a contiguous int32 tensor on {query.device}")
    if query.dim() != 3 or k_cache.dim() != 5 or v_cache.dim() != 4 or block_tables.dim() != 2:
        raise ValueError("query [S, Hq, D], k_cache [B, Hkv, D/8, bs, 8], v_cache [B, Hkv, D, bs], "
                         "block_tables [S, max_blocks]")
    num_seqs, hq, d = query.shape
    num_blocks, hkv, _, bs = v_cache.shape
    lib = load()
    s = _stream_handle(stream, query.device)
    with torch.cuda.device(query.device):
        rc = lib.paged_attn_decode(query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                   block_tables.data_ptr(), seq_lens.data_ptr(), num_seqs, hq,
                                   hkv, d, bs, block_tables.shape[1], num_blocks,
                                   1 if query.dtype == torch.float16 else 0, out.data_ptr(), s)
    if rc != OK:
        raise AttnVarlenError(rc, "paged_attn_decode")
    return out


def chunk_delta_rule_output(q, k, v, h, g, chunk_size=64, scale=None, out=None, stream=None):
    """Chunked gated delta-rule output (include/chunk_delta_rule.h).

    q, k bf16 [B, T, Hq, 128]; v bf16 [B, T, Hv, 128]; h bf16
    [B, ceil(T / 64), Hv, 128, 128]; g float32 [B, T, Hv]; all contiguous CUDA
    tensors on one device.  Returns ``out`` (bf16 [B, T, Hv, 128]).
    """
    import torch
    B, T, hq, kd = q.shape
    hv, vd = v.shape[2], v.shape[3]
    if out is None:
        out = torch.empty((B, T, hv, vd), dtype=torch.bfloat16, device=q.device)
    for name, t in (("q", q), ("k", k), ("v", v), ("h", h), ("out", out)):
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or t.device != q.device:
            raise ValueError(f"{name} must be a contiguous bf16 tensor on {q.device}")
    if g.dtype != torch.float32 or not g.is_contiguous() or g.device != q.device:
        raise ValueError(f"g must be a contiguous float32 tensor on {q.device}")
    if k.shape != q.shape or v.shape[:2] != (B, T) or g.shape != (B, T, hv) \
            or h.shape != (B, (T + chunk_size - 1) // chunk_size, hv, kd, vd):
        raise ValueError("shapes do not match")
    lib = load()
    s = _stream_handle(stream, q.device)
    with torch.cuda.device(q.device):
        rc = lib.chunk_delta_rule_output(q.data_ptr(), k.data_ptr(), v.data_ptr(), h.data_ptr(),
                                         g.data_ptr(), B, T, hq, hv, kd, vd, int(chunk_size),
                                         float(scale or 0.0), out.data_ptr(), s)
    if rc != OK:
        raise AttnVarlenError(rc, "chunk_delta_rule_output")
    return out


# ------------------------------------------- paged cache and drafted tokens
# The operators below take a few microseconds on the GPU, so their checks are
# written for the host's time: one comparison per property, devices as indexes.
# A call for another device or stream than the current ones runs again with
# those made current, so that what it allocates belongs to them.
def _torch():
    global _torch_module, _i32, _types, _raw_stream, _device, _take, _give
    import torch
    _i32, _types = torch.int32, (torch.bfloat16, torch.float16)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    # memory of the caching allocator, on the current device, without a tensor
    # around it (which costs the host 6 us more)
    _take = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None) or (
        lambda n, stream: torch.cuda.caching_allocator_alloc(n, None, stream))
    _give = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None) or \
        torch.cuda.caching_allocator_delete
    _torch_module = torch  # last: other threads take it for all of the above


_torch_module = _i32 = _types = _raw_stream = _device = _take = _give = None


def _ints(t, shape, dev, name):
    if t.dtype is not _i32 or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)} on CUDA device {dev}")


def _cache(k_cache, v_cache):
    """(num_blocks, num_kv_heads, head_size, block_size, device) of a pair of caches."""
    if _torch_module is None:
        _torch()
    shape = v_cache.shape
    if len(shape) != 4 or k_cache.dim() != 5:
        raise ValueError("k_cache [B, Hkv, D/8, bs, 8], v_cache [B, Hkv, D, bs]")
    nb, hkv, d, bs = shape
    if k_cache.shape != (nb, hkv, d // 8, bs, 8) or d % 8:
        raise ValueError(f"k_cache {list(k_cache.shape)} does not fit v_cache {list(shape)}")
    if k_cache.dtype not in _types or v_cache.dtype is not k_cache.dtype:
        raise ValueError("k_cache and v_cache must both be bf16 or both fp16")
    dev = k_cache.get_device()
    if dev < 0 or v_cache.get_device() != dev or not (k_cache.is_contiguous()
                                                      and v_cache.is_contiguous()):
        raise ValueError("k_cache and v_cache must be contiguous tensors on one CUDA device")
    return nb, hkv, d, bs, dev


def _table(block_tables, seq_lens, dev):
    """(rows, entries of a row) of a block table, its lengths checked."""
    shape = block_tables.shape
    if len(shape) != 2:
        raise ValueError("block_tables must be [S, max_blocks]")
    _ints(block_tables, shape, dev, "block_tables")
    _ints(seq_lens, shape[:1], dev, "seq_lens")
    return shape


def _elsewhere(dev, stream):
    """A context that makes the call's device and stream current; None if they are."""
    cuda = _torch_module.cuda
    if stream is None:
        return None if _device() == dev else cuda.device(dev)
    if stream.device.index != dev:
        raise ValueError(f"the stream belongs to CUDA device {stream.device.index}, the tensors "
                         f"to {dev}")
    return cuda.stream(stream)  # makes the stream's device current as well


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(name, *sizes):
    return getattr(load(), f"{name}_workspace_size")(*sizes)


def _done(rc, where):
    if rc != OK:
        raise AttnVarlenError(rc, where)


def paged_attn_cache_write(key, value, k_cache, v_cache, block_tables, seq_lens, cu_seqlens,
                           stream=None):
    """Write new tokens' keys and values into a paged cache (include/paged_attn_cache.h).

    key, value [total, Hkv, D] of the caches' type, packed by cu_seqlens int32
    [S + 1]; the head's elements contiguous, token and head strides multiples
    of 8 (views of a fused projection).  block_tables int32 [S, max_blocks];
    seq_lens int32 [S] counts the new tokens already: the last n of row i are
    the ones written.  The caches are changed in place.
    """
    nb, hkv, d, bs, dev = _cache(k_cache, v_cache)
    s, w = _table(block_tables, seq_lens, dev)
    _ints(cu_seqlens, (s + 1,), dev, "cu_seqlens")
    total = key.shape[0]
    for t in (key, value):
        if t.dtype is not k_cache.dtype or t.shape != (total, hkv, d) or t.get_device() != dev \
                or (t.stride(2) != 1 and total):
            raise ValueError(f"key and value must be {k_cache.dtype} [total, {hkv}, {d}] on CUDA "
                             f"device {dev} with contiguous head elements")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return paged_attn_cache_write(key, value, k_cache, v_cache, block_tables, seq_lens,
                                          cu_seqlens)
    kt, kh, _ = key.stride()
    vt, vh, _ = value.stride()
    if total == 1:  # the stride of a single token or head says nothing
        kt = vt = 0
    if hkv == 1:
        kh = vh = 0
    _done((_LIB or load()).paged_attn_cache_write(
        key.data_ptr(), value.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        block_tables.data_ptr(), seq_lens.data_ptr(), cu_seqlens.data_ptr(), s, total, hkv, d, bs,
        w, nb, kt, kh, vt, vh, _raw_stream(dev)), "paged_attn_cache_write")


def paged_attn_cache_accept(k_cache, v_cache, block_tables, seq_lens, cu_seqlens, accepted,
                            num_accepted, out=None, stream=None):
    """Move each row's accepted drafts up to the end of its context.

    The last n = cu_seqlens[i + 1] - cu_seqlens[i] tokens of row i are drafts;
    accepted int32 [S, A] lists the accepted ones in increasing order,
    num_accepted int32 [S] says how many.  Returns the rows' new lengths
    (int32 [S], not seq_lens itself).
    """
    nb, hkv, d, bs, dev = _cache(k_cache, v_cache)
    s, w = _table(block_tables, seq_lens, dev)
    if accepted.dim() != 2:
        raise ValueError("accepted must be [S, A]")
    a = accepted.shape[1]
    _ints(cu_seqlens, (s + 1,), dev, "cu_seqlens")
    _ints(accepted, (s, a), dev, "accepted")
    _ints(num_accepted, (s,), dev, "num_accepted")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return paged_attn_cache_accept(k_cache, v_cache, block_tables, seq_lens, cu_seqlens,
                                           accepted, num_accepted, out)
    lens = seq_lens.data_ptr()
    if out is None:
        out = _torch_module.empty_like(seq_lens)
    else:
        _ints(out, (s,), dev, "out")
        if s and out.data_ptr() in (lens, num_accepted.data_ptr()):
            raise ValueError("out must not be seq_lens or num_accepted")
    _done((_LIB or load()).paged_attn_cache_accept(
        k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), lens,
        cu_seqlens.data_ptr(), accepted.data_ptr(), num_accepted.data_ptr(), s, a, hkv, d, bs, w,
        nb, out.data_ptr(), _raw_stream(dev)), "paged_attn_cache_accept")
    return out


def paged_attn_cache_free(block_tables, seq_lens, refs, rows, block_size=16, stream=None):
    """Rows give their pages back: counts go down by one, seq_lens[rows] = 0.

    refs int32 [num_blocks] counts the rows that hold each page; rows int32
    [n].  seq_lens and refs are changed in place.
    """
    if _torch_module is None:
        _torch()
    dev = block_tables.get_device()
    if dev < 0 or rows.dim() != 1 or refs.dim() != 1:
        raise ValueError("block_tables [S, max_blocks], refs [num_blocks], rows [n] on a CUDA device")
    s, w = _table(block_tables, seq_lens, dev)
    _ints(refs, refs.shape, dev, "refs")
    _ints(rows, rows.shape, dev, "rows")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return paged_attn_cache_free(block_tables, seq_lens, refs, rows, block_size)
    _done((_LIB or load()).paged_attn_cache_free(
        block_tables.data_ptr(), seq_lens.data_ptr(), refs.data_ptr(), rows.data_ptr(),
        rows.shape[0], s, block_size, w, refs.shape[0], _raw_stream(dev)), "paged_attn_cache_free")


def paged_attn_cache_fork(k_cache, v_cache, block_tables, seq_lens, refs, src, dst, stream=None):
    """Rows dst become copies of rows src: whole pages shared, a partial last
    page copied into the lowest free page (beams, samples of one prompt).

    src, dst int32 [n]; every dst row is empty, no src and named once.
    The caches, block_tables, seq_lens and refs are changed in place.
    """
    nb, hkv, d, bs, dev = _cache(k_cache, v_cache)
    s, w = _table(block_tables, seq_lens, dev)
    if src.dim() != 1:
        raise ValueError("src and dst must be [n]")
    n = src.shape[0]
    _ints(refs, (nb,), dev, "refs")
    _ints(src, (n,), dev, "src")
    _ints(dst, (n,), dev, "dst")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return paged_attn_cache_fork(k_cache, v_cache, block_tables, seq_lens, refs, src, dst)
    lib = _LIB or load()
    size = _workspace_bytes("paged_attn_cache_fork", n, s)
    queue = _raw_stream(dev)
    ws = _take(size, queue)
    try:
        rc = lib.paged_attn_cache_fork(
            k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(),
            refs.data_ptr(), src.data_ptr(), dst.data_ptr(), n, s, hkv, d, bs, w, nb, ws, size,
            queue)
    finally:
        _give(ws)  # later calls on the stream may have it
    _done(rc, "paged_attn_cache_fork")


def paged_attn_cache_compact(k_cache, v_cache, block_tables, seq_lens, refs, out=None, stream=None):
    """Move the used pages (refs > 0) to the lowest ids.

    Returns (block_tables, refs) after the move; ``out``: the pair to write,
    which may be the inputs themselves (in place).  The caches are changed in
    place; seq_lens says how many entries of a row are live.
    """
    nb, hkv, d, bs, dev = _cache(k_cache, v_cache)
    s, w = _table(block_tables, seq_lens, dev)
    _ints(refs, (nb,), dev, "refs")
    if s == 0:
        raise ValueError("block_tables has no row")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return paged_attn_cache_compact(k_cache, v_cache, block_tables, seq_lens, refs, out)
    if out is None:
        tables_out, refs_out = _torch_module.empty_like(block_tables), _torch_module.empty_like(refs)
    else:
        tables_out, refs_out = out
        _ints(tables_out, (s, w), dev, "out block_tables")
        _ints(refs_out, (nb,), dev, "out refs")
    lib = _LIB or load()
    size = _workspace_bytes("paged_attn_cache_compact", nb)
    queue = _raw_stream(dev)
    ws = _take(size, queue)
    try:
        rc = lib.paged_attn_cache_compact(
            k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(),
            refs.data_ptr(), s, hkv, d, bs, w, nb, tables_out.data_ptr(), refs_out.data_ptr(), ws,
            size, queue)
    finally:
        _give(ws)  # later calls on the stream may have it
    _done(rc, "paged_attn_cache_compact")
    return tables_out, refs_out


def paged_attn_tree(query, k_cache, v_cache, block_tables, seq_lens, cu_seqlens, parents=None,
                    scale=None, out=None, stream=None):
    """Attention of drafted tokens over a paged cache (include/paged_attn_tree.h).

    query [total, Hq, D] of the caches' type, packed by cu_seqlens int32
    [S + 1]: the last n tokens of row i, whose keys and values the cache holds
    already (seq_lens counts them).  parents int32 [total]: the draft each
    draft hangs on, an index within its row's drafts below its own, -1 for the
    context; None for chains.  A draft sees the context, its ancestors and
    itself.  scale: default D^-1/2.  Returns ``out`` (allocated like ``query``
    when not given; rows that no sequence covers are left untouched).
    """
    nb, hkv, d, bs, dev = _cache(k_cache, v_cache)
    s, w = _table(block_tables, seq_lens, dev)
    _ints(cu_seqlens, (s + 1,), dev, "cu_seqlens")
    shape = query.shape
    dtype = k_cache.dtype
    for t in (query,) if out is None else (query, out):
        if t.dtype is not dtype or t.shape != shape or len(shape) != 3 or shape[2] != d \
                or t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"query and out must be contiguous {dtype} tensors [total, Hq, {d}] on "
                             f"CUDA device {dev}")
    total, hq, _ = shape
    if out is not None:
        apart = out.data_ptr() - query.data_ptr()
        if total and abs(apart) < total * hq * d * 2:
            raise ValueError("out must not overlap query")
    if parents is not None:
        _ints(parents, (total,), dev, "parents")
    if scale is None:
        scale = 0.0
    elif not 2.0 ** -126 <= scale <= 2.0 ** 126:  # the library takes it in 32 bits
        raise ValueError("scale must be from 2^-126 to 2^126")
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return paged_attn_tree(query, k_cache, v_cache, block_tables, seq_lens, cu_seqlens,
                                   parents, scale or None, out)
    lib = _LIB or load()
    size = _workspace_bytes("paged_attn_tree", d)
    if out is None:
        out = _torch_module.empty_like(query)
    queue = _raw_stream(dev)
    ws = _take(size, queue)
    try:
        rc = lib.paged_attn_tree(
            query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
            seq_lens.data_ptr(), cu_seqlens.data_ptr(),
            None if parents is None else parents.data_ptr(), s, total, hq, hkv, d, bs, w, nb, scale,
            1 if dtype is _types[1] else 0, out.data_ptr(), ws, size, queue)
    finally:
        _give(ws)  # later calls on the stream may have it
    _done(rc, "paged_attn_tree")
    return out
