"""A paged KV cache held in 8 bits: appends that quantise, reading back, and attention over it.  The entry
points of include/attn_kv8.h, and their torch-tensor helpers.

Argument marshalling only, as in the package itself, which re-exports every name here:
  * ``attn_paged_append_fp8``, ``attn_paged_read_fp8``, ``attn_paged_fwd_fp8`` and its
    ``*_workspace_size`` query: the C entry points with raw pointers and a stream handle;
  * ``paged_append_fp8``, ``paged_read_fp8``, ``paged_fwd_fp8``: torch tensors.  A cache is codes,
    float8_e4m3fn [num_pages, page_size, H_kv, d], and scales, fp32 [num_pages, H_kv, page_size / block]:
    their shapes say how many rows share a scale.
"""
import ctypes
import functools
import math

import torch

from . import ATTN_ERR_UNSUPPORTED, AttnError, _raise, lib
from .kv import _check, _dense_heads, _device, _dims, _freqs, _handle, _on, _size


def _declare(L):
    """Result and argument types of this header's functions (called once, when the library loads)."""
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    for name, res, args in (
            ("attn_paged_append_fp8", i, [vp] * 11 + [i] * 9 + [vp, i, f, vp]),
            ("attn_paged_read_fp8", i, [vp] * 6 + [i] * 8 + [vp, vp, i, vp]),
            ("attn_paged_fwd_fp8_workspace_size", sz, [i] * 8),
            ("attn_paged_fwd_fp8", i, [vp] * 8 + [i] * 10 + [f, i] + [vp] * 3 + [sz, vp])):
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args


# ---------------------------------------------------------------- C entry points

def attn_paged_append_fp8(q, q_out, k, v, k_cache, v_cache, k_scale, v_scale, slots, positions, inv_freq, freq_bits, T,
                          H, H_kv, d, rot, page_size, block, num_pages, strides, interleaved, amplitude, stream):
    """strides is a C array of 8 long long."""
    return lib().attn_paged_append_fp8(q, q_out, k, v, k_cache, v_cache, k_scale, v_scale, slots, positions, inv_freq,
                                       freq_bits, T, H, H_kv, d, rot, page_size, block, num_pages, strides, interleaved,
                                       amplitude, stream)


def attn_paged_read_fp8(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens_k, B, total_k, H_kv, d, page_size,
                        block, max_pages, num_pages, k, v, elem_bytes, stream):
    return lib().attn_paged_read_fp8(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens_k, B, total_k, H_kv, d,
                                     page_size, block, max_pages, num_pages, k, v, elem_bytes, stream)


def attn_paged_fwd_fp8_workspace_size(B, total_q, max_q_len, H, H_kv, d, page_size, max_pages):
    return lib().attn_paged_fwd_fp8_workspace_size(B, total_q, max_q_len, H, H_kv, d, page_size, max_pages)


def attn_paged_fwd_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens_q, seq_lens, B, total_q, max_q_len,
                       H, H_kv, d, page_size, block, max_pages, num_pages, scale, causal, o, lse, workspace,
                       workspace_bytes, stream):
    return lib().attn_paged_fwd_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens_q, seq_lens, B,
                                    total_q, max_q_len, H, H_kv, d, page_size, block, max_pages, num_pages, scale, causal,
                                    o, lse, workspace, workspace_bytes, stream)


# ---------------------------------------------------------------- torch helpers

_Strides = ctypes.c_longlong * 8
_bf16, _f8, _f32, _i32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.int32

# Decode steps ask for the same few sizes again and again, and the answer is a function of them.
_workspace_bytes = functools.lru_cache(maxsize=1024)(attn_paged_fwd_fp8_workspace_size)


def _cache(k_cache, v_cache, k_scale, v_scale, dev):
    """Checked addresses of a cache's codes and scales, and (num_pages, page_size, block, H_kv, d)."""
    _dims(k_cache, "k_cache", 4)
    _dims(k_scale, "k_scale", 3)
    shape, (num_pages, page_size, H_kv, d) = k_cache.shape, k_cache.shape
    per_page = k_scale.shape[2]
    if per_page < 1 or page_size % per_page:
        raise ValueError("k_scale has %d scales for the %d rows of a page" % (per_page, page_size))
    scales = (num_pages, H_kv, per_page)
    return ((_check(k_cache, "k_cache", _f8, dev, shape), _check(v_cache, "v_cache", _f8, dev, shape),
             _check(k_scale, "k_scale", _f32, dev, scales), _check(v_scale, "v_scale", _f32, dev, scales)),
            (num_pages, page_size, page_size // per_page, H_kv, d))


def _rows(t, name, dev, shape):
    """Address of bf16 rows of heads of this shape, and their strides: of tokens, of heads, the head dim dense."""
    try:
        if t.dtype is _bf16 and t.get_device() == dev and t.shape == shape:
            token, head, dim = t.stride()
            if dim == 1:
                return t.data_ptr(), token, head
    except AttributeError:
        pass
    return (_check(t, name, _bf16, dev, shape, dense=False),) + _dense_heads(t, name)


def paged_append_fp8(q, k, v, k_cache, v_cache, k_scale, v_scale, slots, positions=None, inv_freq=None,
                     interleaved=False, amplitude=1.0, q_out=None, stream=None):
    """Rotates q and k and writes k and v to their cache slots as e4m3 codes, updating the scales of the blocks
    they enter (see attn_paged_append_fp8: rows of a block are filled in order, and its scale is a power of two that
    grows with them).

    q bf16 [T, H, d] (or None), k, v bf16 [T, H_kv, d], any strides with a dense head dim; slots int32 [T],
    negative: the token is skipped, its row of q_out left as it was.  positions int32 [T] and inv_freq as for
    ``rope``; both None: nothing rotates.  q_out may be q.  Returns q_out."""
    dev = _device(k, "k")
    _dims(k, "k", 3)
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    cache, (num_pages, page_size, block, H_kv, d) = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    T = _size(k.shape[0], "the number of tokens")
    H = 0
    qp = qop = None
    qt = qh = qot = qoh = 0
    if q is not None:
        _dims(q, "q", 3)
        H = q.shape[1]
        if q_out is None:
            with _on(stream):
                q_out = torch.empty((T, H, d), dtype=_bf16, device=q.device)
        qp, qt, qh = _rows(q, "q", dev, (T, H, d))
        qop, qot, qoh = _rows(q_out, "q_out", dev, (T, H, d))
    elif q_out is not None:
        raise ValueError("q_out without q")
    kp, kt, kh = _rows(k, "k", dev, (T, H_kv, d))
    vp, vt, vh = _rows(v, "v", dev, (T, H_kv, d))
    fp, bits, rot, pp = None, 64, 0, None
    if inv_freq is not None:
        fp, bits, rot = _freqs(inv_freq, dev)
        pp = _check(positions, "positions", torch.int32, dev, (T,))
    st = lib().attn_paged_append_fp8(qp, qop, kp, vp, *cache, _check(slots, "slots", torch.int32, dev, (T,)), pp, fp, bits,
                                     T, H, H_kv, d, rot, page_size, block, num_pages,
                                     _Strides(qt, qh, qot, qoh, kt, kh, vt, vh), int(bool(interleaved)),
                                     float(amplitude), _handle(stream, dev))
    _raise(st, "attn_paged_append_fp8")
    return q_out


def paged_read_fp8(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens_k, total_k, dtype=torch.bfloat16,
                   k_out=None, v_out=None, stream=None):
    """The first cu_seqlens_k[r + 1] - cu_seqlens_k[r] keys and values of each request r, packed: what ``varlen_fwd``
    takes.  block_table int32 [B, max_pages]; cu_seqlens_k int32 [B + 1]; ``total_k`` rows, those from cu_seqlens_k[B]
    on left as they were.  dtype bfloat16 or float32, or that of the outputs
    given.  Returns (k, v) [total_k, H_kv, d]."""
    dev = _device(k_cache, "k_cache")
    cache, (num_pages, page_size, block, H_kv, d) = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    _dims(block_table, "block_table", 2)
    B, max_pages = (_size(n, "a size of block_table") for n in block_table.shape)
    total_k = _size(total_k, "total_k")
    given = k_out if k_out is not None else v_out
    if given is not None:
        _device(given, "k_out" if k_out is not None else "v_out")
        dtype = given.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError("dtype must be bfloat16 or float32, got %s" % dtype)
    if total_k < 1:
        raise ValueError("total_k must be at least 1")
    shape = (total_k, H_kv, d)
    with _on(stream):
        if k_out is None:
            k_out = torch.empty(shape, dtype=dtype, device=k_cache.device)
        if v_out is None:
            v_out = torch.empty(shape, dtype=dtype, device=k_cache.device)
    st = lib().attn_paged_read_fp8(*cache, _check(block_table, "block_table", torch.int32, dev, (B, max_pages)),
                                   _check(cu_seqlens_k, "cu_seqlens_k", torch.int32, dev, (B + 1,)), B, total_k, H_kv, d,
                                   page_size, block, max_pages, num_pages, _check(k_out, "k_out", dtype, dev, shape),
                                   _check(v_out, "v_out", dtype, dev, shape), dtype.itemsize, _handle(stream, dev))
    _raise(st, "attn_paged_read_fp8")
    return k_out, v_out


def paged_fwd_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens_q=None, max_q_len=None,
                  causal=False, scale=None, out=None, lse=None, workspace=None, return_lse=True, stream=None):
    """``paged_fwd`` over a cache of codes: grouped-query attention for decode steps and a few tokens per request.

    q bf16 [total_q, H, d] token-major; block_table int32 [B, max_pages]; seq_lens int32 [B]; cu_seqlens_q int32
    [B + 1] (None: one query token per request).  max_q_len is the largest per-request token count (read from
    cu_seqlens_q, with a device-to-host copy, when not given).  Returns (o bf16 like q, lse fp32 [total_q, H])."""
    dev = _device(q, "q")
    _dims(q, "q", 3)
    _dims(block_table, "block_table", 2)
    T, H, d = q.shape
    cache, (num_pages, page_size, block, H_kv, cd) = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    if cd != d:
        raise ValueError("q has head dim %d, the cache %d" % (d, cd))
    B, max_pages = (_size(n, "a size of block_table") for n in block_table.shape)
    i32 = _i32
    cp = None
    if cu_seqlens_q is not None:
        cp = _check(cu_seqlens_q, "cu_seqlens_q", i32, dev, (B + 1,))
        if max_q_len is None:
            with _on(stream):  # what writes the offsets may be under way there
                max_q_len = int((cu_seqlens_q[1:] - cu_seqlens_q[:-1]).max().item()) if B else 0
    elif max_q_len is None:
        max_q_len = 1
    max_q_len = _size(max_q_len, "max_q_len")
    with _on(stream):
        if out is None:
            out = torch.empty((T, H, d), dtype=torch.bfloat16, device=q.device)
        if lse is None and return_lse:
            lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
        if workspace is None:
            need = _workspace_bytes(B, T, max_q_len, H, H_kv, d, page_size, max_pages)
            if need == 0:
                raise AttnError(ATTN_ERR_UNSUPPORTED, "attn_paged_fwd_fp8_workspace_size")
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:
            need = workspace.numel()
            _check(workspace, "workspace", torch.uint8, dev, (need,))
    st = lib().attn_paged_fwd_fp8(_check(q, "q", torch.bfloat16, dev, (T, H, d)), *cache,
                                  _check(block_table, "block_table", i32, dev, (B, max_pages)), cp,
                                  _check(seq_lens, "seq_lens", i32, dev, (B,)), B, T, max_q_len, H, H_kv, d, page_size,
                                  block, max_pages, num_pages, float(scale) if scale is not None else 1.0 / math.sqrt(d),
                                  int(bool(causal)), _check(out, "out", torch.bfloat16, dev, (T, H, d)),
                                  None if lse is None else _check(lse, "lse", torch.float32, dev, (T, H)),
                                  workspace.data_ptr(), need, _handle(stream, dev))
    _raise(st, "attn_paged_fwd_fp8")
    return out, lse
