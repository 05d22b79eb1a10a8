"""Rotary positions, page plans, cache appends, page sketches and page-sparse attention: the entry
points of include/attn_kv.h, and their torch-tensor helpers.

Argument marshalling only, as in the package itself, which re-exports every name here:
  * ``attn_rope_inv_freq``, ``attn_rope``, ``attn_paged_plan``, ``attn_paged_append``,
    ``attn_page_sketch``, ``attn_page_select``, ``attn_paged_sparse_fwd`` and the
    ``*_workspace_size`` queries: the C entry points with raw pointers and a stream handle;
  * ``rope_inv_freq``, ``rope``, ``paged_plan``, ``paged_append``, ``page_sketch``,
    ``page_select``, ``paged_sparse_fwd``: torch tensors.  All tensors of a call are on the
    current CUDA device; outputs and workspaces that are not given are allocated on the stream
    that the call runs on (``stream``, or the current one).
"""
import contextlib
import ctypes
import math

import torch

from . import ATTN_ERR_INVALID_ARG, ATTN_ERR_WORKSPACE, AttnError, _raise, lib

ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}


def _declare(L):
    """Result and argument types of this header's functions (called once, when the library loads)."""
    vp, i, f, sz, ll, db = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong,
                            ctypes.c_double)
    for name, res, args in (
            ("attn_rope_inv_freq", i, [vp, vp, i, db, i, db, i, db, db]),
            ("attn_rope", i, [vp] * 5 + [ll, vp] + [i] * 8 + [vp, i, i, f, vp]),
            ("attn_paged_plan", i, [vp] * 5 + [i] * 6 + [vp] * 6),
            ("attn_paged_append", i, [vp] * 9 + [i] * 8 + [vp, i, f, vp]),
            ("attn_page_sketch", i, [vp] * 4 + [i] * 7 + [vp] * 3),
            ("attn_page_select_workspace_size", sz, [i] * 4),
            ("attn_page_select", i, [vp] * 6 + [i] * 11 + [vp] * 3 + [sz, vp]),
            ("attn_paged_sparse_fwd_workspace_size", sz, [i] * 7),
            ("attn_paged_sparse_fwd", i, [vp] * 8 + [i] * 11 + [f] + [vp] * 5 + [sz, vp])):
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args


# ---------------------------------------------------------------- C entry points

def attn_rope_inv_freq(inv_freq, amplitude, rot, base, scaling, factor, orig_len, low, high):
    return lib().attn_rope_inv_freq(inv_freq, amplitude, rot, base, scaling, factor, orig_len, low, high)


def attn_rope(q, q_out, k, k_out, positions, pos_stride_b, inv_freq, freq_bits, elem_bytes, B, H, H_k, N, d, rot,
              strides, interleaved, inverse, amplitude, stream):
    """strides is a C array of 12 long long."""
    return lib().attn_rope(q, q_out, k, k_out, positions, pos_stride_b, inv_freq, freq_bits, elem_bytes, B, H, H_k, N,
                           d, rot, strides, interleaved, inverse, amplitude, stream)


def attn_paged_plan(ctx_lens, new_lens, block_table, free_pages, free_count, B, total_q, page_size, max_pages,
                    num_pages, n_free, cu_seqlens_q, seq_lens, positions, slots, free_left, stream):
    return lib().attn_paged_plan(ctx_lens, new_lens, block_table, free_pages, free_count, B, total_q, page_size,
                                 max_pages, num_pages, n_free, cu_seqlens_q, seq_lens, positions, slots, free_left,
                                 stream)


def attn_paged_append(q, q_out, k, v, k_cache, v_cache, slots, positions, inv_freq, freq_bits, T, H, H_kv, d, rot,
                      page_size, num_pages, strides, interleaved, amplitude, stream):
    """strides is a C array of 8 long long."""
    return lib().attn_paged_append(q, q_out, k, v, k_cache, v_cache, slots, positions, inv_freq, freq_bits, T, H, H_kv,
                                   d, rot, page_size, num_pages, strides, interleaved, amplitude, stream)


def attn_page_sketch(k_cache, block_table, cu_seqlens_q, seq_lens, B, max_q_len, H_kv, d, page_size, max_pages,
                     num_pages, sketch, amp, stream):
    return lib().attn_page_sketch(k_cache, block_table, cu_seqlens_q, seq_lens, B, max_q_len, H_kv, d, page_size,
                                  max_pages, num_pages, sketch, amp, stream)


def attn_page_select_workspace_size(total_q, H_kv, max_pages, budget):
    return lib().attn_page_select_workspace_size(total_q, H_kv, max_pages, budget)


def attn_page_select(q, sketch, amp, block_table, cu_seqlens_q, seq_lens, B, total_q, H, H_kv, d, page_size, max_pages,
                     num_pages, budget, first, last, tables, sel_lens, workspace, workspace_bytes, stream):
    return lib().attn_page_select(q, sketch, amp, block_table, cu_seqlens_q, seq_lens, B, total_q, H, H_kv, d,
                                  page_size, max_pages, num_pages, budget, first, last, tables, sel_lens, workspace,
                                  workspace_bytes, stream)


def attn_paged_sparse_fwd_workspace_size(total_q, H, H_kv, d, page_size, max_pages, budget):
    return lib().attn_paged_sparse_fwd_workspace_size(total_q, H, H_kv, d, page_size, max_pages, budget)


def attn_paged_sparse_fwd(q, k_cache, v_cache, block_table, cu_seqlens_q, seq_lens, sketch, amp, B, total_q, H, H_kv,
                          d, page_size, max_pages, num_pages, budget, first, last, scale, o, lse, tables, sel_lens,
                          workspace, workspace_bytes, stream):
    return lib().attn_paged_sparse_fwd(q, k_cache, v_cache, block_table, cu_seqlens_q, seq_lens, sketch, amp, B,
                                       total_q, H, H_kv, d, page_size, max_pages, num_pages, budget, first, last,
                                       scale, o, lse, tables, sel_lens, workspace, workspace_bytes, stream)


# ---------------------------------------------------------------- torch helpers

# The helpers below run once per call of a decode step, whose kernels take a few microseconds: they
# look up each attribute once and take the slow path only to say what is wrong.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _dims(t, name, n):
    """Refuses what is not a tensor of n dims (its dtype, device and shape are checked with the others')."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dim() != n:
        raise ValueError("%s must have %d dims" % (name, n))


def _size(x, name):
    """x as a C int, which would take its low 32 bits without a word."""
    x = int(x)
    if not -0x80000000 <= x <= 0x7fffffff:
        raise ValueError("%s = %d does not fit 32 bits" % (name, x))
    return x


def _device(t, name):
    """Index of the current CUDA device, which t has to be on."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError("%s is on cuda:%d, the current device is cuda:%d" % (name, dev, torch.cuda.current_device()))
    return dev


def _check(t, name, dtype, dev, shape, dense=True):
    """Address of t, a tensor of this dtype, device and shape."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape and (not dense or t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s is on cuda:%d, the call runs on cuda:%d" % (name, t.get_device(), dev))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be contiguous" % name)


def _handle(stream, dev):
    if stream is None:
        return _raw_stream(dev)
    if stream.device.index != dev:
        raise ValueError("stream is on %s, the tensors are on cuda:%d" % (stream.device, dev))
    return stream.cuda_stream


_no_context = contextlib.nullcontext()


def _on(stream):
    """Allocations inside belong to the call's stream."""
    return _no_context if stream is None else torch.cuda.stream(stream)


def _freqs(inv_freq, dev):
    """(address, bits, rotated dims) of the frequencies."""
    _dims(inv_freq, "inv_freq", 1)
    if inv_freq.dtype not in (torch.float64, torch.float32):
        raise TypeError("inv_freq must be float64 or float32, got %s" % inv_freq.dtype)
    return (_check(inv_freq, "inv_freq", inv_freq.dtype, dev, (inv_freq.numel(),)),
            64 if inv_freq.dtype is torch.float64 else 32, 2 * inv_freq.numel())


def _dense_heads(t, name):
    """Strides of all dims but the last, which has to be dense."""
    s = t.stride()
    if s[-1] != 1:
        raise ValueError("the head dim of %s must be dense" % name)
    return s[:-1]


def rope_inv_freq(rot, base=10000.0, scaling="none", factor=1.0, orig_len=8192, low=1.0, high=None):
    """Angle per position of each of the rot / 2 rotated pairs, a float64 CPU tensor, and the amplitude
    that goes with them (see attn_rope_scaling_t; ``low`` and ``high`` are turns over ``orig_len``: 1 and, where
    ``high`` is None, the end that each kind was published with, 4 for bands and 32 for yarn)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be one of %s" % ", ".join(ROPE_SCALINGS))
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    rot, orig_len = _size(rot, "rot"), _size(orig_len, "orig_len")
    out = torch.empty(max(rot, 0) // 2, dtype=torch.float64)
    amplitude = ctypes.c_double()
    st = attn_rope_inv_freq(out.data_ptr(), ctypes.addressof(amplitude), rot, float(base), ROPE_SCALINGS[scaling],
                            float(factor), orig_len, float(low), float(high))
    _raise(st, "attn_rope_inv_freq")
    return out, amplitude.value


def rope(q, k=None, *, inv_freq, positions=None, interleaved=False, inverse=False, amplitude=1.0, q_out=None,
         k_out=None, stream=None):
    """Rotary positions on q [B, H, N, d] (or token-major [T, H, d]) and, in the same launch, k with its own
    head count; bf16 or fp32, any strides with a dense head dim.  inv_freq: float64 or float32 [rot / 2].
    positions: int32 [N], or [B, N] ([T] token-major); None: 0, 1, ...  ``inverse``: the transpose, that is
    the gradient.  q_out, k_out may be q, k (in place).  Returns (q_out, k_out)."""
    dev = _device(q, "q")
    dt = q.dtype
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise TypeError("q must be bfloat16 or float32, got %s" % dt)
    if q.dim() == 4:
        B, H, N, d = q.shape
    elif q.dim() == 3:
        (N, H, d), B = q.shape, 1
    else:
        raise ValueError("q must have 3 or 4 dims")
    shape = q.shape
    H_k = 0
    if k is not None:
        _dims(k, "k", q.dim())
        H_k = k.shape[1]
    elif k_out is not None:
        raise ValueError("k_out without k")
    with _on(stream):
        if q_out is None:
            q_out = torch.empty(shape, dtype=dt, device=q.device)
        if k is not None and k_out is None:
            k_out = torch.empty(k.shape, dtype=dt, device=q.device)

    def strides(t, name, n_heads):
        ptr = _check(t, name, dt, dev, (B, n_heads, N, d) if len(shape) == 4 else (N, n_heads, d), dense=False)
        s = _dense_heads(t, name)
        return ptr, s if len(s) == 3 else (0, s[1], s[0])

    qp, qs = strides(q, "q", H)
    qop, qos = strides(q_out, "q_out", H)
    kp = kop = None
    ks = kos = (0, 0, 0)
    if k is not None:
        kp, ks = strides(k, "k", H_k)
        kop, kos = strides(k_out, "k_out", H_k)
    fp, bits, rot = _freqs(inv_freq, dev)
    pp, pb = None, 0
    if positions is not None:
        if not isinstance(positions, torch.Tensor):
            raise TypeError("positions must be a CUDA tensor")
        if positions.dim() == 2 and len(shape) == 4:
            pp, pb = _check(positions, "positions", torch.int32, dev, (B, N)), N
        else:
            pp = _check(positions, "positions", torch.int32, dev, (N,))
    st = lib().attn_rope(qp, qop, kp, kop, pp, pb, fp, bits, dt.itemsize, B, H, H_k, N, d, rot,
                   (ctypes.c_longlong * 12)(*qs, *qos, *ks, *kos), int(bool(interleaved)),
                   int(bool(inverse)), float(amplitude), _handle(stream, dev))
    _raise(st, "attn_rope")
    return q_out, k_out


def paged_plan(ctx_lens, block_table, free_pages, free_count, page_size, num_pages, total_q, new_lens=None,
               cu_seqlens_q=None, seq_lens=None, positions=None, slots=None, free_left=None, stream=None):
    """Offsets, positions and cache slots of a step's new tokens, all int32 on the GPU.

    ctx_lens [B] cached keys, new_lens [B] new tokens (None: one each), total_q the rows of the token
    buffer (tokens behind the last get position 0 and slot -1).  block_table [B, max_pages] is updated
    in place with pages from the top of free_pages [n] of which the first free_count [1] are free.
    seq_lens may be ctx_lens and free_left may be free_count.
    Returns (cu_seqlens_q [B + 1], seq_lens [B], positions [total_q], slots [total_q], free_left [1])."""
    dev = _device(ctx_lens, "ctx_lens")
    i32, total_q = torch.int32, _size(total_q, "total_q")
    _dims(ctx_lens, "ctx_lens", 1)
    _dims(block_table, "block_table", 2)
    _dims(free_pages, "free_pages", 1)
    if total_q < 1:
        raise ValueError("total_q must be at least 1")
    B, max_pages = ctx_lens.shape[0], block_table.shape[1]
    sizes = (B + 1, B, total_q, total_q, 1)
    given = [cu_seqlens_q, seq_lens, positions, slots, free_left]
    with _on(stream):
        for i in range(5):
            if given[i] is None:
                given[i] = torch.empty(sizes[i], dtype=i32, device=ctx_lens.device)
    names = ("cu_seqlens_q", "seq_lens", "positions", "slots", "free_left")
    outs = [_check(t, name, i32, dev, (n,)) for t, name, n in zip(given, names, sizes)]
    st = lib().attn_paged_plan(_check(ctx_lens, "ctx_lens", i32, dev, (B,)),
                         None if new_lens is None else _check(new_lens, "new_lens", i32, dev, (B,)),
                         _check(block_table, "block_table", i32, dev, (B, max_pages)),
                         _check(free_pages, "free_pages", i32, dev, (free_pages.shape[0],)),
                         _check(free_count, "free_count", i32, dev, (1,)), B, total_q, _size(page_size, "page_size"), max_pages,
                         _size(num_pages, "num_pages"), free_pages.shape[0], *outs, _handle(stream, dev))
    _raise(st, "attn_paged_plan")
    return tuple(given)


def paged_append(q, k, v, k_cache, v_cache, slots, positions=None, inv_freq=None, interleaved=False, amplitude=1.0,
                 q_out=None, stream=None):
    """Rotates q and k and writes k and v to their cache slots, in one pass.

    q bf16 [T, H, d] (or None), k, v bf16 [T, H_kv, d], any strides with a dense head dim (views of a
    fused projection); caches bf16 [num_pages, page_size, H_kv, d]; slots int32 [T], negative: the token
    is skipped, its row of q_out left as it was.  positions int32 [T] and inv_freq as for ``rope``; both
    None: nothing rotates.  q_out may be q.  Returns q_out."""
    dev = _device(k, "k")
    bf = torch.bfloat16
    _dims(k, "k", 3)
    _dims(k_cache, "k_cache", 4)
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    T, H_kv, d = _size(k.shape[0], "the number of tokens"), k.shape[1], k.shape[2]
    num_pages, page_size = k_cache.shape[0], k_cache.shape[1]
    H = 0
    qp = qop = None
    qs = qos = (0, 0)
    if q is not None:
        _dims(q, "q", 3)
        H = q.shape[1]
        if q_out is None:
            with _on(stream):
                q_out = torch.empty((T, H, d), dtype=bf, device=q.device)
        qp, qs = _check(q, "q", bf, dev, (T, H, d), dense=False), _dense_heads(q, "q")
        qop, qos = _check(q_out, "q_out", bf, dev, (T, H, d), dense=False), _dense_heads(q_out, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    kp, ks = _check(k, "k", bf, dev, (T, H_kv, d), dense=False), _dense_heads(k, "k")
    vp, vs = _check(v, "v", bf, dev, (T, H_kv, d), dense=False), _dense_heads(v, "v")
    cache = (num_pages, page_size, H_kv, d)
    fp, bits, rot, pp = None, 64, 0, None
    if inv_freq is not None:
        fp, bits, rot = _freqs(inv_freq, dev)
        pp = _check(positions, "positions", torch.int32, dev, (T,))
    st = lib().attn_paged_append(qp, qop, kp, vp, _check(k_cache, "k_cache", bf, dev, cache),
                           _check(v_cache, "v_cache", bf, dev, cache), _check(slots, "slots", torch.int32, dev, (T,)),
                           pp, fp, bits, T, H, H_kv, d, rot, page_size, num_pages,
                           (ctypes.c_longlong * 8)(*qs, *qos, *ks, *vs), int(bool(interleaved)),
                           float(amplitude), _handle(stream, dev))
    _raise(st, "attn_paged_append")
    return q_out


def page_sketch(k_cache, block_table, seq_lens, sketch, amp, cu_seqlens_q=None, max_q_len=1, stream=None):
    """Renews, in place, the sketches of the pages that hold each request's newest keys: its last
    ``max_q_len`` ones, or with cu_seqlens_q int32 [B + 1] as many as it has new tokens (at most
    ``max_q_len``).  k_cache bf16 [num_pages, page_size, H_kv, d]; block_table int32 [B, max_pages];
    seq_lens int32 [B]; sketch int8 [num_pages, H_kv, 2 d]; amp fp32 [num_pages, H_kv]."""
    dev = _device(k_cache, "k_cache")
    _dims(k_cache, "k_cache", 4)
    _dims(block_table, "block_table", 2)
    num_pages, page_size, H_kv, d = k_cache.shape
    B, max_pages = block_table.shape
    i32 = torch.int32
    st = lib().attn_page_sketch(_check(k_cache, "k_cache", torch.bfloat16, dev, k_cache.shape),
                          _check(block_table, "block_table", i32, dev, (B, max_pages)),
                          None if cu_seqlens_q is None else _check(cu_seqlens_q, "cu_seqlens_q", i32, dev, (B + 1,)),
                          _check(seq_lens, "seq_lens", i32, dev, (B,)), B, _size(max_q_len, "max_q_len"), H_kv, d, page_size,
                          max_pages, num_pages, _check(sketch, "sketch", torch.int8, dev, (num_pages, H_kv, 2 * d)),
                          _check(amp, "amp", torch.float32, dev, (num_pages, H_kv)), _handle(stream, dev))
    _raise(st, "attn_page_sketch")
    return sketch, amp


def _selection_args(q, sketch, amp, block_table, seq_lens, cu_seqlens_q, dev):
    """Checked pointers and sizes that selection and sparse attention share."""
    _dims(q, "q", 3)
    _dims(block_table, "block_table", 2)
    _dims(sketch, "sketch", 3)
    T, H, d = q.shape
    B, max_pages = block_table.shape
    num_pages, H_kv = sketch.shape[0], sketch.shape[1]
    i32 = torch.int32
    ptrs = (_check(q, "q", torch.bfloat16, dev, (T, H, d)),
            _check(sketch, "sketch", torch.int8, dev, (num_pages, H_kv, 2 * d)),
            _check(amp, "amp", torch.float32, dev, (num_pages, H_kv)),
            _check(block_table, "block_table", i32, dev, (B, max_pages)),
            None if cu_seqlens_q is None else _check(cu_seqlens_q, "cu_seqlens_q", i32, dev, (B + 1,)),
            _check(seq_lens, "seq_lens", i32, dev, (B,)))
    return ptrs, (B, T, H, H_kv, d), max_pages, num_pages


def _with_workspace(call, size, workspace, dev, stream, device, what):
    """Runs call(address, bytes) with the workspace given, else with none, and where that is refused with one of
    size() bytes: most calls need none, and asking for the size first would cost each of them."""
    if workspace is not None:
        st = call(_check(workspace, "workspace", torch.uint8, dev, (workspace.numel(),)), workspace.numel())
    else:
        st = call(None, 0)
        if st == ATTN_ERR_WORKSPACE:
            with _on(stream):
                workspace = torch.empty(size(), dtype=torch.uint8, device=device)
            st = call(workspace.data_ptr(), workspace.numel())
    _raise(st, what)


def page_select(q, sketch, amp, block_table, seq_lens, page_size, budget, first=1, last=1, cu_seqlens_q=None,
                tables=None, sel_lens=None, workspace=None, stream=None):
    """The pages each query token attends to: per KV head the ``first`` and ``last`` ones it sees and the
    best-scoring others, ``budget`` in all.  q bf16 [total_q, H, d]; cu_seqlens_q int32 [B + 1] or None (one
    token per request).  Returns (tables int32 [total_q, H_kv, budget] physical page ids, -1 behind the
    chosen ones; sel_lens int32 [total_q], the keys they hold)."""
    dev = _device(q, "q")
    ptrs, (B, T, H, H_kv, d), max_pages, num_pages = _selection_args(q, sketch, amp, block_table, seq_lens,
                                                                     cu_seqlens_q, dev)
    page_size, budget = _size(page_size, "page_size"), _size(budget, "budget")
    first, last = _size(first, "first"), _size(last, "last")
    if budget < 1:
        raise AttnError(ATTN_ERR_INVALID_ARG, "attn_page_select")
    with _on(stream):
        if tables is None:
            tables = torch.empty((T, H_kv, budget), dtype=torch.int32, device=q.device)
        if sel_lens is None:
            sel_lens = torch.empty((T,), dtype=torch.int32, device=q.device)
    tp = _check(tables, "tables", torch.int32, dev, (T, H_kv, budget))
    lp = _check(sel_lens, "sel_lens", torch.int32, dev, (T,))
    h = _handle(stream, dev)
    _with_workspace(lambda wp, wn: lib().attn_page_select(*ptrs, B, T, H, H_kv, d, page_size, max_pages, num_pages, budget,
                                                          first, last, tp, lp, wp, wn, h),
                    lambda: attn_page_select_workspace_size(T, H_kv, max_pages, budget), workspace, dev, stream, q.device,
                    "attn_page_select")
    return tables, sel_lens


def paged_sparse_fwd(q, k_cache, v_cache, block_table, seq_lens, sketch, amp, budget, first=1, last=1,
                     cu_seqlens_q=None, scale=None, out=None, lse=None, return_lse=True, return_tables=False,
                     workspace=None, stream=None):
    """Attention of each query token over the pages that ``page_select`` chooses for it.

    As ``paged_fwd`` with causal=True, plus the sketches of ``page_sketch`` and the selection's budget.
    Returns (o bf16 like q, lse fp32 [total_q, H]); with ``return_tables`` also the selection (tables,
    sel_lens)."""
    dev = _device(q, "q")
    ptrs, (B, T, H, H_kv, d), max_pages, num_pages = _selection_args(q, sketch, amp, block_table, seq_lens,
                                                                     cu_seqlens_q, dev)
    bf = torch.bfloat16
    _dims(k_cache, "k_cache", 4)
    page_size, budget = k_cache.shape[1], _size(budget, "budget")
    first, last = _size(first, "first"), _size(last, "last")
    cache = (num_pages, page_size, H_kv, d)
    kp, vp = _check(k_cache, "k_cache", bf, dev, cache), _check(v_cache, "v_cache", bf, dev, cache)
    tables = sel_lens = None
    with _on(stream):
        if out is None:
            out = torch.empty((T, H, d), dtype=bf, device=q.device)
        if lse is None and return_lse:
            lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
        if return_tables and budget > 0:
            tables = torch.empty((T, H_kv, budget), dtype=torch.int32, device=q.device)
            sel_lens = torch.empty((T,), dtype=torch.int32, device=q.device)
    op = _check(out, "out", bf, dev, (T, H, d))
    lp = None if lse is None else _check(lse, "lse", torch.float32, dev, (T, H))
    tp = None if tables is None else tables.data_ptr()
    sp = None if sel_lens is None else sel_lens.data_ptr()
    sc, h = float(scale) if scale is not None else 1.0 / math.sqrt(d), _handle(stream, dev)
    qp, skp, ap, bp, cp, np_ = ptrs
    _with_workspace(lambda wp, wn: lib().attn_paged_sparse_fwd(qp, kp, vp, bp, cp, np_, skp, ap, B, T, H, H_kv, d, page_size,
                                                               max_pages, num_pages, budget, first, last, sc, op, lp,
                                                               tp, sp, wp, wn, h),
                    lambda: attn_paged_sparse_fwd_workspace_size(T, H, H_kv, d, page_size, max_pages, budget), workspace, dev,
                    stream, q.device, "attn_paged_sparse_fwd")
    return (out, lse, tables, sel_lens) if return_tables else (out, lse)
