"""The entry points of include/attn_kv.h without a GPU: exported and bound, frequencies by their
formulas, and bad arguments refused on the host before anything is enqueued."""
import ctypes
import math
import os
import re

import pytest
import torch

import attention_attn_fwd_03_gb300 as attn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, UNS, WS = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED, attn.ATTN_ERR_WORKSPACE
FAKE = 1 << 20  # a 16-byte aligned non-NULL address; validation fails before any use


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.build()


def test_declared_functions_are_exported_and_bound():
    src = open(os.path.join(ROOT, "include", "attn_kv.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(attn_\w+)\s*\(", src)))
    assert names == sorted(["attn_rope_inv_freq", "attn_rope", "attn_paged_plan", "attn_paged_append",
                            "attn_page_sketch", "attn_page_select_workspace_size", "attn_page_select",
                            "attn_paged_sparse_fwd_workspace_size", "attn_paged_sparse_fwd"])
    raw = ctypes.CDLL(attn.LIB_PATH)
    for n in names:
        assert hasattr(raw, n) and callable(getattr(attn, n))
        args = re.search(r"\b%s\s*\(([^)]*)\)" % n, src, flags=re.S).group(1)
        assert len(getattr(attn.lib(), n).argtypes) == len(args.split(",")), n


# ---------------------------------------------------------------- frequencies

@pytest.mark.parametrize("rot,base,factor,orig", [(128, 10000.0, 8.0, 8192), (64, 500000.0, 1.0, 4096), (2, 100.0, 3.0, 1),
                                                  (96, 10000.0, 16.0, 100000)])
def test_rope_inv_freq_formulas(rot, base, factor, orig):
    def near(got, want):
        # a power, a product or two and a quotient in float64: a few roundings each
        assert len(got) == rot // 2
        for g, w in zip(got.tolist(), want):
            assert abs(g - w) <= 16 * 2.0 ** -53 * w
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    got, amp = attn.rope_inv_freq(rot, base)
    near(got, f)
    assert amp == 1.0 and got.dtype == torch.float64
    near(attn.rope_inv_freq(rot, base, "linear", factor)[0], [x / factor for x in f])
    if rot > 2:
        b2 = base * factor ** (rot / (rot - 2))
        near(attn.rope_inv_freq(rot, base, "ntk", factor)[0], [b2 ** (-2.0 * i / rot) for i in range(rot // 2)])
    got, amp = attn.rope_inv_freq(rot, base, "bands", factor, orig, 1.0, 4.0)
    for g, x in zip(got.tolist(), f):
        turns = orig * x / (2 * math.pi)
        if turns >= 4.0:
            assert abs(g - x) <= 16 * 2.0 ** -53 * x
        elif turns <= 1.0:
            assert abs(g - x / factor) <= 16 * 2.0 ** -53 * x
        else:
            t = (turns - 1.0) / 3.0
            assert abs(g - ((1 - t) * x / factor + t * x)) <= 1e-13 * x
    got, amp = attn.rope_inv_freq(rot, base, "yarn", factor, orig, 1.0, 32.0)
    assert abs(amp - (0.1 * math.log(factor) + 1.0)) < 1e-15
    c = [rot * math.log(orig / (2 * math.pi * n)) / (2 * math.log(base)) for n in (32.0, 1.0)]
    lo, hi = (min(max(x, 0.0), rot - 1.0) for x in (math.floor(c[0]), math.ceil(c[1])))
    for i, (g, x) in enumerate(zip(got.tolist(), f)):
        keep = 1.0 - min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
        assert abs(g - (keep * x + (1 - keep) * x / factor)) <= 1e-13 * x


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=7), dict(rot=1026), dict(base=1.0), dict(base=float("nan")),
                                dict(scaling="linear", factor=0.5), dict(scaling="yarn", factor=float("inf")),
                                dict(scaling="bands", factor=2.0, orig_len=0),
                                dict(scaling="bands", factor=2.0, low=4.0, high=4.0),
                                dict(scaling="yarn", factor=2.0, low=0.0)])
def test_rope_inv_freq_refusals(kw):
    with pytest.raises(attn.AttnError) as e:
        attn.rope_inv_freq(**dict(dict(rot=64), **kw))
    assert e.value.status == BAD


def test_rope_inv_freq_unknown_scaling():
    with pytest.raises(ValueError):
        attn.rope_inv_freq(64, scaling="cubic")


# ---------------------------------------------------------------- refusals of the device calls

def _ll(*v):
    return (ctypes.c_longlong * len(v))(*v)


def _rope(**kw):
    s = kw.pop("s", (2 * 8 * 128, 128, 2 * 128))
    a = dict(q=FAKE, q_out=FAKE, k=None, k_out=None, positions=None, pos_stride_b=0, inv_freq=FAKE, freq_bits=64,
             elem_bytes=2, B=2, H=2, H_k=2, N=8, d=128, rot=128, strides=_ll(*s * 4), interleaved=0, inverse=0,
             amplitude=1.0, stream=None)
    a.update(kw)
    return attn.attn_rope(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), BAD), (dict(q_out=None), BAD), (dict(inv_freq=None), BAD), (dict(strides=None), BAD),
    (dict(k=FAKE), BAD), (dict(k_out=FAKE), BAD), (dict(k=FAKE, k_out=FAKE, H_k=0), BAD), (dict(B=0), BAD),
    (dict(H=0), BAD), (dict(H=65536), BAD), (dict(N=0), BAD), (dict(B=1 << 16, N=1 << 15), BAD),
    (dict(interleaved=2), BAD), (dict(inverse=-1), BAD), (dict(freq_bits=16), BAD), (dict(amplitude=float("nan")), BAD),
    (dict(elem_bytes=8), UNS), (dict(d=96), UNS), (dict(rot=0), UNS), (dict(rot=24), UNS), (dict(rot=144), UNS),
    (dict(q=FAKE + 8), BAD), (dict(q_out=FAKE + 2), BAD), (dict(inv_freq=FAKE + 4), BAD), (dict(positions=FAKE + 2), BAD),
    (dict(positions=FAKE, pos_stride_b=-1), BAD),
    (dict(s=(2048, 132, 256)), BAD),       # rows off the 16-byte grid
    (dict(s=(2048, -128, 256)), BAD),
    (dict(s=(0, 128, 256)), BAD),          # an output whose batch entries coincide
    (dict(s=(2048, 64, 256)), BAD),        # output heads that overlap
    (dict(s=(2048, 1 << 60, 256)), BAD),
])
def test_rope_refusals(kw, code):
    assert _rope(**kw) == code


def _plan(**kw):
    a = dict(ctx_lens=FAKE, new_lens=None, block_table=FAKE, free_pages=FAKE, free_count=FAKE, B=4, total_q=4,
             page_size=64, max_pages=8, num_pages=32, n_free=32, cu_seqlens_q=FAKE, seq_lens=FAKE, positions=FAKE,
             slots=FAKE, free_left=FAKE, stream=None)
    a.update(kw)
    return attn.attn_paged_plan(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(ctx_lens=None), BAD), (dict(block_table=None), BAD), (dict(free_pages=None), BAD), (dict(free_count=None), BAD),
    (dict(slots=None), BAD), (dict(free_left=None), BAD), (dict(B=0), BAD), (dict(total_q=0), BAD), (dict(n_free=0), BAD),
    (dict(num_pages=0), BAD), (dict(max_pages=0), BAD), (dict(new_lens=FAKE + 1), BAD), (dict(positions=FAKE + 2), BAD),
    (dict(B=16385), UNS), (dict(page_size=12), UNS), (dict(page_size=2048), UNS),
    (dict(max_pages=1 << 26), BAD), (dict(num_pages=1 << 26), BAD),
])
def test_plan_refusals(kw, code):
    assert _plan(**kw) == code


def _append(**kw):
    s = kw.pop("s", (5 * 128, 128))
    a = dict(q=FAKE, q_out=FAKE, k=FAKE, v=FAKE, k_cache=FAKE, v_cache=FAKE, slots=FAKE, positions=FAKE, inv_freq=FAKE,
             freq_bits=64, T=4, H=2, H_kv=2, d=128, rot=128, page_size=64, num_pages=4, strides=_ll(*s * 4), interleaved=0,
             amplitude=1.0, stream=None)
    a.update(kw)
    return attn.attn_paged_append(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), BAD), (dict(q_out=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(k_cache=None), BAD),
    (dict(slots=None), BAD), (dict(positions=None), BAD), (dict(inv_freq=None), BAD), (dict(freq_bits=0), BAD),
    (dict(T=0), BAD), (dict(H=0), BAD), (dict(H_kv=0), BAD), (dict(num_pages=0), BAD), (dict(interleaved=3), BAD),
    (dict(amplitude=float("inf")), BAD), (dict(v=FAKE + 8), BAD), (dict(v_cache=FAKE + 4), BAD), (dict(slots=FAKE + 2), BAD),
    (dict(d=80), UNS), (dict(rot=8), UNS), (dict(rot=-16), UNS), (dict(page_size=10), UNS), (dict(num_pages=1 << 25), BAD),
    (dict(s=(640, 130)), BAD), (dict(s=(640, 0)), BAD),
])
def test_append_refusals(kw, code):
    assert _append(**kw) == code


def _sketch(**kw):
    a = dict(k_cache=FAKE, block_table=FAKE, cu_seqlens_q=None, seq_lens=FAKE, B=2, max_q_len=1, H_kv=2, d=128,
             page_size=64, max_pages=4, num_pages=8, sketch=FAKE, amp=FAKE, stream=None)
    a.update(kw)
    return attn.attn_page_sketch(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(k_cache=None), BAD), (dict(seq_lens=None), BAD), (dict(sketch=None), BAD), (dict(amp=None), BAD),
    (dict(B=0), BAD), (dict(max_q_len=0), BAD), (dict(H_kv=0), BAD), (dict(k_cache=FAKE + 8), BAD),
    (dict(sketch=FAKE + 8), BAD), (dict(cu_seqlens_q=FAKE + 1), BAD), (dict(d=32), UNS), (dict(page_size=48), UNS),
    (dict(max_pages=1 << 25), BAD), (dict(B=1 << 20, max_pages=1 << 12, max_q_len=1 << 30), BAD),
])
def test_sketch_refusals(kw, code):
    assert _sketch(**kw) == code


def _select(**kw):
    a = dict(q=FAKE, sketch=FAKE, amp=FAKE, block_table=FAKE, cu_seqlens_q=None, seq_lens=FAKE, B=4, total_q=4, H=8,
             H_kv=2, d=128, page_size=64, max_pages=64, num_pages=256, budget=8, first=1, last=2, tables=FAKE,
             sel_lens=FAKE, workspace=FAKE, workspace_bytes=1 << 20, stream=None)
    a.update(kw)
    return attn.attn_page_select(**a)


SELECTION = [
    (dict(q=None), BAD), (dict(sketch=None), BAD), (dict(amp=None), BAD), (dict(block_table=None), BAD),
    (dict(seq_lens=None), BAD), (dict(total_q=5), BAD), (dict(H=9), BAD), (dict(H_kv=0), BAD), (dict(budget=0), BAD),
    (dict(first=-1), BAD), (dict(last=0), BAD), (dict(first=7), BAD), (dict(first=2 ** 31 - 1), BAD), (dict(q=FAKE + 8), BAD),
    (dict(amp=FAKE + 4), BAD), (dict(sketch=FAKE + 4), BAD), (dict(seq_lens=FAKE + 2), BAD), (dict(num_pages=0), BAD),
    (dict(d=96), UNS), (dict(page_size=24), UNS), (dict(H=516, H_kv=2), UNS), (dict(max_pages=1 << 26), BAD),
    (dict(B=1 << 15, total_q=1 << 15, max_pages=1 << 15), BAD), (dict(budget=1 << 28), BAD),
]


@pytest.mark.parametrize("kw,code", SELECTION + [
    (dict(tables=None), BAD), (dict(sel_lens=None), BAD), (dict(workspace=None), WS), (dict(workspace=FAKE + 8), WS),
    (dict(workspace_bytes=4 * 2 * 64 * 4 - 1), WS)])
def test_select_refusals(kw, code):
    assert _select(**kw) == code


def _sparse(**kw):
    a = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, block_table=FAKE, cu_seqlens_q=None, seq_lens=FAKE, sketch=FAKE, amp=FAKE,
             B=4, total_q=4, H=8, H_kv=2, d=128, page_size=64, max_pages=64, num_pages=256, budget=8, first=1, last=2,
             scale=0.1, o=FAKE, lse=None, tables=None, sel_lens=None, workspace=FAKE, workspace_bytes=1 << 24, stream=None)
    a.update(kw)
    return attn.attn_paged_sparse_fwd(**a)


@pytest.mark.parametrize("kw,code", SELECTION + [
    (dict(k_cache=None), BAD), (dict(v_cache=FAKE + 8), BAD), (dict(o=None), BAD), (dict(o=FAKE + 4), BAD),
    (dict(lse=FAKE + 2), BAD), (dict(tables=FAKE), BAD), (dict(sel_lens=FAKE), BAD), (dict(scale=0.0), BAD),
    (dict(scale=float("nan")), BAD), (dict(H=80, workspace=None), WS), (dict(H=80, workspace_bytes=4000), WS),
    (dict(H=80, workspace=FAKE + 8), WS)])
def test_sparse_refusals(kw, code):
    assert _sparse(**kw) == code


def test_workspace_sizes():
    size = attn.attn_page_select_workspace_size
    assert size(4, 2, 64, 8) == 4 * 2 * 64 * 4
    assert size(4, 2, 8, 8) == 256  # nothing is scored
    assert size(0, 2, 64, 8) == 0 and size(4, 2, 64, 0) == 0 and size(1 << 16, 1 << 10, 64, 8) == 0
    size = attn.attn_paged_sparse_fwd_workspace_size
    assert size(4, 8, 2, 128, 64, 64, 8) == 256  # one kernel, nothing in device memory
    # groups of more than 24 heads (d = 64: 32), budgets of more than 1024 pages, tables of more pages than shared memory
    # holds scores for: scores, selection and work list
    assert size(4, 64, 2, 64, 64, 64, 8) == 256 and size(4, 48, 2, 128, 64, 64, 8) == 256
    for H, max_pages, budget in ((50, 64, 8), (8, 2000, 1025), (8, 30000, 8)):
        assert size(4, H, 2, 128, 64, max_pages, budget) > attn.attn_page_select_workspace_size(4, 2, max_pages, budget)
    assert size(4, 9, 2, 128, 64, 64, 8) == 0 and size(4, 8, 2, 96, 64, 64, 8) == 0 and size(4, 8, 2, 128, 48, 64, 8) == 0


def test_helpers_refuse_host_tensors():
    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    f = attn.rope_inv_freq(128)[0]
    cache = torch.zeros((8, 64, 2, 128), dtype=torch.bfloat16)
    sk, amp = torch.zeros((8, 2, 256), dtype=torch.int8), torch.zeros((8, 2))
    bt = torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: attn.rope(q, inv_freq=f), lambda: attn.paged_plan(i, bt, i, i[:1], 64, 8, 4),
                 lambda: attn.paged_append(q, q[:, :2], q[:, :2], cache, cache, i),
                 lambda: attn.page_sketch(cache, bt, i, sk, amp), lambda: attn.page_select(q, sk, amp, bt, i, 64, 4),
                 lambda: attn.paged_sparse_fwd(q, cache, cache, bt, i, sk, amp, 4)):
        with pytest.raises(TypeError):
            call()
