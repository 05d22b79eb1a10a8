"""The entry points of include/attn_kv8.h without a GPU: exported and bound, workspace sizes, and bad arguments
refused on the host before anything is enqueued."""
import ctypes
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
    src = open(os.path.join(ROOT, "include", "attn_kv8.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(attn_\w+)\s*\(", src)))
    assert names == sorted(["attn_paged_append_fp8", "attn_paged_read_fp8", "attn_paged_fwd_fp8_workspace_size",
                            "attn_paged_fwd_fp8"])
    raw = ctypes.CDLL(attn.LIB_PATH)
    for n in names:
        assert hasattr(raw, n) and callable(getattr(attn, n))
        args = re.search(r"\b%s\s*\(([^)]*)\)" % n, src, flags=re.S).group(1)
        assert len(getattr(attn.lib(), n).argtypes) == len(args.split(",")), n
    for n in ("paged_append_fp8", "paged_read_fp8", "paged_fwd_fp8"):
        assert callable(getattr(attn, n))


def _append(**kw):
    s = kw.pop("s", (5 * 128, 128))
    a = dict(q=FAKE, q_out=FAKE, k=FAKE, v=FAKE, k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE, slots=FAKE,
             positions=FAKE, inv_freq=FAKE, freq_bits=64, T=4, H=2, H_kv=2, d=128, rot=128, page_size=64, block=16, num_pages=4,
             strides=(ctypes.c_longlong * 8)(*s * 4), interleaved=0, amplitude=1.0, stream=None)
    a.update(kw)
    return attn.attn_paged_append_fp8(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), BAD), (dict(q_out=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(k_cache=None), BAD),
    (dict(v_cache=None), BAD), (dict(k_scale=None), BAD), (dict(v_scale=None), BAD), (dict(slots=None), BAD),
    (dict(positions=None), BAD), (dict(inv_freq=None), BAD), (dict(freq_bits=16), BAD), (dict(strides=None), BAD),
    (dict(T=0), BAD), (dict(T=0x7fffffff), BAD), (dict(T=0x7fffffff - 1024), BAD), (dict(H=0), BAD), (dict(H=65536), BAD),
    (dict(H_kv=0), BAD), (dict(H_kv=65536), BAD), (dict(num_pages=0), BAD), (dict(num_pages=1 << 25), BAD),
    (dict(interleaved=2), BAD), (dict(amplitude=float("nan")), BAD), (dict(q=FAKE + 8), BAD), (dict(v=FAKE + 8), BAD),
    (dict(k_cache=FAKE + 4), BAD), (dict(k_scale=FAKE + 2), BAD), (dict(v_scale=FAKE + 1), BAD), (dict(slots=FAKE + 2), BAD),
    (dict(d=96), UNS), (dict(rot=8), UNS), (dict(rot=144), UNS), (dict(rot=-16), UNS), (dict(page_size=12), UNS),
    (dict(page_size=24, block=8), UNS), (dict(page_size=2048), UNS), (dict(block=0), BAD), (dict(block=-16), BAD),
    (dict(block=12), UNS), (dict(block=128), BAD), (dict(s=(640, 130)), BAD), (dict(s=(640, 0)), BAD)])
def test_append_refusals(kw, code):
    assert _append(**kw) == code


def _read(**kw):
    a = dict(k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE, block_table=FAKE, cu_seqlens_k=FAKE, B=2, total_k=100,
             H_kv=2, d=128, page_size=64, block=16, max_pages=4, num_pages=8, k=FAKE, v=FAKE, elem_bytes=2, stream=None)
    a.update(kw)
    return attn.attn_paged_read_fp8(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None, v=None), BAD), (dict(k_cache=None), BAD), (dict(v_cache=None), BAD), (dict(k_scale=None), BAD),
    (dict(v_scale=None), BAD), (dict(block_table=None), BAD), (dict(cu_seqlens_k=None), BAD), (dict(B=0), BAD),
    (dict(total_k=0), BAD), (dict(total_k=0x7fffffff), BAD), (dict(H_kv=0), BAD), (dict(H_kv=65536), BAD), (dict(max_pages=0), BAD),
    (dict(num_pages=0), BAD), (dict(num_pages=1 << 25), BAD), (dict(max_pages=1 << 25), BAD),
    (dict(B=1 << 16, max_pages=1 << 16), BAD), (dict(k=FAKE + 8), BAD), (dict(v_cache=FAKE + 8), BAD),
    (dict(k_scale=FAKE + 2), BAD), (dict(block_table=FAKE + 1), BAD), (dict(cu_seqlens_k=FAKE + 2), BAD), (dict(d=80), UNS),
    (dict(elem_bytes=1), UNS), (dict(elem_bytes=8), UNS), (dict(page_size=20), UNS), (dict(block=3), UNS), (dict(block=128), BAD)])
def test_read_refusals(kw, code):
    assert _read(**kw) == code


def _fwd(**kw):
    a = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE, block_table=FAKE, cu_seqlens_q=None, seq_lens=FAKE,
             B=4, total_q=4, max_q_len=1, H=8, H_kv=2, d=128, page_size=64, block=16, max_pages=16, num_pages=64, scale=0.1,
             causal=1, o=FAKE, lse=None, workspace=FAKE, workspace_bytes=1 << 24, stream=None)
    a.update(kw)
    return attn.attn_paged_fwd_fp8(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), BAD), (dict(k_cache=None), BAD), (dict(v_cache=None), BAD), (dict(k_scale=None), BAD), (dict(v_scale=None), BAD),
    (dict(block_table=None), BAD), (dict(seq_lens=None), BAD), (dict(o=None), BAD), (dict(B=0), BAD), (dict(total_q=0), BAD),
    (dict(total_q=5), BAD), (dict(max_q_len=2), BAD), (dict(cu_seqlens_q=FAKE, max_q_len=5), BAD),
    (dict(cu_seqlens_q=FAKE, max_q_len=0), BAD), (dict(H=9), BAD), (dict(H_kv=0), BAD), (dict(num_pages=0), BAD),
    (dict(num_pages=1 << 25), BAD), (dict(max_pages=0), BAD), (dict(max_pages=1 << 25), BAD), (dict(scale=0.0), BAD),
    (dict(scale=float("inf")), BAD), (dict(scale=-1.0), BAD), (dict(causal=2), BAD), (dict(q=FAKE + 8), BAD), (dict(o=FAKE + 2), BAD),
    (dict(v_cache=FAKE + 8), BAD), (dict(k_scale=FAKE + 2), BAD), (dict(lse=FAKE + 2), BAD), (dict(seq_lens=FAKE + 1), BAD),
    (dict(cu_seqlens_q=FAKE + 2), BAD), (dict(d=32), UNS), (dict(H=258, H_kv=2), UNS), (dict(page_size=40, block=8), UNS),
    (dict(block=0), BAD), (dict(block=24), UNS), (dict(block=128), BAD), (dict(workspace=None), WS), (dict(workspace=FAKE + 8), WS),
    (dict(workspace_bytes=4000), WS), (dict(B=(1 << 30) + 1, total_q=(1 << 30) + 1, H=1, H_kv=1, max_pages=1), BAD)])
def test_fwd_refusals(kw, code):
    assert _fwd(**kw) == code


def test_workspace_sizes():
    size = attn.attn_paged_fwd_fp8_workspace_size
    ok = dict(B=4, total_q=4, max_q_len=1, H=8, H_kv=2, d=128, page_size=64, max_pages=16)
    n = size(**ok)
    assert n > 0
    assert _fwd(workspace_bytes=n - 1) == WS
    for bad in (dict(B=0), dict(H=9), dict(d=96), dict(page_size=48), dict(max_pages=0), dict(max_q_len=5), dict(H=516, H_kv=2)):
        assert size(**dict(ok, **bad)) == 0
    # one allocated for the largest batch, tables and token counts does for the smaller ones
    for H, H_kv, d in ((8, 2, 128), (8, 2, 64), (4, 1, 128), (16, 16, 64), (64, 8, 128), (6, 3, 64)):
        of = lambda B, q, pages: size(B, B * q, q, H, H_kv, d, 64, pages)
        for q in (1, 2, 4, 8, 40):
            for B in (1, 8, 64, 512):
                for pages in (1, 16, 256, 8192):
                    assert of(B, q, pages) <= of(512, q, 8192)
                    assert of(B, q, pages) <= of(B, 40, pages)


def test_helpers_refuse_host_tensors():
    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    cache = torch.zeros((8, 64, 2, 128), dtype=torch.float8_e4m3fn)
    scale = torch.zeros((8, 2, 4))
    bt = torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: attn.paged_append_fp8(q, q[:, :2], q[:, :2], cache, cache, scale, scale, i),
                 lambda: attn.paged_read_fp8(cache, cache, scale, scale, bt, i, 4),
                 lambda: attn.paged_fwd_fp8(q, cache, cache, scale, scale, bt, i),
                 lambda: attn.paged_fwd_fp8(None, cache, cache, scale, scale, bt, i)):
        with pytest.raises(TypeError):
            call()
