"""Page-sparse attention of groups, budgets and tables that one kernel does not take: the selection kernels and
the paged kernel with a table row per token and KV head.  Each case asserts that it is on that path, and
whether its tokens' keys are split over several units."""
import numpy as np
import pytest
import torch

import attention_attn_fwd_03_gb300 as attn

import _kv_ref as ref
from _parity import default_scale
from test_gpu_sparse import _case, _gpu, _want

pytestmark = pytest.mark.gpu
DEV = "cuda"
GROUPS = [(60, 2, 128), (80, 2, 64)]  # G = 30 and 40


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.lib()


def _on_wide_path(T, H, H_kv, d, page, max_pages, budget, split):
    """The workspace holds the scores, tables and work list, and partials (fp32 O) if anything is split."""
    size = attn.attn_paged_sparse_fwd_workspace_size(T, H, H_kv, d, page, max_pages, budget)
    assert size > 256
    rest = attn.attn_page_select_workspace_size(T, H_kv, max_pages, budget) + 4 * T * H_kv * budget
    assert (size >= rest + 2 * T * H * d * 4) == split, (size, rest)


def _sparse(c, g, budget, first=1, last=1, **kw):
    out = attn.paged_sparse_fwd(g["q"], g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], budget, first, last,
                                cu_seqlens_q=g["cu"], **kw)
    return out


@pytest.mark.parametrize("H,H_kv,d", GROUPS)
@pytest.mark.parametrize("budget,split", [(6, False), (32, False), (40, True)])
def test_rows_behind_the_last_request_stay(H, H_kv, d, budget, split):
    c = _case(51, [300, 200], [3, 2], H, H_kv, d, 8)
    g = _gpu(c)
    pad = 4
    _on_wide_path(5 + pad, H, H_kv, d, 8, c["table"].shape[1], budget, split)
    o2, lse2, t2, s2 = _sparse(c, g, budget, return_tables=True)
    g["q"] = torch.cat([g["q"], torch.full((pad, H, d), float("nan"), dtype=torch.bfloat16, device=DEV)])
    o, lse = torch.full_like(g["q"], 3.0), torch.full((5 + pad, H), 3.0, device=DEV)
    _, _, tables, sel = _sparse(c, g, budget, out=o, lse=lse, return_tables=True)
    attn.device_status()
    want, want_sel = _want(c, budget, 1, 1)
    assert np.array_equal(tables[:5].cpu().numpy(), want) and sel.tolist() == want_sel.tolist() + [0] * pad
    assert bool((tables[5:] == -1).all())
    assert bool((o[5:] == 3).all()) and bool((lse[5:] == 3).all())
    assert torch.equal(t2, tables[:5]) and torch.equal(s2, sel[:5])
    ro, rl, bo, bl = ref.attend(c["q"].float().numpy(), c["k"].float().numpy(), c["v"].float().numpy(), want, want_sel,
                                default_scale(d))
    for x, y in ((o[:5], lse[:5]), (o2, lse2)):
        assert np.all(np.abs(x.double().cpu().numpy() - ro) <= bo)
        assert np.all(np.abs(y.double().cpu().numpy() - rl) <= bl)


@pytest.mark.parametrize("H,H_kv,d", GROUPS)
@pytest.mark.parametrize("what", ["page id", "length", "offsets", "negative length"])
def test_bad_device_data_is_reported(H, H_kv, d, what):
    c = _case(14, [300, 200], [3, 2], H, H_kv, d, 8)
    if what == "page id":
        c["table"][0, 5], c["table"][1, 2] = 10 ** 6, -5
    elif what == "length":
        c["lens"][1] = 10 ** 9
    elif what == "negative length":
        c["lens"][0] = -3
    else:
        c["cu"] = [0, 9, 5]
    g = _gpu(c)
    for budget, split in ((4, False), (64, True)):
        _on_wide_path(5, H, H_kv, d, 8, c["table"].shape[1], budget, split)
        _sparse(c, g, budget)
        with pytest.raises(attn.AttnError) as e:
            attn.device_status()
        assert e.value.status == attn.ATTN_ERR_DEVICE_DATA
    attn.device_status()


@pytest.mark.parametrize("H,H_kv,d", GROUPS)
@pytest.mark.parametrize("budget,split", [(8, False), (40, True)])
def test_recorded_timeout_leaves_outputs_alone(H, H_kv, d, budget, split):
    c = _case(16, [900, 300], None, H, H_kv, d, 16)
    g = _gpu(c)
    _on_wide_path(2, H, H_kv, d, 16, c["table"].shape[1], budget, split)
    o_ref, l_ref = _sparse(c, g, budget)
    attn.device_status()
    o, l = torch.full_like(o_ref, 3.0), torch.full_like(l_ref, 3.0)
    assert attn.attn_selftest_wait_timeout(torch.cuda.current_stream().cuda_stream) == attn.ATTN_OK
    _sparse(c, g, budget, out=o, lse=l)
    with pytest.raises(attn.AttnError) as e:
        attn.device_status()
    assert e.value.status == attn.ATTN_ERR_TIMEOUT
    assert bool((o == 3).all()) and bool((l == 3).all())
    _sparse(c, g, budget, out=o, lse=l)
    attn.device_status()
    assert torch.equal(o, o_ref) and torch.equal(l, l_ref)


def test_caches_past_32_bit_offsets():
    """Pages at the end of a cache of more than 2^32 elements (one cache for K and V)."""
    pages, page, H, H_kv, d, n = 66000, 64, 30 * 8, 8, 128, 40
    c = _case(17, [n * page - 7], None, H, H_kv, d, page)
    c["v"] = c["k"]
    ids = c["table"][0, :n].long()
    far = pages - 1 - 3 * torch.arange(n)
    k = torch.empty((pages, page, H_kv, d), dtype=torch.bfloat16, device=DEV)
    sk, amp = torch.zeros((pages, H_kv, 2 * d), dtype=torch.int8, device=DEV), torch.zeros((pages, H_kv), device=DEV)
    k[far.to(DEV)] = c["k"][ids].to(DEV)
    sk[far.to(DEV)], amp[far.to(DEV)] = torch.from_numpy(c["sk"])[ids].to(DEV), torch.from_numpy(c["amp"])[ids].to(DEV)
    g = _gpu(c)
    _on_wide_path(1, H, H_kv, d, page, n, 9, True)
    want = attn.paged_sparse_fwd(g["q"], g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], 9)
    got = attn.paged_sparse_fwd(g["q"], k, k, far.to(torch.int32)[None].contiguous().to(DEV), g["lens"], sk, amp, 9)
    attn.device_status()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("H,H_kv,d", GROUPS)
def test_one_workspace_for_changing_steps(H, H_kv, d):
    """Call after call in one workspace, each with other queries, lengths and offsets, without a pause between
    them: every call reads the tables, offsets and lengths that its own selection has written."""
    c = _case(61, [900, 500, 0, 700], [3, 1, 0, 2], H, H_kv, d, 16)
    g = _gpu(c)
    steps = []
    rng = np.random.default_rng(7)
    for i in range(24):
        cu = np.concatenate([[0], np.sort(rng.integers(0, 7, 3)), [6]]).astype(np.int32)
        lens = np.array([rng.integers(0, n + 1) for n in (900, 500, 0, 700)], dtype=np.int32)
        steps.append((torch.from_numpy(cu).to(DEV), torch.from_numpy(lens).to(DEV),
                      torch.randn(g["q"].shape, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).to(DEV)))
    for budget in (8, 40):
        ws = torch.full((attn.attn_paged_sparse_fwd_workspace_size(6, H, H_kv, d, 16, c["table"].shape[1], budget),), 0xFF,
                        dtype=torch.uint8, device=DEV)

        def run(step, **kw):
            cu, lens, q = step
            return attn.paged_sparse_fwd(q, g["k"], g["v"], g["bt"], lens, g["sk"], g["amp"], budget, cu_seqlens_q=cu, **kw)
        want = []
        for s in steps:
            want.append(run(s))
            torch.cuda.synchronize()
        got = [run(s, workspace=ws) for s in steps]
        torch.cuda.synchronize()
        for (o, l), (o2, l2) in zip(want, got):
            assert torch.equal(o, o2) and torch.equal(l, l2)
    attn.device_status()
