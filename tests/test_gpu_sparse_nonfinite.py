"""NaN in what page-sparse attention reads: the heads that see it get NaN in O and in the LSE, not the
-inf of a token that sees no key, whichever path computes them; every other row keeps its bits."""
import pytest
import torch

import attention_attn_fwd_03_gb300 as attn

from test_gpu_sparse import _case, _gpu

pytestmark = pytest.mark.gpu

# G <= 24 (d = 64: 32) runs as one kernel, more on the selection kernels and the paged kernel; the
# budgets leave that one split per token (256 keys) and several
PATHS = [(16, 2, 128, 8), (16, 2, 128, 24), (60, 2, 128, 8), (60, 2, 128, 24), (16, 2, 64, 8), (80, 2, 64, 8), (80, 2, 64, 24)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.lib()


def _run(g, budget):
    o, lse = attn.paged_sparse_fwd(g["q"], g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], budget)
    attn.device_status()
    return o, lse


@pytest.mark.parametrize("H,H_kv,d,budget", PATHS)
@pytest.mark.parametrize("where", ["query", "key", "first key"])
def test_nan_reaches_output_and_lse(H, H_kv, d, budget, where):
    lens = [700, 20, 690, 0]
    c = _case(31, lens, None, H, H_kv, d, 32)
    g = _gpu(c)
    G = H // H_kv
    o_ref, l_ref = _run(g, budget)
    poisoned = torch.zeros((len(lens), H), dtype=torch.bool)
    if where == "query":
        g["q"][0, 3, 5] = float("nan")
        poisoned[0, 3] = True
        # the head's group may attend to other pages now: scores of a NaN query count as +inf
        same = ~poisoned
        same[0, :G] = False
    else:
        # a key that every token of request 0 sees: in its own, always chosen page, or in the first one
        last = (lens[0] - 1) // 32
        page, row = (int(c["table"][0, last]), 3) if where == "key" else (int(c["table"][0, 0]), 0)
        g["k"][page, row, 1, 7] = float("nan")
        poisoned[0, G:] = True
        same = ~poisoned
    poisoned, same = poisoned.to(o_ref.device), same.to(o_ref.device)
    o, lse = _run(g, budget)
    assert bool(torch.isnan(o[poisoned]).all()) and bool(torch.isnan(lse[poisoned]).all())
    assert torch.equal(o[same], o_ref[same]) and torch.equal(lse[same], l_ref[same])
    assert bool(torch.isneginf(lse[3]).all()) and bool((o[3] == 0).all())


@pytest.mark.parametrize("max_q_len", [1, 3])
def test_paged_attention_reports_nan_alike(max_q_len):
    """attn_paged_fwd, with and without a merge of split ranges."""
    lens = [3000, 40] if max_q_len == 1 else [100, 40]
    c = _case(32, lens, None if max_q_len == 1 else [3, 2], 8, 2, 128, 16)
    g = _gpu(c)
    args = (g["k"], g["v"], g["bt"], g["lens"])
    kw = dict(cu_seqlens_q=g["cu"], max_q_len=None if max_q_len == 1 else max_q_len, causal=True)
    o_ref, l_ref = attn.paged_fwd(g["q"], *args, **kw)
    q = g["q"].clone()
    q[0, 6, 0] = float("nan")
    o, lse = attn.paged_fwd(q, *args, **kw)
    attn.device_status()
    bad = torch.zeros(l_ref.shape, dtype=torch.bool, device=o.device)
    bad[0, 6] = True
    assert bool(torch.isnan(o[bad]).all()) and bool(torch.isnan(lse[bad]).all())
    assert torch.equal(o[~bad], o_ref[~bad]) and torch.equal(lse[~bad], l_ref[~bad])
