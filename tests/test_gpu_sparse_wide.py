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
