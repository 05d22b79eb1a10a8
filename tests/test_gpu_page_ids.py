"""Page ids out of range in the block table: page selection and page-sparse attention report them whether or
not the page was scored, and never hand them on."""
import pytest
import torch

import attention_attn_fwd_03_gb300 as attn

from test_gpu_sparse import _case, _gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.lib()


def _status():
    with pytest.raises(attn.AttnError) as e:
        attn.device_status()
    assert e.value.status == attn.ATTN_ERR_DEVICE_DATA
    attn.device_status()


@pytest.mark.parametrize("bad", [10 ** 6, -5, -1])
@pytest.mark.parametrize("budget,at", [
    (20, 0), (20, 7), (20, 18),  # every page is taken
    (6, 0), (6, 18), (6, 17),    # the first page, the query's own, the last but one
])
@pytest.mark.parametrize("H", [4, 60])  # one kernel; the selection kernels and the paged kernel
def test_bad_page_ids_are_reported_and_become_minus_one(bad, budget, at, H):
    c = _case(41, [300, 150], None, H, 2, 128, 16)  # 19 and 10 pages
    g = _gpu(c)
    args = (g["sk"], g["amp"], g["bt"], g["lens"])
    want, want_sel = attn.page_select(g["q"], *args, 16, budget, 1, 2)
    attn.device_status()
    id_ = int(c["table"][0, at])
    g["bt"][0, at] = bad
    tables, sel = attn.page_select(g["q"], *args, 16, budget, 1, 2)
    _status()
    assert torch.equal(sel, want_sel)
    assert torch.equal(tables, torch.where(want == id_, -1, want))
    _, _, t2, s2 = attn.paged_sparse_fwd(g["q"], g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], budget, 1, 2,
                                         return_tables=True)
    _status()
    assert torch.equal(t2, tables) and torch.equal(s2, sel)


def test_a_bad_id_among_the_scored_pages_is_the_last_to_be_taken():
    c = _case(42, [300], None, 4, 2, 128, 16)
    g = _gpu(c)
    g["bt"][0, 5], g["bt"][0, 9] = 10 ** 6, -5
    for budget, missing in ((16, 0), (17, 0), (18, 1)):  # 19 pages, 17 of them there
        tables, _ = attn.page_select(g["q"], g["sk"], g["amp"], g["bt"], g["lens"], 16, budget, 1, 1)
        _status()
        assert bool(((tables == -1).sum(-1) == missing).all())
        assert bool((tables < c["k"].shape[0]).all())
