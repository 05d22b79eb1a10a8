"""A recorded timeout and attention whose key ranges are split: the merge of the partials, like the kernel that
would have written them, leaves the outputs as they were."""
import pytest
import torch

import attention_attn_fwd_03_gb300 as attn

from test_gpu_sparse import _case, _gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,q_lens", [([3000, 40], None), ([5000, 2500], [3, 2])])
def test_recorded_timeout_leaves_split_requests_alone(lens, q_lens):
    attn.lib()
    c = _case(33, lens, q_lens, 8, 2, 128, 16)
    g = _gpu(c)
    kw = dict(cu_seqlens_q=g["cu"], max_q_len=None if q_lens is None else max(q_lens), causal=True)
    args = (g["q"], g["k"], g["v"], g["bt"], g["lens"])
    o_ref, l_ref = attn.paged_fwd(*args, **kw)
    attn.device_status()
    o, l = torch.full_like(o_ref, 3.0), torch.full_like(l_ref, 3.0)
    assert attn.attn_selftest_wait_timeout(torch.cuda.current_stream().cuda_stream) == attn.ATTN_OK
    attn.paged_fwd(*args, out=o, lse=l, **kw)
    with pytest.raises(attn.AttnError) as e:
        attn.device_status()
    assert e.value.status == attn.ATTN_ERR_TIMEOUT
    assert bool((o == 3).all()) and bool((l == 3).all())
    attn.paged_fwd(*args, out=o, lse=l, **kw)
    attn.device_status()
    assert torch.equal(o, o_ref) and torch.equal(l, l_ref)
