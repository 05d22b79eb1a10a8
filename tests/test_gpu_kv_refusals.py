"""What the helpers around the cache refuse on the host, by kind: TypeError for what is no CUDA tensor or of the
wrong type, ValueError for wrong shapes and values."""
import pytest
import torch

import attention_attn_fwd_03_gb300 as attn

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.lib()


def _calls():
    """name -> (helper, keyword arguments of a call that is right)."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)
    f = attn.rope_inv_freq(64)[0].to(DEV)
    sk, amp = torch.zeros((4, 2, 128), dtype=torch.int8, device=DEV), torch.zeros((4, 2), device=DEV)
    free = torch.arange(4, dtype=torch.int32, device=DEV)
    return {
        "rope": (attn.rope, dict(q=bf(2, 4, 3, 64), k=bf(2, 2, 3, 64), inv_freq=f, positions=i32(3))),
        "paged_plan": (attn.paged_plan, dict(ctx_lens=i32(2), block_table=i32(2, 3), free_pages=free, free_count=i32(1) + 4,
                                             page_size=16, num_pages=4, total_q=2)),
        "paged_append": (attn.paged_append, dict(q=bf(2, 4, 64), k=bf(2, 2, 64), v=bf(2, 2, 64), k_cache=bf(4, 16, 2, 64),
                                                 v_cache=bf(4, 16, 2, 64), slots=i32(2) - 1, positions=i32(2), inv_freq=f)),
        "page_sketch": (attn.page_sketch, dict(k_cache=bf(4, 16, 2, 64), block_table=i32(2, 3), seq_lens=i32(2), sketch=sk,
                                               amp=amp)),
        "page_select": (attn.page_select, dict(q=bf(2, 4, 64), sketch=sk, amp=amp, block_table=i32(2, 3), seq_lens=i32(2),
                                               page_size=16, budget=2)),
        "paged_sparse_fwd": (attn.paged_sparse_fwd, dict(q=bf(2, 4, 64), k_cache=bf(4, 16, 2, 64), v_cache=bf(4, 16, 2, 64),
                                                         block_table=i32(2, 3), seq_lens=i32(2), sketch=sk, amp=amp, budget=2)),
    }


OPTIONAL = {"rope": ("k", "positions"), "paged_append": ("q",)}


@pytest.mark.parametrize("name", ["rope", "paged_plan", "paged_append", "page_sketch", "page_select", "paged_sparse_fwd"])
def test_what_is_no_tensor_is_a_type_error(name):
    call, kw = _calls()[name]
    call(**kw)
    attn.device_status()
    for arg, value in kw.items():
        if not isinstance(value, torch.Tensor):
            continue
        for wrong in (None, [1, 2], 3.0, value.cpu(), value.cpu().numpy() if value.dtype is not torch.bfloat16 else "x"):
            if wrong is None and (arg in OPTIONAL.get(name, ()) or name == "paged_append" and arg in ("positions", "inv_freq")):
                continue
            with pytest.raises(TypeError):
                call(**dict(kw, **{arg: wrong}))
    if name == "paged_append":  # these two go together
        for arg in ("positions", "inv_freq"):
            with pytest.raises(ValueError):
                call(**dict(kw, **{arg: None}))


def test_k_out_without_k_is_refused():
    call, kw = _calls()["rope"]
    out = torch.full((2, 2, 3, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        call(**dict(kw, k=None, k_out=out))
    assert bool((out == 5).all())


@pytest.mark.parametrize("name,arg", [("paged_plan", "page_size"), ("paged_plan", "num_pages"), ("paged_plan", "total_q"),
                                      ("page_sketch", "max_q_len"), ("page_select", "page_size"), ("page_select", "budget"),
                                      ("page_select", "first"), ("page_select", "last"), ("paged_sparse_fwd", "budget"),
                                      ("paged_sparse_fwd", "first"), ("paged_sparse_fwd", "last")])
def test_sizes_past_32_bits_do_not_wrap(name, arg):
    """2^32 more than a good value is not that value."""
    call, kw = _calls()[name]
    good = dict(dict(first=0, last=1, max_q_len=1), **kw)[arg]
    with pytest.raises((ValueError, attn.AttnError)):
        call(**dict(kw, **{arg: good + 2 ** 32}))
    attn.device_status()
