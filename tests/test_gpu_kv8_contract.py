"""The operators on the 8-bit cache at the edges of what include/attn_kv8.h and the helpers promise: every inverted
offset reported, index arrays that are still being written on another stream, tables wider than 32 bits, many blocks
whose scales grow at once."""
import pytest
import torch

import attention_attn_fwd_03_gb300 as attn

import _kv8_ref as ref
from test_gpu_kv8 import BF, DEV, F8, _gpu_cache, _read_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.lib()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- reading back

@pytest.mark.parametrize("cu", [[0, 10, 5, 12], [0, 20, 19, 20, 20], [0, 4, 8, 9, 9, 3], [0, 0, -1, 0, 20], [5, 0, 20],
                                [0, 20, 21, 20], [0, 3, 1 << 30, 3, 20]])
def test_read_reports_every_pair_of_offsets_that_is_not_in_order(cu):
    """Also a pair that no row of the output falls to."""
    c, _ = _read_case(3, [20] * (len(cu) - 1), 16, 16, 1, 64)
    k, v = (torch.full((24, 1, 64), 3.0, dtype=BF, device=DEV) for _ in "kv")
    attn.paged_read_fp8(*_gpu_cache(c), c["table"].to(DEV), _i32(cu), 20, k_out=k[:20], v_out=v[:20])
    with pytest.raises(attn.AttnError) as e:
        attn.device_status()
    assert e.value.status == attn.ATTN_ERR_DEVICE_DATA
    assert (k[20:] == 3).all() and (v[20:] == 3).all()
    for t in range(20):  # a row is one of the requests that have it, or as it was
        rows = [torch.full((1, 64), 3.0, dtype=BF)]
        for r, (a, b) in enumerate(zip(cu, cu[1:])):
            if 0 <= a <= t < b <= 20:
                rows.append(ref.values(c["k_cache"], c["k_scale"], c["table"][r], t - a + 1)[-1].to(BF))
        assert any(torch.equal(k[t].cpu(), x) for x in rows), t


def test_read_many_requests_one_pair_not_in_order():
    """More requests than a launch has threads, the bad pair anywhere among empty ones; and the same in order."""
    B = 5000
    c, _ = _read_case(4, [16], 16, 16, 1, 64)
    cache, table = _gpu_cache(c), c["table"][:1].to(DEV).expand(B, -1).contiguous()
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[B // 3:] = 16
    attn.paged_read_fp8(*cache, table, cu.to(DEV), 16)
    attn.device_status()
    for at in (1, 700, B // 3 + 9, B - 1):
        bad = cu.clone()
        bad[at] = 15 if cu[at] == 16 else 1
        attn.paged_read_fp8(*cache, table, bad.to(DEV), 16)
        with pytest.raises(attn.AttnError) as e:
            attn.device_status()
        assert e.value.status == attn.ATTN_ERR_DEVICE_DATA


# ---------------------------------------------------------------- attention's helper

def test_longest_request_is_read_on_the_calls_stream():
    """cu_seqlens_q is still being written by work on the stream that the call is given."""
    c, g = _read_case(5, [40, 9], 16, 16, 2, 64)
    cache, table, lens = _gpu_cache(c), c["table"].to(DEV), _i32(c["lens"])
    q = torch.randn((7, 4, 64), generator=g).to(BF).to(DEV)
    ready = _i32([0, 5, 7])
    want, want_lse = attn.paged_fwd_fp8(q, *cache, table, lens, cu_seqlens_q=ready, max_q_len=5, causal=True)
    attn.paged_fwd_fp8(q, *cache, table, lens, cu_seqlens_q=ready, causal=True)  # what the helper runs is loaded
    cu, side = torch.zeros_like(ready), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # a tenth of a second
        cu.copy_(ready)
    o, lse = attn.paged_fwd_fp8(q, *cache, table, lens, cu_seqlens_q=cu, causal=True, stream=side)
    torch.cuda.synchronize()
    attn.device_status()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


def test_tables_past_32_bits_are_refused():
    """Sizes that a C int would take the low 32 bits of."""
    c, g = _read_case(6, [40], 16, 16, 2, 64)
    cache, lens, q = _gpu_cache(c), _i32(c["lens"]), torch.zeros((1, 4, 64), dtype=BF, device=DEV)
    wide = torch.empty((1, (1 << 32) + 4), dtype=torch.int32, device=DEV)
    wide[:, :4] = c["table"][:, :4].to(DEV)
    with pytest.raises(ValueError, match="32 bits"):
        attn.paged_fwd_fp8(q, *cache, wide, lens)
    with pytest.raises(ValueError, match="32 bits"):
        attn.paged_read_fp8(*cache, wide, _i32([0, 40]), 40)
    many = wide.view(-1, 1)
    with pytest.raises(ValueError, match="32 bits"):
        attn.paged_fwd_fp8(q, *cache, many, lens)
    with pytest.raises(ValueError, match="32 bits"):
        attn.paged_read_fp8(*cache, many, _i32([0, 40]), 40)
    attn.device_status()
