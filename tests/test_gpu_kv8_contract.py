"""The operators on the 8-bit cache at the edges of what include/attn_kv8.h and the helpers promise: every inverted
offset reported, index arrays that are still being written on another stream, tables wider than 32 bits, many blocks
whose scales grow at once."""
import pytest
import torch

import attention_attn_fwd_03_gb300 as attn

import _kv8_ref as ref
from test_gpu_kv8 import BF, DEV, _append, _append_case, _check_append, _gpu_cache, _read_case

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


# ---------------------------------------------------------------- appends into blocks that hold rows

def _shrink_scales(c, g, share):
    """Some of the scales so small that the new rows need larger ones."""
    for name in ("k_scale", "v_scale"):
        small = torch.rand(c[name].shape, generator=g) < share
        c[name] = torch.where(small, 2.0 ** -torch.randint(10, 16, c[name].shape, generator=g).float(), c[name])


@pytest.mark.parametrize("page,block", [(64, 64), (16, 8), (1024, 256)])
@pytest.mark.parametrize("H_kv,d", [(1, 64), (3, 128), (20, 64)])
@pytest.mark.parametrize("share", [1.0, 0.3])
def test_append_many_blocks_grow_in_one_call(page, block, H_kv, d, share):
    """One token, or a few, to each of many requests, whose blocks hold rows: all of them grow, or some."""
    g = torch.Generator().manual_seed(page + H_kv + d)
    B = 150 if page < 1024 else 70
    ctx = torch.randint(1, 3 * page, (B,), generator=g).tolist()
    ctx[:4] = [block - 1, page - 1, 1, 2 * page]
    new = [1 + (i % 7 == 0) * (i % 3) for i in range(B)]
    c = _append_case(H_kv, ctx, new, page, block, 0, H_kv, d)
    _shrink_scales(c, g, share)
    got = _append(c)
    _check_append(c, got)
    if share == 1.0:
        held = [s for s, n in zip(c["slots"].tolist(), ctx) if s % block]
        assert len(held) > B // 3
        for name, i in (("k_scale", 3), ("v_scale", 4)):  # growth there was, in most heads of most blocks
            grew = [(got[i][s // page, :, s % page // block] > c[name][s // page, :, s % page // block]).float().mean() for s in held]
            assert torch.stack(grew).mean() > 0.5


@pytest.mark.parametrize("d,rot,interleaved,amplitude", [(128, 128, False, 1.0), (128, 64, True, 1.25), (64, 64, False, 0.5),
                                                         (64, 16, True, 1.0)])
@pytest.mark.parametrize("page,block", [(16, 1), (64, 16), (64, 64)])
def test_append_rotated_keys_scales_rows_held_and_rows_elsewhere(d, rot, interleaved, amplitude, page, block):
    """K turned in 32 bits lies within _kv8_ref.rotate's `off` of its value: each scale is that of an amplitude so near,
    the new codes those of values so near over it, the rows held are the old codes over it, and all else is as it was."""
    g = torch.Generator().manual_seed(d + rot + block)
    ctx = [0, 3, page - 1, 5 * page + 7, 1000] + torch.randint(0, 4 * page, (60,), generator=g).tolist()
    new = [page + 3, 2, 1, 40, 1] + [1, 3] * 30
    c = _append_case(rot, ctx, new, page, block, 2, 3, d, rot=rot, pad=5)
    _shrink_scales(c, g, 0.5)
    got = _append(c, interleaved=interleaved, amplitude=amplitude)
    _check_append(c, got, interleaved, amplitude)
    x, off = ref.rotate(c["k"], c["pos"], c["freq"], interleaved, amplitude)
    had, scale_had, have, scale = c["k_cache"].double(), c["k_scale"].double(), got[1].double(), got[3].double()
    slots = c["slots"].tolist()
    elsewhere = torch.ones(had.shape[:2], dtype=torch.bool)
    same_scale = torch.ones(scale.shape, dtype=torch.bool)
    t = 0
    while t < len(slots):
        n = 1
        if slots[t] < 0:
            t += n
            continue
        while slots[t + n] == slots[t] + n and slots[t + n] % block:
            n += 1
        p, row = slots[t] // page, slots[t] % page
        b, held = row // block, row % block
        elsewhere[p, row - held:row - held + block] = False
        same_scale[p, :, b] = False
        for h in range(3):
            low, high = ((x[t:t + n, h].abs() + sign * off[t:t + n, h]).clamp(min=0).max().item() for sign in (-1, 1))
            before = scale_had[p, h, b].item() if held else 0.0
            now = scale[p, h, b].item()
            assert now in {max(before, ref.scale_for(a)) for a in (low, high)}, (t, h)
            lo, hi = (ref.to_e4m3((x[t:t + n, h] + sign * off[t:t + n, h]) / now) for sign in (-1, 1))
            new_codes = have[p, row:row + n, h]
            assert ((lo <= new_codes) & (new_codes <= hi)).all(), (t, h)
            if held:
                old = had[p, row - held:row, h]
                assert torch.equal(have[p, row - held:row, h], ref.to_e4m3(old * (before / now)) if now > before else old), (t, h)
        t += n
    assert torch.equal(have[elsewhere], had[elsewhere]) and torch.equal(scale[same_scale], scale_had[same_scale])
