"""A paged cache in 8 bits: appends that quantise (attn_paged_append_fp8), reading back (attn_paged_read_fp8) and
attention over it (attn_paged_fwd_fp8), against their definitions in 64 bits.

Codes and scales without a rotation are compared for equality; a rotation in 32 bits may move a value by what
_kv8_ref.rotate derives, and a code or scale to what that interval rounds to.  Attention is held to the bounds of
_kv8_ref.attend."""
import math

import pytest
import torch

import attention_attn_fwd_03_gb300 as attn

import _kv8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.lib()


def _bits(x):
    return x.contiguous().view(torch.uint8)


def _random_cache(g, pages, page, block, H_kv, d, spread=1.0):
    """Codes and scales of a cache in use: every code but NaN, scales that are powers of two."""
    codes = torch.randn((pages, page, H_kv, d), generator=g).mul(60).clamp(-448, 448).to(F8)
    scale = torch.exp2(torch.randint(-6, 3, (pages, H_kv, page // block), generator=g).float() * spread)
    return codes, scale


# ---------------------------------------------------------------- append

def _slots(g, ctx, new, page, extra=2):
    """Slots of requests with ctx cached and new appended tokens each, in scattered pages, and the pool's size."""
    need = [(c + n + page - 1) // page - c // page if n else 0 for c, n in zip(ctx, new)]
    pool = sum(need) + extra
    perm = torch.randperm(pool, generator=g).tolist()
    slots, pos = [], []
    for c, n, k in zip(ctx, new, need):
        ids, perm = perm[:k], perm[k:]
        for p in range(c, c + n):
            slots.append(ids[p // page - c // page] * page + p % page)
            pos.append(p)
    return slots, pos, pool


def _append(c, **kw):
    """Runs the append on copies of the case's cache on the GPU; returns (q_out, codes, codes, scale, scale) on the CPU."""
    t = lambda x: None if x is None else x.to(DEV)
    cache = [t(c[n]).clone() for n in ("k_cache", "v_cache", "k_scale", "v_scale")]
    q = attn.paged_append_fp8(t(c["q"]), t(c["k"]), t(c["v"]), *cache, t(c["slots"]), positions=t(c["pos"]),
                              inv_freq=t(c["freq"]), **kw)
    attn.device_status()
    return [None if q is None else q.cpu()] + [x.cpu() for x in cache]


def _append_case(seed, ctx, new, page, block, H, H_kv, d, rot=0, pad=0, size=1.0, order=None):
    g = torch.Generator().manual_seed(seed)
    slots, pos, pool = _slots(g, ctx, new, page)
    T = len(slots) + pad
    c = dict(page=page, block=block, rot=rot)
    c["q"] = torch.randn((T, H, d), generator=g).to(BF) if H else None
    c["k"] = (torch.randn((T, H_kv, d), generator=g) * size).to(BF)
    c["v"] = (torch.randn((T, H_kv, d), generator=g) * torch.exp2(torch.randn((T, 1, 1), generator=g) * 3)).to(BF)
    c["slots"] = torch.tensor(slots + [-1] * pad, dtype=torch.int32)
    c["pos"] = torch.tensor(pos + [0] * pad, dtype=torch.int32) if rot else None
    c["freq"] = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot) if rot else None
    (c["k_cache"], c["k_scale"]), (c["v_cache"], c["v_scale"]) = (_random_cache(g, pool, page, block, H_kv, d) for _ in "kv")
    return c


def _check_append(c, got, interleaved=False, amplitude=1.0):
    q, *cache = got
    keep = c["slots"] >= 0
    if c["q"] is not None:
        want, off = ref.rotate(c["q"][keep], c["pos"][keep] if c["rot"] else None, c["freq"], interleaved, amplitude)
        assert ((q[keep].double() - want).abs() <= 2.0 ** -8 * want.abs() + off * 2 + 1e-38).all()
    for side, i in (("k", 0), ("v", 1)):
        x, off = (ref.rotate(c["k"], c["pos"], c["freq"], interleaved, amplitude) if side == "k"
                  else (c["v"].double(), torch.zeros_like(c["v"], dtype=torch.float64)))
        had, scale_had = c[side + "_cache"].double(), c[side + "_scale"].double()
        codes, scale = had.clone(), scale_had.clone()
        ref.append(x, codes, scale, c["slots"].tolist(), c["block"])
        have, scale_have = cache[i].double(), cache[2 + i].double()
        if not c["rot"] or side == "v":
            assert torch.equal(scale_have, scale)
            valid = _valid(c, codes.shape)
            assert torch.equal(torch.where(valid, have, 0.0).nan_to_num(nan=1e6), torch.where(valid, codes, 0.0).nan_to_num(nan=1e6))
            continue
        # a value within off of the exact one, over the scale it was given
        differs = scale_have != scale
        assert differs.sum() <= 1 + differs.numel() // 1000
        page, per = c["page"], c["page"] // c["block"]
        for t, s in enumerate(c["slots"].tolist()):
            if s < 0:
                continue
            p, row = s // page, s % page
            now = scale_have[p, :, row // c["block"]][:, None]
            lo, hi = ref.to_e4m3((x[t] - off[t]) / now), ref.to_e4m3((x[t] + off[t]) / now)
            assert ((lo <= have[p, row]) & (have[p, row] <= hi)).all(), t
        assert per >= 1


def _valid(c, shape):
    """Rows that the call leaves valid: all but those behind the last that it writes in a block."""
    valid = torch.ones(shape[0] * shape[1], dtype=torch.bool)
    for s in c["slots"].tolist():
        if s >= 0:
            end = s - s % c["block"] + c["block"]
            valid[s + 1:end] = False
    for s in c["slots"].tolist():
        if s >= 0:
            valid[s] = True
    return valid.view(shape[0], shape[1], 1, 1)


@pytest.mark.parametrize("page,block", [(8, 1), (8, 8), (16, 2), (16, 16), (64, 1), (64, 16), (64, 64), (128, 64), (1024, 1024),
                                        (1024, 32)])
@pytest.mark.parametrize("H_kv,d", [(1, 128), (3, 64), (20, 128)])
def test_append_codes_and_scales(page, block, H_kv, d):
    ctx = [0, 5, 63, 64, 200, 1, 700]
    new = [1, 1, 1, 3, 70, 0, 2]
    c = _append_case(page * 7 + block + d, ctx, new, page, block, 2, H_kv, d)
    _check_append(c, _append(c))


@pytest.mark.parametrize("d,rot,interleaved,amplitude", [(128, 128, False, 1.0), (128, 128, True, 1.25), (128, 48, False, 1.0),
                                                         (64, 64, True, 1.0), (64, 16, False, 0.5), (64, 32, True, 1.0)])
@pytest.mark.parametrize("block", [1, 16, 64])
def test_append_rotates(d, rot, interleaved, amplitude, block):
    c = _append_case(rot + block, [0, 17, 130, 40000], [40, 1, 9, 150], 64, block, 4, 2, d, rot=rot, pad=3)
    _check_append(c, _append(c, interleaved=interleaved, amplitude=amplitude), interleaved, amplitude)


@pytest.mark.parametrize("T", [1, 31, 32, 33, 64, 257, 1500])
@pytest.mark.parametrize("block", [1, 128])
def test_append_token_counts(T, block):
    c = _append_case(T + block, [3], [T], 128, block, 1, 1, 128, rot=32)
    _check_append(c, _append(c))


def test_append_grows_a_scale_and_keeps_the_rows_there():
    """Token after token into one page, each larger than the one before: what lies there is the plain form's at each step."""
    page, H_kv, d = 16, 2, 64
    g = torch.Generator().manual_seed(1)
    codes, scale = torch.zeros((2, page, H_kv, d), dtype=F8), torch.zeros((2, H_kv, 1))
    cache = [codes.to(DEV), codes.clone().to(DEV), scale.to(DEV), scale.clone().to(DEV)]
    want_c, want_s = codes.double(), scale.double()
    for i in range(page):
        x = (torch.randn((1, H_kv, d), generator=g) * 1.7 ** i).to(BF)
        attn.paged_append_fp8(None, x.to(DEV), x.to(DEV), *cache, torch.tensor([page + i], dtype=torch.int32, device=DEV))
        ref.append(x.double(), want_c, want_s, [page + i], page)
        for side in (0, 1):
            assert torch.equal(cache[2 + side].cpu().double(), want_s)
            assert torch.equal(cache[side].cpu().double()[1, :i + 1], want_c[1, :i + 1])
    attn.device_status()


@pytest.mark.parametrize("size", [0.0, 1e-38, 2.0 ** -133, 1e-30, 1.0, 3e38])
def test_append_sizes_of_values(size):
    c = _append_case(3, [0, 4], [4, 3], 16, 4, 0, 2, 64, size=1.0)
    c["k"] = (c["k"].double().clamp(-1, 1) * size).to(BF)
    c["v"] = torch.full_like(c["v"], size)
    _check_append(c, _append(c))


def test_append_borders_of_the_scale():
    """Amplitudes at 448 2^e, the next bf16 above and below."""
    c = _append_case(4, [0], [48], 16, 1, 0, 1, 64)
    for t in range(48):
        e, k = t // 3 - 8, t % 3
        top = torch.tensor(448.0 * 2.0 ** e).to(BF).view(torch.int16) + (k - 1)
        c["k"][t] = 0.0
        c["k"][t, 0, t] = -top.view(BF)
    _check_append(c, _append(c))


def test_append_infinities_and_nan_become_nan():
    c = _append_case(5, [2, 0], [5, 8], 16, 8, 0, 2, 128)
    c["k"][1, 0, 7] = float("inf")
    c["k"][3, 1, 0] = float("nan")
    c["v"][0, 0, :] = float("-inf")
    c["v"][7, 1, 99] = float("nan")
    _check_append(c, _append(c))


def test_append_skips_tokens_without_a_slot():
    c = _append_case(6, [0], [40], 16, 8, 3, 2, 64)
    c["slots"][8:16] = -1
    c["slots"][33:] = -7
    q_out = torch.full((40, 3, 64), 5.0, dtype=BF, device=DEV)
    got = _append(c, q_out=q_out)
    _check_append(c, got)
    assert (got[0][8:16] == 5).all() and (got[0][33:] == 5).all()


def test_append_slot_past_the_cache_is_reported_and_skipped():
    c = _append_case(7, [0], [20], 16, 16, 1, 1, 64)
    slots = c["slots"].clone()
    c["slots"][19] = c["k_cache"].shape[0] * 16
    with pytest.raises(attn.AttnError) as e:
        _append(c)
    assert e.value.status == attn.ATTN_ERR_DEVICE_DATA
    c["slots"] = slots
    _check_append(c, _append(c))


def test_append_views_of_a_projection_and_in_place():
    c = _append_case(8, [0, 30], [17, 20], 16, 16, 6, 2, 128, rot=128)
    T = 37
    qkv = torch.cat([c["q"], c["k"], c["v"]], 1).to(DEV)
    q, k, v = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:]
    cache = [c[n].to(DEV) for n in ("k_cache", "v_cache", "k_scale", "v_scale")]
    out = attn.paged_append_fp8(q, k, v, *cache, c["slots"].to(DEV), c["pos"].to(DEV), c["freq"].to(DEV), q_out=q)
    attn.device_status()
    assert out.data_ptr() == qkv.data_ptr() and q.shape == (T, 6, 128)
    _check_append(c, [out.cpu().contiguous()] + [x.cpu() for x in cache])


def test_append_broadcast_k():
    c = _append_case(9, [0], [12], 16, 4, 0, 3, 64)
    one = c["k"][:1, :1].clone()
    c["k"] = one.expand(12, 3, 64)
    g = dict(c, k=None)
    cache = [c[n].to(DEV) for n in ("k_cache", "v_cache", "k_scale", "v_scale")]
    attn.paged_append_fp8(None, one.to(DEV).expand(12, 3, 64), c["v"].to(DEV), *cache, c["slots"].to(DEV))
    attn.device_status()
    assert g["k"] is None
    _check_append(c, [None] + [x.cpu() for x in cache])


def test_append_scales_of_another_writer():
    """Scales that are no powers of two: kept where they are large enough, and codes divided by them."""
    c = _append_case(10, [3, 5], [2, 3], 16, 8, 0, 2, 64)
    c["k_scale"] = c["k_scale"] * 0 + 0.3
    c["v_scale"] = c["v_scale"] * 0 + 0.001
    q, kc, vc, ks, vs = _append(c)
    codes, scale = c["k_cache"].double(), c["k_scale"].double()
    ref.append(c["k"].double(), codes, scale, c["slots"].tolist(), 8)
    assert torch.equal(ks.double(), scale)
    valid = _valid(c, codes.shape)
    # a quotient in 32 bits next to a border between two codes: an e4m3 step, which is at most an eighth, or 2^-9
    d = torch.where(valid, (kc.double() - codes).abs() - 0.125 * codes.abs() - 2.0 ** -9, -1.0)
    assert (d <= 0).all() and (torch.where(valid, kc.double() != codes, False)).sum() <= codes.numel() // 1000
    before = c["v_scale"].double()[0, 0, 0].item()
    grew = vs.double() != before
    assert grew.any()  # a larger one is needed: a power of two takes its place
    assert torch.equal(torch.exp2(torch.round(torch.log2(vs.double()[grew]))), vs.double()[grew])


# ---------------------------------------------------------------- reading back

def _read_case(seed, lens, page, block, H_kv, d, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pool = sum(need) + 2
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32)
    at = 0
    for r, k in enumerate(need):
        table[r, :k] = perm[at:at + k]
        at += k
    c = dict(page=page, block=block, table=table, lens=list(lens))
    (c["k_cache"], c["k_scale"]), (c["v_cache"], c["v_scale"]) = (_random_cache(g, pool, page, block, H_kv, d, spread) for _ in "kv")
    return c, g


def _gpu_cache(c):
    return [c[n].to(DEV) for n in ("k_cache", "v_cache", "k_scale", "v_scale")]


@pytest.mark.parametrize("page,block", [(8, 1), (16, 16), (64, 8), (128, 128), (1024, 512)])
@pytest.mark.parametrize("H_kv,d", [(1, 64), (3, 128), (8, 64)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_read(page, block, H_kv, d, dtype):
    lens = [0, 1, page, page + 3, 0, 133, 7]
    c, _ = _read_case(page + H_kv, lens, page, block, H_kv, d)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
    total = int(cu[-1]) + 5
    k, v = (torch.full((total, H_kv, d), 3.0, dtype=dtype, device=DEV) for _ in "kv")
    out = attn.paged_read_fp8(*_gpu_cache(c), c["table"].to(DEV), cu.to(DEV), total, k_out=k, v_out=v)
    attn.device_status()
    assert out[0] is k and out[1] is v
    for got, name in ((k, "k"), (v, "v")):
        want = torch.cat([ref.values(c[name + "_cache"], c[name + "_scale"], c["table"][r], n) for r, n in enumerate(lens)])
        assert torch.equal(got.cpu()[:total - 5].double(), want)  # powers of two: exact in either type
        assert (got[total - 5:] == 3).all()


def test_read_other_scales_round_once():
    c, g = _read_case(1, [100], 16, 4, 2, 64)
    c["k_scale"] = torch.rand(c["k_scale"].shape, generator=g) + 0.01
    cu = torch.tensor([0, 100], dtype=torch.int32, device=DEV)
    k, _ = attn.paged_read_fp8(*_gpu_cache(c), c["table"].to(DEV), cu, 100)
    k32, _ = attn.paged_read_fp8(*_gpu_cache(c), c["table"].to(DEV), cu, 100, dtype=torch.float32)
    want = ref.values(c["k_cache"], c["k_scale"], c["table"][0], 100)
    assert torch.equal(k32.cpu().double(), want.float().double())
    assert torch.equal(k.cpu(), k32.cpu().to(BF))


def test_read_bad_device_data_is_reported():
    c, _ = _read_case(2, [20, 20], 16, 16, 1, 64)
    cache, total = _gpu_cache(c), 40
    for cu, table in (([0, 20, 41], c["table"]), ([0, 30, 20], c["table"]), ([-1, 20, 40], c["table"]),
                      ([0, 20, 40], torch.full_like(c["table"], 1 << 20))):
        attn.paged_read_fp8(*cache, table.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV), total)
        with pytest.raises(attn.AttnError) as e:
            attn.device_status()
        assert e.value.status == attn.ATTN_ERR_DEVICE_DATA


# ---------------------------------------------------------------- attention

def _fwd_case(seed, lens, q_lens, H, H_kv, d, page, block, q_size=1.0, spread=0.5, pad=0):
    c, g = _read_case(seed, lens, page, block, H_kv, d, spread)
    c["k_scale"] /= 60
    used = set()
    for r, n in enumerate(lens):  # what lies behind the last key, and in no page, is not read
        ids = [int(i) for i in c["table"][r, :-(-n // page)]]
        used |= set(ids)
        if n % page:
            for name in ("k", "v"):
                _bits(c[name + "_cache"])[ids[-1], n % page:] = 0x7f
                c[name + "_scale"][ids[-1], :, (n % page + block - 1) // block:] = float("nan")
    for i in set(range(c["k_cache"].shape[0])) - used:
        for name in ("k", "v"):
            c[name + "_cache"].view(torch.uint8)[i] = 0xff
            c[name + "_scale"][i] = float("nan")
    c["cu"] = None if q_lens is None else torch.tensor([0] + q_lens).cumsum(0).tolist()
    T = len(lens) if q_lens is None else c["cu"][-1]
    c["q"] = (torch.randn((T + pad, H, d), generator=g) * q_size).to(BF)
    c["T"] = T
    return c


def _fwd(c, causal, scale=None, **kw):
    dev = lambda x, dt=torch.int32: None if x is None else torch.tensor(x, dtype=dt, device=DEV)
    q = c["q"].to(DEV)
    out = torch.full(q.shape, 9.0, dtype=BF, device=DEV)
    lse = torch.full(q.shape[:2], 9.0, device=DEV)
    max_q = 1 if c["cu"] is None else max(1, max(b - a for a, b in zip(c["cu"], c["cu"][1:])))
    o, l = attn.paged_fwd_fp8(q, *_gpu_cache(c), c["table"].to(DEV), dev(c["lens"]), cu_seqlens_q=dev(c["cu"]), max_q_len=max_q,
                              causal=causal, scale=scale, out=out, lse=lse, **kw)
    attn.device_status()
    assert o is out and l is lse
    return o.cpu(), l.cpu()


def _check_fwd(c, causal, got, scale=None):
    o, lse = got
    T = c["T"]
    scale = scale or 1.0 / math.sqrt(c["q"].shape[2])
    wo, wl, bo, bl = ref.attend(c["q"][:T], c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], c["table"], c["lens"], c["cu"],
                                scale, causal)
    empty = torch.isinf(wl)
    assert torch.equal(lse[:T][empty].double(), wl[empty]) and (o[:T][empty] == 0).all()
    e = (o[:T].double() - wo).abs()
    assert (e <= bo).all(), ("o", (e / bo).max(), e.max())
    e = torch.where(empty, 0.0, (lse[:T].double() - wl).abs())
    assert (e <= torch.where(empty, 1.0, bl)).all(), ("lse", (e / bl).max(), e.max())
    assert (o[T:] == 9).all() and (lse[T:] == 9).all()  # rows behind the last request


@pytest.mark.parametrize("H,H_kv", [(1, 1), (4, 1), (8, 2), (10, 2), (16, 1), (48, 3), (128, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_fwd_groups(H, H_kv, d):
    c = _fwd_case(H + d, [1, 127, 128, 129, 700], None, H, H_kv, d, 16, 16)
    _check_fwd(c, True, _fwd(c, True))


@pytest.mark.parametrize("page,block", [(8, 1), (8, 8), (16, 4), (32, 32), (64, 1), (64, 64), (128, 16), (256, 256), (1024, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_fwd_pages_and_blocks(page, block, d):
    c = _fwd_case(page + block + d, [5, page, 1023, 0, 300], None, 8, 2, d, page, block)
    _check_fwd(c, True, _fwd(c, True))


@pytest.mark.parametrize("n", [0, 1, 2, 31, 32, 33, 127, 128, 129, 511, 512, 513, 1024, 1025, 5000])
def test_fwd_lengths(n):
    c = _fwd_case(n, [n], None, 8, 1, 128, 16, 16)
    _check_fwd(c, True, _fwd(c, True))
    c = _fwd_case(n + 1, [n], None, 12, 1, 64, 64, 32)
    _check_fwd(c, False, _fwd(c, False))


@pytest.mark.parametrize("q_lens", [[1, 2, 3, 4], [8, 1, 0, 5], [33, 2, 17, 1], [130, 4, 1, 9]])
@pytest.mark.parametrize("H,H_kv,d", [(4, 1, 128), (8, 8, 64), (6, 2, 128), (40, 1, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_fwd_several_tokens(q_lens, H, H_kv, d, causal):
    c = _fwd_case(sum(q_lens) + H, [max(n, 3 * n - 3) + 130 * (i == 1) for i, n in enumerate(q_lens)], q_lens, H, H_kv, d, 16, 8,
                  pad=3)
    _check_fwd(c, causal, _fwd(c, causal))


def test_fwd_more_tokens_than_keys():
    """Query tokens before the first key see nothing: O = 0, LSE = -inf; the others their keys."""
    c = _fwd_case(12, [3, 0, 130], [7, 4, 2], 4, 2, 64, 16, 16)
    _check_fwd(c, True, _fwd(c, True))
    _check_fwd(c, False, _fwd(c, False))


def test_fwd_long_and_many():
    c = _fwd_case(13, [40000, 3, 9000], None, 4, 1, 128, 64, 64)
    _check_fwd(c, True, _fwd(c, True))
    g = torch.Generator().manual_seed(14)
    c = _fwd_case(15, torch.randint(0, 400, (700,), generator=g).tolist(), None, 2, 1, 64, 16, 16)
    _check_fwd(c, True, _fwd(c, True))


@pytest.mark.parametrize("q_size,scale", [(0.0, None), (1e-30, None), (30.0, 0.3), (1e30, 1e-31)])
def test_fwd_sizes_of_queries(q_size, scale):
    c = _fwd_case(16, [300, 900], None, 8, 2, 128, 16, 16, q_size=q_size)
    _check_fwd(c, True, _fwd(c, True, scale), scale)


def test_fwd_scores_that_grow_and_scales_that_differ():
    """The running maximum rises again and again, and the values' scales span 2^40."""
    c = _fwd_case(17, [3000], None, 4, 1, 64, 16, 1)
    n = c["k_scale"].shape[0]
    order = c["table"][0, :-(-3000 // 16)].long()
    ramp = torch.linspace(0.02, 2.0, order.numel())
    c["k_scale"][order] = (ramp[:, None, None] * torch.ones(order.numel(), 1, 16)) / 60
    c["v_scale"][order] = torch.exp2(torch.randint(-20, 20, (order.numel(), 1, 16), generator=torch.Generator().manual_seed(2)).float())
    assert n >= order.numel()
    _check_fwd(c, True, _fwd(c, True))


def test_fwd_a_nan_among_the_scores_and_among_the_values():
    c = _fwd_case(18, [200, 200, 200], None, 4, 2, 64, 16, 16)
    page = lambda r, key: int(c["table"][r, key // 16])
    _bits(c["k_cache"])[page(0, 70), 70 % 16, 1, 5] = 0x7f
    _bits(c["v_cache"])[page(1, 190), 190 % 16, 0, 9] = 0xff
    o, lse = _fwd(c, True)
    assert torch.isnan(o[0, 2:]).all() and torch.isnan(lse[0, 2:]).all()
    assert torch.isnan(o[1, :2, 9]).all()
    for t, heads in ((0, slice(0, 2)), (1, slice(2, 4)), (2, slice(0, 4))):
        assert torch.isfinite(o[t, heads].float()).all() and torch.isfinite(lse[t, heads]).all()


def test_fwd_agrees_with_the_bf16_cache():
    """The same values in a bf16 cache and in codes."""
    c = _fwd_case(19, [700, 130, 64, 1], None, 16, 4, 128, 64, 64)
    k16, v16 = ((c[n + "_cache"].float() * c[n + "_scale"].transpose(1, 2).repeat_interleave(64, 1)[..., None]).nan_to_num(0.0).to(BF).to(DEV)
                for n in "kv")
    lens = torch.tensor(c["lens"], dtype=torch.int32, device=DEV)
    o16, l16 = attn.paged_fwd(c["q"].to(DEV), k16, v16, c["table"].to(DEV), lens)
    o, lse = _fwd(c, True)
    attn.device_status()
    _check_fwd(c, True, (o, lse))
    # The bf16 cache holds the values rounded (half a step, 2^-8, since these scales are no powers of two): a score moves
    # by at most off = scale 2^-8 sum |q k|, so each probability by a factor between e^(-2 off) and e^(2 off), the LSE by
    # off; the values and that kernel's probabilities are rounded by 2^-8 each, O by 2^-8.
    wo, wl, bo, bl = ref.attend(c["q"], c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], c["table"], c["lens"], None,
                                128 ** -0.5, True)
    for r, n in enumerate(c["lens"]):
        k, v = (ref.values(c[x + "_cache"], c[x + "_scale"], c["table"][r], n) for x in "kv")
        for h in range(16):
            x, y = k[:, h // 4], v[:, h // 4]
            off = 128 ** -0.5 * 2.0 ** -8 * (x.abs() @ c["q"][r, h].double().abs()).max()
            spread = torch.softmax(128 ** -0.5 * (x @ c["q"][r, h].double()), 0) @ y.abs()
            near = bo[r, h] + (torch.expm1(2 * off) + 2 * 2.0 ** -8) * 1.01 * torch.exp(2 * off) * spread + 2.0 ** -8 * wo[r, h].abs()
            assert ((o16[r, h].cpu().double() - wo[r, h]).abs() <= near).all()
            assert (l16[r, h].cpu().double() - wl[r, h]).abs() <= bl[r, h] + off


def test_fwd_bad_device_data_is_reported():
    c = _fwd_case(20, [100, 200], [2, 2], 4, 2, 64, 16, 16)
    cache, q = _gpu_cache(c), c["q"].to(DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    good = dict(table=c["table"].to(DEV), lens=i32(100, 200), cu=i32(0, 2, 4))
    cap = c["table"].shape[1] * 16
    for bad in (dict(table=torch.full_like(good["table"], -5)), dict(table=torch.full_like(good["table"], 1 << 28)),
                dict(lens=i32(-3, 200)), dict(lens=i32(100, cap + 1)), dict(cu=i32(0, 3, 2)), dict(cu=i32(0, 2, 5)),
                dict(cu=i32(-1, 2, 4)), dict(cu=i32(0, 0, 4))):
        a = dict(good, **bad)
        attn.paged_fwd_fp8(q, *cache, a["table"], a["lens"], cu_seqlens_q=a["cu"], max_q_len=2, causal=True)
        with pytest.raises(attn.AttnError) as e:
            attn.device_status()
        assert e.value.status == attn.ATTN_ERR_DEVICE_DATA


# ---------------------------------------------------------------- together

def test_serving_steps():
    """A prompt through plan, append and read, then decode steps: each step's attention against that over the cache it
    left, and the cache against the tokens that went in."""
    B, H, H_kv, d, page, block = 3, 8, 2, 64, 16, 16
    g = torch.Generator().manual_seed(21)
    prompt, steps = [37, 5, 64], 6
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    pool = 24
    codes = torch.zeros((pool, page, H_kv, d), dtype=F8, device=DEV)
    cache = [codes, codes.clone(), torch.zeros((pool, H_kv, page // block), device=DEV), torch.zeros((pool, H_kv, page // block), device=DEV)]
    table = torch.full((B, 8), -1, dtype=torch.int32, device=DEV)
    free, count, ctx = torch.randperm(pool, generator=g).to(torch.int32).to(DEV), i32([pool]), i32([0] * B)
    freq, _ = attn.rope_inv_freq(d)
    freq = freq.to(DEV)
    raw = [[] for _ in range(B)]
    for step in range(steps + 1):
        new = prompt if step == 0 else [1] * B
        T = sum(new)
        cu, ctx, pos, slots, count = attn.paged_plan(ctx, table, free, count, page, pool, T, new_lens=i32(new))
        q, k, v = (torch.randn((T, h, d), generator=g).to(BF).to(DEV) for h in (H, H_kv, H_kv))
        q = attn.paged_append_fp8(q, k, v, *cache, slots, pos, freq)
        o, lse = attn.paged_fwd_fp8(q, *cache, table, ctx, cu_seqlens_q=cu, max_q_len=max(new), causal=True)
        c = dict(q=q.cpu(), k_cache=cache[0].cpu(), v_cache=cache[1].cpu(), k_scale=cache[2].cpu(), v_scale=cache[3].cpu(),
                 table=table.cpu(), lens=ctx.tolist(), cu=cu.tolist(), T=T)
        attn.device_status()
        _check_fwd(c, True, (o.cpu(), lse.cpu()))
        at = 0
        for r, n in enumerate(new):
            raw[r].append(v[at:at + n].cpu().double())
            at += n
    lens = ctx.tolist()
    cu_k = i32([0] + torch.tensor(lens).cumsum(0).tolist())
    kk, vv = attn.paged_read_fp8(*cache, table, cu_k, sum(lens))
    attn.device_status()
    at = 0
    for r, n in enumerate(lens):
        x, y = torch.cat(raw[r]), vv[at:at + n].cpu().double()
        # an e4m3 rounding is 2^-4 of the value, or half of 2^-9 of the scale (at most 2^-7 of the largest over 448);
        # a code may have been rounded again, each time that its block's scale grew, by half a subnormal step
        top = x.abs().amax((0, 2), keepdim=True)
        assert ((y - x).abs() <= 2.0 ** -4 * x.abs() + 20 * 2.0 ** -10 * top / 224).all()
        at += n
    # attention of every token by the packed values, which are the cache's own: scales are powers of two
    q = torch.randn((sum(lens), H, d), generator=g).to(BF).to(DEV)
    o1, l1 = attn.varlen_fwd(q, kk, vv, cu_k, cu_k, max_q_len=max(lens), max_k_len=max(lens), causal=True)
    attn.device_status()
    wo, wl, bo, bl = ref.attend(q.cpu(), cache[0].cpu(), cache[1].cpu(), cache[2].cpu(), cache[3].cpu(), table.cpu(), lens,
                                cu_k.tolist(), d ** -0.5, True)
    at = 0
    for n in lens:
        # beside the bounds of _kv8_ref.attend: probabilities in bf16, 2^-8 of their sum over the values' magnitudes,
        # which is at most the largest of them
        top = vv[at:at + n].cpu().double().abs().amax(0).repeat_interleave(H // H_kv, 0)
        assert ((o1[at:at + n].cpu().double() - wo[at:at + n]).abs() <= bo[at:at + n] + 2.0 ** -8 * top).all()
        at += n
    assert ((l1.cpu().double() - wl).abs() <= bl).all()
