"""Attention over the 8-bit cache where one key outweighs a long tail of small ones and its value is zero (an
attention sink): O is the tail's alone, so whatever of a small probability is lost shows in full.

K has one channel that is not zero, so that the scores are exact but for their roundings in 32 bits; the tail's
values have one sign, so that errors are relative to O itself.  Requests are more than the CTAs and share their pages:
each lies in one CTA or two, under one running maximum."""
import math

import pytest
import torch

import attention_attn_fwd_03_gb300 as attn

from test_gpu_kv8 import BF, DEV, F8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.lib()


def _case(n, bits, H, H_kv, d, q_len, B, page=64, block=16):
    """The last q_len tokens of B requests of the same n keys, whose first third ends with a key 2^bits (2^(0.75 bits)
    for some heads) above the others."""
    g = torch.Generator().manual_seed(n + H + d)
    pages = -(-n // page)
    c = dict(page=page, lens=[n] * B, scale=bits * math.log(2) / 16)
    k, v = torch.zeros((pages * page, H_kv, d)), torch.zeros((pages * page, H_kv, d))
    k[:, :, 0] = -8 + 0.5 * (torch.arange(pages * page) % 4)[:, None]
    k[n // 3, :, 0] = 8
    v[:] = torch.randint(64, 449, v.shape, generator=g)
    v[n // 3] = 0
    order = torch.randperm(pages, generator=g)
    c["table"] = torch.argsort(order).to(torch.int32).repeat(B, 1)
    for name, x in (("k", k), ("v", v)):
        c[name + "_cache"] = x.view(pages, page, H_kv, d)[order].to(F8)
        c[name + "_scale"] = torch.ones((pages, H_kv, page // block))
    c["k"], c["v"] = k.double()[:n], v.to(F8).double()[:n]
    c["q"] = torch.randn((q_len, H, d), generator=g).to(BF)
    c["q"][:, :, 0] = 1 - 0.125 * (torch.arange(H) % 3)
    return c


def _run(c):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    T, B = c["q"].shape[0], len(c["lens"])
    cache = [c[x].to(DEV) for x in ("k_cache", "v_cache", "k_scale", "v_scale")]
    o, lse = attn.paged_fwd_fp8(c["q"].repeat(B, 1, 1).to(DEV), *cache, c["table"].to(DEV), i32(c["lens"]),
                                cu_seqlens_q=i32(list(range(0, T * B + 1, T))), max_q_len=T, causal=True, scale=c["scale"])
    attn.device_status()
    return o.cpu().double().unflatten(0, (B, T)), lse.cpu().double().unflatten(0, (B, T))


def _check(c, got):
    """A probability enters O as an fp16 number (half a step, 2^-11, relative), cut into four e5m2 numbers of 3 bits,
    the last two 64 times as large: 12 bits, but for half their smallest step, 2^-16 / 64; with fp16's own, 2^-25, and
    the row's largest at 2^11 at least that is less than 2^-33 of the largest.  Four
    instructions of 32 keys to a tile add in 32 bits, truncating: n / 32 times 2^-23.  A score's factor, its product with it
    and the base-2 exponent are three roundings of half a step, 2^-24, doubled for the largest's own, relative to scores of at most `size`
    on either side: less than 2^-21 size.  Exponentials, sums, the factors at the end: 2^-18.  O in bf16: 2^-8."""
    o, lse = got
    n = c["lens"][0]
    T, H, d = c["q"].shape
    G = H // c["k"].shape[1]
    for t in range(T):
        seen = n - T + 1 + t
        for h in range(H):
            x = c["q"][t, h, 0].double() * c["scale"]
            s = c["k"][:seen, h // G, 0] * x
            p, v = torch.exp(s - s.max()), c["v"][:seen, h // G]
            want = (p @ v) / p.sum()
            off = 2.0 ** -21 * float(s.abs().max()) + 2.0 ** -18
            bound = want * (2.0 ** -8 + 2.0 ** -11 + n / 32 * 2.0 ** -23 + 2 * off) * 1.01 + 2.0 ** -33 * v.sum(0) / p.sum()
            e = (o[:, t, h] - want).abs()
            assert (e <= bound).all(), (t, h, float((e / want).max()), float((bound / want).max()))
            ll = s.max() + torch.log(p.sum())
            assert ((lse[:, t, h] - ll).abs() <= off + 2.0 ** -18 * (1 + ll.abs())).all()


# (heads, KV heads, head dim, tokens): 8, 16 and 32 rows to a unit of one KV head, then of two
FORMS = [(1, 1, 128, 1), (8, 1, 64, 1), (12, 1, 128, 1), (4, 1, 64, 3), (20, 1, 128, 1), (8, 1, 64, 4), (16, 2, 128, 1),
         (16, 2, 64, 1), (32, 2, 128, 1), (8, 2, 128, 3), (32, 2, 64, 1), (8, 2, 64, 5)]


@pytest.mark.parametrize("H,H_kv,d,q_len", FORMS)
@pytest.mark.parametrize("bits", [12.3, 16.9, 20.6, 24.1, 27.7])
def test_tail_under_one_large_key(H, H_kv, d, q_len, bits):
    c = _case(20011, bits, H, H_kv, d, q_len, 640 // H_kv)
    _check(c, _run(c))


@pytest.mark.parametrize("d", [64, 128])
def test_long_tail_under_one_large_key(d):
    """262 thousand keys, each 2^-24.1 of one: 1.5% of the sum, and all of O."""
    c = _case(262144, 24.1, 4, 2, d, 1, 320)
    _check(c, _run(c))


@pytest.mark.parametrize("H,H_kv,d,q_len", FORMS)
@pytest.mark.parametrize("bits,up,down", [(60.4, 50, -40), (113.7, 62, -62), (118.3, 62, -62), (124.6, 80, -50), (100.2, 100, 10),
                                          (20.5, 100, 100), (20.5, -126, -126)])
def test_small_probabilities_of_large_values(H, H_kv, d, q_len, bits, up, down):
    """The scales of the tail's values are 2^up, that of the large key's, which is not zero, 2^down: O is a sum of both, of any size.
    (Not up to 2^120: codes above 255 are no 32-bit numbers there, and O is a sum in 32 bits before it is divided.)"""
    c = _case(1111, bits, H, H_kv, d, q_len, 640 // H_kv, block=1)
    c["q"][:, :, 0] = 1.0
    n, page = 1111, c["page"]
    c["v"][n // 3] = 300.0
    c["v"] = c["v"].to(F8).double()
    i = int(c["table"][0, n // 3 // page])
    c["v_scale"][:] = 2.0 ** up
    c["v_scale"][i, :, n // 3 % page] = 2.0 ** down
    keys = c["k_cache"].float()  # one size of the tail's probabilities
    keys[:, :, :, 0] = torch.where(keys[:, :, :, 0] < 0, -8.0, keys[:, :, :, 0])
    c["k_cache"] = keys.to(F8)
    c["k"] = torch.where(c["k"] < 0, -8.0, c["k"])
    codes = c["v_cache"].float()
    codes[i, n // 3 % page] = 300.0
    c["v_cache"] = codes.to(F8)
    w = torch.full((n, 1), 2.0 ** up, dtype=torch.float64)
    w[n // 3] = 2.0 ** down
    o, lse = _run(c)
    # as in _check, but that the row's largest is that of probability times scale, and that bf16's steps do not get smaller than
    # 2^-133; scales below 2^-112 leave 2^-19 of the largest
    floor = 2.0 ** (-19 if max(up, down) < -112 else -33)
    G = H // H_kv
    for t in range(q_len):
        seen = n - q_len + 1 + t
        for h in range(H):
            s = c["k"][:seen, h // G, 0] * c["scale"]
            p, v = torch.exp(s - s.max())[:, None] * w[:seen], c["v"][:seen, h // G]
            total = torch.exp(s - s.max()).sum()
            want = (p * v).sum(0) / total
            off = 2.0 ** -21 * float(s.abs().max()) + 2.0 ** -18
            bound = want * (2.0 ** -8 + 2.0 ** -11 + n / 32 * 2.0 ** -23 + 2 * off) * 1.01 + floor * p.max() * v.sum(0) / total + 2.0 ** -134
            e = (o[:, t, h] - want).abs()
            assert (e <= bound).all(), (t, h, float((e / want).max()), float((bound / want).max()))
