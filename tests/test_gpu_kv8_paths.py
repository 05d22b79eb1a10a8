"""Attention over the 8-bit cache where its work is cut in other ways (units of two KV heads, many steps to a CTA, many
units to a CTA), and all three operators under capture, on side streams, in large caches and with what a launch must
leave alone.  Bounds: _kv8_ref.attend, as in test_gpu_kv8.py; runs of the same call are compared for equality."""
import os
import random
import subprocess
import sys

import pytest
import torch

import attention_attn_fwd_03_gb300 as attn

import _kv8_ref as ref
from test_gpu_kv8 import BF, DEV, F8, _append, _append_case, _bits, _check_append, _check_fwd, _fwd, _fwd_case, _gpu_cache

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.lib()


def _long_table(c, H_kv):
    """The case with a table of so many columns that its units take two KV heads each, where those are even."""
    B, cols = c["table"].shape
    more = 128 * 40 * 304 // (B * H_kv * c["page"]) + 1
    c["table"] = torch.cat([c["table"], torch.full((B, more), -1, dtype=torch.int32)], 1)
    return c


def _crowd(lens, q_lens, H_kv):
    """Requests (these over and over) that make more units than there are CTAs: two KV heads to a unit."""
    times = -(-(304 // H_kv + 1) // len(lens))
    return lens * times, None if q_lens is None else q_lens * times


def _check_some(c, causal, got, n=30):
    """_check_fwd for the first, last and longest requests and n others, drawn; the rest have to be finite."""
    B, T, (o, lse) = len(c["lens"]), c["T"], got
    cu = c["cu"] or list(range(B + 1))
    pick = sorted({0, B - 1, c["lens"].index(max(c["lens"]))} | set(random.Random(B).sample(range(B), min(n, B))))
    rows = torch.cat([torch.arange(cu[r], cu[r + 1]) for r in pick])
    part = dict(c, table=c["table"][pick], lens=[c["lens"][r] for r in pick], q=c["q"][rows], T=len(rows),
                cu=None if c["cu"] is None else [0] + torch.tensor([cu[r + 1] - cu[r] for r in pick]).cumsum(0).tolist())
    _check_fwd(part, causal, (o[rows], lse[rows]))
    assert torch.isfinite(o[:T].float()).all() and not torch.isnan(lse[:T]).any() and (o[T:] == 9).all() and (lse[T:] == 9).all()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- two KV heads to a unit

@pytest.mark.parametrize("H,H_kv", [(2, 2), (8, 2), (16, 4), (20, 2), (32, 2), (66, 6), (128, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [1, 16])
def test_pairs_groups(H, H_kv, d, block):
    c = _long_table(_fwd_case(H + d + block, [1, 127, 128, 0, 129, 300, 2000], None, H, H_kv, d, 16, block), H_kv)
    _check_fwd(c, True, _fwd(c, True))


@pytest.mark.parametrize("page,block", [(8, 8), (16, 4), (32, 1), (64, 64), (128, 16), (256, 256), (1024, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_pairs_pages_and_blocks(page, block, d):
    c = _long_table(_fwd_case(page + block + d, [5, page, 1023, 0, 300, 2 * page + 1], None, 16, 4, d, page, block), 4)
    _check_fwd(c, False, _fwd(c, False))


@pytest.mark.parametrize("q_lens", [[1, 2, 3, 4], [8, 1, 0, 5], [33, 2, 17, 1]])
@pytest.mark.parametrize("H,H_kv,d", [(4, 2, 128), (8, 8, 64), (6, 2, 128), (20, 2, 64), (16, 4, 64), (16, 4, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_pairs_several_tokens(q_lens, H, H_kv, d, causal):
    c = _fwd_case(sum(q_lens) + H, [max(n, 3 * n - 3) + 130 * (i == 1) + 700 * (i == 2) for i, n in enumerate(q_lens)], q_lens,
                  H, H_kv, d, 16, 8, pad=3)
    _check_fwd(c, causal, _fwd(_long_table(c, H_kv), causal))


@pytest.mark.parametrize("H_kv", [2, 3])
@pytest.mark.parametrize("d", [64, 128])
def test_many_requests(H_kv, d):
    """More units than CTAs, of no keys to several steps: pairs of heads (H_kv even) without a long table."""
    g = torch.Generator().manual_seed(d + H_kv)
    lens = torch.randint(0, 700, (320,), generator=g).tolist()
    c = _fwd_case(d, lens, None, 2 * H_kv, H_kv, d, 32, 8)
    _check_fwd(c, True, _fwd(c, True))


# ---------------------------------------------------------------- many steps to a CTA

@pytest.mark.parametrize("H,H_kv,q_len", [(2, 1, 1), (2, 2, 1), (10, 1, 1), (3, 1, 9), (4, 2, 3), (8, 2, 9)])
@pytest.mark.parametrize("d", [64, 128])
def test_long(H, H_kv, q_len, d):
    """Keys enough for each CTA to take a dozen steps or more, whatever form runs."""
    lens = [200000, 70001, 130, 90000]
    q_lens = None if q_len == 1 else [q_len, 1, q_len, 2]
    c = _fwd_case(H + d, lens, q_lens, H, H_kv, d, 64, 16)
    _check_fwd(c, True, _fwd(c, True))


def test_rows_of_many_tiles_each_cut_many_times():
    """Few units, each in the hands of many CTAs; and one CTA's piece of one tile."""
    for d, n in ((64, 40000), (128, 38913), (64, 130), (128, 257)):
        for H, H_kv in ((1, 1), (16, 2)):
            c = _fwd_case(n, [n], None, H, H_kv, d, 128, 128)
            _check_fwd(c, True, _fwd(c, True))
            _check_fwd(c, True, _fwd(_long_table(c, H_kv), True))


@pytest.mark.parametrize("seed", range(24))
def test_drawn(seed):
    r = random.Random(seed)
    B, H_kv = r.randint(1, 12), r.choice((1, 2, 3, 4, 8))
    G, d = r.choice((1, 2, 3, 4, 7, 8, 12)), r.choice((64, 128))
    page = 1 << r.randint(3, 10)
    block = 1 << r.randint(0, page.bit_length() - 1)
    q_lens = None if r.random() < 0.4 else [r.randint(0, 9) for _ in range(B)]
    if q_lens is not None and sum(q_lens) == 0:
        q_lens[0] = 1
    lens = [r.choice((0, 1, r.randint(2, 200), r.randint(200, 3000))) for _ in range(B)]
    c = _fwd_case(seed, lens, q_lens, G * H_kv, H_kv, d, page, block, pad=r.randint(0, 3) if q_lens else 0)
    if r.random() < 0.6:
        _long_table(c, H_kv)
    causal = r.random() < 0.7
    _check_fwd(c, causal, _fwd(c, causal))


# ---------------------------------------------------------------- values

@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_of_keys_that_some_tokens_do_not_see(d, pairs):
    """A NaN among the values (scores) of a key reaches the tokens that see the key, in its channel (in all), and no other."""
    q_lens, lens = [5, 3], [300, 640]
    c = _fwd_case(31, lens, q_lens, 8, 4, d, 16, 4)
    if pairs:
        _long_table(c, 4)
    want_o, want_l = _fwd(c, True)
    at = lambda r, key: (int(c["table"][r, key // 16]), key % 16)
    hurt = torch.zeros(want_o.shape, dtype=torch.bool)
    hurt_l = torch.zeros(want_l.shape, dtype=torch.bool)
    before = {}
    for r, key, h, ch in ((0, 299, 0, 9), (0, 297, 3, d - 1), (0, 297, 3, 0), (1, 638, 2, 33), (1, 639, 1, 16)):
        p, row = at(r, key)
        before[p, row, h, ch] = int(_bits(c["v_cache"])[p, row, h, ch])
        c["v_cache"].view(torch.uint8)[p, row, h, ch] = 0xff if ch % 2 else 0x7f
        first = key - (lens[r] - q_lens[r])  # the first token that sees it
        hurt[sum(q_lens[:r]) + first:sum(q_lens[:r + 1]), 2 * h:2 * h + 2, ch] = True
    p, row = at(1, 637 + 1)
    c["k_cache"].view(torch.uint8)[p, row, 0, 7] = 0x7f
    hurt[6:8, 0:2] = True
    hurt_l[6:8, 0:2] = True
    o, lse = _fwd(c, True)
    assert torch.isnan(o[hurt].float()).all() and torch.isnan(lse[hurt_l]).all()
    assert torch.isfinite(o[~hurt].float()).all()
    assert torch.equal(lse[~hurt_l], want_l[~hurt_l])
    # where the token does not see the key, nothing has changed
    sees = hurt.any(2)
    assert torch.equal(o[~sees], want_o[~sees])


def test_not_finite_queries_stay_in_their_rows():
    for wide in (False, True):
        c = _fwd_case(32, [300, 500], None, 8, 2, 128, 16, 16)
        if wide:
            _long_table(c, 2)
        want_o, want_l = _fwd(c, True)
        c["q"][0, 1, 5] = float("nan")
        c["q"][1, 6, 0] = float("inf")
        o, lse = _fwd(c, True)
        for t, h in ((0, 1), (1, 6)):
            assert torch.isnan(o[t, h].float()).all() and torch.isnan(lse[t, h])
            o[t, h], lse[t, h] = want_o[t, h], want_l[t, h]
        assert torch.equal(o, want_o) and torch.equal(lse, want_l)


def test_scales_far_from_one():
    """Values' scales times 2^-100 or 2^90, and all at the smallest that an append writes: the result goes with them.
    Below 2^-120 P is up to 2^6 smaller, so that what it loses lies 2^-18 below the row's largest instead of 2^-24."""
    c = _fwd_case(33, [700, 40], None, 4, 2, 64, 16, 4)
    want, lse, bo, bl = ref.attend(c["q"], c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], c["table"], c["lens"], None, 0.125,
                                   True)
    had = c["v_scale"].clone()
    for e in (-100, 90):
        c["v_scale"] = had * 2.0 ** e
        o, l = _fwd(c, True)
        assert ((o.double() * 2.0 ** -e - want).abs() <= bo).all() and ((l.double() - lse).abs() <= bl).all()
    c["v_scale"] = torch.where(had.isnan(), had, 2.0 ** -126)
    one = torch.where(had.isnan(), had, 1.0)
    want, lse, bo, bl = ref.attend(c["q"], c["k_cache"], c["v_cache"], c["k_scale"], one, c["table"], c["lens"], None, 0.125, True)
    o, l = _fwd(c, True)
    # sum over the keys of 2^-18 of the largest probability, which is at most 1, times |code| <= 448; and bf16's smallest
    # steps, 2^-133, of numbers down to 2^-126
    slack = 2.0 ** -18 * 448 * 700 + 2.0 ** -7
    e = (o.double() * 2.0 ** 126 - want).abs()
    assert (e <= bo + slack).all() and ((l.double() - lse).abs() <= bl).all()


def test_scale_of_zero_reads_as_zero():
    c = _fwd_case(34, [200], None, 4, 2, 128, 16, 4)
    live = c["table"][0, :12].long()
    c["v_scale"][live[3:7]] = 0.0
    c["k_scale"][live[5:9], 1] = 0.0
    # the bound's floor divides by the scales: those of zero add nothing to it
    plain = dict(c, v_scale=torch.where(c["v_scale"] == 0, 1.0, c["v_scale"]), v_cache=c["v_cache"].clone())
    plain["v_cache"].view(torch.uint8)[live[3:7]] = 0
    wo, wl, bo, bl = ref.attend(c["q"], c["k_cache"], plain["v_cache"], c["k_scale"], plain["v_scale"], c["table"], c["lens"], None,
                                128 ** -0.5, True)
    o, lse = _fwd(c, True)
    assert ((o.double() - wo).abs() <= bo).all() and ((lse.double() - wl).abs() <= bl).all()


# ---------------------------------------------------------------- what a call may be given

def test_scales_and_tables_off_the_16_byte_grid():
    c = _fwd_case(35, [300, 77], None, 8, 2, 64, 16, 2)
    want = _fwd(c, True)
    cache = _gpu_cache(c)
    shift = lambda x, k: torch.cat([x.new_zeros(k), x.flatten()])[k:].view(x.shape)
    ks, vs = shift(cache[2], 1), shift(cache[3], 3)
    table, lens = shift(c["table"].to(DEV), 1), shift(_i32(c["lens"]), 3)
    assert ks.data_ptr() % 16 == 4 and vs.data_ptr() % 16 == 12
    q, cu = c["q"].to(DEV), _i32([0, 300, 377])
    o, lse = attn.paged_fwd_fp8(q, cache[0], cache[1], ks, vs, table, lens)
    assert torch.equal(o.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])
    k, v = attn.paged_read_fp8(cache[0], cache[1], ks, vs, table, cu, 377)
    k2, v2 = attn.paged_read_fp8(*cache, c["table"].to(DEV), cu, 377)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    a = _append_case(36, [5, 40], [20, 3], 16, 2, 4, 2, 64)
    t = lambda n: a[n].to(DEV).clone()
    out = []
    for place in (lambda x: x, lambda x: shift(x, 3)):
        cache = [t("k_cache"), t("v_cache"), place(t("k_scale")), place(t("v_scale"))]
        attn.paged_append_fp8(t("q"), t("k"), t("v"), *cache, place(t("slots")))
        out.append([_bits(x) for x in cache])
    attn.device_status()
    assert all(torch.equal(x, y) for x, y in zip(*out))


def test_helpers_refuse_what_does_not_fit():
    c = _fwd_case(37, [100, 50], None, 8, 2, 64, 16, 4)
    cache, q, table, lens = _gpu_cache(c), c["q"].to(DEV), c["table"].to(DEV), _i32(c["lens"])
    kc, vc, ks, vs = cache
    fwd = lambda *a, **kw: attn.paged_fwd_fp8(*a, **kw)
    good = (q, kc, vc, ks, vs, table, lens)
    def swap(i, x):
        return good[:i] + (x,) + good[i + 1:]
    for i, x, error in ((0, q.float(), TypeError), (0, q[:, :, :32].contiguous(), ValueError), (0, q[0], ValueError),
                        (0, q.transpose(0, 1), ValueError), (1, kc.view(torch.uint8), TypeError), (1, kc[:-1], ValueError),
                        (2, vc[:, :, :1].contiguous(), ValueError), (3, ks.double(), TypeError), (3, ks[:, :, :3].contiguous(), ValueError),
                        (4, vs[:, :1], ValueError), (4, vs.transpose(1, 2), ValueError), (5, table.long(), TypeError),
                        (5, table[0], ValueError), (6, lens[:1], ValueError), (6, lens.cpu(), TypeError)):
        with pytest.raises(error):
            fwd(*swap(i, x))
    with pytest.raises(attn.AttnError):
        fwd(*good, cu_seqlens_q=None, max_q_len=2)
    with pytest.raises(attn.AttnError):
        fwd(*good, scale=0.0)
    with pytest.raises(attn.AttnError):
        fwd(*good, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        fwd(*good, out=torch.empty_like(q)[:, :4])
    with pytest.raises(ValueError):
        attn.paged_read_fp8(*cache, table, _i32([0, 1, 2]), 0)
    with pytest.raises(ValueError):
        attn.paged_read_fp8(*cache, table, _i32([0, 1]), 2)
    with pytest.raises(TypeError):
        attn.paged_read_fp8(*cache, table, _i32([0, 1, 2]), 2, dtype=torch.float16)
    k = torch.zeros((4, 2, 64), dtype=BF, device=DEV)
    for a, kw, error in (((None, k, k, *cache, _i32([0, 1])), {}, ValueError), ((None, k, k[:, :1], *cache, _i32([0, 1, 2, 3])), {}, ValueError),
                         ((None, k, k, *cache, _i32([0, 1, 2, 3])), dict(positions=_i32([0] * 4)), ValueError),
                         ((None, k, k, *cache, _i32([0, 1, 2, 3])), dict(q_out=k), ValueError),
                         ((k[:, :, ::2], k, k, *cache, _i32([0, 1, 2, 3])), {}, ValueError),
                         ((k, k, k.half(), *cache, _i32([0, 1, 2, 3])), {}, TypeError)):
        with pytest.raises(error):
            attn.paged_append_fp8(*a, **kw)
    attn.device_status()


def test_workspace_of_the_exact_size_with_anything_in_it():
    for lens, q_lens, H, H_kv, d, long in (([30000, 5], None, 8, 2, 128, False), ([3000, 5, 900], [9, 1, 3], 8, 2, 64, True)):
        c = _fwd_case(38, lens, q_lens, H, H_kv, d, 16, 16)
        if long:
            _long_table(c, H_kv)
        want = _fwd(c, True)
        T, max_q = c["T"], 1 if q_lens is None else max(q_lens)
        n = attn.attn_paged_fwd_fp8_workspace_size(len(lens), T, max_q, H, H_kv, d, 16, c["table"].shape[1])
        for fill in (0xff, 0x00, 0x7f):
            room = torch.full((n + 4096,), fill, dtype=torch.uint8, device=DEV)
            got = _fwd(c, True, workspace=room[:n])
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert (room[n:] == fill).all()


def test_without_lse_and_with_outputs_given():
    c = _fwd_case(39, [3000, 5], None, 8, 2, 128, 16, 16)
    want, lse = _fwd(c, True)
    args = (c["q"].to(DEV), *_gpu_cache(c), c["table"].to(DEV), _i32(c["lens"]))
    o, none = attn.paged_fwd_fp8(*args, return_lse=False)
    assert none is None and torch.equal(o.cpu(), want)
    o, l = attn.paged_fwd_fp8(*args)
    assert torch.equal(o.cpu(), want) and torch.equal(l.cpu(), lse)


# ---------------------------------------------------------------- streams, graphs, large caches, failures

def test_two_streams_and_two_workspaces():
    cases = [_fwd_case(40 + i, lens, None, 8, 2, 128, 16, 16) for i, lens in enumerate(([20000, 300], [7000, 9000]))]
    want = [_fwd(c, True) for c in cases]
    args = [(c["q"].to(DEV), *_gpu_cache(c), c["table"].to(DEV), _i32(c["lens"])) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for a, s in zip(args, streams):
            got.append(attn.paged_fwd_fp8(*a, stream=s))
    torch.cuda.synchronize()
    attn.device_status()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o.cpu(), want[i % 2][0]) and torch.equal(l.cpu(), want[i % 2][1])


def test_captured_step_replayed_with_other_lengths():
    """Append and attention in one graph, the lengths, slots and rows changed between replays; two graphs share a workspace."""
    H, H_kv, d, page, block, B = 8, 2, 128, 16, 16, 3
    g = torch.Generator().manual_seed(42)
    pages = 64
    table = torch.randperm(pages * B, generator=g).view(B, pages).to(torch.int32).to(DEV)
    def fresh():
        return [torch.zeros((B * pages, page, H_kv, d), dtype=F8, device=DEV) for _ in "kv"] + \
               [torch.zeros((B * pages, H_kv, page // block), device=DEV) for _ in "kv"]
    cache, eager = fresh(), fresh()
    q, k, v = (torch.zeros((B, h, d), dtype=BF, device=DEV) for h in (H, H_kv, H_kv))
    slots, pos, lens = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(3))
    freq = attn.rope_inv_freq(d)[0].to(DEV)
    n = attn.attn_paged_fwd_fp8_workspace_size(B, B, 1, H, H_kv, d, page, pages)
    room = torch.empty(n, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            turned = attn.paged_append_fp8(q, k, v, *cache, slots, pos, freq)
            outs.append(attn.paged_fwd_fp8(turned, *cache, table, lens, workspace=room))
        graphs.append(graph)
    at = [0, 3, 900]
    for c in (cache, eager):  # something behind the longer contexts
        for x in c[:2]:
            x.copy_((torch.randn(x.shape, generator=torch.Generator().manual_seed(1)) * 50).clamp(-448, 448).to(F8).to(DEV))
        for x in c[2:]:
            x.fill_(0.25)
    for step in range(40):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g).to(BF))
        slots.copy_(_i32([int(table[r, p // page]) * page + p % page for r, p in enumerate(at)]))
        pos.copy_(_i32(at))
        at = [p + 1 for p in at]
        lens.copy_(_i32(at))
        graphs[step % 2].replay()
        turned = attn.paged_append_fp8(q, k, v, *eager, slots, pos, freq)
        o, l = attn.paged_fwd_fp8(turned, *eager, table, lens)
        attn.device_status()
        assert torch.equal(outs[step % 2][0], o) and torch.equal(outs[step % 2][1], l)
        assert all(torch.equal(_bits(x), _bits(y)) for x, y in zip(cache, eager))


PROGRAM = """
import sys, torch
import attention_attn_fwd_03_gb300 as attn
what, d = sys.argv[1], int(sys.argv[2])
DEV, F8 = "cuda", torch.float8_e4m3fn
cache = [torch.ones((600, 16, 2, d), device=DEV).to(F8) for _ in "kv"] + [torch.ones((600, 2, 4), device=DEV) for _ in "kv"]
table = torch.arange(600, dtype=torch.int32, device=DEV).view(2, 300)
lens = torch.tensor([4000, 77], dtype=torch.int32, device=DEV)
q, k, v = (torch.randn((2, h, d), device=DEV).bfloat16() for h in (8, 2, 2))
slots = torch.tensor([5, 4811], dtype=torch.int32, device=DEV)
cu = torch.tensor([0, 4000, 4077], dtype=torch.int32, device=DEV)
start = [x.clone() for x in cache]


def call():
    if what == "append":
        for x, y in zip(cache, start):
            x.copy_(y)
        return [attn.paged_append_fp8(q, k, v, *cache, slots)] + [x.clone() for x in cache]
    if what == "read":
        return attn.paged_read_fp8(*cache, table, cu, 4077)
    return attn.paged_fwd_fp8(q, *cache, table, lens)


torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
    got = call()
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in got]
want = call()
attn.device_status()
b = lambda x: x.contiguous().view(torch.uint8)
assert all(torch.equal(b(x), b(y)) for x, y in zip(got, want)), what
"""


@pytest.mark.parametrize("what,d", [("append", 64), ("append", 128), ("read", 64), ("fwd", 64), ("fwd", 128)])
def test_first_call_is_captured(what, d):
    r = subprocess.run([sys.executable, "-c", PROGRAM, what, str(d)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("H_kv,d", [(8, 128), (8, 64), (3, 64)])
def test_cache_past_32_bit_offsets(H_kv, d):
    """Pages beyond 4 GB of codes hold the same as pages of a small cache."""
    page, block, H = 64, 16, 2 * H_kv
    far = (1 << 32) // (page * H_kv * d) + 50
    ids = [far - 1, far - 30, far - 7, 3, far - 16]
    g = torch.Generator().manual_seed(43)
    small = [(torch.randn((5, page, H_kv, d), generator=g) * 60).clamp(-448, 448).to(F8).to(DEV) for _ in "kv"] + \
            [torch.exp2(torch.randint(-6, 3, (5, H_kv, page // block), generator=g).float()).to(DEV) for _ in "kv"]
    large = [torch.empty((far, page, H_kv, d), dtype=F8, device=DEV) for _ in "kv"] + \
            [torch.empty((far, H_kv, page // block), device=DEV) for _ in "kv"]
    for x, y in zip(large, small):
        for i, p in enumerate(ids):
            x[p] = y[i]
    n = 4 * page + 21
    q, k, v = (torch.randn((3, h, d), generator=g).to(BF).to(DEV) for h in (H, H_kv, H_kv))
    lens = _i32([n + 3])
    got = []
    for cache, table in ((small, list(range(5))), (large, ids)):
        slots = _i32([table[(n + i) // page] * page + (n + i) % page for i in range(3)])
        attn.paged_append_fp8(None, k, v, *cache, slots)
        table = _i32([table])
        o, lse = attn.paged_fwd_fp8(q, *cache, table, lens, cu_seqlens_q=_i32([0, 3]), max_q_len=3, causal=True)
        got.append([o, lse, *attn.paged_read_fp8(*cache, table, _i32([0, n + 3]), n + 3)])
    attn.device_status()
    for x, y in zip(*got):
        assert torch.equal(x, y)
    for x, y in zip(large, small):
        for i, p in enumerate(ids):
            assert torch.equal(_bits(x[p]), _bits(y[i]))


@pytest.mark.parametrize("pairs", [False, True])
def test_recorded_timeout_leaves_outputs_alone(pairs):
    c = _fwd_case(44, [30000, 40, 700], None, 8, 2, 128, 16, 16)
    if pairs:
        _long_table(c, 2)
    args = (c["q"].to(DEV), *_gpu_cache(c), c["table"].to(DEV), _i32(c["lens"]))
    want = attn.paged_fwd_fp8(*args)
    attn.device_status()
    o, l = torch.full_like(want[0], 3.0), torch.full_like(want[1], 3.0)
    assert attn.attn_selftest_wait_timeout(torch.cuda.current_stream().cuda_stream) == attn.ATTN_OK
    attn.paged_fwd_fp8(*args, out=o, lse=l)
    with pytest.raises(attn.AttnError) as e:
        attn.device_status()
    assert e.value.status == attn.ATTN_ERR_TIMEOUT
    assert bool((o == 3).all()) and bool((l == 3).all())
    attn.paged_fwd_fp8(*args, out=o, lse=l)
    attn.device_status()
    assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_the_same_call_gives_the_same_bits():
    for d, H_kv, long in ((64, 2, True), (128, 2, True), (128, 1, False)):
        c = _fwd_case(45, [9000, 300, 0, 4000], None, 4 * H_kv, H_kv, d, 16, 16)
        if long:
            _long_table(c, H_kv)
        first = _fwd(c, True)
        for _ in range(10):
            got = _fwd(c, True)
            assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


def test_bad_pages_of_some_requests_leave_the_others_right():
    """A page id out of range reads as keys of zeros and is reported; every other request is as it was."""
    for H_kv, long in ((2, True), (3, False)):
        c = _fwd_case(46, [900, 400, 3000], None, 2 * H_kv, H_kv, 64, 16, 16)
        if long:
            _long_table(c, H_kv)
        want_o, want_l = _fwd(c, True)
        bad = c["table"].clone()
        bad[1, 7] = 1 << 30
        o, lse = attn.paged_fwd_fp8(c["q"].to(DEV), *_gpu_cache(c), bad.to(DEV), _i32(c["lens"]))
        with pytest.raises(attn.AttnError) as e:
            attn.device_status()
        assert e.value.status == attn.ATTN_ERR_DEVICE_DATA
        for r in (0, 2):
            assert torch.equal(o[r].cpu(), want_o[r]) and torch.equal(lse[r].cpu(), want_l[r])
        assert torch.isfinite(o[1].float()).all()


@pytest.mark.parametrize("seed", range(12))
def test_drawn_appends(seed):
    r = random.Random(100 + seed)
    page = 1 << r.randint(3, 10)
    block = 1 << r.randint(0, page.bit_length() - 1)
    H_kv, d = r.choice((1, 2, 3, 8, 9)), r.choice((64, 128))
    rot = r.choice((0, d, d // 2, 16))
    n = r.randint(1, 8)
    ctx, new = [r.randint(0, 300) for _ in range(n)], [r.choice((0, 1, r.randint(2, 90))) for _ in range(n)]
    new[0] = max(new[0], 1)
    c = _append_case(seed, ctx, new, page, block, r.choice((0, 1, 6)), H_kv, d, rot=rot, pad=r.randint(0, 4))
    inter, amp = r.random() < 0.5, r.choice((1.0, 0.75))
    kw = dict(interleaved=inter, amplitude=amp) if rot else {}
    _check_append(c, _append(c, **kw), **kw)


@pytest.mark.parametrize("H,H_kv,d,max_q", [(8, 2, 128, 2), (8, 2, 128, 9), (4, 1, 64, 3), (16, 2, 64, 9)])
def test_max_q_len_above_the_longest(H, H_kv, d, max_q):
    """Tiles for more rows than any request has: the same results, within their bounds."""
    c = _fwd_case(47, [300, 9, 0, 2000, 64, 1, 700, 128, 5], [1] * 9, H, H_kv, d, 16, 4)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    for long in (False, True):
        if long:
            _long_table(c, H_kv)
        o, lse = torch.full(c["q"].shape, 9.0, dtype=BF, device=DEV), torch.full(c["q"].shape[:2], 9.0, device=DEV)
        attn.paged_fwd_fp8(c["q"].to(DEV), *_gpu_cache(c), c["table"].to(DEV), i32(c["lens"]), cu_seqlens_q=i32(c["cu"]), max_q_len=max_q,
                           causal=True, out=o, lse=lse)
        attn.device_status()
        _check_fwd(c, True, (o.cpu(), lse.cpu()))


@pytest.mark.parametrize("page", [8, 128, 1024])
def test_tables_filled_to_the_last_page(page):
    """Requests whose keys are all that the table can hold, in the last place of the cache and of the table."""
    n = max(page, 256) * 2
    c = _fwd_case(48 + page, [n, n - 1, n], None, 4, 2, 64, page, 8)
    c["table"] = c["table"][:, :n // page].contiguous()
    _check_fwd(c, True, _fwd(c, True))
    cu = torch.tensor([0, n, 2 * n - 1, 3 * n - 1], dtype=torch.int32, device=DEV)
    k, v = attn.paged_read_fp8(*_gpu_cache(c), c["table"].to(DEV), cu, 3 * n - 1, dtype=torch.float32)
    attn.device_status()
    for got, name in ((k, "k"), (v, "v")):
        want = torch.cat([ref.values(c[name + "_cache"], c[name + "_scale"], c["table"][r], m) for r, m in enumerate(c["lens"])])
        assert torch.equal(got.cpu().double(), want.float().double())


# ---------------------------------------------------------------- many requests: two KV heads to a unit

@pytest.mark.parametrize("H,H_kv", [(2, 2), (16, 2), (6, 6), (16, 4), (64, 8)])
@pytest.mark.parametrize("page,block", [(16, 1), (8, 8), (128, 32), (1024, 64)])
def test_two_heads_to_a_unit(H, H_kv, page, block):
    lens, _ = _crowd([1, 127, 128, 0, 129, 300, 900], None, H_kv)
    c = _fwd_case(H + block, lens, None, H, H_kv, 128, page, block)
    _check_some(c, True, _fwd(c, True))


@pytest.mark.parametrize("H,H_kv,d", [(4, 2, 128), (8, 4, 128), (8, 8, 64), (48, 8, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_several_tokens_and_heads_to_a_unit(H, H_kv, d, causal):
    lens, q_lens = _crowd([3, 40, 1, 130, 129, 0, 256, 2], [2, 1, 1, 4, 1, 1, 0, 3], H_kv)
    c = _fwd_case(H + d, lens, q_lens, H, H_kv, d, 16, 8, pad=2)
    _check_some(c, causal, _fwd(c, causal))


@pytest.mark.parametrize("H_kv", [2, 4])
def test_a_long_request_among_many(H_kv):
    """One request in the hands of many CTAs, the others many to a CTA; the same bits each time."""
    lens, _ = _crowd([60, 300, 0, 90], None, H_kv)
    lens[len(lens) // 2] = 50000
    c = _fwd_case(52, lens, None, 2 * H_kv, H_kv, 128, 64, 16)
    first = _fwd(c, True)
    _check_some(c, True, first)
    for _ in range(4):
        got = _fwd(c, True)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


def test_lengths_of_a_captured_call_change():
    """One graph, its lengths changed between replays, from one tile to hundreds for a unit, in one workspace."""
    H, H_kv, d, page, B, pages = 8, 4, 128, 64, 40, 360
    g = torch.Generator().manual_seed(53)
    cache = [(torch.randn((900, page, H_kv, d), generator=g) * 50).clamp(-448, 448).to(F8).to(DEV) for _ in "kv"] + \
            [torch.exp2(torch.randint(-6, 3, (900, H_kv, 4), generator=g).float()).to(DEV) / 60 for _ in "kv"]
    table = torch.randint(0, 900, (B, pages), generator=g).to(torch.int32).to(DEV)
    q, lens = torch.randn((B, H, d), generator=g).to(BF).to(DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    room = torch.empty(attn.attn_paged_fwd_fp8_workspace_size(B, B, 1, H, H_kv, d, page, pages), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        o, lse = attn.paged_fwd_fp8(q, *cache, table, lens, workspace=room)
    host = [x.cpu() for x in cache]
    for n in (50, 15000, 23040, 300, 23040):
        lens.copy_(torch.full((B,), n, dtype=torch.int32) - torch.arange(B, dtype=torch.int32) % 7 * (n < 23040))
        graph.replay()
        got = o.clone(), lse.clone()
        want = attn.paged_fwd_fp8(q, *cache, table, lens)
        attn.device_status()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        few = slice(0, 2)
        wo, wl, bo, bl = ref.attend(q[few].cpu(), *host, table[few].cpu(), lens[few].tolist(), None, d ** -0.5, True)
        assert ((got[0][few].cpu().double() - wo).abs() <= bo).all() and ((got[1][few].cpu().double() - wl).abs() <= bl).all()


def test_not_finite_values_stay_in_their_head():
    """A NaN among a head's values, scores or queries reaches that head's rows that see it, and no other head of the unit."""
    lens, q_lens = _crowd([300, 640, 20, 50], [2, 1, 1, 1], 4)
    c = _fwd_case(50, lens, q_lens, 8, 4, 128, 16, 4)
    want_o, want_l = _fwd(c, True)
    at = lambda r, key: (int(c["table"][r, key // 16]), key % 16)
    p, row = at(0, 299)  # seen by the second token only
    c["v_cache"].view(torch.uint8)[p, row, 2, 77] = 0xff
    p, row = at(1, 5)
    c["k_cache"].view(torch.uint8)[p, row, 3, 127] = 0x7f
    c["q"][0, 1, 9] = float("nan")
    o, lse = _fwd(c, True)
    assert torch.isnan(o[1, 4:6, 77].float()).all() and torch.isnan(o[2, 6:8].float()).all() and torch.isnan(lse[2, 6:8]).all()
    assert torch.isnan(o[0, 1].float()).all() and torch.isnan(lse[0, 1])
    same = torch.ones(want_l.shape, dtype=torch.bool)
    same[1, 4:6] = same[2, 6:8] = same[0, 1] = False
    assert torch.equal(o[same], want_o[same]) and torch.equal(lse[same], want_l[same])
    assert torch.equal(lse[1, 4:6], want_l[1, 4:6]) and torch.isfinite(o[1, 4:6, :77].float()).all()


def test_recorded_timeout_with_several_heads_to_a_unit():
    lens, _ = _crowd([700, 40], None, 4)
    c = _fwd_case(51, lens, None, 16, 4, 128, 16, 16)
    args = (c["q"].to(DEV), *_gpu_cache(c), c["table"].to(DEV), _i32(c["lens"]))
    want = attn.paged_fwd_fp8(*args)
    attn.device_status()
    o, l = torch.full_like(want[0], 3.0), torch.full_like(want[1], 3.0)
    assert attn.attn_selftest_wait_timeout(torch.cuda.current_stream().cuda_stream) == attn.ATTN_OK
    attn.paged_fwd_fp8(*args, out=o, lse=l)
    with pytest.raises(attn.AttnError) as e:
        attn.device_status()
    assert e.value.status == attn.ATTN_ERR_TIMEOUT
    assert bool((o == 3).all()) and bool((l == 3).all())
    attn.paged_fwd_fp8(*args, out=o, lse=l)
    attn.device_status()
    assert torch.equal(o, want[0]) and torch.equal(l, want[1])
