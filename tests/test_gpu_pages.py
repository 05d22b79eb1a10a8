"""Page plans (attn_paged_plan) and page sketches (attn_page_sketch): exact whole numbers."""
import numpy as np
import pytest
import torch

import attention_attn_fwd_03_gb300 as attn

import _kv_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.lib()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _state(seed, B, ctx_hi, new_lo, new_hi, page, spare=3):
    """Requests with cached lengths and new tokens, a table that holds their cached pages, a free stack."""
    g = np.random.default_rng(seed)
    ctx = g.integers(0, ctx_hi + 1, B)
    new = g.integers(new_lo, new_hi + 1, B)
    held, want = -(-ctx // page), -(-(ctx + new) // page)
    max_pages = int(want.max()) + 2
    num_pages = int(want.sum()) + spare
    perm = g.permutation(num_pages).astype(np.int32)
    table = np.full((B, max_pages), -7, dtype=np.int32)
    at = 0
    for r in range(B):
        table[r, :held[r]] = perm[at:at + held[r]]
        at += held[r]
    return ctx.tolist(), new.tolist(), table, perm[at:], num_pages


@pytest.mark.parametrize("B,ctx_hi,new_lo,new_hi,page,pad", [
    (1, 0, 1, 1, 64, 0),          # the first token of the first request
    (64, 8191, 1, 1, 64, 0),
    (7, 100, 0, 40, 8, 5),        # requests without new tokens, padding
    (5, 1000, 900, 3000, 16, 100),
    (300, 70, 0, 9, 24, 17),      # a page size that is no power of two
    (1025, 300, 1, 1, 128, 0),    # more requests than threads: two per thread
    (3000, 64, 0, 3, 16, 1),
    (2, 5, 40000, 60000, 1024, 3),
    (16384, 30, 0, 2, 8, 0),      # the largest batch
])
def test_plan_matches_definition(B, ctx_hi, new_lo, new_hi, page, pad):
    ctx, new, table, free, num_pages = _state(B, B, ctx_hi, new_lo, new_hi, page)
    total = max(1, sum(new) + pad)
    want = ref.plan(ctx, new, table, free, len(free), page, total)
    bt = torch.from_numpy(table.copy()).to(DEV)
    got = attn.paged_plan(_i32(ctx), bt, torch.from_numpy(free).to(DEV), _i32([len(free)]), page, num_pages, total,
                          new_lens=_i32(new))
    attn.device_status()
    for name, a, b in zip(("cu", "lens", "positions", "slots"), got[:4], want[:4]):
        assert a.tolist() == b, name
    assert np.array_equal(bt.cpu().numpy(), np.array(want[4]))
    assert got[4].tolist() == [want[5]]
    # a second call on the same inputs gives the same plan
    again = attn.paged_plan(_i32(ctx), bt, torch.from_numpy(free).to(DEV), _i32([len(free)]), page, num_pages, total,
                            new_lens=_i32(new))
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_captured_plan_advances_itself():
    """seq_lens over ctx_lens and free_left over free_count: each replay is the next decode step."""
    B, page, steps = 37, 8, 40
    rng = np.random.default_rng(0)
    ctx = rng.integers(0, 30, B).tolist()
    held = [-(-c // page) for c in ctx]
    max_pages = max(held) + steps // page + 2
    num_pages = sum(held) + B * (steps // page + 1)
    perm = rng.permutation(num_pages).astype(np.int32)
    table = np.full((B, max_pages), -1, dtype=np.int32)
    at = 0
    for r in range(B):
        table[r, :held[r]] = perm[at:at + held[r]]
        at += held[r]
    free = perm[at:]
    lens, bt, fr, count = _i32(ctx), torch.from_numpy(table.copy()).to(DEV), torch.from_numpy(free.copy()).to(DEV), _i32([len(free)])
    pos, slots, cu = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (B, B, B + 1))

    def step():
        attn.paged_plan(lens, bt, fr, count, page, num_pages, B, cu_seqlens_q=cu, seq_lens=lens, positions=pos,
                        slots=slots, free_left=count)
    keep = [t.clone() for t in (lens, bt, count)]
    step()
    torch.cuda.synchronize()
    for t, k in zip((lens, bt, count), keep):
        t.copy_(k)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    n, tab = len(free), table
    for _ in range(steps):
        graph.replay()
        _, ctx2, p, s, tab, n = ref.plan(ctx, [1] * B, tab, free, n, page, B)
        assert pos.tolist() == p and slots.tolist() == s and lens.tolist() == ctx2 and count.tolist() == [n]
        ctx = ctx2
    assert np.array_equal(bt.cpu().numpy(), np.array(tab))
    attn.device_status()


@pytest.mark.parametrize("over", ["ctx", "new"])
def test_plan_in_place_with_many_tokens(over):
    """Outputs over inputs, more tokens than one CTA has threads: the cluster reads all before it writes."""
    ctx, new, table, free, num_pages = _state(8, 700, 90, 0, 60, 16)
    total = sum(new) + 5
    want = ref.plan(ctx, new, table, free, len(free), 16, total)
    for _ in range(3):
        bt, c, n, count = torch.from_numpy(table.copy()).to(DEV), _i32(ctx), _i32(new), _i32([len(free)])
        cu, lens, pos, slots, left = attn.paged_plan(c, bt, torch.from_numpy(free).to(DEV), count, 16, num_pages, total,
                                                     new_lens=n, seq_lens=c if over == "ctx" else n, free_left=count)
        attn.device_status()
        assert lens is (c if over == "ctx" else n) and left is count
        for name, a, b in zip(("cu", "lens", "positions", "slots"), (cu, lens, pos, slots), want[:4]):
            assert a.tolist() == b, name
        assert np.array_equal(bt.cpu().numpy(), np.array(want[4])) and count.tolist() == [want[5]]


@pytest.mark.parametrize("what", ["too few pages", "negative length", "past the table", "too many tokens", "count", "page id"])
def test_plan_reports_bad_data(what):
    ctx, new, table, free, num_pages = _state(5, 6, 50, 3, 20, 8)
    table = np.where(table == -7, -1, table)
    total, count = sum(new) + 4, len(free)
    if what == "too few pages":
        count = 1
    elif what == "negative length":
        new[2] = -4
    elif what == "past the table":
        ctx[3] = table.shape[1] * 8 + 5
    elif what == "too many tokens":
        total = sum(new) - 3
    elif what == "count":
        count = len(free) + 9
    else:
        ctx[1] = 13
        table[1, 1] = num_pages
    bt = torch.from_numpy(table.copy()).to(DEV)
    cu, lens, pos, slots, left = attn.paged_plan(_i32(ctx), bt, torch.from_numpy(free).to(DEV), _i32([count]), 8,
                                                 num_pages, total, new_lens=_i32(new))
    with pytest.raises(attn.AttnError) as e:
        attn.device_status()
    assert e.value.status == attn.ATTN_ERR_DEVICE_DATA
    s = slots.cpu()
    assert bool(((s >= -1) & (s < num_pages * 8)).all())
    if what == "too few pages":
        want = ref.plan(ctx, new, table, np.concatenate([np.full(999, -1), free[:1]]), 1000, 8, total)
        got = [x if x >= 0 else -1 for x in slots.tolist()]
        assert got == [x if x >= 0 else -1 for x in want[3]] and left.tolist() == [0]


# ---------------------------------------------------------------- sketches

def _cache(seed, pages, page, H_kv, d):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((pages, page, H_kv, d), generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("H_kv,d,page,lens,fresh", [
    (1, 64, 8, [1, 8, 9, 0, 3], 1),
    (8, 128, 64, [64, 65, 1, 130, 640], 1),
    (3, 64, 16, [40, 16, 0, 200], 30),        # 24 pieces a row: groups of threads that do not divide the CTA
    (2, 128, 128, [300, 127, 128], 1000),     # every page
    (16, 128, 32, [70, 33], 64),              # more than 1024 channels: two channel blocks
    (9, 128, 16, [50, 20], 20),               # the second channel block partial
    (5, 64, 1024, [1500, 1], 700),
    (1, 64, 8, [4100, 100, 0, 7], 5000),      # many pages of narrow rows: a warp per page
    (3, 64, 8, [4099, 90], 5000),             # 24 of 32 lanes across a row
    (2, 128, 16, [9000, 41], 9000),
    (5, 64, 16, [8500, 200], 9000),           # many pages of wider rows
])
def test_sketch_matches_definition(H_kv, d, page, lens, fresh):
    B, max_pages = len(lens), max(-(-n // page) for n in lens) + 1
    pages = sum(-(-n // page) for n in lens) + 2
    k = _cache(H_kv + d, pages, page, H_kv, d)
    perm = np.random.default_rng(page).permutation(pages)
    table, at = np.full((B, max_pages), -1, dtype=np.int32), 0
    sk = torch.full((pages, H_kv, 2 * d), 99, dtype=torch.int8)
    amp = torch.full((pages, H_kv), 5.0)
    want_sk, want_amp = sk.clone().numpy(), amp.clone().numpy()
    for r, n in enumerate(lens):
        m = -(-n // page)
        table[r, :m] = perm[at:at + m]
        at += m
        if n % page:
            k[int(table[r, m - 1]), n % page:] = float("nan")  # rows past the last key are not read
        for p in range(max(0, n - fresh) // page if n else m, m):
            rows = min(page, n - p * page)
            want_sk[table[r, p]], want_amp[table[r, p]] = ref.sketch(k[int(table[r, p]), :rows].float().numpy())
    for cu in (None, np.concatenate([[0], np.cumsum([min(n, fresh) for n in lens])])):
        s, a = sk.to(DEV), amp.to(DEV)
        attn.page_sketch(k.to(DEV), torch.from_numpy(table).to(DEV), _i32(lens), s, a,
                         cu_seqlens_q=None if cu is None else _i32(cu.tolist()), max_q_len=fresh)
        attn.device_status()
        assert np.array_equal(s.cpu().numpy(), want_sk) and np.array_equal(a.cpu().numpy(), want_amp)


def test_sketch_of_extreme_pages():
    """Zeros, infinities, NaN, the smallest and largest numbers, and an order that must not matter."""
    H_kv, d, page = 2, 64, 8
    k = _cache(4, 8, page, H_kv, d)
    k[0] = 0
    k[1, 3, 0, 7] = float("inf")
    k[2, 5, 1, 63] = float("nan")
    k[3] *= 1e-38
    k[4] = torch.finfo(torch.bfloat16).max * torch.sign(k[4])
    k[5] = 2.0 ** -133  # the smallest subnormal
    k[6] = -k[6].abs()
    table, lens = _i32([[0, 1, 2, 3, 4, 5, 6, 7]]), _i32([64])
    out = []
    for x in (k, k.flip(1)):
        s = torch.empty((8, H_kv, 2 * d), dtype=torch.int8, device=DEV)
        a = torch.empty((8, H_kv), device=DEV)
        attn.page_sketch(x.contiguous().to(DEV), table, lens, s, a, max_q_len=64)
        attn.device_status()
        out.append((s.cpu(), a.cpu()))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    for p in range(8):
        code, amp = ref.sketch(k[p].float().numpy())
        assert np.array_equal(out[0][0][p].numpy(), code) and np.array_equal(out[0][1][p].numpy(), amp), p


def test_sketch_reports_bad_data():
    k = _cache(1, 4, 8, 1, 64).to(DEV)
    s, a = torch.zeros((4, 1, 128), dtype=torch.int8, device=DEV), torch.full((4, 1), -1.0, device=DEV)
    for table, lens, cu, m in (([[9, 0]], [8], None, 1), ([[-1, 0]], [8], None, 1), ([[0, 1]], [17], None, 1),
                               ([[0, 1]], [-1], None, 1), ([[0, 1]], [16], [0, 9], 4), ([[0, 1]], [16], [4, 0], 4)):
        attn.page_sketch(k, _i32(table), _i32(lens), s, a, cu_seqlens_q=None if cu is None else _i32(cu), max_q_len=m)
        with pytest.raises(attn.AttnError) as e:
            attn.device_status()
        assert e.value.status == attn.ATTN_ERR_DEVICE_DATA
    assert bool((a[2:] == -1).all())


def test_sketch_past_32_bit_offsets():
    H_kv, d, page, pages = 8, 128, 64, 66000
    k = torch.empty((pages, page, H_kv, d), dtype=torch.bfloat16, device=DEV)
    last = _cache(3, 1, page, H_kv, d)
    k[pages - 1] = last[0].to(DEV)
    s, a = torch.zeros((pages, H_kv, 2 * d), dtype=torch.int8, device=DEV), torch.zeros((pages, H_kv), device=DEV)
    attn.page_sketch(k, _i32([[pages - 1]]), _i32([page]), s, a)
    attn.device_status()
    code, amp = ref.sketch(last[0].float().numpy())
    assert np.array_equal(s[pages - 1].cpu().numpy(), code) and np.array_equal(a[pages - 1].cpu().numpy(), amp)
    assert int(s[:pages - 1].abs().max()) == 0


def test_other_stream():
    """The whole chain on a side stream, outputs allocated by the calls: the bits of the default stream."""
    page, H, H_kv, d = 16, 4, 2, 64
    ctx, new, table, free, num_pages = _state(3, 9, 60, 0, 20, page)
    total = sum(new) + 2
    f = attn.rope_inv_freq(d)[0].to(DEV)
    x = torch.randn((total, H + 2 * H_kv, d), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).to(DEV)
    side = torch.cuda.Stream()
    out = []
    for stream in (None, side):
        bt = torch.from_numpy(np.where(table == -7, -1, table)).to(DEV)
        kc, vc = (torch.zeros((num_pages, page, H_kv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        sk, amp = torch.zeros((num_pages, H_kv, 2 * d), dtype=torch.int8, device=DEV), torch.zeros((num_pages, H_kv), device=DEV)
        args = _i32(ctx), bt, torch.from_numpy(free).to(DEV), _i32([len(free)])
        fresh = _i32(new)
        torch.cuda.synchronize()
        cu, lens, pos, slots, left = attn.paged_plan(*args, page, num_pages, total, new_lens=fresh, stream=stream)
        with torch.cuda.stream(side if stream is not None else torch.cuda.current_stream()):
            qo = torch.zeros((total, H, d), dtype=torch.bfloat16, device=DEV)
        attn.paged_append(x[:, :H], x[:, H:H + H_kv], x[:, H + H_kv:], kc, vc, slots, positions=pos, inv_freq=f, q_out=qo, stream=stream)
        attn.page_sketch(kc, bt, lens, sk, amp, cu_seqlens_q=cu, max_q_len=20, stream=stream)
        qr, kr = attn.rope(x[:, :H], x[:, H:H + H_kv], inv_freq=f, positions=pos, stream=stream)
        tables, sel = attn.page_select(qo, sk, amp, bt, lens, page, 2, cu_seqlens_q=cu, stream=stream)
        torch.cuda.synchronize()
        attn.device_status()
        out.append((cu, lens, pos, slots, left, bt, kc, vc, qo, sk, amp, qr, kr, tables, sel))
    assert all(torch.equal(a, b) for a, b in zip(*out))
    with pytest.raises(ValueError):
        attn.paged_plan(*args, page, num_pages, total, new_lens=fresh[:-1])
