"""Page selection (attn_page_select), page-sparse attention (attn_paged_sparse_fwd), and a serving step
made of the cache operators.

The selection is compared for equality: its scores are integers and three fp32 roundings.  Attention is
held to the bounds that _kv_ref.attend derives from the roundings of P and O."""
import numpy as np
import pytest
import torch

import attention_attn_fwd_03_gb300 as attn
from attention_attn_fwd_03_gb300 import inputs

import _kv_ref as ref
from _parity import default_scale

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.lib()


def _sketches(k_cache, page_ok):
    """Sketches of whole pages (garbage for those that are not page_ok, which nothing should score)."""
    n, _, H_kv, d = k_cache.shape
    sk, amp = np.full((n, H_kv, 2 * d), 101, dtype=np.int8), np.full((n, H_kv), np.nan, dtype=np.float32)
    for p in range(n):
        if page_ok[p]:
            sk[p], amp[p] = ref.sketch(k_cache[p].float().numpy())
    return sk, amp


def _case(seed, lens, q_lens, H, H_kv, d, page, extra_pages=2, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pages = [-(-n // page) for n in lens]
    pool = sum(pages) + 3
    perm = torch.randperm(pool, generator=g)
    max_pages = max(pages) + extra_pages
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    k = (torch.randn((pool, 1, H_kv, d), generator=g) * spread + torch.randn((pool, page, H_kv, d), generator=g)).to(torch.bfloat16)
    v = torch.randn((pool, page, H_kv, d), generator=g).to(torch.bfloat16)
    ok, at = np.zeros(pool, dtype=bool), 0
    for r in range(B):
        table[r, :pages[r]] = perm[at:at + pages[r]]
        at += pages[r]
        ok[table[r, :pages[r]].numpy()] = True
    sk, amp = _sketches(k, ok)
    for r, n in enumerate(lens):  # what lies behind the last key, and in no page, is not read
        if n % page:
            k[table[r, pages[r] - 1], n % page:] = float("nan")
            v[table[r, pages[r] - 1], n % page:] = float("nan")
    k[torch.from_numpy(~ok)] = float("nan")
    v[torch.from_numpy(~ok)] = float("nan")
    cu = None if q_lens is None else np.concatenate([[0], np.cumsum(q_lens)]).tolist()
    T = B if cu is None else cu[-1]
    q = torch.randn((T, H, d), generator=g).to(torch.bfloat16)
    return dict(q=q, k=k, v=v, table=table, lens=list(lens), cu=cu, sk=sk, amp=amp, page=page, T=T)


def _gpu(c):
    t = lambda x: torch.as_tensor(x).to(DEV)
    return dict(q=t(c["q"]), k=t(c["k"]), v=t(c["v"]), bt=t(c["table"]), lens=t(np.array(c["lens"], dtype=np.int32)),
                sk=t(c["sk"]), amp=t(c["amp"]), cu=None if c["cu"] is None else t(np.array(c["cu"], dtype=np.int32)))


def _select(c, g, budget, first, last, **kw):
    out = attn.page_select(g["q"], g["sk"], g["amp"], g["bt"], g["lens"], c["page"], budget, first, last,
                           cu_seqlens_q=g["cu"], **kw)
    attn.device_status()
    return out


def _want(c, budget, first, last):
    return ref.select(c["q"].float().numpy(), c["sk"], c["amp"], c["table"].numpy(), c["lens"], c["cu"], c["page"], budget,
                      first, last)


CASES = [
    # lens, q_lens, H, H_kv, d, page, budget, first, last
    ([1000], None, 4, 1, 128, 16, 8, 1, 1),
    ([0, 1, 16, 17, 300, 1], None, 8, 2, 64, 16, 4, 0, 1),       # empty and one-key requests
    ([5000, 640, 3999], None, 32, 8, 128, 64, 10, 1, 2),
    ([700, 90, 1300], [3, 1, 8], 16, 2, 64, 16, 12, 1, 4),       # several tokens per request
    ([260, 3, 0, 130], [5, 3, 0, 2], 6, 2, 128, 8, 6, 2, 2),     # G = 3; a request shorter than its budget; one empty
    ([40, 20], [40, 20], 4, 4, 64, 8, 2, 0, 1),                  # whole prompts: tokens that see one page and more
    ([3000, 2000], None, 128, 1, 128, 32, 20, 0, 1),             # G = 128
    ([2, 5], [4, 5], 2, 1, 64, 8, 1, 0, 1),                      # more tokens than keys: some see none
    ([900, 60], None, 40, 2, 128, 16, 9, 1, 1),                  # G = 20: three column tiles, the last half empty
    ([500, 1], None, 32, 1, 64, 8, 33, 1, 1),                    # G = 32
    ([3000, 20, 1], [2, 1, 1], 12, 1, 128, 8, 50, 2, 1),         # G = 12, two boxes per chunk
    ([700, 2000], None, 33, 1, 64, 32, 12, 1, 1),                # G = 33: the tiles of 128 rows
    ([1700, 400], None, 48, 2, 128, 16, 14, 1, 1),               # G = 24 ..
    ([1700, 400], None, 50, 2, 128, 16, 14, 1, 1),               # .. and 25
    ([2500, 300], None, 10, 2, 128, 128, 3, 0, 1),               # pages of several chunks
    ([9000], None, 8, 8, 64, 1024, 4, 1, 1),                     # G = 1, large pages
    ([9000, 100], None, 4, 2, 64, 8, 1030, 3, 5),                # a budget beyond the fused kernel's list
    ([300, 2000], None, 8, 2, 128, 16, 3, 1, 2),                 # nothing left for the scores to decide
    ([160000], None, 2, 1, 64, 8, 40, 1, 1),                     # 20000 pages
    ([200000], None, 2, 1, 64, 8, 40, 1, 1),                     # more scores than the fused kernel's shared memory holds
    ([20000], None, 2, 1, 64, 8, 700, 3, 5),                     # 2500 pages: several selection runs per thread
]


@pytest.mark.parametrize("lens,q_lens,H,H_kv,d,page,budget,first,last", CASES)
def test_select_and_attend(lens, q_lens, H, H_kv, d, page, budget, first, last):
    c = _case(len(lens) + d + page, lens, q_lens, H, H_kv, d, page)
    g = _gpu(c)
    tables, sel = _select(c, g, budget, first, last)
    want, want_sel = _want(c, budget, first, last)
    assert np.array_equal(sel.cpu().numpy(), want_sel)
    assert np.array_equal(tables.cpu().numpy(), want)
    scale = default_scale(d)
    o, lse, t2, s2 = attn.paged_sparse_fwd(g["q"], g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], budget, first, last,
                                           cu_seqlens_q=g["cu"], scale=scale, return_tables=True)
    attn.device_status()
    assert torch.equal(t2, tables) and torch.equal(s2, sel)
    ro, rl, bo, bl = ref.attend(c["q"].float().numpy(), c["k"].float().numpy(), c["v"].float().numpy(), want, want_sel, scale)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), empty) and np.all(o[empty] == 0)
    assert np.all(np.abs(o - ro) <= bo), np.max(np.abs(o - ro) / np.maximum(bo, 1e-30))
    assert np.all(np.abs(lse[~empty] - rl[~empty]) <= bl[~empty])
    # without tables, without lse: the same bits
    o2, none = attn.paged_sparse_fwd(g["q"], g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], budget, first, last,
                                     cu_seqlens_q=g["cu"], scale=scale, return_lse=False)
    assert none is None and np.array_equal(o2.double().cpu().numpy(), o)


def test_many_scored_pages_and_unsplit_units():
    """Enough (token, head) rows that the score kernel takes its wide chunks and no key range is split."""
    rng = np.random.default_rng(1)
    lens = rng.integers(1, 3000, 120).tolist()
    c = _case(77, lens, None, 16, 8, 64, 8)
    g = _gpu(c)
    tables, sel = _select(c, g, 16, 1, 1)
    want, want_sel = _want(c, 16, 1, 1)
    assert np.array_equal(tables.cpu().numpy(), want) and np.array_equal(sel.cpu().numpy(), want_sel)
    o, lse = attn.paged_sparse_fwd(g["q"], g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], 16)
    attn.device_status()
    ro, rl, bo, bl = ref.attend(c["q"].float().numpy(), c["k"].float().numpy(), c["v"].float().numpy(), want, want_sel,
                                1 / 8.0)
    assert np.all(np.abs(o.double().cpu().numpy() - ro) <= bo) and np.all(np.abs(lse.double().cpu().numpy() - rl) <= bl)


def test_selection_from_many_pages():
    """20000 pages of scores that tie a lot, budgets of a few to all but one."""
    lens, page = [160000], 8
    c = _case(5, [800], None, 2, 1, 64, page)
    g = torch.Generator().manual_seed(11)
    n = lens[0] // page
    c["sk"] = torch.randint(-127, 128, (n, 1, 128), generator=g).to(torch.int8).numpy()
    c["amp"] = (torch.randint(1, 5, (n, 1), generator=g) / 4.0).numpy().astype(np.float32)
    c["table"] = torch.randperm(n, generator=g).to(torch.int32)[None].contiguous()
    c["lens"] = lens
    for budget in (5, 1000, 19999):
        tables, sel = _select(c, _gpu(c), budget, 1, 1)
        want, want_sel = _want(c, budget, 1, 1)
        assert np.array_equal(tables.cpu().numpy(), want) and np.array_equal(sel.cpu().numpy(), want_sel)


def test_ties_go_to_the_earlier_page():
    c = _case(3, [640], None, 4, 2, 64, 8)
    c["sk"][:] = c["sk"][int(c["table"][0, 0])]     # every page scores alike
    c["amp"][:] = 1.5
    for budget, first, last in ((7, 0, 1), (7, 2, 3), (5, 2, 3), (79, 0, 1)):
        tables, _ = _select(c, _gpu(c), budget, first, last)
        t = c["table"][0]
        want = torch.cat([t[:budget - last], t[80 - last:80]])
        assert torch.equal(tables[0, 0].cpu(), want) and torch.equal(tables[0, 1].cpu(), want)
    c["amp"][:] = 0.0                               # zero pages: scores of +0 and -0 tie too
    c["sk"][::2] = -c["sk"][::2]
    tables, _ = _select(c, _gpu(c), 7, 0, 1)
    assert torch.equal(tables[0, 0].cpu(), torch.cat([c["table"][0, :6], c["table"][0, 79:80]]))


@pytest.mark.parametrize("d,H", [(128, 1), (64, 20)])
def test_scores_at_the_ends_of_their_range(d, H):
    """Codes of +-127 throughout: the integer sums reach 2 d 127^2, and pages that differ by one unit in
    one channel differ in their scores."""
    c = _case(2, [320], None, H, 1, d, 8)
    c["q"][:] = torch.where(torch.arange(d) % 3 == 0, -1.0, 1.0)
    full = np.where(np.arange(d) % 3 == 0, -127, 127).astype(np.int8)
    ids = c["table"][0, :40].numpy()
    for p in range(40):
        c["sk"][ids[p], 0] = np.concatenate([full, full])
        c["sk"][ids[p], 0, (p * 7) % (2 * d)] //= 1 + p % 4
        c["sk"][ids[p], 0, 1] = 127 - (p * 11) % 17
    c["amp"][:] = 1.0
    for budget in (2, 9, 30):
        tables, sel = _select(c, _gpu(c), budget, 0, 1)
        want, want_sel = _want(c, budget, 0, 1)
        assert np.array_equal(tables.cpu().numpy(), want) and np.array_equal(sel.cpu().numpy(), want_sel)


def test_non_finite_queries_and_sketches():
    c = _case(8, [400, 400, 400, 400], None, 4, 1, 64, 8)
    c["q"][1, 2, 5] = float("inf")
    c["q"][2, 0, 0] = float("nan")
    c["q"][3] = 0
    for p in (3, 17, 30):
        c["amp"][int(c["table"][0, p])] = np.inf
        c["sk"][int(c["table"][0, p])] = 0
    tables, sel = _select(c, _gpu(c), 9, 1, 1)
    want, want_sel = _want(c, 9, 1, 1)
    assert np.array_equal(tables.cpu().numpy(), want) and np.array_equal(sel.cpu().numpy(), want_sel)
    assert set(c["table"][0, [3, 17, 30]].tolist()) <= set(tables[0, 0].tolist())


@pytest.mark.parametrize("q_lens", [None, [2, 7, 1]])
def test_full_budget_is_dense_attention(q_lens):
    """With a budget that holds every page the call is causal attn_paged_fwd."""
    c = _case(6, [500, 900, 64], q_lens, 8, 2, 128, 16)
    g = _gpu(c)
    o, lse = attn.paged_sparse_fwd(g["q"], g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], 64, cu_seqlens_q=g["cu"])
    o2, lse2 = attn.paged_fwd(g["q"], g["k"], g["v"], g["bt"], g["lens"], cu_seqlens_q=g["cu"],
                              max_q_len=None if q_lens is None else max(q_lens), causal=True)
    attn.device_status()
    # both round P and O to bf16; the running maximum at which P rounds may differ between the two
    tables, sel = (x.cpu().numpy() for x in _select(c, g, 64, 1, 1))
    ro, rl, bo, bl = ref.attend(c["q"].float().numpy(), c["k"].float().numpy(), c["v"].float().numpy(), tables, sel,
                                default_scale(128))
    for x, y in ((o, lse), (o2, lse2)):
        assert np.all(np.abs(x.double().cpu().numpy() - ro) <= bo) and np.all(np.abs(y.double().cpu().numpy() - rl) <= bl)


def test_rows_behind_the_last_request_stay():
    c = _case(9, [300, 200], [3, 2], 4, 2, 64, 8)
    g = _gpu(c)
    pad = torch.full((4, 4, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    q = torch.cat([g["q"], pad])
    for budget in (6, 60):  # with and without a merge of split ranges
        o = torch.full_like(q, 3.0)
        lse = torch.full((9, 4), 3.0, device=DEV)
        _, _, tables, sel = attn.paged_sparse_fwd(q, g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], budget,
                                                  cu_seqlens_q=g["cu"], out=o, lse=lse, return_tables=True)
        attn.device_status()
        o2, lse2 = attn.paged_sparse_fwd(g["q"], g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], budget,
                                         cu_seqlens_q=g["cu"])
        assert torch.equal(o[:5], o2) and torch.equal(lse[:5], lse2)
        assert bool((o[5:] == 3).all()) and bool((lse[5:] == 3).all())
        assert bool((tables[5:] == -1).all()) and sel.tolist()[5:] == [0] * 4


@pytest.mark.parametrize("H", [16, 120])  # the fused kernel; the selection kernels and the paged kernel
def test_replay_other_stream_and_two_at_once(H):
    c = _case(12, [3000, 500, 0, 1700], None, H, 4, 128, 16)
    g = _gpu(c)
    args = (g["q"], g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], 24, 1, 2)
    o_ref, l_ref = attn.paged_sparse_fwd(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for i in range(6):  # two streams, each call with a workspace of its own
        s = streams[i % 2]
        s.wait_stream(torch.cuda.current_stream())
        outs.append(attn.paged_sparse_fwd(*args, stream=s))
    torch.cuda.synchronize()
    for o, l in outs:
        assert torch.equal(o, o_ref) and torch.equal(l, l_ref)
    need = attn.attn_paged_sparse_fwd_workspace_size(4, H, 4, 128, 16, c["table"].shape[1], 24)
    ws = torch.full((need,), 0xAB, dtype=torch.uint8, device=DEV)
    o, l = torch.zeros_like(o_ref), torch.zeros_like(l_ref)
    graphs = []
    for _ in range(2):  # two graphs that share a workspace, replayed one after the other
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            attn.paged_sparse_fwd(*args, out=o, lse=l, workspace=ws)
        torch.cuda.current_stream().wait_stream(side)
        graphs.append(graph)
    for graph in graphs + graphs:
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o_ref) and torch.equal(l, l_ref)
    # the replay follows new lengths and queries
    g["lens"].copy_(torch.tensor([2000, 499, 0, 1], dtype=torch.int32))
    g["q"].copy_(g["q"].flip(0))
    graphs[0].replay()
    torch.cuda.synchronize()
    o2, l2 = attn.paged_sparse_fwd(*args)
    attn.device_status()
    assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("what", ["page id", "length", "offsets", "negative length"])
def test_bad_device_data_is_reported(what):
    c = _case(14, [300, 200], [3, 2], 4, 2, 64, 8)
    if what == "page id":
        c["table"][0, 5], c["table"][1, 2] = 10 ** 6, -5
    elif what == "length":
        c["lens"][1] = 10 ** 9
    elif what == "negative length":
        c["lens"][0] = -3
    else:
        c["cu"] = [0, 9, 5]
    g = _gpu(c)
    for budget in (4, 64):
        attn.paged_sparse_fwd(g["q"], g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], budget, cu_seqlens_q=g["cu"])
        with pytest.raises(attn.AttnError) as e:
            attn.device_status()
        assert e.value.status == attn.ATTN_ERR_DEVICE_DATA
    attn.device_status()


def test_helpers_refuse():
    c = _case(15, [100], None, 4, 2, 64, 8)
    g = _gpu(c)
    args = dict(q=g["q"], k_cache=g["k"], v_cache=g["v"], block_table=g["bt"], seq_lens=g["lens"], sketch=g["sk"],
                amp=g["amp"], budget=4)
    for kw in (dict(q=g["q"].float()), dict(sketch=g["sk"].to(torch.uint8)), dict(lse=torch.zeros((1, 4), device=DEV).double())):
        with pytest.raises(TypeError):
            attn.paged_sparse_fwd(**dict(args, **kw))
    for kw in (dict(amp=g["amp"][:-1]), dict(k_cache=g["k"][:, :, :1].contiguous()), dict(q=g["q"].transpose(1, 2)),
               dict(seq_lens=g["lens"].repeat(2))):
        with pytest.raises(ValueError):
            attn.paged_sparse_fwd(**dict(args, **kw))
    for kw in (dict(budget=0), dict(budget=4, first=4), dict(last=0), dict(scale=-1.0)):
        with pytest.raises(attn.AttnError):
            attn.paged_sparse_fwd(**dict(args, **kw))
    with pytest.raises(attn.AttnError):  # scores do not fit
        _select(c, g, 4, 1, 1, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))


def test_serving_steps():
    """Prompts, then decode steps: plan, append, sketch, sparse attention, from an empty cache; the cache, the
    sketches and the attention are those of the same tokens laid out plainly."""
    g = torch.Generator().manual_seed(21)
    B, H, H_kv, d, page, budget = 3, 4, 2, 64, 8, 6
    prompts, steps = [37, 5, 90], 12
    max_pages, num_pages = 16, 48
    f, _ = attn.rope_inv_freq(d)
    fd = f.to(DEV)
    kc, vc = (torch.full((num_pages, page, H_kv, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sk = torch.zeros((num_pages, H_kv, 2 * d), dtype=torch.int8, device=DEV)
    amp = torch.zeros((num_pages, H_kv), device=DEV)
    bt = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(num_pages, generator=g).to(torch.int32).to(DEV)
    count = torch.tensor([num_pages], dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    keys = [np.zeros((0, H_kv, d)) for _ in range(B)]
    vals = [np.zeros((0, H_kv, d)) for _ in range(B)]
    for step in range(steps):
        new = prompts if step == 0 else [1] * B
        total = sum(new) + (3 if step == 0 else 0)  # the prompt batch is padded
        fused = torch.randn((total, (H + 2 * H_kv) * d), generator=g).to(torch.bfloat16).to(DEV)
        q, k, v = (x.unflatten(1, (-1, d)) for x in fused.split([H * d, H_kv * d, H_kv * d], 1))
        cu, _, pos, slots, _ = attn.paged_plan(lens, bt, free, count, page, num_pages, total, seq_lens=lens, free_left=count,
                                               new_lens=torch.tensor(new, dtype=torch.int32, device=DEV))
        qr = attn.paged_append(q, k, v, kc, vc, slots, positions=pos, inv_freq=fd, q_out=torch.zeros((total, H, d), dtype=torch.bfloat16, device=DEV))
        attn.page_sketch(kc, bt, lens, sk, amp, cu_seqlens_q=cu, max_q_len=max(new))
        o = torch.full((total, H, d), 9.0, dtype=torch.bfloat16, device=DEV)
        _, lse, tables, sel = attn.paged_sparse_fwd(qr, kc, vc, bt, lens, sk, amp, budget, cu_seqlens_q=cu, out=o, return_tables=True)
        dense, _ = attn.paged_fwd(qr[:sum(new)].contiguous(), kc, vc, bt, lens, cu_seqlens_q=cu, max_q_len=max(new), causal=True)
        attn.device_status()
        # the plain layout: each request's keys so far
        offs = np.concatenate([[0], np.cumsum(new)])
        ctx = [len(x) for x in keys]
        for r in range(B):
            rows = slice(int(offs[r]), int(offs[r + 1]))
            at = np.arange(ctx[r], ctx[r] + new[r])
            keys[r] = np.concatenate([keys[r], ref.rope(k[rows].double().cpu().numpy(), at, f.numpy(), d)])
            vals[r] = np.concatenate([vals[r], v[rows].double().cpu().numpy()])
            n, table = len(keys[r]), bt[r].cpu().numpy()
            assert int(lens[r]) == n
            got_k = kc.float().cpu().numpy()[table[:-(-n // page)]].reshape(-1, H_kv, d)[:n]
            got_v = vc.float().cpu().numpy()[table[:-(-n // page)]].reshape(-1, H_kv, d)[:n]
            assert np.all(np.abs(got_k - keys[r]) <= 2.0 ** -8 * np.abs(keys[r]) + 2.0 ** -18) and np.array_equal(got_v, vals[r])
            for p in range(-(-n // page)):
                code, a = ref.sketch(got_k[p * page:(p + 1) * page])
                assert np.array_equal(sk[table[p]].cpu().numpy(), code) and np.array_equal(amp[table[p]].cpu().numpy(), a)
            assert np.all(np.abs(qr[rows].double().cpu().numpy() - ref.rope(q[rows].double().cpu().numpy(), at, f.numpy(), d))
                          <= 2.0 ** -8 * np.abs(qr[rows].double().cpu().numpy()) + 2.0 ** -18)
        want, want_sel = ref.select(qr.float().cpu().numpy(), sk.cpu().numpy(), amp.cpu().numpy(), bt.cpu().numpy(), lens.tolist(),
                                    cu.tolist(), page, budget, 1, 1)
        assert np.array_equal(tables.cpu().numpy(), want) and np.array_equal(sel.cpu().numpy(), want_sel)
        owned = sum(new)
        ro, rl, bo, bl = ref.attend(qr.float().cpu().numpy(), kc.float().cpu().numpy(), vc.float().cpu().numpy(), want, want_sel,
                                    default_scale(d))
        assert np.all(np.abs(o.double().cpu().numpy() - ro)[:owned] <= bo[:owned])
        assert np.all(np.abs(lse.double().cpu().numpy() - rl)[:owned] <= bl[:owned])
        assert bool((o[owned:] == 9).all()) and bool((qr[owned:] == 0).all())
        if step == 0:  # a short prompt fits the budget: sparse is dense there
            rows = slice(37, 42)
            assert np.all(np.abs(dense[rows].double().cpu().numpy() - ro[rows]) <= bo[rows])
    assert int(count) == num_pages - sum(-(-(p + steps - 1) // page) for p in prompts)


def test_captured_decode_step():
    """One decode step (plan in place, append, sketch, sparse attention) captured once and replayed: every
    replay is the next step, to the bits of the same calls made one by one."""
    B, H, H_kv, d, page, budget, steps = 5, 8, 2, 128, 16, 4, 20
    ctx = [0, 15, 40, 100, 63]
    max_pages = 9
    num_pages = 64
    f = attn.rope_inv_freq(d)[0].to(DEV)

    def state():
        g = torch.Generator().manual_seed(3)
        held = [-(-c // page) for c in ctx]
        perm = torch.randperm(num_pages, generator=g).to(torch.int32)
        table = torch.full((B, max_pages), -1, dtype=torch.int32)
        at = 0
        for r in range(B):
            table[r, :held[r]] = perm[at:at + held[r]]
            at += held[r]
        k, v = (torch.randn((num_pages, page, H_kv, d), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
        s = dict(lens=torch.tensor(ctx, dtype=torch.int32, device=DEV), bt=table.to(DEV), free=perm[at:].contiguous().to(DEV),
                 count=torch.tensor([num_pages - at], dtype=torch.int32, device=DEV), k=k, v=v,
                 sk=torch.zeros((num_pages, H_kv, 2 * d), dtype=torch.int8, device=DEV),
                 amp=torch.zeros((num_pages, H_kv), device=DEV), fused=torch.zeros((B, (H + 2 * H_kv) * d), dtype=torch.bfloat16, device=DEV),
                 o=torch.zeros((B, H, d), dtype=torch.bfloat16, device=DEV), lse=torch.zeros((B, H), device=DEV))
        attn.page_sketch(s["k"], s["bt"], s["lens"], s["sk"], s["amp"], max_q_len=max_pages * page)
        s["tmp"] = [torch.empty(n, dtype=torch.int32, device=DEV) for n in (B + 1, B, B)]
        return s

    def step(s):
        cu, pos, slots = s["tmp"]
        attn.paged_plan(s["lens"], s["bt"], s["free"], s["count"], page, num_pages, B, cu_seqlens_q=cu, seq_lens=s["lens"],
                        positions=pos, slots=slots, free_left=s["count"])
        q, k, v = (x.unflatten(1, (-1, d)) for x in s["fused"].split([H * d, H_kv * d, H_kv * d], 1))
        attn.paged_append(q, k, v, s["k"], s["v"], slots, positions=pos, inv_freq=f, q_out=q)
        attn.page_sketch(s["k"], s["bt"], s["lens"], s["sk"], s["amp"])
        attn.paged_sparse_fwd(q.contiguous(), s["k"], s["v"], s["bt"], s["lens"], s["sk"], s["amp"], budget, out=s["o"], lse=s["lse"])
    eager, kept, replayed = state(), state(), state()
    step(kept)  # warm-up
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step(replayed)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(steps):
        x = torch.randn(eager["fused"].shape, generator=torch.Generator().manual_seed(100 + i)).to(torch.bfloat16).to(DEV)
        for s in (eager, replayed):
            s["fused"].copy_(x)
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("lens", "bt", "count", "k", "v", "sk", "amp", "o", "lse"):
            assert torch.equal(eager[name], replayed[name]), (i, name)
    attn.device_status()
    assert eager["lens"].tolist() == [c + steps for c in ctx]


def test_recorded_timeout_leaves_outputs_alone():
    """While a bounded wait's timeout is recorded, page-sparse attention returns without work, as the other
    attention calls do; once the word is read it computes again."""
    c = _case(16, [900, 300], None, 8, 2, 64, 16)
    g = _gpu(c)
    args = (g["q"], g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], 6)
    o_ref, l_ref = attn.paged_sparse_fwd(*args)
    attn.device_status()
    o, l = torch.full_like(o_ref, 3.0), torch.full_like(l_ref, 3.0)
    assert attn.attn_selftest_wait_timeout(torch.cuda.current_stream().cuda_stream) == attn.ATTN_OK
    attn.paged_sparse_fwd(*args, out=o, lse=l)
    with pytest.raises(attn.AttnError) as e:
        attn.device_status()
    assert e.value.status == attn.ATTN_ERR_TIMEOUT
    assert bool((o == 3).all()) and bool((l == 3).all())
    attn.paged_sparse_fwd(*args, out=o, lse=l)
    attn.device_status()
    assert torch.equal(o, o_ref) and torch.equal(l, l_ref)


def test_caches_past_32_bit_offsets():
    """Pages at the end of caches of more than 2^32 elements."""
    pages, page, H_kv, d, n = 66000, 64, 8, 128, 40
    c = _case(17, [n * page - 7], None, 8, H_kv, d, page)
    ids = c["table"][0, :n].long()
    k, v = (torch.empty((pages, page, H_kv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sk, amp = torch.zeros((pages, H_kv, 2 * d), dtype=torch.int8, device=DEV), torch.zeros((pages, H_kv), device=DEV)
    far = pages - 1 - 3 * torch.arange(n)
    k[far.to(DEV)], v[far.to(DEV)] = c["k"][ids].to(DEV), c["v"][ids].to(DEV)
    sk[far.to(DEV)], amp[far.to(DEV)] = torch.from_numpy(c["sk"])[ids].to(DEV), torch.from_numpy(c["amp"])[ids].to(DEV)
    g = _gpu(c)
    want = attn.paged_sparse_fwd(g["q"], g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], 9)
    got = attn.paged_sparse_fwd(g["q"], k, v, far.to(torch.int32)[None].contiguous().to(DEV), g["lens"], sk, amp, 9)
    attn.device_status()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("seed", range(30))
def test_random_shapes(seed):
    """Seeded shapes over the whole range: groups on both kernels, every page size, budgets below and above
    the pages in use, requests that are empty or shorter than their new tokens."""
    rng = np.random.default_rng(1000 + seed)
    d = int(rng.choice([64, 128]))
    page = int(rng.choice([8, 16, 32, 64, 128, 256, 512, 1024]))
    H_kv = int(rng.choice([1, 2, 3, 5]))
    G = int(rng.choice([1, 2, 5, 7, 8, 11, 16, 21, 30, 40]))
    B = int(rng.integers(1, 6))
    top = int(rng.choice([3, 40, 150])) * page
    lens = rng.integers(0, max(2, min(top, 12000)), B).tolist()
    q_lens = None if rng.random() < 0.5 else rng.integers(0, 7, B).tolist()
    if q_lens is not None and sum(q_lens) == 0:
        q_lens[-1] = 2
    if sum(lens) == 0:
        lens[0] = 1
    first, last = int(rng.integers(0, 3)), int(rng.integers(1, 4))
    budget = first + last + int(rng.integers(0, 20))
    c = _case(seed, lens, q_lens, G * H_kv, H_kv, d, page, extra_pages=int(rng.integers(0, 4)))
    g = _gpu(c)
    want, want_sel = _want(c, budget, first, last)
    tables, sel = _select(c, g, budget, first, last)
    assert np.array_equal(tables.cpu().numpy(), want) and np.array_equal(sel.cpu().numpy(), want_sel)
    scale = float(np.float32(rng.uniform(0.02, 0.3)))
    o, lse, t2, s2 = attn.paged_sparse_fwd(g["q"], g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], budget, first, last,
                                           cu_seqlens_q=g["cu"], scale=scale, return_tables=True)
    attn.device_status()
    assert torch.equal(t2, tables) and torch.equal(s2, sel)
    ro, rl, bo, bl = ref.attend(c["q"].float().numpy(), c["k"].float().numpy(), c["v"].float().numpy(), want, want_sel, scale)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), empty) and np.all(o[empty] == 0)
    assert np.all(np.abs(o - ro) <= bo) and np.all(np.abs(lse[~empty] - rl[~empty]) <= bl[~empty])
