"""The cache operators around paged attention, case by case: rotary positions, page plans, cache
appends, page sketches and page-sparse decode, in a plain form and through the library's entry points.

With ``own`` false ``run`` computes each operator with elementary torch operations; with ``own`` true it
makes the library's calls on the same inputs.  ``exact`` computes the same outputs in 64 bits.
"""
import math

import torch

own = False

_DEV = "cuda"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one 32768-token training row, 32 query and 8 KV heads, positions far into a stretched context
        dict(name="rope_long", op="rope", dtype="bf16", B=1, H=32, H_kv=8, N=32768, d=128, rot=128, interleaved=False,
             inverse=False, scaling="bands", factor=8.0, start=98304),
        # gradient of a batch whose upstream gradient is kept in 32 bits: half of the head rotates, pairs adjacent
        dict(name="rope_grad", op="rope", dtype="fp32", B=4, H=16, H_kv=16, N=1999, d=128, rot=64, interleaved=True,
             inverse=True, scaling="none", factor=1.0, start=0),
        # the serving loop's step: 64 requests with one new token each
        dict(name="plan_decode", op="plan", B=64, new_lo=1, new_hi=1, ctx_lo=511, ctx_hi=8191, page=64, max_pages=128,
             pad=0),
        # admission of a ragged batch of prompts and chunks, padded to a fixed token count
        dict(name="plan_chunks", op="plan", B=200, new_lo=0, new_hi=511, ctx_lo=0, ctx_hi=4000, page=16, max_pages=300,
             pad=333),
        # one new token for each of 64 requests, split out of a fused projection
        dict(name="append_decode", op="append", T=64, H=32, H_kv=8, d=128, rot=128, page=64, pad=0),
        # eight prompts' chunks of 2048 tokens in one launch, the batch padded
        dict(name="append_chunk", op="append", T=16301, H=32, H_kv=8, d=128, rot=128, page=64, pad=83),
        # the pages that one decode step has touched
        dict(name="sketch_decode", op="sketch", B=64, H_kv=8, d=128, page=64, max_pages=128, len_lo=512, len_hi=8192,
             new=1),
        # every page of prompts just loaded
        dict(name="sketch_load", op="sketch", B=8, H_kv=8, d=128, page=64, max_pages=128, len_lo=6144, len_hi=8192,
             new=8192),
        # a single conversation: latency
        dict(name="sparse_one", op="sparse", B=1, H=32, H_kv=8, d=128, page=64, max_pages=512, len_lo=32000,
             len_hi=32768, q_hi=1, budget=32, first=1, last=2),
        # a serving batch of mixed lengths, short ones below the budget among them
        dict(name="sparse_batch", op="sparse", B=32, H=32, H_kv=8, d=128, page=64, max_pages=1024, len_lo=0,
             len_hi=65536, q_hi=1, budget=64, first=1, last=2),
        # several drafted tokens per request, small pages, 64-wide heads
        dict(name="sparse_verify", op="sparse", B=16, H=16, H_kv=2, d=64, page=16, max_pages=1024, len_lo=9,
             len_hi=16384, q_hi=8, budget=128, first=1, last=4),
        # four very long documents
        dict(name="sparse_long", op="sparse", B=4, H=32, H_kv=8, d=128, page=64, max_pages=4096, len_lo=200000,
             len_hi=262144, q_hi=1, budget=128, first=1, last=2),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "plan", "append", "sketch", "sparse", "sparse"])
    H_kv = rng.choice([1, 2, 4, 8])
    H = H_kv * rng.choice([1, 2, 4, 5, 8])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        B = rng.choice([1, 2, 3, 4])
        N = _log_int(rng, 1, 8192 // B)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]), B=B, H=H, H_kv=H_kv, N=N, d=d,
                    rot=rng.choice([d, d, d // 2, 16, 48]), interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "bands", "yarn"]), factor=rng.uniform(1.5, 16.0),
                    start=_log_int(rng, 1, 500000))
    if op == "plan":
        B = _log_int(rng, 1, 1024)
        hi = _log_int(rng, 1, max(2, 65536 // B))
        ctx = _log_int(rng, 1, 8000)
        return dict(op=op, B=B, new_lo=rng.choice([0, 1]), new_hi=hi, ctx_lo=rng.choice([0, ctx // 2]), ctx_hi=ctx,
                    page=page, max_pages=-(-(ctx + hi) // page) + rng.randint(0, 5), pad=rng.choice([0, rng.randint(1, 500)]))
    if op == "append":
        return dict(op=op, T=_log_int(rng, 1, 16000), H=H, H_kv=H_kv, d=d, rot=rng.choice([d, d, d // 2, 32]), page=page,
                    pad=rng.choice([0, rng.randint(1, 100)]))
    B = _log_int(rng, 1, 64)
    if op == "sketch":
        hi = _log_int(rng, 16, max(64, 65536 // B))
        return dict(op=op, B=B, H_kv=H_kv, d=d, page=page, max_pages=-(-hi // page) + rng.randint(0, 3),
                    len_lo=rng.choice([0, hi // 2]), len_hi=hi, new=rng.choice([1, 1, rng.randint(2, 600), hi]))
    hi = _log_int(rng, 64, max(128, 262144 // B))
    budget = _log_int(rng, 4, 128)
    q_hi = rng.choice([1, 1, rng.randint(2, 6)])
    return dict(op=op, B=B, H=H, H_kv=H_kv, d=d, page=page, max_pages=-(-hi // page) + rng.randint(0, 3),
                len_lo=rng.choice([0 if q_hi == 1 else q_hi, hi // 2]), len_hi=hi, q_hi=q_hi, budget=budget,
                first=rng.randint(0, 1), last=rng.randint(1, min(3, budget - 1)))


# ---------------------------------------------------------------- inputs

def _freqs(case, base=10000.0):
    """Angle per position of each rotated pair, float64 [rot / 2] on the GPU, and the amplitude factor."""
    rot, s = case["rot"], case.get("factor", 1.0)
    i = torch.arange(rot // 2, dtype=torch.float64)
    kind = case.get("scaling", "none")
    if kind == "ntk" and rot > 2:
        base = base * s ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    amp = 1.0
    if kind == "linear":
        f = f / s
    elif kind == "bands":
        t = ((8192 * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = f * (t + (1 - t) / s)
    elif kind == "yarn":
        dim = [rot * math.log(8192 / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32.0, 1.0)]
        lo, hi = max(math.floor(dim[0]), 0), min(math.ceil(dim[1]), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - ramp) + f / s * ramp
        amp = 0.1 * math.log(s) + 1.0
    return f.to(_DEV), amp


def _lens(g, lo, hi, n):
    """n lengths spread evenly over [lo, hi] in an order of the seed's: their sum is the case's own."""
    spread = lo + (torch.arange(n, dtype=torch.float64) + 0.5) * (hi - lo) / n
    return spread.round().long()[torch.randperm(n, generator=g)]


def _tables(g, pages, max_pages):
    """Block table of requests that hold pages[r] pages each, drawn from a shuffled pool, and the pool's size."""
    pool = int(pages.sum()) + 8
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    start = torch.cumsum(pages, 0) - pages
    j = torch.arange(max_pages)
    at = (start[:, None] + j).clamp(max=pool - 1)
    table = torch.where(j < pages[:, None], perm[at], torch.full((), -1, dtype=torch.int32))
    return table, pool, perm


def _keys(gd, pool, page, H_kv, d):
    """Keys that differ from page to page, as those of a text do: a page's own direction and noise."""
    topic = torch.randn((pool, 1, H_kv, d), generator=gd, device=_DEV) * 0.7
    k = torch.randn((pool, page, H_kv, d), generator=gd, device=_DEV, dtype=torch.bfloat16)
    return k.add_(topic.to(torch.bfloat16))


def _sketch_of(k_pages):
    """Max and min codes and amplitude of whole pages [n, page, H_kv, d]."""
    hi, lo = k_pages.amax(1).float(), k_pages.amin(1).float()
    amp = torch.maximum(hi.abs(), lo.abs()).amax(-1)
    code = torch.round(torch.cat([hi, lo], -1) / amp[..., None] * 127.0)
    return torch.where(amp[..., None] > 0, code, 0.0).to(torch.int8), amp


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device=_DEV).manual_seed(seed)
    op = case["op"]
    st = {"case": case, "op": op}
    if op == "rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        B, N, d = case["B"], case["N"], case["d"]
        st["q"] = torch.randn((B, case["H"], N, d), generator=gd, device=_DEV, dtype=dt)
        st["k"] = torch.randn((B, case["H_kv"], N, d), generator=gd, device=_DEV, dtype=dt)
        st["positions"] = (case["start"] + torch.arange(N, dtype=torch.int32)).to(_DEV)
        st["inv_freq"], st["amplitude"] = _freqs(case)
    elif op == "plan":
        B, page, mp = case["B"], case["page"], case["max_pages"]
        ctx, new = _lens(g, case["ctx_lo"], case["ctx_hi"], B), _lens(g, case["new_lo"], case["new_hi"], B)
        held, want = -(-ctx // page), -(-(ctx + new) // page)
        st["total"] = int(new.sum()) + case["pad"] or 1
        table, pool, perm = _tables(g, want, mp)
        free = torch.cat([table[r, held[r]:want[r]] for r in range(B)] + [perm[-8:]])
        table[torch.arange(mp) >= held[:, None]] = -1
        free = free[torch.randperm(free.numel(), generator=g)]
        st["num_pages"] = pool
        st["count"] = torch.tensor([free.numel()], dtype=torch.int32, device=_DEV)
        st["ctx"], st["new"] = ctx.to(torch.int32).to(_DEV), new.to(torch.int32).to(_DEV)
        st["table"], st["free"] = table.to(_DEV), free.to(_DEV)
    elif op == "append":
        T, H, H_kv, d, page, n = (case[x] for x in ("T", "H", "H_kv", "d", "page", "T"))
        rows = T + case["pad"]
        pool = -(-T // page) + 4
        st["qkv"] = torch.randn((rows, (H + 2 * H_kv) * d), generator=gd, device=_DEV, dtype=torch.bfloat16)
        st["k_cache"] = torch.randn((pool, page, H_kv, d), generator=gd, device=_DEV, dtype=torch.bfloat16)
        st["v_cache"] = torch.randn((pool, page, H_kv, d), generator=gd, device=_DEV, dtype=torch.bfloat16)
        # pages are scattered, tokens within a page follow one another
        base = torch.randperm(pool, generator=g)[: -(-T // page)] * page
        slots = (base[:, None] + torch.arange(page)).reshape(-1)[:T]
        st["slots"] = torch.cat([slots, torch.full((case["pad"],), -1)]).to(torch.int32).to(_DEV)
        st["positions"] = (int(torch.randint(100000, (1,), generator=g)) + torch.arange(rows, dtype=torch.int32)).to(_DEV)
        st["q_out"] = torch.zeros((rows, H, d), dtype=torch.bfloat16, device=_DEV)
        st["inv_freq"], _ = _freqs(case)
        st["n"] = n
    else:
        B, H_kv, d, page, mp = (case[x] for x in ("B", "H_kv", "d", "page", "max_pages"))
        lens = _lens(g, case["len_lo"], case["len_hi"], B)
        pages = -(-lens // page)
        table, pool, _ = _tables(g, pages, mp)
        st["table"], st["lens"] = table.to(_DEV), lens.to(torch.int32).to(_DEV)
        st["k_cache"] = _keys(gd, pool, page, H_kv, d)
        if op == "sketch":
            new = torch.minimum(lens, torch.tensor(case["new"]))
            before = torch.where(new > 0, (lens - new) // page, pages)
            owner = torch.repeat_interleave(torch.arange(B), pages - before)
            nth = torch.arange(owner.numel()) - (torch.cumsum(pages - before, 0) - (pages - before))[owner] + before[owner]
            # the pages the call covers, as a scheduler knows them: page ids and valid rows of each
            st["touched"] = table[owner, nth].long().to(_DEV)
            st["rows"] = (lens[owner] - nth * page).clamp(max=page).to(_DEV)
            st["sketch"] = torch.zeros((pool, H_kv, 2 * d), dtype=torch.int8, device=_DEV)
            st["amp"] = torch.zeros((pool, H_kv), dtype=torch.float32, device=_DEV)
        else:
            st["v_cache"] = torch.randn((pool, page, H_kv, d), generator=gd, device=_DEV, dtype=torch.bfloat16)
            st["sketch"], st["amp"] = _sketch_of(st["k_cache"])
            q_len = _lens(g, 1, case["q_hi"], B)
            cu = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(q_len, 0)])
            T = int(cu[-1])
            st["q"] = torch.randn((T, case["H"], d), generator=gd, device=_DEV, dtype=torch.bfloat16) * 2
            st["cu"] = cu.to(torch.int32).to(_DEV) if case["q_hi"] > 1 else None
            st["o"] = torch.zeros((T, case["H"], d), dtype=torch.bfloat16, device=_DEV)
            st["lse"] = torch.zeros((T, case["H"]), dtype=torch.float32, device=_DEV)
    return st


# ---------------------------------------------------------------- plain forms

def _angles(positions, inv_freq):
    a = positions.double()[:, None] * inv_freq
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, cos, sin, rot, interleaved):
    """x [..., d] with cos, sin broadcast to [..., rot / 2]; 32 bits in, 32 bits out."""
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        out = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = r[..., : rot // 2], r[..., rot // 2:]
        out = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([out, rest], -1)


def _plain_rope(st):
    c = st["case"]
    cos, sin = _angles(st["positions"], st["inv_freq"])
    cos, sin = cos * st["amplitude"], sin * (-st["amplitude"] if c["inverse"] else st["amplitude"])
    return [_rotate(x.float(), cos, sin, c["rot"], c["interleaved"]).to(x.dtype) for x in (st["q"], st["k"])]


def _plain_plan(st):
    c, page, total = st["case"], st["case"]["page"], st["total"]
    ctx, new, table = st["ctx"].long(), st["new"].long(), st["table"]
    cu = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    held = (ctx + page - 1) // page
    want = (ctx + new + page - 1) // page
    before = torch.cumsum(want - held, 0) - (want - held)  # pages given to earlier requests
    t = torch.arange(total, device=_DEV)
    r = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=c["B"] - 1)
    valid = t < cu[-1]
    pos = ctx[r] + t - cu[r]
    pi = pos // page
    fresh = pi >= held[r]
    last = st["free"].numel() - 1
    taken = (st["count"] - 1 - (before[r] + pi - held[r])).clamp(min=0, max=last)
    old = table[r, pi.clamp(max=c["max_pages"] - 1)].long()
    ids = torch.where(fresh, st["free"][taken].long(), old)
    j = torch.arange(c["max_pages"], device=_DEV)
    given = (j >= held[:, None]) & (j < want[:, None])
    at = (st["count"] - 1 - (before[:, None] + j - held[:, None])).clamp(min=0, max=last)
    table.copy_(torch.where(given, st["free"][at], table))
    slots = torch.where(valid, ids * page + pos % page, -1).int()
    left = st["count"] - (want - held).sum(0, keepdim=True).int()
    return [cu.int(), (ctx + new).int(), torch.where(valid, pos, 0).int(), slots, table, left.int()]


def _qkv(st):
    c, x = st["case"], st["qkv"]
    H, H_kv, d = c["H"], c["H_kv"], c["d"]
    return [y.unflatten(1, (-1, d)) for y in x.split([H * d, H_kv * d, H_kv * d], 1)]


def _plain_append(st):
    c, n = st["case"], st["n"]
    q, k, v = _qkv(st)
    cos, sin = _angles(st["positions"][:n], st["inv_freq"])
    cos, sin, at = cos[:, None], sin[:, None], st["slots"][:n].long()
    st["q_out"][:n] = _rotate(q[:n].float(), cos, sin, c["rot"], False).to(torch.bfloat16)
    st["k_cache"].flatten(0, 1)[at] = _rotate(k[:n].float(), cos, sin, c["rot"], False).to(torch.bfloat16)
    st["v_cache"].flatten(0, 1)[at] = v[:n]
    return [st["q_out"], st["k_cache"], st["v_cache"]]


def _plain_sketch(st):
    k = st["k_cache"][st["touched"]].float()
    there = (torch.arange(st["case"]["page"], device=_DEV) < st["rows"][:, None])[:, :, None, None]
    hi = torch.where(there, k, -torch.inf).amax(1)
    lo = torch.where(there, k, torch.inf).amin(1)
    amp = torch.maximum(hi.abs(), lo.abs()).amax(-1)
    code = torch.round(torch.cat([hi, lo], -1) / amp[..., None] * 127.0)
    st["sketch"][st["touched"]] = torch.where(amp[..., None] > 0, code, 0.0).to(torch.int8)
    st["amp"][st["touched"]] = amp
    return [st["sketch"], st["amp"]]


def _plain_sparse(st):
    c = st["case"]
    H, H_kv, d, page, budget = c["H"], c["H_kv"], c["d"], c["page"], c["budget"]
    q, table = st["q"], st["table"].long()
    T, G, P = q.shape[0], H // H_kv, table.shape[1]
    t = torch.arange(T, device=_DEV)
    if st["cu"] is None:
        r, pos = t, st["lens"].long() - 1
    else:
        cu = st["cu"].long()
        r = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=c["B"] - 1)
        pos = st["lens"].long()[r] - cu[r + 1] + t
    n_vis = pos // page + 1
    # scores: 8-bit codes of the query against the pages' extreme codes
    qg = q.float().view(T, H_kv, G, d)
    q_amp = qg.abs().amax(-1, keepdim=True)
    code = torch.where(q_amp > 0, torch.round(qg / q_amp * 127.0), 0.0)
    code = torch.cat([code.clamp(min=0), code.clamp(max=0)], -1)
    ids = table[r].clamp(min=0)
    dots = torch.einsum("thgc,tphc->thgp", code, st["sketch"][ids].float())
    score = (q_amp * dots).amax(2) * st["amp"][ids].transpose(1, 2)
    j = torch.arange(P, device=_DEV)
    kept = (j < c["first"]) | (j >= (n_vis - c["last"])[:, None])
    score = torch.where(kept[:, None], torch.inf, score)
    score = torch.where((j < n_vis[:, None])[:, None], score, -torch.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :budget]
    n_sel = n_vis.clamp(max=budget)
    k = torch.arange(order.shape[-1], device=_DEV)
    order = torch.sort(torch.where(k < n_sel[:, None, None], order, P), dim=-1).values
    there = order < P
    tables = torch.where(there, table[r[:, None, None], order.clamp(max=P - 1)], -1)
    tables = torch.nn.functional.pad(tables, (0, budget - tables.shape[-1]), value=-1).int()
    sel_lens = torch.where(n_sel > 0, (n_sel - 1) * page + pos % page + 1, 0)
    # attention over the chosen pages
    at = tables[..., : order.shape[-1]].long().clamp(min=0)
    head = torch.arange(H_kv, device=_DEV)[:, None]
    kk = st["k_cache"].transpose(1, 2)[at, head].flatten(2, 3).float()
    vv = st["v_cache"].transpose(1, 2)[at, head].flatten(2, 3).float()
    s = torch.einsum("thgc,thkc->thgk", qg, kk) / math.sqrt(d)
    seen = (torch.arange(s.shape[-1], device=_DEV) < sel_lens[:, None])[:, None, None]
    s = torch.where(seen, s, -torch.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m > -torch.inf, m, 0.0)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = torch.einsum("thgk,thkc->thgc", p, vv) / torch.where(l > 0, l, 1.0)
    lse = (m + torch.log(l)).view(T, H)
    return [o.view(T, H, d).to(torch.bfloat16), lse, tables, sel_lens.int()]


# ---------------------------------------------------------------- one pass

def _own(st):
    import attention_attn_fwd_03_gb300 as attn
    c, op = st["case"], st["op"]
    if op == "rope":
        return attn.rope(st["q"], st["k"], inv_freq=st["inv_freq"], positions=st["positions"],
                         interleaved=c["interleaved"], inverse=c["inverse"], amplitude=st["amplitude"])
    if op == "plan":
        cu, lens, pos, slots, left = attn.paged_plan(st["ctx"], st["table"], st["free"], st["count"], c["page"],
                                                     st["num_pages"], st["total"], new_lens=st["new"])
        return [cu, lens, pos, slots, st["table"], left]
    if op == "append":
        q, k, v = _qkv(st)
        attn.paged_append(q, k, v, st["k_cache"], st["v_cache"], st["slots"], positions=st["positions"],
                          inv_freq=st["inv_freq"], q_out=st["q_out"])
        return [st["q_out"], st["k_cache"], st["v_cache"]]
    if op == "sketch":
        attn.page_sketch(st["k_cache"], st["table"], st["lens"], st["sketch"], st["amp"], max_q_len=c["new"])
        return [st["sketch"], st["amp"]]
    o, lse, tables, sel_lens = attn.paged_sparse_fwd(
        st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"], st["sketch"], st["amp"], c["budget"],
        first=c["first"], last=c["last"], cu_seqlens_q=st["cu"], out=st["o"], lse=st["lse"], return_tables=True)
    return [o, lse, tables, sel_lens]


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "plan": _plain_plan, "append": _plain_append, "sketch": _plain_sketch,
            "sparse": _plain_sparse}[state["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def _mean(case, lo, hi):
    return (case[lo] + case[hi]) / 2


def work(case):
    op = case["op"]
    if op == "rope":
        x = case["B"] * case["N"] * (case["H"] + case["H_kv"]) * case["d"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * x * size + 4 * case["N"] + 4 * case["rot"], "flops": 3 * x * case["rot"] / case["d"]}
    if op == "plan":
        tokens = case["B"] * _mean(case, "new_lo", "new_hi")
        pages = tokens / case["page"]
        # lengths in; offsets and lengths out; a position and a slot per token; page ids taken and entered
        return {"bytes": 16 * case["B"] + 8 * (tokens + case["pad"]) + 8 * pages + 4 * case["B"], "flops": 4 * tokens}
    if op == "append":
        x = case["T"] * (case["H"] + 2 * case["H_kv"]) * case["d"]
        return {"bytes": 4 * x + 8 * case["T"] + 4 * case["rot"],
                "flops": 3 * case["T"] * (case["H"] + case["H_kv"]) * case["rot"]}
    length = _mean(case, "len_lo", "len_hi")
    if op == "sketch":
        page = case["page"]
        rows = min(case["new"] + (page - 1) / 2, length)
        x = case["B"] * rows * case["H_kv"] * case["d"]
        return {"bytes": 2 * x + x / page * 2 + case["B"] * 8, "flops": 2 * x}
    T = case["B"] * (1 + case["q_hi"]) / 2
    row = case["H_kv"] * case["d"]
    pages = length / case["page"]
    sketch = case["B"] * pages * (2 * row + 4 * case["H_kv"] + 4)
    keys = case["B"] * min(length, (1 + case["q_hi"]) / 2 * case["budget"] * case["page"])
    each = T * min(length, case["budget"] * case["page"])
    io = 4 * T * case["H"] * case["d"] + 4 * T * case["H"] + 4 * T * case["H_kv"] * case["budget"]
    return {"bytes": sketch + 4 * keys * row + io,
            "flops": 4 * each * case["H"] * case["d"] + 4 * T * pages * case["H"] * case["d"]}


# ---------------------------------------------------------------- the definitions in 64 bits

def _turned(x, positions, freq, rot, interleaved, sign=1.0, amplitude=1.0):
    """Each pair (a, b) as the complex number a + ib, times amplitude * exp(i * sign * position * freq)."""
    y = x.double().clone()
    pairs = [(2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2) for i in range(rot // 2)]
    a, b = (torch.tensor([p[n] for p in pairs], device=_DEV) for n in (0, 1))
    z = torch.complex(y[..., a], y[..., b]) * torch.polar(
        torch.full_like(freq, amplitude).expand(positions.numel(), -1), sign * positions.double()[:, None] * freq)
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_sparse(st):
    c = st["case"]
    H, H_kv, d, page, budget = c["H"], c["H_kv"], c["d"], c["page"], c["budget"]
    G, T = H // H_kv, st["q"].shape[0]
    lens, table = st["lens"].tolist(), st["table"]
    cu = st["cu"].tolist() if st["cu"] is not None else list(range(T + 1))
    o = torch.zeros((T, H, d), dtype=torch.float64, device=_DEV)
    lse = torch.full((T, H), -torch.inf, dtype=torch.float64, device=_DEV)
    for r in range(c["B"]):
        for t in range(cu[r], cu[r + 1]):
            pos = lens[r] - (cu[r + 1] - t)
            if pos < 0:
                continue
            n = pos // page + 1
            mine = table[r, :n].long()
            for h in range(H_kv):
                q = st["q"][t, h * G:(h + 1) * G]
                chosen = list(range(n))
                if n > budget:
                    best = None
                    sk = st["sketch"][mine, h].double()
                    for x in q.float():  # the scores, in the 32-bit steps that define them
                        top = x.abs().max()
                        code = torch.round(x / top * 127).double() if top > 0 else x.double() * 0
                        value = top * (sk[:, :d] @ code.clamp(min=0) + sk[:, d:] @ code.clamp(max=0)).float()
                        best = value if best is None else torch.maximum(best, value)
                    score = (best * st["amp"][mine, h]).tolist()
                    always = set(range(c["first"])) | set(range(n - c["last"], n))
                    rest = sorted((p for p in range(n) if p not in always), key=lambda p: -score[p])
                    chosen = sorted(always | set(rest[: budget - len(always)]))
                at = mine[torch.tensor(chosen, device=_DEV)]
                seen = (len(chosen) - 1) * page + pos % page + 1
                k = st["k_cache"][at, :, h].reshape(-1, d)[:seen].double()
                v = st["v_cache"][at, :, h].reshape(-1, d)[:seen].double()
                s = q.double() @ k.T / math.sqrt(d)
                lse[t, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
                o[t, h * G:(h + 1) * G] = torch.softmax(s, -1) @ v
    return [o, lse, None, None]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None
    if op == "rope":
        sign = -1.0 if case["inverse"] else 1.0
        return [_turned(st[x], st["positions"], st["inv_freq"], case["rot"], case["interleaved"], sign, st["amplitude"])
                for x in ("q", "k")]
    if op == "append":
        n, H, H_kv, d = st["n"], case["H"], case["H_kv"], case["d"]
        rows = st["qkv"][:n].view(n, H + 2 * H_kv, d).transpose(0, 1)
        turned = _turned(rows[: H + H_kv], st["positions"][:n], st["inv_freq"], case["rot"], False).transpose(0, 1)
        q = st["q_out"].double()
        q[:n] = turned[:, :H]
        out = [q]
        for name, new in (("k_cache", turned[:, H:]), ("v_cache", rows[H + H_kv:].transpose(0, 1).double())):
            cache = st[name].double()
            page = st["slots"][:n].long() // case["page"], st["slots"][:n].long() % case["page"]
            cache[page] = new
            out.append(cache)
        return out
    if op == "sketch":
        amp = st["amp"].double()
        for p, n in zip(st["touched"].tolist(), st["rows"].tolist()):
            amp[p] = st["k_cache"][p, :n].double().abs().amax(0).amax(-1)
        return [None, amp]
    if case["B"] * (1 + case["q_hi"]) // 2 * case["H_kv"] > 2000:
        return None
    return _exact_sparse(st)
