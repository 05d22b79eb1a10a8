"""Rotary positions (attn_rope) and the cache append (attn_paged_append) against float64.

Tolerance: the angle enters sincospi rounded to fp32 half turns (2^-25 of a half turn, 1e-7 rad), the
function is good to 1 ulp, the amplitude, two products and their sum round once each: below 2^-21
(|a| + |b|) |amplitude| for a pair (a, b).  bf16 outputs add half a step, 2^-8 of the value."""
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


def _np(t):
    return t.detach().double().cpu().numpy()


def _pair_sum(x, rot, interleaved):
    """|a| + |b| of the pair that each element belongs to (0 where nothing turns)."""
    s = np.zeros_like(x)
    if interleaved:
        s[..., 0:rot:2] = s[..., 1:rot:2] = np.abs(x[..., 0:rot:2]) + np.abs(x[..., 1:rot:2])
    else:
        s[..., :rot // 2] = s[..., rot // 2:rot] = np.abs(x[..., :rot // 2]) + np.abs(x[..., rot // 2:rot])
    return s


def _check(name, got, x, want, rot, interleaved, amplitude, extra=0.0):
    got = _np(got)
    half_step = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24
    tol = (2.0 ** -21 + extra) * abs(amplitude) * _pair_sum(_np(x), rot, interleaved) + half_step * np.abs(want) + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d off, worst %g" % (name, bad.sum(), np.max(np.abs(got - want) / tol))
    still = _pair_sum(np.ones_like(want), rot, interleaved) == 0
    assert np.array_equal(got[still], _np(x)[still])  # dims that do not turn are copied


def _heads_inside(x):
    """[B, H, N, d] -> [B, N, H, d], where positions go with the second dim."""
    return _np(x).transpose(0, 2, 1, 3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,H_k,N,d,rot,inverse,amplitude", [
    (1, 1, 1, 1, 128, 128, False, 1.0),        # one token, one head
    (2, 5, 1, 7, 64, 64, True, 1.0),
    (3, 4, 2, 61, 128, 48, False, 1.25),       # part of the head
    (1, 32, 8, 65, 128, 16, True, 0.5),
    (2, 3, 3, 1031, 64, 32, False, 1.0),       # 512 tokens or more: four to a CTA, the last CTA partial
    (3, 2, 1, 171, 64, 64, True, 1.0),         # 513
    (1, 2, 1, 511, 128, 64, False, 1.0),
    (1, 7, 2, 2051, 128, 128, True, 1.1),
    (1, 40, 0, 5, 128, 112, False, -2.0),      # q alone
])
def test_rope_matches_definition(B, H, H_k, N, d, rot, inverse, amplitude, interleaved, dtype):
    g = torch.Generator().manual_seed(N + d)
    q = torch.randn((B, H, N, d), generator=g).to(dtype).to(DEV)
    k = torch.randn((B, H_k, N, d), generator=g).to(dtype).to(DEV) if H_k else None
    f, _ = attn.rope_inv_freq(rot)
    pos = torch.randint(-5000, 100000, (B, N), generator=g, dtype=torch.int32)
    for p in (None, pos[0].contiguous(), pos):
        qo, ko = attn.rope(q, k, inv_freq=f.to(DEV), positions=None if p is None else p.to(DEV),
                           interleaved=interleaved, inverse=inverse, amplitude=amplitude)
        attn.device_status()
        at = np.arange(N) if p is None else p.numpy()
        for name, x, y in (("q", q, qo), ("k", k, ko)):
            if x is None:
                assert y is None
                continue
            want = ref.rope(_heads_inside(x), at, f.numpy(), rot, interleaved, inverse, amplitude).transpose(0, 2, 1, 3)
            _check(name, y, x, want, rot, interleaved, amplitude)


@pytest.mark.parametrize("freq_dtype", [torch.float64, torch.float32])
def test_far_positions(freq_dtype):
    """Positions up to the ends of int32: the reduced angle is as good as float64's."""
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 999999937, 0, -1], dtype=torch.int32)
    f = attn.rope_inv_freq(128, scaling="linear", factor=1.7)[0].to(freq_dtype)
    x = torch.randn((1, 2, 6, 128), generator=torch.Generator().manual_seed(1)).to(DEV)
    y, _ = attn.rope(x, inv_freq=f.to(DEV), positions=pos.to(DEV))
    want = ref.rope(_heads_inside(x), pos.numpy(), f.double().numpy(), 128).transpose(0, 2, 1, 3)
    # f / 2 pi is rounded to float64, twice (the constant and the product): P f 2^-52 rad; the
    # longdouble angle of the reference rounds at 2^-63 P f at worst
    extra = np.abs(pos.numpy().astype(np.float64))[:, None] * np.concatenate([f.double().numpy()] * 2) * 2.0 ** -51
    _check("far", y, x, want, 128, False, 1.0, extra=extra)


def test_layouts_broadcasts_and_in_place():
    """Token-major views of a fused projection, permuted dims, broadcast inputs, and outputs that replace
    their inputs, all to the bits of the dense call."""
    g = torch.Generator().manual_seed(3)
    T, H, H_k, d, rot = 37, 6, 2, 128, 64
    f = attn.rope_inv_freq(rot)[0].to(DEV)
    pos = torch.randint(0, 4000, (T,), generator=g, dtype=torch.int32).to(DEV)
    fused = torch.randn((T, (H + 2 * H_k) * d), generator=g).to(torch.bfloat16).to(DEV)
    before = fused.clone()
    q, k = fused[:, :H * d].unflatten(1, (H, d)), fused[:, H * d:(H + H_k) * d].unflatten(1, (H_k, d))
    qo, ko = attn.rope(q, k, inv_freq=f, positions=pos)
    assert torch.equal(fused, before)
    q4, k4 = attn.rope(q.transpose(0, 1)[None], k.transpose(0, 1)[None].contiguous(), inv_freq=f, positions=pos)
    assert torch.equal(q4[0].transpose(0, 1), qo) and torch.equal(k4[0].transpose(0, 1), ko)
    # outputs inside a larger buffer: the rest of it stays
    big = torch.full((T, 3 * H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    attn.rope(q, k, inv_freq=f, positions=pos, q_out=big[:, H:2 * H])
    assert torch.equal(big[:, H:2 * H], qo) and bool((big[:, :H] == 7).all()) and bool((big[:, 2 * H:] == 7).all())
    # in place on the fused buffer
    attn.rope(q, k, inv_freq=f, positions=pos, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(fused[:, (H + H_k) * d:], before[:, (H + H_k) * d:])
    # one head vector read by every head and batch entry
    one = torch.randn((1, 1, T, d), generator=g).to(DEV)
    a, _ = attn.rope(one.expand(3, 4, T, d), inv_freq=f, positions=pos)
    b, _ = attn.rope(one, inv_freq=f, positions=pos)
    assert torch.equal(a, b.expand(3, 4, T, d))
    attn.device_status()


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(interleaved):
    """The inverse call against autograd through the float64 formula, and against central differences of the
    call itself (the map is linear, so the step can be large and only rounding is left)."""
    g = torch.Generator().manual_seed(5)
    B, H, N, d, rot, amp = 2, 3, 9, 64, 48, 1.3
    f, _ = attn.rope_inv_freq(rot, scaling="bands", factor=4.0)
    x = torch.randn((B, H, N, d), generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn((B, H, N, d), generator=g)
    t = torch.arange(N, dtype=torch.float64)[:, None] * f
    c, s = torch.cos(t) * amp, torch.sin(t) * amp
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = a * c - b * s, a * s + b * c
    y = torch.cat([torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1), x[..., rot:]], -1)
    (y * w).sum().backward()
    dx, _ = attn.rope(w.to(DEV), inv_freq=f.to(DEV), interleaved=interleaved, inverse=True, amplitude=amp)
    _check("gradient", dx, w, x.grad.numpy(), rot, interleaved, amp)

    def loss(z):
        out, _ = attn.rope(z.float().to(DEV), inv_freq=f.to(DEV), interleaved=interleaved, amplitude=amp)
        return float((out.double().cpu() * w.double()).sum())
    at = x.detach().float().double()
    for i in ((0, 0, 0, 0), (1, 2, 8, 47), (0, 1, 5, 30), (1, 0, 3, 63)):
        e = torch.zeros_like(at)
        e[i] = 8.0
        diff = (loss(at + e) - loss(at - e)) / 16.0
        # every output element is off by at most 2^-21 (|a| + |b|) amp twice, weighed by |w|
        tol = 2 * 2.0 ** -21 * amp * 4 * float((w.abs() * (at.abs() + 8.0)).sum()) / 16.0
        assert abs(diff - float(dx[i])) <= tol


def test_training_step_through_rope_and_attention():
    """rope -> fwd -> bwd -> inverse rope, the gradients of the unrotated q and k, as one chain."""
    g = torch.Generator().manual_seed(9)
    B, H, N, d = 1, 2, 200, 64
    q, k, v, do = (torch.randn((B, H, N, d), generator=g).to(torch.bfloat16) for _ in range(4))
    f, _ = attn.rope_inv_freq(d)
    fd = f.to(DEV)
    qr, kr = attn.rope(q.to(DEV), k.to(DEV), inv_freq=fd)
    o, lse = attn.fwd(qr, kr, v.to(DEV), causal=True)
    dq, dk, dv = attn.bwd(qr, kr, v.to(DEV), o, lse, do.to(DEV), causal=True)
    dq, dk = attn.rope(dq, dk, inv_freq=fd, inverse=True, q_out=dq, k_out=dk)
    attn.device_status()
    x = [t.double().requires_grad_() for t in (q, k, v)]
    t = torch.arange(N, dtype=torch.float64)[:, None] * f
    c, s = torch.cos(t), torch.sin(t)

    def turn(z):
        a, b = z[..., :d // 2], z[..., d // 2:]
        return torch.cat([a * c - b * s, a * s + b * c], -1)
    p = (turn(x[0]) @ turn(x[1]).transpose(-1, -2) / d ** 0.5).masked_fill(torch.ones(N, N).triu(1).bool(), -torch.inf)
    out = torch.softmax(p, -1) @ x[2]
    out.backward(do.double())
    assert float((o.double().cpu() - out.detach()).abs().max()) <= 2e-2
    for name, got, want in (("dq", dq, x[0].grad), ("dk", dk, x[1].grad), ("dv", dv, x[2].grad)):
        # bf16 operands P, dS, rotated q and k, each half a step of 2^-8 per factor: the backward
        # tolerance of the dense tests (2% of the largest entry) covers them
        assert float((got.double().cpu() - want).abs().max()) <= 2e-2 * float(want.abs().max()), name


# ---------------------------------------------------------------- cache append

@pytest.mark.parametrize("T,H,H_kv,d,rot,page,interleaved", [
    (1, 4, 1, 128, 128, 64, False),
    (64, 32, 8, 128, 128, 64, False),
    (33, 5, 5, 64, 32, 16, True),
    (130, 8, 2, 128, 96, 8, True),
    (2500, 4, 2, 64, 64, 128, False),
    (19, 0, 3, 128, 64, 24, False),   # no queries; a page size that is no power of two
    (40, 6, 2, 128, 0, 32, False),    # nothing rotates
])
def test_append_matches_definition(T, H, H_kv, d, rot, page, interleaved):
    g = torch.Generator().manual_seed(T + d)
    pages = -(-T // page) + 3
    fused = torch.randn((T, (H + 2 * H_kv) * d), generator=g).to(torch.bfloat16).to(DEV)
    parts = fused.split([H * d, H_kv * d, H_kv * d], 1)
    q, k, v = (x.unflatten(1, (-1, d)) if x.shape[1] else None for x in parts)
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    skipped = torch.rand(T, generator=g) < 0.2
    slots[skipped] = -1 - torch.randint(0, 100, (int(skipped.sum()),), generator=g, dtype=torch.int32)
    pos = torch.randint(0, 70000, (T,), generator=g, dtype=torch.int32)
    f = attn.rope_inv_freq(rot)[0] if rot else None
    kc = torch.full((pages, page, H_kv, d), 3.0, dtype=torch.bfloat16, device=DEV)
    vc = torch.full_like(kc, 4.0)
    qo = torch.full((T, H, d), 5.0, dtype=torch.bfloat16, device=DEV) if H else None
    got = attn.paged_append(q, k, v, kc, vc, slots.to(DEV), positions=pos.to(DEV) if rot else None,
                            inv_freq=f.to(DEV) if rot else None, interleaved=interleaved, amplitude=1.2, q_out=qo)
    attn.device_status()
    assert got is qo
    ok = ~skipped
    at = slots[ok].long()

    def turned(x):
        return ref.rope(_np(x), pos.numpy(), f.numpy(), rot, interleaved, False, 1.2) if rot else _np(x)
    flat_k, flat_v = kc.flatten(0, 1).cpu(), vc.flatten(0, 1).cpu()
    _check("k", flat_k[at], k[ok.to(DEV)], turned(k)[ok.numpy()], rot, interleaved, 1.2)
    assert torch.equal(flat_v[at], v.cpu()[ok])
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[at] = False
    assert bool((flat_k[rest] == 3).all()) and bool((flat_v[rest] == 4).all())
    if H:
        _check("q", qo[ok.to(DEV)], q[ok.to(DEV)], turned(q)[ok.numpy()], rot, interleaved, 1.2)
        assert bool((qo.cpu()[skipped] == 5).all())


def test_append_in_place_and_as_two_calls():
    g = torch.Generator().manual_seed(2)
    T, H, H_kv, d = 50, 4, 2, 128
    q, k, v = (torch.randn((T, h, d), generator=g).to(torch.bfloat16).to(DEV) for h in (H, H_kv, H_kv))
    slots = torch.randperm(128, generator=g)[:T].to(torch.int32).to(DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    f = attn.rope_inv_freq(d)[0].to(DEV)
    kc, vc = (torch.zeros((2, 64, H_kv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    qr, kr = attn.rope(q, k, inv_freq=f, positions=pos)
    attn.paged_append(q, k, v, kc, vc, slots, positions=pos, inv_freq=f, q_out=q)
    attn.device_status()
    assert torch.equal(q, qr) and torch.equal(kc.flatten(0, 1)[slots.long()], kr)
    assert torch.equal(vc.flatten(0, 1)[slots.long()], v)


def test_append_reports_slots_past_the_cache():
    d = 64
    x = torch.ones((3, 1, d), dtype=torch.bfloat16, device=DEV)
    kc = torch.zeros((2, 8, 1, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    attn.paged_append(None, x, x, kc, vc, torch.tensor([3, 16, 2 ** 31 - 1], dtype=torch.int32, device=DEV))
    with pytest.raises(attn.AttnError) as e:
        attn.device_status()
    assert e.value.status == attn.ATTN_ERR_DEVICE_DATA
    attn.device_status()
    assert float(kc.float().sum()) == d and bool((kc.flatten(0, 1)[3] == 1).all())


def test_append_past_32_bit_offsets():
    """A cache of more than 2^32 elements: slots near its end."""
    H_kv, d, page, pages = 8, 128, 64, 66000
    kc = torch.empty((pages, page, H_kv, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    slots = torch.tensor([pages * page - 1, 0, 65536 * page + 5], dtype=torch.int32, device=DEV)
    kc.flatten(0, 1)[slots.long()] = 0
    x = torch.randn((3, H_kv, d), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).to(DEV)
    attn.paged_append(None, x, x * 2, kc, vc, slots)
    attn.device_status()
    assert torch.equal(kc.flatten(0, 1)[slots.long()], x) and torch.equal(vc.flatten(0, 1)[slots.long()], x * 2)


def test_helpers_refuse():
    q = torch.zeros((2, 4, 3, 128), dtype=torch.bfloat16, device=DEV)
    f = attn.rope_inv_freq(128)[0].to(DEV)
    with pytest.raises(TypeError):
        attn.rope(q.half(), inv_freq=f)
    with pytest.raises(TypeError):
        attn.rope(q, q.float(), inv_freq=f)
    with pytest.raises(TypeError):
        attn.rope(q, inv_freq=f.half())
    with pytest.raises(TypeError):
        attn.rope(q, inv_freq=f.cpu())
    with pytest.raises(ValueError):
        attn.rope(q, inv_freq=f, positions=torch.zeros(4, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        attn.rope(q[..., ::2], inv_freq=f[:32])
    with pytest.raises(attn.AttnError):  # outputs that share memory
        attn.rope(q, inv_freq=f, q_out=q[:1].expand(2, 4, 3, 128))
    with pytest.raises(attn.AttnError):  # rot beyond the head
        attn.rope(q[..., :64].contiguous(), inv_freq=f)
    with pytest.raises(ValueError):
        attn.paged_append(None, q[0], q[0], q, q, torch.zeros(4, dtype=torch.int32, device=DEV), inv_freq=f)


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    """Seeded shapes, strides and types of rope, and the same rotation through the cache append."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if seed % 3 else torch.float32
    d = int(rng.choice([64, 128]))
    rot = int(rng.integers(1, d // 16 + 1)) * 16
    B, N, H, H_k = int(rng.integers(1, 4)), int(rng.choice([1, 3, 30, 400])), int(rng.integers(1, 20)), int(rng.integers(1, 6))
    interleaved, inverse, amp = bool(rng.integers(2)), bool(rng.integers(2)), float(rng.uniform(-2, 2))
    f = attn.rope_inv_freq(rot, base=float(rng.choice([10000.0, 500000.0])))[0]
    pos = torch.randint(-10, 200000, (B, N), generator=g, dtype=torch.int32)
    order = [(0, 1, 2, 3), (0, 2, 1, 3), (2, 0, 1, 3), (1, 0, 2, 3)][int(rng.integers(4))]

    def tensor(heads):  # [B, heads, N, d] stored in another order, inside a wider row
        dims = [(B, heads, N, d + 16)[i] for i in order]
        x = torch.randn(dims, generator=g).to(dt).to(DEV)
        return x.permute([order.index(i) for i in range(4)])[..., :d]
    q, k = tensor(H), tensor(H_k)
    q_out, k_out = tensor(H), None
    qo, ko = attn.rope(q, k, inv_freq=f.to(DEV), positions=pos.to(DEV), interleaved=interleaved, inverse=inverse, amplitude=amp,
                       q_out=q_out, k_out=k_out)
    attn.device_status()
    assert qo is q_out
    for name, x, y in (("q", q, qo), ("k", k, ko)):
        want = ref.rope(_heads_inside(x), pos.numpy(), f.numpy(), rot, interleaved, inverse, amp).transpose(0, 2, 1, 3)
        _check(name, y, x, want, rot, interleaved, amp)
    if dt is torch.bfloat16 and not inverse:
        page, T = int(rng.choice([8, 24, 64, 1024])), B * N
        pages = -(-T // page) + 1
        slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32).to(DEV)
        kc, vc = (torch.zeros((pages, page, H_k, d), dtype=dt, device=DEV) for _ in range(2))
        rows = k.permute(0, 2, 1, 3).reshape(T, H_k, d)
        got = attn.paged_append(q.permute(0, 2, 1, 3).reshape(T, H, d), rows, rows, kc, vc, slots, positions=pos.reshape(-1).to(DEV),
                                inv_freq=f.to(DEV), interleaved=interleaved, amplitude=amp)
        attn.device_status()
        assert torch.equal(got, qo.permute(0, 2, 1, 3).reshape(T, H, d))
        assert torch.equal(kc.flatten(0, 1)[slots.long()], ko.permute(0, 2, 1, 3).reshape(T, H_k, d))
        assert torch.equal(vc.flatten(0, 1)[slots.long()], rows)
