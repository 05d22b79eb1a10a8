"""Page-sparse attention in one kernel against float64, with a bound that leaves no room for probabilities
in bf16: O may be off by its own rounding and by what 32-bit arithmetic brings, no more.

P enters the second product as the sum of two bf16 numbers: the first is off by at most half a step, 2^-8 p,
the second holds that difference to half a step, so P is good to 2^-16.  A score is an fp32 sum of d exact
products (d 2^-24 sum |q k|) times the scale, and the product, the scale and the difference from the maximum
round once each (3 2^-24 of the largest score in natural units); the exponential is good to 2^-22.  All
of that enters twice, in numerator and denominator.  Each accumulation rounds or truncates once per chunk
(2^-23): at most one per 64 keys for the four warps of a CTA, and the merge's 32 partials."""
import numpy as np
import pytest
import torch

import attention_attn_fwd_03_gb300 as attn

import _kv_ref as ref
from _parity import default_scale
from test_gpu_sparse import _case, _gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.lib()


@pytest.mark.parametrize("H,H_kv,d,page,budget", [
    (2, 2, 128, 16, 9), (32, 4, 128, 64, 6), (24, 2, 128, 8, 40), (48, 2, 128, 32, 100), (9, 3, 128, 16, 9),
    (8, 1, 64, 16, 9), (32, 2, 64, 32, 12), (24, 1, 64, 8, 70), (64, 2, 64, 128, 4),
])
def test_output_is_good_to_its_own_rounding(H, H_kv, d, page, budget):
    lens = [900, 1, 333, 64]
    c = _case(H + d, lens, None, H, H_kv, d, page, spread=0.3)
    g = _gpu(c)
    assert attn.attn_paged_sparse_fwd_workspace_size(len(lens), H, H_kv, d, page, c["table"].shape[1], budget) == 256
    scale = default_scale(d)
    o, _, tables, sel = attn.paged_sparse_fwd(g["q"], g["k"], g["v"], g["bt"], g["lens"], g["sk"], g["amp"], budget,
                                              scale=scale, return_tables=True)
    attn.device_status()
    o, tables, sel = o.double().cpu().numpy(), tables.cpu().numpy(), sel.cpu().numpy()
    q, k, v = (c[x].double().numpy() for x in ("q", "k", "v"))
    G = H // H_kv
    for t in range(len(lens)):
        for h in range(H_kv):
            ids = tables[t, h][tables[t, h] >= 0]
            kk, vv = k[ids][:, :, h].reshape(-1, d)[:sel[t]], v[ids][:, :, h].reshape(-1, d)[:sel[t]]
            for x in range(h * G, (h + 1) * G):
                s = scale * (kk @ q[t, x])
                p = np.exp(s - s.max())
                p /= p.sum()
                want, spread = p @ vv, p @ np.abs(vv)
                arg = scale * d * 2.0 ** -24 * (np.abs(kk) @ np.abs(q[t, x])).max() + 3 * 2.0 ** -24 * np.abs(s).max()
                e = (2.0 ** -16 + 2 * (arg + 2.0 ** -22) + (sel[t] // 64 + 1 + 32) * 2.0 ** -23) * spread
                bound = 2.0 ** -8 * (np.abs(want) + e) + e + 1e-30
                off = np.abs(o[t, x] - want)
                assert np.all(off <= bound), (t, x, np.max(off / bound))
