"""The angle of a rotation: exact to the fp32 functions that take it, at any position and frequency."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import attention_attn_fwd_03_gb300 as attn

pytestmark = pytest.mark.gpu
DEV = "cuda"
PI = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.lib()


def _turned(pos, freq):
    """cos and sin of pos * freq, the angle reduced exactly and rounded once to float64."""
    c, s = np.zeros((len(pos), len(freq))), np.zeros((len(pos), len(freq)))
    for n, p in enumerate(pos):
        for i, f in enumerate(freq):
            t = Fraction(int(p)) * Fraction(float(f)) / (2 * PI)
            quarter = round(4 * t)  # the nearest quarter turn comes off exactly
            a = float((4 * t - quarter) * PI / 2)
            cs, sn = np.cos(a), np.sin(a)
            c[n, i], s[n, i] = ((cs, sn), (-sn, cs), (-cs, -sn), (sn, -cs))[quarter % 4]
    return c, s


@pytest.mark.parametrize("freq_dtype", [torch.float64, torch.float32])
def test_far_positions_lose_nothing(freq_dtype):
    """Positions to the ends of int32 and frequencies up to hundreds of turns a position."""
    pos = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 999999937, 1, -1, 0], dtype=np.int32)
    freq = torch.tensor([1.0, 0.75, 0.1, 1e-3, 3.7, 1000.3, 6.25, 1.1e-5], dtype=torch.float64).to(freq_dtype)
    g = torch.Generator().manual_seed(1)
    x = torch.randn((1, 3, len(pos), 64), generator=g)
    y, _ = attn.rope(x.to(DEV), inv_freq=freq.to(DEV), positions=torch.from_numpy(pos).to(DEV))
    attn.device_status()
    c, s = _turned(pos, freq.double().numpy())
    a, b = x[0, :, :, :8].double().numpy(), x[0, :, :, 8:16].double().numpy()
    # the functions are good to 1 ulp, two products and their sum round once each, as does the output: below
    # 2^-21 (|a| + |b|)
    tol = 2.0 ** -21 * (np.abs(a) + np.abs(b))
    got = y[0].double().cpu().numpy()
    for want, out in ((a * c - b * s, got[:, :, :8]), (a * s + b * c, got[:, :, 8:16])):
        assert np.all(np.abs(out - want) <= tol), np.max(np.abs(out - want) / tol)


@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_next_to_whole_quarter_turns(interleaved):
    """Where a cosine or a sine is small it keeps its relative accuracy: the angle is not rounded to the
    steps of fp32 half turns (2^-25 next to a half), which would be off by up to 9e-8 here."""
    off = np.array([1e-3, -3e-4, 1e-4, -7e-5, 3.3e-5, 1.7e-3, -2.9e-3, 5e-6])
    freq = np.pi / 2 + off
    pos = np.array([1, 3, 5, -1, -3, 2, 4], dtype=np.int32)
    x = torch.zeros((len(pos), 1, 64))
    x[:, :, 0:16:2 if interleaved else 1] = 1.0
    if not interleaved:
        x[:, :, 8:] = 0.0
    y, _ = attn.rope(x.to(DEV), inv_freq=torch.from_numpy(freq).to(DEV), positions=torch.from_numpy(pos).to(DEV),
                     interleaved=interleaved)
    attn.device_status()
    c, s = _turned(pos, freq)
    y = y[:, 0].double().cpu().numpy()
    got = (y[:, 0:16:2], y[:, 1:16:2]) if interleaved else (y[:, :8], y[:, 8:16])
    # 1 ulp of the function (2^-23), its correction's rounding (2^-24) and second order, (pi 2^-25)^2 / 2
    for want, out in ((c, got[0]), (s, got[1])):
        tol = (2.0 ** -23 + 2.0 ** -24) * np.abs(want) + 2.0 ** -46
        assert np.all(np.abs(out - want) <= tol), np.max(np.abs(out - want) / tol)
