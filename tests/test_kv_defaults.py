"""Defaults of the frequency helper: each way to stretch the rotation has the ends it was published with."""
import math

import pytest
import torch

import attention_attn_fwd_03_gb300 as attn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.build()


@pytest.mark.parametrize("rot,base,factor,orig", [(128, 10000.0, 8.0, 8192), (64, 500000.0, 32.0, 4096)])
def test_ends_of_each_kind(rot, base, factor, orig):
    for kind, high in (("bands", 4.0), ("yarn", 32.0)):
        got, amp = attn.rope_inv_freq(rot, base, kind, factor, orig)
        want, want_amp = attn.rope_inv_freq(rot, base, kind, factor, orig, 1.0, high)
        assert torch.equal(got, want) and amp == want_amp
        # a chosen end replaces the default, the other one stays
        assert torch.equal(attn.rope_inv_freq(rot, base, kind, factor, orig, high=16.0)[0],
                           attn.rope_inv_freq(rot, base, kind, factor, orig, 1.0, 16.0)[0])
        assert torch.equal(attn.rope_inv_freq(rot, base, kind, factor, orig, low=2.0)[0],
                           attn.rope_inv_freq(rot, base, kind, factor, orig, 2.0, high)[0])


def test_yarn_by_default_matches_its_formula():
    """Pairs that turn 32 times or more over the original length are kept, pairs that turn at most once are
    divided, with the ramp along the pair index between them."""
    rot, base, factor, orig = 128, 10000.0, 8.0, 8192
    got, amp = attn.rope_inv_freq(rot, base, "yarn", factor, orig)
    c = [rot * math.log(orig / (2 * math.pi * n)) / (2 * math.log(base)) for n in (32.0, 1.0)]
    lo, hi = math.floor(c[0]), math.ceil(c[1])
    for i, g in enumerate(got.tolist()):
        f = base ** (-2.0 * i / rot)
        keep = 1.0 - min(max((i - lo) / (hi - lo), 0.0), 1.0)
        assert abs(g - (keep * f + (1 - keep) * f / factor)) <= 1e-13 * f
    assert abs(amp - (0.1 * math.log(factor) + 1.0)) < 1e-15


@pytest.mark.parametrize("kw", [dict(orig_len=2 ** 32 + 8192), dict(orig_len=-2 ** 31 - 1), dict(rot=2 ** 32 + 64)])
def test_sizes_past_32_bits_do_not_wrap(kw):
    with pytest.raises(ValueError):
        attn.rope_inv_freq(**dict(dict(rot=64, scaling="yarn", factor=2.0), **kw))
