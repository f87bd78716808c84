"""Scaled rotary frequencies between their ends, and their refusals (CPU only)."""
import math

import pytest

import speculative_decoding_verification_80_gb300 as sd


# Pairs of more than `fast` turns in the original context stay and those of less than `slow` are divided by the
# factor; between them the share of the divided frequency grows evenly from the pair before the one to the pair after
# the other.  Pair i of 64 values makes original * 10000^(-i / 32) / (2 pi) turns, so `turns` of them at
# i = 32 ln(original / (2 pi turns)) / ln 10000:
#   4096 tokens: 32 turns at 10.47, 1 at 22.51: pairs 10 to 23;
#   8192 tokens: 8 turns at 17.70, 2 at 22.51: pairs 17 to 23;
#   600 tokens: 100 turns at -0.16 (from 0 on), 1 at 15.84: pairs 0 to 16.
@pytest.mark.parametrize("original,fast,slow,low,high", [(4096, 32, 1, 10, 23), (8192, 8, 2, 17, 23), (600, 100, 1, 0, 16)])
def test_yarn_between_its_ends(original, fast, slow, low, high):
    plain, by = sd.rotary_frequencies(64)[0], 16.0
    for turns, near in ((fast, low), (slow, high)):
        i = 32 * math.log(original / (2 * math.pi * turns)) / math.log(10000.0)
        assert near == (max(math.floor(i), 0) if turns == fast else math.ceil(i))
    got, factor = sd.rotary_frequencies(64, scaling=dict(type="yarn", factor=by, original=original, fast=fast, slow=slow))
    assert factor == pytest.approx(0.1 * math.log(by) + 1, rel=1e-15)
    for i, (f, g) in enumerate(zip(plain, got)):
        if i <= low:
            assert g == f
        elif i >= high:
            assert g == pytest.approx(f / by, rel=1e-15)
        else:
            share = (i - low) / (high - low)
            assert g == pytest.approx(f - share * (f - f / by), rel=1e-14) and f / by < g < f


def test_yarn_attention_is_what_is_given():
    ask = lambda a: sd.rotary_frequencies(64, scaling=dict(type="yarn", factor=4, original=4096, attention=a))  # noqa: E731
    assert ask(0.5)[1] == 0.5 and ask(1)[1] == 1.0
    assert ask(None)[1] == pytest.approx(0.1 * math.log(4) + 1)
    for bad in (0, 0.0, -1.0, math.inf, math.nan):
        with pytest.raises(ValueError):
            ask(bad)
