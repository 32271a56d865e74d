"""Frequencies of stretched contexts, every pair against the definition in Python's floats."""
import math

import pytest

import flash_attention_forward_gb300 as fa


def blended(dim, base, factor, length, fast, slow):
    """By the number of turns within `length` positions: the pair that turns `turns` times has the index
    i = dim ln(length / (2 pi turns)) / (2 ln base)."""
    ends = [dim * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (fast, slow)]
    lo, hi = max(0, math.floor(ends[0])), min(dim - 1, math.ceil(ends[1]))
    out = []
    for i in range(dim // 2):
        w = 0.0 if i <= lo else 1.0 if i >= hi else (i - lo) / (hi - lo)
        plain = base ** (-2.0 * i / dim)
        out.append((1.0 - w) * plain + w * plain / factor)
    return out, lo, hi


@pytest.mark.parametrize("dim,base,factor,length,fast,slow", [(64, 10000.0, 32.0, 4096, 32.0, 1.0), (128, 500000.0, 8.0, 8192, 32.0, 1.0),
                                                              (64, 10000.0, 40.0, 4096, 32.0, 1.0), (16, 10000.0, 4.0, 512, 16.0, 2.0),
                                                              (64, 10000.0, 2.0, 20, 32.0, 1.0), (32, 10.0, 3.0, 2000, 32.0, 1.0),
                                                              (64, 10000.0, 1.0, 4096, 32.0, 1.0)])
def test_blended_frequencies(dim, base, factor, length, fast, slow):
    got, attention = fa.sdpa_rope_frequencies(dim, base=base, scaling="by_parts", factor=factor, original_length=length, fast_turns=fast,
                                              slow_turns=slow)
    want, lo, hi = blended(dim, base, factor, length, fast, slow)
    # one rounding to fp32, and the 64-bit powers and products
    assert all(abs(g - w) <= (2.0 ** -24 + 2.0 ** -45) * w for g, w in zip(got.tolist(), want))
    assert math.isclose(attention, 0.1 * math.log(factor) + 1.0, rel_tol=1e-15)
    # the ends are where the turns say: pair lo turns `fast` times or more, pair hi `slow` times or fewer
    turns = [length * base ** (-2.0 * i / dim) / (2 * math.pi) for i in range(dim // 2)]
    assert lo == 0 or turns[min(lo, dim // 2 - 1)] >= fast * (1 - 1e-12)
    assert hi >= dim // 2 or turns[hi] <= slow * (1 + 1e-12)


def test_a_context_shorter_than_a_turn_is_a_step_behind_the_first_pair():
    # no pair turns once within three positions: the blend ends where it starts
    got, _ = fa.sdpa_rope_frequencies(16, scaling="by_parts", factor=4.0, original_length=3)
    plain = [10000.0 ** (-2.0 * i / 16) for i in range(8)]
    want = plain[:1] + [f / 4 for f in plain[1:]]
    assert all(abs(g - w) <= (2.0 ** -24 + 2.0 ** -45) * w for g, w in zip(got.tolist(), want))
