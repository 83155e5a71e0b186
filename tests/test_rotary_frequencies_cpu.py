"""Frequencies of rotary positions that are scaled "by parts": which pairs of
a head are left, divided and blended, for original contexts of any length."""
import math

import pytest

torch = pytest.importorskip("torch")

import routed_expert_ffn_f32_amd as cm


@pytest.mark.parametrize("part,base,original,factor", [
    (128, 10000.0, 4096, 8.0), (128, 10000.0, 65536, 8.0), (128, 10000.0, 131072, 8.0), (64, 10000.0, 1 << 20, 4.0),
    (128, 500000.0, 8192, 16.0), (128, 10000.0, 100, 2.0), (16, 10000.0, 1 << 30, 2.0), (2, 10000.0, 4096, 4.0)])
def test_parts(part, base, original, factor):
    """Pair i turns original / (2 pi) base^(-2 i / part) times in the original
    context.  More than 32 turns: as it is; fewer than one: divided; between:
    the share of the division grows by the same step from pair to pair."""
    got, scale = cm.rotary_frequencies(part, base, scaling="parts", factor=factor, original=original)
    plain = [base ** (-2 * i / part) for i in range(part // 2)]
    turns = [original * f / (2 * math.pi) for f in plain]
    # where a pair would turn 32 times and once, as a (fractional) index
    at = [part * math.log(original / (2 * math.pi * t)) / (2 * math.log(base)) for t in (32, 1)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), part - 1)
    for i, f in enumerate(plain):
        ratio = f / float(got[i])  # float32: half a step of 2^-24
        if turns[i] > 32 or i <= lo < hi:
            want = f
        elif turns[i] < 1:
            want = f / factor
        else:
            share = min(max((i - lo) / (hi - lo), 0), 1)
            want = f * (1 - share) + f / factor * share
        assert abs(float(got[i]) - want) <= 2.0 ** -23 * want, (i, turns[i], ratio)
    assert scale == 0.1 * math.log(factor) + 1


def test_long_originals_leave_pairs_that_turn():
    """A context in which even the slowest pair turns more than once divides no
    pair by the whole factor."""
    got, _ = cm.rotary_frequencies(128, scaling="parts", factor=8.0, original=131072)
    plain, _ = cm.rotary_frequencies(128)
    ratio = plain.double() / got.double()
    assert 131072 * float(plain[-1]) / (2 * math.pi) > 2
    assert (ratio < 2.75).all() and 2.65 < float(ratio[-1])
    assert (ratio[1:] >= ratio[:-1] * (1 - 2.0 ** -22)).all()
