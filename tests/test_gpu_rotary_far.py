"""Rotary positions far out: the angle is a position times a float32 frequency
exactly, whatever the position, up to 2^53."""
import math
from fractions import Fraction

import pytest

torch = pytest.importorskip("torch")

import routed_expert_ffn_f32_amd as cm
from tests.kv_ref import U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def pi(bits):
    """pi 2^bits as a whole number, by Machin's formula, with 16 bits to spare."""
    one = 1 << (bits + 16)

    def arctan(n):  # of 1 / n
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total
    return 4 * (4 * arctan(5) - arctan(239)) >> 16


TWO_PI = Fraction(2 * pi(300), 1 << 300)


def angle(position, freq):
    """position * freq reduced to [-pi, pi], from whole numbers."""
    a = position * Fraction(freq)
    return float(a - TWO_PI * round(a / TWO_PI))


def test_pi():
    assert float(TWO_PI) == 2 * math.pi


@pytest.mark.parametrize("far,dtype", [(1 << 10, torch.int32), (1 << 28, torch.int32), ((1 << 31) - 1, torch.int32),
                                       (1 << 34, torch.int64), (1 << 45, torch.int64), (1 << 53, torch.int64)])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(dev, far, dtype, base, interleaved):
    """The reduced angle is off by less than 2^-50 turns and is rounded to
    float32 in half turns (2^-25 of one: 1.6 half steps of 1), a cosine's or
    sine's 4 steps, product and sum: 16 half steps of the pair's size at most."""
    g = torch.Generator().manual_seed(far % 1000003)
    n = 32
    pos = torch.randint(far // 2, far, (9,), generator=g, dtype=torch.int64)
    pos[0], pos[1::2] = far, -pos[1::2]
    freq = cm.rotary_frequencies(2 * n, base)[0]
    x = torch.randn(9, 2, 2 * n, generator=g)
    got = cm.rotary(x.to(dev), pos.to(dtype).to(dev), freq.to(dev), interleaved=interleaved).cpu().double()
    a = torch.tensor([[angle(int(p), float(f)) for f in freq] for p in pos], dtype=torch.float64)[:, None]
    i = torch.arange(n)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    u, v = x[..., p].double(), x[..., q].double()
    tol = 16 * U * torch.hypot(u, v)
    assert ((got[..., p] - (u * a.cos() - v * a.sin())).abs() <= tol).all()
    assert ((got[..., q] - (u * a.sin() + v * a.cos())).abs() <= tol).all()
