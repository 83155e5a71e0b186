"""Rotary positions against complex multiplication in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import routed_expert_ffn_f32_amd as cm
from tests.kv_ref import HALF_STEP, U

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def reference(x, pos, freq, interleaved, scale, inverse):
    """(result, sizes of its pairs) in float64."""
    a = torch.outer(pos.double(), freq.double()) * (-1 if inverse else 1)
    turn = torch.polar(torch.full_like(a, float(torch.tensor(scale, dtype=F32))), a)[:, None]
    n, out = len(freq), x.double().clone()
    i = torch.arange(n)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    z = torch.complex(out[..., p], out[..., q]) * turn
    size = torch.zeros_like(out)
    size[..., p] = size[..., q] = z.abs()
    out[..., p], out[..., q] = z.real, z.imag
    return out, size


def check(got, x, pos, freq, interleaved, scale, inverse):
    """The angle's error is below 2^-40 turns and a cosine's or sine's 4 steps of float32; with the scale, the product
    and the sum an element is off by at most 8 half steps of float32 of its pair's size, and rounded once."""
    out, size = reference(x, pos, freq, interleaved, scale, inverse)
    tol = HALF_STEP[x.dtype] * out.abs() + 16 * U * size + 2.0 ** -25 * (x.dtype == F16)
    assert ((got.double() - out).abs() <= tol).all()
    n = 2 * len(freq)
    assert torch.equal(got[..., n:], x[..., n:])


@pytest.mark.parametrize("tokens,heads,dim,part,interleaved,dtype,far", [
    (1, 72, 128, 128, False, BF16, 4000), (1, 1, 2, 2, True, F32, 10), (3, 2, 6, 4, False, F16, 100),
    (5, 3, 130, 66, True, F32, 1 << 24), (5, 3, 130, 66, False, F32, 1 << 24), (40, 9, 96, 30, False, BF16, 1 << 20),
    (1300, 4, 64, 64, True, F16, 1 << 20), (1300, 3, 48, 20, False, F32, 50000), (2, 1, 4096, 4096, False, F32, 7),
    (2, 2, 4095, 4094, True, BF16, 7), (4, 2, 16, 0, False, F32, 5), (17, 5, 256, 2, True, BF16, 1 << 22)])
@pytest.mark.parametrize("inverse", [False, True])
def test_against_the_formula(dev, tokens, heads, dim, part, interleaved, dtype, far, inverse):
    g = torch.Generator().manual_seed(tokens + dim + part)
    x = torch.randn(tokens, heads, dim, generator=g).to(dtype)
    pos = torch.randint(-far, far, (tokens,), generator=g).to(torch.int32)
    freq = cm.rotary_frequencies(part)[0] if part else torch.empty(0)
    got = cm.rotary(x.to(dev), pos.to(dev), freq.to(dev), interleaved=interleaved, scale=1.25, inverse=inverse)
    check(got.cpu(), x, pos, freq, interleaved, 1.25, inverse)


def test_views_in_place_and_wide_positions(dev):
    g = torch.Generator().manual_seed(1)
    base = torch.randn(6, 12, 80, generator=g).bfloat16()
    pos = torch.randint(0, 1 << 40, (6,), generator=g)
    freq = cm.rotary_frequencies(32, base=1e6)[0]
    buf = base.to(dev)
    view = buf[:, 2:9, 4:68]
    version = buf._version
    assert cm.rotary(view, pos.to(dev), freq.to(dev), out=view) is view
    assert buf._version == version + 1
    out = buf.cpu()
    # 2^40 times a 24-bit frequency is rounded to 53 bits: 2^-13 of a turn at most, so the check is of the first 2^29
    near = torch.randint(0, 1 << 28, (6,), generator=g)
    buf2 = base.to(dev)
    cm.rotary(buf2[:, 2:9, 4:68], near.to(dev), freq.to(dev), out=buf2[:, 2:9, 4:68])
    check(buf2.cpu()[:, 2:9, 4:68], base[:, 2:9, 4:68], near, freq, False, 1.0, False)
    for got in (out, buf2.cpu()):
        rest = torch.ones(6, 12, 80, dtype=torch.bool)
        rest[:, 2:9, 4:68] = False
        assert torch.equal(got[rest], base[rest])


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(dev, interleaved):
    """<g, R x> = <R' g, x>, and central differences of a sum of the results."""
    g = torch.Generator().manual_seed(2)
    x, up = torch.randn(3, 2, 20, generator=g), torch.randn(3, 2, 20, generator=g)
    pos, freq = torch.tensor([0, 5, 1000], dtype=torch.int32), cm.rotary_frequencies(12)[0]
    kw = dict(interleaved=interleaved, scale=0.7)
    f = lambda v: cm.rotary(v.to(dev), pos.to(dev), freq.to(dev), **kw).cpu().double()  # noqa: E731
    d = cm.rotary(up.to(dev), pos.to(dev), freq.to(dev), inverse=True, **kw).cpu().double()
    lhs, rhs = (up.double() * f(x)).sum(), (d * x.double()).sum()
    assert abs(lhs - rhs) <= 120 * 32 * U * 4
    for i in ((0, 0, 0), (1, 1, 3), (2, 0, 11), (2, 1, 15)):
        e = torch.zeros_like(x)
        e[i] = 0.5  # linear, so a large step is exact but for rounding
        slope = (up.double() * (f(x + e) - f(x - e))).sum()
        assert abs(slope - d[i]) <= 1e-4


def test_frequencies(dev):
    n = 64
    plain, one = cm.rotary_frequencies(2 * n)
    assert one == 1.0 and torch.allclose(plain[0], torch.tensor(1.0))
    lin, _ = cm.rotary_frequencies(2 * n, scaling="linear", factor=8.0)
    assert torch.allclose(lin * 8, plain, rtol=1e-6)
    base, _ = cm.rotary_frequencies(2 * n, scaling="base", factor=8.0)
    assert base[0] == 1 and torch.allclose(base[-1] * 8, plain[-1], rtol=1e-5)
    parts, scale = cm.rotary_frequencies(2 * n, scaling="parts", factor=8.0, original=4096)
    turns = 4096 * plain.double() / (2 * torch.pi)
    assert torch.equal(parts[turns > 40], plain[turns > 40])
    assert torch.allclose(parts[turns < 0.7] * 8, plain[turns < 0.7], rtol=1e-6)
    assert ((parts <= plain) & (parts * 8 >= plain * 0.999999)).all() and 1.2 < scale < 1.21
    assert torch.equal(cm.rotary_frequencies(2 * n, device=dev)[0].cpu(), plain)
