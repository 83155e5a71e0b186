"""GPU parity of coli_moe_rmsnorm (residual addition + root-mean-square norm)
against the formulas in 64 bits and, for the 8-bit codes, against the same
sequence of correctly rounded float32 operations.

Tolerances.  The sum of squares is kept in float64 and r rounded once, then
two float32 products: every y is within 3 half steps of float32 (2^-24 each)
of (s r) w; the output type adds one half step of its own.  The stored sum is
one float32 addition and one rounding, so it is compared bit for bit; so are
scales and codes, whose operations (absolute maximum, division, rounding) are
exact or correctly rounded on both sides."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import routed_expert_ffn_f32_amd as cm

pytestmark = pytest.mark.gpu

F32, BF16, F16, I8, E4 = torch.float32, torch.bfloat16, torch.float16, torch.int8, torch.float8_e4m3fn
HALF = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def make(rows, hidden, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, hidden, generator=g) * scale).to(dtype)


def reference(x, weight, eps, residual=None):
    """(stored sum, y in float64, y in the kernel's float32 operations)."""
    s = x.float()
    stored = None
    if residual is not None:
        stored = (s + residual.float()).to(residual.dtype)
        s = stored.float()
    h = s.shape[1]
    ms = s.double().square().sum(1, keepdim=True) / h + float(np.float32(eps))
    r = 1.0 / ms.sqrt()
    w = torch.ones(h) if weight is None else weight.float()
    y32 = s * r.float()
    if weight is not None:
        y32 = y32 * w
    return stored, s.double() * r * w.double(), y32


def check_float(got, y64, dtype):
    half = torch.finfo(dtype).eps / 2
    tiny = float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps  # one subnormal step
    tol = y64.abs() * ((1 + half) * (1 + 3.01 * HALF) - 1) + tiny
    bad = (got.double() - y64).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside {dtype} tolerance"


def check_codes(codes, scales, y32, y64, dtype, group):
    q = 127.0 if dtype == I8 else 448.0
    h = y32.shape[1]
    for i, lo in enumerate(range(0, h, group or h)):
        blk, exact = y32[:, lo:lo + (group or h)], y64[:, lo:lo + (group or h)]
        s = blk.abs().amax(1) / q
        assert torch.equal(scales[:, i], s), f"scales of group {i}"
        v = torch.where(s[:, None] > 0, blk / s[:, None], torch.zeros_like(blk)).clamp(-q, q)
        want = (v.round() if dtype == I8 else v).to(dtype)
        got = codes[:, lo:lo + (group or h)]
        assert torch.equal(got.view(torch.int8), want.view(torch.int8)), f"codes of group {i}"
        # and the value stands within half a step of the definition's
        val = got.double() * scales[:, i:i + 1].double()
        step = torch.full_like(exact, 0.5) if dtype == I8 else torch.maximum(v.abs().double() * 2.0 ** -4,
                                                                             torch.full_like(exact, 2.0 ** -10))
        assert ((val - exact).abs() <= step * scales[:, i:i + 1].double() * (1 + 2.0 ** -16) + 1e-37).all()


def run(dev, x, weight, eps, residual=None, in_place=False, **kw):
    d = lambda t: None if t is None else t.to(dev)  # noqa: E731
    r = d(residual)
    ro = None if residual is None or in_place else torch.full_like(r, float("nan"))
    got = cm.rms_norm(d(x), d(weight), eps, residual=r, residual_out=ro, **kw)
    torch.cuda.synchronize()
    stored = r if in_place else ro
    if stored is not None and not in_place:
        assert torch.equal(r.cpu(), residual), "the residual was changed though residual_out was given"
    return got, None if stored is None else stored.cpu()


# every launch shape: 1, 2, 4, 6, 8, 12 and 16 waves of one piece a thread, 8 (many rows)
# and 16 of 2, 16 of 4; parts of a wave up to 128 columns
SIZES = [(1, 1), (3, 7), (5, 64), (17, 120), (16, 128), (7, 129), (2, 511), (9, 512), (4, 513), (7, 1024), (3, 1025), (2, 2047), (5, 2048), (2, 2056),
         (3, 2600), (3, 4096), (2, 5001), (1, 6144), (65, 6144), (3, 6145), (2, 8192), (2, 8193), (2, 16384), (1, 16391),
         (2, 32768),
         (1025, 5000)]


@pytest.mark.parametrize("rows,hidden", SIZES)
def test_every_launch_shape(dev, rows, hidden):
    w = (1 + 0.1 * make(1, hidden, F32, 1)[0])
    x, r = make(rows, hidden, F32, 2), make(rows, hidden, F32, 3, 4.0)
    stored, y64, y32 = reference(x, w, 1e-6, r)
    got, kept = run(dev, x, w, 1e-6, r)
    assert torch.equal(kept, stored)
    check_float(got.cpu(), y64, F32)
    for group in (0, 64, 128):
        (codes, scales), kept = run(dev, x, w, 1e-6, r, in_place=True, out_dtype=I8, group=group)
        assert torch.equal(kept, stored)
        check_codes(codes.cpu(), scales.cpu(), y32, y64, I8, group)


@pytest.mark.parametrize("out", [F32, BF16, F16, I8, E4])
@pytest.mark.parametrize("xt,rt,wt", [(F32, F32, F32), (BF16, F32, BF16), (F16, F16, F32), (BF16, BF16, None),
                                      (F32, None, F16), (F16, BF16, F32)])
def test_types(dev, xt, rt, wt, out):
    rows, hidden = 17, 777
    x, r = make(rows, hidden, xt, 5), None if rt is None else make(rows, hidden, rt, 6, 3.0)
    w = None if wt is None else (1 + 0.1 * make(1, hidden, F32, 7)[0]).to(wt)
    stored, y64, y32 = reference(x, w, 1e-5, r)
    got, kept = run(dev, x, w, 1e-5, r, out_dtype=out)
    if r is not None:
        assert torch.equal(kept, stored)
    if out in (I8, E4):
        check_codes(got[0].cpu(), got[1].cpu(), y32, y64, out, 0)
        got, _ = run(dev, x, w, 1e-5, r, out_dtype=out, group=128)
        check_codes(got[0].cpu(), got[1].cpu(), y32, y64, out, 128)
    else:
        check_float(got.cpu(), y64, out)


@pytest.mark.parametrize("xt,out", [(F32, F32), (BF16, I8), (F16, E4), (BF16, F16)])
def test_strided_and_unaligned_rows(dev, xt, out):
    """Rows cut out of a wider matrix at an odd column: nothing is 16-byte
    aligned, and what stands around the written rows stays as it was."""
    rows, hidden, pad = 6, 1003, 13
    big = make(rows, hidden + pad, xt, 8).to(dev)
    x = big[:, 5:5 + hidden]
    w = (1 + 0.1 * make(1, hidden + 1, F32, 9)[0]).to(dev)[1:]
    frame = torch.full((rows, hidden + pad), 3, dtype=F32, device=dev).to(out)
    dst = frame[:, 3:3 + hidden]
    stored, y64, y32 = reference(x.cpu(), w.cpu(), 1e-6)
    scales = torch.full((rows, 11), -1.0, device=dev)
    kw = dict(group=128, scales=scales[:, 2:10]) if out in (I8, E4) else {}
    cm.rms_norm(x, w, 1e-6, out=dst, **kw)
    torch.cuda.synchronize()
    if kw:
        check_codes(dst.cpu(), scales[:, 2:10].cpu(), y32, y64, out, 128)
        assert (scales[:, :2] == -1).all() and (scales[:, 10:] == -1).all()
    else:
        check_float(dst.cpu(), y64, out)
    around = frame.float().cpu()
    assert (around[:, :3] == 3).all() and (around[:, 3 + hidden:] == 3).all()


def test_extreme_rows(dev):
    """Rows of zeros, of float32's largest and smallest values, with one huge
    element; a row with NaN leaves the others alone; eps 0; equal rows read
    through a stride of 0; no rows."""
    h = 640
    x = make(6, h, F32, 10)
    x[0] = 0
    x[1] *= 1e37
    x[2] *= 1e-30
    x[3, 7] = 3e38
    x[5, 1] = float("nan")
    ok = [0, 1, 2, 3, 4]
    stored, y64, y32 = reference(x, None, 1e-6)
    got, _ = run(dev, x, None, 1e-6)
    check_float(got.cpu()[ok], y64[ok], F32)
    (codes, scales), _ = run(dev, x, None, 1e-6, out_dtype=I8, group=64)
    check_codes(codes.cpu()[ok], scales.cpu()[ok], y32[ok], y64[ok], I8, 64)
    assert not codes.cpu()[0].any() and not scales.cpu()[0].any()
    stored, y64, _ = reference(x[4:5], None, 0.0)
    got, _ = run(dev, x[4:5], None, 0.0)
    check_float(got.cpu(), y64, F32)
    zeros = torch.zeros(2, h, device=dev)
    assert not cm.rms_norm(zeros, None, 0.0).any() and not cm.rms_norm(zeros, None, 0.0, out_dtype=E4)[0].float().any()
    same = cm.rms_norm(x[4:5].to(dev).expand(3, h), None, 0.0)
    assert torch.equal(same.cpu(), got.cpu().expand(3, h))
    assert cm.rms_norm(torch.empty(0, h, device=dev)).shape == (0, h)


@pytest.mark.parametrize("exponent", [-148, -140, -126, -100, -70, -61, -60, -59, 50, 99, 100, 101, 110, 119])
def test_codes_at_every_magnitude(dev, exponent):
    """Scales down to float32's subnormals and up to its largest values: the
    codes are those of a correctly rounded division all the same."""
    h = 256
    x = make(3, h, F32, 12) * 3
    w = torch.full((h,), 2.0 ** (exponent / 2 if exponent % 2 == 0 else (exponent + 1) / 2)) * 1.0
    w = w * torch.tensor(2.0 ** (exponent - (exponent // 2 if exponent % 2 == 0 else (exponent + 1) // 2)), dtype=F32)
    stored, y64, y32 = reference(x, w, 1e-6)
    for dtype in (I8, E4):
        for group in (0, 64):
            (codes, scales), _ = run(dev, x, w, 1e-6, out_dtype=dtype, group=group)
            q = 127.0 if dtype == I8 else 448.0
            s = y32.view(3, -1, group or h).abs().amax(2) / q
            assert torch.equal(scales.cpu(), s)
            wide = s.repeat_interleave(group or h, 1)
            v = torch.where(wide > 0, y32 / wide, torch.zeros_like(y32)).clamp(-q, q)
            want = (v.round() if dtype == I8 else v).to(dtype)
            assert torch.equal(codes.cpu().view(torch.int8), want.view(torch.int8)), (exponent, dtype, group)


def test_in_place(dev):
    """out == x, element for element, gives the result of separate buffers."""
    x = make(9, 2100, F32, 11).to(dev)
    want = cm.rms_norm(x, None)
    cm.rms_norm(x, None, out=x)
    assert torch.equal(x, want)


def test_another_stream_and_graph_replays(dev):
    """On a stream of the caller's, and captured: every replay on new inputs
    gives the eager result."""
    rows, hidden = 33, 6144
    w = (1 + 0.1 * make(1, hidden, F32, 12)[0]).to(dev)
    xs = [make(rows, hidden, BF16, 20 + i).to(dev) for i in range(3)]
    rs = [make(rows, hidden, F32, 30 + i).to(dev) for i in range(3)]
    want = []
    for x, r in zip(xs, rs):
        r2 = r.clone()
        want.append((*cm.rms_norm(x, w, residual=r2, out_dtype=I8), r2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r2 = rs[0].clone()
        got = (*cm.rms_norm(xs[0], w, residual=r2, out_dtype=I8), r2)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    x, r = xs[0].clone(), rs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        codes, scales = cm.rms_norm(x, w, residual=r, out_dtype=I8)
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        r.copy_(rs[i])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((codes, scales, r), want[i])), i
        cm.rms_norm(xs[i], w)  # eager work between replays


@pytest.mark.parametrize("hidden", [40, 300, 2050, 6144])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rows_that_are_not_finite_stay_visible(dev, bad, hidden):
    """A row with NaN or Inf is NaN from end to end (8 bits: every scale, with
    codes 0), its stored sum is the plain one, and the rows beside it are
    those of a call without it."""
    x, r = make(5, hidden, BF16, 40).to(dev), make(5, hidden, F32, 41).to(dev)
    x[1, hidden - 1] = bad
    x[3, 3] = bad
    ok, nan = [0, 2, 4], [1, 3]
    w = (1 + 0.1 * make(1, hidden, F32, 42)[0]).to(dev)
    for out in (F32, BF16, F16):
        s = r.clone()
        got = cm.rms_norm(x, w, residual=s, out_dtype=out)
        assert got[nan].isnan().all()
        assert torch.equal(got[ok], cm.rms_norm(x[ok], w, residual=r[ok], out_dtype=out))
        assert torch.equal(s.nan_to_num(7.0), (x.float() + r).nan_to_num(7.0))
    for out in (I8, E4):
        for group in (0, 64, 128):
            codes, scales = cm.rms_norm(x, w, out_dtype=out, group=group)
            assert scales[nan].isnan().all() and not codes[nan].view(torch.int8).any()
            want = cm.rms_norm(x[ok], w, out_dtype=out, group=group)
            assert torch.equal(codes[ok].view(torch.int8), want[0].view(torch.int8)) and torch.equal(scales[ok], want[1])


@pytest.mark.parametrize("hidden", [8, 300, 2050])
def test_signs_of_zero_codes(dev, hidden):
    """e4m3 has a negative zero: the code of -0, and of a negative quotient
    that rounds to it."""
    x = make(3, hidden, F32, 50)
    x[0, ::2], x[0, 1::4] = -0.0, 0.0
    x[1, 1:] *= 2.0 ** -20
    x[2, :4] = torch.tensor([-2.0 ** -149, -0.0, 2.0 ** -149, 0.0])
    _, y64, y32 = reference(x, None, 1e-6)
    for group in (0, 64):
        (codes, scales), _ = run(dev, x, None, 1e-6, out_dtype=E4, group=group)
        check_codes(codes.cpu(), scales.cpu(), y32, y64, E4, group)


@pytest.mark.parametrize("hidden", [8, 120, 300, 1000, 2050, 6144, 16391, 32768])
def test_rows_at_both_ends_of_the_range(dev, hidden):
    """Without eps, rows of float32's and bf16's subnormals and of its largest
    values: 1 / rms is not a (normal) float32 there, the results are of order
    1.  The reference takes the power of two from one factor to the other too,
    which changes no rounding."""
    g = torch.Generator().manual_seed(hidden)
    x = torch.randn(9, hidden, generator=g)
    x[0] = torch.randint(-3, 4, (hidden,), generator=g) * 2.0 ** -149
    x[0, 0], x[0, hidden // 2] = 0.0, 2.0 ** -149
    x[1] = 0
    x[1, hidden - 1] = -2.0 ** -149
    for row, e in ((2, -128), (3, -105), (4, -100), (5, -95), (6, 99), (7, 126)):
        x[row] *= 2.0 ** e
    x[8] *= 1e-37
    x[8, 3] = 3.4e38
    x.clamp_(-3.4e38, 3.4e38)
    assert x[0].any() and torch.isfinite(x).all()
    w = 1 + 0.1 * make(1, hidden, F32, 1)[0]
    for v in (x, x.bfloat16()):
        s = v.float()
        ok = torch.isfinite(s).all(1)  # the largest values round to Inf in bf16: a row of NaN
        assert ok.all() or v.dtype == BF16
        r = 1 / (s.double().square().sum(1, keepdim=True) / hidden).sqrt()
        r = torch.where(torch.isfinite(r), r, torch.zeros_like(r))  # and the smallest to 0: a row of zeros
        far = torch.where(r > 2.0 ** 100, 64.0, torch.where(r < 2.0 ** -100, -64.0, 0.0)).double()
        y32 = (s.double() * 2.0 ** far).float() * (r * 2.0 ** -far).float() * w
        y64 = s.double() * r * w.double()
        for out in (F32, BF16):
            got = run(dev, v, w, 0.0, out_dtype=out)[0].cpu()
            check_float(got[ok], y64[ok], out)
            assert got[~ok].isnan().all()
        for out in (I8, E4):
            for group in (0, 64):
                codes, scales = (t.cpu() for t in run(dev, v, w, 0.0, out_dtype=out, group=group)[0])
                check_codes(codes[ok], scales[ok], y32[ok], y64[ok], out, group)
                assert scales[~ok].isnan().all()


@pytest.mark.parametrize("out", [I8, E4])
def test_results_past_the_range_stay_visible(dev, out):
    """A weight that takes one element past float32's largest: its group's
    scale is Inf, every value of the group Inf * 0; the others are as without
    it."""
    x, w = make(4, 300, F32, 60), 1 + 0.1 * make(1, 300, F32, 61)[0]
    x[2] *= 1e-3
    x[2, 70] = 50.0
    w[70] = 5e37
    for group in (0, 64):
        (codes, scales), _ = run(dev, x, w, 1e-6, out_dtype=out, group=group)
        hit = slice(64, 128) if group else slice(0, 300)
        at = 1 if group else 0
        assert scales[2, at] == float("inf") and not codes[2, hit].view(torch.int8).any()
        _, y64, y32 = reference(x, w, 1e-6)
        rest = [0, 1, 3]
        check_codes(codes.cpu()[rest], scales.cpu()[rest], y32[rest], y64[rest], out, group)
