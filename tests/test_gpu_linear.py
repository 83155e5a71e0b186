"""GPU parity of coli_moe_linear (dense product with its epilogue).

Where every number is a small integer (and every scale a power of two), all
sums are exact whatever their order, and float32 results are compared bit for
bit: that covers sizes, tails, strides and types of the structure.  On real
numbers the results are held to the formulas in 64 bits within
  sums     (k/4 + 16) u sum |x w| (u = 2^-23: a matrix instruction adds at
           least 4 products at a time), none for int8;
  scales   one rounding of the sum to float32, two products: 2 u |v|;
  bias     u |v|;
  act      slopes of at most 1.2, and 8 u |v| for the function itself
           (exponential 3 u, quotient 2 u, product 1 u, and its argument's
           rounding, which the sigmoid's slope damps);
  SwiGLU   both of the above for gate and up, and 2 u for the product;
  residual u |out|, and half a step of the output's type."""
import math

import pytest

torch = pytest.importorskip("torch")

import routed_expert_ffn_f32_amd as cm

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
F32, BF16, F16, I8, E4 = torch.float32, torch.bfloat16, torch.float16, torch.int8, torch.float8_e4m3fn
KINDS = [BF16, F16, I8, E4]
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def ints(shape, top, g):
    return torch.randint(-top, top + 1, shape, generator=g).double()


def step(k, kind):
    """k as a multiple of 16 bytes."""
    e = 8 if kind in (BF16, F16) else 16
    return -(-k // e) * e


def padded(v, kind, dev, pad=16, fill=0.0):
    """v in the given type as the first columns of a wider array."""
    big = torch.full((v.shape[0], v.shape[1] + pad), fill, device=dev).to(kind)
    big[:, :v.shape[1]] = v.to(kind).to(dev) if kind != E4 else v.float().to(dev).to(kind)
    return big[:, :v.shape[1]]


def exact_case(dev, m, n, k, kind, act, seed, bias, residual, out=F32, frame=5):
    """act in none, relu; integers throughout."""
    g = torch.Generator().manual_seed(seed)
    k = step(k, kind)
    x, w = ints((m, k), 3 if kind != I8 else 128, g), ints((n, k), 3 if kind != I8 else 128, g)
    if kind == I8:
        x, w = x.clamp(max=127), w.clamp(max=127)
    # what stands past a row's end must not be used
    fill = float("nan") if kind in (BF16, F16, E4) else 77.0
    xd, wd = padded(x, kind, dev, 16, fill), padded(w, kind, dev, 32, fill)
    want = x @ w.t()
    kw = {}
    if kind in (I8, E4):
        sx, sw = torch.exp2(torch.randint(-3, 4, (m,), generator=g).float()), torch.exp2(
            torch.randint(-3, 4, (n,), generator=g).float())
        kw = dict(x_scale=sx.to(dev), w_scale=sw.to(dev))
        want = want.float().double() * sx[:, None].double() * sw.double()
    if bias:
        b = ints((n,), 9, g)
        kw["bias"] = b.float().to(dev)
        want = (want.float() + b.float()).double()
    if act == "relu":
        want = want.clamp(min=0)
    full = torch.full((m, n + frame), 7.0, device=dev, dtype=out)
    if residual:
        r = ints((m, n), 9, g)
        kw["residual"] = padded(r, out, dev, 3)
        want = (want.float() + r.float()).double()
    cm.linear(xd, wd, act=act, out=full[:, :n], **kw)
    torch.cuda.synchronize()
    got = full.cpu()
    assert (got[:, n:] == 7.0).all(), "outputs beyond n were written"
    assert torch.equal(got[:, :n].float(), want.to(out).float()), (m, n, k, kind, act)


SIZES = [(1, 1, 8), (1, 7, 64), (1, 64, 1024), (1, 513, 2072), (2, 16, 72), (3, 31, 200), (4, 100, 4096), (5, 129, 136),
         (8, 257, 520), (15, 64, 64), (16, 48, 6144), (17, 1001, 256), (31, 33, 1032), (33, 500, 72), (63, 129, 640),
         (64, 255, 2048), (65, 64, 72), (100, 128, 8192), (127, 257, 136), (128, 129, 1024), (129, 1, 64),
         (200, 300, 2072), (255, 513, 200), (257, 1001, 520), (1, 4097, 512), (40, 2048, 128), (1000, 17, 264)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_sizes_exactly(dev, m, n, k, kind):
    exact_case(dev, m, n, k, kind, "none", m + n + k, bias=False, residual=False)
    exact_case(dev, m, n, k, kind, "relu", m + n + k + 1, bias=True, residual=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,k", [(129, 8200, 136), (500, 4096, 328), (1000, 6100, 200), (1000, 5000, 8),
                                   (4000, 6100, 136),
                                   (3500, 3600, 264), (3329, 4000, 520), (4096, 3585, 64), (300, 5000, 8)])
def test_every_block_shape_exactly(dev, m, n, k, kind):
    """Sizes that the choice of blocks sends to each of its shapes beyond the
    smallest; K of less than a step, of whole steps, and with a rest."""
    exact_case(dev, m, n, k, kind, "none", m, bias=True, residual=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,k", [(1, 5, 64), (7, 100, 520), (30, 129, 264), (60, 300, 136), (129, 4099, 136),
                                   (500, 2049, 72), (1000, 3050, 200), (4000, 3050, 72), (3500, 1801, 136)])
def test_swiglu_on_every_block_shape(dev, m, n, k, kind):
    """Gate and up sums are exact integers here, so only the activation's own
    8 u |gate up| and the product's 2 u remain."""
    g = torch.Generator().manual_seed(n)
    k = step(k, kind)
    x, w = ints((m, k), 2, g), ints((2 * n, k), 2, g)
    sx, sw = torch.full((m,), 0.25), torch.full((2 * n,), 0.125)
    kw = dict(x_scale=sx.to(dev), w_scale=sw.to(dev)) if kind in (I8, E4) else {}
    v = (x.float() @ w.float().t()).double() * (0.03125 if kw else 1.0)
    gate, up = v[:, :n], v[:, n:]
    want = gate / (1 + torch.exp(-gate)) * up
    got = cm.linear(padded(x, kind, dev, 0), padded(w, kind, dev, 0), act="swiglu", out_dtype=F32, **kw)
    err = (got.cpu().double() - want).abs()
    assert (err <= 10 * U * (gate * up).abs()).all(), float((err / ((gate * up).abs() + 1e-30)).max() / U)


@pytest.mark.parametrize("out", [BF16, F16])
def test_narrow_outputs_exactly(dev, out):
    """Small sums are whole numbers that 16 bits hold."""
    for m, n in ((3, 70), (70, 133), (300, 260)):
        g = torch.Generator().manual_seed(m)
        x, w, r = ints((m, 16), 1, g), ints((n, 16), 1, g), ints((m, n), 30, g)
        got = cm.linear(x.to(dev, BF16), w.to(dev, BF16), residual=r.to(dev, out))
        assert got.dtype == out and torch.equal(got.cpu().double(), x @ w.t() + r)


def f_act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act in ("silu", "swiglu"):
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,k,out,bt", [(1, 130, 1024, BF16, F32), (6, 77, 136, F32, BF16), (37, 200, 2072, F16, F16),
                                          (150, 90, 264, F32, F32), (290, 270, 1040, BF16, None)])
def test_epilogues(dev, m, n, k, out, bt, kind, act):
    g = torch.Generator().manual_seed(m + len(act))
    k, rows = step(k, kind), 2 * n if act == "swiglu" else n
    x, w = torch.randn(m, k, generator=g), torch.randn(rows, k, generator=g) / math.sqrt(k)
    kw, sx, sw = {}, torch.ones(m), torch.ones(rows)
    if kind in (I8, E4):
        q = 127.0 if kind == I8 else 448.0
        sx, sw = x.abs().amax(1) / q, w.abs().amax(1) / q
        x, w = x / sx[:, None], w / sw[:, None]
        x, w = (x.round(), w.round()) if kind == I8 else (x.clamp(-q, q), w.clamp(-q, q))
        kw = dict(x_scale=sx.to(dev), w_scale=sw[:, None].to(dev).contiguous())
    xq, wq = x.to(kind), w.to(kind)
    x, w, s = xq.double(), wq.double(), sx[:, None].double() * sw.double()
    v = (x @ w.t()) * s
    err = 0 if kind == I8 else (k / 4 + 16) * U * (x.abs() @ w.abs().t()) * s
    err = err + 2 * U * v.abs()
    if bt is not None:
        b = (0.5 * torch.randn(rows, generator=g)).to(bt)
        kw["bias"] = b.to(dev)
        v = v + b.double()
        err = err + U * v.abs()
    if act == "swiglu":
        gate, up, eg, eu = v[:, :n], v[:, n:], err[:, :n], err[:, n:]
        sg = f_act(gate, act)
        err = (1.2 * eg + 8 * U * gate.abs()) * (up.abs() + eu) + sg.abs() * eu + 2 * U * (sg * up).abs()
        v = sg * up
    elif act == "none":
        pass
    else:
        err = 1.2 * err + (0 if act == "relu" else 8 * U * v.abs())
        v = f_act(v, act)
    r = torch.randn(m, n, generator=g).to(out)
    v = v + r.double()
    err = err + U * v.abs()
    err = err + (v.abs() + err) * torch.finfo(out).eps / 2 + 1e-7 * (out == F16)
    res = r.to(dev)
    got = cm.linear(xq.to(dev), wq.to(dev), act=act, residual=res, **kw)
    again = cm.linear(xq.to(dev), wq.to(dev), act=act, residual=res, out=res, **kw)  # onto the residual itself
    torch.cuda.synchronize()
    bad = (got.cpu().double() - v).abs() > err
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {float(((got.cpu().double() - v).abs() / err).max())}"
    assert torch.equal(again, got)


def test_types_by_default(dev):
    x, w = torch.randn(3, 64, device=dev), torch.randn(5, 64, device=dev)
    assert cm.linear(x.half(), w.half()).dtype == F16
    one = torch.ones(3, device=dev), torch.ones(5, device=dev)
    assert cm.linear(x.to(I8), w.to(I8), *one).dtype == BF16
    assert cm.linear(x.bfloat16(), w.bfloat16(), residual=torch.zeros(3, 5, device=dev)).dtype == F32
    assert cm.linear(x[:0].half(), w.half()).shape == (0, 5)


@pytest.mark.parametrize("m", [1, 16, 40, 300])
def test_stride_zero_and_saturated_activations(dev, m):
    """One row read for all of x; activations far outside their middle."""
    g = torch.Generator().manual_seed(m)
    x, w = ints((1, 64), 3, g).to(dev, BF16), ints((70, 64), 3, g).to(dev, BF16)
    want = cm.linear(x, w, out_dtype=F32)
    got = cm.linear(x.expand(m, 64), w, out_dtype=F32)
    assert torch.equal(got, want.expand(m, 70))
    big = (want * 1e20).cpu()
    for act in ("silu", "gelu", "gelu_tanh"):
        y = cm.linear((x.float() * 2.0 ** 33).bfloat16(), (w.float() * 2.0 ** 33).bfloat16(), act=act, out_dtype=F32).cpu()
        assert torch.equal(y == 0, big <= 0) and torch.isfinite(y).all() and (y >= 0).all()


def test_another_stream_and_graph_replays(dev):
    """Captured with the norm that feeds it; every replay on new rows gives
    the eager result."""
    for m in (1, 24, 300):
        g = torch.Generator().manual_seed(m)
        w = torch.randint(-127, 128, (2 * 200, 512), generator=g).to(I8).to(dev)
        sw = (torch.rand(400, generator=g) / 100).to(dev)
        xs = [torch.randn(m, 512, generator=g).to(dev) for _ in range(3)]

        def block(x):
            q, s = cm.rms_norm(x, None, out_dtype=I8)
            return cm.linear(q, w, s, sw, act="swiglu")

        want = [block(x) for x in xs]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = block(xs[1])
        side.synchronize()
        assert torch.equal(got, want[1])
        x = xs[0].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = block(x)
        for i in (2, 1, 0, 2):
            x.copy_(xs[i])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want[i]), (m, i)
            block(xs[0])


@pytest.mark.parametrize("m", [1, 20, 60, 200, 600])
def test_nan_stays_visible(dev, m):
    """A NaN in a row of x makes that row of the result NaN, one in w or the
    bias its column, under every activation; the others are as without it."""
    g = torch.Generator().manual_seed(m)
    x, w = torch.randn(m, 136, generator=g).to(dev, BF16), torch.randn(2 * 96, 136, generator=g).to(dev, BF16)
    bias = torch.randn(2 * 96, generator=g).to(dev)
    xn, wn, bn = x.clone(), w.clone(), bias.clone()
    xn[m // 2, 135], wn[5, 0], bn[90] = float("nan"), float("nan"), float("nan")
    for act in ACTS:
        rows = 2 * 96 if act == "swiglu" else 96
        want = cm.linear(x, w[:rows], bias=bias[:rows], act=act, out_dtype=F32)
        got = cm.linear(xn, wn[:rows], bias=bn[:rows], act=act, out_dtype=F32)
        nan = torch.zeros(m, 96, dtype=torch.bool, device=dev)
        nan[m // 2], nan[:, 5], nan[:, 90] = True, True, True
        assert torch.equal(got.isnan(), nan), act
        assert torch.equal(got[~nan], want[~nan]), act


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n", [(100, 6000), (250, 6100), (380, 5990)])
@pytest.mark.parametrize("k", [8, 64, 128, 192, 320, 576, 1088, 2056])
def test_rings_of_the_small_blocks(dev, m, n, k, kind):
    """Blocks of 64 x 64, 128 x 64 and 128 x 128 with fewer K steps than their
    rings have stages, as many, several times as many, odd and even numbers."""
    exact_case(dev, m, n, k, kind, "none", m + k, bias=False, residual=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,k", [(100, 3000, 1096), (250, 3050, 1480), (380, 2990, 968)])
def test_swiglu_on_the_small_blocks(dev, m, n, k, kind):
    test_swiglu_on_every_block_shape(dev, m, n, k, kind)


@pytest.mark.parametrize("kind", [I8, E4])
@pytest.mark.parametrize("m,n", [(1, 37), (20, 64), (60, 300), (129, 1030), (300, 500), (1000, 6100)])
def test_scales_of_every_magnitude(dev, m, n, kind):
    """Scales whose product alone leaves float32's range, and zeros: what
    counts is the sum times both.  Sums are whole numbers below 2^24, exact;
    two products round (u |v| in all), the last perhaps to a subnormal (half
    of 2^-149)."""
    g = torch.Generator().manual_seed(m)
    x, w = ints((m, 64), 9, g), ints((n, 64), 9, g)
    x[m // 2], w[5] = 0, 0
    x[0], w[1] = -128 if kind == I8 else 448, -128 if kind == I8 else -448
    far = torch.tensor([1e-22, 1e22, 2.0 ** -140, 1e-38, 1e30, 2.0 ** 120, 1e-28, 1e26, 1.0, 0.0])
    sx, sw = far[torch.randint(0, 10, (m,), generator=g)], -far[torch.randint(0, 10, (n,), generator=g)]
    sx[0], sw[1], sw[2], sw[3] = 1e-22, -1e-22, 1e22, 1e30
    want = (x @ w.t()) * sx[:, None].double() * sw.double()
    xd, wd = padded(x, kind, dev, 0), padded(w, kind, dev, 0)
    got = cm.linear(xd, wd, sx.to(dev), sw.to(dev), out_dtype=F32).cpu()
    over = want.float().isinf()
    assert torch.equal(got[over], want.float()[over]) and torch.isfinite(got[~over]).all()
    err = (got.double() - want)[~over].abs()
    assert (err <= U * want[~over].abs() + 2.0 ** -150).all()
    # powers of two that cancel change nothing
    one = torch.ones(m, device=dev), torch.ones(n, device=dev)
    for act in ACTS:
        rows, cols = (wd[:n // 2 * 2], one[1][:n // 2 * 2]) if act == "swiglu" else (wd, one[1])
        plain = cm.linear(xd, rows, one[0], cols, act=act, out_dtype=F32)
        for e in (-110, -80, 80, 110):
            assert torch.equal(cm.linear(xd, rows, one[0] * 2.0 ** e, cols * 2.0 ** -e, act=act, out_dtype=F32), plain)
