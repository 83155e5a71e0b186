"""GPU parity of coli_moe_balance and coli_moe_balance_grad against the
formulas in 64 bits on the host, and of the gradient against differences of
the loss.

Tolerances, in units u = 2^-23 (two half steps of float32).  A score is an
exponential (argument reduced with a two-part ln 2: at most 3 u) and for
sigmoid a quotient (2 u, the derivative 3 u); its sum over the experts adds
at most 14 float32 additions of positive terms (7 u), a share one division
and one product: 14 u.  A loss adds the shares of positive weight in float32
over the at most 4 + 16 additions a wave and its workgroup make of a chunk of
64 tokens (10 u, half a step each) and continues in float64: 26 u.  An element of the gradient is scale * slope
* (c - m), with m a sum of 14 terms c_j p_j of any sign: its error is at most
48 u of scale * slope * (|c| + sum |c_j| p_j)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import routed_expert_ffn_f32_amd as cm

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
ALPHA = 0.01


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def make(T, E, k, seed, drop=0.1):
    rng = np.random.default_rng(seed)
    z = (rng.standard_normal((T, E)) * 2 + rng.standard_normal(E)).astype(np.float32)
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    idx[rng.random((T, k)) < drop] = -1
    return z, np.ascontiguousarray(idx), rng


def shares(z, scores):
    """(shares, derivative factor) of rows z in float64."""
    z = z.astype(np.float64)
    if scores == "softmax":
        top = np.max(z, axis=1, keepdims=True)
        e = np.exp(z - np.where(np.isfinite(top), top, 0.0))
        d = e
    else:
        e = 1 / (1 + np.exp(-z))
        d = e * (1 / (1 + np.exp(z)))
    tot = e.sum(1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        return np.where(tot > 0, e / tot, 0.0), np.where(tot > 0, d / tot, 0.0)


def reference(z, idx, off, mask, scores, alpha, dloss):
    """loss, counts, coef, gradient (NaN in rows of no sequence) and the gradient's error unit."""
    (T, E), S = z.shape, len(off) - 1
    loss, counts, coef = np.zeros(S), np.zeros((S, E), np.int64), np.zeros((S, E))
    d, unit = np.full((T, E), np.nan), np.zeros((T, E))
    for s in range(S):
        rows = np.arange(off[s], off[s + 1])
        d[rows] = 0.0
        rows = rows[mask[rows]]
        ids = idx[rows]
        ids = ids[(ids >= 0) & (ids < E)]
        counts[s] = np.bincount(ids, minlength=E)
        if len(rows) == 0:
            continue
        p, slope = shares(z[rows], scores)
        if len(ids):
            coef[s] = alpha / len(rows) * (E * counts[s] / len(ids) - 1)
            loss[s] = alpha * np.sum(E * counts[s] / len(ids) * p.sum(0) / len(rows))
        m = p @ coef[s]
        d[rows] = dloss[s] * slope * (coef[s] - m[:, None])
        unit[rows] = abs(dloss[s]) * slope * (np.abs(coef[s]) + (p @ np.abs(coef[s]))[:, None])
    return loss, counts, coef, d, unit


def check(dev, z, idx, off, mask, scores, dloss=None, alpha=ALPHA, tokens_per_chunk=64, stride_pad=0):
    T, E = z.shape
    S = len(off) - 1
    up = np.ones(S) if dloss is None else dloss.astype(np.float64)
    loss, counts, coef, d, unit = reference(z, idx, off, np.ones(T, bool) if mask is None else mask, scores,
                                            float(np.float32(alpha)), up)
    zd = torch.full((T, E + stride_pad), float("nan"), device=dev)
    zd[:, :E] = torch.from_numpy(z)
    zd = zd[:, :E]
    kw = dict(scores=scores, offsets=torch.from_numpy(np.asarray(off, np.int32)).to(dev),
              mask=None if mask is None else torch.from_numpy(mask).to(dev))
    gl, gc, gf = cm.balance_loss(zd, torch.from_numpy(idx).to(dev), alpha, **kw)
    out = torch.full((T, E + stride_pad), 7.0, device=dev)
    cm.balance_grad(zd, gf, None if dloss is None else torch.from_numpy(dloss).to(dev), out=out[:, :E], **kw)
    torch.cuda.synchronize()
    assert np.array_equal(gc.cpu().numpy(), counts)
    extra = max(0, tokens_per_chunk - 64) / 16  # additions of a wave beyond the four of 64 tokens
    gl = gl.cpu().numpy().astype(np.float64)
    assert (np.abs(gl - loss) <= (26 + extra / 2) * U * np.abs(loss)).all(), (gl, loss)
    cmax = np.abs(coef) + alpha * 1e-30
    assert (np.abs(gf.cpu().numpy() - coef) <= 2 * U * cmax).all()
    g = out.cpu().numpy().astype(np.float64)
    assert (g[:, E:] == 7.0).all()
    g = g[:, :E]
    none = np.isnan(d[:, 0])
    assert (g[none] == 7.0).all(), "rows of no sequence were written"
    err = np.abs(g[~none] - d[~none])
    assert (err <= 48 * U * unit[~none] + 1e-37).all(), float((err / (unit[~none] + 1e-300)).max() / U)
    return gl, gc, gf, g


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 1), (2, 8, 2), (5, 63, 3), (64, 64, 8), (33, 65, 4), (31, 128, 6),
                                   (257, 200, 8), (300, 256, 8), (100, 257, 32), (77, 512, 16)])
def test_sizes(dev, T, E, k, scores):
    z, idx, rng = make(T, E, k, T * 1000 + E)
    check(dev, z, idx, [0, T], None, scores)
    # ragged sequences (empty ones among them), masked tokens, rows before the first and behind the last
    cuts = np.sort(rng.integers(0, T + 1, size=6))
    check(dev, z, idx, cuts, rng.random(T) < 0.7, scores, rng.standard_normal(5).astype(np.float32), stride_pad=3)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_long_and_many_sequences(dev, scores):
    """More tokens than the sums' largest number of workgroups takes at 64
    each; a sequence per token; one sequence over every workgroup."""
    z, idx, rng = make(20011, 40, 4, 1)
    per = -(-20011 // 256)
    check(dev, z, idx, [0, 20011], rng.random(20011) < 0.9, scores, tokens_per_chunk=per)
    check(dev, z[:700], idx[:700], np.arange(701), None, scores)
    check(dev, z[:700], idx[:700], np.repeat([0, 5, 5, 300, 700], 50), None, scores)
    # more sequences than one load of bounds shows, most of them empty
    rng = np.random.default_rng(8)
    for n in (64, 65, 130, 5000):
        check(dev, z[:900], idx[:900], np.sort(rng.integers(3, 890, size=n + 1)), None, scores)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_masked_and_infinite_logits(dev, scores):
    """Masked rows hold NaN and Inf and are not looked at; -Inf takes an
    expert out of a token's reach; a token and a sequence with nothing left
    give zeros; every slot dropped gives loss 0 and gradient 0."""
    z, idx, rng = make(48, 70, 5, 9)
    mask = rng.random(48) < 0.6
    mask[:16] = False           # the first sequence is masked altogether
    z[~mask] = rng.choice([np.nan, np.inf, -np.inf], size=(int((~mask).sum()), 70))
    mask[20] = mask[21] = True
    z[20] = -np.inf             # a token without any expert
    z[21, 1:] = -np.inf         # and one with a single one
    z[21, 0] = 1.5
    z[mask] = np.where(rng.random((int(mask.sum()), 70)) < 0.2, -np.inf, z[mask])
    z[21, 0] = 1.5
    idx[32:] = -1               # the last sequence kept no assignment
    idx[30, 0], idx[31, 0] = 70, 1 << 30  # not experts
    mask[30] = mask[31] = True
    z[30:32] = rng.standard_normal((2, 70))
    gl, gc, gf, g = check(dev, z, idx, [0, 16, 32, 48], mask, scores)
    assert gl[0] == 0 and gl[2] == 0 and not g[:16].any() and not g[20].any() and not g[32:].any()


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_extreme_logits(dev, scores):
    """Logits of large magnitude overflow nothing."""
    rng = np.random.default_rng(4)
    z = (rng.standard_normal((40, 33)) * np.exp(rng.uniform(-3, 5, size=(40, 1)))).astype(np.float32)
    z[0], z[1], z[2] = 3e38, -80.0, 80.0
    z[3, :5] = [1e30, -1e30, 0, 88, -88]
    z[4] = 0
    idx = np.argsort(-z, axis=1)[:, :4].astype(np.int32)
    with np.errstate(over="ignore"):
        check(dev, z, np.ascontiguousarray(idx), [0, 11, 40], None, scores)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_gradient_against_differences(dev, scores):
    """Central differences of the loss (counts held) in 64 bits: their own
    error is about h^2 and 2^-53 / h of the loss."""
    z, idx, rng = make(6, 12, 3, 3, drop=0.2)
    off, up = [0, 4, 6], np.array([1.5, -0.5], np.float32)
    _, counts, _, g = check(dev, z, idx, off, None, scores, up)
    counts = counts.cpu().numpy()

    def total(zz):
        v = 0.0
        for s in range(2):
            p, _ = shares(zz[off[s]:off[s + 1]], scores)
            f = 12 * counts[s] / counts[s].sum()
            v += float(up[s]) * ALPHA * np.sum(f * p.mean(0))
        return v

    h = 1e-4
    for t in range(6):
        for e in range(12):
            a, b = z.astype(np.float64), z.astype(np.float64)
            a[t, e] += h
            b[t, e] -= h
            assert abs((total(a) - total(b)) / (2 * h) - g[t, e]) <= 1e-6 * ALPHA, (t, e)


def test_default_arguments_and_repeatability(dev):
    """No offsets, mask or upstream gradient; the same call twice gives the
    same bits."""
    z, idx, _ = make(5000, 256, 8, 6)
    zd, id_ = torch.from_numpy(z).to(dev), torch.from_numpy(idx).to(dev)
    a = cm.balance_loss(zd, id_, ALPHA)
    b = cm.balance_loss(zd, id_, ALPHA)
    ga, gb = cm.balance_grad(zd, a[2]), cm.balance_grad(zd, b[2])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((*a, ga), (*b, gb)))
    loss, counts, _, d, unit = reference(z, idx, [0, 5000], np.ones(5000, bool), "sigmoid", float(np.float32(ALPHA)),
                                         [1.0])
    assert np.array_equal(a[1].cpu().numpy(), counts)
    assert abs(float(a[0]) - loss[0]) <= 26 * U * loss[0]
    assert (np.abs(ga.cpu().numpy() - d) <= 48 * U * unit).all()


def test_no_tokens(dev):
    loss, counts, coef = cm.balance_loss(torch.empty(0, 16, device=dev), torch.empty(0, 2, dtype=torch.int32, device=dev),
                                         ALPHA, offsets=torch.zeros(4, dtype=torch.int32, device=dev))
    g = cm.balance_grad(torch.empty(0, 16, device=dev), coef, offsets=torch.zeros(4, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    assert not loss.any() and not counts.any() and not coef.any() and loss.shape == (3,) and g.shape == (0, 16)


def test_graph_replays_and_two_graphs(dev):
    """Two captured graphs, replayed in turn with eager work between them, on
    new inputs each time: every result is the eager one."""
    data = [make(3000, 256, 8, 50 + i)[:2] for i in range(3)]
    data = [(torch.from_numpy(z).to(dev), torch.from_numpy(i).to(dev)) for z, i in data]
    off = torch.tensor([0, 1000, 1010, 2990], dtype=torch.int32, device=dev)
    want = []
    for z, i in data:
        loss, counts, coef = cm.balance_loss(z, i, ALPHA, offsets=off)
        want.append((loss, counts, coef, cm.balance_grad(z, coef, offsets=off)))
    graphs = []
    for _ in range(2):
        z, i = data[0][0].clone(), data[0][1].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            loss, counts, coef = cm.balance_loss(z, i, ALPHA, offsets=off)
            d = cm.balance_grad(z, coef, offsets=off)
        graphs.append((g, z, i, (loss, counts, coef, d)))
    for rep in range(4):
        for n, (g, z, i, out) in enumerate(graphs):
            k = (rep + n) % 3
            z.copy_(data[k][0])
            i.copy_(data[k][1])
            g.replay()
            eager = cm.balance_loss(*data[(k + 1) % 3], ALPHA, offsets=off)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want[k])), (rep, n)
            assert all(torch.equal(a, b) for a, b in zip(eager, want[(k + 1) % 3][:3]))


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E", [(48, 70), (300, 256), (300, 20)])
def test_nan_stays_visible_and_where_it_is(dev, T, E, scores):
    """A valid token's NaN logit makes its sequence's loss and its own row of
    the gradient NaN, and nothing else; so does +Inf under softmax."""
    z, idx, _ = make(T, E, 4, 77)
    off = [0, 10, 20, T - 9, T]
    od = torch.tensor(off, dtype=torch.int32, device=dev)
    zd, ids = torch.from_numpy(z).to(dev), torch.from_numpy(idx).to(dev)
    want = cm.balance_loss(zd, ids, ALPHA, scores, od)
    dwant = cm.balance_grad(zd, want[2], None, scores, od)
    for bad in [float("nan")] + ([float("inf")] if scores == "softmax" else []):
        zn = zd.clone()
        zn[13, E // 2] = bad
        loss, counts, coef = cm.balance_loss(zn, ids, ALPHA, scores, od)
        d = cm.balance_grad(zn, coef, None, scores, od)
        assert loss.isnan().tolist() == [False, True, False, False]
        assert torch.equal(loss[[0, 2, 3]], want[0][[0, 2, 3]]) and torch.equal(counts, want[1])
        assert torch.equal(coef, want[2])
        assert d[13].isnan().all() and torch.equal(d[:13], dwant[:13]) and torch.equal(d[14:], dwant[14:])


def test_scores_at_the_end_of_their_range(dev):
    """All of a token's sigmoid scores just above 2^-126: shares and gradient
    hold, also with a large upstream gradient.  All below: shares and
    gradient 0."""
    z, idx, rng = make(20, 12, 3, 5)
    z = (rng.uniform(-87.3, -84.0, size=z.shape)).astype(np.float32)  # exp(-87.3) = 2^-125.95
    up = np.array([3e4, -3e4], np.float32)
    # the error unit of d carries dloss: 3e4 * alpha / 20 * 48 U, far above 1e-37
    check(dev, z, idx, [0, 10, 20], None, "sigmoid", up)
    low = torch.full((20, 12), -95.0, device=dev)
    ids = torch.from_numpy(idx).to(dev)
    loss, _, coef = cm.balance_loss(low, ids, ALPHA)
    assert loss.tolist() == [0.0] and not cm.balance_grad(low, coef).any()


def many_sequences(kind):
    rng = np.random.default_rng(31)
    if kind == "63 short, one long":    # the long one is the last that the first window of bounds shows
        return 32768, np.r_[np.arange(64), 32768]
    if kind == "64 short, one long":
        return 32768, np.r_[np.arange(65), 32768]
    if kind == "random":
        return 65536, np.r_[0, np.sort(rng.integers(0, 65537, 3899)), 65536]
    if kind == "equal":
        return 78000, np.arange(0, 78001, 20)
    if kind == "empty between":         # rows before the first and behind the last, windows of empty sequences
        return 40000, np.sort(np.r_[np.repeat([5, 5, 700, 20001], 100), rng.integers(5, 39001, 200)])
    return 1 << 20, np.r_[0, np.sort(rng.integers(0, (1 << 20) + 1, 16383)), 1 << 20]


@pytest.mark.parametrize("kind", ["63 short, one long", "64 short, one long", "random", "equal", "empty between", "largest"])
def test_many_sequences_over_several_batches(dev, kind):
    """More sequences than one load of bounds shows, in workgroups of several
    batches: every token and choice is counted once, in its own sequence.  The
    workspace holds NaN before the call, so that a sum of anything unwritten
    shows.  The logits are equal, so every token's shares are 1 / E, and E = 4
    makes the shares and their sums (under 2^24 tokens of 1/4) exact: a loss
    is alpha up to the float32 rounding of alpha's product, 2 half steps."""
    T, off = many_sequences(kind)
    S, E, k = len(off) - 1, 4, 2
    rng = np.random.default_rng(T)
    idx = rng.integers(-1, E, size=(T, k)).astype(np.int32)
    mask = rng.random(T) < 0.9
    seq = np.searchsorted(off[1:], np.arange(T), side="right")
    inside = (np.arange(T) >= off[0]) & (seq < S) & mask
    rows = np.repeat(np.where(inside, seq, S), k)
    flat = idx.reshape(-1)
    keep = (flat >= 0) & (rows < S)
    counts = np.zeros((S, E), np.int64)
    np.add.at(counts, (rows[keep], flat[keep]), 1)
    valid = np.bincount(seq[inside], minlength=S)[:S]
    n = counts.sum(1)
    some = (n > 0) & (valid > 0)
    with np.errstate(invalid="ignore", divide="ignore"):
        coef = np.where(some[:, None], float(np.float32(ALPHA)) / valid[:, None] * (E * counts / n[:, None] - 1), 0.0)
    z = torch.zeros(T, E, device=dev)
    it, ot, mt = (torch.from_numpy(np.ascontiguousarray(v)).to(dev) for v in (idx, off.astype(np.int32), mask))
    loss, cnt = torch.full((S,), float("nan"), device=dev), torch.full((S, E), -1, dtype=torch.int32, device=dev)
    cf = torch.full((S, E), float("nan"), device=dev)
    ws = torch.full((cm.coli_moe_balance_workspace_bytes(T, E, S) // 4,), float("nan"), device=dev)
    args = cm.coli_moe_balance_t(T, E, k, S, cm.COLI_MOE_SCORES_SOFTMAX, ALPHA, z.data_ptr(), E, it.data_ptr(),
                                 ot.data_ptr(), mt.data_ptr())
    cm.coli_moe_balance(args, loss.data_ptr(), cnt.data_ptr(), cf.data_ptr(), ws.data_ptr(), 4 * ws.numel(),
                        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert np.array_equal(cnt.cpu().numpy(), counts)
    want = np.where(some, float(np.float32(ALPHA)), 0.0)
    assert (np.abs(loss.cpu().numpy() - want) <= U * want).all()
    # one rounding to float32; in 64 bits a quotient, a product and a difference, each off by 2^-53 of E n_e / N or 1
    got = cf.cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        off64 = np.where(some[:, None], 4 * 2.0 ** -53 * ALPHA / valid[:, None] * (E * counts / n[:, None] + 1), 0.0)
    assert (np.abs(got - coef) <= U * np.abs(coef) + off64).all()
    dl = torch.full((T, E), 7.0, device=dev)
    cm.coli_moe_balance_grad(args, cf.data_ptr(), None, dl.data_ptr(), E, torch.cuda.current_stream().cuda_stream)
    d = dl.cpu().numpy().astype(np.float64)
    nowhere = (np.arange(T) < off[0]) | (seq >= S)
    assert (d[nowhere] == 7.0).all() and not d[~nowhere & ~mask].any()
    c = got[seq[inside]]
    unit = 0.25 * (np.abs(c) + 0.25 * np.abs(c).sum(1, keepdims=True))
    assert (np.abs(d[inside] - 0.25 * (c - c.mean(1, keepdims=True))) <= 48 * U * unit + 1e-37).all()


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_gradient_reaches_a_router(dev, scores):
    """The documented way from the loss to a router's weights, against autograd
    of the formula in 64 bits.  Tolerance: the gradient's 48 u on every element
    and the float32 product's sum of T terms, both of sum |x| |dz|."""
    g = torch.Generator().manual_seed(11)
    T, E, h, k = 50, 24, 40, 3
    x, w = torch.randn(T, h, generator=g), torch.randn(h, E, generator=g) / 6
    wd = w.to(dev).requires_grad_()
    logits = x.to(dev) @ wd
    idx = torch.topk(logits.detach(), k, dim=1).indices.to(torch.int32)
    off = torch.tensor([0, 20, T], dtype=torch.int32, device=dev)
    loss, counts, coef = cm.balance_loss(logits, idx, ALPHA, scores, off)
    assert not loss.requires_grad
    d = cm.balance_grad(logits, coef, None, scores, off)
    logits.backward(d)
    # the same logits in 64 bits (as rounded by the product), their gradient by autograd
    z = logits.detach().cpu().double().requires_grad_()
    total = 0.0
    for s in range(2):
        zs = z[off[s]:off[s + 1]]
        e = torch.exp(zs - zs.detach().amax(1, keepdim=True)) if scores == "softmax" else 1 / (1 + torch.exp(-zs))
        p = e / e.sum(1, keepdim=True)
        n = counts[s].cpu().double()
        total = total + float(np.float32(ALPHA)) * (E * n / n.sum() * p.mean(0)).sum()
    total.backward()
    total = float(total.detach())
    assert abs(float(loss.sum()) - total) <= 27 * U * total
    _, _, _, _, unit = reference(logits.detach().cpu().numpy(), idx.cpu().numpy(), off.tolist(), np.ones(T, bool), scores,
                                 float(np.float32(ALPHA)), np.ones(2))
    want = x.double().t() @ z.grad
    tol = x.double().abs().t() @ (48 * U * torch.from_numpy(unit) + T * U * z.grad.abs())
    assert ((wd.grad.cpu().double() - want).abs() <= tol).all()
