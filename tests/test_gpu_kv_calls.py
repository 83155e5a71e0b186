"""Rotary positions and the 4-bit cache as a program uses them: together in a
block, captured and replayed, on other streams and from threads, in caches
whose offsets pass 32 bits, with values that are no numbers, and the calls
that are refused on the device."""
import threading

import pytest

torch = pytest.importorskip("torch")

import routed_expert_ffn_f32_amd as cm
import synth
from tests import kv_ref
from tests.gpu_util import DeviceLayer
from tests.kv_ref import Pool, U, offsets_of, unpack

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def ints(values, dev):
    return torch.tensor(values, dtype=I32, device=dev)


def test_block(dev):
    """norm, projections, rotary positions, append, attention, projection and
    the routed layer, a prompt and then single tokens; every operator's result
    against its formula on what it was given."""
    shape = synth.TINY
    H, heads, group, dim, page, prompt, steps = shape.hidden, 2, 2, 64, 16, 37, 3
    hq = heads * group
    layer = DeviceLayer(shape, 1, 0, dev, max_tokens=64)
    g = torch.Generator().manual_seed(5)
    wqkv = (torch.randn((hq + 2 * heads) * dim, H, generator=g) / 16).bfloat16()
    wo = (torch.randn(H, hq * dim, generator=g) / 16).bfloat16()
    d_wqkv, d_wo = wqkv.to(dev), wo.to(dev)
    freq, fscale = cm.rotary_frequencies(dim, device=dev)
    pool = Pool([prompt + steps], heads, dim, page, seed=1)
    cache = pool.to(dev, cm, weights=False)
    table = pool.table.to(dev)
    at = 0
    for n in [prompt] + [1] * steps:
        x = (torch.randn(n, H, generator=g)).bfloat16().to(dev)
        pos = torch.arange(at, at + n, device=dev)
        at += n
        lengths, off = ints([at], dev), ints([0, n], dev) if n > 1 else None
        y = cm.rms_norm(x)
        qkv = cm.linear(y, d_wqkv).view(n, hq + 2 * heads, dim)
        ref = y.cpu().double() @ wqkv.double().t()
        mass = y.cpu().double().abs() @ wqkv.double().abs().t()
        assert ((qkv.flatten(1).cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + H * U * mass).all()
        before = qkv.clone()
        qk = qkv[:, : hq + heads]
        assert cm.rotary(qk, pos, freq, scale=fscale, out=qk) is qk
        angle = pos.cpu().double()[:, None] * freq.cpu().double()
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        a, b = before[:, : hq + heads].cpu().double().split(dim // 2, -1)
        want = torch.cat([a * c - b * s, a * s + b * c], -1)
        # angles reduced in 64 bits, then a handful of float32 roundings and the type's
        size = (a.abs() + b.abs()).repeat(1, 1, 2)
        assert ((qk.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 16 * U * size).all()
        assert torch.equal(qkv[:, hq + heads:], before[:, hq + heads:])
        cache.append(qkv[:, hq: hq + heads], qkv[:, hq + heads:], table, lengths, off)
        host = qkv.cpu().float()
        for i in range(n):
            pool.write(0, at - n + i, host[i, hq: hq + heads], host[i, hq + heads:])
        pool.lengths = [at]
        o = cache.attention(qkv[:, :hq], table, lengths, off)
        out, tol, _, _ = kv_ref.attention(pool, host[:, :hq].bfloat16(), [n])
        assert ((o.cpu().double() - out).abs() <= tol).all()
        z = cm.linear(o.flatten(1), d_wo, residual=x)
        ref = o.flatten(1).cpu().double() @ wo.double().t()
        mass = o.flatten(1).cpu().double().abs() @ wo.double().abs().t()
        total = ref + x.cpu().double()
        size = mass + total.abs()
        assert ((z.cpu().double() - total).abs() <= 2.0 ** -8 * total.abs() + (hq * dim + 2) * U * size).all()
        got, want = layer.moe.forward_normed(z), layer.moe.forward(cm.rms_norm(z.float()))
        assert torch.isfinite(got).all() and (got != 0).any() and got.shape == want.shape == (n, H)
    layer.close()
    for name in ("k_codes", "v_codes"):
        assert torch.equal(getattr(cache, name).cpu(), getattr(pool, name))


def step(cache, table, lengths, off, x, heads, q_heads, pos, freq, **kw):
    """One attention step on a fused [tokens, q + 2 kv, dim] projection."""
    qk = cm.rotary(x[:, : q_heads + heads], pos, freq)
    cache.append(qk[:, q_heads:], x[:, q_heads + heads:], table, lengths, off)
    return cache.attention(qk[:, :q_heads], table, lengths, off, **kw)


@pytest.mark.parametrize("new,window", [([1, 1, 1], 0), ([3, 0, 6], 0), ([90, 1, 40], 70)])
def test_captured(dev, new, window):
    """A captured step replayed as the sequences grow, with eager work between,
    beside another graph of the same kind: each replay equals the eager step
    on a copy of the cache, bit for bit."""
    heads, group, dim, page = 2, 4, 64, 16
    T, hq = sum(new), heads * group
    lengths = [140, 40, 100]
    order = torch.randperm(3 * 32, generator=torch.Generator().manual_seed(1)).to(I32)
    caches = [cm.KVCache.empty(3 * 32, heads, dim, page, weights=True, device=dev) for _ in range(2)]
    twin = cm.KVCache.empty(3 * 32, heads, dim, page, weights=True, device=dev)
    table = order.view(3, 32).to(dev)
    freq, _ = cm.rotary_frequencies(dim, device=dev)
    off = offsets_of(new).to(dev) if max(new) > 1 else None
    x = torch.zeros(T, hq + 2 * heads, dim, dtype=BF16, device=dev)
    lens, pos = ints(lengths, dev), torch.zeros(T, dtype=torch.int64, device=dev)
    kw = dict(window=window, accumulate=True)
    outs, graphs = [], []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # first calls outside of a capture
        step(caches[0], table, lens, off, x, heads, hq, pos, freq, **kw)
        caches[0].weights.zero_()
    side.synchronize()
    for c in caches:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(c, table, lens, off, x, heads, hq, pos, freq, **kw))
        graphs.append(graph)
    for c in caches:
        for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales, c.weights):
            t.zero_()
    g = torch.Generator().manual_seed(4)
    for turn in range(5):
        x.copy_(torch.randn(x.shape, generator=g))
        pos.copy_(torch.arange(T) + 10 * turn)
        lens.copy_(ints([n + turn * m for n, m in zip(lengths, [7, 3, 11])], dev))
        for graph in graphs:
            graph.replay()
        want = step(twin, table, lens, off, x, heads, hq, pos, freq, **kw)
        if turn % 2:
            torch.cuda.synchronize()
        for out, c in zip(outs, caches):
            assert torch.equal(out, want), turn
            assert torch.equal(c.weights, twin.weights) and torch.equal(c.k_codes, twin.k_codes), turn
    assert float(twin.weights.sum()) > 0


def test_eviction_captured(dev):
    pool = Pool([90, 20], 2, 64, 16, seed=3, spare=48).fill()
    a, b = pool.to(dev, cm), pool.to(dev, cm)
    table, into, lens = pool.table.to(dev), pool.into.to(dev), ints([90, 20], dev)
    want = a.evict(40, table, lens, into, first=2, recent=5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.evict(40, table, lens, into, first=2, recent=5)
    for turn in range(3):
        graph.replay()
        want = a.evict(40, table, lens, into, first=2, recent=5)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(b.k_codes, a.k_codes) and torch.equal(b.weights, a.weights)
        for c in (a, b):
            c.weights.mul_(-1)


def test_side_stream_and_threads(dev):
    """Calls on streams of their own, from threads of their own, each on its
    own cache: the results of the calls made alone."""
    def work(seed):
        pool = Pool([200, 70], 2, 128, 32, seed=seed).fill(seed)
        q = torch.randn(12, 4, 128, generator=torch.Generator().manual_seed(seed)).bfloat16()
        return pool, q
    jobs = [work(s) for s in range(3)]
    args = [(p.to(dev, cm), p.table.to(dev), ints(p.lengths, dev), offsets_of([5, 7]).to(dev), q.to(dev)) for p, q in jobs]
    alone = [c.attention(q, t, n, o, accumulate=True) for c, t, n, o, q in args]
    sums = [a[0].weights.clone() for a in args]
    again = [p.to(dev, cm) for p, _ in jobs]
    torch.cuda.synchronize()
    results, errors = [None] * 3, []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                _, t, n, o, q = args[i]
                for _ in range(20):
                    results[i] = again[i].attention(q, t, n, o, weights_out=torch.zeros_like(again[i].weights))
                results[i] = again[i].attention(q, t, n, o, accumulate=True)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for i in range(3):
        assert torch.equal(results[i], alone[i]) and torch.equal(again[i].weights, sums[i])


@pytest.mark.parametrize("tokens", [2, 80])
def test_offsets_past_32_bits(dev, tokens):
    """A pool whose rows of codes lie past 4 GiB: append, read, attention,
    weights and eviction at its far end."""
    dim, page, heads, pages = 256, 256, 8, 17000  # 4.15 GiB of codes each
    shape = (pages, heads, page)
    cache = cm.KVCache(torch.empty((*shape, dim // 2), dtype=torch.uint8, device=dev),
                       torch.empty((pages, heads, dim // 64, page), dtype=BF16, device=dev),
                       torch.empty((*shape, dim // 2), dtype=torch.uint8, device=dev),
                       torch.empty((pages, heads, dim // 64, page), dtype=BF16, device=dev),
                       torch.zeros(shape, device=dev))
    n = 300
    g = torch.Generator().manual_seed(7)
    small = cm.KVCache.empty(4, heads, dim, page, weights=True, device=dev)
    k, v = (torch.randn(n, heads, dim, generator=g).bfloat16().to(dev) for _ in "kv")
    q = torch.randn(tokens, heads, dim, generator=g).bfloat16().to(dev)
    results = []
    for c, pagenos, into in ((cache, [pages - 1, pages - 7], [pages - 3, pages - 2]), (small, [0, 2], [1, 3])):
        table, lens = ints([pagenos], dev), ints([n], dev)
        c.append(k, v, table, lens, ints([0, n], dev))
        out = c.attention(q, table, lens, ints([0, tokens], dev), accumulate=True)
        kept, new = c.evict(100, table, lens, ints([into], dev))
        results.append((out, *c.read(n, table, lens, ints([0, n], dev)), c.weights[pagenos], kept, new,
                        *c.read(100, ints([into], dev), new, ints([0, 100], dev))))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    far = torch.empty(((1 << 31) // 4096 + 2) * 4096, dtype=BF16, device=dev)  # rows of heads past 2^31 elements
    x = far.as_strided((2, 3, 64), (1 << 31, 64, 1))
    x.copy_(torch.randn(2, 3, 64, generator=g))
    freq, _ = cm.rotary_frequencies(64, device=dev)
    pos = ints([3, 1 << 20], dev)
    near = cm.rotary(x.contiguous(), pos, freq)
    assert torch.equal(cm.rotary(x, pos, freq), near)
    cm.rotary(x, pos, freq, out=x)
    assert torch.equal(x, near)


@pytest.mark.parametrize("tokens", [5, 90])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_queries_that_are_no_numbers(dev, tokens, bad):
    """A row with one stays its own matter, whatever rows share its tile."""
    pool = Pool([200], 1, 128, 64, seed=9).fill()
    q = torch.randn(tokens, 4, 128, generator=torch.Generator().manual_seed(1)).half()
    out, tol, _, _ = kv_ref.attention(pool, q, [tokens])
    q[3, 1, 70] = bad
    got = pool.to(dev, cm).attention(q.to(dev), pool.table.to(dev), ints([200], dev), ints([0, tokens], dev)).cpu()
    assert not torch.isfinite(got[3, 1]).any()
    got[3, 1], out[3, 1] = 0, 0
    assert ((got.double() - out).abs() <= tol).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("far", [2.0 ** 40, 2.0 ** 90, 2.0 ** -90])
@pytest.mark.parametrize("tokens", [3, 40])
def test_values_far_apart(dev, dim, far, tokens):
    """64 rows of values many powers of two from the later ones, rows of zeros
    and a page that is not there in between: queries that see all and weigh
    the early ones, and queries that weigh the late ones alone."""
    pool = Pool([330], 1, dim, 64, seed=35)
    g = torch.Generator().manual_seed(36)
    toward = torch.randn(1, dim, generator=g)
    for r in range(330):
        early = r < 64
        k = (-8 if early else 1) * toward + 0.1 * torch.randn(1, dim, generator=g)
        v = torch.randn(1, dim, generator=g) * (far if early else 0.0 if 128 <= r < 192 else 1.0)
        pool.write(0, r, k, v)
    pool.table[0, 3] = -1
    way = 1.0 - 2.0 * (torch.arange(tokens) % 2).view(-1, 1, 1)
    q = (torch.randn(tokens, 2, dim, generator=g) + 3 * toward * way).bfloat16()
    out, tol, _, _ = kv_ref.attention(pool, q, [tokens])
    got = pool.to(dev, cm).attention(q.to(dev), pool.table.to(dev), ints([330], dev), ints([0, tokens], dev)).cpu()
    assert 1e-3 < float(out[0].abs().max()) < 1e3 and 1e-3 < float((out[1] / far).abs().max()) < 1e3
    assert ((got.double() - out).abs() <= tol).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("far", [2.0 ** 35, 2.0 ** 90])
@pytest.mark.parametrize("tokens", [3, 60])
def test_keys_far_apart(dev, dim, far, tokens):
    """One new row's key is many powers of two above all others: those that do
    not see it keep their results, and for those that do it is out of the
    question, or all of it."""
    pool, near = (Pool([150], 1, dim, 32, seed=37).fill() for _ in range(2))
    g = torch.Generator().manual_seed(38)
    toward, value = torch.randn(1, dim, generator=g), torch.randn(1, dim, generator=g)
    row = 150 - tokens + 1
    pool.write(0, row, -far * toward, value)
    near.write(0, row, -12 * toward, value)
    way = 1.0 - 2.0 * (torch.arange(tokens) % 3 == 2).float().view(-1, 1, 1)
    q = (torch.randn(tokens, 2, dim, generator=g) + toward * way).bfloat16()
    # 12 times is as good as far: either way its weight, or all others', is below 2^-36
    z = q.double() @ near.rows(0, 150)[0][:, 0].t() * dim ** -0.5
    far_z, rest = z[1:, :, row], torch.cat([z[1:, :, :row], z[1:, :, row + 1:]], -1)
    assert ((far_z < rest.amin(-1) - 30) | (far_z > rest.amax(-1) + 30)).all() and (far_z > 0).any()
    out, tol, _, _ = kv_ref.attention(near, q, [tokens])
    got = pool.to(dev, cm).attention(q.to(dev), pool.table.to(dev), ints([150], dev), ints([0, tokens], dev)).cpu()
    assert ((got.double() - out).abs() <= tol + 2.0 ** -30).all()


@pytest.mark.parametrize("dim,page", [(64, 32), (128, 16), (256, 64)])
@pytest.mark.parametrize("tokens", [1, 3, 45])
def test_codes_and_scales_of_a_users_own(dev, dim, page, tokens):
    """Codes of -8 and scales below 0, which append never makes, through the
    attention, its weights and reads."""
    pool = Pool([190], 2, dim, page, seed=61)
    g = torch.Generator().manual_seed(62)
    for scales in (pool.k_scales, pool.v_scales):
        scales.copy_(torch.randn(scales.shape, generator=g) / 3)
    assert (unpack(pool.k_codes) == -8).any() and (pool.k_scales < 0).any()
    q = torch.randn(tokens, 4, dim, generator=g).half()
    out, tol, w, wtol = kv_ref.attention(pool, q, [tokens])
    cache = pool.to(dev, cm)
    args = pool.table.to(dev), ints([190], dev), ints([0, tokens], dev)
    got = cache.attention(q.to(dev), *args, accumulate=True).cpu()
    assert ((got.double() - out).abs() <= tol).all()
    want = pool.weights.double() + w
    assert ((cache.weights.cpu().double() - want).abs() <= wtol + 2 * U * want)[w > 0].all()
    k, v, _, _, _ = pool.rows(0, 190)
    for a, b in zip(cache.read(tokens, *args, dtype=torch.float32), (k, v)):
        assert torch.equal(a.cpu().double(), b[190 - tokens:])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("tokens", [2, 50])
@pytest.mark.parametrize("length", [130, 2600])
def test_large_scores(dev, dim, tokens, length):
    """Scores of 10^8, far beyond what float32 tells apart, and of zeros: one
    key has all the weight, and queries of zeros weigh all keys alike, in
    splits too."""
    pool = Pool([length], 1, dim, 64, seed=41)
    pool.weights.zero_()
    g = torch.Generator().manual_seed(42)
    signs = 2.0 * torch.randint(0, 2, (length, 1, dim), generator=g) - 1
    for r in range(length):
        pool.write(0, r, signs[r] * 8192, torch.randn(1, dim, generator=g))
    q = torch.zeros(tokens, 3, dim)
    at = length - tokens + torch.arange(tokens)
    chosen = (at * 7919) % (length - tokens)
    q[:, 0], q[:, 1] = signs[chosen, 0] * 30000, signs[chosen, 0] * -30000
    q = q.half()
    cache = pool.to(dev, cm)
    sums = torch.zeros_like(cache.weights)
    args = pool.table.to(dev), ints([length], dev), ints([0, tokens], dev)
    got = cache.attention(q.to(dev), *args, weights_out=sums).cpu().double()
    v = pool.rows(0, length)[1][:, 0]
    assert (got[:, 0] - v[chosen]).abs().le(2.0 ** -11 * v[chosen].abs() + 2.0 ** -25).all()
    assert torch.isfinite(got).all()
    mean = v.cumsum(0)[at] / (at + 1).view(-1, 1)
    size = v.abs().cumsum(0)[at] / (at + 1).view(-1, 1)
    # a float32 sum, and weights of 22 bits
    assert (got[:, 2] - mean).abs().le(2.0 ** -11 * mean.abs() + (length + 128) * U * 8 * size + 2.0 ** -25).all()
    # Weights come from scores computed once more.  Neighbouring float32 numbers are 128 apart at 2^30, where these
    # scores are, so a sum in another order may fall short of the maximum by 2^-100 of its weight, or pass it, where
    # it counts 2^8 at most.  The queries of zeros have no such scores: each gives 1 in all.
    total = sums.double().sum().item()
    assert tokens * (1 - 2.0 ** -18) <= total <= 3 * 2 ** 8 * tokens


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 32)])
def test_weights_of_prompts_in_wide_tables(dev, dim, page):
    """The tables have room for far more rows than the sequences have, so that
    the weights are summed by workgroups of more keys; rows before the window,
    behind the end and on no page keep theirs."""
    new, lengths, heads, group = [40, 1, 70, 80], [600, 30, 71, 95], 2, 2
    pool = Pool(lengths, heads, dim, page, seed=31, capacity=1 << 15).fill()
    pool.table[0, 3] = -1
    q = torch.randn(sum(new), heads * group, dim, generator=torch.Generator().manual_seed(2)).bfloat16()
    for window in (0, 45):
        out, tol, w, wtol = kv_ref.attention(pool, q, new, window=window)
        cache = pool.to(dev, cm)
        sums = torch.full_like(cache.weights, -1.0)
        got = cache.attention(q.to(dev), pool.table.to(dev), ints(lengths, dev), offsets_of(new).to(dev), window=window,
                              weights_out=sums).cpu()
        assert ((got.double() - out).abs() <= tol).all()
        seen, sums, want = w > 0, sums.cpu(), pool.weights.double() + w
        assert ((sums.double() - want).abs() <= wtol + 2 * U * want)[seen].all()
        # a weight of no query that float32 rounds to nothing is still added
        assert ((sums == -1) | (sums.double() - want).abs().le(wtol + 2 * U * want))[~seen].all()


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 32)])
@pytest.mark.parametrize("seqs", [3, 700])
def test_weights_of_single_tokens_in_wide_tables(dev, dim, page, seqs):
    """As above, and more sequences than there are waves for parts of each."""
    lengths = [(37 * i) % 90 if i != 1 else 700 for i in range(seqs)]
    pool = Pool(lengths, 2, dim, page, seed=33, capacity=1 << 13)
    pool.k_scales.nan_to_num_(0.01)
    pool.v_scales.nan_to_num_(0.02)
    q = torch.randn(seqs, 4, dim, generator=torch.Generator().manual_seed(2)).half()
    few = [i for i in range(seqs) if i < 8 or i % 97 == 0]  # the oracle's
    cache = pool.to(dev, cm)
    sums = torch.full_like(cache.weights, -1.0)
    got = cache.attention(q.to(dev), pool.table.to(dev), ints(lengths, dev), weights_out=sums).cpu()
    for i in few:
        one = Pool([lengths[i]], 2, dim, page, seed=1)
        one.pages, one.table = pool.pages, pool.table[i: i + 1]
        one.k_codes, one.v_codes, one.k_scales, one.v_scales = pool.k_codes, pool.v_codes, pool.k_scales, pool.v_scales
        one.weights = pool.weights
        out, tol, w, wtol = kv_ref.attention(one, q[i: i + 1], [1])
        assert ((got[i: i + 1].double() - out).abs() <= tol).all()
        want = pool.weights.double() + w
        assert ((sums.cpu().double() - want).abs() <= wtol + 2 * U * want)[w > 0].all()
    # nothing but the rows of sequences is touched
    assert int((sums != -1).sum()) == 2 * sum(lengths)


@pytest.mark.parametrize("capacity", [64, 1 << 14])
def test_many_sequences(dev, capacity):
    """300 sequences of which a few have new tokens, so that hundreds begin
    at the same token; tokens before the first and behind the last."""
    new, lengths, dim = [0] * 300, [13 * i % 50 + 6 for i in range(300)], 64
    for i, n in ((0, 2), (1, 1), (95, 3), (96, 1), (200, 6), (299, 2)):
        new[i] = n
    pool = Pool(lengths, 1, dim, 16, seed=51, capacity=capacity).fill()
    T = sum(new) + 4
    g = torch.Generator().manual_seed(52)
    k, v, q = (torch.randn(T, 1, dim, generator=g).bfloat16() for _ in range(3))
    q = torch.cat([q, -q, q * 2], 1)
    cache = pool.to(dev, cm)
    args = pool.table.to(dev), ints(lengths, dev), (offsets_of(new) + 1).to(dev)
    cache.append(k.to(dev), v.to(dev), *args)
    want, t = torch.zeros(2, T, 1, dim), 1
    for s, n in enumerate(new):
        for i in range(n):
            pool.write(s, lengths[s] - n + i, k[t].float(), v[t].float())
            for x, into in ((k, want[0]), (v, want[1])):
                codes, scale = kv_ref.quantise(x[t].float())
                into[t] = (codes * scale.double().repeat_interleave(64, -1)).float()
            t += 1
    for name in ("k_codes", "v_codes"):
        assert torch.equal(getattr(cache, name).cpu(), getattr(pool, name))
    for a, b in zip(cache.read(T, *args, dtype=torch.float32), want):
        assert torch.equal(a.cpu(), b)
    out, tol, _, _ = kv_ref.attention(pool, q[1: 1 + sum(new)], new)
    got = cache.attention(q.to(dev), *args).cpu()
    assert ((got[1: 1 + sum(new)].double() - out).abs() <= tol).all()
    assert (got[0] == 0).all() and (got[1 + sum(new):] == 0).all()


def test_long_eviction(dev):
    """More rows than LDS holds keys of, many of them alike."""
    L, keep, page = 40000, 11111, 256
    pages = -(-L // page) + -(-keep // page)
    cache = cm.KVCache.empty(pages, 1, 64, page, weights=True, device=dev)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(I32)
    table, into = order[: -(-L // page)][None], order[-(-L // page):][None]
    w = torch.randint(0, 7, (L,), generator=torch.Generator().manual_seed(2)).float() / 8
    w[::1000] = float("nan")
    w[1::1000] = -0.0
    flat = torch.zeros(-(-L // page) * page)
    flat[:L] = w
    cache.weights[table[0].long().to(dev), 0] = flat.view(-1, page).to(dev)
    cache.k_codes.copy_(torch.randint(0, 256, cache.k_codes.shape, generator=torch.Generator().manual_seed(3)))
    before = cache.k_codes[:, 0].clone()
    kept, new = cache.evict(keep, table.to(dev), ints([L], dev), into.to(dev), first=4, recent=100)
    key = torch.where(w.isnan(), torch.tensor(9.0), w)
    key[:4] = 99
    key[-100:] = 99
    want = torch.sort(torch.sort(key, descending=True, stable=True).indices[:keep]).values
    assert torch.equal(kept[0, 0].cpu().long(), want) and int(new[0]) == keep
    rows = before[table[0].long().to(dev)].flatten(0, 1)[want.to(dev)]
    assert torch.equal(cache.k_codes[into[0].long().to(dev), 0].flatten(0, 1)[:keep], rows)


def test_lengths_of_any_value(dev):
    """Negative lengths, lengths past the table and no sequences at all."""
    pool = Pool([50, 50, 50], 1, 64, 16, seed=4).fill()
    cache, table = pool.to(dev, cm), pool.table.to(dev)
    x = torch.randn(3, 1, 64, generator=torch.Generator().manual_seed(1)).bfloat16().to(dev)
    lens = ints([-5, 2 ** 31 - 1, -2 ** 31], dev)
    cache.append(x, x, table, lens)
    for got, kept in zip((cache.k_codes, cache.k_scales, cache.weights), (pool.k_codes, pool.k_scales, pool.weights)):
        assert torch.equal(got.cpu().nan_to_num(3), kept.nan_to_num(3))
    out = cache.attention(x, table, lens, accumulate=True)
    assert (out[0] == 0).all() and (out[2] == 0).all()
    k, v = cache.read(3, table, lens)
    assert (k == 0).all() and (v == 0).all()
    kept, new = cache.evict(10, table, ints([-1, 0, -2 ** 31], dev), pool.table[:, :2].contiguous().to(dev))
    assert (kept == -1).all() and (new == 0).all()
    none, off = torch.empty(0, 4, dtype=I32, device=dev), ints([0], dev)
    empty = torch.empty(0, dtype=I32, device=dev)
    assert (cache.attention(x, none, empty, off) == 0).all()
    assert all((t == 0).all() for t in cache.read(3, none, empty, off))
    assert cache.evict(4, none, empty, none)[0].shape == (0, 1, 4)
    cache.append(x, x, none, empty, off)
    assert cache.attention(x[:0], table, lens, ints([0, 0, 0, 0], dev)).shape == (0, 1, 64)


def test_refusals_on_the_device(dev):
    cache = cm.KVCache.empty(4, 2, 64, 16, weights=True, device=dev)
    plain = cm.KVCache.empty(4, 2, 64, 16, device=dev)
    x = torch.zeros(3, 2, 64, dtype=BF16, device=dev)
    table, lens, off = ints([[0, 1], [2, 3]], dev), ints([5, 6], dev), ints([0, 1, 3], dev)
    freq, _ = cm.rotary_frequencies(64, device=dev)
    pos = ints([0, 1, 2], dev)
    cache.append(x, x, table, lens, off)
    for bad in (lambda: cache.append(x, x[:2], table, lens, off),
                lambda: cache.append(x, x.half(), table, lens, off),
                lambda: cache.append(x[:, :1], x[:, :1], table, lens, off),
                lambda: cache.append(x.int(), x.int(), table, lens, off),
                lambda: cache.append(x.cpu(), x, table, lens, off),
                lambda: cache.append(x, x, table, lens),
                lambda: cache.append(x, x, table.long(), lens, off),
                lambda: cache.append(x, x, table, lens[:1], off),
                lambda: cache.append(x, x, table, lens, off[:2]),
                lambda: cache.append(x, x, table.cpu(), lens, off),
                lambda: cache.append(x.transpose(1, 2), x, table, lens, off),
                lambda: cache.read(3, table, lens, off, dtype=torch.int8),
                lambda: cache.read(3, table, lens),
                lambda: cache.attention(x.float(), table, lens, off),
                lambda: cache.attention(x[:, :1], table, lens, off),
                lambda: cache.attention(torch.zeros(3, 3, 64, dtype=BF16, device=dev), table, lens, off),
                lambda: cache.attention(x, table, lens, off, window=-1),
                lambda: cache.attention(x, table, lens, off, out=x[:2]),
                lambda: cache.attention(x, table, lens, off, weights_out=cache.weights[:2]),
                lambda: cache.attention(x, table, lens, off, weights_out=cache.weights.cpu()),
                lambda: plain.attention(x, table, lens, off, accumulate=True),
                lambda: plain.evict(4, table, lens, table),
                lambda: cache.evict(0, table, lens, table),
                lambda: cache.evict(33, table, lens, table),
                lambda: cache.evict(8, table, lens, table, first=5, recent=4),
                lambda: cache.evict(8, table, lens, table[:1]),
                lambda: cm.rotary(x, pos[:2], freq),
                lambda: cm.rotary(x, pos.float(), freq),
                lambda: cm.rotary(x, pos, freq.double()),
                lambda: cm.rotary(x, pos, torch.ones(33, device=dev)),
                lambda: cm.rotary(x, pos, freq, out=x[:, :1]),
                lambda: cm.rotary(x.int(), pos, freq),
                lambda: cm.rotary(x[0], pos, freq),
                lambda: cm.KVCache(cache.k_codes, cache.k_scales, cache.v_codes[:2], cache.v_scales),
                lambda: cm.KVCache(cache.k_codes, cache.k_scales.half(), cache.v_codes, cache.v_scales),
                lambda: cm.KVCache.empty(4, 2, 96, 16, device=dev),
                lambda: cm.KVCache.empty(4, 2, 64, 8, device=dev)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cm.rotary(x, pos, freq, scale=float("inf")),  # the entry points' own checks
                lambda: cache.attention(x, table, lens, off, scale=float("nan")),
                lambda: cache.attention(x, table, lens, off, out=x),
                lambda: cache.evict(8, table, lens, table)):
        with pytest.raises(cm.ColiMoeError):
            bad()
    assert torch.equal(cache.attention(x, table, lens, off), torch.zeros_like(x))
