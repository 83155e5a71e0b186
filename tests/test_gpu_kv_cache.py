"""Append to, read from and evict from the 4-bit cache against the same on the
CPU: whole numbers, so everything has to be equal."""
import pytest

torch = pytest.importorskip("torch")

import routed_expert_ffn_f32_amd as cm
from tests.kv_ref import Pool, offsets_of, pack, quantise, unpack

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def same(cache, pool):
    """All of the cache's tensors hold the pool's bits."""
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        a, b = getattr(cache, name).cpu(), getattr(pool, name)
        if a.dtype == BF16:
            nan = b.isnan()
            assert torch.equal(a.isnan(), nan), name
            a, b = a.masked_fill(nan, 0), b.masked_fill(nan, 0)
        assert torch.equal(a, b), name


@pytest.mark.parametrize("dim,page,heads,dtype", [(64, 16, 1, F32), (64, 32, 3, BF16), (128, 64, 8, BF16),
                                                  (128, 16, 2, F16), (256, 16, 5, F32), (256, 256, 1, F16)])
def test_append_and_read(dev, dim, page, heads, dtype):
    """Ragged tokens on ragged pasts, views, tokens in no sequence, more tokens
    than rows, a page that is not there; every other place keeps its bits."""
    new, lengths = [3, 0, 70, 1, 6], [40, 20, 70, 1, 4]
    pool = Pool(lengths, heads, dim, page, seed=dim).fill()
    if page == 16:  # sequence 2 has several pages
        pool.table[2, 1] = -5
    g = torch.Generator().manual_seed(1)
    T = sum(new) + 5
    kv = torch.randn(T, 2 * heads + 1, dim + 8, generator=g) * torch.exp(2 * torch.randn(T, 1, 1, generator=g))
    kv[4] = 0
    kv[6, 0, 3] = float("inf")
    kv[7, 0, 5] = float("nan")
    kv = kv.to(dtype)
    k, v = kv[:, :heads, 2: 2 + dim], kv[:, heads + 1:, 8:]
    cache = pool.to(dev, cm)
    off = (offsets_of(new) + 2).to(dev)
    args = pool.table.to(dev), torch.tensor(lengths, dtype=torch.int32, device=dev), off
    d = kv.to(dev)
    cache.append(d[:, :heads, 2: 2 + dim], d[:, heads + 1:, 8:], *args)
    weights, want_k, want_v = pool.weights.clone(), torch.zeros(T, heads, dim), torch.zeros(T, heads, dim)
    t = 2
    for s, n in enumerate(new):
        for i in range(n):
            row = lengths[s] - n + i
            pool.write(s, row, k[t].float(), v[t].float())
            p = pool.place(s, row)
            if p is not None:
                weights[p[0], :, p[1]] = 0
                for x, want in ((k, want_k), (v, want_v)):
                    q, sc = quantise(x[t].float())
                    want[t] = (q * sc.double().repeat_interleave(64, -1)).float()
            t += 1
    same(cache, pool)
    assert torch.equal(cache.weights.cpu(), weights)
    for out in (F32, BF16, F16):
        for got, want in zip(cache.read(T, *args, dtype=out), (want_k, want_v)):
            got, w = got.cpu(), want.to(out)
            assert torch.equal(got.isnan(), w.isnan()) and torch.equal(got.nan_to_num(0), w.nan_to_num(0)), out


def test_borders(dev):
    """Ties, quotients next to them, subnormal scales and the largest values:
    the float32 path picks what 64 bits pick."""
    g = torch.Generator().manual_seed(3)
    rows = []
    for s in (1.0, 0.375, 1.9921875, 2.0 ** -126, 3 * 2.0 ** -130, 2.0 ** -133, 4.5e37):
        x = torch.randint(-14, 15, (64,), generator=g).float() / 2 * s
        x[0] = 7 * s
        up = torch.nextafter(x, torch.full_like(x, 1e38))
        down = torch.nextafter(x, torch.full_like(x, -1e38))
        for r in (x, up, down):
            r[0] = 7 * s
            rows.append(r)
    rows += [torch.rand(64, generator=g) * 2 - 1 for _ in range(400)]
    x = torch.stack(rows)[:, None, :]
    n = len(rows)
    pool = Pool([n], 1, 64, 16, seed=4)
    cache = pool.to(dev, cm)
    cache.append(x.to(dev), -x.to(dev), pool.table.to(dev), torch.tensor([n], dtype=torch.int32, device=dev),
                 offsets_of([n]).to(dev))
    for r in range(n):
        pool.write(0, r, x[r], -x[r])
    same(cache, pool)


def test_one_token_each_without_offsets(dev):
    lengths = [5, 1, 0, 33]
    pool = Pool(lengths, 2, 128, 16, seed=5)
    g = torch.Generator().manual_seed(6)
    k, v = torch.randn(4, 2, 128, generator=g), torch.randn(4, 2, 128, generator=g)
    cache = pool.to(dev, cm, weights=False)
    args = pool.table.to(dev), torch.tensor(lengths, dtype=torch.int32, device=dev)
    cache.append(k.to(dev), v.to(dev), *args)
    for s, n in enumerate(lengths):
        pool.write(s, n - 1, k[s], v[s])
    same(cache, pool)
    got, _ = cache.read(4, *args, dtype=F32)
    assert (got[2] == 0).all() and (got[3] != 0).any()


def evicted(pool, keep, first, recent):
    """(kept lists, new lengths), rows copied in the pool itself."""
    S, H = len(pool.lengths), pool.heads
    kept = torch.full((S, H, keep), -1, dtype=torch.int32)
    moves = []
    for s, n in enumerate(pool.lengths):
        for h in range(H):
            w = [float(pool.weights[p[0], h, p[1]]) if (p := pool.place(s, r)) else 0.0 for r in range(n)]
            if n <= keep:
                rows = list(range(n))
            else:
                middle = range(first, n - recent)
                key = lambda r: (-(float("inf") if w[r] != w[r] else w[r]), w[r] == w[r], r)  # noqa: E731, B023
                rows = sorted([*range(first), *sorted(middle, key=key)[: keep - first - recent], *range(n - recent, n)])
            for i, r in enumerate(rows):
                kept[s, h, i] = r
                src, page = pool.place(s, r), int(pool.into[s, i // pool.page])
                if src is not None and 0 <= page < pool.pages:
                    moves.append((src, (page, i % pool.page), h))
    old = [t.clone() for t in (pool.k_codes, pool.v_codes, pool.k_scales, pool.v_scales, pool.weights)]
    for (sp, ss), (dp, ds), h in moves:
        pool.k_codes[dp, h, ds], pool.v_codes[dp, h, ds] = old[0][sp, h, ss], old[1][sp, h, ss]
        pool.k_scales[dp, h, :, ds], pool.v_scales[dp, h, :, ds] = old[2][sp, h, :, ss], old[3][sp, h, :, ss]
        pool.weights[dp, h, ds] = old[4][sp, h, ss]
    return kept, torch.tensor([min(n, keep) for n in pool.lengths], dtype=torch.int32)


@pytest.mark.parametrize("dim,page,heads,keep,first,recent", [
    (64, 16, 2, 10, 4, 3), (128, 32, 1, 1, 0, 0), (128, 64, 3, 100, 4, 96), (256, 16, 1, 33, 33, 0), (64, 128, 2, 64, 0, 64),
    (128, 16, 2, 500, 4, 60)])
def test_evict(dev, dim, page, heads, keep, first, recent):
    lengths = [0, 1, 9, 10, 11, 100, 101, 1200, 2100]
    pool = Pool(lengths, heads, dim, page, seed=keep, spare=keep, capacity=2100)
    g = torch.Generator().manual_seed(keep)
    # few different weights: ties everywhere; some negative, infinite, -0 and NaN
    pool.weights = torch.randint(0, 4, pool.weights.shape, generator=g).float() / 4
    for value in (float("nan"), float("inf"), -0.0, -1.5, 1e-40):
        pool.weights[torch.rand(pool.weights.shape, generator=g) < 0.02] = value
    pool.table[8, 1] = -1
    pool.into[7, 0] = -1
    cache = pool.to(dev, cm)
    kept, new = cache.evict(keep, pool.table.to(dev), torch.tensor(lengths, dtype=torch.int32, device=dev),
                            pool.into.to(dev), first=first, recent=recent)
    want, lens = evicted(pool, keep, first, recent)
    assert torch.equal(new.cpu(), lens)
    assert torch.equal(kept.cpu(), want)
    same(cache, pool)
    a, b = cache.weights.cpu(), pool.weights
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(7.5), b.nan_to_num(7.5))


def test_codes_round_trip():
    q = torch.randint(-8, 8, (5, 64))
    assert torch.equal(unpack(pack(q)), q.double())
