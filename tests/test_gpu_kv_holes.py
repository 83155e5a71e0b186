"""Eviction from sequences some of whose rows do not exist: what is kept are
rows that exist, so that an attention over the pages they go to sees rows of
the sequence and nothing that stood there before."""
import pytest

torch = pytest.importorskip("torch")

import routed_expert_ffn_f32_amd as cm
from tests import kv_ref
from tests.kv_ref import Pool

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def chosen(weights, there, keep, first, recent):
    """Rows kept of one sequence's key head: of those that exist the first, the
    last and the heaviest between, ties to the lower row, NaN above all."""
    rows = [r for r, t in enumerate(there) if t]
    if len(rows) <= keep:
        return rows
    middle = rows[first: len(rows) - recent]
    rank = sorted(middle, key=lambda r: (0, 0.0, r) if weights[r] != weights[r] else (1, -weights[r], r))
    return sorted(rows[:first] + rank[: keep - first - recent] + rows[len(rows) - recent:])


@pytest.mark.parametrize("dim,page,heads", [(64, 16, 2), (128, 64, 1), (256, 32, 2)])
@pytest.mark.parametrize("keep,first,recent", [(48, 4, 8), (33, 33, 0), (64, 0, 64), (20, 0, 0), (150, 20, 50)])
def test_evict_with_holes(dev, dim, page, heads, keep, first, recent):
    """Pages missing at the start (freed behind a window), in the middle, at the
    end, everywhere; in sequences of fewer rows than are kept too."""
    lengths = [300, 300, 300, 290, 5 * page + 3, 40, 300, 0, 300]
    holes = [(0, [0, 1]), (1, [2, 3]), (2, [-1]), (3, [0, 2, -1]), (4, [0, 1, 2, 3, 4]), (5, [0]),
             (6, range(400)), (8, [])]
    pool = Pool(lengths, heads, dim, page, seed=dim + keep, spare=keep).fill()
    g = torch.Generator().manual_seed(keep)
    pool.weights = torch.randint(-1, 4, pool.weights.shape, generator=g).float() / 4  # ties, some below 0
    pool.weights[torch.rand(pool.weights.shape, generator=g) < 0.02] = float("nan")
    for s, pages in holes:
        last = (lengths[s] - 1) // page
        for i in pages:
            if i <= last:
                pool.table[s, last if i < 0 else i] = -1 if i % 2 else pool.pages
    cache = pool.to(dev, cm)
    kept, new = cache.evict(keep, pool.table.to(dev), torch.tensor(lengths, dtype=I32, device=dev), pool.into.to(dev),
                            first=first, recent=recent)
    kept, new = kept.cpu(), new.cpu()
    after = Pool(lengths, heads, dim, page, seed=1)  # the same pool as it is now, its rows those of `into`
    after.pages, after.table, after.lengths = pool.pages, pool.into, new.tolist()
    for name in ("k_codes", "v_codes", "k_scales", "v_scales", "weights"):
        setattr(after, name, getattr(cache, name).cpu())
    for s, n in enumerate(lengths):
        there = [pool.place(s, r) is not None for r in range(n)]
        assert int(new[s]) == min(keep, sum(there)), s
        k, v, _, _, _ = pool.rows(s, n)
        ak, av, _, _, _ = after.rows(s, int(new[s]))
        for h in range(heads):
            w = [float(pool.weights[p[0], h, p[1]]) if (p := pool.place(s, r)) else 0.0 for r in range(n)]
            rows = chosen(w, there, keep, first, recent)
            assert kept[s, h].tolist() == rows + [-1] * (keep - len(rows)), (s, h)
            assert torch.equal(ak[:, h], k[rows, h]) and torch.equal(av[:, h], v[rows, h]), (s, h)
            for i, r in enumerate(rows):
                p = after.place(s, i)
                assert str(float(after.weights[p[0], h, p[1]])) == str(w[r])
    q = torch.randn(len(lengths), 2 * heads, dim, generator=g).bfloat16()
    out, tol, _, _ = kv_ref.attention(after, q, [1] * len(lengths))
    got = cache.attention(q.to(dev), pool.into.to(dev), new.to(dev)).cpu().double()
    assert ((got - out).abs() <= tol).all()


@pytest.mark.parametrize("first,recent", [(4, 100), (0, 0), (10000, 1111)])
def test_long_evict_with_holes(dev, first, recent):
    """More rows than LDS holds keys of; every third page is not there."""
    L, keep, page = 60000, 11111, 256
    pages = -(-L // page)
    cache = cm.KVCache.empty(pages + -(-keep // page), 2, 64, page, weights=True, device=dev)
    g = torch.Generator().manual_seed(first)
    order = torch.randperm(cache.pages, generator=g).to(I32)
    table, into = order[:pages].clone()[None], order[pages:][None]
    w = torch.randint(0, 1000, cache.weights.shape, generator=g).float()
    cache.weights.copy_(w)
    rows = w[table[0].long()].permute(1, 0, 2).flatten(1)[:, :L].tolist()
    table[0, 1::3] = -1
    there = [r // page % 3 != 1 for r in range(L)]
    kept, new = cache.evict(keep, table.to(dev), torch.tensor([L], dtype=I32, device=dev), into.to(dev), first=first,
                            recent=recent)
    assert int(new[0]) == keep
    for h in range(2):
        assert kept[0, h].tolist() == chosen(rows[h], there, keep, first, recent)
