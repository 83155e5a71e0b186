"""Accumulated weights of rows that several sequences of a call see: pages of a
common prefix, pages at different places of their sequences, a page twice in
one: each place gets the sum over all that see it."""
import pytest

torch = pytest.importorskip("torch")

import routed_expert_ffn_f32_amd as cm
from tests import kv_ref
from tests.kv_ref import Pool, U, offsets_of

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def check(dev, pool, q, new, window=0, turns=1):
    """Both forms against the oracle, which adds up place by place.  Each of a
    place's sums is added with a rounding of its own."""
    _, _, w, wtol = kv_ref.attention(pool, q, new, window=window)
    off = None if all(n == 1 for n in new) else offsets_of(new).to(dev)
    args = pool.table.to(dev), torch.tensor(pool.lengths, dtype=I32, device=dev), off
    seen = torch.zeros_like(w, dtype=torch.bool)
    for s, (n, length) in enumerate(zip(new, pool.lengths)):
        for r in range(max(0, length - n - window + 1) if window else 0, length):
            p = pool.place(s, r)
            if n > 0 and p is not None:
                seen[p[0], :, p[1]] = True
    for _ in range(turns):
        cache = pool.to(dev, cm)
        sums = torch.full_like(cache.weights, -1.0)
        a = cache.attention(q.to(dev), *args, window=window, weights_out=sums)
        assert torch.equal(cache.weights.cpu(), pool.weights)
        b = cache.attention(q.to(dev), *args, window=window, accumulate=True)
        assert torch.equal(a, b)
        want = pool.weights.double() + w
        tol = wtol + (len(new) + 4) * U * want
        for got in (sums.cpu(), cache.weights.cpu()):
            assert ((got.double() - want).abs() <= tol)[seen].all()
        assert (sums.cpu()[~seen] == -1).all() and torch.equal(cache.weights.cpu()[~seen], pool.weights[~seen])


@pytest.mark.parametrize("dim,page,heads,group", [(64, 16, 2, 2), (128, 64, 1, 4), (256, 32, 1, 3)])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [2, 0, 3, 1], [30, 1, 9, 2]])
@pytest.mark.parametrize("window", [0, 70])
def test_shared_pages(dev, dim, page, heads, group, new, window):
    pool = Pool([200, 180, 150, 199], heads, dim, page, seed=dim).fill()
    pool.table[1, :2] = pool.table[0, :2]  # a common prefix
    pool.table[2, :1] = pool.table[0, :1]
    pool.table[3, 1] = pool.table[0, 0]  # at another place
    pool.table[3, 2] = pool.table[3, 0]  # twice in one sequence
    q = torch.randn(sum(new), heads * group, dim, generator=torch.Generator().manual_seed(1)).half()
    check(dev, pool, q, new, window)


@pytest.mark.parametrize("dim,group", [(64, 4), (128, 8)])
def test_many_sharers(dev, dim, group):
    """60 sequences on one prefix of eight pages, single tokens, several times."""
    pool = Pool([128 + 2 * i for i in range(60)], 1, dim, 16, seed=3).fill()
    pool.weights *= 2.0 ** -10
    pool.table[:, :8] = pool.table[0, :8].clone()
    q = torch.randn(60, group, dim, generator=torch.Generator().manual_seed(4)).bfloat16()
    check(dev, pool, q, [1] * 60, turns=4)


@pytest.mark.parametrize("out", [False, True])
def test_as_many_sequences_as_there_may_be(dev, out):
    """65536 sequences of one row, the same one, and 17 key heads: more parts of
    the work than workgroups.

    A weight is 1 - e with 0 <= e <= 2^-23 (an exponential's last bit), so a sum
    of n is at most n.  From n = 4 on e is below half a step of float32 there,
    and with n - k steps n + 1 - k steps is a float32 number too (or, where
    steps double, n + 1 - k / 2 of them, rounded down to k at most), so no
    further step is lost: 4 of 2^-8 at most, from the first four additions."""
    S, H = 65536, 17
    cache = cm.KVCache.empty(1, H, 64, 16, weights=True, device=dev)
    cache.k_scales.fill_(0.5)
    cache.k_codes.fill_(0x21)
    cache.weights.copy_(torch.arange(16.0).expand(1, H, 16))
    q = torch.ones(S, H, 64, dtype=torch.bfloat16, device=dev)
    table = torch.zeros(S, 1, dtype=I32, device=dev)
    lengths = torch.ones(S, dtype=I32, device=dev)
    sums = torch.full_like(cache.weights, -1.0) if out else None
    got = cache.attention(q, table, lengths, weights_out=sums, accumulate=True)
    assert (got == 0).all()  # the value's scale is 0
    got = (sums if out else cache.weights).cpu()
    assert ((got[:, :, 0] <= S) & (got[:, :, 0] >= S - 2.0 ** -6)).all()
    want = torch.full((1, H, 16), -1.0) if out else torch.arange(16.0).expand(1, H, 16)
    assert torch.equal(got[:, :, 1:], want[:, :, 1:])


@pytest.mark.parametrize("new", [[1, 1, 1], [20, 1, 3]])
def test_captured_sums_of_their_own(dev, new):
    """Sums in a tensor of their own, replayed while the cache's weights change
    between: each replay starts from the weights as they are."""
    pool = Pool([90, 70, 40], 2, 64, 16, seed=5).fill()
    q = torch.randn(sum(new), 4, 64, generator=torch.Generator().manual_seed(6)).bfloat16().to(dev)
    off = None if max(new) == 1 else offsets_of(new).to(dev)
    args = pool.table.to(dev), torch.tensor(pool.lengths, dtype=I32, device=dev), off
    cache = pool.to(dev, cm)
    sums, want = torch.full_like(cache.weights, -1.0), torch.full_like(cache.weights, -1.0)
    cache.attention(q, *args, weights_out=sums)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = cache.attention(q, *args, weights_out=sums)
    for turn in range(4):
        sums.fill_(-1.0)
        graph.replay()
        out = cache.attention(q, *args, weights_out=want)
        if turn % 2:
            torch.cuda.synchronize()
        assert torch.equal(got, out) and torch.equal(sums, want), turn
        cache.weights.mul_(1.5)
