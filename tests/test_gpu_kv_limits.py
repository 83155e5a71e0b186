"""The 4-bit cache at the ends of its numbers and of its rows: scales that are
no numbers or next to the largest, in every kernel of the attention."""
import pytest

torch = pytest.importorskip("torch")

import routed_expert_ffn_f32_amd as cm
from tests import kv_ref
from tests.kv_ref import Pool, U, offsets_of, pack

pytestmark = pytest.mark.gpu
BF16, F16, I32 = torch.bfloat16, torch.float16, torch.int32
INF = float("inf")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def ints(values, dev):
    return torch.tensor(values, dtype=I32, device=dev)


# tokens of 3 query heads on one key head: rows of one tile, of several tiles, of a prompt; one workgroup, and splits
ROWS = pytest.mark.parametrize("tokens,length", [(1, 150), (9, 150), (22, 150), (1, 900), (9, 900)])


@pytest.mark.parametrize("dim,page", [(64, 32), (128, 16), (128, 64), (256, 64)])
@ROWS
@pytest.mark.parametrize("bad", [INF, -INF, float("nan")])
def test_key_scales_that_are_no_numbers(dev, dim, page, tokens, length, bad):
    """A row whose key has such a scale makes every query that sees it NaN,
    whatever the sign of its product; the others keep their results."""
    pool = Pool([length], 1, dim, page, seed=1).fill()
    g = torch.Generator().manual_seed(2)
    q = torch.randn(tokens, 3, dim, generator=g).bfloat16()
    row = length - tokens + tokens // 2  # queries from the middle on see it
    p = pool.place(0, row)
    out, tol, w, wtol = kv_ref.attention(pool, q, [tokens])
    group = dim // 64 - 1
    pool.k_scales[p[0], 0, group, p[1]] = bad
    codes = torch.randint(1, 8, (dim,), generator=g)
    # the group's product is above 0, below 0 and 0 for three of the heads
    codes[dim - 64:] *= torch.where(q[tokens // 2, 1, dim - 64:] > 0, -1, 1)
    pool.k_codes[p[0], 0, p[1]] = pack(codes)
    q[:, 2, dim - 64:] = 0
    for dtype in (BF16, F16):
        cache = pool.to(dev, cm)
        got = cache.attention(q.to(dtype).to(dev), pool.table.to(dev), ints([length], dev),
                              offsets_of([tokens]).to(dev), accumulate=True).cpu().double()
        see = tokens // 2
        assert got[see:].isnan().all()
        keep = [0, 1]  # head 2's queries are other ones now
        assert ((got[:see, keep] - out[:see, keep]).abs() <= tol[:see, keep] + 2.0 ** -8 * out[:see, keep].abs()).all()
        sums = cache.weights.cpu()
        for r in (0, row):
            at = pool.place(0, r)
            assert sums[at[0], 0, at[1]].isnan()


@pytest.mark.parametrize("dim,page", [(64, 32), (128, 16), (128, 64), (256, 64)])
@ROWS
@pytest.mark.parametrize("bad", [INF, -INF, float("nan")])
def test_value_scales_that_are_no_numbers(dev, dim, page, tokens, length, bad):
    """A value with such a scale makes the columns of its group NaN in the
    queries that see it, also where its codes are not 0; nothing else."""
    pool = Pool([length], 1, dim, page, seed=3).fill()
    g = torch.Generator().manual_seed(4)
    q = torch.randn(tokens, 3, dim, generator=g).bfloat16()
    row = length - tokens + tokens // 2
    p = pool.place(0, row)
    pool.v_codes[p[0], 0, p[1]] = pack(torch.arange(dim) % 15 - 7)
    out, tol, w, wtol = kv_ref.attention(pool, q, [tokens])
    pool.v_scales[p[0], 0, dim // 64 - 1, p[1]] = bad
    for dtype in (BF16, F16):
        cache = pool.to(dev, cm)
        got = cache.attention(q.to(dtype).to(dev), pool.table.to(dev), ints([length], dev),
                              offsets_of([tokens]).to(dev), accumulate=True).cpu().double()
        see, cut = tokens // 2, dim - 64
        assert got[see:, :, cut:].isnan().all()
        for a, b, t in ((got[:see], out[:see], tol[:see]), (got[see:, :, :cut], out[see:, :, :cut], tol[see:, :, :cut])):
            assert ((a - b).abs() <= t).all()
        # weights are the keys' matter
        want = pool.weights.double() + w
        assert ((cache.weights.cpu().double() - want).abs() <= wtol + 2 * U * want)[w > 0].all()


@pytest.mark.parametrize("dim,page", [(64, 32), (128, 16), (128, 64), (256, 64)])
@ROWS
@pytest.mark.parametrize("power", [95, 105, 120])
def test_key_scales_next_to_the_largest(dev, dim, page, tokens, length, power):
    """Keys of 2^power and queries as small: scores of ordinary size, from
    products that are within float32's range whatever the order."""
    pool = Pool([length], 1, dim, page, seed=5).fill()
    g = torch.Generator().manual_seed(6)
    pool.k_scales *= 2.0 ** power
    q = (torch.randn(tokens, 3, dim, generator=g) * 2.0 ** -power).bfloat16()
    q[:, 1] *= 2.0 ** 4  # scores far apart
    out, tol, w, wtol = kv_ref.attention(pool, q, [tokens])
    cache = pool.to(dev, cm)
    got = cache.attention(q.to(dev), pool.table.to(dev), ints([length], dev), offsets_of([tokens]).to(dev),
                          accumulate=True).cpu().double()
    assert ((got - out).abs() <= tol).all()
    want = pool.weights.double() + w
    assert ((cache.weights.cpu().double() - want).abs() <= wtol + 2 * U * want)[w > 0].all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("tokens", [1, 9, 22])
@pytest.mark.parametrize("power", [110, 124])
def test_one_large_key_among_small_ones(dev, dim, tokens, power):
    """A key of 2^power that takes all of a query's weight, or none, beside keys
    of ordinary size whose scores are next to nothing then; queries of another
    size that see the ordinary ones alone."""
    pool = Pool([150], 1, dim, 64, seed=7).fill()
    g = torch.Generator().manual_seed(8)
    toward = torch.sign(torch.randn(1, dim, generator=g))
    row, see = 150 - tokens + tokens // 2, tokens // 2
    q = torch.randn(tokens, 3, dim, generator=g).bfloat16()
    q[see:, 0] = (toward * 2.0 ** -20).bfloat16()
    q[see:, 1] = (toward * -(2.0 ** -20)).bfloat16()
    q[see:, 2] = (toward * 2.0 ** (1 - power)).bfloat16()
    # all scores of heads 0 and 1 are below 2^-10 where the row is of zeros, so the weights are alike: without the row,
    # or with it in full, what they are off by is at most a hundredth more
    pool.write(0, row, 0 * toward, torch.randn(1, dim, generator=g))
    _, small, _, _ = kv_ref.attention(pool, q, [tokens])
    v = pool.rows(0, 150)[1][row, 0]
    pool.write(0, row, toward * 2.0 ** power, v.float()[None])
    assert torch.equal(pool.rows(0, 150)[1][row, 0], v)
    out, tol, _, _ = kv_ref.attention(pool, q, [tokens])
    tol[see:, 1] = 1.01 * small[see:, 1]
    tol[see:, 0] = 2.0 ** -8 * v.abs()
    got = pool.to(dev, cm).attention(q.to(dev), pool.table.to(dev), ints([150], dev), offsets_of([tokens]).to(dev)).cpu()
    assert ((got.double() - out).abs() <= tol).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("tokens", [2, 50, 120])
@pytest.mark.parametrize("length", [130, 900])
def test_a_weight_is_at_most_one(dev, dim, tokens, length):
    """Scores of 2^30, where neighbouring float32 numbers are 128 apart, so that
    a score computed once more may pass its row's maximum by far: still no query
    adds more than 1 to a key."""
    g = torch.Generator().manual_seed(dim + tokens + length)
    pool = Pool([length], 1, dim, 64, seed=9)
    pool.weights.zero_()
    keys = torch.randn(length, 1, dim, generator=g) * 8192
    for r in range(length):
        pool.write(0, r, keys[r], torch.randn(1, dim, generator=g))
    at = length - tokens + torch.arange(tokens)
    chosen = (at * 7919) % (length - tokens)
    q = torch.zeros(tokens, 2, dim)
    q[:, 0] = keys[chosen, 0] * 4  # of its own key by far the largest score
    q = q.bfloat16()
    cache = pool.to(dev, cm)
    cache.attention(q.to(dev), pool.table.to(dev), ints([length], dev), ints([0, tokens], dev), accumulate=True)
    # head 1 is of zeros: all it sees alike
    most = torch.zeros(length, dtype=torch.float64)
    z = (q[:, 0].double() @ pool.rows(0, length)[0][:, 0].t()) * dim ** -0.5
    for i in range(tokens):
        seen = z[i, : at[i] + 1]
        top = seen.argmax()
        assert seen.topk(2).values.diff() < -1e7  # all others' weights are 0
        most[top] += 1
        most[: at[i] + 1] += 1 / (int(at[i]) + 1)
    sums = cache.weights.cpu().double()
    got = torch.stack([sums[p[0], 0, p[1]] for p in (pool.place(0, r) for r in range(length))])
    assert (got <= most * (1 + (2 * tokens + 256) * U)).all()
