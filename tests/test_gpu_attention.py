"""Attention over the 4-bit cache against its formulas in 64 bits: head
layouts, lengths and pages that end inside a step, several queries of a
sequence, windows, rows that see nothing, junk in every place that is not
read, and the accumulated weights."""
import pytest

torch = pytest.importorskip("torch")

import routed_expert_ffn_f32_amd as cm
from tests import kv_ref
from tests.kv_ref import HALF_STEP, Pool, offsets_of

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def check(got, out, tol, dtype, what=""):
    err = (got.double() - out).abs()
    assert torch.isfinite(got).all(), what
    over = err / (tol + 1e-300)
    at = [int(i) for i in torch.unravel_index(over.argmax(), over.shape)]
    assert bool((err <= tol).all()), \
        f"{what}: {int((err > tol).sum())} beyond, worst at {at}: {float(got[tuple(at)])} for " \
        f"{float(out[tuple(at)])} +- {float(tol[tuple(at)])}"
    # one rounding of the type, weights rounded to an eighth of its half step or less, float32 sums
    if out.norm() > 0:
        assert float(err.norm() / out.norm()) <= 1.25 * HALF_STEP[dtype], what


def run(dev, pool, q, new, weights=False, table=None, **kw):
    cache = pool.to(dev, cm)
    off = None if all(n == 1 for n in new) and kw.pop("plain", True) else offsets_of(new).to(dev)
    lengths = torch.tensor(pool.lengths, dtype=torch.int32, device=dev)
    wo = torch.full_like(cache.weights, -1.0) if weights else None
    got = cache.attention(q.to(dev), pool.table.to(dev), lengths, off, weights_out=wo, **kw)
    torch.cuda.synchronize()
    return got.cpu(), None if wo is None else wo.cpu(), cache


def queries(tokens, heads, dim, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (2 * torch.randn(tokens, heads, dim, generator=g)).to(dtype)


@pytest.mark.parametrize("dim,page,heads,group,dtype", [
    (64, 16, 2, 1, BF16), (64, 64, 1, 16, F16), (64, 32, 3, 5, F16), (64, 16, 1, 40, BF16),
    (128, 64, 2, 8, BF16), (128, 16, 1, 6, F16), (128, 256, 2, 1, BF16), (128, 32, 1, 20, F16),
    (256, 16, 2, 4, BF16), (256, 128, 1, 1, F16), (256, 64, 1, 9, F16)])
def test_one_token_each(dev, dim, page, heads, group, dtype):
    """Lengths from 0 (a token that sees nothing) to several steps of keys."""
    lengths = [1, 0, 2, 15, 16, 17, 63, 64, 65, 200, 330]
    pool = Pool(lengths, heads, dim, page, seed=dim + group).fill()
    q = queries(len(lengths), heads * group, dim, dtype, 1)
    out, tol, w, wtol = kv_ref.attention(pool, q, [1] * len(lengths))
    got, wo, _ = run(dev, pool, q, [1] * len(lengths), weights=True)
    assert (got[1] == 0).all()
    check(got, out, tol, dtype)
    written = torch.zeros_like(w, dtype=torch.bool)
    for s, n in enumerate(lengths):
        for r in range(n):
            p = pool.place(s, r)
            written[p[0], :, p[1]] = True
    assert (wo[~written] == -1).all()
    want = pool.weights.double() + w
    assert ((wo.double() - want).abs() <= wtol + 2 * kv_ref.U * want)[written].all()


@pytest.mark.parametrize("dim,page,heads,group,dtype", [
    (64, 16, 2, 2, F16), (128, 64, 1, 8, BF16), (128, 16, 2, 3, F16), (256, 32, 1, 4, BF16)])
@pytest.mark.parametrize("window", [0, 1, 40])
def test_several_tokens(dev, dim, page, heads, group, dtype, window):
    """Prompts and drafts: causal within the call, sequences without a token,
    more tokens than rows, a window."""
    new, lengths = [5, 1, 0, 33, 7, 70], [90, 1, 12, 33, 3, 131]
    pool = Pool(lengths, heads, dim, page, seed=3).fill()
    q = queries(sum(new), heads * group, dim, dtype, 2)
    out, tol, w, wtol = kv_ref.attention(pool, q, new, window=window)
    got, wo, _ = run(dev, pool, q, new, weights=True, window=window)
    assert (got[5 + 1 + 33: 5 + 1 + 33 + 4] == 0).all()  # rows before 0
    check(got, out, tol, dtype)
    seen = w > 0
    want = pool.weights.double() + w
    assert ((wo.double() - want).abs() <= wtol + 2 * kv_ref.U * want)[seen].all()
    touched = wo != -1
    assert touched[seen].all() and (wo[touched & ~seen] == pool.weights[touched & ~seen]).all()


@pytest.mark.parametrize("new", [[1], [3], [150]])
def test_long_and_split(dev, new):
    """One sequence over many workgroups, its last split short."""
    pool = Pool([1500], 1, 128, 64, seed=5).fill()
    q = queries(sum(new), 8, 128, F16, 6)
    out, tol, w, wtol = kv_ref.attention(pool, q[:1] if new == [1] else q, new)
    got, wo, _ = run(dev, pool, q, new, weights=True)
    check(got, out, tol, F16)
    want = pool.weights.double() + w
    assert ((wo.double() - want).abs() <= wtol + 2 * kv_ref.U * want)[w > 0].all()


def test_tokens_in_no_sequence(dev):
    """Left as they were in a given result, zeros in a fresh one."""
    new, lengths = [2, 3], [20, 40]
    pool = Pool(lengths, 1, 128, 16, seed=7).fill()
    q = queries(9, 4, 128, BF16, 8)
    out, tol, _, _ = kv_ref.attention(pool, q[2:7], new)
    cache = pool.to(dev, cm)
    off = (offsets_of(new) + 2).to(dev)
    lengths = torch.tensor(lengths, dtype=torch.int32, device=dev)
    fresh = cache.attention(q.to(dev), pool.table.to(dev), lengths, off).cpu()
    given = torch.full((9, 4, 128), 7.0, dtype=BF16, device=dev)
    assert cache.attention(q.to(dev), pool.table.to(dev), lengths, off, out=given) is given
    given = given.cpu()
    for got, rest in ((fresh, 0.0), (given, 7.0)):
        check(got[2:7], out, tol, BF16)
        assert (got[:2] == rest).all() and (got[7:] == rest).all()


def test_missing_pages_and_strides(dev):
    """A page that is not there in the middle; queries and results as views;
    the table as a view; a scale of its own."""
    pool = Pool([200], 2, 128, 16, seed=9).fill()
    pool.table[0, 3] = -1
    pool.table[0, 5] = 1 << 20
    g = torch.Generator().manual_seed(10)
    wide = torch.randn(6, 9, 200, generator=g).bfloat16()
    q = wide[1:4, 2:8, 40:168]
    out, tol, _, _ = kv_ref.attention(pool, q, [3], scale=0.3)
    cache = pool.to(dev, cm)
    table = torch.zeros(1, 50, dtype=torch.int32, device=dev)
    table[:, 20: 20 + pool.table.shape[1]] = pool.table.to(dev)
    res = torch.zeros(3, 7, 140, dtype=BF16, device=dev)
    cache.attention(wide.to(dev)[1:4, 2:8, 40:168], table[:, 20: 20 + pool.table.shape[1]],
                    torch.tensor([200], dtype=torch.int32, device=dev), offsets_of([3]).to(dev), scale=0.3,
                    out=res[:, 1:, 6:134])
    res = res.cpu()
    check(res[:, 1:, 6:134], out, tol, BF16)
    assert (res[:, 0] == 0).all() and (res[:, :, :6] == 0).all() and (res[:, :, 134:] == 0).all()


def test_uneven_values(dev):
    """Value scales many powers of two apart, the largest where the weight is
    next to nothing and the other way round: nothing is lost to the range of
    half precision."""
    for far in (2.0 ** 40, 2.0 ** -40):
        pool = Pool([130], 1, 128, 16, seed=11).fill(v_gain=lambda s, r: far if r % 7 == 3 else 1.0)
        q = queries(1, 8, 128, F16, 12)
        k, _, _, _, _ = pool.rows(0, 130)
        q[0, 0] = -4 * k[3, 0].half()  # against the outlier
        q[0, 1] = 4 * k[3, 0].half()
        out, tol, _, _ = kv_ref.attention(pool, q, [1])
        got, _, _ = run(dev, pool, q.bfloat16(), [1])
        out, tol, _, _ = kv_ref.attention(pool, q.bfloat16(), [1])
        check(got, out, tol, BF16, str(far))


def test_large_and_small_queries(dev):
    for gain in (1e-30, 1e-3, 300.0):
        pool = Pool([75], 1, 64, 16, seed=13).fill()
        q = (queries(1, 4, 64, torch.float32, 14) * gain).bfloat16()
        out, tol, _, _ = kv_ref.attention(pool, q, [1])
        got, _, _ = run(dev, pool, q, [1])
        check(got, out, tol, BF16, str(gain))


def test_nan_reaches_who_sees_it(dev):
    """A row of NaN: every query that sees it is NaN, the others are not."""
    pool = Pool([40], 1, 128, 16, seed=15).fill()
    nan = torch.full((1, 128), float("nan"))
    pool.write(0, 37, nan, torch.zeros(1, 128))
    q = queries(5, 2, 128, BF16, 16)
    got, _, _ = run(dev, pool, q, [5])
    assert torch.isfinite(got[:2]).all() and got[2:].isnan().all()


def test_accumulates_in_place(dev):
    pool = Pool([70, 30], 2, 64, 32, seed=17).fill()
    q = queries(2, 4, 64, F16, 18)
    cache = pool.to(dev, cm)
    lengths = torch.tensor(pool.lengths, dtype=torch.int32, device=dev)
    version = cache.weights._version
    once = cache.attention(q.to(dev), pool.table.to(dev), lengths, accumulate=True)
    again = cache.attention(q.to(dev), pool.table.to(dev), lengths, accumulate=True)
    assert torch.equal(once, again) and cache.weights._version == version + 2
    _, _, w, wtol = kv_ref.attention(pool, q, [1, 1])
    want = pool.weights.double() + 2 * w
    assert ((cache.weights.cpu().double() - want).abs() <= 2 * wtol + 4 * kv_ref.U * want)[w > 0].all()
    assert torch.equal(cache.weights.cpu()[w == 0], pool.weights[w == 0])


# --- many query rows: prompts ---------------------------------------------

@pytest.mark.parametrize("dim,page,heads,group,dtype", [
    (64, 16, 2, 3, F16), (64, 64, 1, 16, BF16), (128, 64, 1, 8, BF16), (128, 16, 2, 5, F16), (256, 32, 1, 4, BF16),
    (256, 16, 1, 7, F16)])
@pytest.mark.parametrize("window", [0, 50])
def test_prompts(dev, dim, page, heads, group, dtype, window):
    """Rows on both sides of the limits of a workgroup, beside a sequence of
    one token and an empty one, on pasts that end inside a step."""
    new = [70, 1, 0, 33, 130]
    lengths = [70, 55, 9, 90, 259]
    pool = Pool(lengths, heads, dim, page, seed=21).fill()
    q = queries(sum(new), heads * group, dim, dtype, 22)
    out, tol, w, wtol = kv_ref.attention(pool, q, new, window=window)
    got, wo, _ = run(dev, pool, q, new, weights=True, window=window)
    check(got, out, tol, dtype)
    want = pool.weights.double() + w
    assert ((wo.double() - want).abs() <= wtol + 2 * kv_ref.U * want)[w > 0].all()


@pytest.mark.parametrize("dim,dtype", [(64, BF16), (128, F16), (256, BF16)])
@pytest.mark.parametrize("far", [2.0 ** 30, 2.0 ** 60, 2.0 ** -30, 2.0 ** -50])
def test_uneven_values_in_prompts(dev, dim, dtype, far):
    """Values of one step many powers of two apart: where the large rows have
    no weight the small ones still count in full."""
    if dtype == F16 and far > 1:
        far = 1 / far  # results stay in the type's range
    pool = Pool([150], 1, dim, 16, seed=23)
    g = torch.Generator().manual_seed(24)
    toward = torch.randn(1, dim, generator=g)
    for r in range(150):
        big = far > 1 and r % 5 == 3
        k = -8 * toward if big else torch.randn(1, dim, generator=g) + toward
        pool.write(0, r, k, torch.randn(1, dim, generator=g) * (far if r % 5 == 3 else 1.0))
    q = (torch.randn(75, 2, dim, generator=g) + 3 * toward).to(dtype)
    out, tol, _, _ = kv_ref.attention(pool, q, [75])
    got, _, _ = run(dev, pool, q, [75])
    assert float(out.abs().max()) < 1e3  # the large rows have no weight
    check(got, out, tol, dtype)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_nan_in_prompts(dev, dim):
    """NaN keys and NaN values of one group reach exactly the queries that see
    them, and of the values exactly the group's columns."""
    new = 100
    pool = Pool([140], 1, dim, 16, seed=25).fill()
    one = torch.ones(1, dim)
    bad = one.clone()
    bad[0, dim - 3] = float("nan")
    pool.write(0, 90, one, bad)
    bad_key = one.clone()
    bad_key[0, 0] = float("inf")
    pool.write(0, 120, bad_key, one)
    q = queries(new, 2, dim, BF16, 26)
    got, _, _ = run(dev, pool, q, [new])
    first = 140 - new
    assert torch.isfinite(got[: 90 - first]).all()
    assert torch.isfinite(got[90 - first: 120 - first, :, : dim - 64]).all()
    assert got[90 - first: 120 - first, :, dim - 64:].isnan().all()
    assert got[120 - first:].isnan().all()
    windowed, _, _ = run(dev, pool, q, [new], window=10)
    assert torch.isfinite(windowed[130 - first:]).all() and windowed[120 - first: 130 - first].isnan().all()


@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
@pytest.mark.parametrize("tokens", [4, 90])
def test_scales_and_missing_pages(dev, scale, tokens):
    pool = Pool([300], 1, 128, 16, seed=27).fill()
    for i in (0, 4, 5, 12):
        pool.table[0, i] = -7
    q = queries(tokens, 2, 128, BF16, 28)
    out, tol, _, _ = kv_ref.attention(pool, q, [tokens], scale=scale)
    got, _, _ = run(dev, pool, q, [tokens], scale=scale)
    check(got, out, tol, BF16)


def test_split_prompt(dev):
    """Few rows over a long past: the keys are split over workgroups; and the
    tokens of no sequence around it."""
    pool = Pool([2300], 1, 64, 64, seed=29).fill()
    q = queries(75, 2, 64, F16, 30)
    out, tol, _, _ = kv_ref.attention(pool, q[3:73], [70])
    cache = pool.to(dev, cm)
    got = cache.attention(q.to(dev), pool.table.to(dev), torch.tensor([2300], dtype=torch.int32, device=dev),
                          (offsets_of([70]) + 3).to(dev)).cpu()
    check(got[3:73], out, tol, F16)
    assert (got[:3] == 0).all() and (got[73:] == 0).all()
