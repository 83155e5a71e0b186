"""Queries and results that are views of one buffer, between each other's heads
and tokens but with no element in common, are calls like any other; those that
have some in common are refused."""
import pytest

torch = pytest.importorskip("torch")

import routed_expert_ffn_f32_amd as cm
from tests.kv_ref import Pool, offsets_of

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("layout", ["parts of a token", "heads in turn", "tokens in turn", "halves of heads", "heads first",
                                    "wider steps from head to head"])
def test_results_between_the_inputs(dev, layout):
    T, H, D = 7, 4, 64
    g = torch.Generator().manual_seed(1)
    if layout == "parts of a token":
        buf = torch.randn(T, 2 * H, D, generator=g).to(BF16).to(dev)
        x, out = buf[:, :H], buf[:, H:]
    elif layout == "heads in turn":
        buf = torch.randn(T, 2 * H, D, generator=g).to(BF16).to(dev)
        x, out = buf[:, 1::2], buf[:, 0::2]
    elif layout == "tokens in turn":
        buf = torch.randn(2 * T, H, D, generator=g).to(BF16).to(dev)
        x, out = buf[0::2], buf[1::2]
    elif layout == "halves of heads":
        buf = torch.randn(T, H, 2 * D, generator=g).to(BF16).to(dev)
        x, out = buf[..., D:], buf[..., :D]
    elif layout == "wider steps from head to head":
        buf = torch.randn(T, 4 * H * D, generator=g).to(BF16).to(dev)
        x, out = buf[:, : 3 * H * D].view(T, H, 3 * D)[..., :D], buf[:, 3 * H * D:].view(T, H, D)
    else:
        buf = torch.randn(H, 2 * T, D, generator=g).to(BF16).to(dev)
        x, out = buf[:, :T].transpose(0, 1), buf[:, T:].transpose(0, 1)
    before = x.clone()
    pos, (freq, _) = torch.arange(T, device=dev), cm.rotary_frequencies(D, device=dev)
    want = cm.rotary(before, pos, freq)
    assert cm.rotary(x, pos, freq, out=out) is out
    assert torch.equal(out, want) and torch.equal(x, before)
    pool = Pool([40], 2, D, 16, seed=2).fill()
    args = pool.table.to(dev), torch.tensor([40], dtype=I32, device=dev), offsets_of([T]).to(dev)
    cache = pool.to(dev, cm)
    want = cache.attention(before, *args)
    cache.attention(x, *args, out=out)
    assert torch.equal(out, want) and torch.equal(x, before)


def test_results_across_the_inputs(dev):
    buf = torch.zeros(7, 9, 64, dtype=BF16, device=dev)
    pos, (freq, _) = torch.arange(7, device=dev), cm.rotary_frequencies(64, device=dev)
    cache = cm.KVCache.empty(3, 2, 64, 16, weights=True, device=dev)
    table, lengths = torch.zeros(1, 1, dtype=I32, device=dev), torch.tensor([9], dtype=I32, device=dev)
    off = offsets_of([7]).to(dev)
    args = table, lengths, off
    flat = buf.view(-1)
    for x, out in ((buf[:, :4], buf[:, 1:5]), (buf[:, 4:8], buf[:, 1:5]), (buf[:6, :4], buf[1:, :4]),
                   (buf[:, :4], flat[1: 1 + 7 * 4 * 64].view(7, 4, 64))):
        n = x.shape[0]
        with pytest.raises(cm.ColiMoeError):
            cm.rotary(x, pos[:n], freq, out=out)
        with pytest.raises(cm.ColiMoeError):
            cache.attention(x, table, lengths, offsets_of([n]).to(dev), out=out)
    both = torch.zeros(4, 2, 16, device=dev)
    shared = cm.KVCache(cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, both[:3])
    with pytest.raises(cm.ColiMoeError):
        shared.attention(buf[:, :4], *args, weights_out=both[1:])
