"""The operators together with the layer, as a model's block runs them: the
residual addition and norm in front of the layer (forward_normed), the
balance of what its router chose, and its gradient."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import routed_expert_ffn_f32_amd as cm
import synth
from tests.gpu_util import DeviceLayer, rel_err
from tests.test_gpu_balance import ALPHA, U, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("T", [1, 3, 16, 70])
def test_normed_forward_and_balance(dev, T):
    """Against the CPU oracle on the rows that the norm gives, with the
    layer's own bar of 2e-3; the balance of the oracle's routing."""
    shape = synth.LayerShape(hidden=256, n_experts=16, top_k=4, inter=512, n_shared=1, rsf=2.5, bias_sigma=0.05)
    L = DeviceLayer(shape, 3, 0, dev, max_tokens=128, keep_host=True)
    try:
        g = torch.Generator().manual_seed(T)
        x = torch.randn(T, 256, generator=g).to(torch.bfloat16).to(dev)
        res = torch.randn(T, 256, generator=g).to(dev)
        w = (1 + 0.1 * torch.randn(256, generator=g)).to(dev)
        want_sum = res + x.float()
        rows = cm.rms_norm(want_sum, w, 1e-6)
        out = L.moe.forward_normed(x, w, 1e-6, residual=res)
        torch.cuda.synchronize()
        assert torch.equal(res, want_sum)
        ref, _, _ = L.oracle_forward(rows.cpu().numpy())
        assert rel_err(out.cpu().numpy(), ref) <= 2e-3
        assert torch.equal(out, L.moe(rows))

        z = L.moe.last_logits()
        cut = T // 3
        off = torch.tensor([0, cut, T], dtype=torch.int32, device=dev)
        loss, counts, coef = L.moe.balance(ALPHA, offsets=off)
        d = cm.balance_grad(z, coef, offsets=off)
        torch.cuda.synchronize()
        idx = L.oracle_route(rows.cpu().numpy())
        l64, n, _, d64, unit = reference(z.cpu().numpy(), idx, [0, cut, T], np.ones(T, bool), "sigmoid",
                                         float(np.float32(ALPHA)), np.ones(2))
        assert np.array_equal(counts.cpu().numpy(), n)
        assert (np.abs(loss.cpu().numpy() - l64) <= 26 * U * np.abs(l64)).all()
        assert (np.abs(d.cpu().numpy() - d64) <= 48 * U * unit + 1e-37).all()
    finally:
        L.close()


def test_balance_with_routing_limits_and_cache(dev):
    """Slots that the routing limits dropped count for no expert; a cached
    layer gives the resident layer's balance."""
    shape = synth.TINY
    L = DeviceLayer(shape, 1, 0, dev, max_tokens=4, keep_host=True)
    host = {k: torch.from_numpy(np.ascontiguousarray(v)).pin_memory() for k, v in L.host_routed.items()}
    cache = cm.ExpertCache(L.moe.cfg, L.tensors, host, n_slots=8)
    try:
        x = torch.from_numpy(synth.hidden(shape, 1, 4)).to(dev)
        L.moe(x)
        a = L.moe.balance(ALPHA)
        cache(x)
        b = cache.balance(ALPHA)
        assert torch.equal(cache.last_logits(), L.moe.last_logits())
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        assert int(a[1].sum()) == 4 * shape.top_k
        L.set_routing(1)
        L.moe(x)
        assert int(L.moe.balance(ALPHA)[1].sum()) == 4
    finally:
        cache.close()
        L.close()


def test_a_refused_call_leaves_the_residual(dev):
    """More rows than the layer takes: refused, and the same rows in two calls
    afterwards give what two calls on the first residual give."""
    shape = synth.TINY
    L = DeviceLayer(shape, 1, 0, dev, max_tokens=4)
    try:
        x = torch.from_numpy(synth.hidden(shape, 1, 6)).to(dev)
        res = torch.randn(6, shape.hidden, generator=torch.Generator().manual_seed(5)).to(dev)
        before = res.clone()
        with pytest.raises(cm.ColiMoeError) as e:
            L.moe.forward_normed(x, residual=res)
        assert e.value.code == cm.COLI_MOE_ECAPACITY
        torch.cuda.synchronize()
        assert torch.equal(res, before)
        for lo, hi in ((0, 4), (4, 6)):
            L.moe.forward_normed(x[lo:hi], residual=res[lo:hi])
        torch.cuda.synchronize()
        assert torch.equal(res, before + x)
    finally:
        L.close()


def test_balance_is_never_a_prefetchs(dev):
    """A prefetch routes other rows: no logits and no balance until the next
    forward, which gives its own."""
    shape = synth.TINY
    L = DeviceLayer(shape, 1, 0, dev, max_tokens=4, keep_host=True)
    host = {k: torch.from_numpy(np.ascontiguousarray(v)).pin_memory() for k, v in L.host_routed.items()}
    cache = cm.ExpertCache(L.moe.cfg, L.tensors, host, n_slots=8)
    try:
        x = torch.from_numpy(synth.hidden(shape, 1, 4)).to(dev)
        cache(x)
        z, want = cache.last_logits(), cache.balance(ALPHA)
        cache.prefetch(-x[:2], 1)
        for call in (cache.last_logits, lambda: cache.balance(ALPHA)):
            with pytest.raises(cm.ColiMoeError) as e:
                call()
            assert e.value.code == cm.COLI_MOE_EARG
        cache(x)
        assert torch.equal(cache.last_logits(), z)
        assert all(torch.equal(p, q) for p, q in zip(cache.balance(ALPHA), want))
    finally:
        cache.close()
        L.close()
