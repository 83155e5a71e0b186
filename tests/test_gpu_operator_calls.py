"""Calls of the operators around the layer that go wrong easily: arrays whose
offsets pass 32 bits, extreme integers, a side stream, two graphs, several
threads, empty results, and refusals that need device tensors."""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import routed_expert_ffn_f32_amd as cm
import synth
from tests.gpu_util import DeviceLayer
from tests.test_gpu_rmsnorm import check_float, reference

pytestmark = pytest.mark.gpu

F32, BF16, I8, E4 = torch.float32, torch.bfloat16, torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def far_rows(rows, cols, stride, dtype, dev):
    """A [rows, cols] view whose rows lie `stride` elements apart."""
    return torch.empty((rows - 1) * stride + cols, dtype=dtype, device=dev).as_strided((rows, cols), (stride, 1))


def test_norm_offsets_past_32_bits(dev):
    x = far_rows(3, 264, (1 << 30) + 8, BF16, dev)  # 4 GiB
    x.copy_(torch.randn(3, 264, generator=torch.Generator().manual_seed(1)))
    out = far_rows(3, 264, (1 << 30) + 64, BF16, dev)
    cm.rms_norm(x, None, 1e-6, out=out)
    _, y64, _ = reference(x.cpu(), None, 1e-6)
    check_float(out.cpu(), y64, BF16)


@pytest.mark.parametrize("m", [40, 300])
def test_linear_offsets_past_32_bits(dev, m):
    g = torch.Generator().manual_seed(m)
    rows = torch.randint(-3, 4, (m, 64), generator=g).float()
    x = far_rows(m, 64, (1 << 22) // 2 if m > 40 else 1 << 21, BF16, dev)
    x.copy_(rows)
    w = torch.randint(-3, 4, (70, 64), generator=g).float()
    out = far_rows(m, 70, ((1 << 31) // m + 64) // 8 * 8, BF16, dev)
    res = torch.randint(-3, 4, (m, 70), generator=g).float()
    cm.linear(x, w.to(dev, BF16), residual=res.to(dev, BF16), out=out)
    assert torch.equal(out.cpu().float(), (rows @ w.t() + res).bfloat16().float())


def test_balance_offsets_past_32_bits(dev):
    T, E = 40, 16
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(2))
    far = far_rows(T, E, 1 << 26, F32, dev)
    far.copy_(z)
    idx = torch.topk(z, 2, dim=1).indices.to(torch.int32).to(dev)
    a, b = cm.balance_loss(far, idx, 0.1), cm.balance_loss(z.to(dev), idx, 0.1)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    d = cm.balance_grad(far, a[2], out=far_rows(T, E, 1 << 26, F32, dev))
    assert torch.equal(d.cpu(), cm.balance_grad(z.to(dev), b[2]).cpu())


@pytest.mark.parametrize("m", [1, 40, 200])
def test_int8_at_its_largest(dev, m):
    """-128 everywhere over the longest K: a sum of 2^30, exact."""
    x = torch.full((m, 65536), -128, dtype=I8, device=dev)
    w = torch.full((17, 65536), -128, dtype=I8, device=dev)
    got = cm.linear(x, w, torch.ones(m, device=dev), torch.ones(17, device=dev), out_dtype=F32)
    assert (got == 2.0 ** 30).all()


@pytest.mark.parametrize("rows,hidden", [((1 << 20) * 16 + 5, 8), ((1 << 20) * 4 + 5, 136), ((1 << 20) + 3, 520)])
def test_many_short_rows(dev, rows, hidden):
    """More workgroups than one axis of the grid is given: several rows a wave,
    a row a wave, a row a workgroup."""
    x = torch.zeros(rows, hidden, dtype=BF16, device=dev)
    x[-3:] = 2.0
    out = cm.rms_norm(x, None, 0.0)
    assert (out[-3:] == 1).all() and not out[:-3].any()


def test_forward_normed_from_another_stream(dev):
    """The layer's own stream carries the norm too, whatever stream is current."""
    shape = synth.TINY
    L = DeviceLayer(shape, 1, 0, dev, max_tokens=4)
    try:
        x = torch.from_numpy(synth.hidden(shape, 1, 4)).to(dev)
        w = torch.ones(shape.hidden, device=dev)
        res = torch.randn(4, shape.hidden, device=dev)
        r1, r2 = res.clone(), res.clone()
        want = L.moe.forward_normed(x, w, residual=r1)
        bal = L.moe.balance(0.01)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            got = L.moe.forward_normed(x, w, residual=r2)
            bal2 = L.moe.balance(0.01)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(r1, r2)
        assert all(torch.equal(p, q) for p, q in zip(bal, bal2))
    finally:
        L.close()


def test_whole_block_captured(dev):
    """Norm to int8, SwiGLU product, projection onto the residual, norm, MoE
    layer: one graph, replayed on new rows with eager work in between, gives
    the eager results each time."""
    shape = synth.TINY
    h, inter, T = shape.hidden, 256, 4
    L = DeviceLayer(shape, 1, 0, dev, max_tokens=T)
    g = torch.Generator().manual_seed(4)
    side = torch.cuda.Stream()
    try:
        wq = torch.randint(-127, 128, (2 * inter, h), generator=g).to(I8).to(dev)
        ws = (torch.rand(2 * inter, generator=g) / 500).to(dev)
        wd = (torch.randn(h, inter, generator=g) / 16).to(dev, BF16)
        nw = (1 + 0.1 * torch.randn(h, generator=g)).to(dev)
        xs = [torch.randn(T, h, generator=g).to(dev) for _ in range(3)]
        L.moe.stream = side.cuda_stream

        def block(x):
            q, s = cm.rms_norm(x, nw, out_dtype=I8)
            mid = cm.linear(q, wq, s, ws, act="swiglu")
            stream = x.clone()
            cm.linear(mid, wd, residual=stream, out=stream)
            out = L.moe.forward_normed(stream, nw)
            return stream, out

        with torch.cuda.stream(side):
            want = [tuple(t.clone() for t in block(x)) for x in xs]
            x = xs[0].clone()
            side.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                got = block(x)
            for i in (1, 2, 0, 2):
                x.copy_(xs[i])
                graph.replay()
                side.synchronize()
                assert all(torch.equal(p, q) for p, q in zip(got, want[i])), i
                block(xs[(i + 1) % 3])
    finally:
        torch.cuda.synchronize()
        L.close()


def test_threads(dev):
    """Calls from several threads, each on a stream of its own."""
    x = [torch.randn(50, 640, device=dev, dtype=F32).bfloat16() for _ in range(4)]
    w = torch.randn(96, 640, device=dev).bfloat16()
    want = [cm.linear(cm.rms_norm(v), w) for v in x]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got[i] = cm.linear(cm.rms_norm(x[i]), w)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals_on_the_device(dev):
    x, w = torch.zeros(4, 64, device=dev), torch.zeros(6, 64, device=dev)
    h, q = x.half(), x.to(I8)
    one4, one6 = torch.ones(4, device=dev), torch.ones(6, device=dev)
    bad = [lambda: cm.rms_norm(x[0]), lambda: cm.rms_norm(x.t()), lambda: cm.rms_norm(x.double()), lambda: cm.rms_norm(q),
           lambda: cm.rms_norm(x, one4), lambda: cm.rms_norm(x, torch.ones(64)), lambda: cm.rms_norm(x, residual=w),
           lambda: cm.rms_norm(x, residual_out=x), lambda: cm.rms_norm(x, residual=x, residual_out=h),
           lambda: cm.rms_norm(x, out=h, out_dtype=F32), lambda: cm.rms_norm(x, out_dtype=torch.float64),
           lambda: cm.rms_norm(x, out_dtype=I8, group=32), lambda: cm.rms_norm(x, scales=torch.ones(4, 1, device=dev)),
           lambda: cm.rms_norm(x, out_dtype=I8, scales=torch.ones(4, 2, device=dev)),
           lambda: cm.linear(x, w), lambda: cm.linear(h, w), lambda: cm.linear(h, w.half()[:, :32]),
           lambda: cm.linear(h, w.half(), act="tanh"), lambda: cm.linear(h, w.half()[:5], act="swiglu"),
           lambda: cm.linear(q, w.to(I8)), lambda: cm.linear(q, w.to(I8), one6, one6), lambda: cm.linear(q, w.to(I8), one4, one6.half()),
           lambda: cm.linear(h, w.half(), one4, one6), lambda: cm.linear(h, w.half(), bias=one4),
           lambda: cm.linear(h, w.half(), residual=torch.zeros(4, 5, device=dev)), lambda: cm.linear(h, w.half(), out_dtype=I8),
           lambda: cm.linear(h, w.half(), out=torch.zeros(4, 6, device=dev).half(), residual=torch.zeros(4, 6, device=dev)),
           lambda: cm.balance_loss(h, torch.zeros(4, 2, dtype=torch.int32, device=dev), 1.0),
           lambda: cm.balance_loss(x, torch.zeros(4, 2, device=dev), 1.0),
           lambda: cm.balance_loss(x, torch.zeros(3, 2, dtype=torch.int32, device=dev), 1.0),
           lambda: cm.balance_loss(x, torch.zeros(4, 4, dtype=torch.int32, device=dev)[:, :2], 1.0),
           lambda: cm.balance_loss(x, torch.zeros(4, 2, dtype=torch.int32, device=dev), 1.0, scores="relu"),
           lambda: cm.balance_loss(x, torch.zeros(4, 2, dtype=torch.int32, device=dev), 1.0, mask=one4),
           lambda: cm.balance_loss(x, torch.zeros(4, 2, dtype=torch.int32, device=dev), 1.0,
                                   offsets=torch.zeros(1, dtype=torch.int32, device=dev)),
           lambda: cm.balance_loss(x, torch.zeros(4, 2, dtype=torch.int32, device=dev), 1.0,
                                   offsets=torch.zeros(3, dtype=torch.int64, device=dev)),
           lambda: cm.balance_grad(x, torch.zeros(2, 64, device=dev)), lambda: cm.balance_grad(x, torch.zeros(1, 64, device=dev), one4),
           lambda: cm.balance_grad(x, torch.zeros(1, 64, device=dev), out=h)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    codes = [(lambda: cm.rms_norm(x, eps=-1.0), -4), (lambda: cm.rms_norm(torch.zeros(1, 32769, device=dev)), -4),
             (lambda: cm.rms_norm(x, residual=x[:1].expand(4, 64)), -4),
             (lambda: cm.linear(torch.zeros(2, 12, device=dev).half(), torch.zeros(3, 12, device=dev).half()), -4),
             (lambda: cm.linear(torch.zeros(2, 72, device=dev).half()[:, 4:68], w.half()), -4),
             (lambda: cm.balance_loss(torch.zeros(2, 600, device=dev), torch.zeros(2, 1, dtype=torch.int32, device=dev), 1.0), -2),
             (lambda: cm.balance_loss(x, torch.zeros(4, 33, dtype=torch.int32, device=dev), 1.0), -2)]
    for i, (call, code) in enumerate(codes):
        with pytest.raises(cm.ColiMoeError) as e:
            call()
        assert e.value.code == code, i
    torch.cuda.synchronize()


def test_layer_on_its_own_stream(dev):
    """A layer on one stream, called while another is current, with work still
    going on both: arguments made on the current stream just before a call are
    read as made, results can be used there, and memory that the calls drop or
    that the caller reuses afterwards is not written late."""
    shape = synth.TINY
    L = DeviceLayer(shape, 1, 0, dev, max_tokens=16)
    own, side = torch.cuda.Stream(), torch.cuda.Stream()
    a = torch.randn(2048, 2048, device=dev)

    def delay():
        for _ in range(20):
            torch.mm(a, a)

    try:
        T, h = 16, shape.hidden
        x0 = torch.from_numpy(synth.hidden(shape, 1, T)).to(dev)
        res0, off0 = torch.randn(T, h, device=dev), torch.tensor([0, 5, T], dtype=torch.int32, device=dev)
        keep0 = torch.arange(T, device=dev) % 3 != 0
        r = res0.clone()
        want = (L.moe.forward_normed(x0, residual=r).clone(), r.clone(), *L.moe.balance(0.01, offsets=off0, mask=keep0),
                L.moe.last_logits(), L.moe.last_routing()[1]["idx"])
        x, res, off, keep = torch.zeros_like(x0), torch.zeros_like(res0), torch.zeros_like(off0), torch.zeros_like(keep0)
        torch.cuda.synchronize()
        L.moe.stream = own.cuda_stream
        for _ in range(3):
            with torch.cuda.stream(own):
                delay()
            with torch.cuda.stream(side):
                delay()
                for dst, src in ((x, x0), (res, res0), (off, off0), (keep, keep0)):
                    dst.copy_(src)
                out = L.moe.forward_normed(x, residual=res)
                x.fill_(float("nan"))                                  # the caller's again
                got = [out.clone(), res.clone()]
                with torch.cuda.stream(own):
                    delay()
                got += L.moe.balance(0.01, offsets=off, mask=keep)
                off.zero_(), keep.zero_()
                # blocks of the sizes that balance has just dropped
                later = [torch.full((n,), -7, dtype=torch.int32, device=dev)
                         for n in (T * shape.top_k, T * shape.n_experts, shape.n_experts, 1) for _ in range(8)]
                with torch.cuda.stream(own):
                    delay()
                got += [L.moe.last_logits(), L.moe.last_routing()[1]["idx"]]
                got = [t.clone() for t in got]
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want))
            assert all((t == -7).all() for t in later)
    finally:
        torch.cuda.synchronize()
        L.close()


@pytest.mark.parametrize("own_stream", [False, True])
def test_layer_calls_captured(dev, own_stream):
    """The norm with the layer, the balance of its routing, the gradient and
    the logits in one graph, on the layer's stream or beside it: replays on new
    rows, with eager calls of the same layer in between, give the eager
    results each time."""
    shape, T = synth.TINY, 8
    L = DeviceLayer(shape, 1, 0, dev, max_tokens=T)
    own, side = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.Generator().manual_seed(6)

    def block(x, res):
        out = L.moe.forward_normed(x, residual=res)
        balance = L.moe.balance(0.01)
        z = L.moe.last_logits()
        return out, *balance, z, cm.balance_grad(z, balance[2]), res

    try:
        xs, rs = ([torch.randn(T, shape.hidden, generator=g).to(dev) for _ in range(3)] for _ in range(2))
        want = [[t.clone() for t in block(x, r.clone())] for x, r in zip(xs, rs)]
        x, res = xs[0].clone(), rs[0].clone()
        torch.cuda.synchronize()
        L.moe.stream = (own if own_stream else side).cuda_stream
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                got = block(x, res)
            for i in (1, 2, 0, 1):
                x.copy_(xs[i])
                res.copy_(rs[i])
                graph.replay()
                side.synchronize()
                assert all(torch.equal(p, q) for p, q in zip(got, want[i])), i
                block(xs[(i + 1) % 3], rs[0].clone())
                side.synchronize()
    finally:
        torch.cuda.synchronize()
        L.close()
