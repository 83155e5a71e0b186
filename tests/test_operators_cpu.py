"""The operators around the layer without a GPU: every refusal is made on the
host before any HIP call, by the C entry points (error codes) and by the
Python functions (ValueError), and calls with nothing to do succeed."""
import contextlib
import ctypes

import pytest

import routed_expert_ffn_f32_amd as cm

torch = pytest.importorskip("torch")

A = 0x7f0000001000  # addresses that are checked but never read


def norm_args(**kw):
    a = dict(rows=0, hidden=64, x_type=0, residual_type=0, weight_type=0, out_type=0, group=0, eps=1e-6, x=A,
             x_stride=64, residual=None, residual_stride=0, residual_out=None, residual_out_stride=0, weight=A,
             out=A + 0x10000, out_stride=64, scales=None, scales_stride=0)
    a.update(kw)
    return cm.coli_moe_rmsnorm_t(**a)


def norm_rc(**kw):
    return cm.load_library().coli_moe_rmsnorm(norm_args(**kw), None)


def test_rmsnorm_refusals():
    assert cm.load_library().coli_moe_rmsnorm(None, None) == -4
    assert norm_rc() == 0  # no rows: a dry run
    for bad in (dict(rows=-1), dict(hidden=0), dict(hidden=32769), dict(eps=-1.0), dict(eps=float("nan")),
                dict(x_type=3), dict(x_type=-1), dict(out_type=5), dict(out_type=-1), dict(group=64),
                dict(out_type=3, group=32), dict(out_type=4, group=-64), dict(weight_type=4),
                dict(residual=A), dict(residual_out=A), dict(residual=A, residual_out=A, residual_type=3)):
        assert norm_rc(**bad) == -4, bad
    two = dict(rows=2)
    for bad in (dict(x=None), dict(out=None), dict(x=A + 2), dict(out=A + 0x10002), dict(weight=A + 1),
                dict(x_type=1, x=A + 1), dict(out_stride=63), dict(out_stride=-64), dict(x_stride=-1),
                dict(x_stride=1 << 56), dict(out_type=3), dict(out_type=3, scales=A + 2, scales_stride=1),
                dict(out_type=3, scales=A, scales_stride=0),
                dict(out_type=4, group=64, hidden=65, x_stride=65, out_stride=65, scales=A, scales_stride=1),
                dict(residual=A, residual_stride=64, residual_out=A + 0x20000, residual_out_stride=63),
                dict(residual=A, residual_stride=128, residual_out=A, residual_out_stride=64),
                dict(residual=A, residual_stride=0, residual_out=A, residual_out_stride=0),
                dict(out=A, out_type=1), dict(out=A, x_stride=128)):
        assert norm_rc(**two, **bad) == -4, bad
    with pytest.raises(cm.ColiMoeError) as e:
        cm.coli_moe_rmsnorm(norm_args(hidden=0))
    assert e.value.code == -4


def balance_args(**kw):
    a = dict(tokens=0, n_experts=8, top_k=2, n_seqs=1, scores=0, alpha=0.01, logits=A, logits_stride=8, idx=A,
             seq_offsets=None, mask=None)
    a.update(kw)
    return cm.coli_moe_balance_t(**a)


def balance_rc(loss=A, counts=A, coef=A, ws=A, nbytes=1 << 30, **kw):
    return cm.load_library().coli_moe_balance(balance_args(**kw), loss, counts, coef, ws, nbytes, None)


def grad_rc(coef=A, dloss=None, out=A, stride=8, **kw):
    return cm.load_library().coli_moe_balance_grad(balance_args(**kw), coef, dloss, out, stride, None)


def test_balance_refusals():
    lib = cm.load_library()
    assert lib.coli_moe_balance(None, A, A, A, A, 1 << 30, None) == -4
    assert lib.coli_moe_balance_grad(None, A, None, A, 8, None) == -4
    assert grad_rc() == 0  # no tokens
    sizes = [(dict(tokens=-1), -4), (dict(n_seqs=0), -4), (dict(n_seqs=65537, seq_offsets=A), -4),
             (dict(n_experts=0), -2), (dict(n_experts=513, top_k=1), -2), (dict(top_k=0), -2), (dict(top_k=9), -2),
             (dict(n_experts=64, top_k=33), -2), (dict(tokens=(1 << 26) + 1), -4), (dict(scores=2), -4),
             (dict(n_seqs=2), -4), (dict(n_seqs=2, seq_offsets=A + 2), -4), (dict(tokens=4, logits=None), -4),
             (dict(tokens=4, logits=A + 2), -4), (dict(tokens=4, logits_stride=-1), -4)]
    for bad, code in sizes:
        assert balance_rc(**bad) == code, bad
        assert grad_rc(**bad) == code, bad
    for bad in (dict(loss=None), dict(counts=None), dict(coef=None), dict(ws=None), dict(ws=A + 8), dict(loss=A + 1),
                dict(tokens=4, idx=None), dict(tokens=4, idx=A + 1)):
        assert balance_rc(**bad) == -4, bad
    assert balance_rc(tokens=100, nbytes=cm.coli_moe_balance_workspace_bytes(100, 8, 1) - 1) == -1
    for bad in (dict(coef=None), dict(tokens=4, out=None), dict(tokens=4, stride=7), dict(dloss=A + 1)):
        assert grad_rc(**bad) == -4, bad
    for bad in ((-1, 8, 1), ((1 << 26) + 1, 8, 1), (4, 0, 1), (4, 513, 1), (4, 8, 0), (4, 8, 65537)):
        assert cm.coli_moe_balance_workspace_bytes(*bad) == 0
    assert lib.coli_moe_last_logits(None, A, None) == -4


def test_python_functions_refuse_host_tensors_and_wrong_shapes():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="GPU"):
        cm.rms_norm(x)
    with pytest.raises(ValueError, match="GPU"):
        cm.balance_loss(x, torch.zeros(2, 2, dtype=torch.int32), 0.01)
    with pytest.raises(ValueError, match="GPU"):
        cm.balance_grad(x, torch.zeros(1, 64))
    m = torch.zeros(2, 64, device="meta")
    with pytest.raises(ValueError):
        cm.rms_norm(m)


def linear_args(**kw):
    a = dict(m=0, n=8, k=64, type=1, out_type=0, bias_type=0, act=0, x=A, ldx=64, w=A, ldw=64, x_scale=None,
             w_scale=None, bias=None, residual=None, ldr=0, out=A, ldo=8)
    a.update(kw)
    return cm.coli_moe_linear_t(**a)


def linear_rc(**kw):
    return cm.load_library().coli_moe_linear(linear_args(**kw), None)


def test_linear_refusals():
    assert cm.load_library().coli_moe_linear(None, None) == -4
    assert linear_rc() == 0  # no rows
    for bad in (dict(m=-1), dict(m=(1 << 22) + 1), dict(n=0), dict(n=(1 << 22) + 1), dict(k=0), dict(k=65552),
                dict(k=4), dict(k=60), dict(type=3, k=72), dict(type=4, k=8), dict(type=0), dict(type=5),
                dict(type=-1), dict(out_type=3), dict(out_type=-1), dict(act=-1), dict(act=6),
                dict(bias=A, bias_type=3)):
        assert linear_rc(**bad) == -4, bad
    for bad in (dict(x=None), dict(w=None), dict(out=None), dict(x=A + 8), dict(w=A + 2), dict(out=A + 2),
                dict(out_type=1, out=A + 1), dict(ldx=63), dict(ldx=-64), dict(ldw=68), dict(ldx=1 << 23),
                dict(ldw=1 << 40), dict(ldo=7), dict(bias=A + 2), dict(bias=A + 1, bias_type=1),
                dict(residual=A + 2), dict(residual=A + 64, ldr=-1), dict(residual=A, ldr=16),
                dict(x_scale=A), dict(w_scale=A), dict(type=3), dict(type=3, x_scale=A),
                dict(type=4, x_scale=A, w_scale=A + 2), dict(type=3, ldx=72, x_scale=A, w_scale=A)):
        assert linear_rc(m=2, **bad) == -4, bad
    with pytest.raises(cm.ColiMoeError) as e:
        cm.coli_moe_linear(linear_args(k=0))
    assert e.value.code == -4


def test_linear_python_refusals():
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        cm.linear(x, w)


def test_overlapping_results_are_refused():
    """Arrays that begin at the same address and cannot be the same array."""
    res = dict(rows=2, residual=A + 0x40000, residual_stride=64, residual_out=A + 0x40000, residual_out_stride=64)
    for bad in (dict(out=A + 0x40000), dict(residual_out=A + 0x10000),  # out is the residual, or the sum
                dict(residual_out=A, residual_type=1), dict(residual_out=A, residual_out_stride=72)):
        assert norm_rc(**{**res, **bad}) == -4, bad
    assert norm_rc(eps=float("inf")) == -4
    for bad in (dict(x=A + 0x10000, w=A, out=A), dict(x=A, w=A + 0x10000, out=A)):
        assert linear_rc(m=2, **bad) == -4, bad


def test_a_layers_device_is_current_in_its_calls(monkeypatch):
    """The default streams of two devices have the same handle: with another
    device current, the layer's has to be set all the same."""
    from types import SimpleNamespace
    entered = []

    @contextlib.contextmanager
    def device(d):
        entered.append(d)
        yield

    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    one = torch.device("cuda", 1)
    with cm._layer_stream(0, torch.device("cuda", 0)):
        assert not entered
    with cm._layer_stream(0, one):
        assert entered == [one]


class HostLayer(cm._RoutedCalls):
    """A layer's public calls with nothing behind them: a norm or a forward
    that is reached shows in `reached`."""

    def __init__(self, monkeypatch):
        self.cfg = cm.make_config(hidden=128, n_experts=8, top_k=2, inter=64, n_shared=0, routed_scaling_factor=1.0,
                                  max_tokens=4)
        self.workspace, self.stream, self.handle, self.reached = torch.empty(0), 0, 1, []
        monkeypatch.setattr(cm, "rms_norm", lambda *a, **kw: self.reached.append("norm"))
        monkeypatch.setattr(cm, "_layer_stream", lambda *a: contextlib.nullcontext())

    def forward(self, hidden, out):
        self.reached.append("forward")
        return out

    def _layer(self):
        return self.handle


def test_forward_normed_refuses_shapes_that_are_not_the_layers(monkeypatch):
    """The layer reads and writes rows of its own width: narrower ones would
    be left behind."""
    layer = HostLayer(monkeypatch)
    x = torch.zeros(3, 128)
    assert layer.forward_normed(x).shape == (3, 128) and layer.reached == ["norm", "forward"]
    assert layer.forward_normed(x[:1], out=torch.empty(1, 200)[:, :128]).shape == (1, 128)
    layer.reached.clear()
    for bad in (dict(x=x[:, :64]), dict(x=torch.zeros(3, 256)), dict(x=x[0]), dict(x=torch.zeros(128, 3).t()),
                dict(x=torch.zeros(3, 128, device="meta")), dict(x=x, out=torch.zeros(2, 128)),
                dict(x=x, out=torch.zeros(3, 64)), dict(x=x, out=x.half()), dict(x=x, out=torch.zeros(3, 256)[:, :128]),
                dict(x=x, out=torch.zeros(3, 128, device="meta"))):
        with pytest.raises(ValueError):
            layer.forward_normed(**bad)
    assert not layer.reached


def test_forward_normed_refuses_before_the_residual_changes(monkeypatch):
    """Calls that the layer refuses are refused before the norm stores the sum:
    a caller that splits the batch and calls again adds once."""
    layer = HostLayer(monkeypatch)
    many, wide = torch.zeros(5, 128), torch.zeros(3 * 128 + 1)
    with pytest.raises(cm.ColiMoeError) as e:
        layer.forward_normed(many, residual=many.clone())
    assert e.value.code == cm.COLI_MOE_ECAPACITY
    off = wide[1:].view(3, 128) if wide.data_ptr() % 16 == 0 else wide[:-1].view(3, 128)
    closed = HostLayer(monkeypatch)
    closed.handle = None
    for refused, kw in ((layer, dict(out=off)), (closed, {})):
        with pytest.raises(cm.ColiMoeError) as e:
            refused.forward_normed(many[:3], residual=many[:3].clone(), **kw)
        assert e.value.code == cm.COLI_MOE_EARG
    assert not layer.reached and not closed.reached


def test_tensors_written_in_place_are_marked_as_changed(monkeypatch):
    """A backward pass that saved the old contents of a residual or a result
    raises; nothing else is marked."""
    monkeypatch.setattr(cm, "_gpu", lambda t, what: t.device)
    monkeypatch.setattr(cm, "_enqueue", lambda *a: None)
    x, w = torch.zeros(2, 64), torch.zeros(8, 64)
    h, q = x.bfloat16(), torch.zeros(2, 64, dtype=torch.int8)
    res, kept, out, scales = torch.zeros(2, 64), torch.zeros(2, 64), torch.zeros(2, 64), torch.zeros(2, 1)
    cm.rms_norm(x, residual=res)
    assert res._version == 1
    cm.rms_norm(x, residual=res, residual_out=kept, out=out)
    assert (res._version, kept._version, out._version) == (1, 1, 1)
    cm.rms_norm(x, out=q, scales=scales)
    assert (q._version, scales._version) == (1, 1)
    y = torch.zeros(2, 8)
    cm.linear(h, w.bfloat16(), residual=y, out=y)
    assert y._version == 1
    cm.balance_grad(x, torch.zeros(1, 64), out=out)
    assert out._version == 2
    assert x._version == h._version == w._version == 0
    leaf = torch.ones(2, 64, requires_grad=True)
    stream = leaf * 1
    square = stream * stream
    assert not cm.rms_norm(x, residual=stream).requires_grad
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        square.sum().backward()


def test_more_choices_than_a_count_holds_are_refused():
    """2^26 tokens of 32 choices, all of which may name one expert, pass int32
    by one.  The gradient, which reads no choices, has no such bound."""
    most = dict(tokens=1 << 26, n_experts=32, logits_stride=32, top_k=32)
    nbytes = cm.coli_moe_balance_workspace_bytes(1 << 26, 32, 1)
    assert balance_rc(**most, nbytes=nbytes) == -4
    assert balance_rc(**{**most, "top_k": 31}, nbytes=nbytes - 1) == -1  # the next check: nothing is enqueued
    assert grad_rc(**most, stride=31) == -4


def test_sizes_past_32_bits_are_refused(monkeypatch):
    """They would wrap around on their way into the C structs: 2^32 + 4 rows
    would be 4."""
    monkeypatch.setattr(cm, "_gpu", lambda t, what: t.device)
    monkeypatch.setattr(cm, "_enqueue", lambda *a: pytest.fail("enqueued"))
    monkeypatch.setattr(cm, "_vector", lambda *a: None)
    many = (1 << 32) + 4

    def shaped(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="meta")

    x, w, bf16 = shaped(many, 64), shaped(8, 64), torch.bfloat16
    calls = [lambda: cm.rms_norm(x), lambda: cm.rms_norm(shaped(4, many)), lambda: cm.linear(x.to(bf16), w.to(bf16)),
             lambda: cm.linear(w.to(bf16), x.to(bf16)),
             lambda: cm.linear(shaped(2, many, dtype=bf16), shaped(3, many, dtype=bf16)),
             lambda: cm.balance_loss(x, shaped(many, 2, dtype=torch.int32), 0.1),
             lambda: cm.balance_grad(x, shaped(1, 64)),
             lambda: cm.balance_loss(w, shaped(8, 2, dtype=torch.int32), 0.1, offsets=shaped(many, dtype=torch.int32))]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="2\\^31|65536"):
            call()
            pytest.fail(f"call {i} was not refused")


def test_a_layers_given_result_is_marked_as_changed(monkeypatch):
    layer = HostLayer(monkeypatch)
    x, out = torch.zeros(3, 128), torch.zeros(3, 128)
    assert layer.forward_normed(x, out=out) is out and out._version == 1 and x._version == 0
