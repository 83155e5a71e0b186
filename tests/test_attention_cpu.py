"""Rotary positions and the 4-bit cache without a GPU: refusals are made on
the host before any HIP call, and calls with nothing to do succeed."""
import pytest

import routed_expert_ffn_f32_amd as cm

torch = pytest.importorskip("torch")

A = 0x7f0000001000  # addresses that are checked but never read
B, C, D = A + (1 << 20), A + (2 << 20), A + (3 << 20)


def rotary_rc(**kw):
    a = dict(tokens=0, heads=2, dim=64, part=32, type=1, interleaved=0, inverse=0, wide=0, scale=1.0, x=A, x_token=128,
             x_head=64, positions=C, freq=D, out=B, out_token=128, out_head=64)
    a.update(kw)
    return cm.load_library().coli_moe_rotary(cm.coli_moe_rotary_t(**a), None)


def test_rotary_refusals():
    assert cm.load_library().coli_moe_rotary(None, None) == -4
    assert rotary_rc() == 0  # no tokens: a dry run
    for bad in (dict(tokens=-1), dict(tokens=(1 << 26) + 1), dict(heads=0), dict(heads=4097), dict(dim=0), dict(dim=4097),
                dict(part=-2), dict(part=31), dict(part=66), dict(type=3), dict(type=-1), dict(interleaved=2),
                dict(inverse=-1), dict(wide=2), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert rotary_rc(**bad) == -4, bad
    for bad in (dict(x=None), dict(x=A + 1), dict(out=None), dict(out=B + 1), dict(positions=None), dict(positions=C + 2),
                dict(wide=1, positions=C + 4), dict(freq=None), dict(freq=D + 2), dict(x_token=-1), dict(x_head=-64),
                dict(out_head=63), dict(out_token=127), dict(out_token=0), dict(out_head=0), dict(out_head=100),
                dict(x_token=1 << 41), dict(out=A, out_token=256), dict(out=A, out_head=65, out_token=130)):
        assert rotary_rc(tokens=2, **bad) == -4, bad


def kv(**kw):
    a = dict(n_pages=4, page_size=16, kv_heads=2, head_dim=64, k_codes=A, k_scales=B, v_codes=C, v_scales=D, weights=None)
    a.update(kw)
    return cm.coli_moe_kv_t(**a)


def rows(**kw):
    a = dict(tokens=0, seqs=2, table_width=2, table=A, table_stride=2, lengths=B, offsets=C)
    a.update(kw)
    return cm.coli_moe_kv_rows_t(**a)


def values(**kw):
    a = dict(type=1, clear=0, k=A, k_token=128, k_head=64, v=B, v_token=128, v_head=64)
    a.update(kw)
    return cm.coli_moe_kv_values_t(**a)


def att(**kw):
    a = dict(q_heads=4, type=1, window=0, clear=0, scale=0.1, q=A, q_token=256, q_head=64, out=B, out_token=256, out_head=64,
             weights_out=None)
    a.update(kw)
    return cm.coli_moe_kv_attention_t(**a)


def evi(**kw):
    a = dict(keep=8, first=2, recent=3, into_width=1, into=C, into_stride=1, kept=D, new_lengths=D + 4096)
    a.update(kw)
    return cm.coli_moe_kv_evict_t(**a)


BAD_KV = (dict(n_pages=0), dict(n_pages=-1), dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(kv_heads=0),
          dict(kv_heads=1025), dict(head_dim=96), dict(head_dim=0), dict(head_dim=512))
BAD_KV_POINTERS = (dict(k_codes=None), dict(k_codes=A + 8), dict(k_scales=B + 2), dict(v_codes=None), dict(v_scales=None),
                   dict(weights=A + 4))
BAD_ROWS = (dict(seqs=0), dict(seqs=65537), dict(table_width=0), dict(table_width=(1 << 26) + 1))
BAD_TOKENS = (dict(tokens=-1), dict(tokens=(1 << 22) + 1), dict(offsets=None), dict(offsets=None, tokens=3))
BAD_ROW_POINTERS = (dict(table=None), dict(table=A + 2), dict(lengths=None), dict(lengths=B + 1), dict(offsets=C + 2),
                    dict(table_stride=-1), dict(table_stride=1 << 41))


@pytest.mark.parametrize("entry", ["coli_moe_kv_append", "coli_moe_kv_read"])
def test_append_and_read_refusals(entry):
    call = lambda k=kv(), r=rows(), v=values(): getattr(cm.load_library(), entry)(k, r, v, None)  # noqa: E731, B008
    assert call() == 0  # no tokens: a dry run
    assert call(k=None) == call(r=None) == call(v=None) == -4
    for bad in BAD_KV + BAD_KV_POINTERS:
        assert call(k=kv(**bad)) == -4, bad
    for bad in BAD_ROWS + BAD_TOKENS + BAD_ROW_POINTERS:
        assert call(r=rows(**bad)) == -4, bad
    two = rows(tokens=2)
    for bad in (dict(type=3), dict(type=-1), dict(clear=-1),
                dict(clear=2 if entry.endswith("read") else 1), dict(k=None), dict(k=A + 1), dict(v=None),
                dict(v=B + 1), dict(k_token=-1),
                dict(k_head=-1), dict(v_token=1 << 41)):
        assert call(r=two, v=values(**bad)) == -4, bad
    if entry == "coli_moe_kv_read":
        for bad in (dict(k_head=63), dict(k_token=127), dict(v_token=0), dict(v=A)):
            assert call(r=two, v=values(**bad)) == -4, bad


def test_attention_refusals():
    lib = cm.load_library()
    call = lambda k=kv(), r=rows(), a=att(), ws=A, n=1 << 40: lib.coli_moe_kv_attention(k, r, a, ws, n, None)  # noqa: E731, B008
    size = lambda k=kv(), r=rows(), a=att(): lib.coli_moe_kv_attention_workspace_bytes(k, r, a)  # noqa: E731, B008
    assert call() == 0 and size() > 0
    assert call(k=None) == call(r=None) == call(a=None) == -4
    assert size(k=None) == size(r=None) == size(a=None) == 0
    for bad in BAD_KV:
        assert call(k=kv(**bad)) == -4 and size(k=kv(**bad)) == 0, bad
    for bad in BAD_KV_POINTERS:
        assert call(k=kv(**bad)) == -4, bad
    for bad in BAD_ROWS + BAD_TOKENS:
        assert call(r=rows(**bad)) == -4 and size(r=rows(**bad)) == 0, bad
    for bad in BAD_ROW_POINTERS:
        assert call(r=rows(**bad)) == -4, bad
    for bad in (dict(q_heads=0), dict(q_heads=3), dict(q_heads=1), dict(q_heads=514), dict(type=0), dict(type=3),
                dict(window=-1), dict(clear=2), dict(scale=float("nan")), dict(scale=float("-inf"))):
        assert call(a=att(**bad)) == -4 and size(a=att(**bad)) == 0, bad
    assert call(a=att(weights_out=A)) == -4  # the cache keeps none
    assert call(k=kv(weights=A), a=att(weights_out=A + 4)) == -4
    two = rows(tokens=2)
    for bad in (dict(q=None), dict(q=A + 1), dict(out=None), dict(out=A), dict(q_token=-1), dict(out_head=63),
                dict(out_token=255), dict(out_token=0)):
        assert call(r=two, a=att(**bad)) == -4, bad
    assert call(r=two, ws=None) == call(r=two, ws=A + 8) == -4
    assert call(r=two, n=size(r=two) - 1) == -1
    # more keys in the table: more splits, so more workspace, up to a bound; the weights need a place too
    wide = size(r=rows(tokens=2, table_width=4096))
    assert size(r=two) < wide == size(r=rows(tokens=2, table_width=1 << 20)) < 1 << 28
    assert size(r=rows(tokens=2, table_width=4096), a=att(weights_out=A)) > wide


def test_evict_refusals():
    lib = cm.load_library()
    call = lambda k=kv(weights=A), r=rows(), a=evi(): lib.coli_moe_kv_evict(k, r, a, None)  # noqa: E731, B008
    assert call(k=None) == call(r=None) == call(a=None) == -4
    for bad in BAD_KV + BAD_KV_POINTERS:
        assert call(k=kv(**{**dict(weights=A), **bad})) == -4, bad
    assert call(k=kv()) == -4  # no weights
    for bad in BAD_ROWS + tuple(b for b in BAD_ROW_POINTERS if "offsets" not in b):
        assert call(r=rows(**bad)) == -4, bad
    for bad in (dict(keep=0), dict(keep=17), dict(first=-1), dict(recent=-1), dict(first=6), dict(first=1 << 31 - 1 - 1),
                dict(recent=2147483647), dict(into_width=0), dict(into_width=(1 << 26) + 1), dict(into=None),
                dict(into=C + 2), dict(into=A), dict(into_stride=-1), dict(kept=None), dict(kept=D + 1),
                dict(new_lengths=None), dict(new_lengths=B)):
        assert call(a=evi(**bad)) == -4, bad


def test_python_refusals_need_no_gpu():
    x = torch.zeros(2, 3, 64)
    with pytest.raises(ValueError):
        cm.rotary(x, torch.zeros(2, dtype=torch.int32), torch.zeros(4))
    with pytest.raises(ValueError):
        cm.KVCache(torch.zeros(2, 2, 16, 32, dtype=torch.uint8), None, None, None)
    with pytest.raises(ValueError):
        cm.KVCache.empty(2, 2, 96)
    for bad in (dict(part=0), dict(part=7), dict(part=8, base=1.0), dict(part=8, factor=0.5), dict(part=8, scaling="yes"),
                dict(part=2, scaling="base"), dict(part=8, scaling="parts", beta_fast=1.0, beta_slow=2.0),
                dict(part=8, original=0)):
        with pytest.raises(ValueError):
            cm.rotary_frequencies(**bad)
