"""Results of rotary positions and of the cache's calls that overlap what the
call reads, or each other, are refused on the host before any HIP call."""
import pytest

import routed_expert_ffn_f32_amd as cm
from tests.test_attention_cpu import A, B, att, evi, kv, rotary_rc, rows, values

BAD = -4


@pytest.mark.parametrize("out", [
    dict(out=A + 2 * 64),            # a head further in the same buffer
    dict(out=A - 2 * 64),
    dict(out=A + 2),                 # an element further
    dict(out=A + 2 * 128),           # a token further
    dict(out=A + 2 * (4 * 128 + 64)),
    dict(out=A, out_token=256),      # other strides from the same place
    dict(out=A + 2 * 32, out_token=192, out_head=96),
])
def test_rotary(out):
    assert rotary_rc(**{**dict(tokens=5, x=A, x_token=128, x_head=64, out_token=128, out_head=64), **out}) == BAD


@pytest.mark.parametrize("out", [
    dict(x_token=512, out=A + 2 * 64, out_token=512),   # heads 0, 1 to heads 1, 2 of a wider row
    dict(x_token=512, out=A + 2 * (512 * 3 + 100), out_token=512),
    dict(x_token=64, x_head=1024, out=A + 2 * 64, out_token=64, out_head=1024),  # tokens side by side in a head
    dict(x_token=0, out=A + 2 * 64, out_token=128),     # one token for all, inside of the result
    dict(x_token=0, x_head=0, out=A - 2 * (3 * 128 + 1), out_token=128),
    dict(x_token=128, x_head=0, out=A + 2 * 127, out_token=128),
    dict(x_token=1024, x_head=192, out=A + 2 * (64 + 65), out_token=1024, out_head=64),  # heads of other steps
    dict(x_token=1024, x_head=64, out=A + 2 * 127, out_token=1024, out_head=192),
])
def test_rotary_in_fused_buffers(out):
    assert rotary_rc(**{**dict(tokens=5, x=A, x_head=64, out_head=64), **out}) == BAD


def test_attention():
    lib = cm.load_library()
    call = lambda r=rows(tokens=2), k=kv(), **a: lib.coli_moe_kv_attention(k, r, att(**a), A + (8 << 20), 1 << 40, None)  # noqa: E731, B008
    for out in (A + 2 * 64, A - 2 * 64, A + 2 * 256, A + 2 * 3, A):
        assert call(out=out) == BAD, out
    assert call(q_token=1024, out=A + 2 * 64, out_token=1024) == BAD
    # sums beside the cache's weights, not across them
    n = 4 * 2 * 16 * 4  # bytes of the weights
    far = A + (16 << 20)
    for at in (far + 16, far - 16, far + n - 16, far - n + 16):
        assert call(k=kv(weights=far), weights_out=at) == BAD, at


def test_read():
    lib = cm.load_library()
    call = lambda **a: lib.coli_moe_kv_read(kv(), rows(tokens=2), values(**a), None)  # noqa: E731
    for v in (A, A + 2 * 64, A + 2 * 128, A - 2 * 64):
        assert call(k=A, v=v) == BAD, v
    assert call(k=A, k_token=512, v=A + 2 * 64, v_token=512) == BAD


def test_evict():
    lib = cm.load_library()
    call = lambda **a: lib.coli_moe_kv_evict(kv(weights=A), rows(), evi(**a), None)  # noqa: E731
    for a in (dict(new_lengths=B + 4), dict(new_lengths=B - 4), dict(kept=B - 2 * 2 * 8 * 4 + 4), dict(kept=B + 4),
              dict(kept=A + (5 << 20), new_lengths=A + (5 << 20) + 2 * 2 * 8 * 4 - 4)):
        assert call(**a) == BAD, a


def test_sizes_at_their_limits():
    """The longest steps and the most tokens are looked at without overflow."""
    far = dict(tokens=1 << 26, heads=4096, x_token=1 << 40, x_head=1 << 40, out=A + 2, out_token=1 << 40, out_head=64)
    assert rotary_rc(**far) == BAD
    assert rotary_rc(**{**far, "heads": 1, "out_token": (1 << 40) - 64}) == BAD
    assert rotary_rc(**{**far, "heads": 1, "x_token": 0}) == BAD
