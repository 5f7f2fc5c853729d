"""CPU-only checks of the cache operators' largest sizes: what is too large is refused before any launch, and alike by a
call and by the function that sizes its workspace. Pointers are made up; every refused call returns before it would use
them."""
import pytest

from test_cache_ops_host import by, decode_args, evict_args, lib, shape
from test_cache_ops_host import J_ as WEIGHTS

UNSUPPORTED = -2
TOO_MANY = [  # sequences, longest context: too many (sequence, KV head) pairs, or too many pieces of weights
    ((1 << 28), 1, shape(kv_fp8=2)), ((1 << 31) - 1, 1 << 30, shape()), ((1 << 31) - 1, 16, shape(kv_fp8=3)),
    ((1 << 28), 1 << 30, shape(kv_fp8=2)),
]
TOO_MANY_PIECES = [((1 << 27), 1 << 30, shape()), ((1 << 27), 16385, shape(kv_fp8=2)), ((1 << 20), 1 << 20, shape())]


@pytest.mark.parametrize("B,top,s", TOO_MANY)
def test_too_many_sequences(B, top, s):
    if s.kv_fp8:
        assert lib().pa_decode_block8_workspace_bytes(B, top, 0, by(s)) == UNSUPPORTED
        assert lib().pa_decode_block8(*decode_args(B=B, top=top, shape=s, n=1 << 62)) == UNSUPPORTED
    _weights_refused(B, top, s)


@pytest.mark.parametrize("B,top,s", TOO_MANY_PIECES)
def test_too_many_weights(B, top, s):
    _weights_refused(B, top, s)


def _weights_refused(B, top, s):
    assert lib().pa_decode_weights_workspace_bytes(B, top, 0, by(s)) == UNSUPPORTED
    for n in (16, 1 << 62):  # not for its workspace
        a = decode_args(B=B, top=top, shape=s, n=n)
        assert lib().pa_decode_weights(a[0], WEIGHTS, 1 << 30, *a[1:]) == UNSUPPORTED


def test_largest_sizes_have_a_workspace():
    # just inside: 2^31 - 8 pairs of one short context, 2^30 pairs of one piece each
    for B, top in (((1 << 28) - 1, 16), (1 << 27, 1024)):
        for s in (shape(), shape(kv_fp8=2)):
            n = lib().pa_decode_weights_workspace_bytes(B, top, 0, by(s))
            assert n > B * 32 * top * 4  # the scores alone
    assert lib().pa_decode_block8_workspace_bytes((1 << 28) - 1, 1 << 30, 0, by(shape(kv_fp8=2))) > 0


@pytest.mark.parametrize("kw", [
    dict(B=1 << 15, db=(1 << 16) + 1, top=16, keep=16), dict(B=1 << 28, db=8, top=16, keep=16),
    dict(B=1 << 26, top=1 << 20, width=1 << 20, keep=16, db=1),
    dict(B=1, shape=shape(num_heads=262141, num_kv_heads=262141)),
])
def test_evict_refuses_before_its_first_launch(kw):
    # Without a GPU the first launch gives another error.
    assert lib().pa_evict(*evict_args(**dict(dict(sinks=0, recent=0), **kw))) == UNSUPPORTED


@pytest.mark.parametrize("mscale", [1e39, -1e39, 3.4028236e38])
def test_rope_plan_refuses_a_factor_past_fp32(mscale):
    # the plan holds it in fp32, and the rotary calls refuse an infinite one
    from paged_kv_cache_366_b200 import pa
    plan = pa.PaRopePlan()
    assert lib().pa_rope_init(by(plan), 64, 0, 1e4, 0, 1.0, 1.0, 32.0, 0.0, mscale) == -1
    assert lib().pa_rope_init(by(plan), 64, 0, 1e4, 0, 1.0, 1.0, 32.0, 0.0, 3.4e38) == 0
