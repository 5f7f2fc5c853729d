"""CPU-only checks of the cache operators' host side: refusals before any launch, workspace sizes, the rotary plan.
Pointers here are made-up device addresses: every refused call returns before it would use them."""
import ctypes
import math

import numpy as np
import pytest

import cache_ops_ref as R

P = ctypes.c_void_p
A, B_, C_, D_, E_, F_, G_, H_, I_, J_ = (P(0x10000 * i) for i in range(1, 11))


def shape(**kw):
    from paged_kv_cache_366_b200 import pa
    d = dict(num_heads=32, num_kv_heads=8, head_dim=128, block_size=16, num_blocks=1000, dtype=1)
    d.update(kw)
    return pa.PaShape(**d)


def lib():
    from paged_kv_cache_366_b200 import pa
    return pa.lib


def by(x):
    return ctypes.byref(x)


# ---- the rotary plan


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=8.0), dict(scaling="base", factor=8.0),
                                dict(scaling="parts", factor=8.0, low=1.0, high=4.0, original_len=8192.0),
                                dict(scaling="parts", factor=40.0, original_len=4096.0)])
@pytest.mark.parametrize("rot,base", [(16, 10000.0), (128, 10000.0), (64, 500000.0), (48, 1.0)])
def test_rope_plan_turns(kw, rot, base):
    from paged_kv_cache_366_b200 import pa
    plan = pa.pa_rope_init(rot, base, interleaved=True, mscale=0.5, **kw)
    assert (plan.rot_dim, plan.interleaved, plan.mscale) == (rot, 1, 0.5)
    kw = dict(kw)
    freq = R.frequencies(rot, base, **kw)
    got = np.array([plan.step[i] for i in range(rot // 2)], dtype=np.float64) / 2.0 ** 64
    # the reference's frequencies are within a few roundings of 64-bit floats
    assert np.all(np.abs(got - freq / (2 * math.pi)) <= 2.0 ** -48 * freq + 2.0 ** -64)
    assert all(plan.step[i] == 0 for i in range(rot // 2, 64))


@pytest.mark.parametrize("args,code", [
    ((8, 0, 1e4, 0, 1, 1, 32, 0, 1), -2), ((20, 0, 1e4, 0, 1, 1, 32, 0, 1), -2), ((144, 0, 1e4, 0, 1, 1, 32, 0, 1), -2),
    ((64, 2, 1e4, 0, 1, 1, 32, 0, 1), -1), ((64, 0, 0.5, 0, 1, 1, 32, 0, 1), -1),
    ((64, 0, math.inf, 0, 1, 1, 32, 0, 1), -1), ((64, 0, 1e4, 4, 1, 1, 32, 0, 1), -1),
    ((64, 0, 1e4, 1, 0.5, 1, 32, 0, 1), -1), ((64, 0, 1e4, 1, math.nan, 1, 32, 0, 1), -1),
    ((64, 0, 1e4, 3, 8, 32, 32, 4096, 1), -1), ((64, 0, 1e4, 3, 8, 1, 32, 0, 1), -1),
    ((64, 0, 1e4, 3, 8, -1, 32, 4096, 1), -1), ((64, 0, 1e4, 0, 1, 1, 32, 0, math.nan), -1),
])
def test_rope_plan_refusals(args, code):
    from paged_kv_cache_366_b200 import pa
    plan = pa.PaRopePlan()
    assert lib().pa_rope_init(by(plan), *args) == code
    assert lib().pa_rope_init(None, 64, 0, 1e4, 0, 1.0, 1.0, 32.0, 0.0, 1.0) == -1
    with pytest.raises(ValueError):
        pa.pa_rope_init(64, scaling="other")


def rope_args(**kw):
    from paged_kv_cache_366_b200 import pa
    d = dict(q_out=A, q=B_, k=C_, v=D_, qs=32 * 128, ks=8 * 128, vs=8 * 128, kc=E_, vc=F_, slots=G_, pos=H_, T=3,
             plan=pa.pa_rope_init(128), shape=shape())
    d.update(kw)
    plan = by(d["plan"]) if d["plan"] is not None else None
    return (d["q_out"], d["q"], d["k"], d["v"], d["qs"], d["ks"], d["vs"], d["kc"], d["vc"], d["slots"], d["pos"],
            d["T"], plan, by(d["shape"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q_out=None), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(kc=None), -1),
    (dict(vc=None), -1), (dict(slots=None), -1), (dict(pos=None), -1), (dict(plan=None), -1), (dict(T=-1), -1),
    (dict(T=0, q=None), 0), (dict(qs=32 * 128 - 8), -1), (dict(qs=32 * 128 + 4), -3), (dict(ks=8 * 128 + 1), -3),
    (dict(vs=0), -1), (dict(q=P(0x20008)), -3), (dict(q_out=P(0x10004)), -3), (dict(pos=P(0x20004)), -3),
    (dict(q_out=B_, qs=6144), -1), (dict(shape=shape(head_dim=64), qs=4096), -2), (dict(shape=shape(block_size=32)), -2),
    (dict(shape=shape(kv_fp8=1)), -1), (dict(shape=shape(kv_fp8=2)), -1), (dict(shape=shape(kv_fp8=3)), -1),
    (dict(T=1 << 31), -2),
])
def test_rope_and_cache_refusals(kw, code):
    assert lib().pa_rope_and_cache(*rope_args(**kw)) == code


def test_rope_refusals():
    from paged_kv_cache_366_b200 import pa
    s, plan = shape(), pa.pa_rope_init(64, interleaved=True)
    f = lib().pa_rope
    ok = [A, B_, C_, D_, 4096, 1024, E_, 2, by(plan), by(s), None]

    def but(**at):
        a = list(ok)
        for i, x in at.items():
            a[int(i[1:])] = x
        return f(*a)

    assert but(_7=0) == 0 and but(_7=-1) == -1 and but(_0=None) == -1 and but(_1=None) == -1 and but(_2=None) == -1
    assert but(_3=None) == -1 and but(_6=None) == -1 and but(_8=None) == -1 and but(_4=4095) == -1
    assert but(_4=4100) == -3 and but(_0=P(8)) == -3
    assert but(_2=A, _4=8192) == -1 and but(_3=B_, _5=2048) == -1  # in place, strided
    bad = pa.pa_rope_init(64)
    bad.rot_dim = 24
    assert but(_8=by(bad)) == -1
    bad.rot_dim = 1 << 20
    assert but(_8=by(bad)) == -2


# ---- block8 pools


@pytest.mark.parametrize("i", [0, 1, 2, 3, 4, 5, 6])
def test_write_null_and_misaligned(i):
    s = shape(kv_fp8=2)
    args = [A, B_, C_, D_, E_, F_, G_]
    args[i] = None
    assert lib().pa_cache_block8(*args, 3, by(s), None) == -1
    args[i] = P(0x10002)
    assert lib().pa_cache_block8(*args, 3, by(s), None) == -3


def test_write_refusals():
    f = lib().pa_cache_block8
    args = [A, B_, C_, D_, E_, F_, G_]
    assert f(*args, 0, by(shape(kv_fp8=2)), None) == 0
    assert f(*args, -1, by(shape(kv_fp8=2)), None) == -1
    assert f(*args, 3, by(shape()), None) == -2  # not a block8 pool
    assert f(*args, 3, by(shape(kv_fp8=1, k_scale=1, v_scale=1)), None) == -2
    assert f(*args, 3, by(shape(kv_fp8=3, dtype=0)), None) == -2
    assert f(*args, 3, by(shape(kv_fp8=4)), None) == -1
    assert f(*args, 3, by(shape(kv_fp8=2, head_dim=96)), None) == -2
    assert f(*args, 3, None, None) == -1


def test_plain_calls_refuse_block8_pools():
    """The calls from before take no block8 shape: they would read codes without their scales."""
    l = lib()
    for code in (2, 3):
        s = shape(kv_fp8=code)
        assert l.pa_reshape_and_cache(A, B_, C_, D_, E_, 3, by(s), None) == -1
        assert l.pa_decode(A, B_, C_, D_, E_, 4, F_, 2, 64, 1.0, 0, G_, 1 << 30, by(s), None) == -1
        assert l.pa_decode_workspace_bytes(2, 64, 0, by(s)) == -1
        assert l.pa_prefill_chunk(A, B_, C_, D_, E_, 4, F_, G_, 1, 8, 8, 1.0, by(s), None) == -1


def decode_args(**kw):
    d = dict(out=A, q=B_, k=C_, v=D_, ks=E_, vs=F_, t=G_, mb=4, lens=H_, B=2, top=64, scale=0.1, part=0, ws=I_,
             n=1 << 40, shape=shape(kv_fp8=2))
    d.update(kw)
    return (d["out"], d["q"], d["k"], d["v"], d["ks"], d["vs"], d["t"], d["mb"], d["lens"], d["B"], d["top"],
            d["scale"], d["part"], d["ws"], d["n"], by(d["shape"]), None)


REFUSED = [(dict(out=None), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(ks=None), -1),
           (dict(vs=None), -1), (dict(t=None), -1), (dict(lens=None), -1), (dict(mb=0), -1), (dict(mb=-1), -1),
           (dict(B=-1), -1), (dict(top=-1), -1), (dict(scale=math.nan), -1), (dict(scale=math.inf), -1),
           (dict(part=100), -1), (dict(part=-64), -1), (dict(ws=None), -4), (dict(n=16), -4), (dict(ws=P(0x10008)), -3),
           (dict(q=P(0x10008)), -3), (dict(ks=P(0x10002)), -3), (dict(lens=P(0x10002)), -3), (dict(B=0, q=None), 0),
           (dict(top=(1 << 30) + 1), -2), (dict(mb=(1 << 26) + 1), -2), (dict(mb=(1 << 31) - 1), -2),
           (dict(shape=shape(kv_fp8=2, num_heads=24)), -2), (dict(shape=shape(kv_fp8=3, dtype=0)), -2)]


@pytest.mark.parametrize("kw,code", REFUSED + [(dict(shape=shape()), -2)])
def test_decode_block8_refusals(kw, code):
    assert lib().pa_decode_block8(*decode_args(**kw)) == code


@pytest.mark.parametrize("kw,code", REFUSED + [(dict(w=None), -1), (dict(width=63), -1), (dict(w=P(0x10002)), -3)])
def test_decode_weights_refusals(kw, code):
    kw = dict(kw)
    w, width = kw.pop("w", J_), kw.pop("width", max(64, kw.get("top", 0)))
    a = decode_args(**kw)
    assert lib().pa_decode_weights(a[0], w, width, *a[1:]) == code


def test_workspace_sizes():
    from paged_kv_cache_366_b200 import pa

    def r16(n):
        return (n + 15) // 16 * 16

    b8 = shape(kv_fp8=2)
    for s in (shape(), b8, shape(kv_fp8=1, k_scale=1.0, v_scale=1.0), shape(dtype=0)):
        plain = (pa.pa_decode_block8_workspace_bytes if s is b8 else pa.pa_decode_workspace_bytes)(64, 2041, 0, s)
        # the decode's own, then 64 * 32 rows of 2048 scores, then 64 * 32 sums
        assert pa.pa_decode_weights_workspace_bytes(64, 2041, 0, s) == r16(plain) + 64 * 32 * (2048 + 1) * 4
        assert pa.pa_decode_weights_workspace_bytes(0, 2041, 0, s) == 0
    # past 32 bits
    assert pa.pa_decode_weights_workspace_bytes(256, 1 << 20, 0, b8) > 256 * 32 * (1 << 20) * 4
    with pytest.raises(pa.PaError):
        pa.pa_decode_block8_workspace_bytes(4, 100, 0, shape())
    with pytest.raises(pa.PaError):
        pa.pa_decode_block8_workspace_bytes(4, 100, 100, b8)
    with pytest.raises(pa.PaError):
        pa.pa_decode_weights_workspace_bytes(-1, 100, 0, b8)


# ---- eviction


def evict_args(**kw):
    d = dict(k=A, v=B_, ks=None, vs=None, w=C_, width=64, t=D_, mb=4, lens=E_, dst=F_, db=2, nw=G_, nl=H_, kept=I_, B=2,
             top=64, keep=32, sinks=4, recent=8, shape=shape())
    d.update(kw)
    return (d["k"], d["v"], d["ks"], d["vs"], d["w"], d["width"], d["t"], d["mb"], d["lens"], d["dst"], d["db"],
            d["nw"], d["nl"], d["kept"], d["B"], d["top"], d["keep"], d["sinks"], d["recent"], by(d["shape"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(w=None), -1), (dict(t=None), -1), (dict(lens=None), -1),
    (dict(dst=None), -1), (dict(nw=None), -1), (dict(nl=None), -1), (dict(kept=None), -1), (dict(width=63), -1),
    (dict(mb=0), -1), (dict(db=1), -1), (dict(db=0), -1), (dict(B=-1), -1), (dict(top=-1), -1), (dict(keep=0), -1),
    (dict(sinks=-1), -1), (dict(recent=-1), -1), (dict(sinks=20, recent=13), -1), (dict(nl=E_), -1), (dict(nw=C_), -1),
    (dict(sinks=(1 << 31) - 1, recent=(1 << 31) - 1), -1),
    (dict(shape=shape(kv_fp8=2)), -1), (dict(shape=shape(kv_fp8=3), ks=A), -1), (dict(k=P(0x10008)), -3),
    (dict(kept=P(0x10002)), -3), (dict(shape=shape(kv_fp8=1)), -1), (dict(shape=shape(kv_fp8=9)), -1),
    (dict(B=0, k=None), 0), (dict(shape=shape(head_dim=80)), -2), (dict(keep=(1 << 30) + 1), -2),
    (dict(db=1 << 27), -2), (dict(mb=1 << 27), -2), (dict(top=(1 << 30) + 1, width=(1 << 31) - 1, keep=8, sinks=0), -2),
])
def test_evict_refusals(kw, code):
    assert lib().pa_evict(*evict_args(**kw)) == code


# ---- the Python binding's own checks


def test_binding_refusals():
    """Wrong devices, types and shapes are ValueErrors before the library is called (CPU tensors here)."""
    import torch
    from paged_kv_cache_366_b200 import pa
    bf, i32, i64 = torch.bfloat16, torch.int32, torch.int64
    q, kv = torch.zeros(2, 8, 64, dtype=bf), torch.zeros(2, 2, 64, dtype=bf)
    pool, codes, scales = torch.zeros(4, 16, 2, 64, dtype=bf), torch.zeros(4, 16, 2, 64, dtype=torch.int8), torch.ones(4, 2)
    n64, tables, lens, w = torch.zeros(2, dtype=i64), torch.zeros(2, 3, dtype=i32), torch.ones(2, dtype=i32), torch.zeros(2, 2, 48)
    kept, plan = torch.zeros(2, 2, 8, dtype=i32), pa.pa_rope_init(64)
    calls = {
        "rope": (pa.pa_rope, [q, kv, q, kv, n64, plan]),
        "rope_and_cache": (pa.pa_rope_and_cache, [q, q, kv, kv, pool, pool, n64, n64, plan]),
        "write": (pa.pa_cache_block8, [kv, kv, codes, codes, scales, scales, n64]),
        "decode": (pa.pa_decode_block8, [q, q, codes, codes, scales, scales, tables, lens, 48, 0.1]),
        "weights": (pa.pa_decode_weights, [q, w, q, pool, pool, tables, lens, 48, 0.1]),
        "evict": (pa.pa_evict, [pool, pool, w, tables, lens, tables, w, lens, kept, 0, 0, 48]),
    }
    for name, (fn, args) in calls.items():
        with pytest.raises(ValueError, match="CUDA device"):
            fn(*args)  # everything right but the device
    wrong = {
        "rope": {0: q[:, :4], 1: kv.float(), 3: kv[:1], 4: n64.int()},
        "rope_and_cache": {1: q.float(), 2: kv[:, :1], 4: pool[..., :32], 5: pool[:2], 6: n64[:1], 7: n64.int()},
        "write": {0: kv.float(), 1: kv[:1], 2: codes.float(), 3: codes[:2], 4: scales.double(), 5: scales[:2], 6: n64.int()},
        "decode": {0: q[:1], 1: q.float(), 2: pool, 4: scales[:, :1], 6: tables.long(), 7: lens[:1]},
        "weights": {0: q.float(), 1: w[:, :1], 2: q[..., :32], 3: pool.float(), 4: pool[:1], 5: tables[0], 6: lens.long()},
        "evict": {1: pool[:2], 2: w.double(), 3: tables[:1], 5: tables.long(), 6: w[..., :40], 8: kept[:, :1]},
    }
    for name, changes in wrong.items():
        fn, args = calls[name]
        for i, bad in changes.items():
            with pytest.raises(ValueError) as e:
                fn(*(bad if j == i else a for j, a in enumerate(args)))
            assert "CUDA device" not in str(e.value), (name, i)
    with pytest.raises(ValueError, match="both"):
        pa.pa_decode_weights(*calls["weights"][1], k_scales=scales)
    with pytest.raises(ValueError):
        pa.shape_of_block8(pool, 8)
    a, b = pa.shape_of_block8(codes, 8), pa.shape_of_block8(codes, 8)
    a.num_heads = 2
    assert b.num_heads == 8  # each caller has its own


# ---- the reference's own pieces


def test_reference_codes():
    import torch
    x = torch.cat([torch.randn(4000) * 2.0 ** e for e in range(-12, 8)])
    got = R.encode(x.double().numpy(), "e4m3")
    ref = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got, ref)
    codes = np.arange(256, dtype=np.uint8)
    back = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.values(codes, "e4m3"), back, equal_nan=True)
    assert R.least_scale(np.array([448.0]), "e4m3") == 1.0 and R.least_scale(np.array([448.1]), "e4m3") == 2.0
    assert R.least_scale(np.array([127.0]), "int8") == 1.0 and R.least_scale(np.array([63.5]), "int8") == 0.5
    assert R.least_scale(np.zeros(3), "int8") == 2.0 ** -64
