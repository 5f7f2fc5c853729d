"""GPU checks of the rotary calls against the 64-bit definition: layouts, partial heads, scaled frequencies, far
positions, strided projections, padding slots and every pool type."""
import numpy as np
import pytest
import torch

import cache_ops_ref as R

pytestmark = pytest.mark.gpu

SCALINGS = {
    "none": {},
    "linear": dict(scaling="linear", factor=4.0),
    "base": dict(scaling="base", factor=8.0),
    "parts": dict(scaling="parts", factor=8.0, low=1.0, high=4.0, original_len=8192.0),
}


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_366_b200 import pa as _pa
    assert _pa.pa_get_status() == 0
    return _pa


def _positions(rng, T, far):
    p = rng.integers(0, far, T)
    p[:min(T, 4)] = [0, far - 1, 1, far // 2][:min(T, 4)]
    return p


def _near(got, x, pos, rot, inter, freq, mscale, half_step):
    """|got - exact| <= half a step of the result, and the angle's and the products' fp32 error: the turn is
    rounded to 2^-33 and then to fp32 (2^-25 of a half turn), cos and sin to 2 ulp, the products once each."""
    ref = R.rotate(x, pos, rot, inter, freq, mscale)
    size = np.zeros_like(x)  # |x| + |y| of each rotated pair
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    size[..., i] = size[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    angle = 2 * np.pi * 2.0 ** -33 + np.pi * 2.0 ** -25
    tol = abs(mscale) * size * (angle + 2 * 2.0 ** -23 + 3 * 2.0 ** -24) + half_step * np.abs(ref) * (1 + 2.0 ** -20)
    bad = np.abs(got - ref) - tol
    assert np.all(bad <= 0), float(bad.max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("scaling", sorted(SCALINGS))
@pytest.mark.parametrize("H,Hk,D,rot,T", [(32, 8, 128, 128, 5), (16, 2, 64, 16, 33), (8, 8, 128, 48, 1),
                                          (64, 8, 128, 64, 300), (4, 1, 64, 64, 7)])
def test_rotation(pa, dtype, inter, scaling, H, Hk, D, rot, T):
    rng = np.random.default_rng([H, Hk, rot, T])
    pos = _positions(rng, T, 1 << 21)
    mscale = 1.25 if scaling == "parts" else 1.0
    plan = pa.pa_rope_init(rot, 500000.0, interleaved=inter, mscale=mscale, **SCALINGS[scaling])
    qkv = torch.from_numpy(rng.standard_normal((T, (H + Hk) * D + 16))).to("cuda", dtype)
    q = qkv[:, :H * D].unflatten(1, (H, D))
    k = qkv[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D))
    q_out, k_out = torch.full((T, H, D), float("nan"), dtype=dtype, device="cuda"), torch.empty(T, Hk, D, dtype=dtype, device="cuda")
    before = qkv.clone()
    pa.pa_rope(q_out, k_out, q, k, torch.from_numpy(pos).cuda(), plan)
    assert pa.pa_get_status() == 0 and torch.equal(qkv, before)
    freq = R.frequencies(rot, 500000.0, **SCALINGS[scaling])
    half = torch.finfo(dtype).eps / 2
    for x, y in ((q, q_out), (k, k_out)):
        _near(y.double().cpu().numpy(), x.double().cpu().numpy(), pos, rot, inter, freq, mscale, half)
        assert torch.equal(y[..., rot:], x[..., rot:])  # the rest of the head passes through


def test_rotation_in_place_is_the_same(pa):
    T, H, Hk, D = 19, 16, 4, 128
    q, k = (torch.randn(T, h, D, device="cuda", dtype=torch.bfloat16) for h in (H, Hk))
    pos = torch.arange(T, device="cuda") * 977
    plan = pa.pa_rope_init(D)
    q2, k2 = torch.empty_like(q), torch.empty_like(k)
    pa.pa_rope(q2, k2, q, k, pos, plan)
    pa.pa_rope(q, k, q, k, pos, plan)
    assert torch.equal(q, q2) and torch.equal(k, k2)


def test_rotation_turns_back(pa):
    # position p and then -p: the identity, up to two roundings to fp32 of numbers up to |x| + |y|
    T, H, D = 9, 4, 64
    q = torch.randn(T, H, D, device="cuda")
    pos = torch.arange(T, device="cuda") * 12345
    plan = pa.pa_rope_init(D)
    a, b = torch.empty_like(q), torch.empty_like(q)
    pa.pa_rope(a, b, q, q, pos, plan)
    pa.pa_rope(a, b, a, a.clone(), -pos, plan)
    size = q.abs() + q.abs().roll(D // 2, -1)
    assert bool(((a - q).abs() <= size * 2 * (2.0 ** -22 + np.pi * 2.0 ** -25 + 3 * 2.0 ** -24) * 1.5).all())


@pytest.mark.parametrize("cache", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("H,Hk,D,rot,T", [(32, 8, 128, 128, 64), (16, 2, 64, 32, 1), (8, 8, 128, 16, 200), (32, 8, 128, 64, 2),
                                          (64, 8, 64, 64, 3)])
def test_rotate_and_cache(pa, cache, H, Hk, D, rot, T):
    rng = np.random.default_rng([3, H, D, T])
    dt = torch.float32 if cache == "f32" else torch.bfloat16
    ks, vs = (0.03125, 1.0 / 48) if cache == "fp8" else (0.0, 0.0)
    nb = R.blocks(T) + 3
    qkv = torch.from_numpy(rng.standard_normal((T, (H + 2 * Hk) * D))).to("cuda", dt)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([H * D, Hk * D, Hk * D], 1))
    slots = rng.permutation(nb * 16)[:T]
    slots[T // 2] = -1  # padding
    pos = _positions(rng, T, 1 << 17)
    kc = torch.randint(0, 120, (nb, 16, Hk, D), device="cuda").to(torch.uint8) if cache == "fp8" else torch.randn(nb, 16, Hk, D, device="cuda").to(dt)
    vc = kc.flip(0).contiguous()
    kc0, vc0 = kc.clone(), vc.clone()
    q_out = torch.empty(T, H, D, device="cuda", dtype=dt)
    plan = pa.pa_rope_init(rot, interleaved=True)
    pa.pa_rope_and_cache(q_out, q, k, v, kc, vc, torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda(), plan,
                         k_scale=ks, v_scale=vs)
    assert pa.pa_get_status() == 0
    freq = R.frequencies(rot)
    _near(q_out.double().cpu().numpy(), q.double().cpu().numpy(), pos, rot, True, freq, 1.0, torch.finfo(dt).eps / 2)
    live = np.flatnonzero(slots >= 0)
    rows = torch.from_numpy(slots[live]).cuda()
    new_k, new_v = kc.flatten(0, 1)[rows], vc.flatten(0, 1)[rows]
    x = k.double().cpu().numpy()[live]
    if cache == "fp8":
        ref = R.rotate(x, pos[live], rot, True, freq, 1.0) / ks
        got = new_k.view(torch.float8_e4m3fn).double().cpu().numpy()
        # half a step of E4M3 (2^-4 of the value, 2^-10 below its normal numbers), and fp32 before it
        assert np.all(np.abs(got - ref) <= 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 + 2.0 ** -18 * np.abs(x).max(initial=0) / ks)
        code_v = (v.float()[torch.from_numpy(live).cuda()] * float(np.float32(1) / np.float32(vs))).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(new_v, code_v.view(torch.uint8))
    else:
        _near(new_k.double().cpu().numpy(), x, pos[live], rot, True, freq, 1.0, torch.finfo(dt).eps / 2)
        assert torch.equal(new_v, v[torch.from_numpy(live).cuda()])
    # nothing else changed
    kc.flatten(0, 1)[rows] = kc0.flatten(0, 1)[rows]
    vc.flatten(0, 1)[rows] = vc0.flatten(0, 1)[rows]
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)


def test_bad_slot_is_flagged_and_skipped(pa):
    T, H, Hk, D = 3, 4, 4, 64
    q, k, v = (torch.randn(T, h, D, device="cuda", dtype=torch.bfloat16) for h in (H, Hk, Hk))
    kc, vc = (torch.zeros(2, 16, Hk, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q_out = torch.empty_like(q)
    slots = torch.tensor([0, 32, 31], device="cuda")
    pa.pa_rope_and_cache(q_out, q, k, v, kc, vc, slots, torch.zeros(T, dtype=torch.int64, device="cuda"),
                         pa.pa_rope_init(16))
    assert pa.pa_get_status() == pa.PA_STATUS_BAD_SLOT
    assert torch.equal(q_out, q)  # position 0 turns nothing
    assert torch.equal(kc.flatten(0, 1)[0], k[0]) and torch.equal(kc.flatten(0, 1)[31], k[2])
    assert int(kc.count_nonzero()) <= 2 * Hk * D


def test_rotate_write_then_decode_in_a_graph(pa):
    """A captured rotate-write-decode step, replayed on new inputs, gives the eager calls' outputs."""
    B, H, Hk, D, nb = 3, 32, 8, 128, 12
    dt = torch.bfloat16
    kc, vc = (torch.randn(nb, 16, Hk, D, device="cuda").to(dt) for _ in range(2))
    tables = torch.arange(nb, device="cuda", dtype=torch.int32).view(B, 4)
    lens = torch.tensor([17, 1, 50], dtype=torch.int32, device="cuda")
    pos = (lens - 1).long()
    slots = tables.long().gather(1, (pos // 16)[:, None])[:, 0] * 16 + pos % 16
    qkv = torch.randn(B, (H + 2 * Hk) * D, device="cuda").to(dt)
    plan = pa.pa_rope_init(D)
    n = pa.pa_decode_workspace_bytes(B, 64, 0, pa.shape_of(kc, H))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def step(qkv, kc, vc):
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([H * D, Hk * D, Hk * D], 1))
        q_out = torch.empty(B, H, D, device="cuda", dtype=dt)
        out = torch.empty_like(q_out)
        pa.pa_rope_and_cache(q_out, q, k, v, kc, vc, slots, pos, plan)
        pa.pa_decode(out, q_out, kc, vc, tables, lens, 64, 0.1, 0, ws)
        return out

    stream = torch.cuda.Stream()
    kg, vg, xg = kc.clone(), vc.clone(), qkv.clone()
    with torch.cuda.stream(stream):
        step(xg, kg, vg)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out_g = step(xg, kg, vg)
    for seed in range(2):
        new = torch.randn_like(qkv) + seed
        with torch.cuda.stream(stream):
            xg.copy_(new)
            graph.replay()
        stream.synchronize()
        out = step(new, kc, vc)
        torch.cuda.synchronize()
        assert torch.equal(out, out_g) and torch.equal(kc, kg) and torch.equal(vc, vg)
    assert pa.pa_get_status() == 0


def test_rotate_many_tokens(pa):
    # enough tokens for four to a CTA, the last CTA not full; every row against the one-token calls
    T, H, Hk, D = 16 * 148 + 3, 8, 1, 64
    q, k = (torch.randn(T, h, D, device="cuda", dtype=torch.bfloat16) for h in (H, Hk))
    pos = torch.randint(0, 1 << 20, (T,), device="cuda")
    plan = pa.pa_rope_init(32, interleaved=True)
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    pa.pa_rope(q_out, k_out, q, k, pos, plan)
    a, b = torch.empty_like(q), torch.empty_like(k)
    for lo in range(0, T, 500):
        s = slice(lo, lo + 500)
        pa.pa_rope(a[s], b[s], q[s], k[s], pos[s], plan)
    assert torch.equal(a, q_out) and torch.equal(b, k_out)
    _near(q_out.double().cpu().numpy(), q.double().cpu().numpy(), pos.cpu().numpy(), 32, True, R.frequencies(32), 1.0, 2.0 ** -8)


def test_rotate_and_cache_past_32_bits(pa):
    # a pool of 4.6 GB: slots whose byte offsets need more than 32 bits
    NB, H, Hk, D, T = 140000, 8, 8, 128, 3
    kc, vc = (torch.zeros(NB, 16, Hk, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, k, v = (torch.randn(T, H, D, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    slots = torch.tensor([NB * 16 - 1, 0, 2200000], device="cuda")
    q_out = torch.empty_like(q)
    pos = torch.tensor([5, (1 << 31) - 1, 0], device="cuda")
    pa.pa_rope_and_cache(q_out, q, k, v, kc, vc, slots, pos, pa.pa_rope_init(D))
    assert pa.pa_get_status() == 0
    assert torch.equal(vc.flatten(0, 1)[slots], v) and int(vc.count_nonzero()) == int(v.count_nonzero())
    _near(kc.flatten(0, 1)[slots].double().cpu().numpy(), k.double().cpu().numpy(), pos.cpu().numpy(), D, False, R.frequencies(D), 1.0, 2.0 ** -8)
