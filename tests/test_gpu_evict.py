"""GPU checks of weight-counting decode and of eviction against their 64-bit definitions, over every pool type,
and of a run of them together."""
import numpy as np
import pytest
import torch

import cache_ops_ref as R
from test_gpu_block8 import bf16, bounds, dev, make_pool, poison, tables_of

pytestmark = pytest.mark.gpu

K_SCALE, V_SCALE = 0.03125, 1.0 / 48
POOLS = ["bf16", "f32", "fp8", "e4m3", "int8"]


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_366_b200 import pa as _pa
    assert _pa.pa_get_status() == 0
    return _pa


def host(t):
    """A device tensor's bits on the host (bf16 as int16)."""
    return (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).cpu().numpy()


class Pool:
    """K and V of one type on the device, and their values in 64 bits."""

    def __init__(self, rng, kind, nb, Hk, D, t, lens):
        self.kind, self.kw, self.one = kind, {}, {}
        self.dtype = torch.float32 if kind == "f32" else torch.bfloat16
        parts = []
        for one in (K_SCALE, V_SCALE):
            if kind in R.CODE_MAX:
                c, s = make_pool(rng, nb, Hk, D, kind, 1.0)
                poison(c, s, t, lens, kind)
                parts.append((dev(c), dev(s), R.dequantized(c, s, kind)))
            elif kind == "fp8":
                c = R.encode(rng.standard_normal((nb, 16, Hk, D)) / one, "e4m3")
                s = np.ones((nb, Hk), np.float32)
                poison(c, s, t, lens, "e4m3")
                parts.append((dev(c), None, R.values(c, "e4m3") * one))
            else:
                x = torch.from_numpy(rng.standard_normal((nb, 16, Hk, D))).to(self.dtype)
                parts.append((x.cuda(), None, x.double().numpy()))
        (self.k, ks, self.k64), (self.v, vs, self.v64) = parts
        if ks is not None:
            self.kw = dict(k_scales=ks, v_scales=vs)
        if kind == "fp8":
            self.one = dict(k_scale=K_SCALE, v_scale=V_SCALE)

    def shape(self, pa, H):
        if self.kw:
            return pa.shape_of_block8(self.k, H)
        return pa.shape_of(self.k, H, K_SCALE, V_SCALE)


def count(pa, pool, q, weights, t, lens, scale, part=0, top=None):
    top = max(lens) if top is None else top
    n = pa.pa_decode_weights_workspace_bytes(len(lens), top, part, pool.shape(pa, q.shape[1]))
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=pool.dtype, device="cuda")
    pa.pa_decode_weights(out, weights, q, pool.k, pool.v, dev(t), dev(np.asarray(lens, np.int32)), top, scale, part,
                         ws, **pool.kw, **pool.one)
    return out


def check_count(pa, rng, kind, lens, H, Hk, D, part=0, steps=1):
    nb, t = tables_of(rng, lens)
    pool = Pool(rng, kind, nb, Hk, D, t, lens)
    width = max(lens) + 5
    w0 = rng.random((len(lens), Hk, width)).astype(np.float32)
    weights = dev(w0)
    ref = w0.astype(np.float64)
    tol = np.zeros_like(ref)
    scale = 1 / np.sqrt(D)
    for _ in range(steps):
        q = torch.from_numpy(rng.standard_normal((len(lens), H, D)) * 2).to(pool.dtype)
        out = count(pa, pool, q.cuda(), weights, t, lens, scale, part)
        assert pa.pa_get_status() == 0
        att = R.attend(q.double().numpy(), pool.k64, pool.v64, t, lens, scale, host(pool.kw["v_scales"]) if pool.kw else None)
        got, o_ref = out.double().cpu().numpy(), np.stack([a[0] for a in att])
        assert np.all(np.abs(got - o_ref) <= bounds(att, torch.finfo(pool.dtype).eps / 2))
        for b, n in enumerate(lens):
            p = att[b][1].reshape(Hk, H // Hk, n)
            s = att[b][3].reshape(Hk, H // Hk, 1)
            ref[b, :, :n] += p.sum(1)
            # each p: scores in fp32 (2^-17 of their size, in p and in the sum) and the exponential; then fp32 sums
            tol[b, :, :n] += (p * (2 * 2.0 ** -17 * s + 2.0 ** -20)).sum(1) + (H // Hk + 1) * 2.0 ** -24 * ref[b, :, :n]
    got = weights.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= tol + 1e-37), float(np.abs(got - ref).max())
    for b, n in enumerate(lens):  # entries past the context are left alone
        assert np.array_equal(got[b, :, n:], w0.astype(np.float64)[b, :, n:])


@pytest.mark.parametrize("kind", POOLS)
@pytest.mark.parametrize("H,Hk,D", [(32, 8, 128), (16, 2, 64), (8, 8, 128), (16, 8, 64), (4, 1, 128)])
def test_counting_ragged(pa, kind, H, Hk, D):
    rng = np.random.default_rng([H, Hk, D])
    check_count(pa, rng, kind, [1, 15, 0, 16, 17, 64, 65, 200, 1031], H, Hk, D)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_counting_cut_units_and_several_steps(pa, kind):
    check_count(pa, np.random.default_rng(41), kind, [5000, 3, 700], 8, 2, 128, steps=3)
    check_count(pa, np.random.default_rng(42), kind, [700, 16], 32, 8, 128, part=64)


def test_counting_gives_decodes_output(pa):
    # bit for bit over block8 pools; the plain pools' decode cuts short lists differently, so there each of the two
    # is within its bound of the exact output
    rng = np.random.default_rng(43)
    lens = [400, 17, 1]
    nb, t = tables_of(rng, lens)
    for kind in POOLS:
        pool = Pool(rng, kind, nb, 8, 128, t, lens)
        q = torch.randn(3, 32, 128, device="cuda").to(pool.dtype)
        out = count(pa, pool, q, torch.zeros(3, 8, 400, device="cuda"), t, lens, 0.1)
        ref = torch.empty_like(out)
        args = (dev(t), dev(np.asarray(lens, np.int32)), 400, 0.1, 0, torch.empty(1 << 24, dtype=torch.uint8, device="cuda"))
        if pool.kw:
            pa.pa_decode_block8(ref, q, pool.k, pool.v, pool.kw["k_scales"], pool.kw["v_scales"], *args)
        else:
            pa.pa_decode(ref, q, pool.k, pool.v, *args, **pool.one)
        if pool.kw:
            assert torch.equal(out, ref), kind
        else:
            att = R.attend(q.double().cpu().numpy(), pool.k64, pool.v64, t, lens, 0.1)
            tol = bounds(att, torch.finfo(pool.dtype).eps / 2)
            assert np.all(np.abs((out.double() - ref.double()).cpu().numpy()) <= 2 * tol), kind


# ---- eviction


def evicted(pool, scales, kind, t, dst, lens, kept):
    """A pool and its scales (host copies) with the kept entries' rows in the new blocks."""
    pool, new = pool, pool.copy()
    new_s = None if scales is None else scales.copy()
    for b, n in enumerate(lens):
        for h in range(pool.shape[2]):
            idx = kept[b][h]
            rows = pool[t[b, idx // 16], idx % 16, h]
            for j in range(R.blocks(len(idx))):
                r = rows[16 * j:16 * j + 16]
                if scales is not None:
                    x = R.values(r, kind) * scales[t[b, idx // 16], h].astype(np.float64)[16 * j:16 * j + 16, None]
                    new_s[dst[b, j], h] = R.least_scale(x, kind)
                    r = R.encode(x / float(new_s[dst[b, j], h]), kind)
                new[dst[b, j], :len(r), h] = r
    return new, new_s


def check_evict(pa, rng, kind, lens, Hk, D, keep, sinks, recent, weights=None, top=None):
    B = len(lens)
    nb0, t = tables_of(rng, lens)
    top = max(lens) if top is None else top
    per = max(1, R.blocks(min(keep, top)))
    nb = nb0 + per * B
    dst = (nb0 + rng.permutation(per * B)).astype(np.int32).reshape(B, per)
    pool = Pool(rng, kind, nb, Hk, D, t, lens)
    if weights is None:
        weights = np.exp2(rng.standard_normal((B, Hk, top + 3)) * 4).astype(np.float32)
    new_w = torch.full((B, Hk, per * 16), float("nan"), device="cuda")
    kept = torch.full((B, Hk, keep), -7, dtype=torch.int32, device="cuda")
    new_lens = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    before = [host(x) for x in (pool.k, pool.v)]
    scales = [host(pool.kw[n]) for n in ("k_scales", "v_scales")] if pool.kw else [None, None]
    pa.pa_evict(pool.k, pool.v, dev(weights), dev(t), dev(np.asarray(lens, np.int32)), dev(dst), new_w, new_lens,
                kept, sinks, recent, top, **pool.kw)
    assert pa.pa_get_status() == 0
    want = [[R.select(weights[b, h], n, keep, sinks, recent) for h in range(Hk)] for b, n in enumerate(lens)]
    want_kept = np.full((B, Hk, keep), -1)
    want_w = np.zeros((B, Hk, per * 16), np.float32)
    for b in range(B):
        for h in range(Hk):
            idx = want[b][h]
            want_kept[b, h, :len(idx)] = idx
            want_w[b, h, :len(idx)] = weights[b, h, idx]
    assert np.array_equal(host(new_lens), [min(n, keep) for n in lens])
    assert np.array_equal(host(kept), want_kept)
    assert np.array_equal(host(new_w), want_w, equal_nan=True)
    for x, name, old, s in zip((pool.k, pool.v), ("k_scales", "v_scales"), before, scales):
        new, new_s = evicted(old, s, kind, t, dst, lens, want)
        assert np.array_equal(host(x), new)
        if s is not None:
            assert np.array_equal(host(pool.kw[name]), new_s, equal_nan=True)


@pytest.mark.parametrize("kind", POOLS)
@pytest.mark.parametrize("Hk,D", [(8, 128), (2, 64), (1, 128), (3, 64)])
@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (1, 0, 1), (16, 4, 8), (33, 0, 0), (100, 4, 50), (5000, 2, 2)])
def test_evict_ragged(pa, kind, Hk, D, keep, sinks, recent):
    rng = np.random.default_rng([Hk, D, keep])
    check_evict(pa, rng, kind, [1, 15, 0, 16, 17, 33, 34, 101, 300], Hk, D, keep, sinks, recent)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_evict_long(pa, kind):
    # rows of a cluster of CTAs, short ones beside them
    check_evict(pa, np.random.default_rng(51), kind, [20000, 9, 5000], 2, 64, 4097, 4, 1000)
    check_evict(pa, np.random.default_rng(52), kind, [60000, 1000], 1, 64, 777, 0, 10)


def test_evict_row_too_long_for_shared_memory(pa):
    # 430000 keys over eight CTAs: more than they hold, so each pass reads the weights again
    check_evict(pa, np.random.default_rng(59), "fp8", [430000, 70], 1, 64, 100001, 4, 5000)


def test_evict_ties_and_odd_weights(pa):
    rng = np.random.default_rng(53)
    for fill in (0.0, 1.0, float("nan"), float("inf"), float("-inf")):
        check_evict(pa, rng, "bf16", [200, 50], 2, 64, 40, 3, 5, np.full((2, 2, 200), fill, np.float32))
    w = rng.integers(0, 3, (2, 2, 900)).astype(np.float32)  # many equal weights, cut among them
    check_evict(pa, rng, "bf16", [900, 333], 2, 64, 250, 0, 0, w)
    w = rng.standard_normal((2, 2, 900)).astype(np.float32)
    w[rng.random(w.shape) < 0.3] = np.nan
    w[rng.random(w.shape) < 0.1] = -0.0
    w[rng.random(w.shape) < 0.1] = 0.0
    w[rng.random(w.shape) < 0.05] = np.inf
    w[rng.random(w.shape) < 0.05] = -np.inf
    w[rng.random(w.shape) < 0.05] = 1e-42
    check_evict(pa, rng, "bf16", [900, 777], 2, 64, 400, 10, 20, w)


def test_evict_loose_bound(pa):
    # a host bound far above the lengths, and a table wider than what is left needs
    check_evict(pa, np.random.default_rng(54), "e4m3", [100, 20], 2, 128, 64, 4, 16, top=4000)


def test_evict_bad_blocks_are_flagged(pa):
    rng = np.random.default_rng(55)
    lens = [64, 64]
    nb0, t = tables_of(rng, lens)
    dst = np.array([[nb0, nb0 + 1], [nb0 + 2, nb0 + 9]], np.int32)  # the last is outside the pool
    t[0, 2] = -3
    pool = Pool(rng, "bf16", nb0 + 4, 2, 64, t[1:], lens[1:])
    before = host(pool.k)
    w = torch.rand(2, 2, 64, device="cuda")
    new_w, kept = torch.empty(2, 2, 32, device="cuda"), torch.empty(2, 2, 32, dtype=torch.int32, device="cuda")
    new_lens = torch.empty(2, dtype=torch.int32, device="cuda")
    pa.pa_evict(pool.k, pool.v, w, dev(t), dev(np.asarray(lens, np.int32)), dev(dst), new_w, new_lens, kept, 0, 0, 64)
    assert pa.pa_get_status() == pa.PA_STATUS_BAD_BLOCK_ID
    assert np.array_equal(host(pool.k)[:nb0], before[:nb0])  # nothing but new blocks was written
    pa.pa_evict(pool.k, pool.v, w[:1], dev(t[1:]), dev(np.asarray([70], np.int32)), dev(dst[:1]), new_w[:1], new_lens[:1],
                kept[:1], 0, 0, 64)
    assert pa.pa_get_status() == pa.PA_STATUS_BAD_CONTEXT


def test_evict_again_and_shared_prefix(pa):
    """Two sequences that share a prefix are evicted; the shared blocks stay, and a second eviction of what is left
    keeps what a direct one would."""
    rng = np.random.default_rng(56)
    Hk, D, nb = 2, 64, 40
    t = np.array([[0, 1, 2, 3], [0, 1, 4, 5]], np.int32)
    lens = [64, 60]
    pool = Pool(rng, "bf16", nb, Hk, D, t, lens)
    before = host(pool.k)
    w = dev(rng.random((2, Hk, 64)).astype(np.float32))
    args = dict(sinks=2, recent=8)

    def evict(weights, tables, lengths, dst, keep, top):
        new_w = torch.empty(2, Hk, dst.shape[1] * 16, device="cuda")
        kept = torch.empty(2, Hk, keep, dtype=torch.int32, device="cuda")
        new_lens = torch.empty(2, dtype=torch.int32, device="cuda")
        pa.pa_evict(pool.k, pool.v, weights, tables, lengths, dst, new_w, new_lens, kept, max_context_len=top, **args)
        return new_w, new_lens, kept

    d1, d2, d3 = (torch.arange(a, a + 2 * n, dtype=torch.int32, device="cuda").view(2, n) for a, n in ((6, 3), (12, 2), (16, 2)))
    w1, l1, k1 = evict(w, dev(t), dev(np.asarray(lens, np.int32)), d1, 40, 64)
    w2, l2, k2 = evict(w1, d1, l1, d2, 24, 40)
    w3, l3, k3 = evict(w, dev(t), dev(np.asarray(lens, np.int32)), d3, 24, 64)
    assert pa.pa_get_status() == 0
    assert np.array_equal(host(pool.k)[:6], before[:6])
    # the 24 best are among the 40 best, and age order is kept
    assert torch.equal(torch.gather(k1, 2, k2.long()), k3) and torch.equal(w2, w3) and torch.equal(l2, l3)
    assert torch.equal(pool.k[d2.long()].flatten(1, 2)[:, :24], pool.k[d3.long()].flatten(1, 2)[:, :24])


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_rotate_write_count_evict_run(pa, kind):
    """The calls as a server uses them: rotate, write, decode with counting, evict, and go on from the new blocks;
    after each decode the output equals plain decode over a pool of the same entries."""
    rng = np.random.default_rng(57)
    B, H, Hk, D, nb = 2, 16, 4, 128, 64
    start = [70, 33]
    tables = torch.arange(2 * 8, dtype=torch.int32, device="cuda").view(2, 8)
    free = 16
    block8 = kind == "int8"
    k, v = (torch.zeros(nb, 16, Hk, D, dtype=torch.int8 if block8 else torch.bfloat16, device="cuda") for _ in range(2))
    sc = [torch.zeros(nb, Hk, device="cuda") for _ in range(2)] if block8 else []
    kw = dict(k_scales=sc[0], v_scales=sc[1]) if block8 else {}
    shape = pa.shape_of_block8(k, H) if block8 else pa.shape_of(k, H)
    plan = pa.pa_rope_init(D, scaling="parts", factor=4.0, original_len=64.0)
    ws = torch.empty(pa.pa_decode_weights_workspace_bytes(B, 128, 0, shape), dtype=torch.uint8, device="cuda")
    weights = torch.zeros(B, Hk, 128, device="cuda")

    def append(pos, entry, seqs):
        """New tokens at positions `pos`, entries `entry` of sequences `seqs`; returns rotated q."""
        T = len(pos)
        qkv = bf16(rng.standard_normal((T, (H + 2 * Hk) * D))).cuda()
        q, kn, vn = (x.unflatten(1, (-1, D)) for x in qkv.split([H * D, Hk * D, Hk * D], 1))
        e, b = torch.tensor(entry, device="cuda"), torch.tensor(seqs, device="cuda")
        slots = tables[b, e // 16].long() * 16 + e % 16
        p = torch.tensor(pos, device="cuda")
        q_out = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
        if block8:
            k_out = torch.empty(T, Hk, D, dtype=torch.bfloat16, device="cuda")
            pa.pa_rope(q_out, k_out, q, kn, p, plan)
            pa.pa_cache_block8(k_out, vn.contiguous(), k, v, *sc, slots)
        else:
            pa.pa_rope_and_cache(q_out, q, kn, vn, k, v, slots, p, plan)
        return q_out

    def values(x, i):
        x = x.double().cpu().numpy()
        return x * sc[i].double().cpu().numpy()[:, None, :, None] if block8 else x

    append([p for n in start for p in range(n)], [p for n in start for p in range(n)], [b for b, n in enumerate(start) for _ in range(n)])
    pos, lens = list(start), list(start)
    for step in range(12):
        q = append(pos, lens, [0, 1])
        pos, lens = [p + 1 for p in pos], [n + 1 for n in lens]
        ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
        out = torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda")
        before = weights.clone()
        pa.pa_decode_weights(out, weights, q, k, v, tables, ld, 128, 0.1, 0, ws, **kw)
        att = R.attend(q.double().cpu().numpy(), values(k, 0), values(v, 1), host(tables), lens, 0.1,
                       host(sc[1]) if block8 else None)
        assert np.all(np.abs(out.double().cpu().numpy() - np.stack([a[0] for a in att])) <= bounds(att, 2.0 ** -8))
        added = (weights - before).sum(2).cpu().numpy()  # every head's probabilities sum to 1
        assert np.all(np.abs(added - H // Hk) <= 1e-3)
        if step % 4 == 3:
            keep, width = 40, 4
            dst = torch.arange(free, free + 2 * 8, dtype=torch.int32, device="cuda").view(2, 8)
            free = free + 16 if free < 48 else 0
            new_w = torch.empty(B, Hk, 128, device="cuda")
            kept = torch.empty(B, Hk, keep, dtype=torch.int32, device="cuda")
            new_lens = torch.empty(B, dtype=torch.int32, device="cuda")
            pa.pa_evict(k, v, weights, tables, ld, dst, new_w, new_lens, kept, 4, 8, 128, **kw)
            assert new_lens.tolist() == [min(n, keep) for n in lens]
            assert float(new_w[:, :, width * 16:].abs().sum()) == 0
            lens, tables, weights = new_lens.tolist(), dst, new_w
    assert pa.pa_get_status() == 0


def test_counting_and_evicting_in_a_graph(pa):
    rng = np.random.default_rng(58)
    lens = [300, 80]
    nb0, t = tables_of(rng, lens)
    pool = Pool(rng, "e4m3", nb0 + 16, 2, 128, t, lens)
    dst = torch.arange(nb0, nb0 + 16, dtype=torch.int32, device="cuda").view(2, 8)
    q = torch.randn(2, 8, 128, device="cuda").to(torch.bfloat16)
    td, ld = dev(t), dev(np.asarray(lens, np.int32))
    ws = torch.empty(pa.pa_decode_weights_workspace_bytes(2, 300, 0, pool.shape(pa, 8)), dtype=torch.uint8, device="cuda")

    def buffers():
        return [torch.empty_like(q), torch.zeros(2, 2, 300, device="cuda"), torch.empty(2, 2, 128, device="cuda"),
                torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(2, 2, 100, dtype=torch.int32, device="cuda")]

    def step(out, w, new_w, new_lens, kept):
        pa.pa_decode_weights(out, w, q, pool.k, pool.v, td, ld, 300, 0.1, 0, ws, **pool.kw)
        pa.pa_evict(pool.k, pool.v, w, td, ld, dst, new_w, new_lens, kept, 4, 16, 300, **pool.kw)

    eager, captured = buffers(), buffers()
    step(*eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*captured)
    for _ in range(2):
        captured[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            assert torch.equal(a, b)
    assert pa.pa_get_status() == 0
