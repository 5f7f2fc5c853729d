"""GPU checks of the decodes where their pieces meet: the prologue's scratch under the first loads, table entries outside
the pool, NaN over cut contexts, and the ends of the ranges that the pools' scales have."""
import numpy as np
import pytest
import torch

import cache_ops_ref as R
from test_gpu_block8 import bf16, bounds, dev, make_pool, tables_of
from test_gpu_evict import POOLS, Pool, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_366_b200 import pa as _pa
    assert _pa.pa_get_status() == 0
    return _pa


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_first_blocks_land_where_the_length_scan_was(pa, kind):
    # 20000 sequences: the scan of their lengths lies over most of every warp's ring, in which the first blocks land
    # at once. One token or none each, so an output row is its value row, whatever the softmax rounds.
    rng = np.random.default_rng(61)
    B, H, Hk, D = 20000, 4, 2, 128
    t = rng.integers(0, 50, (B, 1)).astype(np.int32)
    lens = rng.integers(0, 2, B).astype(np.int32)
    q = bf16(rng.standard_normal((B, H, D))).cuda()
    out = torch.empty_like(q)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    if kind == "int8":
        (kc, ks), (vc, vs) = (make_pool(rng, 50, Hk, D, "int8") for _ in range(2))
        v = R.dequantized(vc, vs, "int8")
        pool = [dev(a) for a in (kc, vc, ks, vs)]
        call = pa.pa_decode_block8
    else:
        k, v = (bf16(rng.standard_normal((50, 16, Hk, D))) for _ in range(2))
        pool, v = [k.cuda(), v.cuda()], v.double().numpy()
        call = pa.pa_decode
    td, ld = dev(t), dev(lens)
    ref = bf16(v[t[:, 0], 0] * lens[:, None, None]).repeat_interleave(H // Hk, 1).cuda()
    for _ in range(20):
        out.fill_(float("nan"))
        call(out, q, *pool, td, ld, 1, 0.1, 0, ws)
        assert torch.equal(out, ref)
    assert pa.pa_get_status() == 0


# ---- table entries outside the pool


def _without(t, lens, bad):
    """Tables and lengths as if the entries of the blocks in bad[b] were not there, and the places of those left."""
    rows, left, places = [], [], []
    for b, n in enumerate(lens):
        keep = [i for i in range(R.blocks(n)) if i not in bad[b]]
        places.append(np.array([p for p in range(n) if p // 16 in keep], np.int64))
        left.append(len(places[-1]))
        rows.append([t[b, i] for i in keep])
    width = max(1, max(len(r) for r in rows))
    return np.array([r + [0] * (width - len(r)) for r in rows], np.int32), left, places


@pytest.mark.parametrize("kind", POOLS)
@pytest.mark.parametrize("H,Hk,D", [(32, 8, 128), (8, 8, 64), (16, 2, 128), (6, 3, 64)])
@pytest.mark.parametrize("part", [0, 64, 4096])
@pytest.mark.parametrize("left_over", [0xFF, 0x40])  # what the workspace holds: NaN, or about 3.0
def test_counting_leaves_out_bad_entries(pa, kind, H, Hk, D, part, left_over):
    # The entries of a block outside the pool take no part: their weights stay, the others' are those of a softmax
    # without them, and a sequence of nothing else gives zeros and leaves all its weights. (Of the whole blocks that are
    # left, every row is valid; the last block of a sequence may be bad too.)
    rng = np.random.default_rng([62, H, Hk, D, part])
    lens = [100, 37, 77, 16, 1, 640]
    bad = [{1, 4}, {0, 1, 2}, {4}, set(), {0}, {0, 7, 20, 21, 22, 39}]
    nb, t = tables_of(rng, lens)
    pool = Pool(rng, kind, nb, Hk, D, t, lens)
    good = t.copy()
    for b, blocks in enumerate(bad):
        for i in blocks:
            t[b, i] = (-1, nb, 2 ** 31 - 1)[i % 3]
    q = torch.from_numpy(rng.standard_normal((len(lens), H, D))).to(pool.dtype)
    w0 = rng.random((len(lens), Hk, max(lens) + 3)).astype(np.float32)
    scale = 1 / np.sqrt(D)

    def run(table):
        n = pa.pa_decode_weights_workspace_bytes(len(lens), max(lens), part, pool.shape(pa, H))
        ws = torch.full((n,), left_over, dtype=torch.uint8, device="cuda")
        out, w = torch.full(q.shape, float("nan"), dtype=pool.dtype, device="cuda"), dev(w0)
        pa.pa_decode_weights(out, w, q.cuda(), pool.k, pool.v, dev(table), dev(np.asarray(lens, np.int32)), max(lens),
                             scale, part, ws, **pool.kw, **pool.one)
        return out.double().cpu().numpy(), w.cpu().numpy()

    out_good, w_good = run(good)
    assert pa.pa_get_status() == 0
    out, w = run(t)
    assert pa.pa_get_status() == pa.PA_STATUS_BAD_BLOCK_ID
    assert np.array_equal(out[3], out_good[3]) and np.array_equal(w[3], w_good[3])  # untouched by its neighbours
    rows, left, places = _without(t, lens, bad)
    att = R.attend(q.double().numpy(), pool.k64, pool.v64, rows, left, scale,
                   host(pool.kw["v_scales"]) if pool.kw else None)
    tol = bounds(att, torch.finfo(pool.dtype).eps / 2)
    for b, n in enumerate(lens):
        assert np.all(np.abs(out[b] - att[b][0]) <= tol[b])
        p = att[b][1].reshape(Hk, H // Hk, left[b])
        s = att[b][3].reshape(Hk, H // Hk, 1)
        ref = w0[b].astype(np.float64)
        ref[:, places[b]] += p.sum(1)
        # p: scores in fp32 (2^-17 of their size, in p and in the sum) and the exponential; then fp32 sums
        near = np.zeros_like(ref)
        near[:, places[b]] = (p * (2 * 2.0 ** -17 * s + 2.0 ** -20)).sum(1) + (H // Hk + 1) * 2.0 ** -24 * ref[:, places[b]]
        assert np.all(np.abs(w[b] - ref) <= near)  # no tolerance where nothing is added


# ---- NaN over cut contexts


def _decode(pa, pool, q, t, lens, scale, part, weights=None):
    """pa_decode or pa_decode_block8, or pa_decode_weights where weights are given."""
    td, ld, top = dev(t), dev(np.asarray(lens, np.int32)), max(lens)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    out = torch.zeros(q.shape, dtype=pool.dtype, device="cuda")
    if weights is not None:
        pa.pa_decode_weights(out, weights, q, pool.k, pool.v, td, ld, top, scale, part, ws, **pool.kw, **pool.one)
    elif pool.kw:
        pa.pa_decode_block8(out, q, pool.k, pool.v, pool.kw["k_scales"], pool.kw["v_scales"], td, ld, top, scale, part, ws)
    else:
        pa.pa_decode(out, q, pool.k, pool.v, td, ld, top, scale, part, ws, **pool.one)
    assert pa.pa_get_status() == 0
    return out


@pytest.mark.parametrize("kind", POOLS)
@pytest.mark.parametrize("counting", [False, True])
@pytest.mark.parametrize("part", [0, 64, 65536])
def test_nan_query_gives_nan(pa, kind, counting, part):
    # One head's query holds a NaN: all its scores are NaN, in every slice that its context is cut into. Its output is
    # NaN (and so are its KV head's weights), wherever the cuts lie; the other heads' outputs are what they were.
    rng = np.random.default_rng([63, part])
    lens, H, Hk, D = [1000, 16, 5], 8, 2, 128
    nb, t = tables_of(rng, lens)
    pool = Pool(rng, kind, nb, Hk, D, t, lens)
    q = torch.from_numpy(rng.standard_normal((3, H, D))).to(pool.dtype)
    att = R.attend(q.double().numpy(), pool.k64, pool.v64, t, lens, 0.1, host(pool.kw["v_scales"]) if pool.kw else None)
    tol = bounds(att, torch.finfo(pool.dtype).eps / 2)
    q[0, 3, 5] = q[1, 0, 0] = float("nan")
    w = torch.zeros(3, Hk, 1000, device="cuda") if counting else None
    out = _decode(pa, pool, q.cuda(), t, lens, 0.1, part, w).double().cpu().numpy()
    hit = np.zeros((3, H), bool)
    hit[0, 3] = hit[1, 0] = True
    assert np.all(np.isnan(out[hit]))
    ref = np.stack([a[0] for a in att])
    assert np.all(np.abs(out - ref)[~hit] <= tol[~hit])
    if counting:
        nan = w.isnan().cpu().numpy()
        for b, n in enumerate(lens):
            assert np.array_equal(nan[b, :, :n], np.repeat([[b < 2], [False]], n, 1)) and not nan[b, :, n:].any()


@pytest.mark.parametrize("kind", ["bf16", "f32", "fp8", "e4m3"])
@pytest.mark.parametrize("part", [0, 64, 65536])
def test_block_of_nan_keys_gives_nan(pa, kind, part):
    # A slice of its own may hold nothing but a block of NaN keys; the heads that read it give NaN all the same.
    rng = np.random.default_rng([64, part])
    lens, H, Hk, D = [333, 40], 8, 2, 64
    nb, t = tables_of(rng, lens)
    pool = Pool(rng, kind, nb, Hk, D, t, lens)
    q = torch.from_numpy(rng.standard_normal((2, H, D))).to(pool.dtype)
    att = R.attend(q.double().numpy(), pool.k64, pool.v64, t, lens, 0.1, host(pool.kw["v_scales"]) if pool.kw else None)
    pool.k[int(t[0, 7]), :, 1] = 0x7F if pool.k.dtype == torch.uint8 else float("nan")
    out = _decode(pa, pool, q.cuda(), t, lens, 0.1, part).double().cpu().numpy()
    assert np.all(np.isnan(out[0, 4:]))
    ref, tol = np.stack([a[0] for a in att]), bounds(att, torch.finfo(pool.dtype).eps / 2)
    assert np.all(np.abs(out - ref)[0, :4] <= tol[0, :4]) and np.all(np.abs(out - ref)[1] <= tol[1])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("part", [0, 64, 65536])
def test_scores_of_minus_infinity(pa, kind, part):
    # Keys of -inf and positive queries: scores of -inf. A context of nothing else gives zeros and leaves the weights;
    # among others they count for nothing.
    rng = np.random.default_rng([65, part])
    lens, H, Hk, D = [300, 50, 20], 8, 2, 64
    nb, t = tables_of(rng, lens)
    pool = Pool(rng, kind, nb, Hk, D, t, lens)
    q = torch.from_numpy(np.abs(rng.standard_normal((3, H, D))) + 0.01).to(pool.dtype)
    places = [np.arange(16 * 5, 300), np.arange(0), np.arange(20)]
    for i in list(range(5)):
        pool.k[int(t[0, i])] = float("-inf")
    for i in range(4):
        pool.k[int(t[1, i])] = float("-inf")
    rows = np.full_like(t, 0)
    rows[0, :t.shape[1] - 5], rows[2] = t[0, 5:], t[2]
    att = R.attend(q.double().numpy(), pool.k64, pool.v64, rows, [220, 0, 20], 0.1, None)
    tol = bounds(att, torch.finfo(pool.dtype).eps / 2)
    w = torch.zeros(3, Hk, 300, device="cuda")
    for weights in (None, w):
        out = _decode(pa, pool, q.cuda(), t, lens, 0.1, part, weights).double().cpu().numpy()
        assert np.all(np.abs(out - np.stack([a[0] for a in att])) <= tol)
    w = w.double().cpu().numpy()
    for b in range(3):
        ref = np.zeros((Hk, 300))
        p, s = (x.reshape(Hk, H // Hk, -1) for x in (att[b][1], att[b][3]))
        ref[:, places[b]] = p.sum(1)
        near = np.zeros((Hk, 300))
        near[:, places[b]] = (p * (2 * 2.0 ** -17 * s + 2.0 ** -20)).sum(1) + (H // Hk + 1) * 2.0 ** -24 * p.sum(1)
        assert np.all(np.abs(w[b] - ref) <= near)


# ---- how many digits the probabilities keep


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("H,Hk,D", [(32, 8, 128), (64, 8, 128), (4, 2, 64), (3, 3, 128)])
@pytest.mark.parametrize("counting", [False, True])
def test_block8_probabilities_keep_their_digits(pa, code, H, Hk, D, counting):
    # Queries of zero: every probability is 1 / n and no score has an error. The value scales are no powers of two, so
    # each block's p v_scale is another number, and whatever rounding it meets shows where values cancel.
    rng = np.random.default_rng([66, H, D])
    lens = [32] * 24 + [31, 17, 16, 1]
    nb, t = tables_of(rng, lens)
    pool = Pool(rng, code, nb, Hk, D, t, lens)
    vs = np.exp2(rng.random((nb, Hk)) * 2).astype(np.float32)
    pool.kw["v_scales"] = dev(vs)
    v64 = R.dequantized(host(pool.v), vs, code)
    q = torch.zeros(len(lens), H, D, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(len(lens), Hk, 32, device="cuda") if counting else None
    att = R.attend(q.double().cpu().numpy(), pool.k64, v64, t, lens, 0.1, vs)
    ref, a = np.stack([x[0] for x in att]), np.stack([x[2] for x in att])
    # p v_scale = 2^(log2(v_scale) - r): the logarithm to 2^-21, r and the difference rounded to fp32 (numbers below 16:
    # 2^-21 each), two exponentials to 2^-21, p's two f16 parts 2^-21: less than 2^-18 in all; a few sums in fp32 that
    # may cut (2^-23 each): 2^-17 covers both.
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -17 * a
    for part in (0, 64, 65536):
        got = _decode(pa, pool, q, t, lens, 0.1, part, w).double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= tol), float((np.abs(got - ref) / (tol + 1e-30)).max())


# ---- the ends of the scales' range


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("H,Hk,D", [(16, 4, 128), (64, 8, 64), (2, 2, 128)])
@pytest.mark.parametrize("part", [0, 64, 65536])
@pytest.mark.parametrize("counting", [False, True])
def test_value_scales_over_their_whole_range(pa, code, H, Hk, D, part, counting):
    # The write makes scales from 2^-64 to 2^120. Sequences of scales near either end, of all sizes mixed, and of scales
    # below the write's that a caller may have; sums of 2^100 * 448 * 400 are still bf16 numbers.
    rng = np.random.default_rng([67, H, D, part])
    lens = [400, 399, 17, 100, 33, 1]
    ends = [(-64, -60), (96, 100), (-64, 100), (-64, 100), (-100, -90), (100, 100)]
    nb, t = tables_of(rng, lens)
    pool = Pool(rng, code, nb, Hk, D, t, lens)
    vs = host(pool.kw["v_scales"]).copy()
    for b, (lo, hi) in enumerate(ends):
        at = t[b, :R.blocks(lens[b])]
        vs[at] = np.exp2(rng.integers(lo, hi + 1, (len(at), Hk)))
    pool.kw["v_scales"] = dev(vs)
    v64 = R.dequantized(host(pool.v), vs, code)
    q = bf16(rng.standard_normal((len(lens), H, D)))
    w = torch.zeros(len(lens), Hk, 400, device="cuda") if counting else None
    got = _decode(pa, pool, q.cuda(), t, lens, 0.1, part, w).double().cpu().numpy()
    att = R.attend(q.double().numpy(), pool.k64, v64, t, lens, 0.1, vs)
    ref, tol = np.stack([x[0] for x in att]), bounds(att, 2.0 ** -8)
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - ref) <= tol)
    if counting:
        for b, n in enumerate(lens):
            p = att[b][1].reshape(Hk, H // Hk, n)
            s = att[b][3].reshape(Hk, H // Hk, 1)
            near = (p * (2 * 2.0 ** -17 * s + 2.0 ** -20)).sum(1) + (H // Hk + 1) * 2.0 ** -24 * p.sum(1)
            assert np.all(np.abs(w[b, :, :n].double().cpu().numpy() - p.sum(1)) <= near)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_key_scales_over_their_whole_range(pa, code):
    # Key scales from far below to 2^120, undone by the softmax scale: a sequence of one size each.
    rng = np.random.default_rng(68)
    H, Hk, D = 16, 4, 64
    for e in (-64, -20, 60, 100, 120):
        lens = [77, 300, 16]
        nb, t = tables_of(rng, lens)
        pool = Pool(rng, code, nb, Hk, D, t, lens)
        ks = np.full((nb, Hk), 2.0 ** e, np.float32)
        pool.kw["k_scales"] = dev(ks)
        q = bf16(rng.standard_normal((3, H, D)) * 2.0 ** -6)
        scale = 0.01 * 2.0 ** -e
        got = _decode(pa, pool, q.cuda(), t, lens, scale, 0).double().cpu().numpy()
        att = R.attend(q.double().numpy(), R.dequantized(host(pool.k), ks, code), pool.v64, t, lens, scale,
                       host(pool.kw["v_scales"]))
        assert np.all(np.abs(got - np.stack([x[0] for x in att])) <= bounds(att, 2.0 ** -8))
