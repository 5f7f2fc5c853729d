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
