"""GPU checks of the decodes where their pieces meet: the prologue's scratch under the first loads, table entries outside
the pool, NaN over cut contexts, and the ends of the ranges that the pools' scales have."""
import numpy as np
import pytest
import torch

import cache_ops_ref as R
from test_gpu_block8 import bf16, dev, make_pool

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
