"""GPU checks of eviction at the ends of its ranges, and of both sizes of its selection's blocks."""
import numpy as np
import pytest
import torch

import test_gpu_evict as E
from test_gpu_block8 import dev
from test_gpu_evict import check_evict

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_366_b200 import pa as _pa
    assert _pa.pa_get_status() == 0
    return _pa


# ---- values at the end of bf16's range


def test_largest_values_survive_eviction(pa):
    # The write codes bf16's largest numbers as 256 at its largest scale, 2^120: a value that fp32 cannot hold, although
    # its code and its scale can. Cut to entries of the same block, it stays what it was.
    Hk, D = 2, 64
    top = float(torch.finfo(torch.bfloat16).max)
    x = torch.full((32, Hk, D), 1.0, dtype=torch.bfloat16, device="cuda")
    x[:16] = top
    x[3, 1] = -top
    k, v = (torch.zeros(3, 16, Hk, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(3, Hk, device="cuda") for _ in range(2))
    pa.pa_cache_block8(x, x, k, v, ks, vs, torch.arange(32, device="cuda"))
    assert ks[0].tolist() == [2.0 ** 120] * Hk and torch.equal(k[0] & 127, torch.full_like(k[0], 0x78))
    w = torch.zeros(1, Hk, 32, device="cuda")
    w[0, :, 2:6] = 1.0
    new_w, kept = torch.empty(1, Hk, 16, device="cuda"), torch.empty(1, Hk, 4, dtype=torch.int32, device="cuda")
    new_lens = torch.empty(1, dtype=torch.int32, device="cuda")
    pa.pa_evict(k, v, w, dev(np.array([[0, 1]], np.int32)), dev(np.array([32], np.int32)),
                dev(np.array([[2]], np.int32)), new_w, new_lens, kept, 0, 0, 32, k_scales=ks, v_scales=vs)
    assert pa.pa_get_status() == 0 and kept[0].tolist() == [[2, 3, 4, 5]] * Hk
    for codes, scales in ((k, ks), (v, vs)):
        assert torch.equal(scales[2], scales[0]) and torch.equal(codes[2, :4], codes[0, 2:6])


@pytest.mark.parametrize("D", [64, 128])
def test_largest_scales_among_others(pa, monkeypatch, D):
    class Huge(E.Pool):
        """A third of the blocks at scale 2^120, with codes up to 256, as the write leaves them."""

        def __init__(self, rng, kind, nb, *a):
            super().__init__(rng, kind, nb, *a)
            at = torch.from_numpy(rng.random(nb) < 1 / 3).cuda()
            for codes, scales in ((self.k, self.kw["k_scales"]), (self.v, self.kw["v_scales"])):
                mag = torch.minimum(codes & 127, torch.full_like(codes, 0x78))
                codes[at] = (codes & 128 | mag)[at]
                scales[at] = 2.0 ** 120

    monkeypatch.setattr(E, "Pool", Huge)
    check_evict(pa, np.random.default_rng(81), "e4m3", [300, 16, 17, 200], 2, D, 60, 2, 4)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_any_finite_scales(pa, monkeypatch, code):
    class Odd(E.Pool):
        """Scales that are no powers of two, from far below the write's least to above its largest, and zeros."""

        def __init__(self, rng, kind, nb, *a):
            super().__init__(rng, kind, nb, *a)
            for scales in (self.kw["k_scales"], self.kw["v_scales"]):
                x = rng.choice([-130.0, -66.0, -3.0, 0.0, 50.0, 119.0, 120.0, 125.0], (nb, scales.shape[1]))
                x = np.exp2(x + rng.random(x.shape))
                scales.copy_(torch.from_numpy(np.where(rng.random(x.shape) < 0.1, 0.0, x).astype(np.float32)))

    # rows of one scale and code times ratio rounds to fp32 and then to the code; the definition rounds once, which a
    # scale of few bits keeps the same: code times scale is then exact in fp32 too
    class Few(Odd):
        def __init__(self, *a):
            super().__init__(*a)
            for scales in (self.kw["k_scales"], self.kw["v_scales"]):
                scales.copy_((scales.view(torch.int32) & ~0xFFF).view(torch.float32))

    monkeypatch.setattr(E, "Pool", Few)
    check_evict(pa, np.random.default_rng(82), code, [300, 16, 17, 200], 2, 64, 60, 2, 4)


# ---- the selection's two sizes: 256 threads where many rows fill the GPU, else 512, each with clusters for long rows


RAGGED = [0, 1, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 400, 511, 512, 513, 600, 700, 777, 800,
          900, 1000, 1023, 1024, 1025, 1200, 1500, 1535, 1536, 1537, 1800, 2000, 2046, 2047, 2048]


@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (256, 4, 128), (300, 0, 0), (1025, 0, 1025), (2047, 4, 32)])
def test_many_short_rows(pa, keep, sinks, recent):
    # 39 sequences of 8 heads are more rows than SMs
    check_evict(pa, np.random.default_rng([91, keep]), "bf16", RAGGED, 8, 64, keep, sinks, recent)


@pytest.mark.parametrize("kind", ["f32", "fp8", "e4m3", "int8"])
def test_many_short_rows_of_every_pool(pa, kind):
    check_evict(pa, np.random.default_rng(92), kind, RAGGED, 8, 64, 256, 4, 128)


@pytest.mark.parametrize("top", [2048, 2049, 40000])
def test_many_rows_around_the_border(pa, top):
    # the same rows with a host bound at the border, past it and far past it: both sizes, with and without clusters
    check_evict(pa, np.random.default_rng(93), "bf16", RAGGED, 8, 64, 100, 4, 10, top=top)


def test_many_rows_one_too_long_for_shared_memory(pa):
    # 56 rows of a host bound that takes clusters of eight; one row is longer than they hold
    check_evict(pa, np.random.default_rng(96), "fp8", [430000, 70] + RAGGED + [5] * 15, 1, 64, 777, 4, 500)


def test_many_short_rows_ties_and_odd_weights(pa):
    rng = np.random.default_rng(94)
    shape = (len(RAGGED), 8, 2048)
    for fill in (0.0, 1.0, float("nan"), float("inf"), float("-inf")):
        check_evict(pa, rng, "bf16", RAGGED, 8, 64, 260, 3, 5, np.full(shape, fill, np.float32))
    w = rng.integers(0, 3, shape).astype(np.float32)  # many equal weights, cut among them
    check_evict(pa, rng, "bf16", RAGGED, 8, 64, 250, 0, 0, w)
    # equal but for the last bits: the digits decide in their last round
    w = (0x3F800000 + rng.integers(0, 64, shape)).astype(np.uint32).view(np.float32)
    check_evict(pa, rng, "bf16", RAGGED, 8, 64, 500, 1, 2, w)
    w = rng.standard_normal(shape).astype(np.float32)
    w[rng.random(shape) < 0.3] = np.nan
    w[rng.random(shape) < 0.1] = -0.0
    w[rng.random(shape) < 0.1] = 0.0
    w[rng.random(shape) < 0.05] = np.inf
    w[rng.random(shape) < 0.05] = -np.inf
    w[rng.random(shape) < 0.05] = 1e-42
    check_evict(pa, rng, "bf16", RAGGED, 8, 64, 400, 10, 20, w)


# ---- counting for more sequences than the merge scans


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3", "int8"])
@pytest.mark.parametrize("part", [0, 64])
def test_counting_many_sequences(pa, kind, part):
    # more than 256: the merge before the counting takes its slices from the records that the decode kernel leaves
    rng = np.random.default_rng([95, part])
    lens = [int(n) for n in rng.integers(0, 90, 299)] + [1500]
    E.check_count(pa, rng, kind, lens, 8, 2, 64, part=part, steps=2)
