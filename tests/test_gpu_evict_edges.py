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
