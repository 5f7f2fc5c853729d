"""GPU checks of the rotary calls' cosines and sines: how far each may be from the plan's angle."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_366_b200 import pa as _pa
    assert _pa.pa_get_status() == 0
    return _pa


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot,far", [(128, 128, 1 << 21), (64, 64, 300), (128, 32, 2 ** 31 - 1)])
def test_cosines_and_sines_near_the_angle(pa, inter, D, rot, far):
    # Pairs (1, 0) in fp32 come out as (cos, sin) themselves. The reference turns by the plan's own steps, reduced to
    # an eighth of a turn in integers.
    rng = np.random.default_rng([71, D, rot])
    T, half = 4096, rot // 2
    pos = rng.integers(-far, far, T)
    pos[:5] = [0, far, 1, -1, -far]
    plan = pa.pa_rope_init(rot, interleaved=inter)
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, half), slice(half, rot))
    q = torch.zeros(T, 1, D, device="cuda")
    q[..., i] = 1.0
    out, k_out = torch.empty_like(q), torch.empty_like(q)
    pa.pa_rope(out, k_out, q, q, torch.from_numpy(pos).cuda(), plan)
    assert pa.pa_get_status() == 0 and torch.equal(out, k_out)
    got = out[:, 0].double().cpu().numpy()

    step = np.array([plan.step[f] for f in range(half)], np.uint64)
    phase = pos.astype(np.int64).view(np.uint64)[:, None] * step  # of a turn, times 2^64, wrapping around
    quarter = (phase + np.uint64(1 << 61)) >> np.uint64(62)
    a = (phase - (quarter << np.uint64(62))).view(np.int64).astype(np.float64) * (2 * np.pi * 2.0 ** -64)
    c, s, n = np.cos(a), np.sin(a), quarter.astype(np.int64)
    cos = np.choose(n, [c, -s, -c, s])
    sin = np.choose(n, [s, c, -s, -c])
    for x, ref in ((got[:, i], cos), (got[:, j], sin)):
        # the reduced angle rounds to fp32 once and moves each function by no more than that; each function is within
        # one step of fp32. (A number just above a power of two P rounds by up to half a step of 2^-23 P: 2^-24 of it.)
        tol = 2.0 ** -24 * np.abs(a) * (1 + 2.0 ** -20) + np.spacing(np.abs(ref).astype(np.float32))
        assert np.all(np.abs(x - ref) <= tol), float((np.abs(x - ref) / tol).max())
