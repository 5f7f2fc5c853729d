"""GPU checks of the cache operators in the ways a server calls them: captured and replayed with new contents, on two
streams at once, with blocks swapped out between calls."""
import numpy as np
import pytest
import torch

import cache_ops_ref as R
from test_gpu_block8 import bf16, decode_case, dev, make_pool, run_decode, tables_of
from test_gpu_evict import Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_366_b200 import pa as _pa
    assert _pa.pa_get_status() == 0
    return _pa


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("T", [3, 40])
def test_write_replayed_with_new_tokens(pa, code, T):
    # one graph of the write, replayed for other rows and slots: appended to one sequence, over its blocks' borders
    rng = np.random.default_rng([101, T])
    Hk, D, steps = 2, 128, 6
    nb = R.blocks(T * steps)
    order = rng.permutation(nb)
    pools = [make_pool(rng, nb, Hk, D, code) for _ in range(2)]
    d = [dev(a) for a in (pools[0][0], pools[1][0], pools[0][1], pools[1][1])]
    mirror = [list(p) for p in pools]
    k, v = (torch.zeros(T, Hk, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        pa.pa_cache_block8(k, v, *d, slots)
    for step in range(steps):
        x = [bf16(rng.standard_normal((T, Hk, D)) * 2.0 ** step) for _ in range(2)]
        at = [int(order[p // 16]) * 16 + p % 16 for p in range(step * T, (step + 1) * T)]
        k.copy_(x[0])
        v.copy_(x[1])
        slots.copy_(torch.tensor(at))
        graph.replay()
        for i in range(2):
            mirror[i] = R.write(x[i].double().numpy(), *mirror[i], at, code)
    assert pa.pa_get_status() == 0
    for got, ref in zip(d, (mirror[0][0], mirror[1][0], mirror[0][1], mirror[1][1])):
        assert np.array_equal(got.cpu().numpy(), ref)


def test_rotation_replayed_with_new_positions(pa):
    T, H, Hk, D = 9, 8, 2, 128
    plan = pa.pa_rope_init(D, scaling="linear", factor=2.0)
    q, k = (torch.randn(T, h, D, device="cuda").to(torch.bfloat16) for h in (H, Hk))
    pos = torch.zeros(T, dtype=torch.int64, device="cuda")
    out, ref = [torch.empty_like(q), torch.empty_like(k)], [torch.empty_like(q), torch.empty_like(k)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        pa.pa_rope(*out, q, k, pos, plan)
    for step in range(4):
        pos.copy_(torch.arange(T) * 1001 + step * 70000)
        graph.replay()
        pa.pa_rope(*ref, q, k, pos, plan)
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    assert pa.pa_get_status() == 0


def test_counting_and_evicting_on_two_streams(pa):
    # two batches of different pools, each with its own workspace, at once: what each gives alone
    rng = np.random.default_rng(102)
    jobs = []
    for kind, lens in (("bf16", [700, 31, 0, 2000]), ("e4m3", [900] * 5)):
        nb0, t = tables_of(rng, lens)
        B, Hk, H, D, keep = len(lens), 4, 16, 64, 100
        per = R.blocks(keep)
        pool = Pool(rng, kind, nb0 + B * per, Hk, D, t, lens)
        dst = torch.arange(nb0, nb0 + B * per, dtype=torch.int32, device="cuda").view(B, per)
        q = torch.randn(B, H, D, device="cuda").to(pool.dtype)
        ld, td, top = dev(np.asarray(lens, np.int32)), dev(t), max(lens)
        n = pa.pa_decode_weights_workspace_bytes(B, top, 0, pool.shape(pa, H))

        def step(stream, pool=pool, dst=dst, q=q, ld=ld, td=td, top=top, n=n, B=B):
            o = dict(out=torch.empty_like(q), w=torch.zeros(B, Hk, top, device="cuda"),
                     new_w=torch.empty(B, Hk, per * 16, device="cuda"),
                     new_lens=torch.empty(B, dtype=torch.int32, device="cuda"),
                     kept=torch.empty(B, Hk, keep, dtype=torch.int32, device="cuda"),
                     ws=torch.empty(n, dtype=torch.uint8, device="cuda"))
            torch.cuda.synchronize()
            return o, lambda: (pa.pa_decode_weights(o["out"], o["w"], q, pool.k, pool.v, td, ld, top, 0.1, 0, o["ws"],
                                                    stream=stream, **pool.kw),
                               pa.pa_evict(pool.k, pool.v, o["w"], td, ld, dst, o["new_w"], o["new_lens"], o["kept"], 4, 20,
                                           top, stream=stream, **pool.kw))

        jobs.append((pool, step))
    alone = []
    for pool, step in jobs:
        o, go = step(None)
        for _ in range(5):
            go()
        torch.cuda.synchronize()
        alone.append((o, pool.k.clone(), pool.v.clone()))
    both = [step(torch.cuda.Stream()) for _, step in jobs]
    for _ in range(5):
        for _, go in both:
            go()
    torch.cuda.synchronize()
    assert pa.pa_get_status() == 0
    for (pool, _), (ref, k, v), (o, _) in zip(jobs, alone, both):
        assert torch.equal(pool.k, k) and torch.equal(pool.v, v)
        for name in ("out", "w", "new_w", "new_lens", "kept"):
            assert torch.equal(o[name], ref[name]), name


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_swapped_blocks_decode_the_same(pa, code):
    # a block8 pool's codes go to pinned host memory and come back to other blocks; the caller moves the scales' rows
    rng = np.random.default_rng(103)
    lens = [50, 33]
    q, kc, vc, ks, vs, t = decode_case(rng, lens, 8, 2, 64, code)
    ref = run_decode(pa, q, kc, vc, ks, vs, t, lens, 0.1)
    blocks = t[t >= 0]
    pairs = torch.from_numpy(np.stack([blocks, np.arange(len(blocks))], 1).astype(np.int64)).cuda()
    k, v, s_k, s_v = (dev(a) for a in (kc, vc, ks, vs))
    host = [torch.empty((len(blocks),) + x.shape[1:], dtype=x.dtype, pin_memory=True) for x in (k, v)]
    scales = [s[dev(blocks)] for s in (s_k, s_v)]
    for h, x in zip(host, (k, v)):
        pa.pa_swap_blocks(h, x, pairs)
    torch.cuda.synchronize()
    for x in (k, v):
        x.zero_()
    new = rng.permutation(kc.shape[0])[:len(blocks)]
    back = torch.from_numpy(np.stack([np.arange(len(blocks)), new], 1).astype(np.int64)).cuda()
    for h, x in zip(host, (k, v)):
        pa.pa_swap_blocks(x, h, back)
    for s, rows in zip((s_k, s_v), scales):
        s[dev(new)] = rows
    t2 = np.full_like(t, -1)
    t2[t >= 0] = new
    out = run_decode(pa, q, k.cpu().numpy(), v.cpu().numpy(), s_k.cpu().numpy(), s_v.cpu().numpy(), t2, lens, 0.1)
    assert torch.equal(out, ref) and pa.pa_get_status() == 0
