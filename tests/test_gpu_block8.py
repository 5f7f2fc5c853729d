"""GPU checks of the block8 pools (8-bit codes, a scale for each block and KV head): the write bit for bit against
the definition, and decode within bounds derived from its roundings."""
import numpy as np
import pytest
import torch

import cache_ops_ref as R
from paged_kv_cache_366_b200 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from paged_kv_cache_366_b200 import pa as _pa
    assert _pa.pa_get_status() == 0
    return _pa


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def make_pool(rng, nb, Hk, D, code, spread=2.0):
    """Codes and scales of normal values whose size differs by block and head."""
    x = rng.standard_normal((nb, 16, Hk, D)) * np.exp2(rng.standard_normal((nb, 1, Hk, 1)) * spread)
    return R.quantized_pool(x, code)


def tables_of(rng, lens, slack=1, extra=5):
    need = [R.blocks(n) for n in lens]
    nb = sum(need) + extra
    perm = rng.permutation(nb).astype(np.int32)
    t = np.full((len(lens), max(max(need), 1) + slack), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return nb, t


# ---- the write


def check_write(pa, x_k, x_v, codes, scales, slots, code):
    (kc, vc), (ks, vs) = codes, scales
    d = [dev(a) for a in (kc, vc, ks, vs)]
    k, v = bf16(x_k).cuda(), bf16(x_v).cuda()
    pa.pa_cache_block8(k, v, *d, dev(np.asarray(slots, np.int64)))
    status = pa.pa_get_status()
    kr, ksr = R.write(k.double().cpu().numpy(), kc, ks, slots, code)
    vr, vsr = R.write(v.double().cpu().numpy(), vc, vs, slots, code)
    for got, ref in zip(d, (kr, vr, ksr, vsr)):
        g = got.cpu().numpy()
        if g.dtype == np.uint8:  # either NaN code is NaN
            g, ref = np.where((g & 127) == 127, 127, g), np.where((ref & 127) == 127, 127, ref)
        assert np.array_equal(g, ref, equal_nan=g.dtype == np.float32)
    return status, d


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("Hk,D", [(8, 128), (2, 64), (1, 128), (3, 64)])
@pytest.mark.parametrize("new", [1, 2, 15, 16, 17, 130])
def test_write_matches_definition(pa, code, Hk, D, new):
    rng = np.random.default_rng([Hk, D, new])
    lens = [0, 1, 15, 16, 31, 7, 200]
    nb, t = tables_of(rng, [n + new for n in lens])
    pools = [make_pool(rng, nb, Hk, D, code) for _ in range(2)]
    slots = [t[b, p // 16] * 16 + p % 16 for b, n in enumerate(lens) for p in range(n, n + new)]
    # sizes that make some scales grow, some not, by much and by little
    x = [rng.standard_normal((len(slots), Hk, D)) * np.exp2(rng.integers(-6, 7, (len(slots), 1, 1))) for _ in range(2)]
    status, _ = check_write(pa, *x, [p[0] for p in pools], [p[1] for p in pools], slots, code)
    assert status == 0


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_write_token_by_token_equals_its_definition(pa, code):
    # forty calls of one token each for two sequences: blocks start, fill, and their scales grow step by step
    rng = np.random.default_rng(9)
    Hk, D = 2, 128
    nb, t = tables_of(rng, [40, 40])
    codes = [np.full((nb, 16, Hk, D), 0x7F, np.int8 if code == "int8" else np.uint8) for _ in range(2)]
    scales = [np.full((nb, Hk), np.nan, np.float32) for _ in range(2)]  # never read for a fresh block
    for p in range(40):
        slots = [int(t[b, p // 16] * 16 + p % 16) for b in range(2)]
        x = [rng.standard_normal((2, Hk, D)) * 2.0 ** (p % 16) for _ in range(2)]
        _, d = check_write(pa, *x, codes, scales, slots, code)
        codes, scales = [d[0].cpu().numpy(), d[1].cpu().numpy()], [d[2].cpu().numpy(), d[3].cpu().numpy()]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_write_extremes(pa, code):
    """Zeros, the smallest and largest bf16 numbers, infinities and NaN; padding at both ends and between sequences."""
    rng = np.random.default_rng(11)
    Hk, D = 2, 64
    rows = np.zeros((12, Hk, D))
    rows[1] = 1e-38
    rows[2, :, 0] = 3.0e38
    rows[3] = rng.standard_normal((Hk, D))
    rows[3, 0, 5], rows[3, 1, 6] = np.inf, -np.inf
    rows[4] = np.nan
    rows[5] = rng.standard_normal((Hk, D))
    rows[5, :, 3] = np.nan
    rows[6] = 448.0
    rows[7] = 450.0
    rows[8] = 127.0
    rows[9] = 2.0 ** -70
    rows[10:] = rng.standard_normal((2, Hk, D))
    slots = [-1, 16, 32, 48, 64, 80, 96, 112, 128, -5, 144, 145]
    pool = make_pool(rng, 12, Hk, D, code)
    status, _ = check_write(pa, rows, -rows, (pool[0], pool[0]), (pool[1], pool[1]), slots, code)
    assert status == 0


def test_write_bad_slot(pa):
    rng = np.random.default_rng(12)
    pool = make_pool(rng, 4, 2, 64, "e4m3")
    x = rng.standard_normal((3, 2, 64))
    status, _ = check_write(pa, x, x, (pool[0], pool[0]), (pool[1], pool[1]), [5, 64, 1 << 40], "e4m3")
    assert status == pa.PA_STATUS_BAD_SLOT


def test_write_many_tokens(pa):
    # enough tokens for a warp to look through 16 of them; sequences end inside blocks
    rng = np.random.default_rng(13)
    Hk, D = 8, 128
    lens = [rng.integers(1, 900) for _ in range(20)]
    nb, t = tables_of(rng, lens)
    pools = [make_pool(rng, nb, Hk, D, "int8", 0.0) for _ in range(2)]
    slots = [t[b, p // 16] * 16 + p % 16 for b, n in enumerate(lens) for p in range(n)]
    x = [rng.standard_normal((len(slots), Hk, D)) for _ in range(2)]
    check_write(pa, *x, [p[0] for p in pools], [p[1] for p in pools], slots, "int8")


# ---- decode


def bounds(attended, half_step):
    """Error bound of every output: half a step of its type; p rounded to f16 (2^-11) and its exponential (2^-20);
    scores summed in fp32 over at most 128 products (2^-17 of the sum of their sizes S), which moves p and the
    softmax sum each by that factor. (q and the codes are exact in f16.)

    Over a block8 pool p v_scale enters as f16 in units of 2^r, where 2^(r + 7) <= its largest: below f16's normal
    numbers the rounding is 2^-25 units, at most 2^-32 of that largest, for each of n codes of at most 448."""
    return np.stack([half_step * np.abs(o) + a * (2.0 ** -11 + 2.0 ** -20 + 2 * 2.0 ** -17 * s[:, None]) +
                     2.0 ** -32 * u[:, None] + 1e-30 for o, _, a, s, u in attended])


def poison(codes, scales, tables, lens, code):
    """Free blocks and rows past each context hold NaN codes (E4M3) or large ones, free blocks' scales NaN."""
    bad = 0x7F
    used = np.zeros(codes.shape[:2], bool)
    for b, n in enumerate(lens):
        for p in range(n):
            used[tables[b, p // 16], p % 16] = True
    codes[~used] = bad
    scales[~used.any(1)] = np.nan


def decode_case(rng, lens, H, Hk, D, code, spread=2.0):
    nb, t = tables_of(rng, lens)
    kc, ks = make_pool(rng, nb, Hk, D, code, spread)
    vc, vs = make_pool(rng, nb, Hk, D, code, spread)
    for c, s in ((kc, ks), (vc, vs)):
        poison(c, s, t, lens, code)
    q = bf16(rng.standard_normal((len(lens), H, D)) * 2)
    return q, kc, vc, ks, vs, t


def run_decode(pa, q, kc, vc, ks, vs, t, lens, scale, part=0):
    d = [dev(a) for a in (kc, vc, ks, vs, t, np.asarray(lens, np.int32))]
    top = max(lens)
    n = pa.pa_decode_block8_workspace_bytes(len(lens), top, part, pa.shape_of_block8(d[0], q.shape[1]))
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    pa.pa_decode_block8(out, q.cuda(), *d, top, scale, part, ws)
    return out


def check_decode(pa, rng, lens, H, Hk, D, code, part=0, spread=2.0):
    q, kc, vc, ks, vs, t = decode_case(rng, lens, H, Hk, D, code, spread)
    scale = 1 / np.sqrt(D)
    out = run_decode(pa, q, kc, vc, ks, vs, t, lens, scale, part)
    assert pa.pa_get_status() == 0
    att = R.attend(q.double().numpy(), R.dequantized(kc, ks, code), R.dequantized(vc, vs, code), t, lens, scale, vs)
    ref, tol = np.stack([a[0] for a in att]), bounds(att, 2.0 ** -8)
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    worst = float((np.abs(got - ref) / tol).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("H,Hk,D", [(32, 8, 128), (16, 2, 64), (8, 8, 128), (64, 8, 128), (16, 8, 128), (4, 1, 64),
                                    (8, 1, 64), (3, 3, 64), (6, 3, 64)])
@pytest.mark.parametrize("part", [0, 64])
def test_decode_ragged(pa, code, H, Hk, D, part):
    rng = np.random.default_rng([H, Hk, D, part])
    check_decode(pa, rng, [1, 15, 16, 17, 0, 64, 65, 200, 1031], H, Hk, D, code, part)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_decode_long_and_short(pa, code):
    rng = np.random.default_rng(21)
    check_decode(pa, rng, [9000, 1, 0, 33, 4097], 8, 2, 128, code)


def test_decode_one_token(pa):
    check_decode(pa, np.random.default_rng(22), [1], 32, 8, 128, "e4m3")
    check_decode(pa, np.random.default_rng(23), [1], 8, 8, 64, "int8")


def test_decode_all_empty(pa):
    q, kc, vc, ks, vs, t = decode_case(np.random.default_rng(24), [0, 0, 0], 8, 2, 128, "e4m3")
    out = run_decode(pa, q, kc, vc, ks, vs, t, [0, 0, 0], 0.1)
    assert int(out.count_nonzero()) == 0 and not bool(out.isnan().any())


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_decode_scales_far_apart(pa, code):
    # block scales over 2^+-60: f16 alone could not hold the spread
    rng = np.random.default_rng(25)
    lens = [100, 400, 17]
    q, kc, vc, ks, vs, t = decode_case(rng, lens, 16, 4, 128, code)
    vs = np.exp2(rng.integers(-30, 31, vs.shape)).astype(np.float32)
    ks = (ks * np.float32(0.25)).astype(np.float32)
    poison(vc, vs, t, lens, code)
    out = run_decode(pa, q, kc, vc, ks, vs, t, lens, 0.1)
    att = R.attend(q.double().numpy(), R.dequantized(kc, ks, code), R.dequantized(vc, vs, code), t, lens, 0.1, vs)
    ref, tol = np.stack([a[0] for a in att]), bounds(att, 2.0 ** -8)
    worst = float((np.abs(out.double().cpu().numpy() - ref) / tol).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** 60])
def test_decode_tiny_and_huge_queries(pa, size):
    # q far outside f16's range, scaled back by the softmax scale
    rng = np.random.default_rng(26)
    lens = [50, 3]
    q, kc, vc, ks, vs, t = decode_case(rng, lens, 8, 2, 64, "e4m3", 0.0)
    scale = 0.125 / size
    out = run_decode(pa, (q.float() * size).to(torch.bfloat16), kc, vc, ks, vs, t, lens, scale)
    att = R.attend(q.double().numpy() * size, R.dequantized(kc, ks, "e4m3"), R.dequantized(vc, vs, "e4m3"), t, lens, scale, vs)
    ref, tol = np.stack([a[0] for a in att]), bounds(att, 2.0 ** -8)
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)


def test_decode_zero_scales(pa):
    # blocks of zeros may carry a zero scale: their entries count in the softmax and add nothing
    rng = np.random.default_rng(27)
    lens = [60, 16]
    q, kc, vc, ks, vs, t = decode_case(rng, lens, 8, 2, 64, "int8", 0.0)
    ks[t[0, 1]], vs[t[0, 1]], vs[t[1, 0]] = 0, 0, 0
    out = run_decode(pa, q, kc, vc, ks, vs, t, lens, 0.2)
    att = R.attend(q.double().numpy(), R.dequantized(kc, ks, "int8"), R.dequantized(vc, vs, "int8"), t, lens, 0.2, vs)
    ref, tol = np.stack([a[0] for a in att]), bounds(att, 2.0 ** -8)
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= tol)


def test_decode_bad_block_and_context_are_flagged(pa):
    rng = np.random.default_rng(28)
    lens = [40, 20]
    q, kc, vc, ks, vs, t = decode_case(rng, lens, 8, 2, 64, "e4m3")
    good = run_decode(pa, q, kc, vc, ks, vs, t, lens, 0.1)
    t2 = t.copy()
    t2[0, 1] = kc.shape[0]
    out = run_decode(pa, q, kc, vc, ks, vs, t2, lens, 0.1)
    assert pa.pa_get_status() == pa.PA_STATUS_BAD_BLOCK_ID
    assert torch.equal(out[1], good[1])
    d = [dev(a) for a in (kc, vc, ks, vs, t, np.asarray([40, 20], np.int32))]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    pa.pa_decode_block8(torch.empty_like(good), q.cuda(), *d, 32, 0.1, 0, ws)  # 40 > the host's bound of 32
    assert pa.pa_get_status() == pa.PA_STATUS_BAD_CONTEXT


def test_write_then_decode_step_by_step(pa):
    """Prefill two sequences, then decode twenty tokens: the pool that the calls leave gives the definition's output."""
    rng = np.random.default_rng(29)
    H, Hk, D, code = 32, 8, 128, "int8"
    lens = np.array([37, 120])
    nb, t = tables_of(rng, [n + 20 for n in lens])
    z = [torch.zeros(nb, 16, Hk, D, dtype=torch.int8, device="cuda") for _ in range(2)]
    s = [torch.zeros(nb, Hk, device="cuda") for _ in range(2)]
    mirror = [(np.zeros((nb, 16, Hk, D), np.int8), np.zeros((nb, Hk), np.float32)) for _ in range(2)]

    def append(lo, hi):
        slots = [t[b, p // 16] * 16 + p % 16 for b in range(2) for p in range(lo[b], hi[b])]
        x = [bf16(rng.standard_normal((len(slots), Hk, D))) for _ in range(2)]
        pa.pa_cache_block8(x[0].cuda(), x[1].cuda(), *z, *s, dev(np.asarray(slots, np.int64)))
        for i in range(2):
            mirror[i] = R.write(x[i].double().numpy(), *mirror[i], slots, code)

    append([0, 0], lens)
    for step in range(20):
        append(lens + step, lens + step + 1)
    for i in range(2):
        assert np.array_equal(z[i].cpu().numpy(), mirror[i][0]) and np.array_equal(s[i].cpu().numpy(), mirror[i][1])
    q = bf16(rng.standard_normal((2, H, D)))
    now = list(lens + 20)
    out = run_decode(pa, q, *[z[i].cpu().numpy() for i in range(2)], *[s[i].cpu().numpy() for i in range(2)], t, now, 0.1)
    att = R.attend(q.double().numpy(), *[R.dequantized(*m, code) for m in mirror], t, now, 0.1, mirror[1][1])
    assert np.all(np.abs(out.double().cpu().numpy() - np.stack([a[0] for a in att])) <= bounds(att, 2.0 ** -8))


def test_decode_in_a_graph_and_on_another_stream(pa):
    rng = np.random.default_rng(30)
    lens = [300, 17, 90]
    q, kc, vc, ks, vs, t = decode_case(rng, lens, 32, 8, 128, "e4m3")
    ref = run_decode(pa, q, kc, vc, ks, vs, t, lens, 0.1)
    d = [dev(a) for a in (kc, vc, ks, vs, t, np.asarray(lens, np.int32))]
    n = pa.pa_decode_block8_workspace_bytes(3, 300, 0, pa.shape_of_block8(d[0], 32))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    qd, out = q.cuda(), torch.zeros_like(ref)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    pa.pa_decode_block8(out, qd, *d, 300, 0.1, 0, ws, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.pa_decode_block8(out, qd, *d, 300, 0.1, 0, ws)
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


def test_decode_many_sequences(pa):
    # more than 256 sequences: the merge finds its slices in the records the decode kernel leaves
    rng = np.random.default_rng(31)
    lens = [int(n) for n in rng.integers(0, 90, 300)]
    check_decode(pa, rng, lens, 8, 2, 64, "e4m3")
    check_decode(pa, rng, lens[:270] + [3000], 4, 4, 128, "int8")


def test_decode_more_sequences_than_one_scan_holds(pa):
    # 30000 sequences of one token or none: an output row is its value row
    rng = np.random.default_rng(32)
    B, H, Hk, D = 30000, 4, 2, 64
    kc, ks = make_pool(rng, 50, Hk, D, "int8")
    vc, vs = make_pool(rng, 50, Hk, D, "int8")
    t = rng.integers(0, 50, (B, 1)).astype(np.int32)
    lens = rng.integers(0, 2, B).astype(np.int32)
    q = bf16(rng.standard_normal((B, H, D)))
    out = run_decode(pa, q, kc, vc, ks, vs, t, lens, 0.1)
    assert pa.pa_get_status() == 0
    ref = bf16(R.dequantized(vc, vs, "int8")[t[:, 0], 0] * lens[:, None, None]).repeat_interleave(H // Hk, 1)
    # one code times a power of two: exact up to the division by the softmax sum, which is 1
    assert torch.equal(out.cpu().float(), ref.float())


def test_decode_on_two_streams_at_once(pa):
    rng = np.random.default_rng(33)
    cases = []
    for code, lens in (("e4m3", [2000, 300, 5]), ("int8", [700] * 6)):
        q, kc, vc, ks, vs, t = decode_case(rng, lens, 32, 8, 128, code)
        ref = run_decode(pa, q, kc, vc, ks, vs, t, lens, 0.1)
        d = [dev(a) for a in (kc, vc, ks, vs, t, np.asarray(lens, np.int32))]
        n = pa.pa_decode_block8_workspace_bytes(len(lens), max(lens), 0, pa.shape_of_block8(d[0], 32))
        cases.append((q.cuda(), d, max(lens), torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(ref), ref,
                      torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for q, d, top, ws, out, _, stream in cases:
            pa.pa_decode_block8(out, q, *d, top, 0.1, 0, ws, stream=stream)
    torch.cuda.synchronize()
    for _, _, _, _, out, ref, _ in cases:
        assert torch.equal(out, ref)


def test_high_blocks_past_32_bits(pa):
    # a pool of 4.9 GB of codes: rows whose byte offsets need more than 32 bits are written, read and evicted
    NB, Hk, D, H, n = 300000, 8, 128, 32, 40
    rng = np.random.default_rng(34)
    k, v = (torch.zeros(NB, 16, Hk, D, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(NB, Hk, device="cuda") for _ in range(2))
    t = np.array([[NB - 1, NB - 7, 270000]], np.int32)
    slots = np.array([int(t[0, p // 16]) * 16 + p % 16 for p in range(n)], np.int64)
    x = [bf16(rng.standard_normal((n, Hk, D))) for _ in range(2)]
    pa.pa_cache_block8(x[0].cuda(), x[1].cuda(), k, v, ks, vs, dev(slots))
    td, ld = dev(t), torch.tensor([n], dtype=torch.int32, device="cuda")
    q = bf16(rng.standard_normal((1, H, D)))
    w = torch.zeros(1, Hk, 48, device="cuda")
    out = torch.empty(1, H, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(pa.pa_decode_weights_workspace_bytes(1, 48, 0, pa.shape_of_block8(k, H)), dtype=torch.uint8, device="cuda")
    pa.pa_decode_weights(out, w, q.cuda(), k, v, td, ld, 48, 0.1, 0, ws, k_scales=ks, v_scales=vs)
    small = [np.zeros((3, 16, Hk, D), np.int8) for _ in range(2)], [np.zeros((3, Hk), np.float32) for _ in range(2)]
    local = [p for p in range(n)]
    (kc, ksr), (vc, vsr) = (R.write(x[i].double().numpy(), small[0][i], small[1][i], local, "int8") for i in range(2))
    att = R.attend(q.double().numpy(), R.dequantized(kc, ksr, "int8"), R.dequantized(vc, vsr, "int8"), np.arange(3)[None], [n], 0.1, vsr)
    assert np.all(np.abs(out.double().cpu().numpy() - att[0][0]) <= bounds(att, 2.0 ** -8))
    dst = torch.tensor([[NB - 20]], dtype=torch.int32, device="cuda")
    kept, new_w = torch.empty(1, Hk, 16, dtype=torch.int32, device="cuda"), torch.empty(1, Hk, 16, device="cuda")
    new_lens = torch.empty(1, dtype=torch.int32, device="cuda")
    pa.pa_evict(k, v, w, td, ld, dst, new_w, new_lens, kept, 2, 4, 48, k_scales=ks, v_scales=vs)
    assert pa.pa_get_status() == 0
    wh = w.cpu().numpy()
    for h in range(Hk):
        idx = R.select(wh[0, h], n, 16, 2, 4)
        assert np.array_equal(kept[0, h].cpu().numpy(), idx)
        for pool, scales, codes, s in ((v, vs, vc, vsr), (k, ks, kc, ksr)):
            rows = R.values(codes[idx // 16, idx % 16, h], "int8") * s[idx // 16, h].astype(np.float64)[:, None]
            scale = R.least_scale(rows, "int8")
            assert float(scales[NB - 20, h]) == scale
            assert np.array_equal(pool[NB - 20, :, h].cpu().numpy(), R.encode(rows / scale, "int8"))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_several_query_tokens_as_rows(pa, code):
    # a verify chunk of 4 tokens at the end of each sequence: rows with one table and growing lengths
    rng = np.random.default_rng(35)
    lens = [4, 21, 100, 333]
    q, kc, vc, ks, vs, t = decode_case(rng, lens, 16, 4, 128, code)
    rows = np.repeat(t, 4, axis=0)
    row_lens = [n - 3 + j for n in lens for j in range(4)]
    q = bf16(rng.standard_normal((16, 16, 128)))
    out = run_decode(pa, q, kc, vc, ks, vs, rows, row_lens, 0.1)
    assert pa.pa_get_status() == 0
    att = R.attend(q.double().numpy(), R.dequantized(kc, ks, code), R.dequantized(vc, vs, code), rows, row_lens, 0.1, vs)
    assert np.all(np.abs(out.double().cpu().numpy() - np.stack([a[0] for a in att])) <= bounds(att, 2.0 ** -8))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_copied_blocks_decode_the_same(pa, code):
    # copy-on-write of a block8 pool: codes by pa_copy_blocks, scales' rows by the caller
    rng = np.random.default_rng(36)
    lens = [50, 33]
    q, kc, vc, ks, vs, t = decode_case(rng, lens, 8, 2, 64, code)
    ref = run_decode(pa, q, kc, vc, ks, vs, t, lens, 0.1)
    free = np.setdiff1d(np.arange(kc.shape[0]), t[t >= 0])[:3]
    src = np.array([t[0, 0], t[0, 3], t[1, 2]])
    k, v, s_k, s_v = (dev(a) for a in (kc, vc, ks, vs))
    pa.pa_copy_blocks(k, v, dev(np.stack([src, free], 1).astype(np.int64)))
    for s in (s_k, s_v):
        s[dev(free)] = s[dev(src)]
    t2 = t.copy()
    t2[0, 0], t2[0, 3], t2[1, 2] = free
    out = run_decode(pa, q, k.cpu().numpy(), v.cpu().numpy(), s_k.cpu().numpy(), s_v.cpu().numpy(), t2, lens, 0.1)
    assert torch.equal(out, ref) and pa.pa_get_status() == 0
