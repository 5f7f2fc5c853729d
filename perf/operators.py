"""The cache operators as measurable cases: rotary positions with the cache write, the 8-bit cache with a scale
for each block and KV head, decode that counts attention weights, and eviction by those weights.

`run` computes each in plain torch operations, or (where `own` is true) through the library's calls.
"""
import math
import random

import torch

own = False  # set from outside: False = plain torch, True = the library's kernels

BLOCK = 16
CODE_MAX = {"e4m3": 448.0, "int8": 127.0}
# the least and largest exponent of a block's scale 2^e
E_MIN, E_MAX = -64, 120


# ---------------------------------------------------------------------------
# The cases


def listed():
    heads = {"H": 32, "Hk": 8, "D": 128}
    return [
        # one token of one sequence: what an idle server adds to its latency
        dict(name="rope_one", op="rope", T=1, span=2048, rot=128, layout="half", scaling="none", cache="bf16", **heads),
        # a decode step of 64 sequences, a quarter of the head rotated in pairs, odd positions, FP8 pool
        dict(name="rope_decode64", op="rope", T=64, span=32768, rot=32, layout="pairs", scaling="linear", cache="fp8",
             **heads),
        # a step of four 2048-token prefill chunks, frequencies scaled by parts for a long context
        dict(name="rope_prefill8k", op="rope", T=8192, span=131072, rot=128, layout="half", scaling="parts",
             cache="bf16", **heads),
        # the write of a decode step: one token for each of 64 sequences, into partly filled blocks
        dict(name="write8_decode64", op="write8", B=64, new=1, lo=1, hi=2048, code="e4m3", **heads),
        # the write of a mixed step's chunks, lengths that end inside a block
        dict(name="write8_prefill", op="write8", B=5, new=1637, lo=1, hi=700, code="int8", **heads),
        # one short sequence: latency
        dict(name="decode8_one", op="decode8", B=1, lo=333, hi=333, code="e4m3", **heads),
        # the decode batch: 64 sequences of ragged lengths
        dict(name="decode8_batch", op="decode8", B=64, lo=128, hi=2048, code="e4m3", **heads),
        # long contexts
        dict(name="decode8_long", op="decode8", B=8, lo=32768, hi=32768, code="int8", **heads),
        # the decode batch, counting weights, over the plain pool
        dict(name="weights_batch", op="weights", B=64, lo=128, hi=2048, cache="bf16", **heads),
        # long contexts over the 8-bit pool, counting weights
        dict(name="weights8_long", op="weights", B=8, lo=9000, hi=32768, cache="e4m3", **heads),
        # a batch's caches cut to a budget of 512 entries
        dict(name="evict_batch", op="evict", B=64, lo=128, hi=2048, keep=512, sinks=4, recent=128, cache="bf16",
             **heads),
        # long contexts cut to a quarter, over the 8-bit pool
        dict(name="evict8_long", op="evict", B=8, lo=9000, hi=32768, keep=8191, sinks=4, recent=1024, cache="e4m3",
             **heads),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    H, Hk = rng.choice([(32, 8), (16, 2), (8, 8), (64, 8), (16, 8), (4, 1)])
    heads = {"H": H, "Hk": Hk, "D": rng.choice([64, 128, 128])}
    op = rng.choice(["rope", "write8", "decode8", "weights", "evict"])
    if op == "rope":
        return dict(op=op, T=_log_int(rng, 1, 4096), span=_log_int(rng, 256, 1 << 20),
                    rot=rng.choice([heads["D"], heads["D"] // 2, heads["D"] // 4]),
                    layout=rng.choice(["half", "pairs"]), scaling=rng.choice(["none", "linear", "base", "parts"]),
                    cache=rng.choice(["bf16", "fp8", "f32"]), **heads)
    if op == "write8":
        new = rng.choice([1, 1, _log_int(rng, 2, 1024)])
        return dict(op=op, B=_log_int(rng, 1, 256 if new == 1 else 8), new=new, lo=1, hi=_log_int(rng, 2, 2048),
                    code=rng.choice(["e4m3", "int8"]), **heads)
    hi = _log_int(rng, 1, 32768)
    lo = rng.choice([hi, _log_int(rng, 1, hi), 1])
    B = _log_int(rng, 1, max(1, min(128, (1 << 17) // hi)))
    if op == "decode8":
        return dict(op=op, B=B, lo=lo, hi=hi, code=rng.choice(["e4m3", "int8"]), **heads)
    cache = rng.choice(["bf16", "f32", "fp8", "e4m3", "int8"])
    if op == "weights":
        return dict(op=op, B=B, lo=lo, hi=hi, cache=cache, **heads)
    keep = _log_int(rng, 1, max(1, hi))
    sinks = rng.randint(0, min(4, keep))
    return dict(op=op, B=B, lo=lo, hi=hi, keep=keep, sinks=sinks, recent=rng.randint(0, (keep - sinks) // 2),
                cache=cache, **heads)


def _lens(case):
    """The context lengths, from the case alone: the first is the longest, the others spread between lo and hi."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    lens[0] = case["hi"]
    return lens


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


# ---------------------------------------------------------------------------
# Inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _tables(g, lens, spare=0):
    """Tables of every sequence's blocks in a shuffled pool with free blocks among them, int32, -1 past the end;
    `spare` more blocks for each sequence in a second table."""
    need = [_blocks(n) for n in lens]
    nb = sum(need) + spare * len(lens) + 7
    perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    width = max(max(need), 1)
    col = torch.arange(width, device="cuda")
    n = torch.tensor(need, device="cuda")
    first = torch.cumsum(n, 0) - n
    at = (first[:, None] + col[None]).clamp(max=nb - 1)
    table = torch.where(col[None] < n[:, None], perm[at], torch.full_like(perm[at], -1))
    other = perm[sum(need):sum(need) + spare * len(lens)].view(len(lens), spare) if spare else None
    return nb, table.contiguous(), other.contiguous() if spare else None


def _kv(g, nb, Hk, D, like):
    """A pool's keys or values: normal, heads of different sizes, some blocks much larger than others."""
    x = _randn(g, nb, BLOCK, Hk, D)
    x *= torch.exp2(_randn(g, 1, 1, Hk, 1) * 0.5)
    x *= torch.exp2(_randn(g, nb, 1, Hk, 1) * 0.5)
    return x.to(like)


def _exponent(amax, code):
    """The least e with amax <= CODE_MAX 2^e, in [E_MIN, E_MAX]."""
    f, x = torch.frexp(amax)  # amax = f 2^x, f in [0.5, 1)
    f9, x9 = math.frexp(CODE_MAX[code])
    e = x - x9 + (f > f9).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _encode(x, code):
    return x.to(torch.float8_e4m3fn) if code == "e4m3" else torch.round(x).clamp(-127, 127).to(torch.int8)


def _as_codes(x, code):
    """The pool's own type: E4M3 codes are bytes."""
    return x.view(torch.uint8) if code == "e4m3" else x


def _as_values(codes, code):
    return codes.view(torch.float8_e4m3fn) if code == "e4m3" else codes


def _quantized(x, code):
    """Whole blocks [NB][16][Hk][D] as codes and scales [NB][Hk]."""
    e = _exponent(x.float().abs().amax(dim=(1, 3)), code)
    s = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    return _as_codes(_encode(x.float() / s[:, None, :, None], code), code), s


FP8_SCALES = (0.0625, 0.046875)  # k_scale, v_scale of the pool with one scale


def _pools(g, nb, case):
    Hk, D, cache = case["Hk"], case["D"], case["cache"]
    s = {}
    if cache in CODE_MAX:
        s["k"], s["ks"] = _quantized(_kv(g, nb, Hk, D, torch.bfloat16), cache)
        s["v"], s["vs"] = _quantized(_kv(g, nb, Hk, D, torch.bfloat16), cache)
    elif cache == "fp8":
        for name, sc in zip("kv", FP8_SCALES):
            x = _kv(g, nb, Hk, D, torch.bfloat16).float() / sc
            s[name] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        dt = torch.bfloat16 if cache == "bf16" else torch.float32
        s["k"], s["v"] = _kv(g, nb, Hk, D, dt), _kv(g, nb, Hk, D, dt)
    return s


def _frequencies(case):
    """rot / 2 angular frequencies per position, in 64 bits, and the factor on cos and sin."""
    rot, base, factor = case["rot"], 10000.0, 8.0
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    if case["scaling"] == "base":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "parts":  # turns over the original context: below `low` interpolated, above `high` kept
        low, high, original = 1.0, 32.0, 4096.0
        keep = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
        return f, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = _gen(seed)
    H, Hk, D, op = case["H"], case["Hk"], case["D"], case["op"]
    s = {"case": case}
    if op == "rope":
        T = case["T"]
        dt = torch.float32 if case["cache"] == "f32" else torch.bfloat16
        # q, k and v as a projection leaves them: columns of one matrix
        s["qkv"] = _randn(g, T, (H + 2 * Hk) * D).to(dt)
        s["positions"] = torch.randint(0, case["span"], (T,), generator=g, device="cuda")
        nb = _blocks(T) + 7
        s |= _pools(g, nb, case)
        s["slots"] = torch.randperm(nb * BLOCK, generator=g, device="cuda")[:T].contiguous()
        s["q_out"] = torch.empty(T, H, D, dtype=dt, device="cuda")
        s["freq"], s["mscale"] = _frequencies(case)
        if own:
            from paged_kv_cache_366_b200 import pa
            s["rope"] = pa.pa_rope_init(case["rot"], 10000.0, interleaved=case["layout"] == "pairs",
                                        scaling=case["scaling"], factor=8.0, low=1.0, high=32.0, original_len=4096.0,
                                        mscale=s["mscale"])
        return s
    lens = _lens(case)
    if op == "write8":
        B, new = case["B"], case["new"]
        nb, table, _ = _tables(g, [n + new for n in lens])
        s |= _pools(g, nb, dict(case, cache=case["code"]))
        s["k_new"] = _kv(g, B * new, Hk, D, torch.bfloat16)[:, 0].contiguous()
        s["v_new"] = _kv(g, B * new, Hk, D, torch.bfloat16)[:, 0].contiguous()
        p = torch.tensor(lens, device="cuda")[:, None] + torch.arange(new, device="cuda")[None]
        block = torch.gather(table.long(), 1, p // BLOCK)
        s["slots"] = (block * BLOCK + p % BLOCK).reshape(-1).contiguous()
        return s
    case = dict(case, cache=case.get("cache") or case["code"])
    spare = _blocks(min(case["keep"], case["hi"])) if op == "evict" else 0
    nb, s["tables"], s["dst"] = _tables(g, lens, spare)
    s |= _pools(g, nb, case)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["max_len"] = max(lens)
    width = s["tables"].shape[1] * BLOCK
    if op != "decode8":  # what some steps of decoding have left: a few entries hold most of the weight
        w = torch.exp2(_randn(g, case["B"], Hk, width) * 3 - 4)
        s["weights"] = w * (torch.arange(width, device="cuda")[None] < s["lens"][:, None])[:, None]
    if op == "evict":
        s["kept"] = torch.empty(case["B"], Hk, case["keep"], dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.empty_like(s["lens"])
        s["new_weights"] = torch.empty(case["B"], Hk, spare * BLOCK, device="cuda")
    else:
        dt = torch.float32 if case["cache"] == "f32" else torch.bfloat16
        s["q"] = (_randn(g, case["B"], H, D) * 2).to(dt)
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = 1.0 / math.sqrt(D)
    if own:  # scratch that a serving loop keeps
        from paged_kv_cache_366_b200 import pa
        if op == "evict":
            n = 0
        elif op == "decode8":
            n = pa.pa_decode_block8_workspace_bytes(case["B"], s["max_len"], 0, pa.shape_of_block8(s["k"], H))
        else:
            shape = pa.shape_of_block8(s["k"], H) if case["cache"] in CODE_MAX else pa.shape_of(s["k"], H, *FP8_SCALES)
            n = pa.pa_decode_weights_workspace_bytes(case["B"], s["max_len"], 0, shape)
        s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# One pass


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "rope":
        _rope_own(s) if own else _rope_plain(s)
        fp8 = case["cache"] == "fp8"
        k, v = (x.view(torch.float8_e4m3fn) if fp8 else x for x in (s["k"], s["v"]))
        return {"q": s["q_out"], "k": k, "v": v}
    if op == "write8":
        _write8_own(s) if own else _write8_plain(s)
        return {"k": _as_values(s["k"], case["code"]), "v": _as_values(s["v"], case["code"]), "ks": s["ks"],
                "vs": s["vs"]}
    if op == "evict":
        _evict_own(s) if own else _evict_plain(s)
        b8 = case["cache"] in CODE_MAX
        codes = case["cache"] if b8 else "e4m3"
        k, v = (_as_values(x, codes) if x.dtype in (torch.uint8, torch.int8) else x for x in (s["k"], s["v"]))
        out = {"kept": s["kept"], "lens": s["new_lens"], "weights": s["new_weights"], "k": k, "v": v}
        return out | ({"ks": s["ks"], "vs": s["vs"]} if b8 else {})
    if op == "decode8":
        _decode8_own(s) if own else _attend_plain(s)
        return s["out"]
    _weights_own(s) if own else _attend_plain(s)
    return {"out": s["out"], "weights": s["weights"]}


# ---- the library's calls


def _split(s):
    case = s["case"]
    H, Hk, D = case["H"], case["Hk"], case["D"]
    return (x.unflatten(1, (-1, D)) for x in s["qkv"].split([H * D, Hk * D, Hk * D], 1))


def _rope_own(s):
    from paged_kv_cache_366_b200 import pa
    q, k, v = _split(s)
    ks, vs = FP8_SCALES if s["case"]["cache"] == "fp8" else (0.0, 0.0)
    pa.pa_rope_and_cache(s["q_out"], q, k, v, s["k"], s["v"], s["slots"], s["positions"], s["rope"], k_scale=ks,
                         v_scale=vs)


def _write8_own(s):
    from paged_kv_cache_366_b200 import pa
    pa.pa_cache_block8(s["k_new"], s["v_new"], s["k"], s["v"], s["ks"], s["vs"], s["slots"])


def _decode8_own(s):
    from paged_kv_cache_366_b200 import pa
    pa.pa_decode_block8(s["out"], s["q"], s["k"], s["v"], s["ks"], s["vs"], s["tables"], s["lens"], s["max_len"],
                        s["scale"], 0, s["workspace"])


def _weights_own(s):
    from paged_kv_cache_366_b200 import pa
    ks, vs = FP8_SCALES if s["case"]["cache"] == "fp8" else (0.0, 0.0)
    pa.pa_decode_weights(s["out"], s["weights"], s["q"], s["k"], s["v"], s["tables"], s["lens"], s["max_len"],
                         s["scale"], 0, s["workspace"], k_scale=ks, v_scale=vs, k_scales=s.get("ks"),
                         v_scales=s.get("vs"))


def _evict_own(s):
    from paged_kv_cache_366_b200 import pa
    case = s["case"]
    pa.pa_evict(s["k"], s["v"], s["weights"], s["tables"], s["lens"], s["dst"], s["new_weights"], s["new_lens"],
                s["kept"], case["sinks"], case["recent"], s["max_len"], k_scales=s.get("ks"), v_scales=s.get("vs"))


# ---- the plain forms


def _rope_plain(s):
    case = s["case"]
    r, half = case["rot"], case["rot"] // 2
    a = s["positions"].double()[:, None] * s["freq"][None]  # far positions: angles in 64 bits
    cos, sin = ((f(a) * s["mscale"]).float()[:, None] for f in (torch.cos, torch.sin))

    def rotated(x):
        x = x.float()
        y = x.clone()
        if case["layout"] == "half":
            x0, x1 = x[..., :half], x[..., half:r]
            y[..., :half], y[..., half:r] = x0 * cos - x1 * sin, x1 * cos + x0 * sin
        else:
            x0, x1 = x[..., 0:r:2], x[..., 1:r:2]
            y[..., 0:r:2], y[..., 1:r:2] = x0 * cos - x1 * sin, x1 * cos + x0 * sin
        return y

    q, k, v = _split(s)
    s["q_out"].copy_(rotated(q))
    k, v = rotated(k), v.float()
    if case["cache"] == "fp8":
        k, v = ((x * (1.0 / sc)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                for x, sc in zip((k, v), FP8_SCALES))
    else:
        k, v = k.to(s["k"].dtype), v.to(s["v"].dtype)
    s["k"].flatten(0, 1)[s["slots"]] = k
    s["v"].flatten(0, 1)[s["slots"]] = v


def _write8_plain(s):
    code = s["case"]["code"]
    block, row = s["slots"] // BLOCK, s["slots"] % BLOCK
    used, of = torch.unique(block, return_inverse=True)
    first = torch.full_like(used, BLOCK).scatter_reduce(0, of, row, "amin")  # rows below it hold earlier tokens
    earlier = torch.arange(BLOCK, device="cuda")[None] < first[:, None]
    for codes, scales, x in ((s["k"], s["ks"], s["k_new"]), (s["v"], s["vs"], s["v_new"])):
        x = x.float()
        amax = x.abs().amax(dim=2)
        top = torch.zeros_like(scales[used]).scatter_reduce(0, of[:, None].expand_as(amax), amax, "amax")
        need = torch.ldexp(torch.ones_like(top), _exponent(top, code))
        old = scales[used]
        scale = torch.where(first[:, None] > 0, torch.maximum(old, need), need)
        held = codes[used]
        again = _as_codes(_encode(_as_values(held, code).float() * (old / scale)[:, None, :, None], code), code)
        codes[used] = torch.where(earlier[:, :, None, None], again, held)
        codes[block, row] = _as_codes(_encode(x / scale[of][:, :, None], code), code)
        scales[used] = scale


def _values(codes, scales, code):
    return _as_values(codes, code).float() * scales[:, None, :, None]


def _cached(s, tables):
    """Keys and values of every sequence, [B][W][Hk][D] in 32 bits (rows past a context hold whatever is there)."""
    cache = s["case"].get("cache") or s["case"]["code"]
    t = tables.long().clamp(min=0)
    both = []
    for x, scales, one in ((s["k"], s.get("ks"), FP8_SCALES[0]), (s["v"], s.get("vs"), FP8_SCALES[1])):
        x = x[t]  # [B][MB][16][Hk][D]
        if cache in CODE_MAX:
            x = _as_values(x, cache).float() * scales[t][:, :, None, :, None]
        elif cache == "fp8":
            x = x.view(torch.float8_e4m3fn).float() * one
        both.append(x.float().flatten(1, 2))
    return both


def _attend_plain(s):
    case = s["case"]
    B, H, Hk, D = case["B"], case["H"], case["Hk"], case["D"]
    k, v = _cached(s, s["tables"])
    valid = torch.arange(k.shape[1], device="cuda")[None] < s["lens"][:, None]  # [B][W]
    v = v * valid[:, :, None, None]
    q = s["q"].float().view(B, Hk, H // Hk, D)
    x = (q @ k.permute(0, 2, 3, 1)) * s["scale"]  # [B][Hk][G][W]
    x = x.masked_fill(~valid[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(dim=-1, keepdim=True))
    p = p / p.sum(dim=-1, keepdim=True)
    s["out"].copy_((p @ v.permute(0, 2, 1, 3)).view(B, H, D))
    if case["op"] == "weights":
        s["weights"] += p.sum(dim=2)


def _evict_plain(s):
    case = s["case"]
    keep, Hk = case["keep"], case["Hk"]
    w = s["weights"]
    width = w.shape[2]
    at = torch.arange(width, device="cuda")[None]
    n = s["lens"].long()[:, None]
    always = (at < case["sinks"]) | (at >= n - case["recent"])
    key = w.masked_fill(always[:, None], math.inf).masked_fill((at >= n)[:, None], -math.inf)
    order = torch.sort(key, dim=2, descending=True, stable=True).indices[..., :keep]
    m = n.clamp(max=keep)  # entries left, [B][1]
    slot = torch.arange(keep, device="cuda")[None]
    left = (slot < m)[:, None].expand(-1, Hk, -1)  # [B][Hk][keep]
    if order.shape[2] < keep:
        order = torch.nn.functional.pad(order, (0, keep - order.shape[2]), value=0)
    kept = torch.where(left, order, width).sort(dim=2).values
    s["kept"].copy_(torch.where(left, kept, -1))
    s["new_lens"].copy_(m[:, 0])
    kept = torch.where(left, kept, 0)
    s["new_weights"].zero_()
    count = min(keep, s["new_weights"].shape[2])  # no sequence is longer than the new table
    kept, left, slot = kept[..., :count], left[..., :count], slot[:, :count]
    s["new_weights"][..., :count] = torch.gather(w, 2, kept) * left
    # the rows: from (source block, row, head) to (new block, row, head)
    src = torch.gather(s["tables"].long()[:, None].expand(-1, Hk, -1), 2, kept // BLOCK)
    dst = s["dst"].long()[:, None, :].expand(-1, Hk, -1)
    to = torch.gather(dst, 2, (slot // BLOCK)[:, None].expand(kept.shape[0], Hk, -1))
    head = torch.arange(Hk, device="cuda")[None, :, None].expand_as(kept)
    b, h, i = torch.nonzero(left, as_tuple=True)
    src, row, to, trow, head = src[b, h, i], kept[b, h, i] % BLOCK, to[b, h, i], i % BLOCK, head[b, h, i]
    code = case["cache"] if case["cache"] in CODE_MAX else None
    for name in "kv":
        x = s[name][src, row, head]  # [rows][D]
        if code:
            scales = s[name + "s"]
            x = _as_values(x, code).float() * scales[src, head][:, None]
            amax = torch.zeros_like(scales).index_put((to, head), torch.zeros((), device="cuda"))
            amax = amax.flatten().scatter_reduce(0, to * Hk + head, x.abs().amax(dim=1), "amax").view_as(scales)
            scale = torch.ldexp(torch.ones_like(amax), _exponent(amax, code))
            scales[to, head] = scale[to, head]
            x = _as_codes(_encode(x / scale[to, head][:, None], code), code)
        s[name][to, trow, head] = x


# ---------------------------------------------------------------------------
# Work


def work(case):
    H, Hk, D, op = case["H"], case["Hk"], case["D"], case["op"]
    if op == "rope":
        e = 4 if case["cache"] == "f32" else 2
        c = 1 if case["cache"] == "fp8" else e
        return {"bytes": case["T"] * (2 * H * D * e + 2 * Hk * D * (e + c) + 16), "flops": case["T"] * (H + Hk) * case["rot"] * 3}
    lens = _lens(case)
    tokens, blocks = sum(lens), sum(_blocks(n) for n in lens)
    if op == "write8":
        new = case["B"] * case["new"]
        touched = sum(_blocks(n + case["new"]) - n // BLOCK for n in lens)
        return {"bytes": new * (2 * Hk * D * 3 + 8) + touched * Hk * 2 * 8, "flops": new * 2 * Hk * D * 2}
    cache = case.get("cache") or case["code"]
    e = {"f32": 4, "bf16": 2}.get(cache, 1)
    scales = blocks * Hk * 2 * 4 if cache in CODE_MAX else 0
    if op == "evict":
        left = sum(min(n, case["keep"]) for n in lens)
        new_scales = sum(_blocks(min(n, case["keep"])) for n in lens) * Hk * 2 * 4 if cache in CODE_MAX else 0
        b = tokens * Hk * 4 + left * Hk * (2 * 2 * D * e + 12) + scales + new_scales + blocks * 4
        return {"bytes": b, "flops": tokens * Hk}
    b = tokens * 2 * Hk * D * e + scales + blocks * 4 + 2 * case["B"] * H * D * (4 if cache == "f32" else 2)
    if op == "weights":
        b += tokens * Hk * 8
    return {"bytes": b, "flops": tokens * H * D * 4}


# ---------------------------------------------------------------------------
# The definition, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _rope_exact(s)
    if op == "write8":
        return _write8_exact(s)
    if op == "evict":
        return _evict_exact(s)
    return _attend_exact(s)


def _e4m3_nearest(x):
    """The E4M3 value nearest to x (ties to even), saturating at 448, in 64 bits."""
    a = x.abs().clamp(max=448.0)
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (e - 4).clamp(min=-9))
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), x)


def _rope_exact(s):
    case = s["case"]
    H, Hk, D, r = case["H"], case["Hk"], case["D"], case["rot"]
    x = s["qkv"].double().view(case["T"], H + 2 * Hk, D)
    a = s["positions"].double()[:, None, None] * s["freq"]
    turn = torch.polar(torch.full_like(a, s["mscale"]), a)
    rq = x[:, :H + Hk, :r]
    z = torch.complex(rq[..., :r // 2], rq[..., r // 2:]) if case["layout"] == "half" else torch.view_as_complex(
        rq.reshape(case["T"], H + Hk, r // 2, 2).contiguous())
    z = z * turn
    x[:, :H + Hk, :r] = torch.cat((z.real, z.imag), -1) if case["layout"] == "half" else torch.view_as_real(z).flatten(-2)
    pools = []
    for name, sc, new in (("k", FP8_SCALES[0], x[:, H:H + Hk]), ("v", FP8_SCALES[1], x[:, H + Hk:])):
        pool = s[name].view(torch.float8_e4m3fn).double() if case["cache"] == "fp8" else s[name].double()
        pool.flatten(0, 1)[s["slots"]] = _e4m3_nearest(new / sc) if case["cache"] == "fp8" else new
        pools.append(pool)
    return {"q": x[:, :H], "k": pools[0], "v": pools[1]}


def _exact_scale(amax, code):
    """The least power of two s with amax <= CODE_MAX s."""
    e = torch.ceil(torch.log2(amax / CODE_MAX[code]))
    s = torch.exp2(e)
    s = torch.where(amax > CODE_MAX[code] * s, s * 2, s)
    s = torch.where(amax <= CODE_MAX[code] * s / 2, s / 2, s)
    return s.clamp(2.0 ** E_MIN, 2.0 ** E_MAX)


def _exact_code(x, code):
    return _e4m3_nearest(x) if code == "e4m3" else torch.round(x).clamp(-127, 127)


def _write8_exact(s):
    case = s["case"]
    code, B, new = case["code"], case["B"], case["new"]
    lens = _lens(case)
    slots = s["slots"].view(B, new)
    out = {}
    for name in "kv":
        codes = _as_values(s[name], code).double()
        scales = s[name + "s"].double()
        x = s[name + "_new"].double().view(B, new, case["Hk"], case["D"])
        group = {}  # the sequences that fill as many rows, from the same row, go together
        for b, n in enumerate(lens):
            t = 0
            while t < new:
                row = (n + t) % BLOCK
                m = min(BLOCK - row, new - t)
                group.setdefault((row, m), []).append((b, t))
                t += m
        for (row, m), at in group.items():
            b = torch.tensor([i[0] for i in at], device="cuda")
            t = torch.tensor([i[1] for i in at], device="cuda")
            rows = x[b[:, None], t[:, None] + torch.arange(m, device="cuda")]  # [n][m][Hk][D]
            block = slots[b, t] // BLOCK
            scale = _exact_scale(rows.abs().amax(dim=(1, 3)), code)
            if row:
                scale = torch.maximum(scale, scales[block])
                held = codes[block, :row] * scales[block][:, None, :, None]
                codes[block, :row] = _exact_code(held / scale[:, None, :, None], code)
            codes[block, row:row + m] = _exact_code(rows / scale[:, None, :, None], code)
            scales[block] = scale
        out[name] = codes if code == "e4m3" else codes.to(torch.int8)
        out[name + "s"] = scales
    return out


def _rows64(s, b, n):
    """Keys and values of sequence b's first n entries, [n][Hk][D] in 64 bits."""
    cache = s["case"].get("cache") or s["case"]["code"]
    t = s["tables"][b, :_blocks(n)].long()
    both = []
    for name, one in zip("kv", FP8_SCALES):
        x = s[name][t]
        if cache in CODE_MAX:
            x = _as_values(x, cache).double() * s[name + "s"][t].double()[:, None, :, None]
        elif cache == "fp8":
            x = x.view(torch.float8_e4m3fn).double() * one
        both.append(x.double().flatten(0, 1)[:n])
    return both


def _attend_exact(s):
    case = s["case"]
    H, Hk, D = case["H"], case["Hk"], case["D"]
    out = torch.zeros(case["B"], H, D, dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if case["op"] == "weights" else None
    for b, n in enumerate(_lens(case)):
        k, v = _rows64(s, b, n)
        q = s["q"][b].double().view(Hk, H // Hk, D)
        x = torch.einsum("hgd,nhd->hgn", q, k) * s["scale"]
        p = torch.softmax(x, dim=-1)
        out[b] = torch.einsum("hgn,nhd->hgd", p, v).reshape(H, D)
        if weights is not None:
            weights[b, :, :n] += p.sum(1)
    return out if weights is None else {"out": out, "weights": weights}


def _evict_exact(s):
    case = s["case"]
    keep, Hk, cache = case["keep"], case["Hk"], case["cache"]
    code = cache if cache in CODE_MAX else None
    kept, weights = torch.full_like(s["kept"], -1), torch.zeros_like(s["new_weights"], dtype=torch.float64)
    lens = _lens(case)
    pools = {}
    for name in "kv":
        x = s[name]
        pools[name] = (_as_values(x, code or "e4m3") if x.dtype in (torch.uint8, torch.int8) else x).double()
        if code:
            pools[name + "s"] = s[name + "s"].double()
    heads = torch.arange(Hk, device="cuda")
    for b, n in enumerate(lens):
        m = min(n, keep)
        w = s["weights"][b, :, :n]
        rank = w.double().clone()
        rank[:, :case["sinks"]] = math.inf
        rank[:, max(0, n - case["recent"]):] = math.inf
        index = torch.argsort(-rank, dim=1, stable=True)[:, :m].sort(dim=1).values  # [Hk][m]
        kept[b, :, :m] = index.int()
        weights[b, :, :m] = torch.gather(w, 1, index).double()
        src = s["tables"][b].long()[index // BLOCK]
        full = _blocks(m) * BLOCK
        to = s["dst"][b, :_blocks(m)].long()
        for name in "kv":
            x = (_as_values(s[name], code or "e4m3") if s[name].dtype in (torch.uint8, torch.int8) else s[name])
            x = x[src, index % BLOCK, heads[:, None]].double()  # [Hk][m][D]
            at = torch.arange(m, device="cuda")
            if code:
                x = x * s[name + "s"].double()[src, heads[:, None]][..., None]
                blocked = torch.nn.functional.pad(x, (0, 0, 0, full - m)).unflatten(1, (-1, BLOCK))
                scale = _exact_scale(blocked.abs().amax(dim=(2, 3)), code)  # [Hk][blocks]
                pools[name + "s"][to] = scale.t()
                x = _exact_code(x / scale[:, at // BLOCK][..., None], code)
            pools[name][to[at // BLOCK], at % BLOCK] = x.transpose(0, 1)
    if code == "int8":
        pools["k"], pools["v"] = pools["k"].to(torch.int8), pools["v"].to(torch.int8)
    return {"kept": kept, "lens": torch.tensor([min(n, keep) for n in lens], dtype=torch.int32, device="cuda"),
            "weights": weights} | pools
