"""64-bit references of the cache operators, written from their definitions (numpy, one sequence at a time).

Pools here are numpy arrays: codes uint8 (E4M3) or int8 [NB, 16, Hk, D], scales float32 [NB, Hk]; plain pools are
float64 values.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 16
CODE_MAX = {"e4m3": 448.0, "int8": 127.0}


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _e4m3_table():
    out = np.zeros(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = math.nan if (c & 127) == 127 else (-v if c & 128 else v)
    return out


E4M3 = _e4m3_table()


def values(codes, code):
    return E4M3[codes] if code == "e4m3" else codes.astype(np.float64)


def encode(x, code):
    """Nearest code, ties to even, saturating; NaN is E4M3's NaN (0x7f or 0xff) or 0."""
    x = np.asarray(x, np.float64)
    if code == "int8":
        return np.where(np.isnan(x), 0, np.clip(np.round(np.nan_to_num(x, posinf=1e9, neginf=-1e9)), -127, 127)).astype(np.int8)
    a = np.minimum(np.abs(np.nan_to_num(x, posinf=1e9, neginf=-1e9)), 448.0)
    _, e = np.frexp(a)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))
    r = np.round(a / step) * step
    mag = np.searchsorted(E4M3[:127], r).astype(np.uint8)
    assert np.array_equal(E4M3[mag], r)
    return np.where(np.isnan(x), 0x7F, mag | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)).astype(np.uint8)


def least_scale(x, code):
    """The least power of two s in [2^-64, 2^120] with |x| <= CODE_MAX s over the finite x."""
    a = np.abs(x[np.isfinite(x)])
    top = float(a.max()) if a.size else 0.0
    e = -64
    while top > CODE_MAX[code] * 2.0 ** e and e < 120:
        e += 1
    return 2.0 ** e


def quantized_pool(x, code):
    """Codes and scales of whole blocks of float64 values [NB, 16, Hk, D]."""
    nb, _, hk, _ = x.shape
    scales = np.array([[least_scale(x[b, :, h], code) for h in range(hk)] for b in range(nb)])
    return encode(x / scales[:, None, :, None], code), scales.astype(np.float32)


def write(x, codes, scales, slots, code):
    """pa_cache_block8 for one of K and V: (codes, scales) after x float64 [T, Hk, D] goes to its slots."""
    codes, scales = codes.copy(), scales.copy()
    groups = {}
    for t, s in enumerate(slots):
        if 0 <= s < codes.shape[0] * BLOCK:
            groups.setdefault(int(s) // BLOCK, []).append((int(s) % BLOCK, t))
    for b, rows in groups.items():
        first = min(r for r, _ in rows)
        for h in range(codes.shape[2]):
            new = np.stack([x[t, h] for _, t in rows])
            s = least_scale(new, code)
            if first > 0:
                old = float(scales[b, h])
                s = max(s, old)
                if s > old:
                    codes[b, :first, h] = encode(values(codes[b, :first, h], code) * (old / s), code)
            for r, t in rows:
                codes[b, r, h] = encode(x[t, h] / s, code)
            scales[b, h] = s
    return codes, scales


def dequantized(codes, scales, code):
    return values(codes, code) * scales.astype(np.float64)[:, None, :, None]


def attend(q, k, v, tables, lens, scale, v_scales=None):
    """Per sequence: out [H, D], p [H, n], and what error bounds need: A = sum_i p_i |v_i| [H, D],
    S = max_i scale sum_d |q_d k_id| [H] and, with a block8 pool's v_scales, U = n * 448 * max_i p_i v_scale_i [H].
    k, v: float64 pools of values."""
    hk = k.shape[2]
    out = []
    for b, n in enumerate(lens):
        g = q.shape[1] // hk
        H, D = q.shape[1:]
        if n == 0:
            out.append((np.zeros((H, D)), np.zeros((H, 0)), np.zeros((H, D)), np.zeros(H), np.zeros(H)))
            continue
        t = tables[b][:blocks(n)]
        kk, vv = k[t].reshape(-1, hk, D)[:n], v[t].reshape(-1, hk, D)[:n]
        o, p, a, s, u = np.zeros((H, D)), np.zeros((H, n)), np.zeros((H, D)), np.zeros(H), np.zeros(H)
        for h in range(H):
            x = kk[:, h // g] @ q[b, h] * scale
            e = np.exp(x - x.max())
            p[h] = e / e.sum()
            o[h] = p[h] @ vv[:, h // g]
            a[h] = p[h] @ np.abs(vv[:, h // g])
            s[h] = (np.abs(kk[:, h // g]) @ np.abs(q[b, h])).max() * abs(scale)
            if v_scales is not None:
                u[h] = n * 448 * (p[h] * np.repeat(v_scales[t, h // g].astype(np.float64), BLOCK)[:n]).max()
        out.append((o, p, a, s, u))
    return out


def select(w, n, keep, sinks, recent):
    """Indices that one (sequence, KV head) keeps, in order."""
    if n <= keep:
        return np.arange(n)
    rank = np.where(np.isnan(w[:n]), -np.inf, w[:n].astype(np.float64))
    always = (np.arange(n) < sinks) | (np.arange(n) >= n - recent)
    order = sorted(range(n), key=lambda i: (not always[i], -rank[i], i))
    return np.sort(np.array(order[:keep], dtype=np.int64))


def rotate(x, pos, rot, interleaved, freq, mscale):
    """x float64 [T, heads, D] rotated; freq float64 [rot / 2]."""
    y = x.copy()
    a = pos.astype(np.float64)[:, None, None] * freq
    c, s = np.cos(a) * mscale, np.sin(a) * mscale
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, low=1.0, high=32.0, original_len=0.0):
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        t = np.clip((original_len * f / (2 * math.pi) - low) / (high - low), 0, 1)
        f = t * f + (1 - t) * f / factor
    return f
