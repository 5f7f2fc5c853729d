// Eviction by accumulated attention weight: which entries of each (sequence, KV head)
// stay, and the copy of those that do into other blocks.
//
// Kept: all of the first `sinks` and last `recent` entries, and of the others those
// with the largest weights, `keep` in all (ties to the lower index); everything when
// the context is no longer than `keep`. They go, in their order, to entries 0, 1, ...
// of the blocks of dst_block_tables, and their weights with them. Order is age, so
// `recent` keeps its meaning after any number of evictions; blocks shared with other
// sequences stay as they are; and since nothing is read that is written, all copies
// run at once.
#pragma once

#include <cooperative_groups.h>
#include <math_constants.h>

#include "block8.cuh"

namespace pa {

struct EvictParams {
    unsigned char *k_cache, *v_cache;
    float *k_scales, *v_scales;  // block8 pools
    const float *weights;        // [B][Hk][width]
    const int *block_tables, *context_lens, *dst_tables;
    float *new_weights;          // [B][Hk][dst_blocks * 16]
    int *new_lens;               // [B]
    int *kept;                   // [B][Hk][keep]
    long long num_blocks;
    int num_seqs, num_kv_heads, width, max_blocks, dst_blocks;
    int keep, sinks, recent, max_context_len;
};

__device__ __forceinline__ int evict_cap(const EvictParams &p) {
    return min(min(p.max_blocks * kBlockSize, p.max_context_len), p.width);
}

// Order of weights as unsigned: NaN lowest (with -inf), -0 as +0. Entries that always
// stay come above all.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) w = -CUDART_INF_F;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// ---- which entries stay ---------------------------------------------------------
//
// A radix select over the 32-bit keys, a bin a thread, finds the smallest kept key
// and how many of its equals stay (it ends early once all keys that share the digits so
// far stay); then warps count what they keep of their part of the row, a scan gives each
// its place, and a second look writes. A (sequence, KV head) is the work of one CTA, or
// of a cluster of up to 8 for long rows: each takes a contiguous share, adds the bins it
// has keys in to the first CTA's through distributed shared memory, and that one tells
// the others the digit. (Every CTA reading all the others' bins instead made the select
// of 64 rows of up to 32 K weights 109 us; one CTA a row took 42.) Bound by latency: up
// to four rounds of histogram, barrier and scan over a few thousand keys a CTA, which stay
// in shared memory, so that HBM sees the weights once. 64 sequences of 128 to 2048 entries
// with 8 KV heads: 14 to 15 us under ncu (512 threads and three rounds of 2048 bins were a
// microsecond slower); eight of 9 to 32 K: 27 to 28.
constexpr int kSelectShare = 4096;          // keys of a CTA, while 8 CTAs are enough for that
constexpr int kSelectKeys = 50 * 1024;      // keys a CTA's shared memory holds at most
constexpr int kSelectMaxCluster = 8;        // the portable cluster size

// Sum of v over the CTA's threads before this one; total over the CTA in `all`.
template <int WARPS>
__device__ __forceinline__ int scan_before(int v, int *warp_sums, int &all) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    int inc = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += t;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    const int w = lane < WARPS ? warp_sums[lane] : 0;
    all = __reduce_add_sync(0xffffffffu, w);
    return inc - v + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
}

// THREADS: 512, digits of 9 + 9 + 9 + 5 bits, or 256, four of 8. 2048 threads an SM: a CTA
// mostly waits (for loads, shared-memory atomics, barriers), and the rows of a batch of 64
// sequences with 8 KV heads then fit the GPU at once.
template <int THREADS>
__global__ void __launch_bounds__(THREADS, 2048 / THREADS) evict_select_kernel(const EvictParams prm, int keys_held) {
    extern __shared__ __align__(16) uint32_t select_keys[];
    constexpr int WARPS = THREADS / 32, BITS = THREADS == 512 ? 9 : 8;
    static_assert(THREADS == 1 << BITS, "a bin a thread");
    __shared__ int hist[THREADS];         // this CTA's keys
    __shared__ int total[THREADS];        // rank 0 of a cluster: all CTAs' keys
    __shared__ int warp_sums[WARPS];
    __shared__ int found[3];              // the digit, the keys above it, the keys in it
    __shared__ int counts[2];             // this CTA's keys above the threshold, and equal to it
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int u = blockIdx.x / ranks, b = u / prm.num_kv_heads;
    const int tix = threadIdx.x, warp = tix / 32, lane = tix % 32;
    const bool first = u % prm.num_kv_heads == 0 && rank == 0 && tix == 0;
    const int n = clamp_context(__ldg(prm.context_lens + b), evict_cap(prm), first);
    const float *w = prm.weights + static_cast<size_t>(u) * prm.width;
    int *kept = prm.kept + static_cast<size_t>(u) * prm.keep;
    const int new_width = prm.dst_blocks * kBlockSize;
    float *new_w = prm.new_weights + static_cast<size_t>(u) * new_width;
    const int m = min(n, prm.keep);
    const int tid = rank * THREADS + tix, threads = ranks * THREADS;
    if (first) prm.new_lens[b] = m;
    for (int i = m + tid; i < prm.keep; i += threads) kept[i] = -1;
    for (int i = m + tid; i < new_width; i += threads) new_w[i] = 0.f;
    if (n <= prm.keep) {  // the same for the whole cluster
        for (int i = tid; i < n; i += threads) {
            kept[i] = i;
            new_w[i] = __ldg(w + i);
        }
        return;
    }
    const int old = n - prm.recent;  // entries from here on always stay
    const int share = (n + ranks - 1) / ranks;
    const int lo = min(n, rank * share), hi = min(n, lo + share);
    const bool held = hi - lo <= keys_held;
    auto key_from = [&](int i, float x) -> uint32_t {
        return i < prm.sinks || i >= old ? 0xffffffffu : weight_key(x);
    };
    auto key_of = [&](int i) -> uint32_t { return key_from(i, __ldg(w + i)); };

    // a cluster: rank 0's totals start at zero before any peer adds to them
    int *sums = ranks > 1 ? cluster.map_shared_rank(total, 0) : total;
    if (ranks > 1) {
        if (rank == 0)
            total[tix] = 0;
        cluster.sync();
    }
    uint32_t prefix = 0, mask = 0;  // the smallest kept key's digits so far
    int need = prm.keep;            // keys to keep among those that share them
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int above_digit = 32 - BITS * pass, shift = max(0, above_digit - BITS);
        const int bins = 1 << (above_digit - shift);
        hist[tix] = 0;
        __syncthreads();
        if (pass == 0) {
            for (int i0 = lo + tix; i0 < hi; i0 += 4 * THREADS) {
                float x[4];  // loads in flight together
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = i0 + j * THREADS < hi ? __ldg(w + i0 + j * THREADS) : 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = i0 + j * THREADS;
                    if (i < hi) {
                        const uint32_t key = key_from(i, x[j]);
                        if (held) select_keys[i - lo] = key;
                        atomicAdd(&hist[key >> shift], 1);
                    }
                }
            }
        } else {
#pragma unroll 4
            for (int i = lo + tix; i < hi; i += THREADS) {
                const uint32_t key = held ? select_keys[i - lo] : key_of(i);
                if ((key & mask) == prefix) atomicAdd(&hist[key >> shift & (bins - 1)], 1);
            }
        }
        __syncthreads();
        int c = tix < bins ? hist[tix] : 0;
        if (ranks > 1) {
            if (c) atomicAdd(&sums[tix], c);
            cluster.sync();
        }
        if (rank == 0) {
            // thread t: bin t from the top; the digit is where the running count from the top
            // first reaches `need`
            const int bin = bins - 1 - tix;
            const int *h = ranks > 1 ? total : hist;
            c = bin >= 0 ? h[bin] : 0;
            int all;
            const int above = scan_before<WARPS>(c, warp_sums, all);
            if (above < need && above + c >= need) {  // one thread: its digit to every CTA
                for (int r = 0; r < ranks; ++r) {
                    int *f = ranks > 1 ? cluster.map_shared_rank(found, r) : found;
                    f[0] = bin;
                    f[1] = above;
                    f[2] = c;
                }
            }
            total[tix] = 0;  // for the next round (scan_before's barriers are behind every read)
        }
        if (ranks > 1) cluster.sync();
        else __syncthreads();
        prefix |= static_cast<uint32_t>(found[0]) << shift;
        mask |= static_cast<uint32_t>(bins - 1) << shift;
        need -= found[1];
        if (found[2] == need) break;  // all of them stay
    }

    // keys whose digits are above `prefix` stay, and the first `need` of those that share it
    const int span = (hi - lo + THREADS - 1) / THREADS * 32;  // entries of a warp, a multiple of 32
    const int wlo = min(hi, lo + warp * span), whi = min(hi, wlo + span);
    int gt = 0, eq = 0;
#pragma unroll 4
    for (int i = wlo + lane; i < whi; i += 32) {
        const uint32_t key = (held ? select_keys[i - lo] : key_of(i)) & mask;
        gt += key > prefix;
        eq += key == prefix;
    }
    int gt_all, eq_all;
    gt = __shfl_sync(0xffffffffu, scan_before<WARPS>(gt, warp_sums, gt_all), 0);  // of the warps before
    eq = __shfl_sync(0xffffffffu, scan_before<WARPS>(eq, warp_sums, eq_all), 0);
    if (ranks > 1) {  // and of the CTAs before
        if (tix == 0) {
            counts[0] = gt_all;
            counts[1] = eq_all;
        }
        cluster.sync();
        for (int r = 0; r < rank; ++r) {
            const int *peer = cluster.map_shared_rank(counts, r);
            gt += peer[0];
            eq += peer[1];
        }
    }
    const uint32_t below = (1u << lane) - 1;
#pragma unroll 4
    for (int i0 = wlo; i0 < whi; i0 += 32) {
        const int i = i0 + lane;
        const float x = i < whi ? __ldg(w + i) : 0.f;  // every entry's, so that loads run ahead of the counting
        const uint32_t key = i < whi ? (held ? select_keys[i - lo] : key_from(i, x)) & mask : 0u;
        const bool is_gt = i < whi && key > prefix, is_eq = i < whi && key == prefix;
        const uint32_t vg = __ballot_sync(0xffffffffu, is_gt), ve = __ballot_sync(0xffffffffu, is_eq);
        const int g = gt + __popc(vg & below), e = eq + __popc(ve & below);
        if (is_gt || (is_eq && e < need)) {
            const int at = g + min(e, need);
            kept[at] = i;
            new_w[at] = x;
        }
        gt += __popc(vg);
        eq += __popc(ve);
    }
    if (ranks > 1) cluster.sync();  // no CTA leaves while a peer may read its shared memory
}

// ---- the copy --------------------------------------------------------------------
//
// One warp per (sequence, new block, KV head), and for block8 pools K or V: 16 rows, each
// a contiguous D * E bytes of a source block, to 16 rows of the new one. Bound by HBM:
// 2 * rows * 2 * D * E bytes. A lane holds its 16-byte pieces of all 16 rows in registers,
// so that they are in flight together. (A persistent grid whose warps look up their next
// piece while they copy took longer, 48 against 39 us for the batch: the registers of the
// look-ahead cost more warps than it hides.) Measured: a bf16 batch of 64 sequences cut to 512
// entries, 249 MB, 37 to 39 us (6.4 to 6.7 TB/s); eight E4M3 contexts cut to 8191, 270 MB, 57
// to 60 us (4.5 to 4.7 TB/s). On one box 60 us, 58 with scales that need no re-coding, 54
// where neighbouring rows are kept, and 54 with both: neither is most of what it lacks.
//
// FMT >= 0 (block8): a new block's rows come from blocks of different scales; the new
// scale is the least power of two for its rows' largest magnitude, and the codes are
// divided by the ratio, as in the write. Codes widen exactly to f16, where their largest
// is found, and where a product with a power of two from 2^-24 to 2^15 rounds once, to
// the new code (below 2^-24 every code becomes 0, as there). Other ratios, which only
// scales that are not powers of two or far apart have, go through fp32.

// 16 codes of one row times ratio (exact in f16) to codes.
template <int FMT>
__device__ __forceinline__ uint4 rescale16(const uint32_t (&h)[8], float ratio) {
    const __half2 r2 = __float2half2_rn(ratio);
    const uint32_t r = *reinterpret_cast<const uint32_t *>(&r2);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (FMT == kBlockE4M3) {
            asm("{\n\t.reg .b32 a, b;\n\t.reg .b16 x, y;\n\t"
                "mul.rn.f16x2 a, %1, %3;\n\t"
                "mul.rn.f16x2 b, %2, %3;\n\t"
                "cvt.rn.satfinite.e4m3x2.f16x2 x, a;\n\t"
                "cvt.rn.satfinite.e4m3x2.f16x2 y, b;\n\t"
                "mov.b32 %0, {x, y};\n\t}"
                : "=r"(w[i])
                : "r"(h[2 * i]), "r"(h[2 * i + 1]), "r"(r));
        } else {
            // code * ratio + 1536 in one rounding: an f16 whose unit is 1, its low byte the code
            uint32_t a, b;
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(a) : "r"(h[2 * i]), "r"(r), "r"(0x66006600u));
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(b) : "r"(h[2 * i + 1]), "r"(r), "r"(0x66006600u));
            w[i] = __byte_perm(a, b, 0x6420);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int FMT>
__device__ __forceinline__ void widen16(const uint4 &v, uint32_t (&h)[8]) {
    widen4_f16<FMT>(v.x, h[0], h[1]);
    widen4_f16<FMT>(v.y, h[2], h[3]);
    widen4_f16<FMT>(v.z, h[4], h[5]);
    widen4_f16<FMT>(v.w, h[6], h[7]);
}

// The same through fp32, for any finite ratio. Rare, and out of line: its registers
// would cost the copy a third of its warps.
template <int FMT>
__device__ __noinline__ uint4 rescale16_any(uint4 v, float ratio) {
    uint32_t h[8], w[4];
    widen16<FMT>(v, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&h[2 * i]));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&h[2 * i + 1]));
        w[i] = encode4<FMT>(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The largest |code| of 16, NaN aside.
__device__ __forceinline__ float largest16(const uint32_t (&h)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("max.xorsign.abs.f16x2 %0, %0, %1;" : "+r"(top) : "r"(h[i]));
    top &= 0x7fff7fffu;
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&top));
    return fmaxf(f.x, f.y);
}

__device__ __forceinline__ bool power_of_two(float x) { return (__float_as_uint(x) & 0x807fffffu) == 0; }

template <int ROW, int FMT>
__device__ __forceinline__ void copy_rows(unsigned char *pool, float *scales, int kept, int rows, int src_blk,
                                          long long dst_blk, int Hk, int hk) {
    constexpr int L = ROW / 16;             // lanes of a row
    constexpr int RS = 32 / L;              // rows a step
    constexpr int STEPS = kBlockSize / RS;
    static_assert(L <= 32, "a row is one 16-byte piece of up to 32 lanes");
    const int lane = threadIdx.x % 32, j = lane % L, rg = lane / L;
    const size_t pitch = static_cast<size_t>(Hk) * ROW;
    uint4 v[STEPS];
    float s[STEPS];  // block8: the row's scale
    float mine = 0.f;  // lane t: row t's
    if constexpr (FMT >= 0) {
        if (lane < rows && src_blk >= 0) mine = __ldcg(scales + static_cast<size_t>(src_blk) * Hk + hk);
    }
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
        const int t = st * RS + rg;
        const int e = __shfl_sync(0xffffffffu, kept, t), sb = __shfl_sync(0xffffffffu, src_blk, t);
        v[st] = make_uint4(0u, 0u, 0u, 0u);
        if (t < rows && sb >= 0)
            v[st] = __ldcs(reinterpret_cast<const uint4 *>(
                pool + (static_cast<size_t>(sb) * kBlockSize + e % kBlockSize) * pitch + hk * ROW + j * 16));
    }
#pragma unroll
    for (int st = 0; st < STEPS; ++st) s[st] = FMT >= 0 ? __shfl_sync(0xffffffffu, mine, st * RS + rg) : 0.f;
    if constexpr (FMT >= 0) {
        float amax = 0.f;
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
            uint32_t h[8];
            widen16<FMT>(v[st], h);
            // a finite code times a finite scale may pass fp32's range (the write makes 256 * 2^120)
            amax = fmaxf(amax, fminf(largest16(h) * s[st], kLargestFloat));
        }
        const int e = scale_exponent<FMT>(warp_max(amax));
        const float scale = exp2_int(e), inv = exp2_int(-e);
        if (lane == 0) scales[dst_blk * Hk + hk] = scale;
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
            const float ratio = s[st] * inv;
            if (ratio == 1.f) continue;
            if (power_of_two(ratio) && ratio <= 0x1p15f && s[st] <= 0x1p120f) {
                uint32_t h[8];
                widen16<FMT>(v[st], h);
                v[st] = rescale16<FMT>(h, fmaxf(ratio, 0x1p-24f));
            } else {
                // an infinite ratio has codes of zero only: the new scale holds every other
                v[st] = rescale16_any<FMT>(v[st], fminf(ratio, kLargestFloat));
            }
        }
    }
    unsigned char *dst = pool + static_cast<size_t>(dst_blk) * kBlockSize * pitch + hk * ROW + j * 16;
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
        const int t = st * RS + rg;
        const int sb = __shfl_sync(0xffffffffu, src_blk, t);
        if (t < rows && sb >= 0) __stcs(reinterpret_cast<uint4 *>(dst + t * pitch), v[st]);
    }
}

// Grid: x (sequence, new block), y four warps' pieces each.
template <int ROW, int FMT>
__global__ void __launch_bounds__(128, FMT >= 0 ? 8 : 1) evict_copy_kernel(const EvictParams prm) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the selection
    const int lane = threadIdx.x % 32, Hk = prm.num_kv_heads;
    const int part = blockIdx.y * 4 + threadIdx.x / 32;
    if (part >= (FMT >= 0 ? 2 * Hk : Hk)) return;
    const int hk = part < Hk ? part : part - Hk;
    const unsigned b = blockIdx.x / static_cast<unsigned>(prm.dst_blocks);
    const int blk = static_cast<int>(blockIdx.x - b * prm.dst_blocks);
    const int n = clamp_context(__ldg(prm.context_lens + b), evict_cap(prm), false);
    const int rows = min(min(n, prm.keep) - blk * kBlockSize, kBlockSize);
    if (rows <= 0) return;
    const long long dst = __ldg(prm.dst_tables + blockIdx.x);
    // lane t < rows: the entry that row t holds, and its block
    int kept = 0, src = -1;
    if (lane < rows) {
        kept = __ldcg(prm.kept + (static_cast<size_t>(b) * Hk + hk) * prm.keep + blk * kBlockSize + lane);
        src = __ldg(prm.block_tables + static_cast<size_t>(b) * prm.max_blocks + kept / kBlockSize);
        if (src < 0 || src >= prm.num_blocks) {
            flag_status(PA_STATUS_BAD_BLOCK_ID);
            src = -1;
        }
    }
    if (dst < 0 || dst >= prm.num_blocks) {
        if (lane == 0) flag_status(PA_STATUS_BAD_BLOCK_ID);
        return;
    }
    if constexpr (FMT >= 0) {
        const bool k = part < Hk;
        copy_rows<ROW, FMT>(k ? prm.k_cache : prm.v_cache, k ? prm.k_scales : prm.v_scales, kept, rows, src, dst, Hk, hk);
    } else {
        copy_rows<ROW, FMT>(prm.k_cache, nullptr, kept, rows, src, dst, Hk, hk);
        copy_rows<ROW, FMT>(prm.v_cache, nullptr, kept, rows, src, dst, Hk, hk);
    }
}

}  // namespace pa
