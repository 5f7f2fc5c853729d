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
// One CTA per (sequence, KV head): a radix select over the 32-bit keys, 11 + 11 + 10
// bits, finds the smallest kept key and how many of its equals stay; then warps count
// what they keep of their part of the row, a scan gives each its place, and a second
// look writes. Bound by latency (a row of 32 K weights is 128 KB); the row's keys stay in
// shared memory when they fit, so HBM sees them once.
constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kSelectBins = 2048;
constexpr int kSelectKeys = 50 * 1024;  // keys held in shared memory

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictParams prm, int keys_held) {
    extern __shared__ __align__(16) uint32_t select_keys[];
    __shared__ int hist[kSelectBins];
    __shared__ int warp_a[kSelectWarps], warp_b[kSelectWarps];
    __shared__ int found[2];  // the digit, and the keys above it
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int u = blockIdx.x, b = u / prm.num_kv_heads;
    const int tix = threadIdx.x, warp = tix / 32, lane = tix % 32;
    const int n = clamp_context(__ldg(prm.context_lens + b), evict_cap(prm), u % prm.num_kv_heads == 0 && tix == 0);
    const float *w = prm.weights + static_cast<size_t>(u) * prm.width;
    int *kept = prm.kept + static_cast<size_t>(u) * prm.keep;
    const int new_width = prm.dst_blocks * kBlockSize;
    float *new_w = prm.new_weights + static_cast<size_t>(u) * new_width;
    const int m = min(n, prm.keep);
    if (u % prm.num_kv_heads == 0 && tix == 0) prm.new_lens[b] = m;
    for (int i = m + tix; i < prm.keep; i += kSelectThreads) kept[i] = -1;
    for (int i = m + tix; i < new_width; i += kSelectThreads) new_w[i] = 0.f;
    if (n <= prm.keep) {
        for (int i = tix; i < n; i += kSelectThreads) {
            kept[i] = i;
            new_w[i] = __ldg(w + i);
        }
        return;
    }
    const int old = n - prm.recent;  // entries from here on always stay
    const bool held = n <= keys_held;
    auto key_of = [&](int i) -> uint32_t {
        return i < prm.sinks || i >= old ? 0xffffffffu : weight_key(__ldg(w + i));
    };
    if (held)
        for (int i = tix; i < n; i += kSelectThreads) select_keys[i] = key_of(i);

    uint32_t prefix = 0, mask = 0;  // the smallest kept key's digits so far
    int need = prm.keep;            // keys to keep among those that share them
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const int bins = pass == 2 ? 1024 : 2048;
        for (int i = tix; i < bins; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
        for (int i = tix; i < n; i += kSelectThreads) {
            const uint32_t key = held ? select_keys[i] : key_of(i);
            if ((key & mask) == prefix) atomicAdd(&hist[key >> shift & (bins - 1)], 1);
        }
        __syncthreads();
        // thread t: the bins / 1024 bins from the top; the digit is where the running
        // count from the top first reaches `need`
        const int per = bins / kSelectThreads;
        int c[2] = {0, 0}, sum = 0;
        for (int i = 0; i < per; ++i) {
            c[i] = hist[bins - 1 - (tix * per + i)];
            sum += c[i];
        }
        int inc = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += t;
        }
        if (lane == 31) warp_a[warp] = inc;
        __syncthreads();
        if (warp == 0) {
            int t = warp_a[lane];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int p = __shfl_up_sync(0xffffffffu, t, off);
                if (lane >= off) t += p;
            }
            warp_b[lane] = t;
        }
        __syncthreads();
        int above = inc - sum + (warp ? warp_b[warp - 1] : 0);
        for (int i = 0; i < per; ++i) {
            if (above < need && above + c[i] >= need) {
                found[0] = bins - 1 - (tix * per + i);
                found[1] = above;
            }
            above += c[i];
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(found[0]) << shift;
        mask |= static_cast<uint32_t>(bins - 1) << shift;
        need -= found[1];
        __syncthreads();
    }

    // keys above `prefix` stay, and the first `need` equal to it
    const int span = (n + kSelectThreads - 1) / kSelectThreads * 32;  // entries of a warp, a multiple of 32
    const int lo = warp * span, hi = min(n, lo + span);
    int gt = 0, eq = 0;
    for (int i = lo + lane; i < hi; i += 32) {
        const uint32_t key = held ? select_keys[i] : key_of(i);
        gt += key > prefix;
        eq += key == prefix;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        warp_a[warp] = gt;
        warp_b[warp] = eq;
    }
    __syncthreads();
    gt = __reduce_add_sync(0xffffffffu, lane < warp ? warp_a[lane] : 0);
    eq = __reduce_add_sync(0xffffffffu, lane < warp ? warp_b[lane] : 0);
    const uint32_t below = (1u << lane) - 1;
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t key = i < hi ? (held ? select_keys[i] : key_of(i)) : 0u;
        const bool is_gt = i < hi && key > prefix, is_eq = i < hi && key == prefix;
        const uint32_t vg = __ballot_sync(0xffffffffu, is_gt), ve = __ballot_sync(0xffffffffu, is_eq);
        const int g = gt + __popc(vg & below), e = eq + __popc(ve & below);
        if (is_gt || (is_eq && e < need)) {
            const int at = g + min(e, need);
            kept[at] = i;
            new_w[at] = __ldg(w + i);
        }
        gt += __popc(vg);
        eq += __popc(ve);
    }
}

// ---- the copy --------------------------------------------------------------------
//
// One warp per (sequence, new block, KV head): 16 rows of K and V, each a contiguous
// D * E bytes of a source block, to 16 rows of the new one. Bound by HBM: 2 * rows *
// 2 * D * E bytes. A lane holds its 16-byte pieces of all 16 rows of K (then of V)
// in registers, so that they are in flight together.
//
// FMT >= 0 (block8): a new block's rows come from blocks of different scales; the new
// scale is the least power of two for its rows' largest magnitude, and the codes are
// divided by the ratio, as in the write.
template <int ROW, int FMT>
__device__ __forceinline__ void copy_rows(unsigned char *pool, float *scales, int kept, int rows, int src_blk,
                                          long long dst_blk, int Hk, int hk) {
    constexpr int L = ROW / 16 < 32 ? ROW / 16 : 32;  // lanes of a row
    constexpr int RS = 32 / L;                         // rows a step
    constexpr int STEPS = kBlockSize / RS;
    constexpr int VPL = ROW / 16 / L;                  // 16-byte pieces of a row per lane
    const int lane = threadIdx.x % 32, j = lane % L, rg = lane / L;
    const size_t pitch = static_cast<size_t>(Hk) * ROW;
    uint4 v[STEPS][VPL];
    float s[STEPS];  // block8: the row's scale
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
        const int t = st * RS + rg;
        const int e = __shfl_sync(0xffffffffu, kept, t), sb = __shfl_sync(0xffffffffu, src_blk, t);
        if (t < rows && sb >= 0) {
            const unsigned char *p =
                pool + (static_cast<size_t>(sb) * kBlockSize + e % kBlockSize) * pitch + hk * ROW + j * 16;
#pragma unroll
            for (int i = 0; i < VPL; ++i) v[st][i] = __ldcs(reinterpret_cast<const uint4 *>(p + i * L * 16));
            if constexpr (FMT >= 0) s[st] = __ldcg(scales + static_cast<size_t>(sb) * Hk + hk);
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) v[st][i] = make_uint4(0u, 0u, 0u, 0u);
            s[st] = 0.f;
        }
    }
    float scale = 1.f;
    if constexpr (FMT >= 0) {
        float amax = 0.f;
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
            const uint32_t w[4] = {v[st][0].x, v[st][0].y, v[st][0].z, v[st][0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float f[4];
                widen4_f32<FMT < 0 ? 0 : FMT>(w[i], f);
#pragma unroll
                for (int e = 0; e < 4; ++e) amax = fmaxf(amax, finite_abs(f[e] * s[st]));
            }
        }
        scale = exp2_int(scale_exponent<FMT < 0 ? 0 : FMT>(warp_max(amax)));
        if (lane == 0) scales[dst_blk * Hk + hk] = scale;
    }
    unsigned char *dst = pool + static_cast<size_t>(dst_blk) * kBlockSize * pitch + hk * ROW + j * 16;
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
        const int t = st * RS + rg;
        const int sb = __shfl_sync(0xffffffffu, src_blk, t);
        if (t >= rows || sb < 0) continue;
        if constexpr (FMT >= 0) {
            if (s[st] != scale) {
                const float inv = 1.f / scale;
                uint32_t w[4] = {v[st][0].x, v[st][0].y, v[st][0].z, v[st][0].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float f[4];
                    widen4_f32<FMT < 0 ? 0 : FMT>(w[i], f);
                    w[i] = encode4<FMT < 0 ? 0 : FMT>(f[0] * s[st] * inv, f[1] * s[st] * inv, f[2] * s[st] * inv,
                                                      f[3] * s[st] * inv);
                }
                v[st][0] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) __stcs(reinterpret_cast<uint4 *>(dst + t * pitch + i * L * 16), v[st][i]);
    }
}

template <int ROW, int FMT>
__global__ void __launch_bounds__(128) evict_copy_kernel(const EvictParams prm) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the selection
    const int lane = threadIdx.x % 32, Hk = prm.num_kv_heads;
    const long long item = static_cast<long long>(blockIdx.x) * 4 + threadIdx.x / 32;
    const int hk = static_cast<int>(item % Hk);
    const long long bb = item / Hk;
    const int blk = static_cast<int>(bb % prm.dst_blocks);
    const long long b = bb / prm.dst_blocks;
    if (b >= prm.num_seqs) return;
    const int n = clamp_context(__ldg(prm.context_lens + b), evict_cap(prm), false);
    const int rows = min(min(n, prm.keep) - blk * kBlockSize, kBlockSize);
    if (rows <= 0) return;
    const long long dst = __ldg(prm.dst_tables + b * prm.dst_blocks + blk);
    // lane t < rows: the entry that row t holds, and its block
    int kept = 0, src = -1;
    if (lane < rows) {
        kept = __ldcg(prm.kept + (b * Hk + hk) * prm.keep + blk * kBlockSize + lane);
        src = __ldg(prm.block_tables + b * prm.max_blocks + kept / kBlockSize);
        if (src < 0 || src >= prm.num_blocks) {
            flag_status(PA_STATUS_BAD_BLOCK_ID);
            src = -1;
        }
    }
    if (dst < 0 || dst >= prm.num_blocks) {
        if (lane == 0) flag_status(PA_STATUS_BAD_BLOCK_ID);
        return;
    }
    copy_rows<ROW, FMT>(prm.k_cache, prm.k_scales, kept, rows, src, dst, Hk, hk);
    copy_rows<ROW, FMT>(prm.v_cache, prm.v_scales, kept, rows, src, dst, Hk, hk);
}

}  // namespace pa
