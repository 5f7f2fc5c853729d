// Rotary positions: rotate q and the new tokens' k by position, and put the
// rotated k with v straight into the paged cache.
//
// The first rot_dim dims of a head are pairs (x, y), turned by the angle
// a = position * f_i: x' = x cos a - y sin a, y' = y cos a + x sin a. The pairs
// are (i, i + rot_dim / 2) in the half layout, (2i, 2i + 1) in the interleaved one.
//
// Angles. f_i reaches the kernel as the fraction of a turn per position in 64-bit
// fixed point (pa_rope_plan.step), so position * step mod 2^64 is the angle's
// fraction of a turn for any position: integer wrap-around is the range reduction,
// exact, where a 32-bit product of a position in the millions would be off by
// hundredths of a radian. The quarter turns come off in integers too, so that what is
// rounded to fp32 for sincospif is at most an eighth of a turn: off by 2^-24 of itself,
// at most 2^-28 of a turn, less than the step of an fp32 cosine. (Half a turn would be
// off by 2^-26 of a turn, more than that step.)
//
// Bound by memory: a token moves 2 H D (q) + 4 Hk D (k, v) elements and computes
// rot_dim / 2 angles, shared by all heads. A CTA takes four tokens (one when there are few,
// with more CTAs to a token while they would leave SMs idle): its threads issue their
// first loads, then compute the tokens' angles once into shared memory while those fly.
// 8192 tokens of 32 + 2 * 8 heads of 128 in bf16: 35.4 us, 0.87 of the measured copy
// bandwidth (a token a CTA of 384 threads, one unit a thread: 45.8 us, waiting for angles).
// One token: 2.7 us.

#pragma once

#include <cstring>

#include "pa_common.cuh"

namespace pa {

struct RopeParams {
    const void *q, *k, *v;           // rows of [heads][D], token strides below
    void *q_out;                     // [T][H][D]
    void *k_out, *v_out;             // the caches, or k_out [T][Hk][D] and no v
    const int64_t *slot_mapping;     // null: k_out is [T][Hk][D]
    const int64_t *positions;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    int64_t num_slots, num_tokens;
    int num_heads, num_kv_heads;
    float k_inv, v_inv;              // 1 / scale of an FP8 cache
    pa_rope_plan plan;
};

// V elements in 16 bytes, to and from fp32.
__device__ __forceinline__ void widen_vec(const uint4 &r, float (&f)[8]) { Widen<__nv_bfloat16>::apply(r, f); }
__device__ __forceinline__ void widen_vec(const uint4 &r, float (&f)[4]) { Widen<float>::apply(r, f); }
__device__ __forceinline__ uint4 narrow_vec(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 narrow_vec(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint2 e4m3_vec(const float (&f)[8], float inv) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = f32x2_to_e4m3x2(f[2 * i] * inv, f[2 * i + 1] * inv);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;  // tokens of a CTA at most

// T: float or bf16. FP8: the caches hold E4M3 codes (T is bf16); the rotated k is
// quantized from fp32, without a rounding to bf16 in between.
// A unit is two 16-byte vectors of one head: for a rotated pair column u the
// vectors that hold its x and its y (half layout) or two neighbours (interleaved,
// and dims past rot_dim, which pass through). A thread keeps its column u and goes
// through the rows (q's, k's and v's heads of each of the CTA's tokens), two at a time.
// Grid: x groups of `tokens` tokens, y parts of their rows.
template <typename T, bool FP8, int D>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams prm, int tokens) {
    constexpr int V = 16 / sizeof(T);             // elements of a vector
    constexpr int UNITS = D / V / 2;              // units of a head
    constexpr int ROWS = kRopeThreads / UNITS;    // rows the CTA takes at once
    // (cos, sin) of pair u * V + i at i * UNITS + u: neighbouring threads read neighbouring entries
    __shared__ float2 turn[kRopeTokens][D / 2];
    __shared__ int64_t slots[kRopeTokens];
    // a paged decode that follows is a programmatic dependent: it may launch now and waits for this grid
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens;
    const int count = static_cast<int>(min(static_cast<int64_t>(tokens), prm.num_tokens - t0));
    const int H = prm.num_heads, Hk = prm.num_kv_heads, heads = H + Hk + (prm.v ? Hk : 0);
    const int half = prm.plan.rot_dim / 2, u = threadIdx.x % UNITS;
    const bool split = !prm.plan.interleaved, turns = u * V < half;
    // first elements of the two vectors, in rows that are rotated and in v's
    const int e0 = split && turns ? u * V : 2 * u * V, e1 = split && turns ? u * V + half : e0 + V;

    struct Row {
        int t, head;  // of the CTA's tokens; of q's, k's, v's heads in a line
        uint4 a, b;
    };
    const int step = ROWS * gridDim.y;
    Row next{0, static_cast<int>(blockIdx.y) * ROWS + static_cast<int>(threadIdx.x) / UNITS, {}, {}};
    auto settle = [&]() {
        while (next.head >= heads) {
            next.head -= heads;
            ++next.t;
        }
    };
    auto fetch = [&]() {  // the row at `next`, which moves on
        Row r = next;
        if (r.t < count) {
            const int64_t t = t0 + r.t;
            const T *p;
            if (r.head < H) p = static_cast<const T *>(prm.q) + t * prm.q_stride + r.head * D;
            else if (r.head < H + Hk) p = static_cast<const T *>(prm.k) + t * prm.k_stride + (r.head - H) * D;
            else p = static_cast<const T *>(prm.v) + t * prm.v_stride + (r.head - H - Hk) * D;
            const bool v = r.head >= H + Hk;
            r.a = __ldcs(reinterpret_cast<const uint4 *>(p + (v ? 2 * u * V : e0)));
            r.b = __ldcs(reinterpret_cast<const uint4 *>(p + (v ? 2 * u * V + V : e1)));
        }
        next.head += step;
        settle();
        return r;
    };
    settle();
    Row r0 = fetch(), r1 = fetch();
    for (int i = threadIdx.x; i < count * half; i += kRopeThreads) {
        const int t = i / half, f = i - t * half;
        const uint64_t phase = static_cast<uint64_t>(__ldg(prm.positions + t0 + t)) * prm.plan.step[f];
        // the nearest quarter of a turn, and the signed rest: an eighth of a turn at most, rounded to fp32
        const int quarter = static_cast<int>((phase + (1ull << 61)) >> 62);
        const int64_t rest = static_cast<int64_t>(phase - (static_cast<uint64_t>(quarter) << 62));
        float s, c;
        sincospif(static_cast<float>(rest) * 0x1p-63f, &s, &c);
        if (quarter & 1) {
            const float x = c;
            c = -s;
            s = x;
        }
        if (quarter & 2) {
            c = -c;
            s = -s;
        }
        turn[t][f % V * UNITS + f / V] = make_float2(c * prm.plan.mscale, s * prm.plan.mscale);
    }
    if (threadIdx.x < count) {
        int64_t slot = t0 + threadIdx.x;
        if (prm.slot_mapping) {
            slot = __ldg(prm.slot_mapping + slot);
            if (slot >= prm.num_slots) {
                if (blockIdx.y == 0) flag_status(PA_STATUS_BAD_SLOT);
                slot = -1;
            }
        }
        slots[threadIdx.x] = slot;
    }
    __syncthreads();
    auto finish = [&](const Row &r) {
        if (r.t >= count) return;
        const bool is_v = r.head >= H + Hk;
        float a[V], b[V];
        widen_vec(r.a, a);
        widen_vec(r.b, b);
        if (turns && !is_v) {
            const float2 *cs = turn[r.t] + u;
            if (split) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float2 p = cs[i * UNITS];
                    const float x = a[i], y = b[i];
                    a[i] = x * p.x - y * p.y;
                    b[i] = y * p.x + x * p.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    const float2 p = cs[i / 2 * UNITS], w = cs[(V + i) / 2 * UNITS];
                    const float x = a[i], y = a[i + 1], z = b[i], v = b[i + 1];
                    a[i] = x * p.x - y * p.y;
                    a[i + 1] = y * p.x + x * p.y;
                    b[i] = z * w.x - v * w.y;
                    b[i + 1] = v * w.x + z * w.y;
                }
            }
        }
        const int f0 = is_v ? 2 * u * V : e0, f1 = is_v ? 2 * u * V + V : e1;
        if (r.head < H) {
            T *o = static_cast<T *>(prm.q_out) + ((t0 + r.t) * H + r.head) * D;
            *reinterpret_cast<uint4 *>(o + f0) = narrow_vec(a);
            *reinterpret_cast<uint4 *>(o + f1) = narrow_vec(b);
            return;
        }
        const int64_t slot = slots[r.t];
        if (slot < 0) return;  // padding
        const int hk = r.head - H - (is_v ? Hk : 0);
        const int64_t row = (slot * Hk + hk) * D;
        if constexpr (FP8) {
            const float inv = is_v ? prm.v_inv : prm.k_inv;
            uint8_t *o = static_cast<uint8_t *>(is_v ? prm.v_out : prm.k_out) + row;
            *reinterpret_cast<uint2 *>(o + f0) = e4m3_vec(a, inv);
            *reinterpret_cast<uint2 *>(o + f1) = e4m3_vec(b, inv);
        } else {
            T *o = static_cast<T *>(is_v ? prm.v_out : prm.k_out) + row;
            *reinterpret_cast<uint4 *>(o + f0) = narrow_vec(a);
            *reinterpret_cast<uint4 *>(o + f1) = narrow_vec(b);
        }
    };
    while (r0.t < count) {
        const Row a = r0, b = r1;
        r0 = fetch();
        r1 = fetch();
        finish(a);
        finish(b);
    }
}

}  // namespace pa
