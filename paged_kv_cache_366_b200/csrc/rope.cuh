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
// hundredths of a radian. The top 32 bits go through sincospif.
//
// Bound by memory: a token moves 2 H D (q) + 4 Hk D (k, v) elements and computes
// rot_dim / 2 angles, shared by all heads. One CTA a token (more when few tokens
// would leave SMs idle, each taking some of the heads): its threads issue their
// loads, then compute the token's angles once in shared memory while they fly.
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
    int64_t num_slots;
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

constexpr int kRopeThreads = 384;  // 32 + 2 * 8 heads of 128 bf16: one unit each

// T: float or bf16. FP8: the caches hold E4M3 codes (T is bf16); the rotated k is
// quantized from fp32, without a rounding to bf16 in between.
// A unit is two 16-byte vectors of one head: for a rotated pair column u the
// vectors that hold its x and its y (half layout) or two neighbours (interleaved,
// and dims past rot_dim, which pass through).
template <typename T, bool FP8, int D>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams prm) {
    constexpr int V = 16 / sizeof(T);    // elements of a vector
    constexpr int UNITS = D / V / 2;     // units of a head
    // (cos, sin) of pair u * V + i at i * UNITS + u: neighbouring threads read neighbouring entries
    __shared__ float2 turn[D / 2];
    // a paged decode that follows is a programmatic dependent: it may launch now and waits for this grid
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t t = blockIdx.x;
    const int H = prm.num_heads, Hk = prm.num_kv_heads;
    const int rot = prm.plan.rot_dim, half = rot / 2;
    const bool split = !prm.plan.interleaved;
    int64_t slot = t;
    if (prm.slot_mapping) {
        slot = __ldg(prm.slot_mapping + t);
        if (slot >= prm.num_slots) {
            if (blockIdx.y == 0 && threadIdx.x == 0) flag_status(PA_STATUS_BAD_SLOT);
            slot = -1;
        }
    }
    // items: the units of q's heads, of k's and of v's
    const int total = (H + Hk + (prm.v ? Hk : 0)) * UNITS;
    const int step = blockDim.x * gridDim.y;
    int item = blockIdx.y * blockDim.x + threadIdx.x;

    auto place = [&](int it, const uint4 *&src, int &head, int &u, int &kind, int &e0, int &e1) {
        head = it / UNITS;
        u = it % UNITS;
        kind = head < H ? 0 : head < H + Hk ? 1 : 2;
        const T *base;
        if (kind == 0) {
            base = static_cast<const T *>(prm.q) + t * prm.q_stride + head * D;
        } else if (kind == 1) {
            head -= H;
            base = static_cast<const T *>(prm.k) + t * prm.k_stride + head * D;
        } else {
            head -= H + Hk;
            base = static_cast<const T *>(prm.v) + t * prm.v_stride + head * D;
        }
        const bool apart = kind != 2 && split && u * V < half;
        e0 = apart ? u * V : 2 * u * V;  // first element of either vector
        e1 = apart ? u * V + half : e0 + V;
        src = reinterpret_cast<const uint4 *>(base);
    };

    const uint4 *src;
    int head, u, kind, e0, e1;
    uint4 r0, r1;
    if (item < total) {
        place(item, src, head, u, kind, e0, e1);
        r0 = __ldcs(src + e0 / V);
        r1 = __ldcs(src + e1 / V);
    }
    if (threadIdx.x < half) {
        const uint64_t phase = static_cast<uint64_t>(__ldg(prm.positions + t)) * prm.plan.step[threadIdx.x];
        // nearest 32-bit fraction of a turn, as a signed one in half turns
        const int32_t frac = static_cast<int32_t>((phase + 0x80000000ull) >> 32);
        float s, c;
        sincospif(static_cast<float>(frac) * 0x1p-31f, &s, &c);
        turn[threadIdx.x % V * UNITS + threadIdx.x / V] = make_float2(c * prm.plan.mscale, s * prm.plan.mscale);
    }
    __syncthreads();
    for (; item < total; item += step) {
        if (item >= step) {  // past the thread's first item
            place(item, src, head, u, kind, e0, e1);
            r0 = __ldcs(src + e0 / V);
            r1 = __ldcs(src + e1 / V);
        }
        float a[V], b[V];
        widen_vec(r0, a);
        widen_vec(r1, b);
        if (kind != 2 && u * V < half) {
            const float2 *cs = turn + u;
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
                    const float2 p = cs[i / 2 * UNITS], r = cs[(V + i) / 2 * UNITS];
                    const float x = a[i], y = a[i + 1], z = b[i], w = b[i + 1];
                    a[i] = x * p.x - y * p.y;
                    a[i + 1] = y * p.x + x * p.y;
                    b[i] = z * r.x - w * r.y;
                    b[i + 1] = w * r.x + z * r.y;
                }
            }
        }
        if (kind == 0) {
            uint4 *o = reinterpret_cast<uint4 *>(static_cast<T *>(prm.q_out) + (t * H + head) * D);
            o[e0 / V] = narrow_vec(a);
            o[e1 / V] = narrow_vec(b);
        } else if (slot >= 0) {  // a negative slot is padding
            void *pool = kind == 1 ? prm.k_out : prm.v_out;
            const int64_t row = (slot * Hk + head) * D;
            if constexpr (FP8) {
                const float inv = kind == 1 ? prm.k_inv : prm.v_inv;
                uint8_t *o = static_cast<uint8_t *>(pool) + row;
                *reinterpret_cast<uint2 *>(o + e0) = e4m3_vec(a, inv);
                *reinterpret_cast<uint2 *>(o + e1) = e4m3_vec(b, inv);
            } else {
                uint4 *o = reinterpret_cast<uint4 *>(static_cast<T *>(pool) + row);
                o[e0 / V] = narrow_vec(a);
                o[e1 / V] = narrow_vec(b);
            }
        }
    }
}

}  // namespace pa
