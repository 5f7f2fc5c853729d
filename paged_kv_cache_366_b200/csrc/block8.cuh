// The 8-bit cache with a scale for each block of 16 tokens and KV head: codes
// (E4M3 or INT8) and their conversions, and the write of new tokens.
//
// A cached value is code * scale[block][KV head]; the write only makes scales that
// are powers of two, the least 2^e with largest magnitude <= 448 * 2^e (E4M3) or
// 127 * 2^e (INT8). Why powers of two: a decode step appends one row to a block
// whose scale may then have to grow, and the rows already there are re-coded.
// Dividing E4M3 codes by a power of two is exact (short of its subnormals); for INT8
// each growth rounds at half the new step, so all growths together stay within one
// step, where arbitrary ratios would add up. The price is up to one bit of an INT8
// code and none of an E4M3 one.
#pragma once

#include <cuda_fp16.h>

#include "pa_common.cuh"

namespace pa {

enum Block8Format { kBlockE4M3 = 0, kBlockInt8 = 1 };

constexpr int kScaleExpMin = -64, kScaleExpMax = 120;  // 2^e and 2^-e are normal fp32 numbers
constexpr float kLargestFloat = 3.402823466e38f;

// The least e with amax <= CODE_MAX * 2^e, clamped; amax finite, >= 0.
// CODE_MAX is 1.75 * 2^8 or 127/128 * 2^7, so e follows from amax's exponent and
// whether its significand exceeds CODE_MAX's.
template <int FMT>
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int x = static_cast<int>(u >> 23) - 127;  // amax = 1.f * 2^x (a subnormal or 0 gives -127: clamped)
    const uint32_t top = FMT == kBlockE4M3 ? 0x600000u : 0x7e0000u;  // fractions of 1.75 and 1.984375
    const int e = x - (FMT == kBlockE4M3 ? 8 : 6) + ((u & 0x7fffffu) > top ? 1 : 0);
    return min(max(e, kScaleExpMin), kScaleExpMax);
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// |x| for the block's largest magnitude: infinities and NaN do not count (they
// would leave nothing of the block's other rows; an infinity saturates instead).
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= kLargestFloat ? a : 0.f;
}

// Four fp32 values, already divided by the scale, to four codes (low byte first):
// nearest, ties to even, saturating. NaN becomes E4M3's NaN, and 0 in INT8.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if constexpr (FMT == kBlockE4M3) {
        return f32x2_to_e4m3x2(a, b) | (f32x2_to_e4m3x2(c, d) << 16);
    } else {
        const float v[4] = {a, b, c, d};
        uint32_t r = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int q = __float2int_rn(fminf(fmaxf(v[i] == v[i] ? v[i] : 0.f, -127.f), 127.f));
            r |= (static_cast<uint32_t>(q) & 0xffu) << (8 * i);
        }
        return r;
    }
}

// The same for values known to be finite and within the code's range.
template <int FMT>
__device__ __forceinline__ uint32_t encode4_in_range(float a, float b, float c, float d) {
    if constexpr (FMT == kBlockE4M3) {
        return encode4<FMT>(a, b, c, d);
    } else {
        // x + 1.5 * 2^23 is a number whose unit is 1: its low byte is x to the nearest, ties to even
        const uint32_t lo = __byte_perm(__float_as_uint(a + 12582912.f), __float_as_uint(b + 12582912.f), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(c + 12582912.f), __float_as_uint(d + 12582912.f), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    }
}

// Four codes of one word to two f16 pairs, (codes 0, 1) and (codes 2, 3), exactly:
// E4M3 by the hardware conversion; INT8 as the low byte of 1024 + (code + 128),
// an f16 whose unit is 1, less 1152.
template <int FMT>
__device__ __forceinline__ void widen4_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (FMT == kBlockE4M3) {
        asm("{\n\t.reg .b16 a, b;\n\t"
            "mov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t bias = 0x64806480u;  // two f16 1152
        uint32_t l = __byte_perm(u, 0x64646464u, 0x4140), h = __byte_perm(u, 0x64646464u, 0x4342);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(l), "r"(bias));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(h), "r"(bias));
    }
}

// Four codes to fp32.
template <int FMT>
__device__ __forceinline__ void widen4_f32(uint32_t w, float (&f)[4]) {
    uint32_t lo, hi;
    widen4_f16<FMT>(w, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
    return x;
}

// ---- the write ----------------------------------------------------------------
//
// A run is a maximal series of tokens next to one another in the call whose slots
// lie in one block. One warp takes a run for one KV head and one of K and V: it
// reads the run's rows into registers (a lane holds D / 32 elements of each), takes
// their largest magnitude, and writes codes. Rows of the block below the run's
// lowest hold earlier tokens: when that largest magnitude outgrows the block's
// scale they are re-coded, else they are left alone. A run from row 0 starts the
// block afresh.
//
// Bound by memory (2 D bytes read and D written a row) and nearly as much by its
// conversions for prefill chunks: 8185 tokens with 8 KV heads of 128 to INT8 in 13.0 us,
// 3.9 TB/s, the ALU 56 % busy. Bound by latency for a decode step's one row a block: 64
// tokens in 2.9 us. A warp looks for runs among
// `chunk` tokens: 16 when there are many tokens (few runs start among 16 tokens of
// a prefill chunk, and a warp for each token would mostly find nothing to do), 1
// when there are few (every token of a decode step is a run).

struct Block8WriteParams {
    const __nv_bfloat16 *k, *v;  // [T][Hk][D]
    uint8_t *k_codes, *v_codes;  // [NB][16][Hk][D]
    float *k_scales, *v_scales;  // [NB][Hk]
    const int64_t *slot_mapping;
    int64_t num_tokens, num_slots;
    int num_kv_heads, chunk;
};

template <int FMT, int D>
__global__ void __launch_bounds__(128, 6) block8_write_kernel(const Block8WriteParams prm) {
    constexpr int EPL = D / 32;  // elements of a row per lane: 4 or 2
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x % 32, Hk = prm.num_kv_heads;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 32;
    const int which = static_cast<int>(w % (2 * Hk));
    const int64_t t0 = w / (2 * Hk) * prm.chunk;
    if (t0 >= prm.num_tokens) return;
    const int hk = which % Hk;
    const bool is_v = which >= Hk;
    const __nv_bfloat16 *src = is_v ? prm.v : prm.k;
    uint8_t *codes = is_v ? prm.v_codes : prm.k_codes;
    float *scales = is_v ? prm.v_scales : prm.k_scales;

    // lane i: the slot of token t0 - 1 + i (negative: padding, or out of range). Runs that
    // start among tokens t0 .. t0 + chunk - 1, chunk <= 16, end by t0 + 30: lane 31.
    int64_t mine = -1;
    {
        const int64_t t = t0 - 1 + lane;
        if (t >= 0 && t < prm.num_tokens) mine = __ldg(prm.slot_mapping + t);
        if (mine >= prm.num_slots) {
            if (which == 0) flag_status(PA_STATUS_BAD_SLOT);
            mine = -1;
        }
    }
    const int64_t my_block = mine < 0 ? -1 : mine / kBlockSize;
    const int64_t before = __shfl_up_sync(0xffffffffu, my_block, 1);
    uint32_t starts = __ballot_sync(0xffffffffu, lane >= 1 && lane <= prm.chunk && mine >= 0 && my_block != before);
    while (starts) {
        const int at = __ffs(starts) - 1;
        starts &= starts - 1;
        const int64_t t = t0 - 1 + at;
        const int64_t blk = __shfl_sync(0xffffffffu, my_block, at);
        // the run: token t + i in lane i, at most 16
        const int64_t slot = __shfl_sync(0xffffffffu, mine, min(at + lane, 31));
        int row = lane < kBlockSize && slot >= 0 && slot / kBlockSize == blk ? static_cast<int>(slot % kBlockSize)
                                                                             : kBlockSize;
        const uint32_t in = __ballot_sync(0xffffffffu, row < kBlockSize);
        const int n = __ffs(~in) - 1;  // in's low bits in a row
        if (lane >= n) row = kBlockSize;
        const int first = __reduce_min_sync(0xffffffffu, row);

        const int64_t pitch = static_cast<int64_t>(Hk) * D;  // elements of a token, bytes of its codes
        const __nv_bfloat16 *first_row = src + (t * Hk + hk) * D + lane * EPL;
        uint32_t raw[kBlockSize][EPL / 2];  // bf16 pairs
#pragma unroll
        for (int i = 0; i < kBlockSize; ++i) {
            if (i < n) {
                const uint32_t *p = reinterpret_cast<const uint32_t *>(first_row + i * pitch);
                if constexpr (EPL == 4) {
                    const uint2 r = *reinterpret_cast<const uint2 *>(p);
                    raw[i][0] = r.x;
                    raw[i][1] = r.y;
                } else {
                    raw[i][0] = *p;
                }
            }
        }
        float *scale_at = scales + blk * Hk + hk;
        const float held = first > 0 ? *scale_at : 0.f;
        // The largest magnitude, by bf16 pairs: NaN if there is one, infinite if there is one;
        // then (rarely) again over the finite ones, and with the careful conversion below.
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kBlockSize; ++i)
            if (i < n)
#pragma unroll
                for (int j = 0; j < EPL / 2; ++j)
                    asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(raw[i][j]));
        // bf16 magnitudes order as their bits, NaN above infinity
        uint32_t bits = max(top & 0x7fffu, top >> 16 & 0x7fffu);
        bits = __reduce_max_sync(0xffffffffu, bits);
        float amax = __uint_as_float(bits << 16);
        const bool odd = bits >= 0x7f80u;
        if (odd) {
            amax = 0.f;
#pragma unroll
            for (int i = 0; i < kBlockSize; ++i)
                if (i < n)
#pragma unroll
                    for (int j = 0; j < EPL / 2; ++j) {
                        amax = fmaxf(amax, finite_abs(__uint_as_float(raw[i][j] << 16)));
                        amax = fmaxf(amax, finite_abs(__uint_as_float(raw[i][j] & 0xffff0000u)));
                    }
            amax = warp_max(amax);
        }
        const float need = exp2_int(scale_exponent<FMT>(amax));
        const float scale = fmaxf(held, need);
        uint8_t *block = codes + (blk * kBlockSize * Hk + hk) * D + lane * EPL;  // this lane's columns of row 0
        if (first > 0 && scale > held) {
            const float ratio = held / scale;
            for (int r = 0; r < first; ++r) {
                float f[4];
                if constexpr (EPL == 4) {
                    uint32_t *p = reinterpret_cast<uint32_t *>(block + r * pitch);
                    widen4_f32<FMT>(*p, f);
                    *p = encode4<FMT>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
                } else {
                    uint16_t *p = reinterpret_cast<uint16_t *>(block + r * pitch);
                    widen4_f32<FMT>(*p, f);
                    *p = static_cast<uint16_t>(encode4<FMT>(f[0] * ratio, f[1] * ratio, 0.f, 0.f));
                }
            }
        }
        const float inv = 1.f / scale;
        auto put = [&](auto encode) {
#pragma unroll
            for (int i = 0; i < kBlockSize; ++i) {
                const int r = __shfl_sync(0xffffffffu, row, i);
                if (i < n) {
                    const float x0 = __uint_as_float(raw[i][0] << 16) * inv;
                    const float x1 = __uint_as_float(raw[i][0] & 0xffff0000u) * inv;
                    if constexpr (EPL == 4) {
                        const float x2 = __uint_as_float(raw[i][EPL / 2 - 1] << 16) * inv;
                        const float x3 = __uint_as_float(raw[i][EPL / 2 - 1] & 0xffff0000u) * inv;
                        *reinterpret_cast<uint32_t *>(block + r * pitch) = encode(x0, x1, x2, x3);
                    } else {
                        *reinterpret_cast<uint16_t *>(block + r * pitch) =
                            static_cast<uint16_t>(encode(x0, x1, 0.f, 0.f));
                    }
                }
            }
        };
        // in range: finite, and not past the largest scale
        if (!odd && amax * inv <= (FMT == kBlockE4M3 ? 448.f : 127.f))
            put([](float a, float b, float c, float d) { return encode4_in_range<FMT>(a, b, c, d); });
        else
            put([](float a, float b, float c, float d) { return encode4<FMT>(a, b, c, d); });
        if (lane == 0 && scale != held) *scale_at = scale;
    }
}

}  // namespace pa
