// Decode attention over the 8-bit cache with a scale for each block and KV head.
//
//   out[b][h] = softmax(scale * q[b][h] . K^T) V,
//   K[p] = k_codes[block][p % 16] * k_scales[block][hk], V likewise,
//   block = block_tables[b][p / 16].
//
// The work list, its slices, the partials and the merge are decode_kernel's. What
// differs is the block step, because the bytes are half of a bf16 cache's: at the
// copy bandwidth an SM has about 180 cycles for a block of one KV head, and the
// packed-FMA step of decode_kernel takes over 750 issue slots. So here a block is two
// small matrix products on the warp's tensor instructions (m16n8k16, f16 operands,
// fp32 sums), about 220 issue slots:
//  * S^T[16 tokens][8 heads] = K Q^T. K's codes widen exactly to f16 in registers; the
//    group's heads fill the 8 columns (the rest are 0). tcgen05 wants 64 or more rows of
//    a product at once and the operands in shared memory; widening through shared memory
//    would cost more than these 16 instructions do.
//  * O^T[D][8 heads] += V^T P. The block's probabilities go from the first product's
//    accumulator layout to the second's operand layout by a register transpose
//    (movmatrix), and V's codes of two tokens are paired byte by byte before widening.
// Which lane holds which token and column is free as long as both operands agree, so
// each lane reads 16 contiguous bytes of a row (8 of a 64-byte V row), and the tokens
// are ordered (kTau) so that those reads of TMA-swizzled rows meet no bank conflict.
//
// Numbers. Scores, maxima, sums and O are fp32. q enters as f16 after division by its
// head's power of two (so a bf16 value is exact down to 2^-22 of the head's largest);
// p enters P V as f16 (relative 2^-11, under bf16's 2^-9). The key scale multiplies the
// block's scores. The value scale joins the exponent: P V uses
// 2^(s + log2(v_scale) - r), with r a running reference of its own, so that f16 keeps
// its digits whatever the spread of scales between blocks; r stays kHeadroom below the
// largest, so that f16's smallest step is 2^-32 of the largest term (a long flat tail
// must not vanish). The softmax sum uses 2^(s - m). A close multiplies O by 2^(r - m).
#pragma once

#include "block8.cuh"
#include "decode.cuh"

namespace pa {

// The largest term of P V is 2^7 when r moves and may reach 2^15 before it moves
// again (f16 ends at 2^16).
constexpr float kHeadroom = 7.f;

struct Block8Params {
    DecodeParams d;
    const float *k_scales, *v_scales;  // [NB][Hk]
};

template <int D, int G>
struct Block8Cfg {
    static constexpr int STAGE_BYTES = 2 * kBlockSize * D;  // K and V codes of one block of one KV head
    static constexpr int WARPS = 12;
    static constexpr int NSTAGE = D == 128 ? 4 : 8;  // 16 KB in flight per warp
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int WARP_RING = NSTAGE * STAGE_BYTES;
    static constexpr int RING_BYTES = WARPS * WARP_RING;
    static constexpr int OFF_BAR = RING_BYTES;
    static constexpr int OFF_SCALE = OFF_BAR + WARPS * NSTAGE * 8;  // per stage: k_scale, v_scale
    static constexpr int OFF_MISC = OFF_SCALE + WARPS * NSTAGE * 8;
    static constexpr int SMEM = OFF_MISC + WARPS * 5 * 4 + 16;
    static_assert(SMEM <= kCtaSmem, "one CTA must fit an SM");
    static_assert(STAGE_BYTES / 2 % 1024 == 0, "each tile starts on a swizzle period");
};

// d += a b, a [16][16] (row-major fragments), b [16][8], f16 in, fp32 out.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Arrive on `bar` once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Token of score row i (and i + 8: token + 8), 4 bits each from the low end. Rows
// 2i and 2i + 1 must differ in the token bit that decides the half of a 128-byte line
// (bit 2 under the 128-byte swizzle, bit 0 under the 64-byte one), and rows 0, 2, 4, 6
// (and 1, 3, 5, 7) must spread over the line's quarters, so that every eight lanes of a
// 16-byte read cover all banks.
template <int D>
constexpr uint32_t kTau = D == 128 ? 0x37621540u : 0x67542310u;

// Byte offset of 16-byte chunk c of row t in a swizzled tile of D-byte rows.
template <int D>
__device__ __forceinline__ uint32_t tile_at(int t, int c) {
    return t * D + ((D == 128 ? c ^ (t & 7) : c ^ ((t >> 1) & 3)) << 4);
}

template <int FMT, int D, int G, bool EMIT>
__global__ void __launch_bounds__(Block8Cfg<D, G>::THREADS, 1)
    decode_block8_kernel(const Block8Params b8, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v) {
    using C = Block8Cfg<D, G>;
    using T = __nv_bfloat16;
    constexpr int KC = D / 64;     // 16-code chunks of a K row per lane
    constexpr int VW = D / 32;     // 4-code words of a V row per lane
    constexpr int TILES = D / 16;  // 16-column tiles of O^T
    const DecodeParams &prm = b8.d;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int gid = lane / 4, tid = lane % 4;
    const int Hk = prm.num_kv_heads;

    extern __shared__ __align__(1024) unsigned char smem_b8[];
    int *starts = reinterpret_cast<int *>(smem_b8 + C::OFF_MISC);

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    long long N;
    int WS;
    decode_prologue<T, D, C::WARPS, C::RING_BYTES / 8>(prm, reinterpret_cast<long long *>(smem_b8), starts, N, WS);
    const int slice = static_cast<int>(blockIdx.x) * C::WARPS + warp;
    if (slice >= WS) return;  // from here on every warp runs alone on its slice
    const long long s_lo = N * slice / WS, s_hi = N * (slice + 1) / WS;
    const int nb_w = static_cast<int>(s_hi - s_lo);

    unsigned char *ring = smem_b8 + warp * C::WARP_RING;
    const uint32_t ring_s = smem_addr(ring);
    const uint32_t bars = smem_addr(smem_b8 + C::OFF_BAR) + warp * C::NSTAGE * 8;
    const float *scale_slots = reinterpret_cast<const float *>(smem_b8 + C::OFF_SCALE) + warp * C::NSTAGE * 2;
    const uint32_t scale_s = smem_addr(scale_slots);
    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < C::NSTAGE; ++s) mbar_init(bars + 8 * s, 3);  // lane 0's bytes, two scales
        fence_mbar_init();
    }
    __syncwarp();
    Cursor cc{0, starts[5 * warp], starts[5 * warp + 1], starts[5 * warp + 3], starts[5 * warp + 4],
              starts[5 * warp + 2]};

    // ---- issue side, as in decode_kernel: block k at cursor ic into stage k % NSTAGE
    int tb_u = -1, tbase = 0, tw = 0;
    uint32_t bad_mask = 0;
    auto issue = [&](int k, const Cursor &ic) {
        const int u = ic.b * Hk + ic.hk;
        if (u != tb_u || ic.blk >= tbase + 32) {
            tb_u = u;
            tbase = ic.blk;
            const int e = tbase + lane;
            tw = e < min(ic.nblk, prm.max_blocks_per_seq)
                     ? __ldg(prm.block_tables + static_cast<size_t>(ic.b) * prm.max_blocks_per_seq + e)
                     : 0;
        }
        int pb = __shfl_sync(0xffffffffu, tw, ic.blk - tbase);
        const int s = k % C::NSTAGE;
        if (pb < 0 || pb >= prm.num_blocks) {
            if (lane == 0) flag_status(PA_STATUS_BAD_BLOCK_ID);
            pb = 0;
            bad_mask |= 1u << s;
        } else {
            bad_mask &= ~(1u << s);
        }
        const uint32_t bar = bars + 8 * s;
        if (lane == 0) {
            mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
            const uint32_t dst = ring_s + s * C::STAGE_BYTES;
            const uint64_t pol = policy_evict_normal();
            tma_load_3d_policy(dst, &tm_k, 0, ic.hk, pb * kBlockSize, bar, pol);
            tma_load_3d_policy(dst + kBlockSize * D, &tm_v, 0, ic.hk, pb * kBlockSize, bar, pol);
        }
        if (lane < 2) {
            const float *src = (lane == 0 ? b8.k_scales : b8.v_scales) + static_cast<size_t>(pb) * Hk + ic.hk;
            cp_async4(scale_s + 8 * s + 4 * lane, src);
            cp_async_arrive(bar);
        }
    };
    Cursor icur = cc;  // the last block fetched
    for (int i = 0; i < min(C::NSTAGE, nb_w); ++i) {
        if (i > 0) cursor_advance(icur, 1, prm);
        issue(i, icur);
    }

    // The unit's queries as the second operand of K Q^T: lane (gid, tid) holds head gid's
    // dims 16 tid + 4 s + {0..3} (s < 4), and 64 dims further on for s >= 4. factor[j]:
    // what a product of head 2 tid + j is multiplied by, short of the key scale.
    uint32_t qf[4 * KC][2];
    float factor[2];
    auto load_q = [&](const Cursor &x) {
        float f[16 * KC];
        float amax = 0.f;
        if (gid < G) {
            const T *row = static_cast<const T *>(prm.q) + (static_cast<size_t>(x.b) * prm.num_heads + x.hk * G + gid) * D;
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 raw = __ldg(reinterpret_cast<const uint4 *>(row + 64 * c + 16 * tid) + i);
                    float w[8];
                    Widen<T>::apply(raw, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[16 * c + 8 * i + e] = w[e];
                }
#pragma unroll
            for (int e = 0; e < 16 * KC; ++e) amax = fmaxf(amax, finite_abs(f[e]));
        } else {
#pragma unroll
            for (int e = 0; e < 16 * KC; ++e) f[e] = 0.f;
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // amax = 1.f * 2^qe; within fp32's normal exponents, so that both powers exist
        const int qe = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -120), 120);
        const float down = exp2_int(-qe);
#pragma unroll
        for (int s = 0; s < 4 * KC; ++s) {
            qf[s][0] = pack_f16(f[4 * s] * down, f[4 * s + 1] * down);
            qf[s][1] = pack_f16(f[4 * s + 2] * down, f[4 * s + 3] * down);
        }
        const float up = exp2_int(qe) * prm.scale_log2;
        factor[0] = __shfl_sync(0xffffffffu, up, 8 * tid);
        factor[1] = __shfl_sync(0xffffffffu, up, 8 * tid + 4);
    };

    // Running state of heads 2 tid + j. O^T tile i: o[i][0], [1] are column 2 VW... of the
    // lane's D / 8 output columns: column 2 i of heads 2 tid, 2 tid + 1, then column 2 i + 1.
    float o[TILES][4];
    float l[2];   // this lane's share of the sums
    float m[2];   // running max of the scores, or of an older one within 2^8
    float r[2];   // the same of score + log2(v_scale), less kHeadroom: the unit of O
    auto reset_state = [&]() {
#pragma unroll
        for (int i = 0; i < TILES; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            l[j] = 0.f;
            m[j] = -CUDART_INF_F;
            r[j] = -CUDART_INF_F;
        }
    };
    const int t_lo = (kTau<D> >> (4 * gid)) & 7;               // token of this lane's score rows gid, gid + 8 (+ 8)
    const int v_lo = (kTau<D> >> (8 * tid)) & 7;               // tokens of value rows 2 tid, 2 tid + 1 (and + 8)
    const int v_hi = (kTau<D> >> (8 * tid + 4)) & 7;

    auto close_segment = [&]() {
        const long long u_lo = s_lo + cc.r - cc.blk, u_hi = u_lo + cc.nblk;  // the unit's positions
        const bool whole = u_lo >= s_lo && u_hi <= s_hi;
        const int u = cc.b * Hk + cc.hk;
        const size_t slot = static_cast<size_t>(slice) + u;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], off);
            const int g = 2 * tid + j;
            if (g < G) {
                float sc = m[j] == -CUDART_INF_F ? 0.f : exp2f(r[j] - m[j]);
                if (whole) sc = l[j] > 0.f ? sc / l[j] : 0.f;
                constexpr int COLS = 2 * TILES;  // output columns of this lane: gid * COLS ...
#pragma unroll
                for (int i = 0; i < TILES; i += 2) {
                    const float4 x = make_float4(o[i][j] * sc, o[i][2 + j] * sc, o[i + 1][j] * sc, o[i + 1][2 + j] * sc);
                    if (whole)
                        store_out4(static_cast<T *>(prm.out) +
                                       (static_cast<size_t>(cc.b) * prm.num_heads + cc.hk * G + g) * D + gid * COLS + 2 * i,
                                   x);
                    else
                        st_v4_keep(prm.ws_o + (slot * G + g) * D + gid * COLS + 2 * i, x);
                }
                if (gid == 0) {
                    if (!whole) {
                        prm.ws_m[slot * G + g] = m[j];
                        prm.ws_l[slot * G + g] = l[j];
                    } else if constexpr (EMIT) {
                        prm.lse[static_cast<size_t>(u) * G + g] = m[j] + log2f(l[j]);
                    }
                }
            }
        }
        if (lane == 0 && u_lo >= s_lo) {
            int *rec = prm.ws_unit + 2 * static_cast<size_t>(u);
            rec[0] = slice;
            rec[1] = whole ? 1 : slice_of(u_hi - 1, N, WS) - slice + 1;
        }
    };

    reset_state();
    bool need_q = true;
    int k = 0;
    for (; k < nb_w; ++k) {
        const int s = k % C::NSTAGE;
        if (need_q) {
            load_q(cc);
            need_q = false;
        }
        const bool landed = mbar_wait(bars + 8 * s, (k / C::NSTAGE) & 1);
        if (!__all_sync(0xffffffffu, landed)) break;
        const int last_valid = cc.c - (cc.nblk - 1) * kBlockSize;
        const int n_valid = ((bad_mask >> s) & 1u) ? 0 : (cc.blk == cc.nblk - 1 ? last_valid : kBlockSize);
        const unsigned char *kb = ring + s * C::STAGE_BYTES;
        const unsigned char *vb = kb + kBlockSize * D;
        if (n_valid > 0) {
            const float ks = scale_slots[2 * s], vs = scale_slots[2 * s + 1];

            // ---- scores
            float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const uint4 a = *reinterpret_cast<const uint4 *>(kb + tile_at<D>(t_lo, tid + 4 * c));
                const uint4 b = *reinterpret_cast<const uint4 *>(kb + tile_at<D>(t_lo + 8, tid + 4 * c));
                const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t a0, a1, a2, a3;
                    widen4_f16<FMT>(aw[w], a0, a2);
                    widen4_f16<FMT>(bw[w], a1, a3);
                    mma_f16(w % 2 ? c1 : c0, a0, a1, a2, a3, qf[4 * c + w][0], qf[4 * c + w][1]);
                }
            }
            float x[4];  // rows gid, gid + 8 of heads 2 tid, 2 tid + 1: x[2 * row half + j]
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = (c0[e] + c1[e]) * (factor[e & 1] * ks);
            if (n_valid < kBlockSize) {
                if (t_lo >= n_valid) x[0] = x[1] = -CUDART_INF_F;
                if (t_lo + 8 >= n_valid) x[2] = x[3] = -CUDART_INF_F;
            }
            if constexpr (EMIT) {
                float *rows = prm.scores + ((static_cast<size_t>(cc.b) * Hk + cc.hk) * prm.score_rows + cc.blk * kBlockSize) * G;
                if (2 * tid < G) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int t = t_lo + 8 * h;
                        if (t < n_valid) {
                            if constexpr (G == 1) rows[t] = x[2 * h];
                            else *reinterpret_cast<float2 *>(rows + t * G + 2 * tid) = make_float2(x[2 * h], x[2 * h + 1]);
                        }
                    }
                }
            }

            // ---- online softmax: references move only when a score passes one by more than 2^8
            const float lv = __log2f(vs);
            bool grow = false;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float top = fmaxf(x[j], x[2 + j]);
                grow |= top > m[j] + 8.f || top + lv > r[j] + (kHeadroom + 8.f);
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float top = fmaxf(x[j], x[2 + j]);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                    const float m_new = fmaxf(m[j], top), r_new = fmaxf(r[j], top + lv - kHeadroom);
                    l[j] *= m_new == -CUDART_INF_F ? 1.f : exp2f(m[j] - m_new);
                    const float alpha = r_new == -CUDART_INF_F ? 1.f : exp2f(r[j] - r_new);
                    m[j] = m_new;
                    r[j] = r_new;
#pragma unroll
                    for (int i = 0; i < TILES; ++i) {
                        o[i][j] *= alpha;
                        o[i][2 + j] *= alpha;
                    }
                }
            }
            float pv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = e & 1;
                const float mj = m[j] == -CUDART_INF_F ? 0.f : m[j], rj = r[j] == -CUDART_INF_F ? 0.f : r[j];
                l[j] += ex2_approx(x[e] - mj);
                pv[e] = ex2_approx(x[e] + lv - rj);
            }
            const uint32_t b0 = transpose8x8(pack_f16(pv[0], pv[1]));
            const uint32_t b1 = transpose8x8(pack_f16(pv[2], pv[3]));

            // ---- O^T += V^T P
            uint32_t w0[VW], w1[VW], w2[VW], w3[VW];  // rows 2 tid, 2 tid + 1, and + 8
            auto load_v = [&](uint32_t(&w)[VW], int t) {
                if constexpr (VW == 4) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(vb + tile_at<D>(t, gid));
                    w[0] = a.x;
                    w[1] = a.y;
                    w[2] = a.z;
                    w[3] = a.w;
                } else {
                    const uint2 a = *reinterpret_cast<const uint2 *>(vb + tile_at<D>(t, gid / 2) + 8 * (gid % 2));
                    w[0] = a.x;
                    w[1] = a.y;
                }
                // rows past the context may hold NaN codes, and 0 * NaN is NaN
                if (t >= n_valid)
#pragma unroll
                    for (int i = 0; i < VW; ++i) w[i] = 0u;
            };
            load_v(w0, v_lo);
            load_v(w1, v_hi);
            load_v(w2, v_lo + 8);
            load_v(w3, v_hi + 8);
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                // a word's columns 4 w .. 4 w + 3 are rows gid, gid + 8 of tiles 2 w and 2 w + 1
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a0, a1, a2, a3;
                    widen4_f16<FMT>(__byte_perm(w0[w], w1[w], h ? 0x7362 : 0x5140), a0, a1);
                    widen4_f16<FMT>(__byte_perm(w2[w], w3[w], h ? 0x7362 : 0x5140), a2, a3);
                    mma_f16(o[2 * w + h], a0, a1, a2, a3, b0, b1);
                }
            }
        }
        __syncwarp();
        Cursor nx = cc;
        const int passed = k + 1 < nb_w ? cursor_advance(nx, 1, prm) : 0;
        if (k + C::NSTAGE < nb_w) {
            cursor_advance(icur, 1, prm);
            issue(k + C::NSTAGE, icur);
        }
        if (passed > 0 || k + 1 == nb_w) {
            close_segment();
            reset_state();
            need_q = true;
        }
        cc = nx;
    }
    if (k < nb_w) {
        // a bounded wait gave up: let copies still in flight land before the CTA ends
        for (int kk = k; kk < min(k + C::NSTAGE, nb_w); ++kk)
            mbar_wait(bars + 8 * (kk % C::NSTAGE), (kk / C::NSTAGE) & 1);
    }
}

}  // namespace pa
