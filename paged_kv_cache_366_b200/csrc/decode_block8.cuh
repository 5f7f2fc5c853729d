// Decode attention over the 8-bit cache with a scale for each block and KV head.
//
//   out[b][h] = softmax(scale * q[b][h] . K^T) V,
//   K[p] = k_codes[block][p % 16] * k_scales[block][hk], V likewise,
//   block = block_tables[b][p / 16].
//
// The work list, its slices, the partials and the merge are decode_kernel's, but a list
// entry is up to four neighbouring KV heads of a block, which as many warps take from one
// stage: the heads' rows of a token are neighbours in memory. One head at a time, 128-byte
// rows a kilobyte apart streamed at 5.1 TB/s; four together stream at 6.3 (64 contexts of
// 4096 tokens, 8 KV heads of 128: 112.5 and 96.0 us).
//
// Producer warps walk the slices and issue every load, a lane a slice; the consumer warps
// only compute. Four of them: one lane's loads hold up its warp's others, and a single
// producer took 95.5 us for eight 32 K contexts where four took 87.6, and 77.8 instead of
// 52.5 us with one KV head (twelve slices to serve). At the copy bandwidth an SM has about
// 180 cycles for a block of one KV head, half of a bf16 cache's, and the packed-FMA step of
// decode_kernel takes over 750 issue slots. So the block step is two small matrix products
// on the warp's tensor instructions (m16n8k16, f16 operands, fp32 sums), about 300 issue
// slots in all for E4M3 and 400 for INT8:
//  * S^T[16 tokens][8 heads] = K Q^T. K's codes widen exactly to f16 in registers; the
//    group's heads fill the 8 columns, up to four of them twice (below). tcgen05 wants 64
//    or more rows of a product at once and the operands in shared memory; widening through
//    shared memory would cost more than these 16 instructions do.
//  * O^T[D][8 heads] += V^T P. The block's probabilities go from the first product's
//    accumulator layout to the second's operand layout by a register transpose
//    (movmatrix), and V's codes of two tokens are paired byte by byte before widening.
// Which lane holds which token and column is free as long as both operands agree, so
// each lane reads 16 contiguous bytes of a row (8 of a 64-byte V row), and the tokens
// are ordered (kTau) so that those reads of TMA-swizzled rows meet no bank conflict.
//
// Numbers. Scores, maxima, sums and O are fp32. q enters as f16 after division by its
// head's power of two: a bf16 value is exact down to 2^-17 of that power (its 8 bits then
// end at f16's smallest step, 2^-24), and off by at most 2^-25 of it below.
// p enters P V as two f16, its first 11 bits and the next 11. Up to four heads leave half
// of the product's columns free: head g's first part is column g, its second column 4 + g
// (whose scores come from the same queries once more), and a close adds the two, so the
// second costs no instruction of the products (eight instructions a block: 89.9 against
// 88.9 us for eight 32 K contexts over INT8, nothing over E4M3; one f16 alone is off by
// 2^-11 of p, which shows where values cancel). Eight heads take a second product. The key
// scale multiplies the block's scores. The value scale joins the exponent: P V uses
// 2^(s + log2(v_scale) - r), with r a running reference of its own, so that f16 keeps
// its digits whatever the spread of scales between blocks; r stays kHeadroom below the
// largest, so that f16's smallest step is 2^-32 of the largest term (a long flat tail
// must not vanish). The softmax sum uses 2^(s - m). A close multiplies O by 2^(r - m).
//
// Measured (32/8 heads of 128): 64 sequences of 128 to 2048 tokens over E4M3 32.7 us, 0.65
// of the measured copy bandwidth. By time stamps the first blocks have landed after 5 us
// (lengths, their scan, tables, first loads), the median slice ends 5 us before the last
// (equal blocks are not equal time where a slice crosses several short contexts), and the
// merge with its launch takes 3.5. Eight of 32 K tokens over INT8: 103 us, 0.80, in calls
// that follow one another for long, where the 1000 W power cap holds the clock at 1.6 GHz
// and INT8's conversions bound it; 87.5 us, 0.94, in short runs at 1965 MHz.
#pragma once

#include "block8.cuh"
#include "decode.cuh"

namespace pa {

// The largest term of P V is 2^8 when r moves and may reach 2^15 before it moves
// again (f16 ends at 2^16).
constexpr float kHeadroom = 8.f, kHighest = 15.f;

struct Block8Params {
    DecodeParams d;
    const float *k_scales, *v_scales;  // [NB][Hk]
};

// Map over a pool of codes [rows][heads][D] with its two outer dims traded, coordinates (x,
// row, head): a box of 16 rows of `share` heads lands as `share` tiles of 16 rows.
// L2 fetches a row of D bytes and no more: its neighbours are other heads' (with 256-byte
// fetches eight 32 K contexts took 118.6 us instead of 101.9 when a stage was one head's).
inline bool encode_codes(CUtensorMap *m, const void *base, int D, uint64_t heads, uint64_t rows, uint32_t share) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return false;
    const cuuint64_t d = static_cast<cuuint64_t>(D), dims[3] = {d, rows, heads};
    const cuuint64_t strides[2] = {heads * d, d};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(D), kBlockSize, share};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              D == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A CTA is WARPS consumer warps and PRODUCERS producer warps. `share` consumer warps (4, 2 or 1:
// the most that divide the KV heads) form a group that streams one slice, a KV head each:
// a stage is one block's K and V tiles of `share` neighbouring heads.
template <int D>
struct Block8Cfg {
    static constexpr int TILE = kBlockSize * D;      // codes of one block of one KV head, K or V
    static constexpr int WARPS = 12;
    static constexpr int NSTAGE = D == 128 ? 4 : 8;  // 16 KB in flight per consumer warp
    static constexpr int PRODUCERS = 4;
    static constexpr int THREADS = 32 * (WARPS + PRODUCERS);
    static constexpr int RING_BYTES = WARPS * NSTAGE * 2 * TILE;
    // per group (at most WARPS) and stage; the scales per warp and stage
    static constexpr int OFF_META = RING_BYTES;                       // what it holds (an int4, below)
    static constexpr int OFF_SCALE = OFF_META + WARPS * NSTAGE * 16;  // k_scale, v_scale
    static constexpr int OFF_FULL = OFF_SCALE + WARPS * NSTAGE * 8;   // an mbarrier
    static constexpr int OFF_EMPTY = OFF_FULL + WARPS * NSTAGE * 8;
    static constexpr int OFF_MISC = OFF_EMPTY + WARPS * NSTAGE * 8;
    static constexpr int SMEM = OFF_MISC + WARPS * 5 * 4 + 16;
    static_assert(SMEM <= kCtaSmem && WARPS % 4 == 0 && WARPS <= 32, "one CTA must fit an SM, a lane each group");
    static_assert(TILE % 1024 == 0, "each tile starts on a swizzle period");
};

// What a stage holds, as one int4: the list's unit, its block, valid rows (0: a bad
// table entry) with flags, rows within the context.
constexpr int kMetaFirst = 0x100, kMetaLast = 0x200, kMetaWhole = 0x400, kMetaRows = 0xff;

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

// Rounded towards zero: an f16's 11 bits of each.
__device__ __forceinline__ uint32_t cut_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// What the two f16 of `h` leave of lo and hi.
__device__ __forceinline__ uint32_t rest_f16(uint32_t h, float lo, float hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return pack_f16(lo - f.x, hi - f.y);
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

// Non-blocking: whether phase `parity` of an mbarrier has completed.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// A producer warp: each lane walks the slice of one group, a few blocks ahead of its
// consumers. For every block it writes what they need to know, and sends the heads' K
// and V (two TMA boxes of `share` tiles) and scales (4-byte cp.async each) on the stage's
// full barrier.
template <int D>
__device__ __forceinline__ void block8_produce(const Block8Params &b8, const CUtensorMap *tm_k, const CUtensorMap *tm_v,
                                               unsigned char *smem, const int *starts, long long N, int WS) {
    using C = Block8Cfg<D>;
    const DecodeParams &prm = b8.d;
    const int share = prm.share, groups = C::WARPS / share;
    const int g = (threadIdx.x % 32) * C::PRODUCERS + threadIdx.x / 32 - C::WARPS;  // the group served
    const int slice = static_cast<int>(blockIdx.x) * groups + g;
    const bool mine = g < groups && slice < WS;
    const long long s_lo = mine ? N * slice / WS : 0, s_hi = mine ? N * (slice + 1) / WS : 0;
    const int nb = static_cast<int>(s_hi - s_lo);
    Cursor cc{0, 0, 0, 0, 1, 0};
    if (mine) cc = Cursor{0, starts[5 * g], starts[5 * g + 1], starts[5 * g + 3], starts[5 * g + 4], starts[5 * g + 2]};
    const uint32_t tiles = share * C::TILE;  // bytes of one TMA box
    const uint32_t ring = smem_addr(smem) + g * C::NSTAGE * 2 * tiles;
    int4 *meta = reinterpret_cast<int4 *>(smem + C::OFF_META) + g * C::NSTAGE;
    const uint32_t scales = smem_addr(smem + C::OFF_SCALE) + g * share * C::NSTAGE * 8;
    const uint32_t full = smem_addr(smem + C::OFF_FULL) + g * C::NSTAGE * 8;
    const uint32_t empty = smem_addr(smem + C::OFF_EMPTY) + g * C::NSTAGE * 8;
    const uint64_t pol = policy_evict_normal();

    // table entries qbase .. qbase + 3 of the unit, and the four after them
    int qbase = 0, cur[4], nxt[4];
    auto entries = [&](int (&q)[4], int at) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = at + i < min(cc.nblk, prm.max_blocks_per_seq)
                       ? __ldg(prm.block_tables + static_cast<size_t>(cc.b) * prm.max_blocks_per_seq + at + i)
                       : -1;
    };
    auto restart = [&]() {
        qbase = cc.blk;
        entries(cur, qbase);
        entries(nxt, qbase + 4);
    };
    if (mine) restart();

    int k = 0, s = 0;          // the next block, its stage
    uint32_t phase = 1;        // the parity of the stage's last release
    unsigned long long idle_since = 0;
    while (true) {
        const bool todo = k < nb;
        if (!__any_sync(0xffffffffu, todo)) break;
        const bool go = todo && (k < C::NSTAGE || mbar_test(empty + 8 * s, phase));
        if (!__any_sync(0xffffffffu, go)) {
            const unsigned long long now = global_ns();
            if (idle_since == 0) idle_since = now;
            if (now - idle_since > kWaitLimitNs) {  // a consumer gave up: its status says why
                flag_status(PA_STATUS_WAIT_TIMEOUT);
                break;
            }
            __nanosleep(20);
            continue;
        }
        idle_since = 0;
        if (go) {
            const int i = cc.blk - qbase;
            int pb = i == 0 ? cur[0] : i == 1 ? cur[1] : i == 2 ? cur[2] : cur[3];
            const int in_context = cc.blk == cc.nblk - 1 ? cc.c - cc.blk * kBlockSize : kBlockSize;
            int rows = in_context;
            if (pb < 0 || pb >= prm.num_blocks) {
                flag_status(PA_STATUS_BAD_BLOCK_ID);
                pb = 0;
                rows = 0;
            }
            const int u = cc.b * prm.list_heads + cc.hk;
            const long long u_lo = s_lo + k - cc.blk, u_hi = u_lo + cc.nblk;  // the unit's positions in the list
            const bool whole = u_lo >= s_lo && u_hi <= s_hi;
            const bool last = cc.blk == cc.nblk - 1 || k == nb - 1;
            meta[s] = make_int4(u, cc.blk,
                                rows | (cc.blk == 0 || k == 0 ? kMetaFirst : 0) | (last ? kMetaLast : 0) |
                                    (whole ? kMetaWhole : 0),
                                in_context);
            const uint32_t bar = full + 8 * s, dst = ring + s * 2 * tiles;
            const int head = cc.hk * share;
            mbar_arrive_expect_tx(bar, 2 * tiles);
            tma_load_3d_policy(dst, tm_k, 0, pb * kBlockSize, head, bar, pol);
            tma_load_3d_policy(dst + tiles, tm_v, 0, pb * kBlockSize, head, bar, pol);
            const size_t at = static_cast<size_t>(pb) * prm.num_kv_heads + head;
            for (int h = 0; h < share; ++h) {
                cp_async4(scales + (h * C::NSTAGE + s) * 8, b8.k_scales + at + h);
                cp_async4(scales + (h * C::NSTAGE + s) * 8 + 4, b8.v_scales + at + h);
            }
            cp_async_arrive(bar);
            if (cc.blk == 0) {  // where the unit's partials are
                int *rec = prm.ws_unit + 2 * static_cast<size_t>(u);
                rec[0] = slice;
                rec[1] = whole ? 1 : slice_of(u_hi - 1, N, WS) - slice + 1;
            }
            if (++s == C::NSTAGE) {
                s = 0;
                phase ^= 1;
            }
            if (++k < nb) {
                if (cursor_advance(cc, 1, prm) > 0) {
                    restart();
                } else if (cc.blk == qbase + 4) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) cur[j] = nxt[j];
                    qbase += 4;
                    entries(nxt, qbase + 4);
                }
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int FMT, int D, int G, bool EMIT>
__global__ void __launch_bounds__(Block8Cfg<D>::THREADS, 1)
    decode_block8_kernel(const __grid_constant__ Block8Params b8, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v) {
    using C = Block8Cfg<D>;
    using T = __nv_bfloat16;
    constexpr int KC = D / 64;     // 16-code chunks of a K row per lane
    constexpr int VW = D / 32;     // 4-code words of a V row per lane
    constexpr int TILES = D / 16;  // 16-column tiles of O^T
    // Groups of up to four heads leave columns of the products free: column 4 + g is head g once more,
    // and takes what column g's f16 probabilities leave.
    constexpr bool SPARE = G <= 4;
    const DecodeParams &prm = b8.d;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int gid = lane / 4, tid = lane % 4;

    extern __shared__ __align__(1024) unsigned char smem_b8[];
    int *starts = reinterpret_cast<int *>(smem_b8 + C::OFF_MISC);
    const int share = prm.share, group = warp / share, sub = warp - group * share;  // sub: the head of the group
    const uint32_t full = smem_addr(smem_b8 + C::OFF_FULL) + group * C::NSTAGE * 8;
    const uint32_t empty = smem_addr(smem_b8 + C::OFF_EMPTY) + group * C::NSTAGE * 8;
    if (warp < C::WARPS && sub == 0 && lane < C::NSTAGE) {
        mbar_init(full + 8 * lane, 2);       // the producer lane: the tiles' bytes, the scales
        mbar_init(empty + 8 * lane, share);  // the consumers
        fence_mbar_init();
    }

    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    long long N;
    int WS;
    decode_prologue<T, D, C::RING_BYTES / 8, C::THREADS>(prm, reinterpret_cast<long long *>(smem_b8), starts,
                                                         C::WARPS / share, N, WS);
    __syncthreads();  // the barriers, and `starts` where the prologue had no sequences to scan
    if (warp >= C::WARPS) {
        block8_produce<D>(b8, &tm_k, &tm_v, smem_b8, starts, N, WS);
        return;
    }
    const int slice = static_cast<int>(blockIdx.x) * (C::WARPS / share) + group;
    if (slice >= WS) return;
    const int nb_w = static_cast<int>(N * (slice + 1) / WS - N * slice / WS);
    const int stage_bytes = 2 * share * C::TILE;
    const unsigned char *ring = smem_b8 + group * C::NSTAGE * stage_bytes + sub * C::TILE;  // this head's K of stage 0
    const int4 *metas = reinterpret_cast<const int4 *>(smem_b8 + C::OFF_META) + group * C::NSTAGE;
    const float2 *scale_slots = reinterpret_cast<const float2 *>(smem_b8 + C::OFF_SCALE) + warp * C::NSTAGE;

    // The unit's queries as the second operand of K Q^T: lane (gid, tid) holds column gid's head's
    // dims 16 tid + 4 s + {0..3} (s < 4), and 64 dims further on for s >= 4. factor[j]:
    // what a product of head 2 tid + j is multiplied by, short of the key scale.
    uint32_t qf[4 * KC][2];
    float factor[2];
    auto load_q = [&](int u) {
        float f[16 * KC];
        float amax = 0.f;
        const int head = SPARE ? gid % 4 : gid;
        if (head < G) {
            const T *row = static_cast<const T *>(prm.q) + (static_cast<size_t>(u) * G + head) * D;
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

    // Running state of heads 2 tid + j. The lane's output columns are gid * D / 8 + c;
    // o[i][j] is column 2 i, o[i][2 + j] column 2 i + 1 of head 2 tid + j.
    float o[TILES][4];
    float l[2];  // this lane's share of the sums
    float m[2];  // running max of the scores, or of an older one within 2^8
    float r[2];  // the same of score + log2(v_scale), less kHeadroom: the unit of O
    const int t_lo = (kTau<D> >> (4 * gid)) & 7;  // token of this lane's score rows gid, gid + 8 (+ 8)
    const int v_lo = (kTau<D> >> (8 * tid)) & 7;  // tokens of value rows 2 tid, 2 tid + 1 (and + 8)
    const int v_hi = (kTau<D> >> (8 * tid + 4)) & 7;
    const uint32_t first11 = SPARE && tid >= 2 ? 0xffffe000u : 0u;  // what this lane's columns leave out of p

    // A segment ends: the unit's output if the whole unit lies in this slice, else the
    // segment's partial (m, l, O).
    auto close_segment = [&](int lu, bool whole) {
        const size_t u = static_cast<size_t>(lu) * share + sub;  // (sequence, KV head)
        const size_t slot = (static_cast<size_t>(slice) + lu) * share + sub;
        if constexpr (SPARE) {
#pragma unroll
            for (int i = 0; i < TILES; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] += __shfl_xor_sync(0xffffffffu, o[i][e], 2);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], off);
            const int g = 2 * tid + j;
            if (g < G) {
                float sc = m[j] == -CUDART_INF_F ? 0.f : exp2f(r[j] - m[j]);
                if (whole) sc = l[j] > 0.f ? sc / l[j] : 0.f;
                const size_t head = (whole ? u : slot) * G + g;
#pragma unroll
                for (int i = 0; i < TILES; i += 2) {
                    const float4 x = make_float4(o[i][j] * sc, o[i][2 + j] * sc, o[i + 1][j] * sc, o[i + 1][2 + j] * sc);
                    const size_t at = head * D + gid * (2 * TILES) + 2 * i;
                    if (whole) store_out4(static_cast<T *>(prm.out) + at, x);
                    else st_v4_keep(prm.ws_o + at, x);
                }
                if (gid == 0) {
                    if (!whole) {
                        prm.ws_m[head] = m[j];
                        prm.ws_l[head] = l[j];
                    } else if constexpr (EMIT) {
                        prm.lse[head] = m[j] + log2f(l[j]);
                    }
                }
            }
        }
    };

    // the first unit's queries, while its first block is on the way
    load_q((starts[5 * group] * prm.list_heads + starts[5 * group + 1]) * share + sub);
    int s = 0;
    uint32_t phase = 0;
    int k = 0;
    for (; k < nb_w; ++k) {
        const bool landed = mbar_wait(full + 8 * s, phase);
        if (!__all_sync(0xffffffffu, landed)) break;
        const int4 meta = metas[s];
        const int n_valid = meta.z & kMetaRows;
        if (meta.z & kMetaFirst) {
            if (k > 0) load_q(meta.x * share + sub);
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
        }
        const unsigned char *kb = ring + s * stage_bytes;
        const unsigned char *vb = kb + share * C::TILE;
        if (n_valid > 0) {
            const float2 scales = scale_slots[s];

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
            // V's words are read now, so that they are there when the softmax is done
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
            };
            load_v(w0, v_lo);
            load_v(w1, v_hi);
            load_v(w2, v_lo + 8);
            load_v(w3, v_hi + 8);
            float x[4];  // rows gid, gid + 8 of heads 2 tid, 2 tid + 1: x[2 * row half + j]
            const float f0 = factor[0] * scales.x, f1 = factor[1] * scales.x;
            x[0] = (c0[0] + c1[0]) * f0;
            x[1] = (c0[1] + c1[1]) * f1;
            x[2] = (c0[2] + c1[2]) * f0;
            x[3] = (c0[3] + c1[3]) * f1;
            if (n_valid < kBlockSize) {
                if (t_lo >= n_valid) x[0] = x[1] = -CUDART_INF_F;
                if (t_lo + 8 >= n_valid) x[2] = x[3] = -CUDART_INF_F;
                // rows past the context may hold NaN codes, and 0 * NaN is NaN
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    if (v_lo >= n_valid) w0[i] = 0u;
                    if (v_hi >= n_valid) w1[i] = 0u;
                    if (v_lo + 8 >= n_valid) w2[i] = 0u;
                    if (v_hi + 8 >= n_valid) w3[i] = 0u;
                }
            }
            if constexpr (EMIT) {
                float *rows = prm.scores + (static_cast<size_t>(meta.x * share + sub) * prm.score_rows + meta.y * kBlockSize) * G;
                if (2 * tid < G) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int t = t_lo + 8 * h;
                        if (t < n_valid) {
                            st_scores<(G == 1 ? 1 : 2)>(rows + t * G + 2 * tid, x + 2 * h);
                        }
                    }
                }
            }

            // ---- online softmax: references move only when a score passes one by more than 2^8
            const float lv = __log2f(scales.y);
            const float top0 = fmaxf(x[0], x[2]), top1 = fmaxf(x[1], x[3]);
            const bool grow = top0 > m[0] + 8.f || top1 > m[1] + 8.f || top0 + lv > r[0] + kHighest ||
                              top1 + lv > r[1] + kHighest;
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float top = j ? top1 : top0;
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
            for (int j = 0; j < 2; ++j) {
                const float mj = m[j] == -CUDART_INF_F ? 0.f : m[j];
                const float rj = lv - (r[j] == -CUDART_INF_F ? 0.f : r[j]);
                l[j] += ex2_approx(x[j] - mj) + ex2_approx(x[2 + j] - mj);
                pv[j] = ex2_approx(x[j] + rj);
                pv[2 + j] = ex2_approx(x[2 + j] + rj);
            }
            // each enters as two f16: its first 11 bits, and the first 11 of what they leave
            uint32_t b0, b1, rest0 = 0, rest1 = 0;
            if constexpr (SPARE) {
#pragma unroll
                for (int e = 0; e < 4; ++e) pv[e] -= __uint_as_float(__float_as_uint(pv[e]) & first11);
                b0 = transpose8x8(cut_f16(pv[0], pv[1]));
                b1 = transpose8x8(cut_f16(pv[2], pv[3]));
            } else {
                const uint32_t p0 = pack_f16(pv[0], pv[1]), p1 = pack_f16(pv[2], pv[3]);
                b0 = transpose8x8(p0);
                b1 = transpose8x8(p1);
                rest0 = transpose8x8(rest_f16(p0, pv[0], pv[1]));
                rest1 = transpose8x8(rest_f16(p1, pv[2], pv[3]));
            }

            // ---- O^T += V^T P
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                // a word's columns 4 w .. 4 w + 3 are rows gid, gid + 8 of tiles 2 w and 2 w + 1
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a0, a1, a2, a3;
                    widen4_f16<FMT>(__byte_perm(w0[w], w1[w], h ? 0x7362 : 0x5140), a0, a1);
                    widen4_f16<FMT>(__byte_perm(w2[w], w3[w], h ? 0x7362 : 0x5140), a2, a3);
                    mma_f16(o[2 * w + h], a0, a1, a2, a3, b0, b1);
                    if constexpr (!SPARE) mma_f16(o[2 * w + h], a0, a1, a2, a3, rest0, rest1);
                }
            }
        } else if constexpr (EMIT) {
            // A block outside the pool takes no part; its scores say so, as the workspace holds whatever was there.
            float *rows = prm.scores + (static_cast<size_t>(meta.x * share + sub) * prm.score_rows + meta.y * kBlockSize) * G;
            for (int i = lane; i < meta.w * G; i += 32) rows[i] = -CUDART_INF_F;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + 8 * s);
        if (++s == C::NSTAGE) {
            s = 0;
            phase ^= 1;
        }
        if (meta.z & kMetaLast) close_segment(meta.x, meta.z & kMetaWhole);
    }
    if (k < nb_w) {
        // a bounded wait gave up: let copies still in flight land before the CTA ends
        for (int kk = k; kk < min(k + C::NSTAGE, nb_w); ++kk)
            mbar_wait(full + 8 * (kk % C::NSTAGE), (kk / C::NSTAGE) & 1);
    }
}

}  // namespace pa
