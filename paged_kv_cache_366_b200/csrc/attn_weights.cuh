// Attention weights, counted over decode steps: weights[b][hk][i] grows by the sum
// over the KV head's query heads of the softmax probability of entry i.
//
// A probability is known only once its head's whole denominator is, so the decode
// kernels (EMIT) leave every score, and each head's log2 denominator lse, and this pass
// adds 2^(score - lse) (a bad block's entries have score -inf and add 0). That costs 4 H
// bytes written and read back for an entry whose K and V are 2 Hk D elements (3 % of a
// bf16 cache's bytes at 32/8 heads of 128, mostly kept by L2), where a second pass over K
// would cost half of them again. Each weight is one thread's: no atomics, the same sums
// every run.
//
// Sharing one launch with the merge, each counting CTA summing its unit's partial
// denominators itself, was slower (decode batch 64.3 us against 58.3): that sum is a chain
// of loads in every CTA. Here the scores, the weights and the denominators are loaded at
// once. Counting adds 8 us to the decode batch over bf16 (48 to 56 us) and 20 us to 64
// contexts of 4096 tokens over E4M3 (88 to 108): bound by launch latency there, and here by
// the scores' way through L2 and back.
#pragma once

#include "decode.cuh"

namespace pa {

constexpr int kCountThreads = 256;
constexpr int kCountEntries = 4 * kCountThreads;  // entries of a CTA: four a thread, a CTA's width apart

// A programmatic dependent of the merge. Grid: units * chunks.
template <int G>
__global__ void __launch_bounds__(kCountThreads) count_weights_kernel(const DecodeParams prm, float *weights,
                                                                      int width, int chunks) {
    const int u = blockIdx.x / chunks, b = u / prm.num_kv_heads;
    const int i0 = (blockIdx.x - u * chunks) * kCountEntries + threadIdx.x;
    const int n = clamp_context(__ldg(prm.context_lens + b), decode_cap(prm), false);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (i0 >= n) return;
    constexpr int VEC = G < 4 ? G : 4;  // an entry's scores by 4, 8 or 16 bytes, lanes side by side
    float s[4][G], w[4], lse[G];
    const float *rows = prm.scores + static_cast<size_t>(u) * prm.score_rows * G;
    float *at = weights + static_cast<size_t>(u) * width;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = i0 + e * kCountThreads;
        if (i >= n) continue;
#pragma unroll
        for (int g = 0; g < G; g += VEC) {
            const float *p = rows + static_cast<size_t>(i) * G + g;
            if constexpr (VEC == 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(p));
                s[e][g] = v.x;
                s[e][g + 1] = v.y;
                s[e][g + 2] = v.z;
                s[e][g + 3] = v.w;
            } else if constexpr (VEC == 2) {
                const float2 v = __ldcg(reinterpret_cast<const float2 *>(p));
                s[e][g] = v.x;
                s[e][g + 1] = v.y;
            } else {
                s[e][g] = __ldcg(p);
            }
        }
        w[e] = at[i];
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
        lse[g] = __ldcg(prm.lse + static_cast<size_t>(u) * G + g);
        if (lse[g] == -CUDART_INF_F) lse[g] = 0.f;  // every score is -inf (all blocks bad, say): 0 for each
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = i0 + e * kCountThreads;
        if (i >= n) continue;
        float p = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) p += ex2_approx(s[e][g] - lse[g]);
        at[i] = w[e] + p;
    }
}

}  // namespace pa
