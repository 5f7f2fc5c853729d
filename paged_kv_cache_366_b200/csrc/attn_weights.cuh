// Attention weights, counted over decode steps: weights[b][hk][i] grows by the sum
// over the KV head's query heads of the softmax probability of entry i.
//
// A probability is known only once its head's whole denominator is, so the decode
// kernels (EMIT) leave every score, and each head's log2 denominator lse, and this pass
// adds 2^(score - lse). That costs 4 H bytes written and read back for an entry whose
// K and V are 2 Hk D elements (3 % of a bf16 cache's bytes at 32/8 heads of 128, mostly
// kept by L2), where a second pass over K would cost half of them again. Each weight is
// one thread's: no atomics, the same sums every run.
#pragma once

#include "decode.cuh"

namespace pa {

constexpr int kCountThreads = 256;
constexpr int kCountEntries = 4 * kCountThreads;  // entries of a CTA

// Grid: (units * chunks). Four neighbouring entries a thread.
template <int G>
__global__ void __launch_bounds__(kCountThreads) count_weights_kernel(const DecodeParams prm, float *weights,
                                                                      int width, int chunks) {
    const int u = blockIdx.x / chunks, b = u / prm.num_kv_heads;
    const int n = clamp_context(__ldg(prm.context_lens + b), decode_cap(prm), false);
    const int i0 = (blockIdx.x % chunks) * kCountEntries + 4 * threadIdx.x;
    if (i0 >= n) return;
    float lse[G];
#pragma unroll
    for (int g = 0; g < G; ++g) lse[g] = __ldcg(prm.lse + static_cast<size_t>(u) * G + g);
    float s[4 * G];  // rows are padded to 16 entries: four are always there
    const float4 *row = reinterpret_cast<const float4 *>(prm.scores + (static_cast<size_t>(u) * prm.score_rows + i0) * G);
#pragma unroll
    for (int i = 0; i < G; ++i) {
        const float4 v = __ldcg(row + i);
        s[4 * i] = v.x;
        s[4 * i + 1] = v.y;
        s[4 * i + 2] = v.z;
        s[4 * i + 3] = v.w;
    }
    float *w = weights + static_cast<size_t>(u) * width + i0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i0 + i < n) {
            float p = 0.f;
#pragma unroll
            for (int g = 0; g < G; ++g) p += ex2_approx(s[i * G + g] - lse[g]);
            w[i] += p;
        }
    }
}

}  // namespace pa
