// Host side of the cache operators declared in include/pa.h: rotary positions, the
// block-scaled 8-bit cache, weight-counting decode and eviction. Argument checks,
// launch geometry and template dispatch; included by pa_api.cu after its own helpers.
#pragma once

#include "block8.cuh"
#include "decode_block8.cuh"
#include "evict.cuh"
#include "rope.cuh"

namespace {

bool is_block8(const pa_shape *s) { return s && (s->kv_fp8 == PA_KV_BLOCK_E4M3 || s->kv_fp8 == PA_KV_BLOCK_INT8); }

// check_shape for calls that also take block8 pools.
int check_shape_b8(const pa_shape *s) {
    if (!is_block8(s)) return check_shape(s);
    pa_shape plain = *s;
    plain.kv_fp8 = 0;
    const int rc = check_shape(&plain);
    if (rc != PA_OK) return rc;
    return s->dtype == PA_DTYPE_BF16 ? PA_OK : PA_ERR_UNSUPPORTED;
}

int cache_bytes(const pa_shape *s) { return is_block8(s) ? 1 : cache_elem_bytes(s); }

int sms_or_default() {
    const int n = sm_count();
    return n > 0 ? n : 148;
}

// ---- rotary positions -----------------------------------------------------------

template <typename T, bool FP8>
int launch_rope(pa::RopeParams p, int64_t num_tokens, int D, cudaStream_t st) {
    p.num_tokens = num_tokens;
    const int heads = p.num_heads + p.num_kv_heads + (p.v ? p.num_kv_heads : 0);
    const int rows = pa::kRopeThreads / (D * static_cast<int>(sizeof(T)) / 32);  // rows a CTA takes at once
    // four tokens a CTA once that fills the SMs four times; while single tokens leave SMs idle, their
    // rows are spread over as many CTAs as hold one round of them each
    const int64_t sms = sms_or_default();
    const int tokens = num_tokens >= 16 * sms ? pa::kRopeTokens : 1;
    const int split = (heads + rows - 1) / rows;
    const int by = num_tokens * split <= sms ? split : 1;
    const dim3 grid(static_cast<unsigned>((num_tokens + tokens - 1) / tokens), by);
    if (D == 128) pa::rope_kernel<T, FP8, 128><<<grid, pa::kRopeThreads, 0, st>>>(p, tokens);
    else pa::rope_kernel<T, FP8, 64><<<grid, pa::kRopeThreads, 0, st>>>(p, tokens);
    return check_launch();
}

int check_plan(const pa_rope_plan *plan, int head_dim) {
    if (!plan) return PA_ERR_INVALID_ARGUMENT;
    if (plan->rot_dim < 16 || plan->rot_dim % 16 != 0 || (plan->interleaved != 0 && plan->interleaved != 1) ||
        !std::isfinite(plan->mscale))
        return PA_ERR_INVALID_ARGUMENT;
    return plan->rot_dim <= head_dim ? PA_OK : PA_ERR_UNSUPPORTED;
}

// q, k, v rows of heads * D elements at a token stride: 16-byte aligned, apart.
int check_rows(const void *p, int64_t stride, int heads, const pa_shape *s) {
    if (!p) return PA_ERR_INVALID_ARGUMENT;
    if (stride < static_cast<int64_t>(heads) * s->head_dim) return PA_ERR_INVALID_ARGUMENT;
    if (!aligned16(p) || stride * elem_bytes(s) % 16 != 0) return PA_ERR_ALIGNMENT;
    return PA_OK;
}

// ---- decode over block8 pools and with weights -----------------------------------

template <int FMT, int D, int G, bool EMIT>
int launch_decode_block8(const pa::Block8Params &b8, const DecodeGeometry &geo, cudaStream_t st) {
    using C = pa::Block8Cfg<D>;
    auto kernel = pa::decode_block8_kernel<FMT, D, G, EMIT>;
    static std::atomic<bool> ready[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev < 0 || dev >= kMaxDevices) return PA_ERR_DEVICE;
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return cuda_fail(e);
        ready[dev].store(true, std::memory_order_release);
    }
    pa::Block8Params p = b8;
    p.d.warps_total = geo.ctas * (C::WARPS / p.d.share);
    CUtensorMap tm_k{}, tm_v{};
    const uint64_t rows = static_cast<uint64_t>(p.d.num_blocks) * pa::kBlockSize;
    if (!pa::encode_codes(&tm_k, p.d.k_cache, D, p.d.num_kv_heads, rows, p.d.share) ||
        !pa::encode_codes(&tm_v, p.d.v_cache, D, p.d.num_kv_heads, rows, p.d.share))
        return PA_ERR_UNSUPPORTED;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(geo.ctas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    e = cudaLaunchKernelEx(&cfg, kernel, p, tm_k, tm_v);
    if (e != cudaSuccess) return cuda_fail(e);
    return launch_merge<__nv_bfloat16, G, D, EMIT, true>(p.d, cfg);
}

template <int FMT, int D, bool EMIT>
int dispatch_block8_g(int g, const pa::Block8Params &p, const DecodeGeometry &geo, cudaStream_t st) {
    switch (g) {
        case 1: return launch_decode_block8<FMT, D, 1, EMIT>(p, geo, st);
        case 2: return launch_decode_block8<FMT, D, 2, EMIT>(p, geo, st);
        case 4: return launch_decode_block8<FMT, D, 4, EMIT>(p, geo, st);
        default: return launch_decode_block8<FMT, D, 8, EMIT>(p, geo, st);
    }
}

template <bool EMIT>
int dispatch_block8(const pa_shape *s, const pa::Block8Params &p, const DecodeGeometry &geo, cudaStream_t st) {
    const int g = s->num_heads / s->num_kv_heads;
    if (s->kv_fp8 == PA_KV_BLOCK_E4M3)
        return s->head_dim == 128 ? dispatch_block8_g<pa::kBlockE4M3, 128, EMIT>(g, p, geo, st)
                                  : dispatch_block8_g<pa::kBlockE4M3, 64, EMIT>(g, p, geo, st);
    return s->head_dim == 128 ? dispatch_block8_g<pa::kBlockInt8, 128, EMIT>(g, p, geo, st)
                              : dispatch_block8_g<pa::kBlockInt8, 64, EMIT>(g, p, geo, st);
}

// Lengths and table widths up to this keep the kernels' int arithmetic in range.
constexpr int32_t kMaxContext = 1 << 30;

// KV heads that share a stage of the block8 decode.
int block8_share(const pa_shape *s) { return s->num_kv_heads % 4 == 0 ? 4 : s->num_kv_heads % 2 == 0 ? 2 : 1; }

// Geometry of a counting decode over any pool, or a decode over a block8 pool. A block8
// list entry is block8_share heads, and a slice is a group of as many warps. Short lists are
// cut down to one block a slice: against four, one 333-token sequence took 8.1 us instead of 10.3, 64
// sequences of 16 tokens 8.1 instead of 15.0 (graph replays, 32/8 heads of 128).
int geometry_of(int32_t num_seqs, int32_t max_context_len, int32_t partition_tokens, const pa_shape *s,
                DecodeGeometry *g) {
    if (max_context_len > kMaxContext) return PA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(num_seqs) * s->num_kv_heads > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    if (!is_block8(s)) {
        DecodeFit fit = decode_fit(s);
        fit.min_blocks = 1;
        return decode_geometry(num_seqs, max_context_len, partition_tokens, s, g, fit);
    }
    const int share = block8_share(s);
    pa_shape list = *s;
    list.num_kv_heads /= share;
    list.num_heads /= share;
    const int rc = decode_geometry(num_seqs, max_context_len, partition_tokens, &list, g,
                                   DecodeFit{1, pa::Block8Cfg<128>::WARPS / share, 1});
    if (rc != PA_OK || g->slots == 0) return rc;
    g->slots *= share;
    const int64_t heads = g->slots * (s->num_heads / s->num_kv_heads);
    g->ws_bytes = heads * s->head_dim * 4 + round16(heads * 4) * 2 +
                  round16(static_cast<int64_t>(num_seqs) * list.num_kv_heads * 8);
    return PA_OK;
}

// Scores (fp32 [B * Hk][score_rows][G]) and denominators (fp32 [B][H]) of a
// weight-counting decode, after the decode's own workspace.
struct CountSpace {
    int64_t score_rows, scores_at, lse_at, bytes;
};

// Whether the counting grid holds every piece of every (sequence, KV head)'s weights; the sizes of a
// workspace for it then fit 64 bits.
bool count_fits(int32_t num_seqs, int32_t max_context_len, const pa_shape *s) {
    return static_cast<int64_t>(num_seqs) * s->num_kv_heads *
               ((max_context_len + pa::kCountEntries - 1) / pa::kCountEntries) <= 0x7fffffff;
}

CountSpace count_space(const DecodeGeometry &g, int32_t num_seqs, int32_t max_context_len, const pa_shape *s) {
    CountSpace c;
    c.score_rows = (static_cast<int64_t>(max_context_len) + PA_BLOCK_SIZE - 1) / PA_BLOCK_SIZE * PA_BLOCK_SIZE;
    c.scores_at = round16(g.ws_bytes);
    c.lse_at = c.scores_at + c.score_rows * num_seqs * s->num_heads * 4;
    c.bytes = c.lse_at + round16(static_cast<int64_t>(num_seqs) * s->num_heads * 4);
    return c;
}

// The checks and parameters that decode over a block8 pool and weight-counting decode share.
int fill_decode(pa::DecodeParams *prm, DecodeGeometry *g, void *out, const void *q, const void *k_cache,
                const void *v_cache, const int32_t *block_tables, int32_t max_blocks_per_seq,
                const int32_t *context_lens, int32_t num_seqs, int32_t max_context_len, float scale,
                int32_t partition_tokens, void *workspace, const pa_shape *s) {
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens) return PA_ERR_INVALID_ARGUMENT;
    if (max_blocks_per_seq < 1 || !std::isfinite(scale)) return PA_ERR_INVALID_ARGUMENT;
    if (max_blocks_per_seq > kMaxContext / PA_BLOCK_SIZE) return PA_ERR_UNSUPPORTED;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4))
        return PA_ERR_ALIGNMENT;
    const int rc = geometry_of(num_seqs, max_context_len, partition_tokens, s, g);
    if (rc != PA_OK) return rc;
    if (!workspace) return PA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return PA_ERR_ALIGNMENT;
    place_partials(prm, *g, s, workspace);
    prm->out = out;
    prm->q = q;
    prm->k_cache = k_cache;
    prm->v_cache = v_cache;
    prm->block_tables = block_tables;
    prm->context_lens = context_lens;
    prm->num_blocks = s->num_blocks;
    prm->num_seqs = num_seqs;
    prm->max_blocks_per_seq = max_blocks_per_seq;
    prm->num_heads = s->num_heads;
    prm->num_kv_heads = s->num_kv_heads;
    prm->share = is_block8(s) ? block8_share(s) : 1;
    prm->list_heads = s->num_kv_heads / prm->share;
    prm->max_context_len = max_context_len;
    prm->scale_log2 = scale * 1.4426950408889634f;
    prm->v_scale = 1.f;
    if (s->kv_fp8 == 1) {
        prm->scale_log2 *= s->k_scale;
        prm->v_scale = s->v_scale;
    }
    return PA_OK;
}

// ---- eviction --------------------------------------------------------------------

// CTAs of a row's selection: as many as bring their share to kSelectShare keys, up to a portable cluster.
int select_ranks(int32_t max_context_len) {
    int ranks = 1;
    while (ranks < pa::kSelectMaxCluster && static_cast<int64_t>(ranks) * pa::kSelectShare < max_context_len) ranks *= 2;
    return ranks;
}

// Four warps' pieces each, a KV head, of K and V apart for block8 pools.
int64_t copy_rows_of_grid(const pa_shape *s) {
    return (static_cast<int64_t>(s->num_kv_heads) * (is_block8(s) ? 2 : 1) + 3) / 4;
}

template <int THREADS>
int launch_evict_select(const pa::EvictParams &p, int64_t units, cudaStream_t st) {
    auto kernel = pa::evict_select_kernel<THREADS>;
    static std::atomic<bool> ready[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev < 0 || dev >= kMaxDevices) return PA_ERR_DEVICE;
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, pa::kSelectKeys * 4);
        if (e != cudaSuccess) return cuda_fail(e);
        ready[dev].store(true, std::memory_order_release);
    }
    const int ranks = select_ranks(p.max_context_len);
    const int held = std::min((p.max_context_len + ranks - 1) / ranks, pa::kSelectKeys);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(units * ranks));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = held * 4;
    e = cudaLaunchKernelEx(&cfg, kernel, p, held);
    return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

template <int ROW, int FMT>
int launch_evict_copy(const pa::EvictParams &p, unsigned y, cudaStream_t st) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(p.num_seqs) * p.dst_blocks, y);
    cfg.blockDim = dim3(128);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, pa::evict_copy_kernel<ROW, FMT>, p);
    return e == cudaSuccess ? PA_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

int pa_rope_init(pa_rope_plan *plan, int32_t rot_dim, int32_t interleaved, double base, int32_t scaling, double factor,
                 double low, double high, double original_len, double mscale) {
    if (!plan || (interleaved != 0 && interleaved != 1)) return PA_ERR_INVALID_ARGUMENT;
    if (rot_dim < 16 || rot_dim > PA_ROPE_MAX_DIM || rot_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (!std::isfinite(base) || base < 1.0 || !std::isfinite(static_cast<float>(mscale))) return PA_ERR_INVALID_ARGUMENT;
    if (scaling < PA_ROPE_NONE || scaling > PA_ROPE_PARTS) return PA_ERR_INVALID_ARGUMENT;
    if (scaling != PA_ROPE_NONE && !(std::isfinite(factor) && factor >= 1.0)) return PA_ERR_INVALID_ARGUMENT;
    if (scaling == PA_ROPE_PARTS &&
        !(std::isfinite(low) && std::isfinite(high) && low >= 0.0 && high > low && std::isfinite(original_len) &&
          original_len > 0.0))
        return PA_ERR_INVALID_ARGUMENT;
    // In long double (64 significant bits): a rounding of the frequency grows with the position.
    const long double two_pi = 6.283185307179586476925286766559L;
    std::memset(plan, 0, sizeof *plan);
    plan->rot_dim = rot_dim;
    plan->interleaved = interleaved;
    plan->mscale = static_cast<float>(mscale);
    long double b = base;
    if (scaling == PA_ROPE_BASE)
        b *= powl(static_cast<long double>(factor), static_cast<long double>(rot_dim) / (rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        long double f = powl(b, -2.0L * i / rot_dim);
        if (scaling == PA_ROPE_LINEAR) f /= factor;
        if (scaling == PA_ROPE_PARTS) {
            long double keep = (original_len * f / two_pi - low) / (static_cast<long double>(high) - low);
            keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
            f = f * keep + f / factor * (1 - keep);
        }
        // the fraction of a turn per position, f <= 1 rad: below 2^62 of 2^64
        plan->step[i] = static_cast<uint64_t>(f / two_pi * 18446744073709551616.0L + 0.5L);
    }
    return PA_OK;
}

int pa_rope(void *q_out, void *k_out, const void *q, const void *k, int64_t q_stride, int64_t k_stride,
            const int64_t *positions, int64_t num_tokens, const pa_rope_plan *plan, const pa_shape *shape,
            void *stream) {
    int rc = check_shape_b8(shape);
    if (rc != PA_OK) return rc;
    rc = check_plan(plan, shape->head_dim);
    if (rc != PA_OK) return rc;
    if (num_tokens < 0) return PA_ERR_INVALID_ARGUMENT;
    if (num_tokens == 0) return PA_OK;
    if (num_tokens > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    if (!q_out || !k_out || !positions) return PA_ERR_INVALID_ARGUMENT;
    rc = check_rows(q, q_stride, shape->num_heads, shape);
    if (rc == PA_OK) rc = check_rows(k, k_stride, shape->num_kv_heads, shape);
    if (rc != PA_OK) return rc;
    if (!aligned16(q_out) || !aligned16(k_out) || !aligned(positions, 8)) return PA_ERR_ALIGNMENT;
    // in place is fine only where a row is written over itself
    if ((q_out == q && q_stride != static_cast<int64_t>(shape->num_heads) * shape->head_dim) ||
        (k_out == k && k_stride != static_cast<int64_t>(shape->num_kv_heads) * shape->head_dim))
        return PA_ERR_INVALID_ARGUMENT;
    pa::RopeParams p{};
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    p.positions = positions;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.num_heads = shape->num_heads;
    p.num_kv_heads = shape->num_kv_heads;
    p.plan = *plan;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return shape->dtype == PA_DTYPE_BF16 ? launch_rope<__nv_bfloat16, false>(p, num_tokens, shape->head_dim, st)
                                         : launch_rope<float, false>(p, num_tokens, shape->head_dim, st);
}

int pa_rope_and_cache(void *q_out, const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                      int64_t v_stride, void *k_cache, void *v_cache, const int64_t *slot_mapping,
                      const int64_t *positions, int64_t num_tokens, const pa_rope_plan *plan, const pa_shape *shape,
                      void *stream) {
    int rc = check_shape(shape);
    if (rc != PA_OK) return rc;
    rc = check_plan(plan, shape->head_dim);
    if (rc != PA_OK) return rc;
    if (num_tokens < 0) return PA_ERR_INVALID_ARGUMENT;
    if (num_tokens == 0) return PA_OK;
    if (num_tokens > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    if (!q_out || !k_cache || !v_cache || !slot_mapping || !positions) return PA_ERR_INVALID_ARGUMENT;
    rc = check_rows(q, q_stride, shape->num_heads, shape);
    if (rc == PA_OK) rc = check_rows(k, k_stride, shape->num_kv_heads, shape);
    if (rc == PA_OK) rc = check_rows(v, v_stride, shape->num_kv_heads, shape);
    if (rc != PA_OK) return rc;
    if (!aligned16(q_out) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned(slot_mapping, 8) ||
        !aligned(positions, 8))
        return PA_ERR_ALIGNMENT;
    if (q_out == q && q_stride != static_cast<int64_t>(shape->num_heads) * shape->head_dim)
        return PA_ERR_INVALID_ARGUMENT;  // in place is fine only where a row is written over itself
    pa::RopeParams p{};
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
    p.k_out = k_cache;
    p.v_out = v_cache;
    p.slot_mapping = slot_mapping;
    p.positions = positions;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.num_slots = shape->num_blocks * PA_BLOCK_SIZE;
    p.num_heads = shape->num_heads;
    p.num_kv_heads = shape->num_kv_heads;
    p.plan = *plan;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (shape->kv_fp8) {
        p.k_inv = 1.0f / shape->k_scale;
        p.v_inv = 1.0f / shape->v_scale;
        return launch_rope<__nv_bfloat16, true>(p, num_tokens, shape->head_dim, st);
    }
    return shape->dtype == PA_DTYPE_BF16 ? launch_rope<__nv_bfloat16, false>(p, num_tokens, shape->head_dim, st)
                                         : launch_rope<float, false>(p, num_tokens, shape->head_dim, st);
}

int pa_cache_block8(const void *k, const void *v, void *k_codes, void *v_codes, float *k_scales, float *v_scales,
                    const int64_t *slot_mapping, int64_t num_tokens, const pa_shape *shape, void *stream) {
    int rc = check_shape_b8(shape);
    if (rc != PA_OK) return rc;
    if (!is_block8(shape)) return PA_ERR_UNSUPPORTED;
    if (num_tokens < 0) return PA_ERR_INVALID_ARGUMENT;
    if (num_tokens == 0) return PA_OK;
    if (!k || !v || !k_codes || !v_codes || !k_scales || !v_scales || !slot_mapping) return PA_ERR_INVALID_ARGUMENT;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_codes) || !aligned16(v_codes) || !aligned(k_scales, 4) ||
        !aligned(v_scales, 4) || !aligned(slot_mapping, 8))
        return PA_ERR_ALIGNMENT;
    pa::Block8WriteParams p{};
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.k_codes = static_cast<uint8_t *>(k_codes);
    p.v_codes = static_cast<uint8_t *>(v_codes);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.slot_mapping = slot_mapping;
    p.num_tokens = num_tokens;
    p.num_slots = shape->num_blocks * PA_BLOCK_SIZE;
    p.num_kv_heads = shape->num_kv_heads;
    // tokens a warp looks for runs among: as many as leave every SM 48 warps
    const int64_t per_token = 2 * static_cast<int64_t>(shape->num_kv_heads);
    const int64_t full = static_cast<int64_t>(sms_or_default()) * 48;
    p.chunk = static_cast<int>(std::min<int64_t>(16, std::max<int64_t>(1, num_tokens * per_token / full)));
    const int64_t warps = (num_tokens + p.chunk - 1) / p.chunk * per_token;
    if ((warps + 3) / 4 > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    const unsigned grid = static_cast<unsigned>((warps + 3) / 4);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool e4m3 = shape->kv_fp8 == PA_KV_BLOCK_E4M3;
    if (shape->head_dim == 128) {
        if (e4m3) pa::block8_write_kernel<pa::kBlockE4M3, 128><<<grid, 128, 0, st>>>(p);
        else pa::block8_write_kernel<pa::kBlockInt8, 128><<<grid, 128, 0, st>>>(p);
    } else {
        if (e4m3) pa::block8_write_kernel<pa::kBlockE4M3, 64><<<grid, 128, 0, st>>>(p);
        else pa::block8_write_kernel<pa::kBlockInt8, 64><<<grid, 128, 0, st>>>(p);
    }
    return check_launch();
}

int64_t pa_decode_block8_workspace_bytes(int32_t num_seqs, int32_t max_context_len, int32_t partition_tokens,
                                         const pa_shape *shape) {
    int rc = check_shape_b8(shape);
    if (rc != PA_OK) return rc;
    if (!is_block8(shape)) return PA_ERR_UNSUPPORTED;
    DecodeGeometry g;
    rc = geometry_of(num_seqs, max_context_len, partition_tokens, shape, &g);
    return rc == PA_OK ? g.ws_bytes : rc;
}

int pa_decode_block8(void *out, const void *q, const void *k_codes, const void *v_codes, const float *k_scales,
                     const float *v_scales, const int32_t *block_tables, int32_t max_blocks_per_seq,
                     const int32_t *context_lens, int32_t num_seqs, int32_t max_context_len, float scale,
                     int32_t partition_tokens, void *workspace, int64_t workspace_bytes, const pa_shape *shape,
                     void *stream) {
    int rc = check_shape_b8(shape);
    if (rc != PA_OK) return rc;
    if (!is_block8(shape)) return PA_ERR_UNSUPPORTED;
    if (num_seqs < 0 || max_context_len < 0 || max_blocks_per_seq < 0) return PA_ERR_INVALID_ARGUMENT;
    if (num_seqs == 0) return PA_OK;
    if (!k_scales || !v_scales) return PA_ERR_INVALID_ARGUMENT;
    if (!aligned(k_scales, 4) || !aligned(v_scales, 4)) return PA_ERR_ALIGNMENT;
    pa::Block8Params p{};
    DecodeGeometry g;
    rc = fill_decode(&p.d, &g, out, q, k_codes, v_codes, block_tables, max_blocks_per_seq, context_lens, num_seqs,
                     max_context_len, scale, partition_tokens, workspace, shape);
    if (rc != PA_OK) return rc;
    if (workspace_bytes < g.ws_bytes) return PA_ERR_WORKSPACE;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    return dispatch_block8<false>(shape, p, g, static_cast<cudaStream_t>(stream));
}

int64_t pa_decode_weights_workspace_bytes(int32_t num_seqs, int32_t max_context_len, int32_t partition_tokens,
                                          const pa_shape *shape) {
    int rc = check_shape_b8(shape);
    if (rc != PA_OK) return rc;
    DecodeGeometry g;
    rc = geometry_of(num_seqs, max_context_len, partition_tokens, shape, &g);
    if (rc != PA_OK) return rc;
    if (!count_fits(num_seqs, max_context_len, shape)) return PA_ERR_UNSUPPORTED;
    return count_space(g, num_seqs, max_context_len, shape).bytes;
}

int pa_decode_weights(void *out, float *weights, int32_t weights_width, const void *q, const void *k_cache,
                      const void *v_cache, const float *k_scales, const float *v_scales, const int32_t *block_tables,
                      int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t num_seqs,
                      int32_t max_context_len, float scale, int32_t partition_tokens, void *workspace,
                      int64_t workspace_bytes, const pa_shape *shape, void *stream) {
    int rc = check_shape_b8(shape);
    if (rc != PA_OK) return rc;
    if (num_seqs < 0 || max_context_len < 0 || max_blocks_per_seq < 0) return PA_ERR_INVALID_ARGUMENT;
    if (num_seqs == 0) return PA_OK;
    if (!weights || weights_width < max_context_len) return PA_ERR_INVALID_ARGUMENT;
    if (!aligned(weights, 4)) return PA_ERR_ALIGNMENT;
    if (is_block8(shape) && (!k_scales || !v_scales)) return PA_ERR_INVALID_ARGUMENT;
    if (!aligned(k_scales, 4) || !aligned(v_scales, 4)) return PA_ERR_ALIGNMENT;
    pa::Block8Params p{};
    DecodeGeometry g;
    rc = fill_decode(&p.d, &g, out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs,
                     max_context_len, scale, partition_tokens, workspace, shape);
    if (rc != PA_OK) return rc;
    if (!count_fits(num_seqs, max_context_len, shape)) return PA_ERR_UNSUPPORTED;
    const CountSpace c = count_space(g, num_seqs, max_context_len, shape);
    if (workspace_bytes < c.bytes) return PA_ERR_WORKSPACE;
    p.d.scores = reinterpret_cast<float *>(static_cast<char *>(workspace) + c.scores_at);
    p.d.lse = reinterpret_cast<float *>(static_cast<char *>(workspace) + c.lse_at);
    p.d.score_rows = static_cast<int>(c.score_rows);
    p.d.weights = weights;
    p.d.weights_width = weights_width;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int G = shape->num_heads / shape->num_kv_heads;
    if (is_block8(shape)) return dispatch_block8<true>(shape, p, g, st);
    if (shape->kv_fp8)
        return shape->head_dim == 128 ? dispatch_g<__nv_bfloat16, pa::fp8e4m3, 128, true>(G, p.d, g, kBoth, st)
                                      : dispatch_g<__nv_bfloat16, pa::fp8e4m3, 64, true>(G, p.d, g, kBoth, st);
    if (shape->dtype == PA_DTYPE_BF16)
        return shape->head_dim == 128 ? dispatch_g<__nv_bfloat16, __nv_bfloat16, 128, true>(G, p.d, g, kBoth, st)
                                      : dispatch_g<__nv_bfloat16, __nv_bfloat16, 64, true>(G, p.d, g, kBoth, st);
    return shape->head_dim == 128 ? dispatch_g<float, float, 128, true>(G, p.d, g, kBoth, st)
                                  : dispatch_g<float, float, 64, true>(G, p.d, g, kBoth, st);
}

int pa_evict(void *k_cache, void *v_cache, float *k_scales, float *v_scales, const float *weights,
             int32_t weights_width, const int32_t *block_tables, int32_t max_blocks_per_seq,
             const int32_t *context_lens, const int32_t *dst_block_tables, int32_t dst_blocks_per_seq,
             float *new_weights, int32_t *new_context_lens, int32_t *kept, int32_t num_seqs, int32_t max_context_len,
             int32_t keep, int32_t sinks, int32_t recent, const pa_shape *shape, void *stream) {
    int rc = check_shape_b8(shape);
    if (rc != PA_OK) return rc;
    if (num_seqs < 0 || max_context_len < 0 || max_blocks_per_seq < 0 || keep < 1 || sinks < 0 || recent < 0 ||
        static_cast<int64_t>(sinks) + recent > keep)
        return PA_ERR_INVALID_ARGUMENT;
    if (num_seqs == 0) return PA_OK;
    if (!k_cache || !v_cache || !weights || !block_tables || !context_lens || !dst_block_tables || !new_weights ||
        !new_context_lens || !kept)
        return PA_ERR_INVALID_ARGUMENT;
    if (max_blocks_per_seq < 1 || weights_width < max_context_len) return PA_ERR_INVALID_ARGUMENT;
    if (max_context_len > kMaxContext || max_blocks_per_seq > kMaxContext / PA_BLOCK_SIZE ||
        dst_blocks_per_seq > kMaxContext / PA_BLOCK_SIZE || keep > kMaxContext)
        return PA_ERR_UNSUPPORTED;
    // every kept entry has a place in the new tables
    if (dst_blocks_per_seq < 1 ||
        static_cast<int64_t>(dst_blocks_per_seq) * PA_BLOCK_SIZE < std::min(keep, max_context_len))
        return PA_ERR_INVALID_ARGUMENT;
    if (new_context_lens == context_lens || new_weights == weights) return PA_ERR_INVALID_ARGUMENT;
    if (is_block8(shape) && (!k_scales || !v_scales)) return PA_ERR_INVALID_ARGUMENT;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned(k_scales, 4) || !aligned(v_scales, 4) ||
        !aligned(weights, 4) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
        !aligned(dst_block_tables, 4) || !aligned(new_weights, 4) || !aligned(new_context_lens, 4) || !aligned(kept, 4))
        return PA_ERR_ALIGNMENT;
    const int64_t units = static_cast<int64_t>(num_seqs) * shape->num_kv_heads;
    const int64_t copy_y = copy_rows_of_grid(shape);
    // both grids, before either is launched
    if (units * select_ranks(max_context_len) > 0x7fffffff ||
        static_cast<int64_t>(num_seqs) * dst_blocks_per_seq > 0x7fffffff || copy_y > 65535)
        return PA_ERR_UNSUPPORTED;
    pa::EvictParams p{};
    p.k_cache = static_cast<unsigned char *>(k_cache);
    p.v_cache = static_cast<unsigned char *>(v_cache);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.weights = weights;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.dst_tables = dst_block_tables;
    p.new_weights = new_weights;
    p.new_lens = new_context_lens;
    p.kept = kept;
    p.num_blocks = shape->num_blocks;
    p.num_seqs = num_seqs;
    p.num_kv_heads = shape->num_kv_heads;
    p.width = weights_width;
    p.max_blocks = max_blocks_per_seq;
    p.dst_blocks = dst_blocks_per_seq;
    p.keep = keep;
    p.sinks = sinks;
    p.recent = recent;
    p.max_context_len = max_context_len;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // 256 threads where three CTAs an SM or more wait for one another's barriers, fewer where rows are short
    // (a thread's keys are few then). The whole call, 512 against 256 threads: 800 rows of up to 1024 entries 37.3
    // and 33.5 us, 128 rows 11.1 and 11.8; 448 rows of up to 2048 37.0 and 35.6, 208 rows 21.9 and 22.1; 800 rows
    // of up to 4096 106 and 103, 352 rows 50.5 and 52.0; 72 rows of up to 32768 (576 CTAs) 87.8 and 81.3, 24 rows
    // 38.1 and 40.6 (bf16, rows of 64, a quarter kept).
    const int64_t ctas = units * select_ranks(max_context_len);
    rc = ctas >= static_cast<int64_t>(sms_or_default()) * std::min(3, (max_context_len + 1023) / 1024)
             ? launch_evict_select<256>(p, units, st)
             : launch_evict_select<512>(p, units, st);
    if (rc != PA_OK) return rc;
    const int row = shape->head_dim * cache_bytes(shape);
    const unsigned y = static_cast<unsigned>(copy_y);
    if (is_block8(shape)) {
        if (shape->kv_fp8 == PA_KV_BLOCK_E4M3)
            return row == 128 ? launch_evict_copy<128, pa::kBlockE4M3>(p, y, st) : launch_evict_copy<64, pa::kBlockE4M3>(p, y, st);
        return row == 128 ? launch_evict_copy<128, pa::kBlockInt8>(p, y, st) : launch_evict_copy<64, pa::kBlockInt8>(p, y, st);
    }
    switch (row) {
        case 64: return launch_evict_copy<64, -1>(p, y, st);
        case 128: return launch_evict_copy<128, -1>(p, y, st);
        case 256: return launch_evict_copy<256, -1>(p, y, st);
        default: return launch_evict_copy<512, -1>(p, y, st);
    }
}

}  // extern "C"
