// Latent attention in the absorbed form over the paged rows: kda_mla_decode.
//
//   s_j = scale (q_lat . c_j + q_pe . p_j),  o = sum_j e^{s_j - M} c_j / sum_j e^{s_j - M}
//
// one pass over the rows with a running maximum and sum. One CTA of four warps takes one
// (token, head); the warps take every fourth row and their parts are joined at the end.

#include "kda_latent_common.cuh"

namespace kda {
namespace {

struct DecodeArgs {
    const __nv_bfloat16 *q_lat, *q_pe;
    PagedRows<const __nv_bfloat16> cache;
    const int32_t *lens;
    int32_t N, H, m;
    float scale;
    __nv_bfloat16 *o;
    float *lse;
    int32_t *status;
};

__global__ void __launch_bounds__(128) kda_mla_decode_kernel(const __grid_constant__ DecodeArgs p) {
    __shared__ float s_o[4][kLatent], s_m[4], s_l[4];
    __shared__ int s_bad;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;  // (n m + t) H + h
    const int64_t nt = row / p.H;
    const int n = (int)(nt / p.m), t = (int)(nt % p.m);
    const int64_t len = p.lens[n], size = p.cache.page_size;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    const bool bad_len = len < 0 || len > (int64_t)p.cache.max_pages * size;
    const int64_t end = bad_len ? 0 : len - p.m + 1 + t;
    const int32_t *table = p.cache.table + (int64_t)n * p.cache.max_pages;
    if (bad_len) {
        if (threadIdx.x == 0) set_status(p.status, KDA_ERR_SEQLENS), s_bad = 1;
    } else {
        for (int64_t i = threadIdx.x; i < (len + size - 1) / size; i += blockDim.x)
            if (table[i] < 0 || table[i] >= p.cache.num_pages) set_status(p.status, KDA_ERR_PAGES), s_bad = 1;
    }
    __syncthreads();
    const bool bad = s_bad;
    float q[18], o[16], m = -INFINITY, l = 0.f;
    for (int i = 0; i < 16; ++i) q[i] = __bfloat162float(p.q_lat[row * kLatent + lane + 32 * i]) * p.scale, o[i] = 0.f;
    for (int i = 0; i < 2; ++i) q[16 + i] = __bfloat162float(p.q_pe[row * kPos + lane + 32 * i]) * p.scale;
    for (int64_t j = warp; j < end && !bad; j += 4) {
        const __nv_bfloat16 *r = p.cache.rows + table[j / size] * p.cache.page_stride + (j % size) * kRow;
        float x[18], s = 0.f;
        for (int i = 0; i < 18; ++i) x[i] = __bfloat162float(r[lane + 32 * i]), s += q[i] * x[i];
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
        const float f = expf(m - base), e = expf(s - base);
        l = l * f + e;
        for (int i = 0; i < 16; ++i) o[i] = o[i] * f + e * x[i];
        m = mn;
    }
    for (int i = 0; i < 16; ++i) s_o[warp][lane + 32 * i] = o[i];
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
    __syncthreads();
    float M = -INFINITY, L = 0.f, f[4];
    for (int w = 0; w < 4; ++w) M = fmaxf(M, s_m[w]);
    for (int w = 0; w < 4; ++w) f[w] = s_l[w] == 0.f ? 0.f : expf(s_m[w] - M), L += f[w] * s_l[w];
    const float inv = bad ? NAN : (L == 0.f ? 0.f : 1.f / L);
    for (int i = threadIdx.x; i < kLatent; i += 128) {
        float v = 0.f;
        for (int w = 0; w < 4; ++w) v += f[w] * s_o[w][i];
        p.o[row * kLatent + i] = __float2bfloat16(v * inv);
    }
    if (p.lse && threadIdx.x == 0) p.lse[row] = bad ? NAN : M + logf(L);
}

}  // namespace
}  // namespace kda

extern "C" {

size_t kda_mla_decode_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t num_tokens) {
    if (num_seqs < 0 || num_heads < 0 || num_tokens < 0) return 0;
    return 256;
}

int kda_mla_decode(const uint16_t *q_lat, const uint16_t *q_pe, const uint16_t *cache, int64_t page_stride,
                   int32_t num_pages, int32_t page_size, const int32_t *page_table, int32_t max_pages,
                   const int32_t *cache_lens, int32_t num_seqs, int32_t num_heads, int32_t num_tokens, float scale,
                   uint16_t *o, float *lse, void *workspace, size_t workspace_bytes, int32_t *status, void *stream) {
    using namespace kda;
    int rc = check_cache(page_stride, num_pages, page_size, max_pages);
    if (rc != KDA_OK) return rc;
    if (!(scale > 0.0f) || scale > 3.402823466e38f || num_tokens > KDA_MAX_REPLAY_TOKENS) return KDA_ERR_UNSUPPORTED;
    if (num_seqs < 0 || num_heads <= 0 || num_tokens < 0 || num_heads > 65535 ||
        (int64_t)num_seqs * num_heads * num_tokens > INT32_MAX)
        return KDA_ERR_SHAPE;
    if (num_seqs == 0 || num_tokens == 0) return KDA_OK;
    if (!q_lat || !q_pe || !cache || !page_table || !cache_lens || !o || !workspace) return KDA_ERR_NULL;
    if (!mla_aligned(q_lat, 16) || !mla_aligned(q_pe, 16) || !mla_aligned(cache, 16) || !mla_aligned(o, 16) ||
        !mla_aligned(lse, 4) || !mla_aligned(page_table, 4) || !mla_aligned(cache_lens, 4) || !mla_aligned(status, 4) ||
        !mla_aligned(workspace, 256))
        return KDA_ERR_ALIGN;
    if (workspace_bytes < kda_mla_decode_workspace_size(num_seqs, num_heads, num_tokens)) return KDA_ERR_WORKSPACE;
    DecodeArgs a{reinterpret_cast<const __nv_bfloat16 *>(q_lat),
                 reinterpret_cast<const __nv_bfloat16 *>(q_pe),
                 {reinterpret_cast<const __nv_bfloat16 *>(cache), page_stride, num_pages, page_size, page_table, max_pages},
                 cache_lens,
                 num_seqs,
                 num_heads,
                 num_tokens,
                 scale,
                 reinterpret_cast<__nv_bfloat16 *>(o),
                 lse,
                 status};
    kda_mla_decode_kernel<<<(unsigned)((int64_t)num_seqs * num_tokens * num_heads), 128, 0,
                            static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
