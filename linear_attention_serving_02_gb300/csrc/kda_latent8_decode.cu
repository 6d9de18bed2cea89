// Latent attention in the absorbed form over the pages of the 8-bit cache: kda_mla_decode_fp8.
//
//   s_rj = scale s_j (q_r . row_j),  o_r = sum_j e^{s_rj - M_r} s_j c_j / sum_j e^{s_rj - M_r}
//
// A warp takes a query row (one window token and head) and a part of its sequence's cached rows, each
// lane 16 latents and 2 positional values; scores are warp reductions, the running maximum and sum are
// kept in fp32. A second kernel joins the parts.

#include "kda_common.cuh"
#include "kda_latent_common.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8, kMaxParts = 64;

struct Decode8Args {
    const __nv_bfloat16 *q_lat, *q_pe;
    PagedRows<const uint8_t> cache;
    const int32_t *lens;
    int32_t N, H, m, R, parts;
    float scale;
    __nv_bfloat16 *o;
    float *lse;
    float *part_o;    // [parts, N R, 512]
    float2 *part_ml;  // [parts, N R]
    int32_t *status;
};

__global__ void __launch_bounds__(kWarps * 32) kda_mla_decode_fp8_kernel(const __grid_constant__ Decode8Args p) {
    const int lane = threadIdx.x & 31, n = blockIdx.y, r = blockIdx.z * kWarps + (threadIdx.x >> 5);
    pdl_wait();
    if (r >= p.R) return;
    const int64_t len = p.lens[n], row = (int64_t)n * p.R + r, at = blockIdx.x * (int64_t)p.N * p.R + row;
    bool bad = len < 0 || len > (int64_t)p.cache.max_pages * p.cache.page_size;
    if (bad && lane == 0) set_status(p.status, KDA_ERR_SEQLENS);
    float q[16], o[16], qp[2], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = __bfloat162float(p.q_lat[row * kLatent + 16 * lane + i]), o[i] = 0.f;
    qp[0] = __bfloat162float(p.q_pe[row * kPos + 2 * lane]), qp[1] = __bfloat162float(p.q_pe[row * kPos + 2 * lane + 1]);
    const int64_t seen = len - (p.m - 1 - r / p.H), per = bad ? 0 : (len + p.parts - 1) / p.parts;
    const int64_t j0 = blockIdx.x * per, j1 = min(seen, j0 + per);
    for (int64_t j = j0; j < j1; ++j) {
        const uint32_t entry = (uint32_t)j / (uint32_t)p.cache.page_size, in = (uint32_t)j - entry * (uint32_t)p.cache.page_size;
        const int32_t page = p.cache.table[(int64_t)n * p.cache.max_pages + entry];
        if (page < 0 || page >= p.cache.num_pages) {
            bad = true;
            if (lane == 0) set_status(p.status, KDA_ERR_PAGES);
            break;
        }
        const uint8_t *base = p.cache.rows + page * p.cache.page_stride, *src = base + (int64_t)in * kRow8;
        const float s = *(reinterpret_cast<const float *>(base + (int64_t)p.cache.page_size * kRow8) + in);
        const uint4 u = *reinterpret_cast<const uint4 *>(src + 16 * lane);
        const __nv_bfloat162 pe = *reinterpret_cast<const __nv_bfloat162 *>(src + kLatent + 4 * lane);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        float v[16], dot = qp[0] * __low2float(pe) + qp[1] * __high2float(pe);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 a = values_of2(w[i >> 1] >> (16 * (i & 1)));
            v[2 * i] = a.x, v[2 * i + 1] = a.y;
            dot += q[2 * i] * a.x + q[2 * i + 1] * a.y;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        const float x = dot * s * p.scale, top = fmaxf(m, x), f = top == -INFINITY ? 1.f : expf(m - top);
        const float e = x == -INFINITY ? 0.f : expf(x - top);  // NaN for a NaN
        l = l * f + e;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = o[i] * f + e * s * v[i];
        m = top;
    }
    if (lane == 0) p.part_ml[at] = make_float2(m, bad ? __int_as_float(0x7fffffff) : l);
#pragma unroll
    for (int i = 0; i < 16; ++i) p.part_o[at * kLatent + 16 * lane + i] = o[i];
}

__global__ void __launch_bounds__(128) kda_mla_join_fp8_kernel(const __grid_constant__ Decode8Args p) {
    pdl_wait();
    const int64_t row = blockIdx.x, rows = (int64_t)p.N * p.R;
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < p.parts; ++i) m = fmaxf(m, p.part_ml[i * rows + row].x);
    for (int i = 0; i < p.parts; ++i) {
        const float2 ml = p.part_ml[i * rows + row];
        const float f = ml.x == -INFINITY ? 0.f : expf(ml.x - m);
        l += ml.y * (ml.y != ml.y ? 1.f : f);
        for (int k = 0; k < 4; ++k) o[k] += f * p.part_o[(i * rows + row) * kLatent + 4 * threadIdx.x + k];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int k = 0; k < 4; ++k) p.o[row * kLatent + 4 * threadIdx.x + k] = __float2bfloat16(l != l ? l : o[k] * inv);
    if (p.lse && threadIdx.x == 0) p.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

int parts_of(int64_t N, int64_t R) {
    const int64_t blocks = N * ((R + kWarps - 1) / kWarps);
    return (int)max((int64_t)1, min((int64_t)kMaxParts, 608 / blocks));
}

}  // namespace
}  // namespace kda

extern "C" {

size_t kda_mla_decode_fp8_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t num_tokens) {
    if (num_seqs < 0 || num_heads < 0 || num_tokens < 0) return 0;
    const int64_t R = (int64_t)num_heads * num_tokens;
    if (R > INT32_MAX / 2 || R == 0 || num_seqs == 0) return 256;
    return (size_t)kda::parts_of(num_seqs, R) * num_seqs * R * (kda::kLatent * 4 + 8);
}

int kda_mla_decode_fp8(const uint16_t *q_lat, const uint16_t *q_pe, const uint8_t *cache, int64_t page_stride,
                       int32_t num_pages, int32_t page_size, const int32_t *page_table, int32_t max_pages,
                       const int32_t *cache_lens, int32_t num_seqs, int32_t num_heads, int32_t num_tokens, float scale,
                       uint16_t *o, float *lse, void *workspace, size_t workspace_bytes, int32_t *status, void *stream) {
    using namespace kda;
    int rc = check_cache<uint8_t>(page_stride, num_pages, page_size, max_pages);
    if (rc != KDA_OK) return rc;
    if (!(scale > 0.0f) || scale > 3.402823466e38f || num_tokens > KDA_MAX_REPLAY_TOKENS) return KDA_ERR_UNSUPPORTED;
    if (num_seqs < 0 || num_heads <= 0 || num_tokens < 0 || num_heads > 65535 ||
        (int64_t)num_seqs * num_heads * num_tokens > INT32_MAX)
        return KDA_ERR_SHAPE;
    if (page_stride >= ((int64_t)1 << 39)) return KDA_ERR_SHAPE;
    if (num_seqs == 0 || num_tokens == 0) return KDA_OK;
    if (!q_lat || !q_pe || !cache || !page_table || !cache_lens || !o || !workspace) return KDA_ERR_NULL;
    if (!mla_aligned(q_lat, 16) || !mla_aligned(q_pe, 16) || !mla_aligned(cache, 16) || !mla_aligned(o, 16) ||
        !mla_aligned(lse, 4) || !mla_aligned(page_table, 4) || !mla_aligned(cache_lens, 4) || !mla_aligned(status, 4) ||
        !mla_aligned(workspace, 256))
        return KDA_ERR_ALIGN;
    if (workspace_bytes < kda_mla_decode_fp8_workspace_size(num_seqs, num_heads, num_tokens)) return KDA_ERR_WORKSPACE;
    if (num_seqs > 65535) return KDA_ERR_SHAPE;
    Decode8Args a{};
    a.q_lat = reinterpret_cast<const __nv_bfloat16 *>(q_lat);
    a.q_pe = reinterpret_cast<const __nv_bfloat16 *>(q_pe);
    a.cache = {cache, page_stride, num_pages, page_size, page_table, max_pages};
    a.lens = cache_lens;
    a.N = num_seqs, a.H = num_heads, a.m = num_tokens, a.R = num_heads * num_tokens;
    a.parts = parts_of(a.N, a.R);
    a.scale = scale;
    a.o = reinterpret_cast<__nv_bfloat16 *>(o);
    a.lse = lse;
    const int64_t rows = (int64_t)a.N * a.R;
    a.part_o = static_cast<float *>(workspace);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + a.parts * rows * kLatent);
    a.status = status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (launch_after(kda_mla_decode_fp8_kernel, dim3(a.parts, a.N, (a.R + kWarps - 1) / kWarps), dim3(kWarps * 32), 0, st, a) != cudaSuccess ||
        launch_after(kda_mla_join_fp8_kernel, dim3((unsigned)rows), dim3(128), 0, st, a) != cudaSuccess)
        return KDA_ERR_CUDA;
    return KDA_OK;
}

}  // extern "C"
