// Latent attention in the expanded form: kda_mla_prefill.
//
//   s_ij = scale (q_i . k_j),  o_i = sum_j e^{s_ij - M_i} v_j / sum_j e^{s_ij - M_i},
//   lse_i = M_i + log sum_j e^{s_ij - M_i}
//
// one pass over the keys with a running maximum and sum. One warp takes one (query row,
// head); a lane holds 6 of the query's 192 values and 4 of the output's 128.

#include "kda_latent_common.cuh"

namespace kda {
namespace {

struct PrefillArgs {
    const __nv_bfloat16 *q, *kv, *k_pe;
    int64_t k_pe_stride;
    const int32_t *cu_q, *cu_k;
    int64_t Tq, Tk;
    int32_t N, H, causal;
    float scale;
    __nv_bfloat16 *o;
    float *lse;
    int32_t *status;
};

__global__ void __launch_bounds__(256) kda_mla_prefill_kernel(const __grid_constant__ PrefillArgs p) {
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t t = item / p.H;
    const int h = (int)(item - t * p.H);
    if (t >= p.Tq) return;
    const int n = warp_find_seq(p.cu_q, p.N, t);
    if (n < 0) return;
    const int64_t q0 = p.cu_q[n], q1 = p.cu_q[n + 1], k0 = p.cu_k[n], k1 = p.cu_k[n + 1];
    if (q0 < 0 || q1 > p.Tq || q1 < q0 || k0 < 0 || k1 > p.Tk || k1 < k0) {
        if (lane == 0) set_status(p.status, KDA_ERR_SEQLENS);
        return;
    }
    if (t >= q1) return;
    int64_t end = k1 - k0;
    if (p.causal) end = (k1 - k0) - (q1 - q0) + (t - q0) + 1;
    float q[6], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
    for (int i = 0; i < 6; ++i) q[i] = __bfloat162float(p.q[(t * p.H + h) * kQk + lane + 32 * i]) * p.scale;
    for (int64_t j = 0; j < end; ++j) {
        const __nv_bfloat16 *kv = p.kv + ((k0 + j) * p.H + h) * (2 * kNope);
        const __nv_bfloat16 *pe = p.k_pe + (k0 + j) * p.k_pe_stride;
        float s = 0.f;
        for (int i = 0; i < 4; ++i) s += q[i] * __bfloat162float(kv[lane + 32 * i]);
        for (int i = 0; i < 2; ++i) s += q[4 + i] * __bfloat162float(pe[lane + 32 * i]);
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
        const float f = expf(m - base), e = expf(s - base);
        l = l * f + e;
        for (int i = 0; i < 4; ++i) o[i] = o[i] * f + e * __bfloat162float(kv[kNope + lane + 32 * i]);
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int i = 0; i < 4; ++i) p.o[(t * p.H + h) * kNope + lane + 32 * i] = __float2bfloat16(o[i] * inv);
    if (p.lse && lane == 0) p.lse[t * p.H + h] = m + logf(l);
}

}  // namespace
}  // namespace kda

extern "C" int kda_mla_prefill(const uint16_t *q, const uint16_t *kv, const uint16_t *k_pe, int64_t k_pe_stride,
                               const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int64_t total_q,
                               int64_t total_k, int32_t num_seqs, int32_t num_heads, int32_t causal, float scale,
                               uint16_t *o, float *lse, int32_t *status, void *stream) {
    using namespace kda;
    if (!(scale > 0.0f) || scale > 3.402823466e38f || (causal != 0 && causal != 1)) return KDA_ERR_UNSUPPORTED;
    if (total_q < 0 || total_k < 0 || total_q > INT32_MAX || total_k > INT32_MAX || num_seqs < 0 || num_heads <= 0 ||
        num_heads > 65535 || k_pe_stride < kPos || k_pe_stride % 8)
        return KDA_ERR_SHAPE;
    if (num_seqs == 0 || total_q == 0) return KDA_OK;
    if (!q || !cu_seqlens_q || !cu_seqlens_k || !o || (total_k > 0 && (!kv || !k_pe))) return KDA_ERR_NULL;
    if (!mla_aligned(q, 16) || !mla_aligned(kv, 16) || !mla_aligned(k_pe, 16) || !mla_aligned(o, 16) ||
        !mla_aligned(lse, 4) || !mla_aligned(cu_seqlens_q, 4) || !mla_aligned(cu_seqlens_k, 4) || !mla_aligned(status, 4))
        return KDA_ERR_ALIGN;
    PrefillArgs a{reinterpret_cast<const __nv_bfloat16 *>(q),
                  reinterpret_cast<const __nv_bfloat16 *>(kv),
                  reinterpret_cast<const __nv_bfloat16 *>(k_pe),
                  k_pe_stride,
                  cu_seqlens_q,
                  cu_seqlens_k,
                  total_q,
                  total_k,
                  num_seqs,
                  num_heads,
                  causal,
                  scale,
                  reinterpret_cast<__nv_bfloat16 *>(o),
                  lse,
                  status};
    const int64_t blocks = (total_q * num_heads + 7) / 8;
    if (blocks > INT32_MAX) return KDA_ERR_SHAPE;
    kda_mla_prefill_kernel<<<(unsigned)blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
