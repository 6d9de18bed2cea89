// The rows of the latent cache: kda_mla_append writes them, kda_mla_gather reads them back.
//
// append: row = ( c / sqrt(mean(c^2) + eps) * w , R(pos) k_pe ), q_out = R(pos) q_pe, in fp32
// and rounded once. gather: a copy. Both are bound by their bytes: a token's row is read
// once and written once (2304 B), a query head's 64 values too (256 B).
//
// One warp takes one item of a token: item 0 its row, the others 16 query heads each. A
// lane holds 16 latent values in two 16-byte accesses, so the sum of squares is one warp
// reduction and nothing passes through shared memory; 8 lanes rotate one head, four pairs a
// lane. gather gives a warp four rows, nine 16-byte accesses a lane, all in flight at once.

#include "kda_latent_common.cuh"

namespace kda {
namespace {

constexpr int kRowThreads = 256;
constexpr int kHeadsPerItem = 16;
constexpr int kGatherRows = 4;
constexpr int kRowUnits = kRow * 2 / 16;  // 16-byte units of a row: 72

struct AppendArgs {
    const __nv_bfloat16 *c, *k_pe;
    int64_t c_stride, k_pe_stride;
    const float *norm_w;
    float eps;
    const float *rope;
    int32_t rope_len, interleaved;
    const __nv_bfloat16 *q_pe;
    int64_t q_ts, q_hs;
    __nv_bfloat16 *q_out;
    int64_t qo_ts, qo_hs;
    int32_t H, items;  // items of a token: 1 + ceil(H / 16), or 1
    const int32_t *cu, *lens;
    PagedRows<__nv_bfloat16> cache;
    int64_t T;
    int32_t N;
    int64_t per_seq;  // tokens of each sequence without cu
    int32_t *status;
};

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// The 64 positional values of one head, by 8 lanes. A lane loads the two 8-byte pieces that
// hold its four pairs: pairs (i, i + 32) for i = 4 j .. 4 j + 3, or (2 i, 2 i + 1) of the
// same i, whose pieces are adjacent.
struct PosPiece {
    uint2 a, b;
};
__device__ __forceinline__ PosPiece load_pos(const __nv_bfloat16 *p, int j, bool interleaved) {
    PosPiece v;
    if (interleaved) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p + 8 * j);
        v.a = make_uint2(u.x, u.y);
        v.b = make_uint2(u.z, u.w);
    } else {
        v.a = *reinterpret_cast<const uint2 *>(p + 4 * j);
        v.b = *reinterpret_cast<const uint2 *>(p + 32 + 4 * j);
    }
    return v;
}
__device__ __forceinline__ void store_pos(__nv_bfloat16 *p, int j, bool interleaved, const PosPiece &v) {
    if (interleaved) {
        *reinterpret_cast<uint4 *>(p + 8 * j) = make_uint4(v.a.x, v.a.y, v.b.x, v.b.y);
    } else {
        *reinterpret_cast<uint2 *>(p + 4 * j) = v.a;
        *reinterpret_cast<uint2 *>(p + 32 + 4 * j) = v.b;
    }
}
__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    const float x = a * c - b * s;
    b = b * c + a * s;
    a = x;
}
__device__ __forceinline__ PosPiece rotate(const PosPiece &v, const float4 &c, const float4 &s, bool interleaved) {
    float x[8];
    unpack8(make_uint4(v.a.x, v.a.y, v.b.x, v.b.y), x);
    if (interleaved) {
        turn(x[0], x[1], c.x, s.x);
        turn(x[2], x[3], c.y, s.y);
        turn(x[4], x[5], c.z, s.z);
        turn(x[6], x[7], c.w, s.w);
    } else {
        turn(x[0], x[4], c.x, s.x);
        turn(x[1], x[5], c.y, s.y);
        turn(x[2], x[6], c.z, s.z);
        turn(x[3], x[7], c.w, s.w);
    }
    const uint4 u = pack8(x);
    return PosPiece{make_uint2(u.x, u.y), make_uint2(u.z, u.w)};
}

__global__ void __launch_bounds__(kRowThreads) kda_mla_append_kernel(const __grid_constant__ AppendArgs p) {
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = item / p.items;
    const int part = (int)(item - t * p.items);
    if (t >= p.T) return;

    // the loads that need no position first
    uint4 lo, hi;
    PosPiece pe[kHeadsPerItem / 4];
    const bool il = p.interleaved != 0;
    const int j = lane & 7, h0 = (part - 1) * kHeadsPerItem + (lane >> 3);
    if (part == 0) {
        const __nv_bfloat16 *c = p.c + t * p.c_stride;
        lo = *reinterpret_cast<const uint4 *>(c + 8 * lane);
        hi = *reinterpret_cast<const uint4 *>(c + 256 + 8 * lane);
        if (lane < 8) pe[0] = load_pos(p.k_pe + t * p.k_pe_stride, j, il);
    } else {
#pragma unroll
        for (int i = 0; i < kHeadsPerItem / 4; ++i)
            if (h0 + 4 * i < p.H) pe[i] = load_pos(p.q_pe + t * p.q_ts + (h0 + 4 * i) * p.q_hs, j, il);
    }

    int n;
    int64_t end;
    if (p.cu) {
        n = warp_find_seq(p.cu, p.N, t);
        if (n < 0) return;  // before the first sequence
        end = p.cu[n + 1];
        if (t >= end) return;  // behind the last one
    } else {
        n = (int)(t / p.per_seq);
        end = (n + 1) * p.per_seq;
    }
    const int64_t pos = p.lens[n] - (end - t);
    const int64_t entry = pos >= 0 ? pos / p.cache.page_size : -1;
    bool good = entry >= 0 && entry < p.cache.max_pages && (p.rope == nullptr || pos < p.rope_len);
    if (!good && lane == 0) set_status(p.status, KDA_ERR_SEQLENS);

    float4 co = make_float4(1.f, 1.f, 1.f, 1.f), si = make_float4(0.f, 0.f, 0.f, 0.f);
    if (good && p.rope) {
        co = *reinterpret_cast<const float4 *>(p.rope + pos * kPos + 4 * j);
        si = *reinterpret_cast<const float4 *>(p.rope + pos * kPos + kPos / 2 + 4 * j);
    }
    int32_t page = -1;
    if (good) page = p.cache.table[(int64_t)n * p.cache.max_pages + entry];
    if (good && (page < 0 || page >= p.cache.num_pages)) {
        good = false;
        if (lane == 0) set_status(p.status, KDA_ERR_PAGES);
    }

    if (part == 0) {
        if (!good) return;
        __nv_bfloat16 *row = p.cache.rows + page * p.cache.page_stride + (pos - entry * p.cache.page_size) * kRow;
        if (p.norm_w) {
            float x[8], y[8];
            unpack8(lo, x);
            unpack8(hi, y);
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += x[i] * x[i] + y[i] * y[i];
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            const float r = 1.0f / sqrtf(ss * (1.0f / kLatent) + p.eps);
            float w[8];
            *reinterpret_cast<float4 *>(&w[0]) = __ldg(reinterpret_cast<const float4 *>(p.norm_w + 8 * lane));
            *reinterpret_cast<float4 *>(&w[4]) = __ldg(reinterpret_cast<const float4 *>(p.norm_w + 8 * lane + 4));
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
            lo = pack8(x);
            *reinterpret_cast<float4 *>(&w[0]) = __ldg(reinterpret_cast<const float4 *>(p.norm_w + 256 + 8 * lane));
            *reinterpret_cast<float4 *>(&w[4]) = __ldg(reinterpret_cast<const float4 *>(p.norm_w + 256 + 8 * lane + 4));
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = y[i] * r * w[i];
            hi = pack8(y);
        }
        *reinterpret_cast<uint4 *>(row + 8 * lane) = lo;
        *reinterpret_cast<uint4 *>(row + 256 + 8 * lane) = hi;
        if (lane < 8) store_pos(row + kLatent, j, il, p.rope ? rotate(pe[0], co, si, il) : pe[0]);
        return;
    }
    const PosPiece nan{make_uint2(0x7fff7fffu, 0x7fff7fffu), make_uint2(0x7fff7fffu, 0x7fff7fffu)};
#pragma unroll
    for (int i = 0; i < kHeadsPerItem / 4; ++i)
        if (h0 + 4 * i < p.H)
            store_pos(p.q_out + t * p.qo_ts + (h0 + 4 * i) * p.qo_hs, j, il, good ? rotate(pe[i], co, si, il) : nan);
}

__global__ void __launch_bounds__(kRowThreads)
    kda_mla_gather_kernel(const PagedRows<const __nv_bfloat16> cache, const int32_t *cu, int32_t N, int64_t T,
                          __nv_bfloat16 *out, int32_t *status) {
    const int lane = threadIdx.x & 31;
    const int64_t t0 = ((int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * kGatherRows;
    if (t0 >= T) return;
    // the four rows' places: nullptr = none (outside every sequence), NaN rows flagged
    const __nv_bfloat16 *src[kGatherRows];
    unsigned nan_rows = 0;
    int n = warp_find_seq(cu, N, t0);
#pragma unroll
    for (int r = 0; r < kGatherRows; ++r) {
        const int64_t t = t0 + r;
        src[r] = nullptr;
        while (n + 1 < N && t >= cu[n + 1]) ++n;  // empty sequences are stepped over
        if (n < 0 || t >= T || t >= cu[n + 1] || t < cu[n]) continue;
        const int64_t i = t - cu[n], entry = i / cache.page_size;
        int32_t page = -1;
        if (entry < cache.max_pages) page = cache.table[(int64_t)n * cache.max_pages + entry];
        if (page < 0 || page >= cache.num_pages) {
            nan_rows |= 1u << r;
            if (lane == 0) set_status(status, entry < cache.max_pages ? KDA_ERR_PAGES : KDA_ERR_SEQLENS);
            continue;
        }
        src[r] = cache.rows + page * cache.page_stride + (i - entry * cache.page_size) * kRow;
    }
    constexpr int kAcc = kGatherRows * kRowUnits / 32;  // 9
    uint4 v[kAcc];
    bool there[kAcc];
#pragma unroll
    for (int k = 0; k < kAcc; ++k) {
        const int u = k * 32 + lane, r = u / kRowUnits, c = u - r * kRowUnits;
        const __nv_bfloat16 *s = r == 0 ? src[0] : (r == 1 ? src[1] : (r == 2 ? src[2] : src[3]));
        const bool nan = (nan_rows >> r) & 1;
        there[k] = nan || s != nullptr;
        v[k] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
        if (s) v[k] = __ldg(reinterpret_cast<const uint4 *>(s + 8 * c));
    }
#pragma unroll
    for (int k = 0; k < kAcc; ++k)
        if (there[k]) reinterpret_cast<uint4 *>(out + t0 * kRow)[k * 32 + lane] = v[k];
}

}  // namespace
}  // namespace kda

extern "C" {

int kda_mla_append(const uint16_t *c, int64_t c_stride, const uint16_t *k_pe, int64_t k_pe_stride,
                   const float *norm_w, float eps, const float *rope, int32_t rope_len, int32_t rope_interleaved,
                   const uint16_t *q_pe, int64_t q_token_stride, int64_t q_head_stride, uint16_t *q_out,
                   int64_t q_out_token_stride, int64_t q_out_head_stride, int32_t num_heads,
                   const int32_t *cu_seqlens, const int32_t *cache_lens, const int32_t *page_table, int32_t max_pages,
                   uint16_t *cache, int64_t page_stride, int32_t num_pages, int32_t page_size, int64_t total_tokens,
                   int32_t num_seqs, int32_t *status, void *stream) {
    using namespace kda;
    int rc = check_cache(page_stride, num_pages, page_size, max_pages);
    if (rc != KDA_OK) return rc;
    if (!(eps >= 0.0f) || (rope_interleaved != 0 && rope_interleaved != 1)) return KDA_ERR_UNSUPPORTED;
    if ((q_pe != nullptr) != (q_out != nullptr) || (q_pe && !rope)) return KDA_ERR_UNSUPPORTED;
    if (total_tokens < 0 || total_tokens > INT32_MAX || num_seqs < 0 || rope_len < 0) return KDA_ERR_SHAPE;
    if (num_seqs == 0 && total_tokens > 0 && !cu_seqlens) return KDA_ERR_SHAPE;
    if (!cu_seqlens && num_seqs > 0 && total_tokens % num_seqs != 0) return KDA_ERR_SHAPE;
    if (c_stride < kLatent || c_stride % 8 || k_pe_stride < kPos || k_pe_stride % 8) return KDA_ERR_SHAPE;
    if (q_pe) {
        if (num_heads <= 0 || num_heads > 65535) return KDA_ERR_SHAPE;
        if (q_token_stride < 0 || q_head_stride < 0 || q_token_stride % 8 || q_head_stride % 8) return KDA_ERR_SHAPE;
        // distinct heads and tokens must not overlap in the output, in either order of the axes
        const int64_t ts = q_out_token_stride, hs = q_out_head_stride;
        if (ts < 0 || hs < 0 || ts % 8 || hs % 8) return KDA_ERR_SHAPE;
        auto apart = [](int64_t inner_n, int64_t inner, int64_t outer_n, int64_t outer) {
            return (inner_n <= 1 || inner >= kPos) &&
                   (outer_n <= 1 || (__int128)outer >= (__int128)(inner_n - 1) * inner + kPos);
        };
        if (!apart(num_heads, hs, total_tokens, ts) && !apart(total_tokens, ts, num_heads, hs)) return KDA_ERR_SHAPE;
    }
    if (num_seqs == 0 || total_tokens == 0) return KDA_OK;
    if (!c || !k_pe || !cache_lens || !page_table || !cache) return KDA_ERR_NULL;
    if (!mla_aligned(c, 16) || !mla_aligned(k_pe, 16) || !mla_aligned(norm_w, 16) || !mla_aligned(rope, 16) ||
        !mla_aligned(q_pe, 16) || !mla_aligned(q_out, 16) || !mla_aligned(cache, 16) || !mla_aligned(cu_seqlens, 4) ||
        !mla_aligned(cache_lens, 4) || !mla_aligned(page_table, 4) || !mla_aligned(status, 4))
        return KDA_ERR_ALIGN;
    AppendArgs a{};
    a.c = reinterpret_cast<const __nv_bfloat16 *>(c);
    a.k_pe = reinterpret_cast<const __nv_bfloat16 *>(k_pe);
    a.c_stride = c_stride;
    a.k_pe_stride = k_pe_stride;
    a.norm_w = norm_w;
    a.eps = eps;
    a.rope = rope;
    a.rope_len = rope_len;
    a.interleaved = rope_interleaved;
    a.q_pe = reinterpret_cast<const __nv_bfloat16 *>(q_pe);
    a.q_ts = q_token_stride;
    a.q_hs = q_head_stride;
    a.q_out = reinterpret_cast<__nv_bfloat16 *>(q_out);
    a.qo_ts = q_out_token_stride;
    a.qo_hs = q_out_head_stride;
    a.H = num_heads;
    a.items = 1 + (q_pe ? (num_heads + kHeadsPerItem - 1) / kHeadsPerItem : 0);
    a.cu = cu_seqlens;
    a.lens = cache_lens;
    a.cache = {reinterpret_cast<__nv_bfloat16 *>(cache), page_stride, num_pages, page_size, page_table, max_pages};
    a.T = total_tokens;
    a.N = num_seqs;
    a.per_seq = cu_seqlens ? 0 : total_tokens / num_seqs;
    a.status = status;
    const int64_t blocks = (total_tokens * a.items + kRowThreads / 32 - 1) / (kRowThreads / 32);
    if (blocks > INT32_MAX) return KDA_ERR_SHAPE;
    kda_mla_append_kernel<<<(unsigned)blocks, kRowThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int kda_mla_gather(const uint16_t *cache, int64_t page_stride, int32_t num_pages, int32_t page_size,
                   const int32_t *cu_seqlens, const int32_t *page_table, int32_t max_pages, uint16_t *out,
                   int64_t total_rows, int32_t num_seqs, int32_t *status, void *stream) {
    using namespace kda;
    int rc = check_cache(page_stride, num_pages, page_size, max_pages);
    if (rc != KDA_OK) return rc;
    if (total_rows < 0 || total_rows > INT32_MAX || num_seqs < 0) return KDA_ERR_SHAPE;
    if (num_seqs == 0 || total_rows == 0) return KDA_OK;
    if (!cache || !cu_seqlens || !page_table || !out) return KDA_ERR_NULL;
    if (!mla_aligned(cache, 16) || !mla_aligned(out, 16) || !mla_aligned(cu_seqlens, 4) || !mla_aligned(page_table, 4) ||
        !mla_aligned(status, 4))
        return KDA_ERR_ALIGN;
    const int64_t per_block = kGatherRows * (kRowThreads / 32);
    const unsigned blocks = (unsigned)((total_rows + per_block - 1) / per_block);
    const PagedRows<const __nv_bfloat16> pr{reinterpret_cast<const __nv_bfloat16 *>(cache), page_stride, num_pages,
                                            page_size, page_table, max_pages};
    kda_mla_gather_kernel<<<blocks, kRowThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        pr, cu_seqlens, num_seqs, total_rows, reinterpret_cast<__nv_bfloat16 *>(out), status);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
