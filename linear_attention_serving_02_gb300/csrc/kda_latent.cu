// The rows of the latent cache: kda_mla_append writes them, kda_mla_gather reads them back; the _fp8 calls are the same
// for the cache in 8 bits.
//
// append: row = ( c / sqrt(mean(c^2) + eps) * w , R(pos) k_pe ), q_out = R(pos) q_pe, in fp32
// and rounded once; in 8 bits the row is divided by its scale before, the least power of two 2^e with
// max|latent| 2^-e <= 448, which moves no bit of the bf16 part. gather: a copy, or the values times their scale. All
// are bound by their bytes: a token's row is read once and written once (2304 B, in 8 bits 1796 B), a query
// head's 64 values too (256 B).
//
// A warp takes a token's row and its first 16 query heads; further heads go 16 to a warp. A
// lane holds 16 latent values in two 16-byte accesses, so the sum of squares and the largest magnitude are one warp
// reduction each and nothing passes through shared memory; four lanes rotate one head, eight pairs a
// lane in two 16-byte accesses. All of a warp's loads are issued before it looks up where the
// token goes; the queries, which then wait for nothing more, are through before the row, so that fewer values live
// at once (65536 tokens x 12 heads in 8 bits: 61.0 us, 59.7 so). gather gives a warp four rows, nine 16-byte
// accesses a lane, all in flight at once. Blocks are one or two warps: a larger one waits for its slowest token and
// frees its registers late (append in 8 bits with 1, 2 and 4 warps 59.7, 57.0 and 58.6 us).
//
// Measured: append of 65536 tokens x 12 heads 56.4 us (6.2 TB/s), in 8 bits 56.7 (5.6 TB/s: fewer bytes, the same
// chain of a token's loads), of 256 tokens x 96 heads 3.0 us (a launch and three dependent loads); gather of 108000 rows
// 40.6 us (6.2 TB/s), in 8 bits 32.9 (5.9 TB/s), of 330 rows 3.3 us (eight rows a warp: 43.7 and 6.0 us).

#include "kda_common.cuh"
#include "kda_latent_common.cuh"

namespace kda {
namespace {

constexpr int kRowThreads = 32, kAppendThreads = 64, kGather8Threads = 64;
constexpr int kHeadsPerItem = 16;
constexpr int kGatherRows = 4;
constexpr int kRowUnits = kRow * 2 / 16;  // 16-byte units of a row: 72

// T: the cache's elements, bf16 values or the bytes of its 8-bit form
template <typename T>
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
    int32_t H;  // 0 without queries
    const int32_t *cu, *lens;
    PagedRows<T> cache;
    int64_t tokens;
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

// The 64 positional values of one head, by 4 lanes. A lane loads the two 16-byte pieces that
// hold its eight pairs: pairs (i, i + 32) for i = 8 j .. 8 j + 7, or (2 i, 2 i + 1) of the
// same i, whose pieces are adjacent.
struct PosPiece {
    uint4 a, b;
};
__device__ __forceinline__ int piece_at(int j, int second, bool interleaved) {
    return interleaved ? 16 * j + 8 * second : 8 * j + 32 * second;
}
__device__ __forceinline__ PosPiece load_pos(const __nv_bfloat16 *p, int j, bool interleaved) {
    return PosPiece{*reinterpret_cast<const uint4 *>(p + piece_at(j, 0, interleaved)),
                    *reinterpret_cast<const uint4 *>(p + piece_at(j, 1, interleaved))};
}
__device__ __forceinline__ void store_pos(__nv_bfloat16 *p, int j, bool interleaved, const PosPiece &v) {
    *reinterpret_cast<uint4 *>(p + piece_at(j, 0, interleaved)) = v.a;
    *reinterpret_cast<uint4 *>(p + piece_at(j, 1, interleaved)) = v.b;
}
__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    const float x = a * c - b * s;
    b = b * c + a * s;
    a = x;
}
__device__ __forceinline__ PosPiece rotate(const PosPiece &v, const float (&c)[8], const float (&s)[8], bool interleaved) {
    float x[8], y[8];
    unpack8(v.a, x);
    unpack8(v.b, y);
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            turn(x[2 * i], x[2 * i + 1], c[i], s[i]);
            turn(y[2 * i], y[2 * i + 1], c[i + 4], s[i + 4]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn(x[i], y[i], c[i], s[i]);
    }
    return PosPiece{pack8(x), pack8(y)};
}
// eight bf16 values times a power of two
__device__ __forceinline__ uint4 scaled8(const uint4 &u, float by) {
    float x[8];
    unpack8(u, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= by;
    return pack8(x);
}
// eight values times a power of two, each rounded to the nearest e4m3
__device__ __forceinline__ uint2 e4m3_of8(const float (&x)[8], float by) {
    return make_uint2(e4m3_of2(x[0] * by, x[1] * by) | (e4m3_of2(x[2] * by, x[3] * by) << 16),
                      e4m3_of2(x[4] * by, x[5] * by) | (e4m3_of2(x[6] * by, x[7] * by) << 16));
}
__device__ __forceinline__ void load8(float (&x)[8], const float *p) {
    *reinterpret_cast<float4 *>(&x[0]) = *reinterpret_cast<const float4 *>(p);
    *reinterpret_cast<float4 *>(&x[4]) = *reinterpret_cast<const float4 *>(p + 4);
}

template <typename T>
__global__ void __launch_bounds__(kAppendThreads) kda_mla_append_kernel(const __grid_constant__ AppendArgs<T> p) {
    constexpr bool kBits8 = sizeof(T) == 1;
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const int part = blockIdx.y;
    pdl_wait();
    if (t >= p.tokens) return;

    // the loads that need no position first
    uint4 lo, hi;
    PosPiece k_pe, q[kHeadsPerItem / 8];
    const bool il = p.interleaved != 0;
    const int j = lane & 3, h0 = part * kHeadsPerItem + (lane >> 2);
    if (part == 0) {
        const __nv_bfloat16 *c = p.c + t * p.c_stride;
        lo = *reinterpret_cast<const uint4 *>(c + 8 * lane);
        hi = *reinterpret_cast<const uint4 *>(c + 256 + 8 * lane);
        if (lane < 4) k_pe = load_pos(p.k_pe + t * p.k_pe_stride, j, il);
    }
#pragma unroll
    for (int i = 0; i < kHeadsPerItem / 8; ++i)
        if (h0 + 8 * i < p.H) q[i] = load_pos(p.q_pe + t * p.q_ts + (h0 + 8 * i) * p.q_hs, j, il);

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
    const uint32_t entry = (uint32_t)max(pos, (int64_t)0) / (uint32_t)p.cache.page_size;
    bool good = pos >= 0 && entry < (uint32_t)p.cache.max_pages && (p.rope == nullptr || pos < p.rope_len);
    if (!good && lane == 0) set_status(p.status, KDA_ERR_SEQLENS);

    float co[8], si[8];
    int32_t page = -1;
    if (good) {
        if (p.rope) {
            load8(co, p.rope + pos * kPos + 8 * j);
            load8(si, p.rope + pos * kPos + kPos / 2 + 8 * j);
        }
        page = p.cache.table[(int64_t)n * p.cache.max_pages + entry];
        if (page < 0 || page >= p.cache.num_pages) {
            good = false;
            if (lane == 0) set_status(p.status, KDA_ERR_PAGES);
        }
    }

    const uint4 nan4 = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
#pragma unroll
    for (int i = 0; i < kHeadsPerItem / 8; ++i)
        if (h0 + 8 * i < p.H)
            store_pos(p.q_out + t * p.qo_ts + (h0 + 8 * i) * p.qo_hs, j, il,
                      good ? rotate(q[i], co, si, il) : PosPiece{nan4, nan4});

    if (part == 0 && good) {
        T *page_at = p.cache.rows + page * p.cache.page_stride;
        const uint32_t r_in_page = (uint32_t)pos - entry * (uint32_t)p.cache.page_size;
        float x[8], y[8];
        auto normalise = [&] {
            float w[8];
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += x[i] * x[i] + y[i] * y[i];
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            const float r = 1.0f / sqrtf(ss * (1.0f / kLatent) + p.eps);
            load8(w, p.norm_w + 8 * lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
            load8(w, p.norm_w + 256 + 8 * lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = y[i] * r * w[i];
        };
        if constexpr (kBits8) {
            unpack8(lo, x);
            unpack8(hi, y);
            if (p.norm_w) normalise();
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaxf(fabsf(x[i]), fabsf(y[i])));
            // magnitudes are in the order of their bits
            top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
            const int e = scale_exponent(top);
            const float inv = exp2_of(-e);
            uint8_t *row = page_at + (int64_t)r_in_page * kRow8;
            *reinterpret_cast<uint2 *>(row + 8 * lane) = e4m3_of8(x, inv);
            *reinterpret_cast<uint2 *>(row + 256 + 8 * lane) = e4m3_of8(y, inv);
            if (lane < 4) {
                __nv_bfloat16 *at = reinterpret_cast<__nv_bfloat16 *>(row + kLatent);
                const PosPiece turned = p.rope ? rotate(k_pe, co, si, il) : k_pe;
                // a power of two: the bf16 values stay what they are
                store_pos(at, j, il, PosPiece{scaled8(turned.a, inv), scaled8(turned.b, inv)});
            }
            if (lane == 0)
                *reinterpret_cast<float *>(page_at + (int64_t)p.cache.page_size * kRow8 + 4 * r_in_page) = exp2_of(e);
        } else {
            __nv_bfloat16 *row = page_at + (int64_t)r_in_page * kRow;
            if (p.norm_w) {
                unpack8(lo, x);
                unpack8(hi, y);
                normalise();
                lo = pack8(x);
                hi = pack8(y);
            }
            *reinterpret_cast<uint4 *>(row + 8 * lane) = lo;
            *reinterpret_cast<uint4 *>(row + 256 + 8 * lane) = hi;
            if (lane < 4) store_pos(row + kLatent, j, il, p.rope ? rotate(k_pe, co, si, il) : k_pe);
        }
    }
}

__global__ void __launch_bounds__(kRowThreads)
    kda_mla_gather_kernel(const PagedRows<const __nv_bfloat16> cache, const int32_t *cu, int32_t N, int64_t T,
                          __nv_bfloat16 *out, int32_t *status) {
    const int lane = threadIdx.x & 31;
    const int64_t t0 = ((int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * kGatherRows;
    pdl_wait();
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
        const uint32_t i = (uint32_t)(t - cu[n]), entry = i / (uint32_t)cache.page_size;
        int32_t page = -1;
        if (entry < (uint32_t)cache.max_pages) page = cache.table[(int64_t)n * cache.max_pages + entry];
        if (page < 0 || page >= cache.num_pages) {
            nan_rows |= 1u << r;
            if (lane == 0) set_status(status, entry < (uint32_t)cache.max_pages ? KDA_ERR_PAGES : KDA_ERR_SEQLENS);
            continue;
        }
        src[r] = cache.rows + page * cache.page_stride + (int64_t)(i - entry * (uint32_t)cache.page_size) * kRow;
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
        if (s) v[k] = *reinterpret_cast<const uint4 *>(s + 8 * c);
    }
#pragma unroll
    for (int k = 0; k < kAcc; ++k)
        if (there[k]) reinterpret_cast<uint4 *>(out + t0 * kRow)[k * 32 + lane] = v[k];
}

// four e4m3 values (a 32-bit word) times s, as two words of bf16 pairs
__device__ __forceinline__ uint2 bf16_of4(uint32_t v, float s) {
    const float2 a = values_of2(v), b = values_of2(v >> 16);
    return make_uint2(pack2(a.x * s, a.y * s), pack2(b.x * s, b.y * s));
}

__global__ void __launch_bounds__(kGather8Threads)
    kda_mla_gather_fp8_kernel(const PagedRows<const uint8_t> cache, const int32_t *cu, const int32_t *starts, int32_t N,
                              int64_t T, __nv_bfloat16 *out, int32_t *status) {
    const int lane = threadIdx.x & 31;
    const int64_t t0 = ((int64_t)blockIdx.x * (kGather8Threads / 32) + (threadIdx.x >> 5)) * kGatherRows;
    pdl_wait();
    if (t0 >= T) return;
    const uint8_t *src[kGatherRows];
    const float *scale_at[kGatherRows];
    unsigned nan_rows = 0;
    int n = warp_find_seq(cu, N, t0);
#pragma unroll
    for (int r = 0; r < kGatherRows; ++r) {
        const int64_t t = t0 + r;
        src[r] = nullptr;
        scale_at[r] = nullptr;
        while (n + 1 < N && t >= cu[n + 1]) ++n;  // empty sequences are stepped over
        if (n < 0 || t >= T || t >= cu[n + 1] || t < cu[n]) continue;
        const int64_t i = t - cu[n] + (starts ? starts[n] : 0);
        const bool there = i >= 0 && i < (int64_t)cache.max_pages * cache.page_size;
        const uint32_t entry = there ? (uint32_t)i / (uint32_t)cache.page_size : 0;
        const int32_t page = there ? cache.table[(int64_t)n * cache.max_pages + entry] : -1;
        if (page < 0 || page >= cache.num_pages) {
            nan_rows |= 1u << r;
            if (lane == 0) set_status(status, there ? KDA_ERR_PAGES : KDA_ERR_SEQLENS);
            continue;
        }
        const uint8_t *at = cache.rows + page * cache.page_stride;
        const uint32_t in_page = (uint32_t)i - entry * (uint32_t)cache.page_size;
        src[r] = at + (int64_t)in_page * kRow8;
        scale_at[r] = reinterpret_cast<const float *>(at + (int64_t)cache.page_size * kRow8) + in_page;
    }
    // lane l takes bytes 8 l and 256 + 8 l of every row's latents, so that a store is 512 bytes in one piece (16 bytes read and 32
    // written a lane: 108000 rows 35.7 us, 33.8 so, 33.0 with two warps a block), and unit l % 8 of 16 bytes of row l / 8's positional key
    uint2 v[kGatherRows][2];
    uint4 pe = make_uint4(0, 0, 0, 0);
    float s[kGatherRows];
#pragma unroll
    for (int r = 0; r < kGatherRows; ++r) {
        v[r][0] = v[r][1] = make_uint2(0, 0);
        s[r] = ((nan_rows >> r) & 1) ? __uint_as_float(0x7fffffffu) : 1.f;
        if (src[r]) {
            v[r][0] = *reinterpret_cast<const uint2 *>(src[r] + 8 * lane);
            v[r][1] = *reinterpret_cast<const uint2 *>(src[r] + 256 + 8 * lane);
            s[r] = *scale_at[r];
        }
    }
    const int pr = lane >> 3;
    const uint8_t *ps = pr == 0 ? src[0] : (pr == 1 ? src[1] : (pr == 2 ? src[2] : src[3]));
    if (ps) pe = *reinterpret_cast<const uint4 *>(ps + kLatent + 16 * (lane & 7));
#pragma unroll
    for (int r = 0; r < kGatherRows; ++r) {
        if (!src[r] && !((nan_rows >> r) & 1)) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint2 a = bf16_of4(v[r][i].x, s[r]), b = bf16_of4(v[r][i].y, s[r]);
            reinterpret_cast<uint4 *>(out + (t0 + r) * kRow + 256 * i)[lane] = make_uint4(a.x, a.y, b.x, b.y);
        }
    }
    if (ps || ((nan_rows >> pr) & 1)) {
        const float sp = pr == 0 ? s[0] : (pr == 1 ? s[1] : (pr == 2 ? s[2] : s[3]));
        reinterpret_cast<uint4 *>(out + (t0 + pr) * kRow + kLatent)[lane & 7] = scaled8(pe, sp);
    }
}

// The checks and the launch of both forms of append.
template <typename T>
int append_call(const uint16_t *c, int64_t c_stride, const uint16_t *k_pe, int64_t k_pe_stride,
                const float *norm_w, float eps, const float *rope, int32_t rope_len, int32_t rope_interleaved,
                const uint16_t *q_pe, int64_t q_token_stride, int64_t q_head_stride, uint16_t *q_out,
                int64_t q_out_token_stride, int64_t q_out_head_stride, int32_t num_heads, const int32_t *cu_seqlens,
                const int32_t *cache_lens, const int32_t *page_table, int32_t max_pages, T *cache, int64_t page_stride,
                int32_t num_pages, int32_t page_size, int64_t total_tokens, int32_t num_seqs, int32_t *status,
                void *stream) {
    const int rc = check_cache<T>(page_stride, num_pages, page_size, max_pages);
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
    AppendArgs<T> a{};
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
    a.H = q_pe ? num_heads : 0;
    a.cu = cu_seqlens;
    a.lens = cache_lens;
    a.cache = {cache, page_stride, num_pages, page_size, page_table, max_pages};
    a.tokens = total_tokens;
    a.N = num_seqs;
    a.per_seq = cu_seqlens ? 0 : total_tokens / num_seqs;
    a.status = status;
    const int64_t blocks = (total_tokens + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
    const int parts = a.H > kHeadsPerItem ? (a.H + kHeadsPerItem - 1) / kHeadsPerItem : 1;
    return launch_after(kda_mla_append_kernel<T>, dim3((unsigned)blocks, (unsigned)parts), dim3(kAppendThreads), 0,
                        static_cast<cudaStream_t>(stream), a) == cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
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
    return kda::append_call(c, c_stride, k_pe, k_pe_stride, norm_w, eps, rope, rope_len, rope_interleaved, q_pe,
                            q_token_stride, q_head_stride, q_out, q_out_token_stride, q_out_head_stride, num_heads,
                            cu_seqlens, cache_lens, page_table, max_pages, reinterpret_cast<__nv_bfloat16 *>(cache),
                            page_stride, num_pages, page_size, total_tokens, num_seqs, status, stream);
}

int kda_mla_gather(const uint16_t *cache, int64_t page_stride, int32_t num_pages, int32_t page_size,
                   const int32_t *cu_seqlens, const int32_t *page_table, int32_t max_pages, uint16_t *out,
                   int64_t total_rows, int32_t num_seqs, int32_t *status, void *stream) {
    using namespace kda;
    int rc = check_cache<__nv_bfloat16>(page_stride, num_pages, page_size, max_pages);
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
    return launch_after(kda_mla_gather_kernel, dim3(blocks), dim3(kRowThreads), 0, static_cast<cudaStream_t>(stream), pr,
                        cu_seqlens, num_seqs, total_rows, reinterpret_cast<__nv_bfloat16 *>(out), status) == cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

int kda_mla_append_fp8(const uint16_t *c, int64_t c_stride, const uint16_t *k_pe, int64_t k_pe_stride,
                       const float *norm_w, float eps, const float *rope, int32_t rope_len, int32_t rope_interleaved,
                       const uint16_t *q_pe, int64_t q_token_stride, int64_t q_head_stride, uint16_t *q_out,
                       int64_t q_out_token_stride, int64_t q_out_head_stride, int32_t num_heads,
                       const int32_t *cu_seqlens, const int32_t *cache_lens, const int32_t *page_table,
                       int32_t max_pages, uint8_t *cache, int64_t page_stride, int32_t num_pages, int32_t page_size,
                       int64_t total_tokens, int32_t num_seqs, int32_t *status, void *stream) {
    return kda::append_call(c, c_stride, k_pe, k_pe_stride, norm_w, eps, rope, rope_len, rope_interleaved, q_pe,
                            q_token_stride, q_head_stride, q_out, q_out_token_stride, q_out_head_stride, num_heads,
                            cu_seqlens, cache_lens, page_table, max_pages, cache, page_stride, num_pages, page_size,
                            total_tokens, num_seqs, status, stream);
}

int kda_mla_gather_fp8(const uint8_t *cache, int64_t page_stride, int32_t num_pages, int32_t page_size,
                       const int32_t *cu_seqlens, const int32_t *starts, const int32_t *page_table, int32_t max_pages,
                       uint16_t *out, int64_t total_rows, int32_t num_seqs, int32_t *status, void *stream) {
    using namespace kda;
    int rc = check_cache<uint8_t>(page_stride, num_pages, page_size, max_pages);
    if (rc != KDA_OK) return rc;
    if (total_rows < 0 || total_rows > INT32_MAX || num_seqs < 0) return KDA_ERR_SHAPE;
    if (num_seqs == 0 || total_rows == 0) return KDA_OK;
    if (!cache || !cu_seqlens || !page_table || !out) return KDA_ERR_NULL;
    if (!mla_aligned(cache, 16) || !mla_aligned(out, 16) || !mla_aligned(cu_seqlens, 4) || !mla_aligned(starts, 4) ||
        !mla_aligned(page_table, 4) || !mla_aligned(status, 4))
        return KDA_ERR_ALIGN;
    const int64_t per_block = kGatherRows * (kGather8Threads / 32);
    const unsigned blocks = (unsigned)((total_rows + per_block - 1) / per_block);
    const PagedRows<const uint8_t> pr{cache, page_stride, num_pages, page_size, page_table, max_pages};
    return launch_after(kda_mla_gather_fp8_kernel, dim3(blocks), dim3(kGather8Threads), 0, static_cast<cudaStream_t>(stream), pr,
                        cu_seqlens, starts, num_seqs, total_rows, reinterpret_cast<__nv_bfloat16 *>(out), status) == cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}

}  // extern "C"
