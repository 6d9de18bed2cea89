// What the two decode kernels of latent attention (the cache in bf16 and in 8 bits) share: the cached
// rows of a batch as one list of tiles that is cut into equal runs, the walk over a run, the sums of
// long stretches, and the join of the sequences that a run's border cuts.
//
// Beginning and ending a sequence costs a run time too. In the list a sequence may therefore stand for
// some units more than its tiles, in front of them (SplitArgs::extra: none in the bf16 form; the 8-bit form's
// are measured there), so that a run of many short sequences is given fewer tiles.
#pragma once

#include "kda_common.cuh"
#include "kda_latent_common.cuh"
#include "kda_tma.cuh"

namespace kda {
namespace {

constexpr int kKvTile = 64;           // cached rows of a tile
constexpr int kMaxGroups = 160;       // CTAs that share the list at most
constexpr int kFold = 1024;           // tiles of a stretch that O^T sums in tensor memory (a power of two)

struct SplitGeom {
    int32_t R;        // query rows of a sequence: m H
    int32_t RT, rows; // row tiles and query rows of each (a multiple of 8)
    int32_t npad;     // MMA columns of O^T: rows rounded up to 16
};

struct SplitArgs {
    const int32_t *table, *lens;
    int32_t max_pages, num_pages, page_size;
    int32_t N, H, m, G;
    int32_t extra;    // units that a sequence counts in front of its tiles, where the runs are long enough (extra_of)
    SplitGeom split;
    float scale;      // what a unit of part_ml's maxima is as a natural logarithm
    __nv_bfloat16 *o;
    float *lse;
    float *part_o;   // [2 G, RT, npad, 512]
    float2 *part_ml; // [2 G, RT, npad] reference maximum, in units of `scale`, and sum
    int64_t *head;   // [0]: tiles of the batch; then per group {sequence, first tile, tiles of the sequence}
    int32_t *status;
};

__device__ __forceinline__ bool bad_len(const SplitArgs &p, int64_t len) {
    return len < 0 || len > (int64_t)p.max_pages * p.page_size;
}
// tiles of a sequence in the list: one at least, so that every sequence's output is written
__device__ __forceinline__ int32_t tiles_of(const SplitArgs &p, int32_t len) {
    return bad_len(p, len) || len == 0 ? 1 : (int32_t)(((int64_t)len + kKvTile - 1) / kKvTile);
}

// A run of fewer tiles than four per group gains nothing from evening out.
__device__ __forceinline__ int32_t extra_of(const SplitArgs &p, int64_t tiles) { return tiles >= 4 * (int64_t)p.G ? p.extra : 0; }

// The list's cut into G runs: the first `longer` of them one unit longer than the others.
struct Runs {
    int64_t each;
    int32_t longer;
    __device__ __forceinline__ Runs(int64_t total, int32_t G)
        : each(total <= INT32_MAX ? (int32_t)total / G : total / G), longer((int32_t)(total - each * G)) {}
    __device__ __forceinline__ int64_t begin(int32_t g) const { return g * each + min(g, longer); }
    // the run that holds unit x
    __device__ __forceinline__ int32_t of(int64_t x) const {
        const int64_t in_longer = longer * (each + 1);
        return (int32_t)(x < in_longer ? x / (each + 1) : longer + (x - in_longer) / each);
    }
};

// a run of the list in shared memory: its ends, and where it begins
struct Run {
    int32_t first_seq, first_unit, first_len, extra;  // where it begins: a sequence, a unit of it, its length
    int64_t begin, end;
};

// Group g's run, found by one warp; row tile 0 leaves its place for the join.
__device__ __forceinline__ void find_run(const SplitArgs &p, int g, int rt, Run &run) {
    const int lane = threadIdx.x & 31;
    int64_t total = 0;
    int32_t own = 0;  // length of sequence `lane`: with up to 32 of them the second look loads nothing
    for (int n = lane; n < p.N; n += 32) {
        const int32_t len = p.lens[n];
        if (n == lane) own = len;
        total += tiles_of(p, len);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    const int32_t extra = extra_of(p, total);
    total += (int64_t)p.N * extra;
    const Runs runs(total, p.G);
    const int64_t begin = runs.begin(g), end = runs.begin(g + 1);
    int64_t before = 0;
    int seq = p.N - 1;
    int64_t first = 0;
    int32_t of = 0, first_len = 0;
    for (int n0 = 0; n0 < p.N; n0 += 32) {
        const int n = n0 + lane;
        const int32_t len = n0 == 0 || n >= p.N ? own : p.lens[n];
        const int32_t t = n < p.N ? tiles_of(p, len) : 0, units = n < p.N ? t + extra : 0;
        int64_t incl = units;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += x;
        }
        const int64_t lo = before + incl - units;
        const unsigned mine = __ballot_sync(0xffffffffu, begin >= lo && begin < lo + units);
        if (mine) {
            const int src = __ffs(mine) - 1;
            seq = n0 + src;
            first = begin - __shfl_sync(0xffffffffu, lo, src);
            of = __shfl_sync(0xffffffffu, t, src);
            first_len = __shfl_sync(0xffffffffu, len, src);
            break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
        run.first_seq = seq;
        run.first_unit = (int32_t)first;
        run.first_len = first_len;
        run.extra = extra;
        run.begin = begin;
        run.end = end;
        if (rt == 0) {
            if (g == 0) p.head[0] = total;
            int32_t *e = reinterpret_cast<int32_t *>(p.head + 1) + 4 * g;
            e[0] = seq;
            e[1] = max(0, (int32_t)first - extra);
            e[2] = of;
        }
    }
}

// A walk over a run of the list, one stretch of tiles of one sequence after the other.
struct Walk {
    int32_t n, unit, j0, j1, tiles, len, extra;
    int64_t left;
    bool work;  // the sequence has cached rows and a sound length
    __device__ __forceinline__ void open(const SplitArgs &p) {
        // where it stands and not again: with a load that the compiler may repeat, two tiles of 72 rows take
        // longer (64 sequences x 130 rows 138 us, 131 so)
        asm volatile("ld.global.b32 %0, [%1];\n" : "=r"(len) : "l"(p.lens + n));
        enter(p);
    }
    __device__ __forceinline__ void enter(const SplitArgs &p) {
        tiles = tiles_of(p, len);
        j0 = max(0, unit - extra);
        j1 = (int32_t)min((int64_t)tiles, unit - extra + left);
        work = len > 0 && !bad_len(p, len);
        if (j1 <= j0) left = 0;  // the run ends in front of the sequence's first tile
    }
    __device__ __forceinline__ void start(const SplitArgs &p, const Run &run) {
        n = run.first_seq;
        unit = run.first_unit;
        extra = run.extra;
        left = run.end - run.begin;
        len = run.first_len;
        if (left > 0) enter(p);
    }
    __device__ __forceinline__ bool done() const { return left <= 0; }
    __device__ __forceinline__ void next(const SplitArgs &p) {
        left -= j1 + extra - unit;
        ++n;
        unit = 0;
        if (left > 0) open(p);
    }
    __device__ __forceinline__ void skip_idle(const SplitArgs &p) {
        while (!done() && !work) next(p);
    }
};

// barrier of the softmax warps (N threads) that also tells whether any thread's flag is set
template <int N>
__device__ __forceinline__ bool softmax_any(bool flag) {
    uint32_t r;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbarrier.cta.red.or.pred q, 1, %2, p;\nselp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)flag), "n"(N)
                 : "memory");
    return r != 0;
}

// kept = factor kept + O^T of this thread's latent, by query row; for the output (back) into O^T instead
__device__ __forceinline__ void fold_o(float *kept, uint32_t o_addr, int npad, const float *factor, bool start, bool back) {
    tc::fence_after_sync();
    for (int e = 0; e < npad; e += 16) {
        uint32_t x[16];
        tma::tmem_ld16_nowait(o_addr + e, x);
        tc::tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < 16; ++y) {
            float *at = kept + (int64_t)(e + y) * kLatent;
            const float v = __uint_as_float(x[y]) + (start ? 0.f : *at * factor[e + y]);
            x[y] = __float_as_uint(v);
            if (!back) *at = v;
        }
        if (back) tc::tmem_st16(o_addr + e, x);
    }
    if (back) tc::tmem_wait_st();
}

// The join of the sequences that a run's border cuts. With fewer sequences than groups block x
// belongs to sequence x, whose place in the list it adds up itself; with more it belongs to
// the border before group x + 1, where the main kernel left the place, and the first border
// inside a sequence joins it. W warps share a row's parts, each lane 16 / Z of the 512 latents, Z
// blocks a row; the parts are added in list order within a
// warp and the warps' sums in warp order, so the result does not depend on timing. With W = 1 no
// shared memory is needed, but 32 KB asked for keep these blocks off the SMs until the main kernel's
// are through: without them they wait beside it, and 256 x 96 takes 2% longer.
// (256 threads: 64 x 96 x 4 in 8 bits 226.9 us, with 512 228.4.)
constexpr int join_threads(int W) { return W == 1 ? 256 : 512; }
template <int W, int Z>
__global__ void __launch_bounds__(join_threads(W)) kda_mla_join_kernel(const __grid_constant__ SplitArgs p) {
    constexpr int kRows = join_threads(W) / 32 / W;  // rows of a block
    constexpr int kLat = kLatent / Z, kVec = kLat / 128;  // its latents, and float4 of a lane
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t n, tiles, b;  // the sequence, its tiles, the run after the one that holds its first tile
    int64_t first;        // list index of that tile's unit
    int count;            // parts
    if (p.N < p.G) {
        // The lengths are read before the wait: whatever wrote them had finished before the main kernel
        // let this one start, which it does behind its own wait. From L2, where that writing is.
        n = blockIdx.x;
        int64_t total = 0, before = 0;
        for (int i = lane; i < p.N; i += 32) {
            const int32_t t = tiles_of(p, __ldcg(p.lens + i));
            total += t;
            if (i < n) before += t;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            total += __shfl_xor_sync(0xffffffffu, total, off);
            before += __shfl_xor_sync(0xffffffffu, before, off);
        }
        const int32_t extra = extra_of(p, total);
        const Runs runs(total + (int64_t)p.N * extra, p.G);
        first = before + (int64_t)(n + 1) * extra;
        tiles = tiles_of(p, __ldcg(p.lens + n));
        b = runs.of(first) + 1;
        count = runs.of(first + tiles - 1) - b + 2;
        pdl_wait();  // in every block: a join that ended early would let the next kernel start before the main one's end
        if (count == 1) return;
    } else {
        b = blockIdx.x + 1;
        pdl_wait();
        const int64_t total = p.head[0];
        const Runs runs(total, p.G);
        const int64_t at = runs.begin(b);
        if (at >= total) return;
        const int32_t *e = reinterpret_cast<const int32_t *>(p.head + 1) + 4 * b;
        n = e[0];
        tiles = e[2];
        first = at - e[1];
        if (e[1] == 0 || runs.of(first) != b - 1) return;
        count = runs.of(first + tiles - 1) - b + 2;
    }
    const int rl = warp / W, part = warp % W, rr = blockIdx.y * kRows + rl;
    const bool live = rr < p.split.R;
    const int rt = (live ? rr : 0) / p.split.rows, r = (live ? rr : 0) % p.split.rows;
    const float c = p.scale * 1.4426950408889634f;
    // parts: run b - 1 (slot 1, it holds the sequence's start), then the following runs (slot 0)
    const int lat0 = blockIdx.z * kLat;
    float m = -INFINITY, l = 0.f, o[4 * kVec];
#pragma unroll
    for (int i = 0; i < 4 * kVec; ++i) o[i] = 0.f;
    auto row_of = [&](int i) {
        const int64_t gq = b - 1 + i;
        return ((2 * gq + (i == 0 ? 1 : 0)) * p.split.RT + rt) * p.split.npad + r;
    };
    if (live) {
        // The common maximum of this warp's parts, then one weighted sum; the first kBatch parts are on their way meanwhile. (With
        // 1, 2 and 4 for W = 1: 256 x 96 in 8 bits 260, 266 and 271 us, 64 x 48 59, 61.6 and 66; with 2 and 4 otherwise 32 x 16
        // 26.9 and 29.6.)
        constexpr int kBatch = W == 1 ? 1 : 2;
        float4 x[kBatch][kVec];
        auto load = [&](int i0) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + W * k;
                const float4 *src = reinterpret_cast<const float4 *>(p.part_o + row_of(i) * kLatent + lat0) + lane;
#pragma unroll
                for (int v = 0; v < kVec; ++v) x[k][v] = i < count ? __ldcs(src + 32 * v) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        };
        load(part);
        float2 mine = make_float2(-INFINITY, 0.f);  // of the lane's part of the first 32
        if (part + W * lane < count) mine = p.part_ml[row_of(part + W * lane)];
        m = mine.x;
        for (int i = part + W * (lane + 32); i < count; i += W * 32) m = fmaxf(m, p.part_ml[row_of(i)].x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        const float ms = m == -INFINITY ? 0.f : m;
        for (int i0 = part, at = 0; i0 < count; i0 += W * kBatch, at += kBatch) {
            if (at > 0) load(i0);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                float2 ml = make_float2(__shfl_sync(0xffffffffu, mine.x, (at + k) & 31), __shfl_sync(0xffffffffu, mine.y, (at + k) & 31));
                if (i0 + W * k >= count) continue;
                if (at + k >= 32) ml = p.part_ml[row_of(i0 + W * k)];
                const float f = tc::ex2((ml.x - ms) * c);
                l += f * ml.y;
#pragma unroll
                for (int v = 0; v < kVec; ++v) {
                    o[4 * v] += f * x[k][v].x;
                    o[4 * v + 1] += f * x[k][v].y;
                    o[4 * v + 2] += f * x[k][v].z;
                    o[4 * v + 3] += f * x[k][v].w;
                }
            }
        }
    }
    const int64_t row = (int64_t)n * p.split.R + rr;
    if constexpr (W == 1) {
        if (!live) return;
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        if (lane == 0 && blockIdx.z == 0 && p.lse) p.lse[row] = l == 0.f ? -INFINITY : m * p.scale + logf(l);
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(o[4 * v] * inv, o[4 * v + 1] * inv),
                                 bb = __floats2bfloat162_rn(o[4 * v + 2] * inv, o[4 * v + 3] * inv);
            *reinterpret_cast<uint2 *>(p.o + row * kLatent + lat0 + 4 * (32 * v + lane)) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&bb));
        }
    } else {
        __shared__ float s_o[kRows][W][kLat];
        __shared__ float s_m[kRows][W], s_l[kRows][W];
#pragma unroll
        for (int v = 0; v < kVec; ++v)
            *reinterpret_cast<float4 *>(&s_o[rl][part][4 * (32 * v + lane)]) = make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
        if (lane == 0) s_m[rl][part] = m, s_l[rl][part] = l;
        __syncthreads();
        if (!live) return;
        float M = -INFINITY, L = 0.f;
        for (int i = 0; i < W; ++i) M = fmaxf(M, s_m[rl][i]);
        const float Ms = M == -INFINITY ? 0.f : M;
        float f[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            f[i] = tc::ex2((s_m[rl][i] - Ms) * c);
            L += f[i] * s_l[rl][i];
        }
        const float inv = L == 0.f ? 0.f : 1.0f / L;
        if (part == 0 && lane == 0 && blockIdx.z == 0 && p.lse) p.lse[row] = L == 0.f ? -INFINITY : M * p.scale + logf(L);
        for (int x = 2 * (part * 32 + lane); x < kLat; x += 2 * 32 * W) {
            float a = 0.f, bb = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                a += f[i] * s_o[rl][i][x];
                bb += f[i] * s_o[rl][i][x + 1];
            }
            *reinterpret_cast<__nv_bfloat162 *>(p.o + row * kLatent + lat0 + x) = __floats2bfloat162_rn(a * inv, bb * inv);
        }
    }
}

// groups of CTAs that share the list: one CTA an SM
int32_t groups_of(int32_t RT, int32_t sms) { return sms / RT > 0 ? sms / RT : 1; }

struct SplitWs {
    size_t head, ml, o, total;
};
// widest: the most query rows of a CTA
SplitWs split_ws(const SplitGeom &q, int widest_rows) {
    SplitWs w;
    size_t parts = 2 * (size_t)groups_of(q.RT, kMaxGroups) * q.RT * q.npad;
    const size_t widest = 2 * (size_t)kMaxGroups * widest_rows;
    if (q.RT > 1 && parts < widest) parts = widest;  // more rows never need less
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    w.head = 0;
    w.ml = up(8 + 16 * kMaxGroups);
    w.o = w.ml + up(parts * sizeof(float2));
    w.total = w.o + parts * kLatent * sizeof(float);
    return w;
}

template <int W, int Z>
cudaError_t launch_join(const SplitArgs &a, cudaStream_t st) {
    const int rows = join_threads(W) / 32 / W;
    const int cuts = a.N < a.G ? a.N : a.G - 1;
    return launch_after(kda_mla_join_kernel<W, Z>, dim3(cuts, (a.split.R + rows - 1) / rows, Z), dim3(join_threads(W)),
                        W == 1 ? 32768 : 0, st, a);
}

// the join behind the main kernel
cudaError_t join_parts(const SplitArgs &a, cudaStream_t st) {
    if (a.G <= 1) return cudaSuccess;
    // As many warps a row, and blocks a row, as leave about 256 blocks of 16 warps: with fewer a warp goes through its parts
    // too long, with more the blocks come in waves. In 8 bits, with 1 x 1, 2 x 2, 4 x 2, 8 x 2, 16 x 2 and 16 x 4 warps x
    // blocks a row: 12 rows of 152 parts (100000 cached rows) -, 49.9, 37.4, 28.9, 25.4 and 24.1 us; 96 of 152 -, 75.2, 54.8,
    // 47.0, 43.6 and 46.7; 192 of 12 (2 x 12 x 8) 14.6, 11.6, 11.4, 11.4, 13.6 and 18.0; 768 of 19 33.7, 25.9, 26.2, 28.1,
    // 36.3 and 52.3; 1024 of 9 31.3, 25.9, 28.4, 32.6, 44.4 and 65.9; 2048 of 6 35.6, 37.0, 40.8, 51.3, 74.6 and 115.6.
    const int64_t rows = (int64_t)(a.N < a.G ? a.N : a.G - 1) * a.split.R;
    if (rows <= 64) return launch_join<16, 4>(a, st);
    if (rows <= 128) return launch_join<16, 2>(a, st);
    if (rows <= 256) return launch_join<8, 2>(a, st);
    if (rows <= 512) return launch_join<4, 2>(a, st);
    if (rows <= 1024) return launch_join<2, 2>(a, st);
    return launch_join<1, 1>(a, st);
}

}  // namespace
}  // namespace kda
