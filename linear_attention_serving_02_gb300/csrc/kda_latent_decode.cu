// Latent attention in the absorbed form over the paged rows: kda_mla_decode.
//
//   s_rj = scale (q_r . row_j),  o_r = sum_j e^{s_rj - M_r} c_j / sum_j e^{s_rj - M_r}
//
// A query row r is one (window token, head); all m H rows of a sequence read the same cached
// rows, and c_j is the first 512 of row_j's 576 values: one read of 1152 B serves the score
// and the value product of every head. 2176 flop a (row, cached row).
//
// Work. The sequences' cached rows are cut into tiles of 64; all tiles of the batch form one
// list, and each of G groups of CTAs takes an equal run of it, so long and short sequences
// load every SM alike whatever their lengths. The CTAs of a group take up to 96 query rows
// each (row tiles) and walk the same tiles, each loading them for itself: the first read brings a
// tile from HBM, its neighbours' come from L2. A sequence that a run cuts leaves partial (O, max,
// sum), joined by a second kernel in list order; the others are finished in place. No CTA waits
// for another.
//
// A tile in a CTA. TMA lays the 64 rows down once as 9 chunks of 64 columns (128-byte
// swizzle). S = Q K^T: M = 64 or 128 query rows, N = 64 cached rows, read K-major. Eight softmax
// warps take S from TMEM, one thread a query row and half of the tile, and write P (bf16) to
// shared memory. The value product runs transposed, O^T = C^T P^T: M = 128 latents (the same
// chunks, read MN-major), N = query rows. TMEM: O^T takes 4 N columns (O itself, rows x 512,
// would take every column), S 64 a tile, two of them with M = 64; past 64 rows of a sequence the
// rest holds Q's first latents. An MMA of K = 16 takes N / 2 cycles, but at
// least 25 with M = 64 and 39 with M = 128, or its operands' bytes in shared memory at 128 a
// cycle: 96 rows need about 28 x 48 + 8 x 32 + 16 x 56 = 2500 cycles a tile and 16 rows 1780, where
// the tile's 72 KB take an SM's share of HBM about 3100.
//
// Measured: 1M cached rows x 12 heads 192 us with the join (6.3 TB/s), bound by the rows' bytes;
// 256 sequences of up to 8000 rows x 96 heads 297 us (4.3 TB/s). There a tile takes 4000
// cycles, of which shared memory is busy about 3000: the operands' 2500 and 576 for the rows'
// arrival. In the rest load, last scores, softmax (1200) and value product of a tile follow one
// another, as the ring holds a little less than two tiles; and the join of the parts that the 151
// borders leave (59 MB written and read) takes 20 us when it runs alone. Tiles of 48 rows, of which
// the ring holds two and a quarter, take the same time in all; two CTAs with 48 query rows each 346;
// two CTAs that split the columns and trade partial scores 427.
//
// P is rounded to bf16 for the value product, which takes 16-bit operands (two of them a weight would
// double it); the sum of the weights is that of the fp32 values.
//
// The reference M_r only has to stay within 2^8 of the row's maximum (P is then far inside
// bf16 and fp32), so a tile costs a comparison a score and one barrier; the halves' maxima are
// exchanged, and O^T rescaled, on a sequence's first tile and where a score passes its
// reference by 2^8.
//
// The tensor core drops what falls below an accumulator's last bit, always towards zero: a sum over n rows
// comes out low by about n / 16 * 0.7 * 2^-23 of itself, 0.5% at a million. O^T therefore sums 1024 tiles
// of a stretch at a time (4096 additions, 2^-11 at most); then it is added, with roundings to nearest, to
// fp32 rows in the stretch's place among the partials, which a stretch of fewer tiles does not touch, and
// the denominator, whose roundings go one way too where tiles are alike, to one in a register.
//
// Shared memory. Q takes 1152 B a row less what TMEM holds; the rest is a ring of 16 KB pairs of
// chunks and a ring of 8 KB positional chunks, two tiles or more, with M = 128 a little less: there
// the coming tile is asked into L2. One thread issues the score products chunk by chunk as they
// land, another the value products as their P is written; each pair of chunks is given back as
// soon as its 128 latents are done.
//
// Rows of a tile behind the sequence's length (the rest of a page, or stale shared memory)
// may hold anything: their scores are replaced by -inf, the product's 16-row steps past the
// length are left out, and value rows inside the last step are zeroed in shared memory.

#include "kda_common.cuh"
#include "kda_latent_common.cuh"
#include "kda_tma.cuh"

namespace kda {
namespace {

constexpr int kKvTile = 64;                     // cached rows of a tile
constexpr int kRowTile = 64, kWideRows = 96;    // query rows of a CTA at most: M = 64, and M = 128 (TMEM holds 96)
constexpr uint32_t kChunkB = kKvTile * 128;     // bytes of a chunk: 8 KB
constexpr uint32_t kPairB = 2 * kChunkB;
constexpr int kPairs = kLatent / 128;         // chunk pairs of a tile's latent: 4
constexpr int kMaxPair = 12, kMaxPos = 4;     // ring slots at most
constexpr int kDecThreads = 352;              // 8 softmax warps, S issue, value issue, TMA
constexpr int kMaxGroups = 160;               // CTAs that share the list at most
constexpr float kGrow = 8.0f;
constexpr int kSoftmaxThreads = 256;
constexpr int kFold = 1024;                   // tiles of a stretch that O^T sums in tensor memory (a power of two)
constexpr int kHalf = kKvTile / 2;            // cached rows of a tile that a softmax thread takes

struct DecodeGeom {
    int32_t R;        // query rows of a sequence: m H
    int32_t RT, rows; // row tiles and query rows of each (a multiple of 8)
    int32_t npad;     // MMA columns of O^T: rows rounded up to 16
    int32_t qt;       // pairs of Q's latent chunks (128 latents) kept in TMEM; the others in shared memory
    int32_t np, nr;   // ring slots
    uint32_t smem;    // dynamic shared memory
};

struct DecodeArgs {
    CUtensorMap q_lat, q_pe, cache;
    const __nv_bfloat16 *q;  // q_lat again
    const __nv_bfloat16 *rows;  // the cache again, for the prefetch of a coming tile into L2
    int64_t page_stride;
    const int32_t *table, *lens;
    int32_t max_pages, num_pages, page_size, rb;  // rb: rows of a TMA box (64, 32 or 16)
    int32_t N, H, m, G;
    DecodeGeom geo;
    float scale;
    __nv_bfloat16 *o;
    float *lse;
    float *part_o;   // [2 G, RT, npad, 512]
    float2 *part_ml; // [2 G, RT, npad] reference maximum (raw scores), sum
    int64_t *head;   // [0]: tiles of the batch; then per group {sequence, first tile, tiles of the sequence}
    int32_t *status;
};

struct DecodeSmem {
    uint64_t q_full, q_empty, q_ready, s_full[2], s_free[2], p_full, pv_done, drained;
    uint64_t pair_full[kMaxPair], pair_empty[kMaxPair], pos_full[kMaxPos], pos_empty[kMaxPos];
    float factor[128], half[2][128];  // by query row: scale of O^T, the halves' maxima or sums
    uint32_t tmem;
    int32_t failed, bad[4];
    int32_t first_seq, first_tile;
    int64_t begin, end;
    int32_t pair_issued, pos_issued, q_issued;
};

__device__ __forceinline__ bool bad_len(const DecodeArgs &p, int64_t len) {
    return len < 0 || len > (int64_t)p.max_pages * p.page_size;
}
// tiles of a sequence in the list: one at least, so that every sequence's output is written
__device__ __forceinline__ int32_t tiles_of(const DecodeArgs &p, int32_t len) {
    return bad_len(p, len) || len == 0 ? 1 : (int32_t)(((int64_t)len + kKvTile - 1) / kKvTile);
}

// The list's cut into G runs: the first `extra` of them one tile longer than the others.
struct Runs {
    int64_t each;
    int32_t extra;
    __device__ __forceinline__ Runs(int64_t total, int32_t G) : each(total / G), extra((int32_t)(total - each * G)) {}
    __device__ __forceinline__ int64_t begin(int32_t g) const { return g * each + min(g, extra); }
    // the run that holds tile x
    __device__ __forceinline__ int32_t of(int64_t x) const {
        const int64_t longer = extra * (each + 1);
        return (int32_t)(x < longer ? x / (each + 1) : extra + (x - longer) / each);
    }
};

// A walk over a run of the list, one stretch of tiles of one sequence after the other.
struct Walk {
    int32_t n, j0, j1, tiles, len;
    int64_t left;
    bool work;  // the sequence has cached rows and a sound length
    __device__ __forceinline__ void open(const DecodeArgs &p) {
        // where it stands and not again: with a load that the compiler may repeat, two tiles of 72 rows take
        // longer (64 sequences x 130 rows 138 us, 131 so)
        asm volatile("ld.global.b32 %0, [%1];\n" : "=r"(len) : "l"(p.lens + n));
        tiles = tiles_of(p, len);
        j1 = (int32_t)min((int64_t)tiles, j0 + left);
        work = len > 0 && !bad_len(p, len);
    }
    __device__ __forceinline__ void start(const DecodeArgs &p, const DecodeSmem &sm) {
        n = sm.first_seq;
        j0 = sm.first_tile;
        left = sm.end - sm.begin;
        if (left > 0) open(p);
    }
    __device__ __forceinline__ bool done() const { return left <= 0; }
    __device__ __forceinline__ void next(const DecodeArgs &p) {
        left -= j1 - j0;
        ++n;
        j0 = 0;
        if (left > 0) open(p);
    }
    __device__ __forceinline__ void skip_idle(const DecodeArgs &p) {
        while (!done() && !work) next(p);
    }
};

// barrier of the softmax warps that also tells whether any thread's flag is set
__device__ __forceinline__ bool softmax_any(bool flag) {
    uint32_t r;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbarrier.cta.red.or.pred q, 1, 256, p;\nselp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)flag)
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

// MS: rows of the score product's M. QT: the first QT pairs of Q's latent chunks are kept in TMEM.
// (Constants, so that the issue loop has no choice to make.)
template <int MS, int QT>
__global__ void __launch_bounds__(kDecThreads, 1) kda_mla_decode_kernel(const __grid_constant__ DecodeArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    constexpr int kS = MS == 128 ? 1 : 2;      // S tiles in TMEM
    const DecodeGeom &geo = p.geo;
    const uint32_t q_chunk = (uint32_t)geo.rows * 128;
    constexpr int q_chunks = 9 - 2 * QT;      // of Q in shared memory, the positions last
    uint8_t *s_q = base;                      // chunks of `rows` rows; M = 64 reads run on into what
    uint8_t *s_p = s_q + q_chunks * q_chunk;  // follows (P and the rings are longer), rows of S that nobody reads
    uint8_t *s_pair = s_p + (uint32_t)geo.npad * 128;  // P: npad rows of 64 cached rows
    uint8_t *s_pos = s_pair + (uint32_t)geo.np * kPairB;
    DecodeSmem &sm = *reinterpret_cast<DecodeSmem *>(s_pos + (uint32_t)geo.nr * kChunkB);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rt = blockIdx.x % geo.RT, g = blockIdx.x / geo.RT;

    pdl_wait();
    // ---- this group's run of the list ----
    if (warp == 10 && lane == 0) {
        tma::prefetch_map(&p.q_lat);
        tma::prefetch_map(&p.q_pe);
        tma::prefetch_map(&p.cache);
    }
    if (warp == 0) {
        int64_t total = 0;
        for (int n = lane; n < p.N; n += 32) total += tiles_of(p, p.lens[n]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
        const Runs runs(total, p.G);
        const int64_t begin = runs.begin(g), end = runs.begin(g + 1);
        int64_t before = 0;
        int seq = p.N - 1;
        int64_t first = 0;
        int32_t of = 0;
        for (int n0 = 0; n0 < p.N; n0 += 32) {
            const int n = n0 + lane;
            const int32_t t = n < p.N ? tiles_of(p, p.lens[n]) : 0;
            int64_t incl = t;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += x;
            }
            const int64_t lo = before + incl - t;
            const unsigned mine = __ballot_sync(0xffffffffu, begin >= lo && begin < lo + t);
            if (mine) {
                const int src = __ffs(mine) - 1;
                seq = n0 + src;
                first = begin - __shfl_sync(0xffffffffu, lo, src);
                of = __shfl_sync(0xffffffffu, t, src);
                break;
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            sm.first_seq = seq;
            sm.first_tile = (int32_t)first;
            sm.begin = begin;
            sm.end = end;
            sm.failed = 0;
            sm.pair_issued = sm.pos_issued = sm.q_issued = 0;
            for (int i = 0; i < 4; ++i) sm.bad[i] = 0;
            if (rt == 0) {
                if (g == 0) p.head[0] = total;
                int32_t *e = reinterpret_cast<int32_t *>(p.head + 1) + 4 * g;
                e[0] = seq;
                e[1] = (int32_t)first;
                e[2] = of;
            }
            tc::mbar_init(&sm.q_full, 1);
            tc::mbar_init(&sm.q_empty, 1);
            tc::mbar_init(&sm.q_ready, kSoftmaxThreads / 32);
            tc::mbar_init(&sm.s_full[0], 1);
            tc::mbar_init(&sm.s_full[1], 1);
            tc::mbar_init(&sm.s_free[0], kSoftmaxThreads / 32);
            tc::mbar_init(&sm.s_free[1], kSoftmaxThreads / 32);
            tc::mbar_init(&sm.p_full, kSoftmaxThreads / 32);
            tc::mbar_init(&sm.pv_done, 1);
            tc::mbar_init(&sm.drained, 2);
            for (int i = 0; i < geo.np; ++i) tc::mbar_init(&sm.pair_full[i], 1), tc::mbar_init(&sm.pair_empty[i], 1);
            for (int i = 0; i < geo.nr; ++i) tc::mbar_init(&sm.pos_full[i], 1), tc::mbar_init(&sm.pos_empty[i], 1);
            tc::mbar_init_fence();
        }
    } else if (warp == 8) {
        tc::tmem_alloc(&sm.tmem, 512);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    pdl_trigger();
    const uint32_t tmem = sm.tmem;
    const uint32_t t_s = tmem + 4 * geo.npad;  // two S tiles of 64 columns behind O^T
    const uint32_t t_q = t_s + kS * kKvTile;    // then Q's first latents, two to a column
    const int row_first = rt * geo.rows, rows_here = max(0, min(geo.rows, geo.R - row_first));
    bool ok = true;

    if (warp == 10) {
        // ---- TMA producer: one thread ----
        if (tma::elect()) {
            Walk w;
            w.start(p, sm);
            w.skip_idle(p);
            int seg = 0, ps = 0, pph = 0, rs = 0, rph = 0;
            const int sub = kKvTile / p.rb;  // boxes of rows of a tile: 1, 2 or 4
            while (!w.done() && ok) {
                const int32_t *entry = p.table + (int64_t)w.n * p.max_pages;
                const int64_t row0 = (int64_t)w.j0 * kKvTile;
                entry += row0 / p.page_size;
                int32_t at = (int32_t)(row0 % p.page_size);  // row within the page
                // the places of a tile's boxes, fetched one tile ahead; nothing past the sequence's rows is looked up
                int32_t pg[4], ry[4], pg_next[4], ry_next[4];
                auto look = [&](int j) {
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        pg_next[b] = 0;
                        ry_next[b] = at;
                        if (b < sub && j < w.j1 && (int64_t)j * kKvTile + b * p.rb < w.len) {
                            pg_next[b] = *entry;
                            at += p.rb;
                            if (at == p.page_size) at = 0, ++entry;
                        }
                    }
                };
                look(w.j0);
                ok = seg == 0 || tc::mbar_wait(&sm.q_empty, (seg - 1) & 1);
                if (!ok) break;
                sm.bad[seg & 3] = 0;
                const int row = (int)((int64_t)w.n * geo.R + row_first);
                tc::mbar_arrive_expect_tx(&sm.q_full, q_chunks * q_chunk);
                tma::load_2d(s_q + (q_chunks - 1) * q_chunk, &p.q_pe, &sm.q_full, 0, row);
                for (int c = 2 * QT; c < 8; ++c)
                    tma::load_2d(s_q + (c - 2 * QT) * q_chunk, &p.q_lat, &sm.q_full, 64 * c, row);
                ++sm.q_issued;
                for (int j = w.j0; j < w.j1 && ok; ++j) {
                    bool bad = false;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        ry[b] = ry_next[b];
                        const bool out = (uint32_t)pg_next[b] >= (uint32_t)p.num_pages;
                        bad |= out;
                        pg[b] = out ? INT32_MAX : pg_next[b];  // past every page: loads as zeros
                    }
                    if (bad) {
                        sm.bad[seg & 3] = 1;
                        set_status(p.status, KDA_ERR_PAGES);
                    }
                    look(j + 1);
                    if (MS == 128 && j + 1 < w.j1) {
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const int64_t row = ((int64_t)j + 1) * kKvTile + b * p.rb;
                            if (b < sub && row < w.len && (uint32_t)pg_next[b] < (uint32_t)p.num_pages)
                                tma::prefetch_l2(p.rows + pg_next[b] * p.page_stride + (int64_t)ry_next[b] * kRow,
                                                 (uint32_t)p.rb * kRow * 2);
                        }
                    }
                    const int valid = min(kKvTile, w.len - j * kKvTile), boxes = (valid + p.rb - 1) / p.rb;
                    const uint32_t box = (uint32_t)p.rb * 128, bytes = boxes * box;
                    ok = tc::mbar_wait(&sm.pos_empty[rs], rph ^ 1);
                    if (!ok) break;
                    tc::mbar_arrive_expect_tx(&sm.pos_full[rs], bytes);
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        if (b < boxes)
                            tma::load_3d(s_pos + rs * kChunkB + b * box, &p.cache, &sm.pos_full[rs], kLatent, ry[b], pg[b]);
                    ++sm.pos_issued;
                    if (++rs == geo.nr) rs = 0, rph ^= 1;
                    for (int i = 0; i < kPairs; ++i) {
                        ok = tc::mbar_wait(&sm.pair_empty[ps], pph ^ 1);
                        if (!ok) break;
                        tc::mbar_arrive_expect_tx(&sm.pair_full[ps], 2 * bytes);
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (b < boxes) {
                                uint8_t *dst = s_pair + ps * kPairB + b * box;
                                tma::load_3d(dst, &p.cache, &sm.pair_full[ps], 128 * i, ry[b], pg[b]);
                                tma::load_3d(dst + kChunkB, &p.cache, &sm.pair_full[ps], 128 * i + 64, ry[b], pg[b]);
                            }
                        ++sm.pair_issued;
                        if (++ps == geo.np) ps = 0, pph ^= 1;
                    }
                }
                ++seg;
                w.next(p);
                w.skip_idle(p);
            }
            if (!ok) sm.failed = 1;
        }
        __syncwarp();
    } else if (warp == 8) {
        // ---- score products: one thread; the value products have a thread of their own, so that
        // neither polls for the other (a narrow batch's MMA takes less than a look at a barrier) ----
        if (tma::elect()) {
            const uint32_t id = tma::idesc(MS, kKvTile, 0, 0);
            const uint32_t q_lo = tma::lo_k(tc::smem_addr(s_q)), pos_lo = tma::lo_k(tc::smem_addr(s_pos));
            const uint32_t pair_lo = tma::lo_k(tc::smem_addr(s_pair)), q_step = q_chunk >> 4;
            Walk w;
            w.start(p, sm);
            w.skip_idle(p);
            int k = 0, seg = 0, ps = 0, pph = 0, rs = 0, rph = 0;
            while (!w.done() && ok) {
                ok = tc::mbar_wait(&sm.q_full, seg & 1) && (QT == 0 || tc::mbar_wait(&sm.q_ready, seg & 1));
                for (int j = w.j0; j < w.j1 && ok; ++j, ++k) {
                    ok = tc::mbar_wait(&sm.s_free[k % kS], ((k / kS) & 1) ^ 1) && tc::mbar_wait(&sm.pos_full[rs], rph);
                    if (!ok) break;
                    tc::fence_after_sync();
                    const uint32_t d = t_s + (k % kS) * kKvTile;
                    {
                        const uint32_t a = q_lo + (q_chunks - 1) * q_step, b = pos_lo + rs * (kChunkB >> 4);
#pragma unroll
                        for (int s = 0; s < 4; ++s) tma::mma_ss(d, a + 2 * s, b + 2 * s, id, s != 0);
                        tc::commit(&sm.pos_empty[rs]);
                        if (++rs == geo.nr) rs = 0, rph ^= 1;
                    }
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) {
                        ok = ok && tc::mbar_wait(&sm.pair_full[ps], pph);
                        if (ok && i < QT) {
                            const uint32_t a = t_q + 64 * i, b = pair_lo + ps * (kPairB >> 4);
#pragma unroll
                            for (int s = 0; s < 4; ++s) tma::mma_ts(d, a + 8 * s, b + 2 * s, id, 1);
#pragma unroll
                            for (int s = 0; s < 4; ++s) tma::mma_ts(d, a + 32 + 8 * s, b + (kChunkB >> 4) + 2 * s, id, 1);
                        } else if (ok) {
                            const uint32_t a = q_lo + 2 * (i - QT) * q_step, b = pair_lo + ps * (kPairB >> 4);
#pragma unroll
                            for (int s = 0; s < 4; ++s) tma::mma_ss(d, a + 2 * s, b + 2 * s, id, 1);
#pragma unroll
                            for (int s = 0; s < 4; ++s) tma::mma_ss(d, a + q_step + 2 * s, b + (kChunkB >> 4) + 2 * s, id, 1);
                        }
                        if (++ps == geo.np) ps = 0, pph ^= 1;
                    }
                    if (!ok) break;
                    tc::commit(&sm.s_full[k % kS]);
                    if (j + 1 == w.j1) tc::commit(&sm.q_empty);
                }
                ++seg;
                w.next(p);
                w.skip_idle(p);
            }
            if (!ok) sm.failed = 1;
        }
        __syncwarp();
    } else if (warp == 9) {
        // ---- value products: one thread ----
        if (tma::elect()) {
            const uint32_t id = tma::idesc(128, geo.npad, 1, 0);
            const uint32_t pair_lo = tma::lo_mn(tc::smem_addr(s_pair), kChunkB), p_lo = tma::lo_k(tc::smem_addr(s_p));
            Walk w;
            w.start(p, sm);
            w.skip_idle(p);
            int k = 0, ps = 0;
            while (!w.done() && ok) {
                for (int j = w.j0; j < w.j1; ++j, ++k) {
                    ok = tc::mbar_wait(&sm.p_full, k & 1);
                    if (!ok) break;
                    tc::fence_after_sync();
                    const int steps = (min(kKvTile, w.len - j * kKvTile) + 15) / 16;
                    const uint32_t more = ((j - w.j0) & (kFold - 1)) != 0;
                    uint32_t d = tmem;
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) {
                        const uint32_t a = pair_lo + ps * (kPairB >> 4);
                        if (steps == 4) {
#pragma unroll
                            for (int s = 0; s < 4; ++s) tma::mma_ss(d, a + 128 * s, p_lo + 2 * s, id, s != 0 ? 1 : more);
                        } else {
                            for (int s = 0; s < steps; ++s) tma::mma_ss(d, a + 128 * s, p_lo + 2 * s, id, s != 0 ? 1 : more);
                        }
                        tc::commit(&sm.pair_empty[ps]);
                        d += geo.npad;
                        if (++ps == geo.np) ps = 0;
                    }
                    tc::commit(&sm.pv_done);
                }
                w.next(p);
                w.skip_idle(p);
            }
            if (!ok) sm.failed = 1;
        }
        __syncwarp();
    } else {
        // ---- softmax: one thread a query row and half a tile; then the output ----
        const int quarter = warp & 3, set = warp >> 2;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        // M = 64 puts rows 16 q .. 16 q + 15 into lanes 32 q .. 32 q + 15 of TMEM, M = 128 row r into lane r
        constexpr int kWarpRows = MS / 4;
        const bool low = lane < kWarpRows;
        const int r = quarter * kWarpRows + (lane & (kWarpRows - 1));
        const bool owner = low && r < rows_here, warp_rows = quarter * kWarpRows < rows_here;
        const int unseen = p.m - 1 - (row_first + (owner ? r : 0)) / p.H;  // last cached rows that the row does not see
        const float c = p.scale * 1.4426950408889634f;
        const uint64_t c2 = pk2(c, c);
        uint8_t *p_row = s_p + r * 128;
        int k = 0, seg = 0, ps = 0;  // tiles and stretches worked on, ring slot
        // Q's first latents into TMEM, in the lanes of S's rows: this thread's row, half of each pair. The
        // last stretch's score products are through: its last tile was taken
        auto load_q = [&](const Walk &s) {
            const uint4 *src = reinterpret_cast<const uint4 *>(
                p.q + ((int64_t)s.n * geo.R + min(row_first + r, geo.R - 1)) * kLatent + 64 * set);
            uint32_t x[2 * QT + 1][16];
#pragma unroll
            for (int i = 0; i < 2 * QT; ++i)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint4 v = src[16 * (i >> 1) + 4 * (i & 1) + u];
                    x[i][4 * u] = v.x, x[i][4 * u + 1] = v.y, x[i][4 * u + 2] = v.z, x[i][4 * u + 3] = v.w;
                }
#pragma unroll
            for (int i = 0; i < 2 * QT; ++i) tc::tmem_st16(t_q + lanes + 64 * (i >> 1) + 32 * set + 16 * (i & 1), x[i]);
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tma::arrive_warp(&sm.q_ready);
        };
        Walk w;
        w.start(p, sm);
        if constexpr (QT > 0) {
            Walk first = w;
            first.skip_idle(p);
            if (!first.done()) load_q(first);
        }
        for (; !w.done() && ok; w.next(p)) {
            float m_ref = -INFINITY, l = 0.f;
            // the stretch's place among the partials: a run's first stretch, where it continues a sequence, has
            // the first, the last one, which the run's end cuts, the second; before that any other may use it
            const int64_t part0 = (((int64_t)2 * g + (w.j0 == 0 ? 1 : 0)) * geo.RT + rt) * geo.npad;
            float m_kept = -INFINITY, l_kept = 0.f;  // reference and denominator of the tiles before the last kFold
            if (w.work) {
                bool stopped = false;
                for (int js = w.j0; !stopped; js += kFold) {
                    if (js > w.j0 && w.j1 - w.j0 > kFold) {
                        // kFold tiles, or the last ones, are in O^T (also with a failed wait: all warps meet these barriers)
                        ok = tma::wait_warp(&sm.pv_done, (k - 1) & 1) && ok;
                        const bool start = js == w.j0 + kFold;
                        named_sync(2, kSoftmaxThreads);  // the factors have been read
                        if (set == 0 && low) sm.factor[r] = start || m_kept == m_ref ? 1.0f : tc::ex2((m_kept - m_ref) * c);
                        named_sync(2, kSoftmaxThreads);
                        for (int i = 2 * set; i < 2 * set + 2; ++i) {
                            float *kept = p.part_o + part0 * kLatent + 128 * i + 32 * quarter + lane;
                            fold_o(kept, tmem + lanes + i * geo.npad, geo.npad, sm.factor, start, js >= w.j1);
                        }
                        m_kept = m_ref;
                        if (low) l_kept = l_kept * sm.factor[r] + l;
                        l = js >= w.j1 ? l_kept : 0.f;
                    }
                    if (js >= w.j1) break;
                    const int je = min(w.j1, js + kFold);
                    for (int j = js; j < je; ++j) {
                        ok = tma::wait_warp(&sm.s_full[k % kS], (k / kS) & 1) && ok;
                        // a failed wait still meets the barriers below, so that no warp is left in them
                        if (ok) tc::fence_after_sync();
                        uint32_t s[kHalf];
                        const bool first = j == w.j0;
                        float mb = m_ref == -INFINITY ? 0.f : -m_ref * c, top = -INFINITY;
                        if (warp_rows && ok) {
                            tc::tmem_ld32_nowait(t_s + lanes + (k % kS) * kKvTile + set * kHalf, s);
                            tc::tmem_wait_ld();
                            tc::fence_before_sync();
                            // cached rows of this thread's half that the row sees
                            const int64_t seen = (int64_t)w.len - unseen - ((int64_t)j * kKvTile + set * kHalf);
                            if (__any_sync(0xffffffffu, seen < kHalf)) {
#pragma unroll
                                for (int e = 0; e < kHalf; ++e)
                                    if (e >= seen) s[e] = 0xff800000u;
                            }
#pragma unroll
                            for (int e = 0; e < kHalf; e += 2)
                                top = fmaxf(top, fmaxf(__uint_as_float(s[e]), __uint_as_float(s[e + 1])));
                        }
                        tma::arrive_warp(&sm.s_free[k % kS]);
                        // one barrier a tile: does a row need a new reference (also from -inf to a finite one), did a wait fail
                        const bool any = softmax_any((owner && (first || (top - m_ref) * c > kGrow)) || !ok);
                        if (k > 0) ok = tma::wait_warp(&sm.pv_done, (k - 1) & 1) && ok;
                        if (any) {
                            if (low) sm.half[set][r] = top;
                            // all stop together when any wait failed
                            if (softmax_any(!ok)) {
                                ok = false;
                                stopped = true;
                                break;
                            }
                            top = fmaxf(top, sm.half[set ^ 1][r]);
                            const bool grown = first || (top - m_ref) * c > kGrow;
                            const float m = grown ? top : m_ref, f = grown ? tc::ex2((m_ref - m) * c) : 1.0f;
                            if (!first) {
                                l *= f;
                                if (set == 0 && low) sm.factor[r] = f;
                                named_sync(2, kSoftmaxThreads);
                                tc::fence_after_sync();
                                for (int i = 2 * set; i < 2 * set + 2; ++i)
                                    for (int e = 0; e < geo.npad; e += 16) {
                                        const uint32_t at = tmem + lanes + i * geo.npad + e;
                                        uint32_t x[16];
                                        tma::tmem_ld16_nowait(at, x);
                                        tc::tmem_wait_ld();
#pragma unroll
                                        for (int y = 0; y < 16; ++y) x[y] = __float_as_uint(__uint_as_float(x[y]) * sm.factor[e + y]);
                                        tc::tmem_st16(at, x);
                                    }
                                tc::tmem_wait_st();
                            }
                            m_ref = m;
                            mb = m_ref == -INFINITY ? 0.f : -m_ref * c;
                        }
                        if (warp_rows && ok) {
                            const uint64_t mb2 = pk2(mb, mb);
                            uint64_t l2[2] = {0, 0};
#pragma unroll
                            for (int u = 0; u < kHalf / 8; ++u) {  // 16-byte units of the row, swizzled
                                uint32_t h[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t *x = &s[8 * u + 2 * e];
                                    const float2 y = upk2(fma2(pk2(__uint_as_float(x[0]), __uint_as_float(x[1])), c2, mb2));
                                    const float a = tc::ex2(y.x), b = tc::ex2(y.y);
                                    l2[e & 1] = add2(l2[e & 1], pk2(a, b));
                                    const __nv_bfloat162 hh = __floats2bfloat162_rn(a, b);
                                    h[e] = *reinterpret_cast<const uint32_t *>(&hh);
                                }
                                if (low && r < geo.npad)
                                    *reinterpret_cast<uint4 *>(p_row + (((4 * set + u) ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                            }
                            const float2 ls = upk2(add2(l2[0], l2[1]));
                            l += ls.x + ls.y;
                        }
                        const int valid = min(kKvTile, w.len - j * kKvTile);
                        if (valid & 15) {  // value rows behind the sequence in the product's last step of 16
                            const int units = (-valid & 15) * 8;
                            for (int u = tid; u < 2 * kPairs * units; u += kSoftmaxThreads) {
                                const int chunk = u / units;
                                const int slot = (ps + (chunk >> 1)) % geo.np;
                                reinterpret_cast<uint4 *>(s_pair + slot * kPairB + (chunk & 1) * kChunkB)[valid * 8 + u % units] =
                                    make_uint4(0, 0, 0, 0);
                            }
                        }
                        ps += kPairs;
                        if (ps >= geo.np) ps -= geo.np;
                        fence_proxy_async();
                        tc::fence_before_sync();
                        tma::arrive_warp(&sm.p_full);
                        ++k;
                    }
                }
                if constexpr (QT > 0) {
                    // the next stretch's queries before this one's output, so that its scores start meanwhile
                    Walk after = w;
                    after.next(p);
                    after.skip_idle(p);
                    if (ok && !after.done()) load_q(after);
                }
                if (ok) ok = tma::wait_warp(&sm.pv_done, (k - 1) & 1);
                tc::fence_after_sync();
            }
            if (low) sm.half[set][r] = l;
            if (softmax_any(!ok)) ok = false;
            l += sm.half[set ^ 1][r];
            // ---- this stretch's part of the sequence: finished, or left for the join ----
            const bool whole = w.j0 == 0 && w.j1 == w.tiles;
            const bool bad = !ok || bad_len(p, w.len) || (w.work && *(volatile int32_t *)&sm.bad[seg & 3] != 0);
            if (bad_len(p, w.len) && tid == 0) set_status(p.status, KDA_ERR_SEQLENS);
            const int64_t row0 = (int64_t)w.n * geo.R + row_first;
            if (set == 0 && low) {
                sm.factor[r] = bad ? NAN : (l == 0.f ? 0.f : 1.0f / l);
                if (owner) {
                    if (!whole)
                        p.part_ml[part0 + r] = make_float2(m_ref, bad ? NAN : l);
                    else if (p.lse)
                        p.lse[row0 + r] = bad ? NAN : (l == 0.f ? -INFINITY : m_ref * p.scale + logf(l));
                }
            }
            named_sync(2, kSoftmaxThreads);
            for (int i = 2 * set; i < 2 * set + 2; ++i) {
                const int lat = 128 * i + 32 * quarter + lane;
                for (int e = 0; 16 * e < rows_here; ++e) {
                    uint32_t x[16];
                    if (w.work && ok) {
                        tma::tmem_ld16_nowait(tmem + lanes + i * geo.npad + 16 * e, x);
                        tc::tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int y = 0; y < 16; ++y) x[y] = 0;
                    }
                    if (whole) {
                        // neighbouring lanes trade a value: each then holds two latents of one row
                        __nv_bfloat16 *dst = p.o + (row0 + 16 * e + (lane & 1)) * kLatent + (lat & ~1);
                        const int left = rows_here - 16 * e - (lane & 1);
#pragma unroll
                        for (int y = 0; y < 16; y += 2) {
                            const float2 f = *reinterpret_cast<const float2 *>(&sm.factor[16 * e + y]);
                            const __nv_bfloat162 h =
                                __floats2bfloat162_rn(__uint_as_float(x[y]) * f.x, __uint_as_float(x[y + 1]) * f.y);
                            const uint32_t own = *reinterpret_cast<const uint32_t *>(&h);
                            const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
                            const uint32_t two_lat = (lane & 1) ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
                            if (y < left) *reinterpret_cast<uint32_t *>(dst + y * kLatent) = two_lat;
                        }
                    } else {  // rows past the last are written too (their columns of O^T are nobody's): parts are npad rows
                        float *dst = p.part_o + (part0 + 16 * e) * kLatent + lat;
#pragma unroll
                        for (int y = 0; y < 16; ++y) dst[y * kLatent] = __uint_as_float(x[y]);
                    }
                }
            }
            // O^T has been read: the next stretch's P (all threads arrive) lets the MMA warp write it
            tc::fence_before_sync();
            named_sync(2, kSoftmaxThreads);
            if (w.work) ++seg;
        }
        if (!ok) sm.failed = 1;
    }
    tc::fence_before_sync();
    __syncthreads();
    if (sm.failed && (warp == 8 || warp == 9)) {
        // a wait gave up: report it, and let what is in flight land before the memory goes
        if (tma::elect()) {
            tc::commit(&sm.drained);  // each issuing thread's own products
            if (warp == 8) {
                set_status(p.status, KDA_ERR_CUDA);
                tc::mbar_wait(&sm.drained, 0);
                if (sm.q_issued > 0) tc::mbar_wait(&sm.q_full, (sm.q_issued - 1) & 1);
                for (int e = max(0, sm.pair_issued - geo.np); e < sm.pair_issued; ++e)
                    tc::mbar_wait(&sm.pair_full[e % geo.np], (e / geo.np) & 1);
                for (int e = max(0, sm.pos_issued - geo.nr); e < sm.pos_issued; ++e)
                    tc::mbar_wait(&sm.pos_full[e % geo.nr], (e / geo.nr) & 1);
            }
        }
        __syncwarp();
    }
    if (warp == 8) tc::tmem_dealloc(tmem, 512);
}

// The join of the sequences that a run's border cuts. With fewer sequences than groups block x
// belongs to sequence x, whose place in the list it adds up itself; with more it belongs to
// the border before group x + 1, where the main kernel left the place, and the first border
// inside a sequence joins it. W warps share a row's parts, each lane 16 / Z of the 512 latents, Z
// blocks a row (1M x 12: 195 us with one, 192 with four); the parts are added in list order within a
// warp and the warps' sums in warp order, so the result does not depend on timing. With W = 1 the
// way through shared memory is not needed, but the 32 KB keep these blocks off the SMs until
// the main kernel's are through: without them they wait beside it, and 256 x 96 takes 2% longer.
constexpr int kJoinThreads = 512;
template <int W, int Z>
__global__ void __launch_bounds__(kJoinThreads) kda_mla_join_kernel(const __grid_constant__ DecodeArgs p) {
    constexpr int kRows = kJoinThreads / 32 / W;  // rows of a block
    constexpr int kLat = kLatent / Z, kVec = kLat / 128;  // its latents, and float4 of a lane
    __shared__ float s_o[kRows][W][kLat];
    __shared__ float s_m[kRows][W], s_l[kRows][W];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t n, tiles, b;  // the sequence, its tiles, the run after the one that holds its first tile
    int64_t first;        // list index of that tile
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
        const Runs runs(total, p.G);
        first = before;
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
    const bool live = rr < p.geo.R;
    const int rt = (live ? rr : 0) / p.geo.rows, r = (live ? rr : 0) % p.geo.rows;
    const float c = p.scale * 1.4426950408889634f;
    // parts: run b - 1 (slot 1, it holds the sequence's start), then the following runs (slot 0)
    const int lat0 = blockIdx.z * kLat;
    float m = -INFINITY, l = 0.f, o[4 * kVec];
#pragma unroll
    for (int i = 0; i < 4 * kVec; ++i) o[i] = 0.f;
    auto row_of = [&](int i) {
        const int64_t gq = b - 1 + i;
        return ((2 * gq + (i == 0 ? 1 : 0)) * p.geo.RT + rt) * p.geo.npad + r;
    };
    if (live) {
        // the common maximum of this warp's parts first, then one weighted sum
        for (int i = part + W * lane; i < count; i += W * 32)
            m = fmaxf(m, p.part_ml[row_of(i)].x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll (Z > 1 ? 8 : 4)
        for (int i = part; i < count; i += W) {
            const int64_t q = row_of(i);
            const float2 ml = p.part_ml[q];
            const float f = tc::ex2((ml.x - ms) * c);
            l += f * ml.y;
            const float4 *src = reinterpret_cast<const float4 *>(p.part_o + q * kLatent + lat0) + lane;
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                const float4 x = __ldcs(src + 32 * v);
                o[4 * v] += f * x.x;
                o[4 * v + 1] += f * x.y;
                o[4 * v + 2] += f * x.z;
                o[4 * v + 3] += f * x.w;
            }
        }
    }
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
    const int64_t row = (int64_t)n * p.geo.R + rr;
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

constexpr size_t kSmemMax = 232448;

// Row tiles of equal size; the rings take what Q and P leave. One tile up to 96 rows and two up to
// 192, with M = 128 past 64 rows. From there on as few as 96 rows each allow, or as 64 do (M = 64, four of
// Q's chunks in TMEM) where that is less than half as many again: 64 sequences of up to 8000 rows take with
// tiles of up to 64 and 96 rows 188 and 213 us (256 rows, 4 and 3 tiles), 222 and 214 (288, 5 and 3), 225
// and 229 (320, 5 and 4), 265 and 269 (384, 6 and 4), 342 and 386 (512, 8 and 6), 395 and 384 (576, 9 and 6),
// 422 and 452 (640, 10 and 7), 512 and 498 (768, 12 and 8), 669 and 694 (1024, 16 and 11).
DecodeGeom geometry(int32_t H, int32_t m) {
    DecodeGeom q{};
    q.R = H * m;
    q.RT = (q.R + kWideRows - 1) / kWideRows;
    const int32_t narrow = (q.R + kRowTile - 1) / kRowTile;
    if (q.RT > 2 && 2 * (int64_t)narrow < 3 * (int64_t)q.RT) q.RT = narrow;
    q.rows = ((q.R + q.RT - 1) / q.RT + 7) / 8 * 8;
    q.npad = (q.rows + 15) / 16 * 16;
    q.qt = q.rows > kRowTile ? 1 : (q.RT == 1 ? 0 : 2);  // 4 npad + 64 or 128 + 64 qt TMEM columns: 512 at most
    const size_t fixed = 1024 + sizeof(DecodeSmem) + (size_t)(9 - 2 * q.qt) * q.rows * 128 + (size_t)q.npad * 128;
    const size_t room = kSmemMax - fixed;
    q.nr = 2;
    q.np = (int32_t)((room - q.nr * kChunkB) / kPairB);
    if (q.np > kMaxPair) q.np = kMaxPair;
    const size_t extra = room - q.nr * kChunkB - (size_t)q.np * kPairB;
    if (extra >= kChunkB) ++q.nr;
    q.smem = (uint32_t)(fixed + (size_t)q.np * kPairB + (size_t)q.nr * kChunkB);
    return q;
}
static_assert(kSmemMax - 1024 - sizeof(DecodeSmem) - 10 * kRowTile * 128 >= 8 * kPairB + 2 * kChunkB, "two tiles' rings");
static_assert(kSmemMax - 1024 - sizeof(DecodeSmem) - 8 * kWideRows * 128 >= 7 * kPairB + 2 * kChunkB, "96 rows leave 7 pairs");

// groups of CTAs that share the list: one CTA an SM
int32_t groups_of(int32_t RT, int32_t sms) { return sms / RT > 0 ? sms / RT : 1; }

struct DecodeWs {
    size_t head, ml, o, total;
};
DecodeWs decode_ws(const DecodeGeom &q) {
    DecodeWs w;
    size_t parts = 2 * (size_t)groups_of(q.RT, kMaxGroups) * q.RT * q.npad;
    const size_t widest = 2 * (size_t)kMaxGroups * kWideRows;
    if (q.RT > 1 && parts < widest) parts = widest;  // more rows never need less
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    w.head = 0;
    w.ml = up(8 + 16 * kMaxGroups);
    w.o = w.ml + up(parts * sizeof(float2));
    w.total = w.o + parts * kLatent * sizeof(float);
    return w;
}

template <int W, int Z>
cudaError_t launch_join(const DecodeArgs &a, cudaStream_t st) {
    const int rows = kJoinThreads / 32 / W;
    const int cuts = a.N < a.G ? a.N : a.G - 1;
    return launch_after(kda_mla_join_kernel<W, Z>, dim3(cuts, (a.geo.R + rows - 1) / rows, Z), dim3(kJoinThreads), 0, st, a);
}

}  // namespace
}  // namespace kda

extern "C" {

size_t kda_mla_decode_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t num_tokens) {
    if (num_seqs < 0 || num_heads < 0 || num_tokens < 0) return 0;
    if ((int64_t)num_heads * num_tokens > INT32_MAX / 2 || num_heads == 0 || num_tokens == 0) return 256;
    return kda::decode_ws(kda::geometry(num_heads, num_tokens)).total;
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
    if (page_stride >= ((int64_t)1 << 38)) return KDA_ERR_SHAPE;
    if (num_seqs == 0 || num_tokens == 0) return KDA_OK;
    if (!q_lat || !q_pe || !cache || !page_table || !cache_lens || !o || !workspace) return KDA_ERR_NULL;
    if (!mla_aligned(q_lat, 16) || !mla_aligned(q_pe, 16) || !mla_aligned(cache, 16) || !mla_aligned(o, 16) ||
        !mla_aligned(lse, 4) || !mla_aligned(page_table, 4) || !mla_aligned(cache_lens, 4) || !mla_aligned(status, 4) ||
        !mla_aligned(workspace, 256))
        return KDA_ERR_ALIGN;
    if (workspace_bytes < kda_mla_decode_workspace_size(num_seqs, num_heads, num_tokens)) return KDA_ERR_WORKSPACE;
    int sms = 0, device = 0;
    rc = device_sms(&sms, &device);
    if (rc != KDA_OK) return rc;
    if (device >= 64) return KDA_ERR_DEVICE;

    DecodeArgs a;
    a.geo = geometry(num_heads, num_tokens);
    const DecodeWs w = decode_ws(a.geo);
    a.rb = page_size % 64 == 0 ? 64 : (page_size % 32 == 0 ? 32 : 16);
    const uint64_t rows = (uint64_t)num_seqs * a.geo.R;
    const uint64_t dl[3] = {kLatent, rows, 0}, sl[3] = {1, kLatent, 0}, dp[3] = {kPos, rows, 0}, sp[3] = {1, kPos, 0};
    // a cache without pages keeps one page of extent: no id is in range, every load is past it
    const uint64_t dc[3] = {kRow, (uint64_t)page_size, (uint64_t)(num_pages > 0 ? num_pages : 1)};
    const uint64_t sc[3] = {1, kRow, (uint64_t)page_stride};
    if (!tma::encode(&a.q_lat, q_lat, 2, dl, sl, a.geo.rows, 1) || !tma::encode(&a.q_pe, q_pe, 2, dp, sp, a.geo.rows, 1) ||
        !tma::encode(&a.cache, cache, 3, dc, sc, a.rb, 1))
        return KDA_ERR_CUDA;
    a.q = reinterpret_cast<const __nv_bfloat16 *>(q_lat);
    a.rows = reinterpret_cast<const __nv_bfloat16 *>(cache);
    a.page_stride = page_stride;
    a.table = page_table;
    a.lens = cache_lens;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.N = num_seqs;
    a.H = num_heads;
    a.m = num_tokens;
    a.scale = scale;
    a.o = reinterpret_cast<__nv_bfloat16 *>(o);
    a.lse = lse;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.head = reinterpret_cast<int64_t *>(ws + w.head);
    a.part_ml = reinterpret_cast<float2 *>(ws + w.ml);
    a.part_o = reinterpret_cast<float *>(ws + w.o);
    a.status = status;
    static std::atomic<bool> configured[64];  // the kernels' shared memory, set once a device
    if (!configured[device].load(std::memory_order_acquire)) {
        for (auto kernel : {kda_mla_decode_kernel<64, 0>, kda_mla_decode_kernel<64, 2>, kda_mla_decode_kernel<128, 1>})
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax) != cudaSuccess)
                return KDA_ERR_CUDA;
        configured[device].store(true, std::memory_order_release);
    }
    // no more groups than the longest page tables could give tiles to
    const int64_t most = (int64_t)num_seqs * (((int64_t)max_pages * page_size + kKvTile - 1) / kKvTile + 1);
    a.G = groups_of(a.geo.RT, sms < kMaxGroups ? sms : kMaxGroups);
    if (a.G > most) a.G = (int32_t)most;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto kernel = a.geo.qt == 2 ? kda_mla_decode_kernel<64, 2> : (a.geo.qt == 1 ? kda_mla_decode_kernel<128, 1> : kda_mla_decode_kernel<64, 0>);
    if (launch_after(kernel, dim3((unsigned)(a.G * a.geo.RT)), dim3(kDecThreads), a.geo.smem, st, a) != cudaSuccess)
        return KDA_ERR_CUDA;
    if (a.G > 1) {
        // a split sequence has about G / N parts: many are shared by a block's 16 warps, a few by four, and
        // two or three are one warp's. With 1, 4 and 16 warps a row: 1M x 12 236, 200 and 193 us; 8 sequences
        // of 30000 rows x 12 heads 50, 36 and 34; 32 of 8000 x 16 42, 37 and 41; 256 of 8000 x 96 293, 347, 440
        const int64_t n = num_seqs;
        const cudaError_t e = n * 16 <= a.G ? launch_join<16, 4>(a, st) : (n * 4 <= a.G ? launch_join<4, 2>(a, st) : launch_join<1, 1>(a, st));
        if (e != cudaSuccess) return KDA_ERR_CUDA;
    }
    return KDA_OK;
}

}  // extern "C"
