// Latent attention in the absorbed form over the pages of the 8-bit cache: kda_mla_decode_fp8.
//
//   x_rj = log2(e) scale s_j (q_r . row_j),  o_r = sum_j 2^{x_rj} s_j c_j / sum_j 2^{x_rj}
//
// with c_j the stored latents and s_j = 2^e_j the row's scale. The work is cut as in the bf16 form: all cached
// rows of the batch are one list of tiles of 64, cut into equal runs; a CTA takes a run for up to 96 query rows
// (window token and head), and a second kernel joins the sequences that a run's border cuts.
//
// The products take the cache as it lies: e4m3, without unpacking. Their other operands have 16 bits, so each
// is two 8-bit ones.
//
//   Scores. A query row in units of a power of two for which its largest latent is in (224, 448] is e4m3 hi and
//   e4m3 lo of the rest: 4 bits and, with the rest's sign, 4 bits more are bf16's 8, so q is exact down to 2^-10 of
//   the unit. Q is M (rows), the cached rows are N and are read K-major; with up to 64 query rows hi and lo
//   are rows of one product, so that a tile is read once, with more two products. The positional part stays
//   bf16 (the key is stored in units of s_j, so one accumulator takes both).
//   Values. The weight w = 2^{x_rj + e_j - m_r} takes the row's scale along; it is e4m3 and, its rest, e5m2, whose
//   range goes on 2^-7 further down. O^T = C^T W^T: M = 128 latents (the same tile, read MN-major), N = query rows.
//
// The two hold a weight of 2^-6 to 448 units as bf16 would, to 2^-8 of itself; a lower one is off by up to 2^-14 units. So
// m_r follows the weights both ways, and is set anew, with O^T rescaled, where
//   a tile's largest weight is over 2^8.75: then at 2^6, so that the others keep 12 binary places below it;
//   four tiles' weights sum to less than 8: then their sum at 2^7 (or the tile's largest at 2^2.5, if that is the larger unit).
// Tiles of weights that sum to more lose at most 256 2^-14 of 8, 2^-9, whatever they hold. A stretch's first tile has its largest at
// 2^2.5, which leaves room to grow; but the first 8 rows of a sequence, which often outweigh all others, may be 2^6.2 above
// that. m_r stays within 2^40 of the largest seen (2^46.2 of those rows), beyond which a tile counts for nothing.
// The other rows' part of the output beside a first key of 0.95 of the sum is off by 0.2% (rms; bf16 weights 0.23%), beside one of
// 0.999 by 1.8%; beside a key of 0.9 or 0.99 in the middle by 0.3% and 1.0%, until the unit has followed. (With the largest of four
// tiles held above 2^-1 by 2^2.5 these were 2.4, 25, 1.0 and 3.7%.) How often the unit is set, emulated: with
// random scores of a deviation of 1.7 natural units in 5% of the tiles of 96 rows, of 3.0 in 65%, which each take a third longer;
// another look a tile behind every new maximum would make 0.15% of the 0.3, and 88% of the 65.
//
// Rows of a tile behind the sequence's length may hold anything: their scores are replaced by -inf, the
// product's 32-row steps past the length are left out, and value rows inside the last step are zeroed in shared
// memory; their scales are never loaded.
//
// Three forms by the CTA's query rows, each with the longest ring that its Q and W leave room for: up to 32 (M = 64, four
// tiles), 64 (M = 128, three) and 96 (hi and lo apart, two). Eight softmax warps hold a tile's scores in registers, a thread
// 8 or 16 cached rows of one or two query rows (with up to 64 rows as the fragments that tcgen05.ld gives, hi and lo added
// in place) or 32 of one; three warps' elected threads issue score products, value products and loads. S and W are double, so
// that a tile's scores are computed under the last one's softmax and value product.
//
// What bounds it (at 2070 MHz): a tile takes 1830 cycles, 0.885 us, with up to 32 rows, which is the rows' arrival (7.1 TB/s); 2360
// to 2440 with 48, the softmax's chain (wait, load, 16 exponentials a thread, a barrier, conversions and 16-bit stores); 3750 with 96,
// of which the products' operands occupy shared memory for 2600. A sequence costs besides what kda_mla_decode_fp8 counts for it
// (extra8), 5 to 16 us, and the join 3 to 16. Measured, whole calls: 1048576 rows x 12 heads 112 us (6.0 TB/s of 6.8), 32
// sequences of up to 8000 rows x 16 25.3 (pages of 64 rows 23.7), 64 x 48 55.5, 256 x 96 251 to 255 (0.87 PFLOP/s as a bf16 form
// counts), 64 x 96 x 4 tokens 220 (0.94). With pages of 32 and 16 rows 1048576 x 12 takes 131 and 159 us: ten and twenty loads a
// tile by one thread.

#include <cstddef>

#include "kda_latent_split.cuh"

namespace kda {
namespace {

constexpr uint32_t kChunk8 = kKvTile * 128;     // 64 rows of 128 bytes: 128 latents, or the positional key
constexpr int kChunks = 5;                      // of a tile: 512 latents, then the positional key
constexpr uint32_t kTile8 = kChunks * kChunk8;
constexpr int kMaxSlots = 4, kMaxPieces = 2 * kChunks;  // of the ring
constexpr int kScales = 8;                      // tiles whose scales are kept: more than the ring has, so that a slot is loaded anew only when
                                                // the softmax is through with its tile
// Two softmax warps a lane quarter: each takes half of a tile's cached rows, and of O^T's blocks of 128 latents. Behind them
// stand four more: score issue, value issue, TMA, none. (Four a quarter: 32 rows 112 -> 142 us, 96 rows 312 -> 324.)
constexpr int kSets = 2, kSetCols = kKvTile / kSets, kBlocks = kLatent / 128 / kSets;
constexpr int kSoft = 128 * kSets, kIssue = kSoft / 32, kThreads = kSoft + 128;  // kIssue: the first warp behind them
// Registers that a block is launched with a thread, and how they are shared out. (208 and 80: 32 x 16 27.2 us, 1M x 12
// 112.8, 64 x 48 58.0, 256 x 96 255.8; 200 and 96: 25.4, 111.5, 57.4, 255.4; 184 and 128: 26.4, 113.2, 56.5, 253.6.)
constexpr int kLaunched = 168;
constexpr int soft_regs(int form) { return form == 0 ? 200 : 184; }
constexpr int issue_regs(int form) { return form == 0 ? 96 : 128; }
static_assert(kSoft * soft_regs(0) + 128 * issue_regs(0) <= kThreads * kLaunched, "the shares' sum");
static_assert(kSoft * soft_regs(1) + 128 * issue_regs(1) <= kThreads * kLaunched, "the shares' sum");
constexpr int kRows8 = 64, kMostRows8 = 96;     // query rows of a CTA at most: with hi and lo in one product, and at all
// Powers of two: where a unit is set below the largest weight of a stretch's first tile, and of one above the unit's range; how far it
// is set below the sum of a low window; what the first rows of a sequence may be above the others of their tile
constexpr float kSet = 2.5f, kSetHigh = 6.0f, kSetLow = 7.0f, kHigh = 8.75f, kEarly = 6.2f, kReach = 40.0f;
constexpr float kMost = 430.0f;                 // weights: below 2^kHigh
constexpr float kLeast = 8.0f, kNothing = 0x1p-14f;  // a window's sum: what is low, and what fp16 has nothing left of
constexpr int kWindow = 4;                      // tiles over which a row's weights have to be low
constexpr int kEarlyRows = 8;
static_assert(kSet + kEarly < kHigh, "the first rows stay in range");
constexpr int kBad = 8;                         // stretches that the loads may be ahead of the output

// Tiles that the ring holds beside Q and W, and the pieces that a tile is loaded in: one (a thread takes 600 cycles
// for a wait and a load, which five a tile would make the bound of few rows, as the small pages' ten and twenty loads do), or
// its five chunks where only two tiles fit, each as soon as its products are through.
// (96 rows with one W and a ring of 12 chunks: 256 x 96 257 -> 268 us, the softmax then waits for the tile before; with two and 11
// chunks 259 to 264, the places of whose chunks take the issuing threads longer to find.)
constexpr int tiles_in(int form) { return 4 - form; }
constexpr int pieces_of(int form) { return form < 2 ? 1 : kChunks; }

struct Geom8 : SplitGeom {
    int32_t form;  // query rows of a CTA: 0 up to 32, 1 up to 64, 2 up to 96
    uint32_t smem;
};

struct Args8 : SplitArgs {
    CUtensorMap map;
    const __nv_bfloat16 *q_lat, *q_pe;
    const uint8_t *rows;
    int64_t page_stride;
    int32_t rb;  // rows of a TMA box: 64 (it then takes all chunks of a tile that is loaded in one piece), 32 or 16
    float c;     // log2(e) scale
    Geom8 geo;
};

struct Smem8 {
    uint64_t q_ready, s_full[2], s_free[2], p_full[2], drained;
    uint64_t full[kMaxPieces], empty[kMaxPieces];  // a piece of a tile is there; may be loaded over
    uint64_t done[kMaxSlots];           // a tile's products are through
    uint64_t sc_full[kScales];
    alignas(16) float sc[kScales][kKvTile];  // scales of a tile's rows (bulk copies land there)
    float row_c[kMostRows8];            // by query row: log2(e) scale times the unit of Q
    float factor[128];                  // by query row: scale of O^T
    float part[kSets][128], recent[kSets][128];  // by query row: the sets' maxima or sums, and sums of a window's weights
    uint32_t tmem;
    int32_t failed, bad[kBad];
    Run run;
    int32_t issued, scaled;  // loads of pieces and of scales
};

// kind::f8f6f4, e4m3 times e4m3 (or e5m2 as B), fp32 accumulator; one step takes 32 of the contraction: 32 bytes
// of a K-major operand, 32 rows of an MN-major one
__host__ __device__ constexpr uint32_t idesc8(int M, int N, int b_e5m2, int a_mn) {
    return (1u << 4) | ((uint32_t)b_e5m2 << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma8(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p;\n.reg .b64 a, b;\nmov.b64 a, {%1, %5};\nmov.b64 b, {%2, %5};\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n}\n" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(id), "r"(accumulate), "n"(tma::kDescHi));
}
// whether the phase of this parity has ended, without waiting: asked for early, used with wait_warp later
__device__ __forceinline__ bool peek(uint64_t *mbar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(done)
                 : "r"(tc::smem_addr(mbar)), "r"(parity)
                 : "memory");
    return done != 0;
}
__device__ __forceinline__ bool wait_peeked(bool there, uint64_t *mbar, uint32_t parity) {
    return __all_sync(0xffffffffu, there) || tma::wait_warp(mbar, parity);
}
// 16 TMEM lanes and 32 columns as a warp's fragments: x[4 g + 0, 1] are columns 8 g + 2 (lane % 4) + 0, 1 of TMEM
// lane lane / 4, x[4 g + 2, 3] the same of TMEM lane 8 + lane / 4. Without the wait
__device__ __forceinline__ void tmem_ld_fragments(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// two values (a first) as a pair of fp16
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
    uint32_t w;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}
__device__ __forceinline__ uint32_t max_half2(uint32_t a, uint32_t b) {
    asm("max.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return a;
}
__device__ __forceinline__ uint32_t add_half2(uint32_t a, uint32_t b) {
    asm("add.rn.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return a;
}
// A pair of fp16 as two bytes of e4m3 and two for the rests: e5m2 for weights, which goes on further down, and e4m3 for
// queries, whose eight bits the two then hold
__device__ __forceinline__ void split_weights(uint32_t w, uint16_t &hi, uint16_t &lo) {
    asm("{\n.reg .b32 v;\ncvt.rn.satfinite.e4m3x2.f16x2 %0, %2;\ncvt.rn.f16x2.e4m3x2 v, %0;\nsub.rn.f16x2 v, %2, v;\n"
        "cvt.rn.satfinite.e5m2x2.f16x2 %1, v;\n}\n"
        : "=&h"(hi), "=h"(lo)
        : "r"(w));
}
__device__ __forceinline__ void split_queries(uint32_t w, uint16_t &hi, uint16_t &lo) {
    asm("{\n.reg .b32 v;\ncvt.rn.satfinite.e4m3x2.f16x2 %0, %2;\ncvt.rn.f16x2.e4m3x2 v, %0;\nsub.rn.f16x2 v, %2, v;\n"
        "cvt.rn.satfinite.e4m3x2.f16x2 %1, v;\n}\n"
        : "=&h"(hi), "=h"(lo)
        : "r"(w));
}

__device__ __forceinline__ void store2(uint32_t at, int more, uint16_t v) {
    asm volatile("st.shared.b16 [%0], %1;\n" ::"r"(at + more), "h"(v) : "memory");
}
__device__ __forceinline__ void store16(uint32_t at, const uint32_t (&v)[4]) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
// The unit 2^a of a query row: its largest latent in (224, 448] of it, unless positional values that dwarf the latents would
// then be over 2^61 (times keys in units of 2^-40 they have to stay in fp32's range). Given the bits of the largest magnitudes as fp32, where NaN is above all.
struct Unit {
    int a;
    float inv;
    bool sound;  // no infinity, no NaN: a row with one has no scores
    __device__ __forceinline__ Unit(uint32_t top, uint32_t top_pe)
        : a(max(max((int)((top + 0x1FFFFFu) >> 23) - 135, (int)(top_pe >> 23) - 187), -100)), inv(exp2_of(-min(a, 120))),
          sound(max(top, top_pe) < 0x7f800000u) {}
    __device__ __forceinline__ uint32_t positions(uint32_t two) const {  // in the unit
        const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(two << 16) * inv, __uint_as_float(two & 0xffff0000u) * inv);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    __device__ __forceinline__ float factor(float c) const { return sound ? c * exp2_of(min(a, 120)) : NAN; }
};
// two bf16 values in the unit as e4m3 and the e4m3 of their rest (in fp16 they are what they were)
__device__ __forceinline__ void split_query(uint32_t two, uint64_t inv2, uint32_t &hi, uint32_t &lo) {
    const float2 x = upk2(mul2(pk2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u)), inv2));
    uint16_t h, l;
    split_queries(half2_of(x.x, x.y), h, l);
    hi = h, lo = l;
}

// FORM: query rows of a CTA, as in Geom8
template <int FORM>
__global__ void __launch_bounds__(kThreads, 1) kda_mla_decode_fp8_kernel(const __grid_constant__ Args8 p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    constexpr int MS = FORM == 0 ? 64 : 128;   // M of the score product
    constexpr bool kStack = FORM < 2;          // hi and lo rows in one product
    constexpr int kRowsQ = kStack ? MS / 8 : 32;   // query rows of a lane quarter (and, stacked, where lo lies behind hi)
    constexpr int kR = FORM == 1 ? 2 : 1;          // query rows of a softmax thread,
    constexpr int kC = kStack ? kSetCols / 4 : kSetCols;  // and cached rows of a tile for each
    constexpr int kTiles = tiles_in(FORM), kPieces = pieces_of(FORM);
    const Geom8 &geo = p.geo;
    // Q: four chunks of 128 latents of hi (and lo, stacked; else four of lo behind), then the positional part
    const uint32_t q_chunk = (uint32_t)(kStack ? MS : geo.rows) * 128;
    constexpr int q_chunks = kStack ? 5 : 9;
    uint8_t *s_q = base;                          // M = 128 reads of fewer rows run on into what follows,
    uint8_t *s_p = s_q + q_chunks * q_chunk;      // rows of S that nobody reads
    const uint32_t p_bytes = (uint32_t)geo.npad * 128;  // W, twice: npad rows of 64 bytes of e4m3, then 64 of e5m2
    uint8_t *s_ring = s_p + 2 * p_bytes;
    Smem8 &sm = *reinterpret_cast<Smem8 *>(s_ring + kTiles * kTile8);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rt = blockIdx.x % geo.RT, g = blockIdx.x / geo.RT;

    pdl_wait();
    if (warp == kIssue + 2 && lane == 0) tma::prefetch_map(&p.map);
    if (warp == 0) {
        find_run(p, g, rt, sm.run);
        if (lane == 0) {
            sm.failed = 0;
            sm.issued = sm.scaled = 0;
            for (int i = 0; i < kScales; ++i) tc::mbar_init(&sm.sc_full[i], 1);
            for (int i = 0; i < kBad; ++i) sm.bad[i] = 0;
            tc::mbar_init(&sm.q_ready, kIssue);
            for (int i = 0; i < 2; ++i) tc::mbar_init(&sm.s_full[i], 2), tc::mbar_init(&sm.s_free[i], kIssue);
            for (int i = 0; i < 2; ++i) tc::mbar_init(&sm.p_full[i], kIssue);
            tc::mbar_init(&sm.drained, 2);
            for (int i = 0; i < kTiles; ++i) {
                tc::mbar_init(&sm.done[i], 1);
                for (int c = 0; c < kPieces; ++c) tc::mbar_init(&sm.full[i * kPieces + c], 1), tc::mbar_init(&sm.empty[i * kPieces + c], 1);
            }
            tc::mbar_init_fence();
        }
    } else if (warp == kIssue) {
        tc::tmem_alloc(&sm.tmem, 512);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    pdl_trigger();
    const uint32_t tmem = sm.tmem;
    const uint32_t t_s = tmem + 4 * geo.npad;  // two S tiles of 64 columns behind O^T
    const int row_first = rt * geo.rows, rows_here = max(0, min(geo.rows, geo.R - row_first));
    bool ok = true;

    if (warp >= kIssue) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(issue_regs(FORM)));
        if (warp == kIssue + 2) {
            // ---- TMA producer: one thread ----
            if (tma::elect()) {
                Walk w;
                w.start(p, sm.run);
                w.skip_idle(p);
                int seg = 0, ps = 0, pph = 0, issued = 0, scaled = 0;
                const int sub = kKvTile / p.rb;  // boxes of rows of a tile: 1, 2 or 4
                while (!w.done() && ok) {
                    const int32_t *entry = p.table + (int64_t)w.n * p.max_pages;
                    const uint32_t row0 = (uint32_t)w.j0 * kKvTile, of = row0 / (uint32_t)p.page_size;
                    entry += of;
                    int32_t at = (int32_t)(row0 - of * (uint32_t)p.page_size);  // row within the page
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
                    sm.bad[seg % kBad] = 0;
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
                            sm.bad[seg % kBad] = 1;
                            set_status(p.status, KDA_ERR_PAGES);
                        }
                        look(j + 1);
                        const int valid = min(kKvTile, w.len - j * kKvTile), boxes = (valid + p.rb - 1) / p.rb;
                        const uint32_t box = (uint32_t)p.rb * 128;
                        uint8_t *dst = s_ring + ps * kTile8;
#pragma unroll
                        for (int c = 0; c < kPieces; ++c) {  // the positional chunk first
                            const int chunk = c == 0 ? kChunks - 1 : c - 1;
                            ok = tc::mbar_wait(kPieces == 1 ? &sm.done[ps] : &sm.empty[ps * kPieces + c], pph ^ 1);
                            if (!ok) break;
                            uint64_t *full = &sm.full[ps * kPieces + c];
                            if (kPieces == 1) {
                                tc::mbar_arrive_expect_tx(full, kChunks * boxes * box);
                                if (p.rb == kKvTile) {
                                    tma::load_4d(dst, &p.map, full, 0, ry[0], 0, pg[0]);
                                } else {
                                    for (int i = 0; i < kChunks; ++i)
#pragma unroll
                                        for (int b = 0; b < 4; ++b)
                                            if (b < boxes) tma::load_4d(dst + i * kChunk8 + b * box, &p.map, full, 0, ry[b], i, pg[b]);
                                }
                            } else {
                                tc::mbar_arrive_expect_tx(full, boxes * box);
                                tma::load_4d(dst + chunk * kChunk8, &p.map, full, 0, ry[0], chunk, pg[0]);
#pragma unroll
                                for (int b = 1; b < 4; ++b)
                                    if (b < boxes) tma::load_4d(dst + chunk * kChunk8 + b * box, &p.map, full, 0, ry[b], chunk, pg[b]);
                            }
                            ++issued;
                            if (c > 0) continue;
                            // the rows' scales stand behind the page's rows; of a page that is not there, none are loaded
                            uint32_t scales = 0;
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                if (b < boxes && pg[b] != INT32_MAX) scales += 4 * p.rb;
                            uint64_t *there = &sm.sc_full[scaled % kScales];
                            tc::mbar_arrive_expect_tx(there, scales);
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                if (b < boxes && pg[b] != INT32_MAX)
                                    tc::bulk_g2s(&sm.sc[scaled % kScales][b * p.rb],
                                                 p.rows + pg[b] * p.page_stride + (int64_t)p.page_size * kRow8 + 4 * ry[b], 4 * p.rb, there);
                            ++scaled;
                            // the next tile into L2: from HBM its load would take longer than the ring has tiles for
                            if (j + 1 < w.j1) {
#pragma unroll
                                for (int b = 0; b < 4; ++b) {
                                    const int64_t row = ((int64_t)j + 1) * kKvTile + b * p.rb;
                                    if (b < sub && row < w.len && (uint32_t)pg_next[b] < (uint32_t)p.num_pages) {
                                        const uint8_t *page = p.rows + pg_next[b] * p.page_stride;
                                        tma::prefetch_l2(page + (int64_t)ry_next[b] * kRow8, (uint32_t)p.rb * kRow8);
                                        tma::prefetch_l2(page + (int64_t)p.page_size * kRow8 + 4 * ry_next[b], 4 * p.rb);
                                    }
                                }
                            }
                        }
                        if (!ok) break;
                        if (++ps == kTiles) ps = 0, pph ^= 1;
                    }
                    ++seg;
                    w.next(p);
                    w.skip_idle(p);
                }
                sm.issued = issued;
                sm.scaled = scaled;
                if (!ok) sm.failed = 1;
            }
            __syncwarp();
        } else if (warp == kIssue) {
            // ---- score products: one thread ----
            if (tma::elect()) {
                constexpr uint32_t id = idesc8(MS, kKvTile, 0, 0), id_pe = tma::idesc(MS, kKvTile, 0, 0);
                const uint32_t q_lo = tma::lo_k(tc::smem_addr(s_q)), ring_lo = tma::lo_k(tc::smem_addr(s_ring)), q_step = q_chunk >> 4;
                Walk w;
                w.start(p, sm.run);
                w.skip_idle(p);
                int k = 0, seg = 0, ps = 0, pph = 0;
                while (!w.done() && ok) {
                    ok = tc::mbar_wait(&sm.q_ready, seg & 1);
                    for (int j = w.j0; j < w.j1 && ok; ++j, ++k) {
                        ok = tc::mbar_wait(&sm.s_free[k & 1], ((k >> 1) & 1) ^ 1);
                        const uint32_t d = t_s + (k & 1) * kKvTile;
                        const uint32_t b = ring_lo + ps * (kTile8 >> 4);
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) {  // the positional chunk first
                            if (c < kPieces) {
                                ok = ok && tc::mbar_wait(&sm.full[ps * kPieces + c], pph);
                                if (!ok) break;
                                tc::fence_after_sync();
                            }
#pragma unroll
                            for (int s = 0; s < 4; ++s) {
                                if (c == 0) {
                                    tma::mma_ss(d, q_lo + (q_chunks - 1) * q_step + 2 * s, b + (4 * kChunk8 >> 4) + 2 * s, id_pe, s != 0);
                                } else {
                                    const uint32_t a = q_lo + (c - 1) * q_step + 2 * s, bb = b + (c - 1) * (kChunk8 >> 4) + 2 * s;
                                    mma8(d, a, bb, id, 1);
                                    if (!kStack) mma8(d, a + 4 * q_step, bb, id, 1);
                                }
                            }
                            if (c == 0 && kPieces > 1) tc::commit(&sm.empty[ps * kPieces]);
                        }
                        if (!ok) break;
                        if (++ps == kTiles) ps = 0, pph ^= 1;
                        // With the scores the softmax may count on the tile's scales, and on the weights of the tile two before
                        // having been used. One thread waits for these instead of every warp, and passes them on by an arrival of
                        // its own: a commit's covers only what the tensor core did.
                        ok = tc::mbar_wait(&sm.sc_full[k % kScales], (k / kScales) & 1) &&
                             (k < 2 || tc::mbar_wait(&sm.done[(k - 2) % kTiles], ((k - 2) / kTiles) & 1));
                        if (!ok) break;
                        tc::commit(&sm.s_full[k & 1]);
                        tma::arrive(&sm.s_full[k & 1]);
                    }
                    ++seg;
                    w.next(p);
                    w.skip_idle(p);
                }
                if (!ok) sm.failed = 1;
            }
            __syncwarp();
        } else if (warp == kIssue + 1) {
            // ---- value products: one thread ----
            if (tma::elect()) {
                const uint32_t id_hi = idesc8(128, geo.npad, 0, 1), id_lo = idesc8(128, geo.npad, 1, 1);
                const uint32_t ring_lo = tma::lo_mn(tc::smem_addr(s_ring), kChunk8), p_lo = tma::lo_k(tc::smem_addr(s_p));
                Walk w;
                w.start(p, sm.run);
                w.skip_idle(p);
                int k = 0, ps = 0;
                while (!w.done() && ok) {
                    for (int j = w.j0; j < w.j1; ++j, ++k) {
                        ok = tc::mbar_wait(&sm.p_full[k & 1], (k >> 1) & 1);
                        if (!ok) break;
                        tc::fence_after_sync();
                        const bool two = w.len - j * kKvTile > 32;  // steps of 32 cached rows
                        const uint32_t more = ((j - w.j0) & (kFold - 1)) != 0;
                        const uint32_t a0 = ring_lo + ps * (kTile8 >> 4), b = p_lo + (k & 1) * (p_bytes >> 4);
#pragma unroll
                        for (int i = 0; i < kChunks - 1; ++i) {
                            const uint32_t a = a0 + i * (kChunk8 >> 4), d = tmem + i * geo.npad;
                            mma8(d, a, b, id_hi, more);
                            mma8(d, a, b + 4, id_lo, 1);
                            if (two) {
                                mma8(d, a + 256, b + 2, id_hi, 1);
                                mma8(d, a + 256, b + 6, id_lo, 1);
                            }
                            if (kPieces > 1) tc::commit(&sm.empty[ps * kPieces + i + 1]);
                        }
                        tc::commit(&sm.done[ps]);
                        if (++ps == kTiles) ps = 0;
                    }
                    w.next(p);
                    w.skip_idle(p);
                }
                if (!ok) sm.failed = 1;
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(soft_regs(FORM)));
        // ---- softmax: a thread takes kC cached rows of a tile for each of kR query rows; then the output ----
        const int quarter = warp & 3, set = warp >> 2;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const bool lead = !kStack || (lane & 3) == 0;  // one lane a row
        int r[kR], unseen[kR];                         // the rows, and the last cached rows that each does not see
        bool owner[kR];
#pragma unroll
        for (int y = 0; y < kR; ++y) {
            r[y] = quarter * kRowsQ + (kStack ? lane / 4 + 8 * y : lane);
            owner[y] = r[y] < rows_here;
            unseen[y] = p.m - 1 - (row_first + (owner[y] ? r[y] : 0)) / p.H;
        }
        const bool warp_rows = quarter * kRowsQ < rows_here;
        // column of a tile of value e
        auto col = [&](int e) { return kSetCols * set + (kStack ? 8 * (e >> 1) + 2 * (lane & 3) + (e & 1) : e); };
        // Where a thread's first weight of a row goes in W, and how far from there those 16 bytes on and the rests lie: a row's
        // 16-byte unit u stands at u ^ (row % 8), its rests four units behind
        uint32_t w_at[kR];
        int w_16[kR], w_64[kR];
        float limit[kR];
#pragma unroll
        for (int y = 0; y < kR; ++y) {
            const int unit = (col(0) >> 4) ^ (r[y] & 7);
            w_at[y] = tc::smem_addr(s_p) + r[y] * 128 + 16 * unit + (col(0) & 15);
            w_16[y] = unit & 1 ? -16 : 16;
            w_64[y] = unit & 4 ? -64 : 64;
            limit[y] = owner[y] ? kMost : INFINITY;
        }
        // the sum of the weights of a row's last window
        auto window = [&](int row) { return sm.recent[0][row] + sm.recent[1][row]; };
        int k = 0, seg = 0;  // tiles and stretches worked on
        // the products of tile t are through: waited for in every tile for the one before the last, so that none is passed over
        auto through = [&](int t) { return tma::wait_warp(&sm.done[t % kTiles], (t / kTiles) & 1); };
        // Q of a stretch, a row a warp at a time; the last stretch's score products are through: its last tile was taken
        auto load_q = [&](int n) {
            const int64_t row0 = (int64_t)n * geo.R + row_first;
            // The loads of kBatch rows are on their way before the first is looked at. (A few rows at a time: this runs once a
            // sequence, and long code that seldom runs is fetched anew each time. 64 x 48 with 1, 2 and 4 56.7, 54.3 and 57.2 us, 256 x 96
            // with 2, 3 and 4 255.3, 252.5 and 254.0.)
            constexpr int kBatch = FORM < 2 ? 2 : 3;
#pragma unroll 1
            for (int q0 = warp; q0 < rows_here; q0 += kIssue * kBatch) {
                struct {
                    uint4 a, b;
                    uint32_t pe;
                } now[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const int64_t row = row0 + min(q0 + kIssue * b, rows_here - 1);
                    const uint4 *src = reinterpret_cast<const uint4 *>(p.q_lat + row * kLatent) + 2 * lane;
                    now[b].a = src[0], now[b].b = src[1];
                    now[b].pe = reinterpret_cast<const uint32_t *>(p.q_pe + row * kPos)[lane];
                }
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const int q = min(q0 + kIssue * b, rows_here - 1);  // (the last row again: the same values)
                    const uint32_t v[8] = {now[b].a.x, now[b].a.y, now[b].a.z, now[b].a.w, now[b].b.x, now[b].b.y, now[b].b.z, now[b].b.w};
                    // bits of the largest magnitudes, as bf16 and then as fp32; NaN is above all
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = __vmaxu2(top, v[i] & 0x7fff7fffu);
                    top = __reduce_max_sync(0xffffffffu, max(top << 16, top & 0xffff0000u));
                    const uint32_t top_pe = __reduce_max_sync(0xffffffffu, max((now[b].pe << 16) & 0x7fffffffu, now[b].pe & 0x7fff0000u));
                    const Unit unit(top, top_pe);
                    const uint64_t inv2 = pk2(unit.inv, unit.inv);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t h[2], l[2];
                        split_query(v[2 * i], inv2, h[0], l[0]);
                        split_query(v[2 * i + 1], inv2, h[1], l[1]);
                        hi[i] = h[0] | (h[1] << 16);
                        lo[i] = l[0] | (l[1] << 16);
                    }
                    // rows of the operand: hi and lo of a quarter one behind the other, or the row itself in chunks of its own
                    const int m_hi = kStack ? (q / kRowsQ) * 2 * kRowsQ + q % kRowsQ : q, m_lo = kStack ? m_hi + kRowsQ : q;
                    uint8_t *at = s_q + (lane >> 3) * q_chunk;
                    *reinterpret_cast<uint4 *>(at + m_hi * 128 + (((lane & 7) ^ (m_hi & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    at += kStack ? 0 : 4 * q_chunk;
                    *reinterpret_cast<uint4 *>(at + m_lo * 128 + (((lane & 7) ^ (m_lo & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    at = s_q + (q_chunks - 1) * q_chunk + (lane & 3) * 4;
                    *reinterpret_cast<uint32_t *>(at + m_hi * 128 + (((lane >> 2) ^ (m_hi & 7)) << 4)) = unit.positions(now[b].pe);
                    if (kStack) *reinterpret_cast<uint32_t *>(at + m_lo * 128 + (((lane >> 2) ^ (m_lo & 7)) << 4)) = 0;
                    if (lane == 0) sm.row_c[q] = unit.factor(p.c);
                }
            }
            fence_proxy_async();
            tma::arrive_warp(&sm.q_ready);
        };
        bool s_there = false;  // of the next tile
        Walk w;
        w.start(p, sm.run);
        {
            Walk first = w;
            first.skip_idle(p);
            if (!first.done()) load_q(first.n);
            named_sync(2, kSoft);
        }
        for (; !w.done() && ok; w.next(p)) {
            float m_ref[kR], m_top[kR], l[kR];
            float recent[kR];  // the sum of the window's weights, and at its end of the whole row
            bool faint[kR];    // the last window's weights were low
            float m_kept[kR], l_kept[kR];  // reference and denominator of the tiles before the last kFold
#pragma unroll
            for (int y = 0; y < kR; ++y) m_ref[y] = m_top[y] = m_kept[y] = -INFINITY, l[y] = l_kept[y] = recent[y] = 0.f, faint[y] = false;
            // the stretch's place among the partials: a run's first stretch, where it continues a sequence, has
            // the first, the last one, which the run's end cuts, the second; before that any other may use it
            const int64_t part0 = (((int64_t)2 * g + (w.j0 == 0 ? 1 : 0)) * geo.RT + rt) * geo.npad;
            if (w.work) {
                float c[kR];
#pragma unroll
                for (int y = 0; y < kR; ++y) c[y] = owner[y] ? sm.row_c[r[y]] : 0.f;
                // the next sequence with rows
                Walk after = w;
                after.next(p);
                after.skip_idle(p);
                const int next_n = after.done() ? -1 : after.n;
                bool stopped = false;
                for (int js = w.j0; !stopped; js += kFold) {
                    if (js > w.j0 && w.j1 - w.j0 > kFold) {
                        // kFold tiles, or the last ones, are in O^T (also with a failed wait: all warps meet these barriers)
                        ok = through(k - 1) && ok;
                        const bool start = js == w.j0 + kFold;
                        named_sync(2, kSoft);  // the factors have been read
#pragma unroll
                        for (int y = 0; y < kR; ++y)
                            if (set == 0 && lead) sm.factor[r[y]] = start || m_kept[y] == m_ref[y] ? 1.0f : tc::ex2(m_kept[y] - m_ref[y]);
                        named_sync(2, kSoft);
                        for (int i = kBlocks * set; i < kBlocks * (set + 1); ++i) {
                            float *kept = p.part_o + part0 * kLatent + 128 * i + 32 * quarter + lane;
                            fold_o(kept, tmem + lanes + i * geo.npad, geo.npad, sm.factor, start, js >= w.j1);
                        }
#pragma unroll
                        for (int y = 0; y < kR; ++y) {
                            m_kept[y] = m_ref[y];
                            l_kept[y] = l_kept[y] * sm.factor[r[y]] + l[y];
                            l[y] = js >= w.j1 ? l_kept[y] : 0.f;
                        }
                    }
                    if (js >= w.j1) break;
                    const int je = min(w.j1, js + kFold);
                    for (int j = js; j < je; ++j) {
                        const bool first = j == w.j0;
                        const int rem = w.len - j * kKvTile;             // cached rows of the sequence from this tile on
                        float sc[kC];                                    // the rows' scales,
                        uint64_t x2[kR][kC / 2];                         // the scores as powers of two, by pairs of cached rows,
                        uint32_t w16[kR][kC / 2];                        // and the weights in fp16
                        auto scales = [&] {
#pragma unroll
                            for (int e = 0; e < kC; e += 2) *reinterpret_cast<float2 *>(&sc[e]) = *reinterpret_cast<const float2 *>(&sm.sc[k % kScales][col(e)]);
                        };
                        ok = wait_peeked(s_there, &sm.s_full[k & 1], (k >> 1) & 1) && ok;
                        // a failed wait still meets the barriers below, so that no warp is left in them
                        if (ok) tc::fence_after_sync();
                        scales();
                        const uint32_t s_at = t_s + lanes + (k & 1) * kKvTile + set * kSetCols;
                        const bool live = warp_rows && ok;
                        float sum[kR], most[kR], mass[kR];               // of a row's weights here: without scales, the largest, the sum
                        // (scores are rounded before a reference is taken off, so that huge ones still differ by 0 from themselves)
                        auto scores = [&] {
                            if constexpr (FORM == 2) {
                                uint32_t x[kC];
                                tc::tmem_ld32_nowait(s_at, x);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < kC / 2; ++e) x2[0][e] = pk2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
                            } else if constexpr (FORM == 1) {
                                uint32_t hi[2 * kC], lo[2 * kC];
                                tmem_ld_fragments(s_at, hi);
                                tmem_ld_fragments(s_at + (16u << 16), lo);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < kC; ++e)
                                    x2[e & 1][e >> 1] = add2(pk2(__uint_as_float(hi[2 * e]), __uint_as_float(hi[2 * e + 1])),
                                                             pk2(__uint_as_float(lo[2 * e]), __uint_as_float(lo[2 * e + 1])));
                            } else {
                                uint32_t x[2 * kC];
                                tmem_ld_fragments(s_at, x);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < kC / 2; ++e)
                                    x2[0][e] = add2(pk2(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1])),
                                                    pk2(__uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3])));
                            }
                            tc::fence_before_sync();
#pragma unroll
                            for (int y = 0; y < kR; ++y)
#pragma unroll
                                for (int e = 0; e < kC / 2; ++e)
                                    x2[y][e] = mul2(mul2(x2[y][e], pk2(sc[2 * e], sc[2 * e + 1])), pk2(c[y], c[y]));
                            if (rem - (p.m - 1) < kKvTile) {  // a tile of which not every row sees all
#pragma unroll
                                for (int y = 0; y < kR; ++y) {
                                    const int seen = rem - unseen[y];
#pragma unroll
                                    for (int e = 0; e < kC / 2; ++e) {
                                        const float2 x = upk2(x2[y][e]);
                                        x2[y][e] = pk2(col(2 * e) >= seen ? -INFINITY : x.x, col(2 * e + 1) >= seen ? -INFINITY : x.y);
                                    }
                                }
                                // scales behind the sequence count as one: 0 times what stands there may be NaN
#pragma unroll
                                for (int e = 0; e < kC; ++e)
                                    if (col(e) >= rem) sc[e] = 1.f;
                            }
                        };
                        auto weights = [&] {
#pragma unroll
                            for (int y = 0; y < kR; ++y) {
                                const float mb = m_ref[y] == -INFINITY ? 0.f : -m_ref[y];
                                const uint64_t mb2 = pk2(mb, mb);
                                uint64_t l2[2] = {0, 0};
                                uint32_t top = 0, all = 0;
#pragma unroll
                                for (int e = 0; e < kC / 2; ++e) {
                                    const float2 x = upk2(add2(x2[y][e], mb2));
                                    const uint64_t pp = pk2(tc::ex2(x.x), tc::ex2(x.y));
                                    l2[e & 1] = add2(l2[e & 1], pp);
                                    const float2 ww = upk2(mul2(pp, pk2(sc[2 * e], sc[2 * e + 1])));
                                    w16[y][e] = half2_of(ww.x, ww.y);
                                    top = max_half2(top, w16[y][e]);
                                    all = add_half2(all, w16[y][e]);
                                }
                                const float2 ls = upk2(add2(l2[0], l2[1]));
                                sum[y] = ls.x + ls.y;
                                const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&top));
                                most[y] = fmaxf(t.x, t.y);
                                const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&all));
                                mass[y] = a.x + a.y;
                            }
                        };
#pragma unroll
                        for (int y = 0; y < kR; ++y) sum[y] = most[y] = mass[y] = 0.f;
                        if (live && !first) {
                            scores();
                            weights();
                        }
                        // one barrier a tile: does a row need a new reference, did a wait fail
                        bool may = first || !ok;
#pragma unroll
                        for (int y = 0; y < kR; ++y) may |= faint[y] || most[y] > limit[y];
                        const bool any = softmax_any<kSoft>(may);
                        bool again = false, anew[kR];
#pragma unroll
                        for (int y = 0; y < kR; ++y) anew[y] = false;
                        if (any) {
                            if (k > 0) ok = through(k - 1) && ok;
                            // the largest exponent of a weight in this tile, over a row's threads
                            float top[kR];
                            scales();
                            if (live) scores();
#pragma unroll
                            for (int y = 0; y < kR; ++y) {
                                top[y] = -INFINITY;
                                if (live) {
                                    auto of_scale = [&](int e) { return (float)((int)(__float_as_uint(sc[e]) >> 23) - 127); };  // its exponent
                                    const float early = j == 0 && set == 0 ? kEarly : 0.f;
#pragma unroll
                                    for (int e = 0; e < kC / 2; ++e) {
                                        const float2 x = upk2(x2[y][e]);
                                        float t = fmaxf(x.x + of_scale(2 * e), x.y + of_scale(2 * e + 1));
                                        if (2 * e < (kStack ? kEarlyRows / 4 : kEarlyRows)) t -= early;
                                        top[y] = fmaxf(top[y], t);
                                    }
                                }
                                if constexpr (kStack) {
                                    top[y] = fmaxf(top[y], __shfl_xor_sync(0xffffffffu, top[y], 1));
                                    top[y] = fmaxf(top[y], __shfl_xor_sync(0xffffffffu, top[y], 2));
                                }
                                if (lead) sm.part[set][r[y]] = top[y];
                            }
                            // all stop together when any wait failed
                            if (softmax_any<kSoft>(!ok)) {
                                ok = false;
                                stopped = true;
                                break;
                            }
                            again = false;
#pragma unroll
                            for (int y = 0; y < kR; ++y) {
                                top[y] = fmaxf(sm.part[0][r[y]], sm.part[1][r[y]]);
                                m_top[y] = fmaxf(m_top[y], top[y]);
                                const bool up = first || top[y] - m_ref[y] > kHigh;
                                // of low weights, the window's sum, which is still in sm.recent
                                const float lately = window(r[y]), low = lately < kNothing ? -INFINITY : m_ref[y] + __log2f(lately) - kSetLow;
                                const float to = fmaxf(up ? top[y] - (first ? kSet : kSetHigh) : fmaxf(top[y] - kSet, low), m_top[y] - kReach);
                                anew[y] = up || (faint[y] && to < m_ref[y]);
                                const float f = anew[y] && !first ? tc::ex2(m_ref[y] - to) : 1.0f;
                                if (set == 0 && lead) sm.factor[r[y]] = f;
                                if (anew[y]) m_ref[y] = to;
                                if (anew[y]) recent[y] = 0.f;
                                // A row that has seen nothing yet looks again. Not one with a NaN in it, which never sees anything
                                // and would take all rows of the block through this in every tile (1.4 to 1.5 times the time).
                                faint[y] = owner[y] && m_ref[y] == -INFINITY && c[y] == c[y];
                                l[y] *= f;
                                again |= owner[y] && anew[y] && !first;
                            }
                            if (softmax_any<kSoft>(again)) {
                                tc::fence_after_sync();
                                for (int e = 0; e < geo.npad; e += 16) {
                                    float fs[16];
                                    bool same = true;
#pragma unroll
                                    for (int y = 0; y < 16; ++y) fs[y] = sm.factor[e + y], same &= fs[y] == 1.0f;
                                    if (same) continue;
                                    for (int i = kBlocks * set; i < kBlocks * (set + 1); ++i) {
                                        const uint32_t at = tmem + lanes + i * geo.npad + e;
                                        uint32_t x[16];
                                        tma::tmem_ld16_nowait(at, x);
                                        tc::tmem_wait_ld();
#pragma unroll
                                        for (int y = 0; y < 16; ++y) x[y] = __float_as_uint(__uint_as_float(x[y]) * fs[y]);
                                        tc::tmem_st16(at, x);
                                    }
                                }
                                tc::tmem_wait_st();
                            }
                            if (live) weights();
                        }
                        tma::arrive_warp(&sm.s_free[k & 1]);
                        if (live) {
#pragma unroll
                            for (int y = 0; y < kR; ++y) {
                                if (r[y] >= geo.npad) continue;
                                const uint32_t a = w_at[y] + (k & 1) * p_bytes, b = a + w_16[y], a_lo = a + w_64[y], b_lo = b + w_64[y];
                                if constexpr (kStack) {
#pragma unroll
                                    for (int e = 0; e < kC / 2; ++e) {
                                        uint16_t hi, lo;
                                        split_weights(w16[y][e], hi, lo);
                                        store2(e < 2 ? a : b, 8 * (e & 1), hi);
                                        store2(e < 2 ? a_lo : b_lo, 8 * (e & 1), lo);
                                    }
                                } else {
#pragma unroll
                                    for (int u = 0; u < kC / 16; ++u) {
                                        uint32_t hi[4], lo[4];
#pragma unroll
                                        for (int e = 0; e < 4; ++e) {
                                            uint16_t q[4];
                                            split_weights(w16[y][8 * u + 2 * e], q[0], q[1]);
                                            split_weights(w16[y][8 * u + 2 * e + 1], q[2], q[3]);
                                            asm("mov.b32 %0, {%1, %2};" : "=r"(hi[e]) : "h"(q[0]), "h"(q[2]));
                                            asm("mov.b32 %0, {%1, %2};" : "=r"(lo[e]) : "h"(q[1]), "h"(q[3]));
                                        }
                                        store16(u ? b : a, hi);
                                        store16(u ? b_lo : a_lo, lo);
                                    }
                                }
                            }
                        }
                        if (rem < kKvTile && (rem & 31)) {  // value rows behind the sequence in the product's last step of 32
                            const int units = (-rem & 31) * 8;
                            for (int u = tid; u < (kChunks - 1) * units; u += kSoft)
                                reinterpret_cast<uint4 *>(s_ring + k % kTiles * kTile8 + u / units * kChunk8)[rem * 8 + u % units] =
                                    make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async();
                        tc::fence_before_sync();
                        tma::arrive_warp(&sm.p_full[k & 1]);
                        s_there = peek(&sm.s_full[(k + 1) & 1], ((k + 1) >> 1) & 1);
                        // low weights: a window's sum is left in shared memory behind its last tile, and looked at behind the next
                        const int of_window = (j - w.j0) & (kWindow - 1);
#pragma unroll
                        for (int y = 0; y < kR; ++y) {
                            l[y] += sum[y];
                            recent[y] += mass[y];
                            if (of_window == kWindow - 1) {
                                if constexpr (kStack) {
                                    recent[y] += __shfl_xor_sync(0xffffffffu, recent[y], 1);
                                    recent[y] += __shfl_xor_sync(0xffffffffu, recent[y], 2);
                                }
                                if (lead) sm.recent[set][r[y]] = recent[y];
                                recent[y] = 0.f;
                            } else if (of_window == 0 && !first && !anew[y]) {  // (a new reference was set by weights that are not low)
                                faint[y] |= owner[y] && window(r[y]) < kLeast && m_ref[y] > m_top[y] - kReach;
                            }
                        }
                        ++k;
                    }
                }
                // the next stretch's queries before this one's output, so that its scores start meanwhile
                if (softmax_any<kSoft>(!ok)) ok = false;
                if (ok && next_n >= 0) load_q(next_n);
                if (ok) ok = through(k - 1);
                tc::fence_after_sync();
            }
#pragma unroll
            for (int y = 0; y < kR; ++y) {
                if constexpr (kStack) {
                    l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
                    l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
                }
                if (lead) sm.part[set][r[y]] = l[y];
            }
            if (softmax_any<kSoft>(!ok)) ok = false;
#pragma unroll
            for (int y = 0; y < kR; ++y) l[y] = sm.part[0][r[y]] + sm.part[1][r[y]];
            // ---- this stretch's part of the sequence: finished, or left for the join ----
            const bool whole = w.j0 == 0 && w.j1 == w.tiles;
            const bool bad = !ok || bad_len(p, w.len) || (w.work && *(volatile int32_t *)&sm.bad[seg % kBad] != 0);
            if (bad_len(p, w.len) && tid == 0) set_status(p.status, KDA_ERR_SEQLENS);
            const int64_t row0 = (int64_t)w.n * geo.R + row_first;
#pragma unroll
            for (int y = 0; y < kR; ++y) {
                if (set != 0 || !lead) continue;
                sm.factor[r[y]] = bad ? NAN : (l[y] == 0.f ? 0.f : 1.0f / l[y]);
                if (owner[y]) {
                    if (!whole)
                        p.part_ml[part0 + r[y]] = make_float2(m_ref[y], bad ? NAN : l[y]);
                    else if (p.lse)
                        p.lse[row0 + r[y]] = bad ? NAN : (l[y] == 0.f ? -INFINITY : m_ref[y] * p.scale + logf(l[y]));
                }
            }
            named_sync(2, kSoft);
            for (int i = kBlocks * set; i < kBlocks * (set + 1); ++i) {
                const int lat = 128 * i + 32 * quarter + lane;
                for (int e0 = 0; e0 < rows_here; e0 += 32) {
                    uint32_t x[2][16];
                    const bool two = e0 + 16 < geo.npad;
                    if (w.work && ok) {
                        tma::tmem_ld16_nowait(tmem + lanes + i * geo.npad + e0, x[0]);
                        if (two) tma::tmem_ld16_nowait(tmem + lanes + i * geo.npad + e0 + 16, x[1]);
                        tc::tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int y = 0; y < 16; ++y) x[0][y] = x[1][y] = 0;
                    }
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int e = e0 + 16 * z;
                        if (z && !two) break;
                        if (whole) {
                            // neighbouring lanes trade a value: each then holds two latents of one row
                            __nv_bfloat16 *dst = p.o + (row0 + e + (lane & 1)) * kLatent + (lat & ~1);
                            const int left = rows_here - e - (lane & 1);
#pragma unroll
                            for (int y = 0; y < 16; y += 2) {
                                const float2 f = *reinterpret_cast<const float2 *>(&sm.factor[e + y]);
                                const __nv_bfloat162 h2 =
                                    __floats2bfloat162_rn(__uint_as_float(x[z][y]) * f.x, __uint_as_float(x[z][y + 1]) * f.y);
                                const uint32_t own = *reinterpret_cast<const uint32_t *>(&h2);
                                const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
                                const uint32_t two_lat = (lane & 1) ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
                                if (y < left) *reinterpret_cast<uint32_t *>(dst + y * kLatent) = two_lat;
                            }
                        } else {  // rows past the last are written too (their columns of O^T are nobody's): parts are npad rows
                            float *dst = p.part_o + (part0 + e) * kLatent + lat;
#pragma unroll
                            for (int y = 0; y < 16; ++y) dst[y * kLatent] = __uint_as_float(x[z][y]);
                        }
                    }
                }
            }
            // O^T has been read: the next stretch's W (all threads arrive) lets the MMA warp write it
            tc::fence_before_sync();
            named_sync(2, kSoft);
            if (w.work) ++seg;
        }
        if (!ok) sm.failed = 1;
    }
    tc::fence_before_sync();
    __syncthreads();
    if (sm.failed && (warp == kIssue || warp == kIssue + 1)) {
        // a wait gave up: report it, and let what is in flight land before the memory goes
        if (tma::elect()) {
            tc::commit(&sm.drained);  // each issuing thread's own products
            if (warp == kIssue) {
                set_status(p.status, KDA_ERR_CUDA);
                tc::mbar_wait(&sm.drained, 0);
                for (int e = max(0, sm.scaled - kScales); e < sm.scaled; ++e) tc::mbar_wait(&sm.sc_full[e % kScales], (e / kScales) & 1);
                for (int e = max(0, sm.issued - kTiles * kPieces); e < sm.issued; ++e)
                    tc::mbar_wait(&sm.full[e % (kTiles * kPieces)], (e / kPieces / kTiles) & 1);
            }
        }
        __syncwarp();
    }
    if (warp == kIssue) tc::tmem_dealloc(tmem, 512);
}

constexpr size_t kSmem8 = 232448;

// Row tiles of equal size, as few as 96 rows each allow, or as few as 64 allow, where these are not more than a third
// more. With tiles of up to 96 and up to 64 rows 64 sequences of up to 8000 rows take 82 and 93 us (96
// rows, 1 and 2 tiles), 131 and 139 (192, 2 and 3), 171 and 169 (200, 3 and 4), 184 and 171 (256, 3 and 4), 189 and 210
// (288, 3 and 5), 216 and 210 (320, 4 and 5), 231 and 248 (384, 4 and 6), 320 and 308 (512, 6 and 8), 426 and 479 (768, 8
// and 12).
// Where the tables hold so little (`most` tiles) that a block has no more than 24 tiles of 32 rows, or 16 of 64, row tiles of
// these: a block then has fewer queries to split and less to write, which counts for more than reading the tiles more
// often. With up to 96, 64 and 32 rows: 96 heads over 500 rows 15.3, - and 10.3 us, 12000 23.9, 18.0 and 16.4, 50000 33.1, 30.3
// and 28.2 (16 tiles), 80000 39.5, 37.4 and 36.6, 120000 47.2, 48.1 and 48.7; 96 x 4 over 20000 35.7, 33.3 (12 tiles) and
// 36.5; 20 x 96 over 3000 38.0, 35.9 and 34.7. (With fewer than three groups of so many tiles too many SMs would have none.)
Geom8 geometry8(int32_t H, int32_t m, int64_t most, int32_t sms) {
    Geom8 q{};
    q.R = H * m;
    q.RT = (q.R + kMostRows8 - 1) / kMostRows8;
    const int32_t narrow = (q.R + kRows8 - 1) / kRows8;
    if (3 * (int64_t)narrow <= 4 * (int64_t)q.RT) q.RT = narrow;
    const int32_t least = (q.R + 31) / 32;
    if (least <= sms / 3 && most * least <= 24 * sms)
        q.RT = least;
    else if (narrow <= sms / 3 && most * narrow <= 16 * sms)
        q.RT = narrow;
    q.rows = ((q.R + q.RT - 1) / q.RT + 7) / 8 * 8;
    q.npad = (q.rows + 15) / 16 * 16;
    q.form = q.rows <= 32 ? 0 : (q.rows <= kRows8 ? 1 : 2);
    const size_t of_q = q.form == 2 ? (size_t)9 * q.rows * 128 : (size_t)(q.form == 0 ? 5 * 64 : 5 * 128) * 128;
    q.smem = (uint32_t)(1024 + sizeof(Smem8) + of_q + (size_t)q.npad * 256 + (size_t)tiles_in(q.form) * kTile8);
    return q;
}
static_assert(1024 + sizeof(Smem8) + 5 * 64 * 128 + 32 * 256 + tiles_in(0) * kTile8 <= kSmem8, "32 rows");
static_assert(1024 + sizeof(Smem8) + 5 * 128 * 128 + 64 * 256 + tiles_in(1) * kTile8 <= kSmem8, "64 rows");
static_assert(1024 + sizeof(Smem8) + 11 * kMostRows8 * 128 + tiles_in(2) * kTile8 <= kSmem8, "96 rows");
static_assert(tiles_in(0) <= kMaxSlots && kMaxSlots + 2 < kScales && tiles_in(2) * pieces_of(2) <= kMaxPieces, "");
static_assert(offsetof(Smem8, sc) % 16 == 0 && kTile8 % 1024 == 0, "bulk copies");
static_assert(kMaxSlots + 2 < kBad, "the loads are fewer stretches ahead than flags are kept");

// The workspace of a call, whatever its page tables hold: row tiles chosen by them are narrower than these, and all groups'
// row tiles are kMaxGroups at most in both.
SplitWs workspace8(int32_t H, int32_t m) { return split_ws(geometry8(H, m, INT32_MAX, 0), kMostRows8); }

// What a sequence costs beside its tiles, in tiles: its queries are split and its output written. (With 0, 0, 0 / 3, 4, 6
// / 4, 6, 8 units: 32 sequences x 16 heads 31.5 / 26.2 / 26.2 us, 64 x 48 71 / 61.4 / 61.3, 64 x 96, four tokens 243 /
// 226.5 / 226, 256 x 96 303 / 256 / 255.)
int32_t extra8(int form) { return form == 0 ? 4 : (form == 1 ? 6 : 8); }

}  // namespace
}  // namespace kda

extern "C" {

size_t kda_mla_decode_fp8_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t num_tokens) {
    if (num_seqs < 0 || num_heads < 0 || num_tokens < 0) return 0;
    if ((int64_t)num_heads * num_tokens > INT32_MAX / 2 || num_heads == 0 || num_tokens == 0) return 256;
    return kda::workspace8(num_heads, num_tokens).total;
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
    int sms = 0, device = 0;
    rc = device_sms(&sms, &device);
    if (rc != KDA_OK) return rc;
    if (device >= 64) return KDA_ERR_DEVICE;

    Args8 a;
    // the longest page tables' tiles; no more groups than these
    const int64_t most = (int64_t)num_seqs * (((int64_t)max_pages * page_size + kKvTile - 1) / kKvTile + 1);
    a.geo = geometry8(num_heads, num_tokens, most, sms);
    a.split = a.geo;
    a.extra = extra8(a.geo.form);
    const SplitWs w = workspace8(num_heads, num_tokens);
    a.rb = page_size % 64 == 0 ? 64 : (page_size % 32 == 0 ? 32 : 16);
    // a cache without pages keeps one page of extent: no id is in range, every load is past it
    // the chunks of a row are a dimension of their own, outside the rows: a box of all of them lands chunk by chunk
    const uint64_t dc[4] = {128, (uint64_t)page_size, kChunks, (uint64_t)(num_pages > 0 ? num_pages : 1)};
    const uint64_t sc[4] = {1, (uint64_t)kRow8, 128, (uint64_t)page_stride};
    if (!tma::encode_bytes(&a.map, cache, dc, sc, a.rb, a.rb == kKvTile && pieces_of(a.geo.form) == 1 ? kChunks : 1)) return KDA_ERR_CUDA;
    a.q_lat = reinterpret_cast<const __nv_bfloat16 *>(q_lat);
    a.q_pe = reinterpret_cast<const __nv_bfloat16 *>(q_pe);
    a.rows = cache;
    a.page_stride = page_stride;
    a.table = page_table;
    a.lens = cache_lens;
    a.max_pages = max_pages;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.N = num_seqs;
    a.H = num_heads;
    a.m = num_tokens;
    a.c = scale * 1.4426950408889634f;
    a.scale = 0.6931471805599453f;  // the maxima count in powers of two
    a.o = reinterpret_cast<__nv_bfloat16 *>(o);
    a.lse = lse;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.head = reinterpret_cast<int64_t *>(ws + w.head);
    a.part_ml = reinterpret_cast<float2 *>(ws + w.ml);
    a.part_o = reinterpret_cast<float *>(ws + w.o);
    a.status = status;
    static std::atomic<bool> configured[64];  // the kernels' shared memory, set once a device
    if (!configured[device].load(std::memory_order_acquire)) {
        for (auto kernel : {kda_mla_decode_fp8_kernel<0>, kda_mla_decode_fp8_kernel<1>, kda_mla_decode_fp8_kernel<2>})
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem8) != cudaSuccess)
                return KDA_ERR_CUDA;
        configured[device].store(true, std::memory_order_release);
    }
    a.G = groups_of(a.geo.RT, sms < kMaxGroups ? sms : kMaxGroups);
    if (a.G > most) a.G = (int32_t)most;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto kernel = a.geo.form == 0 ? kda_mla_decode_fp8_kernel<0> : (a.geo.form == 1 ? kda_mla_decode_fp8_kernel<1> : kda_mla_decode_fp8_kernel<2>);
    if (launch_after(kernel, dim3((unsigned)(a.G * a.geo.RT)), dim3(kThreads), a.geo.smem, st, a) != cudaSuccess ||
        join_parts(a, st) != cudaSuccess)
        return KDA_ERR_CUDA;
    return KDA_OK;
}

}  // extern "C"
