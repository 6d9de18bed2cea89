// Latent attention in the expanded form: kda_mla_prefill.
//
//   s_ij = scale (q_i . k_j),  o_i = sum_j e^{s_ij - M_i} v_j / sum_j e^{s_ij - M_i},
//   lse_i = M_i + log sum_j e^{s_ij - M_i}
//
// with k_j = (k_nope_j, k_pe_j) of 64-column chunks, the first two a head's own and the third
// shared by the heads, so the positional key is never copied per head. One pass over the keys
// with a running maximum and sum.
//
// A CTA takes 256 query rows of one head as two tiles of 128 and walks the keys in tiles of
// 128. Per key tile and query tile the tensor core forms S = Q K^T (128 x 128 x 192, fp32 in
// TMEM); the tile's four warps, one thread a row, turn S into P = 2^{c s - c M} (bf16, written
// over S in TMEM) and the tensor core adds P V (128 x 128 x 128) to O in TMEM. While one tile's
// warps are at their exponentials the tensor core works for the other: its order is PV0(j)
// S0(j+1) PV1(j) S1(j+1). TMEM holds exactly S0 S1 O0 O1 (4 x 128 columns). P is handed over in
// parts of 32 keys, so that P V starts while the rest is at its exponentials.
//
// The grid has a block per 256 rows and head, a sequence's rows with the most keys first. One block fits an
// SM; when its loads come to their end it takes over one that has not started and loads for it
// while the last products and the output still run: the first scores of the next item are issued
// before the last value product of this one. Against blocks that start one after another (8192 new
// tokens x 12 heads, causal; five ragged sequences x 32 heads): 167 and 160 us against 173.6 and 177.5.
// These are times of ten calls replayed from a graph; in a long row of calls, at the clocks that the power
// limit then leaves, the first two take 177 and 167 us.
//
// Bounds: 2 x 1280 cycles of tensor work a key tile at 8192 flop a cycle, and 32 K exponentials,
// 2048 cycles at 16 a cycle. A key tile takes about 3200 cycles: S to P and back is a chain of
// 2000 that the other tile's products cover but for their own waits. 8192 x 12 runs at
// 1.54 PFLOP/s (1.45 in a long row); the ragged case, whose tiles do 19% more than its rows need and
// whose last items end apart, at 1.13 (1.09). Measured and not taken: two threads a row (176 and 169 us,
// more handing over), part of the exponentials as polynomials on the FMA pipe (183 us with an eighth of
// them, 190 with a quarter), a reference that follows the maximum only where 32 weights sum to more than
// 2^24 (167 and 155.5, but 272 us instead of 196 where scores spread by 9). 16384 tokens x 16 heads run at
// 1.77 PFLOP/s.
//
// P is rounded to bf16 for the value product, which takes 16-bit operands (two of them a weight would
// double it); the sum of the weights is that of the fp32 values.
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since its last reference
// (P stays below 2^8, far inside bf16 and fp32), which few tiles do; l sums the fp32 values, a key
// tile's for themselves first, so that small weights behind a large one are not lost.
//
// The tensor core drops what falls below an accumulator's last bit, always towards zero, so a sum over
// n keys comes out low by about n / 16 * 0.7 * 2^-23 of itself: 0.5% at a million keys, 17% at 33 million.
// O therefore sums 512 key tiles at a time (4096 additions, 2^-11 at most); then its row is added to
// one in local memory, with roundings to nearest, and so is l, whose roundings go one way too where tiles
// are alike. That row is touched behind 65536 keys only.
//
// Shared memory: Q 96 KB, K in a ring of four 16 KB chunks (one key tile and the next tile's
// first chunk), V in a ring of two 32 KB tiles. Rows of a tile that lie behind the sequence
// may hold anything: their scores are replaced by -inf, and their value rows are zeroed in
// shared memory before the product (0 x NaN would reach the sums).

#include "kda_common.cuh"
#include "kda_latent_common.cuh"
#include "kda_tma.cuh"

namespace kda {
namespace {

constexpr int kTileQ = 128, kTileK = 128;
constexpr int kRowsCta = 2 * kTileQ;
constexpr uint32_t kChunk = 128 * 128;  // bytes of a 128-row chunk
constexpr int kKSlots = 4, kVSlots = 2;
constexpr int kThreads = 352;  // 2 x 4 softmax warps, the MMA warp, the TMA warp, the scheduler
constexpr float kRescale = 8.0f;
constexpr int kParts = 4;     // P of a key tile is handed over in parts of 32 keys
constexpr int kFold = 512;    // key tiles that O sums in tensor memory (a power of two)
constexpr int kAskAhead = 4;  // key tiles before an item's last whose loads ask for the next item

struct PrefillArgs {
    CUtensorMap q, kv, pe;
    const int32_t *cu_q, *cu_k;
    int64_t Tq, Tk;
    int32_t N, H, causal;
    float scale;
    __nv_bfloat16 *o;
    int32_t o_sectors;  // o is 32-byte aligned
    float *lse;
    int32_t *status;
};

// A CTA's piece of work: 256 query rows of one head of one sequence.
struct Item {
    int32_t q0, nq, k0, nk;  // the sequence's first row and rows, of queries and of keys
    int32_t row0;            // first query row within the sequence
    int32_t h;               // head; -1: no more items
    int32_t nt0, nt1;        // key tiles of each query tile
};

struct PrefillSmem {
    uint8_t q[2][3][kChunk];
    uint8_t k[kKSlots][kChunk];
    uint8_t v[kVSlots][2][kChunk];
    uint4 canceled;  // the answer of a request for a CTA that has not started
    Item item[2];
    uint64_t item_full[2], item_empty[2], ask, cancel_full;
    uint64_t q_full[2], q_empty[2], k_full[kKSlots], k_empty[kKSlots], v_full[kVSlots], v_empty[kVSlots];
    uint64_t s_full[2], p_full[2][kParts], pv_done[2], drained;
    uint32_t tmem;
    int32_t failed;
    int32_t k_issued, v_issued, q_issued[2];  // loads the producer started (read after a failed wait only)
};

// keys that query row r of a sequence sees
__device__ __forceinline__ int keys_of(const Item &w, int causal, int r) {
    return max(0, causal ? min(w.nk, r + w.nk - w.nq + 1) : w.nk);
}

// key tiles of the query tile that starts at row `first`
__device__ __forceinline__ int key_tiles(const Item &w, int causal, int first) {
    const int last = first + min(w.nq - first, kTileQ) - 1;
    return last < first ? 0 : (int)(((int64_t)keys_of(w, causal, last) + kTileK - 1) / kTileK);
}

// Where the last item was found: 32 sequences from n0 on, with `before` tiles before them, whose query rows
// end at `top`. The blocks that a block takes over come mostly in rising order, so that it reads the list of
// sequences about once.
struct Place {
    int32_t n0, top;
    int64_t before;
};

// The item of a slot, by a whole warp: slots are (tile, head) pairs, heads fastest, a sequence's tiles from
// the last one (it sees the most keys) to the first. False for a slot past the last tile.
__device__ __forceinline__ bool find_item(const PrefillArgs &p, int64_t index, Place &at, Item &w) {
    const int lane = threadIdx.x & 31;
    const int64_t slot = index / p.H;
    if (slot < at.before) at = {0, 0, 0};
    for (; at.n0 < p.N; at.n0 += 32) {
        const int n0 = at.n0;
        const int64_t before = at.before;
        const int n = n0 + lane;
        int a = 0, b = 0, c = 0, d = 0;
        int64_t tiles = 0;
        bool sound = true;
        if (n < p.N) {
            a = p.cu_q[n], b = p.cu_q[n + 1], c = p.cu_k[n], d = p.cu_k[n + 1];
            sound = a >= 0 && b <= p.Tq && b >= a && c >= 0 && d <= p.Tk && d >= c;
        }
        // where the rows of the sequences before end. Behind offsets that fell a sequence may begin before that:
        // its rows would be written twice, and the batch have more tiles than the grid has blocks
        const int32_t end = n < p.N && sound ? b : 0;
        int32_t top = at.top;
        if (__any_sync(0xffffffffu, !sound)) {
            int32_t most = end;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int32_t x = __shfl_up_sync(0xffffffffu, most, off);
                if (lane >= off) most = max(most, x);
            }
            most = __shfl_up_sync(0xffffffffu, most, 1);
            if (lane > 0) top = max(top, most);
        }
        if (n < p.N) {
            if (!sound || a < top)
                set_status(p.status, KDA_ERR_SEQLENS);  // every CTA that looks finds it: no tiles
            else
                tiles = ((int64_t)b - a + kRowsCta - 1) / kRowsCta;
        }
        int64_t incl = tiles;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += x;
        }
        const int64_t lo = before + incl - tiles;
        const unsigned mine = __ballot_sync(0xffffffffu, slot >= lo && slot < lo + tiles);
        if (mine) {
            const int src = __ffs(mine) - 1;
            const int tile = (int)(__shfl_sync(0xffffffffu, tiles, src) - 1 - (slot - __shfl_sync(0xffffffffu, lo, src)));
            w.q0 = __shfl_sync(0xffffffffu, a, src);
            w.nq = __shfl_sync(0xffffffffu, b, src) - w.q0;
            w.k0 = __shfl_sync(0xffffffffu, c, src);
            w.nk = __shfl_sync(0xffffffffu, d, src) - w.k0;
            w.row0 = tile * kRowsCta;
            w.h = (int)(index - slot * p.H);
            w.nt0 = key_tiles(w, p.causal, w.row0);
            w.nt1 = key_tiles(w, p.causal, w.row0 + kTileQ);
            return true;
        }
        at.before += __shfl_sync(0xffffffffu, incl, 31);
        at.top = max(at.top, __reduce_max_sync(0xffffffffu, end));
    }
    return false;
}

// scores from `valid` on are hidden
__device__ __forceinline__ void hide(uint32_t (&r)[32], int valid) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (i >= valid) r[i] = 0xff800000u;
}

// max of 32 scores
__device__ __forceinline__ float max32(const uint32_t (&r)[32], float m) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) m = fmaxf(m, fmaxf(__uint_as_float(r[i]), __uint_as_float(r[i + 1])));
    return m;
}

// 32 scores to probabilities 2^{s c - mb}: packed to bf16 pairs, their fp32 values added to l
__device__ __forceinline__ void exp32(const uint32_t (&r)[32], uint32_t (&p)[16], uint64_t c2, uint64_t nmb2, uint64_t (&l)[2]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float2 x = upk2(fma2(pk2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), c2, nmb2));
        const float a = tc::ex2(x.x), b = tc::ex2(x.y);
        l[i & 1] = add2(l[i & 1], pk2(a, b));
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        p[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
}

// kept (+)= O and the denominator l of this thread's row, at their reference m_ref; for the output (back) into
// O instead. Behind kept's values of O stand its reference and its denominator; returns that. A call of its
// own: in the loop's code it made every tile slower (8192 x 12 170.5 us, 168.5 so).
constexpr int kKept = kNope + 2;
__device__ __noinline__ float fold_o(float *kept, uint32_t o_addr, float l, float m_ref, float c, bool first, bool back) {
    const float f = first || kept[kNope] == m_ref ? 1.0f : tc::ex2((kept[kNope] - m_ref) * c);
#pragma unroll 1
    for (int i = 0; i < kNope / 16; ++i) {
        uint32_t x[16];
        tma::tmem_ld16_nowait(o_addr + 16 * i, x);
        tc::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float y = __uint_as_float(x[k]) + (first ? 0.f : kept[16 * i + k] * f);
            kept[16 * i + k] = y;
            x[k] = __float_as_uint(y);
        }
        if (back) tc::tmem_st16(o_addr + 16 * i, x);
    }
    if (back) tc::tmem_wait_st();
    kept[kNope] = m_ref;
    return kept[kNope + 1] = l + (first ? 0.f : kept[kNope + 1] * f);
}

__global__ void __launch_bounds__(kThreads, 1) kda_mla_prefill_kernel(const __grid_constant__ PrefillArgs p) {
    extern __shared__ uint8_t smem_raw[];
    PrefillSmem &sm = *reinterpret_cast<PrefillSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == 9 && lane == 0) {
        tma::prefetch_map(&p.q);
        tma::prefetch_map(&p.kv);
        tma::prefetch_map(&p.pe);
        sm.failed = 0;
        sm.k_issued = sm.v_issued = sm.q_issued[0] = sm.q_issued[1] = 0;
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sm.item_full[i], 1);
            tc::mbar_init(&sm.item_empty[i], 2 + 2 * kTileQ / 32);
            tc::mbar_init(&sm.q_full[i], 1);
            tc::mbar_init(&sm.q_empty[i], 1);
            tc::mbar_init(&sm.s_full[i], 1);
            for (int k = 0; k < kParts; ++k) tc::mbar_init(&sm.p_full[i][k], kTileQ / 32);
            tc::mbar_init(&sm.pv_done[i], 1);
        }
        tc::mbar_init(&sm.ask, 1);
        tc::mbar_init(&sm.cancel_full, 1);
        for (int i = 0; i < kKSlots; ++i) tc::mbar_init(&sm.k_full[i], 1), tc::mbar_init(&sm.k_empty[i], 1);
        for (int i = 0; i < kVSlots; ++i) tc::mbar_init(&sm.v_full[i], 1), tc::mbar_init(&sm.v_empty[i], 1);
        tc::mbar_init(&sm.drained, 1);
        tc::mbar_init_fence();
    }
    if (warp == 8) tc::tmem_alloc(&sm.tmem, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    pdl_wait();
    const uint32_t tmem = sm.tmem;
    bool ok = true;
    // A wait that may last as long as another query tile or role works on an item (10^8 keys take more than a
    // wait's limit): the limit counts from the last load that the item was seen to make
    auto wait_while_loading = [&](uint64_t *mbar, uint32_t parity) {
        auto loads = [&] { return __shfl_sync(0xffffffffu, *(volatile int32_t *)&sm.k_issued, 0); };
        int seen;
        bool got;
        do {
            seen = loads();
            got = tma::wait_warp(mbar, parity);
        } while (!got && loads() != seen);
        return got;
    };

    if (warp == 9) {
        // ---- TMA producer: one thread ----
        if (tma::elect()) {
            int ke = 0, ve = 0, qe[2] = {0, 0};  // loads so far
            for (int n = 0; ok; ++n) {
                ok = tc::mbar_wait(&sm.item_full[n & 1], (n >> 1) & 1);
                if (!ok) break;
                const Item w = sm.item[n & 1];
                if (w.h < 0) break;
                tma::arrive(&sm.item_empty[n & 1]);
                const int tiles = max(w.nt0, w.nt1);
                if (tiles <= kAskAhead) tma::arrive(&sm.ask);
                for (int j = 0; j < tiles && ok; ++j) {
                    if (j + kAskAhead == tiles - 1) tma::arrive(&sm.ask);
                    const int row = w.k0 + j * kTileK;
                    for (int c = 0; c < 3; ++c, ++ke) {
                        const int slot = ke % kKSlots;
                        ok = tc::mbar_wait(&sm.k_empty[slot], ((ke / kKSlots) & 1) ^ 1);
                        if (!ok) break;
                        tc::mbar_arrive_expect_tx(&sm.k_full[slot], kChunk);
                        if (c < 2)
                            tma::load_3d(sm.k[slot], &p.kv, &sm.k_full[slot], 64 * c, w.h, row);
                        else
                            tma::load_2d(sm.k[slot], &p.pe, &sm.k_full[slot], 0, row);
                        ++sm.k_issued;
                    }
                    if (!ok) break;
                    // the queries behind the first keys, which can come while the last item's still are in use;
                    // tile 1's, which stay in use longer, behind the first values
                    auto queries = [&](int g) {
                        if (j > 0 || (g ? w.nt1 : w.nt0) == 0) return;
                        ok = tc::mbar_wait(&sm.q_empty[g], (qe[g] & 1) ^ 1);
                        if (!ok) return;
                        tc::mbar_arrive_expect_tx(&sm.q_full[g], 3 * kChunk);
                        for (int c = 0; c < 3; ++c)
                            tma::load_3d(sm.q[g][c], &p.q, &sm.q_full[g], 64 * c, w.h, w.q0 + w.row0 + g * kTileQ);
                        ++qe[g];
                        ++sm.q_issued[g];
                    };
                    queries(0);
                    if (!ok) break;
                    const int slot = ve % kVSlots;
                    ok = tc::mbar_wait(&sm.v_empty[slot], ((ve / kVSlots) & 1) ^ 1);
                    if (!ok) break;
                    tc::mbar_arrive_expect_tx(&sm.v_full[slot], 2 * kChunk);
                    tma::load_3d(sm.v[slot][0], &p.kv, &sm.v_full[slot], kNope, w.h, row);
                    tma::load_3d(sm.v[slot][1], &p.kv, &sm.v_full[slot], kNope + 64, w.h, row);
                    ++ve;
                    ++sm.v_issued;
                    queries(1);
                }
            }
            if (!ok) sm.failed = 1;
        }
        __syncwarp();
    } else if (warp == 10) {
        // ---- scheduler: this block's item, then those of blocks that have not started, taken over one
        // at a time when the loads of the item at hand come to their end ----
        int64_t index = blockIdx.x;
        Place at = {0, 0, 0};
        int n = 0, asked = 0;
        while (ok) {
            Item w;
            const bool more = index >= 0, found = more && find_item(p, index, at, w);
            if (found || !more) {
                ok = n < 2 || tma::wait_warp(&sm.item_empty[n & 1], ((n >> 1) & 1) ^ 1);
                if (!ok) break;
                if (!more) w.h = -1;
                if (lane == 0) {
                    sm.item[n & 1] = w;
                    tma::arrive(&sm.item_full[n & 1]);
                }
                __syncwarp();
                if (!more) break;
                // its first loads wait for shared memory: meanwhile the rows come to L2
                if (n > 0 && lane < 6 && (lane < 3 ? w.nt0 : w.nt1) > 0)
                    tma::prefetch_3d(&p.q, 64 * (lane % 3), w.h, w.q0 + w.row0 + (lane / 3) * kTileQ);
                if (n > 0 && lane >= 8 && lane < 12 && max(w.nt0, w.nt1) > 0)
                    tma::prefetch_3d(&p.kv, 64 * (lane - 8), w.h, w.k0);
                ok = wait_while_loading(&sm.ask, n & 1);
                ++n;
                if (!ok) break;
            }
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&sm.cancel_full, 16);
                tma::try_cancel(&sm.canceled, &sm.cancel_full);
            }
            ok = tma::wait_warp(&sm.cancel_full, asked & 1);
            ++asked;
            if (!ok) break;
            index = tma::canceled_block(&sm.canceled);
            fence_proxy_async();  // the next answer is written behind this reading
            __syncwarp();
        }
        if (!ok) sm.failed = 1;
    } else if (warp == 8) {
        // ---- MMA issuer: one thread runs the whole loop (votes between the products would hold up their issue) ----
        if (tma::elect()) {
            constexpr uint32_t idS = tma::idesc(kTileQ, kTileK, 0, 0), idO = tma::idesc(kTileQ, kNope, 0, 1);
            const uint32_t q_lo = tma::lo_k(tc::smem_addr(sm.q)), k_lo = tma::lo_k(tc::smem_addr(sm.k));
            const uint32_t v_lo = tma::lo_mn(tc::smem_addr(sm.v), kChunk);
            int ke = 0, ve = 0, qe[2] = {0, 0}, pe[2] = {0, 0};  // K chunks, V tiles; Q tiles and P tiles by query tile
            // S_g = Q_g K^T of the key tile whose chunks start at ring entry e
            auto scores = [&](int g, int e, bool release, bool last) {
                const uint32_t d = tmem + g * 128;
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    const int slot = (e + c) % kKSlots, ph = ((e + c) / kKSlots) & 1;
                    if (ok) ok = tc::mbar_wait(&sm.k_full[slot], ph);
                    if (!ok) return;
                    const uint32_t a = q_lo + (g * 3 + c) * (kChunk >> 4), b = k_lo + slot * (kChunk >> 4);
#pragma unroll
                    for (int s = 0; s < 4; ++s) tma::mma_ss(d, a + 2 * s, b + 2 * s, idS, (c | s) != 0);
                    if (release) tc::commit(&sm.k_empty[slot]);
                }
                tc::commit(&sm.s_full[g]);
                if (last) tc::commit(&sm.q_empty[g]);
            };
            int early = 0;  // whether the item's first scores of query tile 0 went out with the last item
            for (int n = 0; ok; ++n) {
                ok = tc::mbar_wait(&sm.item_full[n & 1], (n >> 1) & 1);
                if (!ok || sm.item[n & 1].h < 0) break;
                const int nt0 = sm.item[n & 1].nt0, nt1 = sm.item[n & 1].nt1;
                tma::arrive(&sm.item_empty[n & 1]);
                const int tiles = max(nt0, nt1);
                for (int g = early; g < 2 && ok; ++g) {
                    const int nt = g ? nt1 : nt0;
                    if (nt == 0) continue;
                    ok = tc::mbar_wait(&sm.q_full[g], qe[g] & 1);
                    ++qe[g];
                    scores(g, ke, g == 1 || nt1 == 0, nt == 1);
                }
                early = 0;
                for (int j = 0; j < tiles && ok; ++j, ++ve) {
                    const int slot = ve % kVSlots;
                    const uint32_t add = (j & (kFold - 1)) != 0;  // to what O holds
                    ok = tc::mbar_wait(&sm.v_full[slot], (ve / kVSlots) & 1);
                    for (int g = 0; g < 2 && ok; ++g) {
                        const int nt = g ? nt1 : nt0;
                        if (j >= nt) continue;
                        const uint32_t d = tmem + 256 + g * 128, a = tmem + g * 128, b = v_lo + slot * (2 * kChunk >> 4);
#pragma unroll
                        for (int k = 0; k < kParts; ++k) {
                            ok = ok && tc::mbar_wait(&sm.p_full[g][k], pe[g] & 1);
                            if (!ok) break;
                            tc::fence_after_sync();
#pragma unroll
                            for (int s = k * (kTileK / 16 / kParts); s < (k + 1) * (kTileK / 16 / kParts); ++s)
                                tma::mma_ts(d, a + 8 * s, b + 128 * s, idO, s != 0 ? 1 : add);
                        }
                        if (!ok) break;
                        ++pe[g];
                        tc::commit(&sm.pv_done[g]);
                        if (g == 1 || j >= nt1) tc::commit(&sm.v_empty[slot]);
                        if (j + 1 < nt) scores(g, ke + 3 * (j + 1), g == 1 || j + 1 >= nt1, j + 2 == nt);
                        if (ok && g == 1 && j + 2 == nt1 && nt0 < nt1) {
                            // query tile 0 is through and tile 1 has its last scores: the next item's first scores
                            // of tile 0 before tile 1's last values
                            ok = tc::mbar_wait(&sm.item_full[(n + 1) & 1], ((n + 1) >> 1) & 1);
                            const Item &next = sm.item[(n + 1) & 1];
                            if (ok && next.h >= 0 && next.nt0 > 0) {
                                ok = tc::mbar_wait(&sm.q_full[0], qe[0] & 1);
                                ++qe[0];
                                scores(0, ke + 3 * tiles, next.nt1 == 0, next.nt0 == 1);
                                early = 1;
                            }
                        }
                    }
                }
                ke += 3 * tiles;
            }
            if (!ok) sm.failed = 1;
        }
        __syncwarp();
    } else {
        // ---- softmax: one thread a query row ----
        const int g = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + g * 128, o_addr = tmem + lane_base + 256 + g * 128;
        const float c = p.scale * 1.4426950408889634f;
        const uint64_t c2 = pk2(c, c);
        int sp = 0, ve = 0;  // score tiles of this query tile so far, V tiles before this item
        for (int n = 0; ok; ++n) {
            ok = wait_while_loading(&sm.item_full[n & 1], (n >> 1) & 1);  // tile 1 may have no rows
            if (!ok) break;
            const Item w = sm.item[n & 1];
            if (w.h < 0) break;
            tma::arrive_warp(&sm.item_empty[n & 1]);
            const int row = w.row0 + g * kTileQ + r, nt = g ? w.nt1 : w.nt0;
            const int keys = row < w.nq ? keys_of(w, p.causal, row) : w.nk;
            float m_ref = -INFINITY;  // reference maximum of O and l, in raw scores
            uint64_t l = pk2(0.f, 0.f);
            float kept[kKept];  // O, reference and denominator of the tiles before the last kFold
            int je = min(nt, kFold);  // the next key tile to stop at
            for (int j = 0;; ++j, ++sp) {
                if (j == je) {
                    if (nt > kFold) {
                        ok = tma::wait_warp(&sm.pv_done[g], (sp - 1) & 1);
                        if (!ok) break;
                        tc::fence_after_sync();
                        const float2 lk = upk2(l);
                        const float all = fold_o(kept, o_addr, lk.x + lk.y, m_ref, c, j == kFold, j == nt);
                        l = pk2(j == nt ? all : 0.f, 0.f);
                    }
                    if (j == nt) break;
                    je = min(nt, j + kFold);
                }
                ok = tma::wait_warp(&sm.s_full[g], sp & 1);
                if (!ok) break;
                tc::fence_after_sync();
                // Twice over the row, for its maximum and for P, 64 scores in registers at a time, in loops
                // that stay loops: unrolled over 128 registers the code spilled, and evicted the other roles'
                // loops from the instruction cache wherever an item ended
                uint32_t s[2][32];
                const int valid = keys - j * kTileK;
                const bool hidden = __any_sync(0xffffffffu, valid < kTileK);
                float mx = -INFINITY;
                tc::tmem_ld32_nowait(s_addr, s[0]);
                tc::tmem_ld32_nowait(s_addr + 32, s[1]);
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    tc::tmem_wait_ld();
                    if (hidden) hide(s[0], valid - 64 * i), hide(s[1], valid - 64 * i - 32);
                    mx = fmaxf(mx, fmaxf(max32(s[0], -INFINITY), max32(s[1], -INFINITY)));
                    // the second half, then the first again
                    tc::tmem_ld32_nowait(s_addr + 64 * (1 - i), s[0]);
                    tc::tmem_ld32_nowait(s_addr + 64 * (1 - i) + 32, s[1]);
                }
                const bool grown = (mx - m_ref) * c > kRescale;  // also from -inf to a finite maximum
                if (j == 0) {
                    m_ref = mx;
                } else if (__any_sync(0xffffffffu, grown)) {
                    const float mn = grown ? mx : m_ref;
                    const float f = grown ? tc::ex2((m_ref - mn) * c) : 1.0f;
                    m_ref = mn;
                    l = mul2(l, pk2(f, f));
                    ok = tma::wait_warp(&sm.pv_done[g], (sp - 1) & 1);
                    if (!ok) break;
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        uint32_t x[16];
                        tma::tmem_ld16_nowait(o_addr + 16 * i, x);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * f);
                        tc::tmem_st16(o_addr + 16 * i, x);
                    }
                }
                const float mb = m_ref == -INFINITY ? 0.f : -m_ref * c;
                const uint64_t nmb2 = pk2(mb, mb);
                const int there = w.nk - j * kTileK;
                if (there < kTileK && (g == 0 || j >= w.nt0)) {
                    // value rows behind the sequence; the first query tile that uses them clears them
                    const int slot = (ve + j) % kVSlots;
                    ok = tma::wait_warp(&sm.v_full[slot], ((ve + j) / kVSlots) & 1);
                    if (!ok) break;
                    for (int u = r; u < 2 * (kTileK - there) * 8; u += kTileQ) {
                        const int chunk = u >= (kTileK - there) * 8, x = u - chunk * (kTileK - there) * 8;
                        reinterpret_cast<uint4 *>(sm.v[slot][chunk])[there * 8 + x] = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async();
                }
                // the value product starts on the first 32 keys while the others are at their exponentials
                uint64_t lj[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    tc::tmem_wait_ld();
                    if (hidden) hide(s[0], valid - 64 * i), hide(s[1], valid - 64 * i - 32);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t pr[16];
                        exp32(s[k], pr, c2, nmb2, lj);
                        if (i == 0) tc::tmem_ld32_nowait(s_addr + 64 + 32 * k, s[k]);
                        tc::tmem_st16(s_addr + 32 * i + 16 * k, pr);
                        tc::tmem_wait_st();
                        tc::fence_before_sync();
                        tma::arrive_warp(&sm.p_full[g][2 * i + k]);
                    }
                }
                l = add2(l, add2(lj[0], lj[1]));
            }
            ve += max(w.nt0, w.nt1);
            if (ok && nt > 0) {
                ok = tma::wait_warp(&sm.pv_done[g], (sp - 1) & 1);
                tc::fence_after_sync();
            }
            const float2 la = upk2(l);
            const float lt = la.x + la.y;
            const float inv = !ok ? NAN : (lt == 0.f ? 0.f : 1.0f / lt);
            const int64_t at = ((int64_t)(w.q0 + row)) * p.H + w.h;
            if (p.lse && row < w.nq) p.lse[at] = !ok ? NAN : (lt == 0.f ? -INFINITY : m_ref * p.scale + logf(lt));
            __nv_bfloat16 *dst = p.o + at * kNope;
            const bool some = nt > 0 && lt != 0.f;  // else the row saw nothing: zeros, whatever O holds
            for (int i = 0; i < 4; ++i) {
                uint32_t x[32];
                if (nt > 0) {
                    tc::tmem_ld32_nowait(o_addr + 32 * i, x);
                    tc::tmem_wait_ld();
                }
                if (row < w.nq) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t o8[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float a = some ? __uint_as_float(x[16 * k + 2 * e]) : 0.f;
                            const float b = some ? __uint_as_float(x[16 * k + 2 * e + 1]) : 0.f;
                            const __nv_bfloat162 hh = __floats2bfloat162_rn(a * inv, b * inv);
                            o8[e] = *reinterpret_cast<const uint32_t *>(&hh);
                        }
                        if (p.o_sectors) {
                            tma::st_global32(dst + 32 * i + 16 * k, o8);
                        } else {
                            uint4 *d = reinterpret_cast<uint4 *>(dst + 32 * i + 16 * k);
                            d[0] = make_uint4(o8[0], o8[1], o8[2], o8[3]);
                            d[1] = make_uint4(o8[4], o8[5], o8[6], o8[7]);
                        }
                    }
                }
            }
            // O has been read: this thread's part of the next P lets the MMA warp write it
            tc::fence_before_sync();
        }
        if (!ok) sm.failed = 1;
    }
    tc::fence_before_sync();
    __syncthreads();
    if (sm.failed && warp == 8) {
        // a wait gave up: report it, and let what is in flight land before the memory goes
        if (tma::elect()) {
            set_status(p.status, KDA_ERR_CUDA);
            tc::commit(&sm.drained);
            tc::mbar_wait(&sm.drained, 0);
            for (int g = 0; g < 2; ++g)
                if (sm.q_issued[g] > 0) tc::mbar_wait(&sm.q_full[g], (sm.q_issued[g] - 1) & 1);
            for (int e = max(0, sm.k_issued - kKSlots); e < sm.k_issued; ++e)
                tc::mbar_wait(&sm.k_full[e % kKSlots], (e / kKSlots) & 1);
            for (int e = max(0, sm.v_issued - kVSlots); e < sm.v_issued; ++e)
                tc::mbar_wait(&sm.v_full[e % kVSlots], (e / kVSlots) & 1);
            const uint64_t t0 = tc::globaltimer();
            while (tc::globaltimer() - t0 < 50000) {  // an answer that may still be on its way: 50 us
            }
        }
        __syncwarp();
    }
    if (warp == 8) tc::tmem_dealloc(tmem, 512);
}

// dynamic shared memory: the structure and the slack of its 1024-byte alignment
constexpr size_t kPrefillSmem = sizeof(PrefillSmem) + 1024;
static_assert(kPrefillSmem <= 232448, "prefill shared memory");

}  // namespace
}  // namespace kda

extern "C" int kda_mla_prefill(const uint16_t *q, const uint16_t *kv, const uint16_t *k_pe, int64_t k_pe_stride,
                               const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int64_t total_q,
                               int64_t total_k, int32_t num_seqs, int32_t num_heads, int32_t causal, float scale,
                               uint16_t *o, float *lse, int32_t *status, void *stream) {
    using namespace kda;
    if (!(scale > 0.0f) || scale > 3.402823466e38f || (causal != 0 && causal != 1)) return KDA_ERR_UNSUPPORTED;
    if (total_q < 0 || total_k < 0 || total_q > INT32_MAX || total_k > INT32_MAX || num_seqs < 0 || num_heads <= 0 ||
        num_heads > 65535 || k_pe_stride < kPos || k_pe_stride % 8 || k_pe_stride >= ((int64_t)1 << 38))
        return KDA_ERR_SHAPE;
    const int64_t slots = total_q / kRowsCta + num_seqs;  // sum of ceil(n_q / 256) at most
    if (slots * num_heads > INT32_MAX) return KDA_ERR_SHAPE;
    if (num_seqs == 0 || total_q == 0) return KDA_OK;
    if (!q || !cu_seqlens_q || !cu_seqlens_k || !o || (total_k > 0 && (!kv || !k_pe))) return KDA_ERR_NULL;
    if (!mla_aligned(q, 16) || !mla_aligned(kv, 16) || !mla_aligned(k_pe, 16) || !mla_aligned(o, 16) ||
        !mla_aligned(lse, 4) || !mla_aligned(cu_seqlens_q, 4) || !mla_aligned(cu_seqlens_k, 4) || !mla_aligned(status, 4))
        return KDA_ERR_ALIGN;
    int sms = 0, device = 0;
    int rc = device_sms(&sms, &device);
    if (rc != KDA_OK) return rc;
    PrefillArgs a;
    const uint64_t H = (uint64_t)num_heads;
    const uint64_t dq[3] = {kQk, H, (uint64_t)total_q}, sq[3] = {1, kQk, H * kQk};
    const uint64_t dk[3] = {2 * kNope, H, (uint64_t)total_k}, sk[3] = {1, 2 * kNope, H * 2 * kNope};
    const uint64_t dp[3] = {kPos, (uint64_t)total_k, 0}, sp[3] = {1, (uint64_t)k_pe_stride, 0};
    if (!tma::encode(&a.q, q, 3, dq, sq, 1, kTileQ)) return KDA_ERR_CUDA;
    if (total_k > 0) {
        if (!tma::encode(&a.kv, kv, 3, dk, sk, 1, kTileK) || !tma::encode(&a.pe, k_pe, 2, dp, sp, kTileK, 1))
            return KDA_ERR_CUDA;
    } else {
        a.kv = a.pe = a.q;  // no key tile exists, nothing loads through them
    }
    a.cu_q = cu_seqlens_q;
    a.cu_k = cu_seqlens_k;
    a.Tq = total_q;
    a.Tk = total_k;
    a.N = num_seqs;
    a.H = num_heads;
    a.causal = causal;
    a.scale = scale;
    a.o = reinterpret_cast<__nv_bfloat16 *>(o);
    a.o_sectors = mla_aligned(o, 32);
    a.lse = lse;
    a.status = status;
    static std::atomic<bool> configured[64];
    if (device >= 64) return KDA_ERR_DEVICE;
    if (!configured[device].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kda_mla_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPrefillSmem) !=
            cudaSuccess)
            return KDA_ERR_CUDA;
        configured[device].store(true, std::memory_order_release);
    }
    return launch_after(kda_mla_prefill_kernel, dim3((unsigned)(slots * num_heads)), dim3(kThreads), kPrefillSmem,
                        static_cast<cudaStream_t>(stream), a) == cudaSuccess
               ? KDA_OK
               : KDA_ERR_CUDA;
}
