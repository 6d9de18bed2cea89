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
// S0(j+1) PV1(j) S1(j+1). TMEM holds exactly S0 S1 O0 O1 (4 x 128 columns). Bounds: 2 x 1280
// cycles of tensor work a key tile at 8192 flop a cycle, and 32 K exponentials.
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since its last reference
// (P stays below 2^8, far inside bf16 and fp32), which few tiles do; l sums the fp32 values.
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
constexpr int kThreads = 320;  // 2 x 4 softmax warps, the MMA warp, the TMA warp
constexpr float kRescale = 8.0f;
constexpr int kParts = 4;  // P of a key tile is handed over in parts of 32 keys

struct PrefillArgs {
    CUtensorMap q, kv, pe;
    const int32_t *cu_q, *cu_k;
    int64_t Tq, Tk;
    int32_t N, H, causal;
    float scale;
    __nv_bfloat16 *o;
    float *lse;
    int32_t *status;
};

struct PrefillSmem {
    uint8_t q[2][3][kChunk];
    uint8_t k[kKSlots][kChunk];
    uint8_t v[kVSlots][2][kChunk];
    uint64_t q_full[2], k_full[kKSlots], k_empty[kKSlots], v_full[kVSlots], v_empty[kVSlots];
    uint64_t s_full[2], p_full[2][kParts], pv_done[2], drained;
    uint32_t tmem;
    int32_t seq, tile, failed;
    int32_t k_issued, v_issued;  // loads the producer started (read after a failed wait only)
};

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

__global__ void __launch_bounds__(kThreads, 1) kda_mla_prefill_kernel(const __grid_constant__ PrefillArgs p) {
    extern __shared__ uint8_t smem_raw[];
    PrefillSmem &sm = *reinterpret_cast<PrefillSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % p.H;

    // ---- which sequence and query tile: the slot's place in the list of all tiles ----
    if (warp == 0) {
        const int64_t slot = blockIdx.x / p.H;
        int64_t before = 0;
        int seq = -1, tile = 0;
        for (int n0 = 0; n0 < p.N && seq < 0; n0 += 32) {
            const int n = n0 + lane;
            int64_t tiles = 0;
            if (n < p.N) {
                const int64_t a = p.cu_q[n], b = p.cu_q[n + 1], c = p.cu_k[n], d = p.cu_k[n + 1];
                if (a < 0 || b > p.Tq || b < a || c < 0 || d > p.Tk || d < c)
                    set_status(p.status, KDA_ERR_SEQLENS);  // every CTA that looks finds it: no tiles
                else
                    tiles = (b - a + kRowsCta - 1) / kRowsCta;
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
                seq = n0 + src;
                // a sequence's last tiles see the most keys: they go first
                tile = (int)(__shfl_sync(0xffffffffu, tiles, src) - 1 - (slot - __shfl_sync(0xffffffffu, lo, src)));
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            sm.seq = seq;
            sm.tile = tile;
            sm.failed = 0;
            sm.k_issued = sm.v_issued = 0;
            for (int i = 0; i < 2; ++i) {
                tc::mbar_init(&sm.q_full[i], 1);
                tc::mbar_init(&sm.s_full[i], 1);
                for (int k = 0; k < kParts; ++k) tc::mbar_init(&sm.p_full[i][k], kTileQ);
                tc::mbar_init(&sm.pv_done[i], 1);
            }
            for (int i = 0; i < kKSlots; ++i) tc::mbar_init(&sm.k_full[i], 1), tc::mbar_init(&sm.k_empty[i], 1);
            for (int i = 0; i < kVSlots; ++i) tc::mbar_init(&sm.v_full[i], 1), tc::mbar_init(&sm.v_empty[i], 1);
            tc::mbar_init(&sm.drained, 1);
            tc::mbar_init_fence();
        }
    }
    __syncthreads();
    const int seq = sm.seq;
    if (seq < 0) return;  // more slots than tiles
    if (warp == 8) tc::tmem_alloc(&sm.tmem, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem;

    const int q0 = p.cu_q[seq], nq = p.cu_q[seq + 1] - q0, k0 = p.cu_k[seq], nk = p.cu_k[seq + 1] - k0;
    const int row0 = sm.tile * kRowsCta;
    // keys that query row r sees: min(nk, r + see), see = nk - nq + 1 under the causal mask
    const int see = p.causal ? nk - nq + 1 : nk;
    auto keys_of = [&](int r) { return max(0, p.causal ? min(nk, r + see) : nk); };
    int nt[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int first = row0 + g * kTileQ, last = min(nq, first + kTileQ) - 1;
        nt[g] = last < first ? 0 : (keys_of(last) + kTileK - 1) / kTileK;
    }
    const int tiles = max(nt[0], nt[1]);
    bool ok = true;

    if (warp == 9) {
        // ---- TMA producer ----
        if (lane == 0 && tiles > 0) {
            for (int g = 0; g < 2; ++g) {
                if (nt[g] == 0) continue;
                tc::mbar_arrive_expect_tx(&sm.q_full[g], 3 * kChunk);
                for (int c = 0; c < 3; ++c) tma::load_3d(sm.q[g][c], &p.q, &sm.q_full[g], 64 * c, h, q0 + row0 + g * kTileQ);
            }
            int ks = 0, kph = 0, vs = 0, vph = 0;
            for (int j = 0; j < tiles && ok; ++j) {
                const int row = k0 + j * kTileK;
                for (int c = 0; c < 3 && ok; ++c) {
                    ok = tc::mbar_wait(&sm.k_empty[ks], kph ^ 1);
                    if (!ok) break;
                    tc::mbar_arrive_expect_tx(&sm.k_full[ks], kChunk);
                    if (c < 2)
                        tma::load_3d(sm.k[ks], &p.kv, &sm.k_full[ks], 64 * c, h, row);
                    else
                        tma::load_2d(sm.k[ks], &p.pe, &sm.k_full[ks], 0, row);
                    ++sm.k_issued;
                    if (++ks == kKSlots) ks = 0, kph ^= 1;
                }
                if (!ok) break;
                ok = tc::mbar_wait(&sm.v_empty[vs], vph ^ 1);
                if (!ok) break;
                tc::mbar_arrive_expect_tx(&sm.v_full[vs], 2 * kChunk);
                tma::load_3d(sm.v[vs][0], &p.kv, &sm.v_full[vs], kNope, h, row);
                tma::load_3d(sm.v[vs][1], &p.kv, &sm.v_full[vs], kNope + 64, h, row);
                ++sm.v_issued;
                if (++vs == kVSlots) vs = 0, vph ^= 1;
            }
            if (!ok) sm.failed = 1;
        }
    } else if (warp == 8) {
        // ---- MMA issuer ----
        constexpr uint32_t idS = tma::idesc(kTileQ, kTileK, 0, 0), idO = tma::idesc(kTileQ, kNope, 0, 1);
        const uint32_t q_lo = tma::lo_k(tc::smem_addr(sm.q)), k_lo = tma::lo_k(tc::smem_addr(sm.k));
        const uint32_t v_lo = tma::lo_mn(tc::smem_addr(sm.v), kChunk);
        // one thread runs the whole loop: votes between the products would hold up their issue
        if (tma::elect()) {
            // S_g(j) = Q_g K(j)^T; chunk c of key tile j is ring entry 3 j + c
            auto scores = [&](int g, int j, bool release) {
                const uint32_t d = tmem + g * 128;
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    const int e = 3 * j + c, slot = e % kKSlots, ph = (e / kKSlots) & 1;
                    if (ok) ok = tc::mbar_wait(&sm.k_full[slot], ph);
                    if (!ok) return;
                    const uint32_t a = q_lo + (g * 3 + c) * (kChunk >> 4), b = k_lo + slot * (kChunk >> 4);
#pragma unroll
                    for (int s = 0; s < 4; ++s) tma::mma_ss(d, a + 2 * s, b + 2 * s, idS, (c | s) != 0);
                    if (release) tc::commit(&sm.k_empty[slot]);
                }
                tc::commit(&sm.s_full[g]);
            };
            for (int g = 0; g < 2 && ok; ++g) {
                if (nt[g] == 0) continue;
                ok = tc::mbar_wait(&sm.q_full[g], 0);
                scores(g, 0, g == 1 || nt[1] == 0);
            }
            for (int j = 0; j < tiles && ok; ++j) {
                const int slot = j % kVSlots;
                ok = tc::mbar_wait(&sm.v_full[slot], (j / kVSlots) & 1);
                for (int g = 0; g < 2 && ok; ++g) {
                    if (j >= nt[g]) continue;
                    const uint32_t d = tmem + 256 + g * 128, a = tmem + g * 128, b = v_lo + slot * (2 * kChunk >> 4);
#pragma unroll
                    for (int k = 0; k < kParts; ++k) {
                        ok = ok && tc::mbar_wait(&sm.p_full[g][k], j & 1);
                        if (!ok) break;
                        tc::fence_after_sync();
#pragma unroll
                        for (int s = k * (kTileK / 16 / kParts); s < (k + 1) * (kTileK / 16 / kParts); ++s)
                            tma::mma_ts(d, a + 8 * s, b + 128 * s, idO, s != 0 ? 1 : j != 0);
                    }
                    if (!ok) break;
                    tc::commit(&sm.pv_done[g]);
                    if (g == 1 || j >= nt[1]) tc::commit(&sm.v_empty[slot]);
                    if (j + 1 < nt[g]) scores(g, j + 1, g == 1 || j + 1 >= nt[1]);
                }
            }
            if (!ok) sm.failed = 1;
        }
        __syncwarp();
    } else {
        // ---- softmax: one thread a query row ----
        const int g = warp >> 2, r = (warp & 3) * 32 + lane, row = row0 + g * kTileQ + r;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + g * 128, o_addr = tmem + lane_base + 256 + g * 128;
        const float c = p.scale * 1.4426950408889634f;
        const uint64_t c2 = pk2(c, c);
        const int keys = row < nq ? keys_of(row) : nk;
        float m_ref = -INFINITY;  // reference maximum of O and l, in raw scores
        uint64_t l[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
        for (int j = 0; j < nt[g]; ++j) {
            ok = tma::wait_warp(&sm.s_full[g], j & 1);
            if (!ok) break;
            tc::fence_after_sync();
            uint32_t s[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i) tc::tmem_ld32_nowait(s_addr + 32 * i, s[i]);
            tc::tmem_wait_ld();
            const int valid = keys - j * kTileK;
            if (__any_sync(0xffffffffu, valid < kTileK)) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (32 * i + k >= valid) s[i][k] = 0xff800000u;
            }
            float m4[4];  // independent chains
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = max32(s[i], -INFINITY);
            const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            const bool grown = (mx - m_ref) * c > kRescale;  // also from -inf to a finite maximum
            if (j == 0) {
                m_ref = mx;
            } else if (__any_sync(0xffffffffu, grown)) {
                const float mn = grown ? mx : m_ref;
                const float f = grown ? tc::ex2((m_ref - mn) * c) : 1.0f;
                m_ref = mn;
                l[0] = mul2(l[0], pk2(f, f));
                l[1] = mul2(l[1], pk2(f, f));
                ok = tma::wait_warp(&sm.pv_done[g], (j - 1) & 1);
                if (!ok) break;
                tc::fence_after_sync();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t x[16];
                    tc::tmem_ld8_nowait(o_addr + 16 * i, *reinterpret_cast<uint32_t(*)[8]>(&x[0]));
                    tc::tmem_ld8_nowait(o_addr + 16 * i + 8, *reinterpret_cast<uint32_t(*)[8]>(&x[8]));
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * f);
                    tc::tmem_st16(o_addr + 16 * i, x);
                }
            }
            const float mb = m_ref == -INFINITY ? 0.f : -m_ref * c;
            const uint64_t nmb2 = pk2(mb, mb);
            const int there = nk - j * kTileK;
            if (there < kTileK && (g == 0 || j >= nt[0])) {
                // value rows behind the sequence; the first query tile that uses them clears them
                ok = tma::wait_warp(&sm.v_full[j % kVSlots], (j / kVSlots) & 1);
                if (!ok) break;
                for (int u = r; u < 2 * (kTileK - there) * 8; u += kTileQ) {
                    const int chunk = u >= (kTileK - there) * 8, x = u - chunk * (kTileK - there) * 8;
                    reinterpret_cast<uint4 *>(sm.v[j % kVSlots][chunk])[there * 8 + x] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
            }
            // the value product starts on the first 32 keys while the others are at their exponentials
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                uint32_t pr[16];
                exp32(s[i], pr, c2, nmb2, l);
                tc::tmem_st16(s_addr + 16 * i, pr);
                tc::tmem_wait_st();
                tc::fence_before_sync();
                tma::arrive(&sm.p_full[g][i]);
            }
        }
        if (ok && nt[g] > 0) {
            ok = tma::wait_warp(&sm.pv_done[g], (nt[g] - 1) & 1);
            tc::fence_after_sync();
        }
        if (!ok) sm.failed = 1;
        const float2 la = upk2(add2(l[0], l[1]));
        const float lt = la.x + la.y;
        const float inv = !ok ? NAN : (lt == 0.f ? 0.f : 1.0f / lt);
        const int64_t at = ((int64_t)(q0 + row)) * p.H + h;
        if (p.lse && row < nq) p.lse[at] = !ok ? NAN : (lt == 0.f ? -INFINITY : m_ref * p.scale + logf(lt));
        uint4 *dst = reinterpret_cast<uint4 *>(p.o + at * kNope);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t x[32];
            if (nt[g] > 0) {  // else O holds nothing: zeros
                tc::tmem_ld32_nowait(o_addr + 32 * i, x);
                tc::tmem_wait_ld();
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a = nt[g] > 0 && lt != 0.f ? __uint_as_float(x[8 * k + 2 * e]) : 0.f;
                    const float b = nt[g] > 0 && lt != 0.f ? __uint_as_float(x[8 * k + 2 * e + 1]) : 0.f;
                    const __nv_bfloat162 hh = __floats2bfloat162_rn(a * inv, b * inv);
                    w[e] = *reinterpret_cast<const uint32_t *>(&hh);
                }
                if (row < nq) dst[4 * i + k] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (sm.failed && warp == 8) {
        // a wait gave up: report it, and let what is in flight land before the memory goes
        if (lane == 0) {
            set_status(p.status, KDA_ERR_CUDA);
            tc::commit(&sm.drained);
            bool land = tc::mbar_wait(&sm.drained, 0);
            for (int g = 0; g < 2; ++g)
                if (nt[g] > 0) land = tc::mbar_wait(&sm.q_full[g], 0) && land;
            for (int e = max(0, sm.k_issued - kKSlots); e < sm.k_issued; ++e)
                land = tc::mbar_wait(&sm.k_full[e % kKSlots], (e / kKSlots) & 1) && land;
            for (int e = max(0, sm.v_issued - kVSlots); e < sm.v_issued; ++e)
                land = tc::mbar_wait(&sm.v_full[e % kVSlots], (e / kVSlots) & 1) && land;
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
    kda_mla_prefill_kernel<<<(unsigned)(slots * num_heads), kThreads, kPrefillSmem, static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
