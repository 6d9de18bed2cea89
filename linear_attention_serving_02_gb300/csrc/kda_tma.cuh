// Tiled TMA loads into 128-byte-swizzled shared memory, and the matrix descriptors that read
// them: the operand path of the latent-attention kernels.
//
// A tile is cut into chunks of 64 bf16 columns (128 bytes). A chunk of R rows is R * 128
// bytes, 1024-byte aligned; TMA stores the 16-byte unit u of row r at unit u ^ (r % 8), and
// the tensor core undoes it. Read with the chunk's columns as the contraction (K-major),
// 8-row groups are 1024 B apart and a step of 16 columns is 32 B further. Read with the
// chunk's rows as the contraction (MN-major), 8-row groups are again 1024 B apart, a step of
// 16 rows is 2048 B further, and the next 64 columns are one chunk further.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kda_tc.cuh"

namespace kda {
namespace tma {

constexpr int kChunkCols = 64;  // bf16 columns of a chunk: one 128-byte swizzle row

// Descriptors as their two halves: the high one is the same for every operand here (8-row
// groups 1024 B apart, version 1, 128-byte swizzle); the low one holds the address and, for an
// MN-major operand, the distance of its 64-column chunks. Adding to the low half moves the
// operand: +2 a 16-column step (K-major), +128 a 16-row step (MN-major), bytes / 16 a chunk.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// (the address field has 14 bits)
__device__ __forceinline__ uint32_t lo_k(uint32_t chunk_saddr) { return ((chunk_saddr >> 4) & 0x3FFF) | (1u << 16); }
__device__ __forceinline__ uint32_t lo_mn(uint32_t chunk_saddr, uint32_t chunk_bytes) {
    return ((chunk_saddr >> 4) & 0x3FFF) | ((chunk_bytes >> 4) << 16);
}
// D[tmem] (+)= A B^T, both in shared memory; issued by one thread
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p;\n.reg .b64 a, b;\nmov.b64 a, {%1, %5};\nmov.b64 b, {%2, %5};\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(id), "r"(accumulate), "n"(kDescHi));
}
// the same with A in tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p;\n.reg .b64 b;\nmov.b64 b, {%2, %5};\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(id), "r"(accumulate), "n"(kDescHi));
}
// 16 consecutive 32-bit TMEM columns of this thread's lane, without the wait
__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// instruction descriptor: kind::f16, bf16 operands, fp32 accumulator; a_mn / b_mn read that
// operand MN-major
__host__ __device__ constexpr uint32_t idesc(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void load_2d(void *dst, const CUtensorMap *map, uint64_t *mbar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n" ::
            "r"(tc::smem_addr(dst)),
        "l"(map), "r"(tc::smem_addr(mbar)), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void load_3d(void *dst, const CUtensorMap *map, uint64_t *mbar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];\n" ::"r"(tc::smem_addr(dst)),
        "l"(map), "r"(tc::smem_addr(mbar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}
// a wait by a whole warp, whose lanes agree on the outcome (what follows is warp-collective)
__device__ __forceinline__ bool wait_warp(uint64_t *mbar, uint32_t parity) {
    return __all_sync(0xffffffffu, tc::mbar_wait(mbar, parity));
}
// true in one lane of a converged warp. Tensor-core and TMA instructions take their operands
// from uniform registers; under this predicate (unlike `lane == 0`) the compiler knows that
// one lane runs and moves them there once, instead of in a loop over the active lanes
__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void arrive(uint64_t *mbar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(tc::smem_addr(mbar)) : "memory");
}
// arrive once for a whole warp, behind what all its lanes did
__device__ __forceinline__ void arrive_warp(uint64_t *mbar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) arrive(mbar);
}
// ask for bytes (16-byte aligned, a multiple of 16) to be in L2
__device__ __forceinline__ void prefetch_l2(const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(src), "r"(bytes) : "memory");
}
// ask for a box of a tiled map to be in L2
__device__ __forceinline__ void prefetch_3d(const CUtensorMap *map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];\n" ::"l"(map), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
// 32 bytes in one store: a whole sector of a row that one thread writes (32-byte aligned)
__device__ __forceinline__ void st_global32(void *dst, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// Ask for a block of this grid that has not started, to do its work in this one: the 16-byte answer
// lands at `answer` and counts on mbar. canceled_block reads it: the block's x index, or -1 when
// none was left (then nothing may be asked for again).
__device__ __forceinline__ void try_cancel(void *answer, uint64_t *mbar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::"r"(
                     tc::smem_addr(answer)),
                 "r"(tc::smem_addr(mbar))
                 : "memory");
}
__device__ __forceinline__ int64_t canceled_block(const void *answer) {
    uint32_t got, x;
    asm volatile(
        "{\n.reg .b128 a;\n.reg .pred p;\nld.shared.b128 a, [%2];\n"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\nselp.u32 %0, 1, 0, p;\nmov.u32 %1, 0;\n"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n}\n"
        : "=r"(got), "=r"(x)
        : "r"(tc::smem_addr(answer))
        : "memory");
    return got ? (int64_t)x : -1;
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
}

// ---- host side ----
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// the driver's encoder, looked up once a process
inline EncodeFn encoder() {
    static std::atomic<EncodeFn> kept{nullptr};
    EncodeFn f = kept.load(std::memory_order_acquire);
    if (f) return f;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult got;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &got) != cudaSuccess ||
        got != cudaDriverEntryPointSuccess)
        return nullptr;
    f = reinterpret_cast<EncodeFn>(p);
    kept.store(f, std::memory_order_release);
    return f;
}

// Map of a bf16 tensor of `rank` (2 or 3) dimensions, innermost first, whose strides count
// elements (dims 1 ..), for boxes of {64, box1, box2}. Out-of-range rows load as zeros.
inline bool encode(CUtensorMap *map, const void *base, int rank, const uint64_t (&dim)[3], const uint64_t (&stride)[3],
                   uint32_t box1, uint32_t box2) {
    const EncodeFn f = encoder();
    if (!f) return false;
    cuuint64_t d[3], s[2];
    for (int i = 0; i < rank; ++i) d[i] = dim[i];
    for (int i = 1; i < rank; ++i) s[i - 1] = stride[i] * 2;
    const cuuint32_t box[3] = {(cuuint32_t)kChunkCols, box1, box2}, one[3] = {1, 1, 1};
    return f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), d, s, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tma
}  // namespace kda
