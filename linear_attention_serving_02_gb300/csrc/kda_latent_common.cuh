// What the latent-attention kernels share: the row geometry, the paged cache, the search of
// a packed batch's offsets, the status word, and host-side checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <climits>

#include "kda.h"

namespace kda {

constexpr int kLatent = KDA_MLA_LATENT;
constexpr int kPos = KDA_MLA_POS;
constexpr int kRow = KDA_MLA_ROW;
constexpr int kNope = KDA_MLA_NOPE;
constexpr int kQk = KDA_MLA_QK;
constexpr int kRow8 = KDA_MLA_ROW_FP8;      // bytes of a row of the 8-bit form, its scale apart
constexpr int kToken8 = KDA_MLA_TOKEN_FP8;  // with its scale

// The kernels are launched so that they may come onto the GPU while the previous kernel on the
// stream ends, and wait for its end (pdl_wait) before they touch memory (the decode's join says why
// it may look at the lengths before): a step of short calls saves about a microsecond a call
// (256-token append 6.1 -> 4.2 us, 330-row gather 6.1 -> 4.2, two windows of 8 tokens x 12 heads
// 16.4 -> 14.1, called one after another). None but the decode's main kernel lets its successor
// start earlier than at its end: in the append that took longer (65536 x 12 70 us, 59 without).
// What they read may thus be written while they are already on the GPU, so they read it with
// ordinary loads: a load through the read-only path claims that nothing writes the data as long as
// the kernel lives, and the compiler may move it to before the wait.

// A cache of rows in pages with its page table (pointers of the caller).
template <typename T>
struct PagedRows {
    T *rows;
    int64_t page_stride;  // elements of T
    int32_t num_pages, page_size;
    const int32_t *table;  // [num_seqs, max_pages]
    int32_t max_pages;
};

// ---- the 8-bit form: a row's latents are e4m3, its positional key bf16, both in units of 2^e ----

// 2^e for e of -126 .. 127
__device__ __forceinline__ float exp2_of(int e) { return __int_as_float((e + 127) << 23); }
// The exponent of a row's scale: the least e of -40 .. 40 with top 2^-e <= 448, the largest e4m3 value, and 0 for
// a row of zeros. 448 is 1.75 2^8: what exceeds 1.75 carries into the exponent. An infinite top gives 40.
__device__ __forceinline__ int scale_exponent(float top) {
    const int e = (int)((__float_as_uint(top) + 0x1FFFFFu) >> 23) - 127 - 8;
    return top == 0.f ? 0 : max(-40, min(40, e));
}
// two values rounded to the nearest e4m3 (a in the low byte); past 448 the nearest is 448, NaN stays NaN
__device__ __forceinline__ uint32_t e4m3_of2(float a, float b) {
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(b), "f"(a));
    return v;
}
// the values of the two e4m3 in the low half of v
__device__ __forceinline__ float2 values_of2(uint32_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Store a status code in the caller's word (the first bad call wins the race or the last;
// both are true, and nothing reads it here).
__device__ __forceinline__ void set_status(int32_t *status, int32_t code) {
    if (status) *status = code;
}

// Largest n in [0, N) with cu[n] <= t, or -1, found by a whole warp: every round splits the
// range into 32 parts with one load a lane (two rounds up to 1024 sequences, where a binary
// search by one thread would chain ten loads). On a table that does not rise the answer is
// some index of the range; callers check what they read with it.
__device__ __forceinline__ int warp_find_seq(const int32_t *cu, int N, int64_t t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = N;  // the answer is in [lo - 1, lo + n)
    while (n > 0) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const bool below = lane * step < n && (int64_t)cu[i] <= t;
        const unsigned m = __ballot_sync(0xffffffffu, below);
        if (m == 0) return lo - 1;
        const int last = 31 - __clz(m);
        const int base = lo + last * step;
        n = min(step, lo + n - base) - 1;  // base itself is <= t: look behind it
        lo = base + 1;
    }
    return lo - 1;
}

// ---- host side ----
inline bool mla_aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The cache's geometry (its pointers apart), T its elements: KDA_OK, KDA_ERR_UNSUPPORTED or KDA_ERR_SHAPE.
template <typename T>
inline int check_cache(int64_t page_stride, int32_t num_pages, int32_t page_size, int32_t max_pages) {
    if (page_size <= 0 || page_size % 16 != 0 || page_size > 65536) return KDA_ERR_UNSUPPORTED;
    constexpr int per_token = sizeof(T) == 1 ? kToken8 : kRow, unit = 16 / sizeof(T);
    if (num_pages < 0 || max_pages < 0 || page_stride < (int64_t)page_size * per_token || page_stride % unit != 0)
        return KDA_ERR_SHAPE;
    if (page_stride > (INT64_MAX >> 2) / (num_pages > 0 ? num_pages : 1)) return KDA_ERR_SHAPE;
    if ((int64_t)max_pages * page_size > INT32_MAX) return KDA_ERR_SHAPE;  // positions are int32
    return KDA_OK;
}

// SMs of the current device, at least compute capability 10.0 (asked anew: both attributes
// are kept by the runtime, so this needs no cache of its own)
inline int device_sms(int *sms, int *device) {
    int major = 0;
    if (cudaGetDevice(device) != cudaSuccess) return KDA_ERR_CUDA;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *device) != cudaSuccess) return KDA_ERR_CUDA;
    if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *device) != cudaSuccess) return KDA_ERR_CUDA;
    if (major < 10 || *sms <= 0) return KDA_ERR_DEVICE;
    return KDA_OK;
}

}  // namespace kda
