// What the latent-attention kernels share: the row geometry, the paged cache, the search of
// a packed batch's offsets, the status word, and host-side checks.
#pragma once

#include <cuda_bf16.h>
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
    int64_t page_stride;  // elements
    int32_t num_pages, page_size;
    const int32_t *table;  // [num_seqs, max_pages]
    int32_t max_pages;
};

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

// The cache's geometry (its pointers apart): KDA_OK, KDA_ERR_UNSUPPORTED or KDA_ERR_SHAPE.
inline int check_cache(int64_t page_stride, int32_t num_pages, int32_t page_size, int32_t max_pages) {
    if (page_size <= 0 || page_size % 16 != 0 || page_size > 65536) return KDA_ERR_UNSUPPORTED;
    if (num_pages < 0 || max_pages < 0 || page_stride < (int64_t)page_size * kRow || page_stride % 8 != 0)
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
