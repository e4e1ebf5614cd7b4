// Device helpers shared by the kernels of a layer of experts.
#pragma once

#include <cstdint>

#include "embedding_device.cuh"
#include "experts.h"

namespace tide {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// a / b where the quotient has 32 bits, as it nearly always can be had: a division of 64 bits takes some hundred instructions.
__device__ __forceinline__ uint32_t quotient(int64_t a, uint32_t b) { return a <= int64_t(UINT32_MAX) ? uint32_t(a) / b : uint32_t(uint64_t(a) / b); }

// v[0..n] = the sums of f(0..n-1) before each index, and their total at n; n <= 1024.  All of the block's
// threads call it; `sums` is 32 words of shared memory.
template <typename F>
__device__ __forceinline__ void exclusive_sums(int32_t* v, int n, int32_t* sums, F&& f) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if (threadIdx.x < 32) sums[threadIdx.x] = 0;
    __syncthreads();
    for (int s = warp; s * 32 < n; s += warps) {
        const int i = s * 32 + lane;
        const int32_t own = i < n ? f(i) : 0;
        int32_t x = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t y = __shfl_up_sync(kFull, x, d);
            if (lane >= d) x += y;
        }
        if (i < n) v[i] = x - own;
        if (lane == 31) sums[s] = x;
    }
    __syncthreads();
    if (warp == 0) {
        const int32_t own = sums[lane];
        int32_t x = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t y = __shfl_up_sync(kFull, x, d);
            if (lane >= d) x += y;
        }
        sums[lane] = x - own;
        if (lane == 31) v[n] = x;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) v[i] += sums[i >> 5];
    __syncthreads();
}

// rows[0..E] = the experts' first rows, inside [0, M] and ascending whatever the offsets hold: none where these descend. Without
// offsets one expert has all M. All of the block's threads call it.
__device__ __forceinline__ void first_rows(int32_t* rows, const int32_t* offsets, int E, int32_t M) {
    bool descends = false;
    for (int e = threadIdx.x; e <= E; e += int(blockDim.x)) {
        const int32_t at = offsets ? load_here(offsets + e) : e ? M : 0;
        descends |= offsets && e < E && load_here(offsets + e + 1) < at;
        rows[e] = min(max(at, 0), M);
    }
    if (__syncthreads_or(descends)) {
        for (int e = threadIdx.x; e <= E; e += int(blockDim.x)) rows[e] = 0;
        __syncthreads();
    }
}

// The last index of starts[0..n) whose value is <= x; starts[0] = 0 <= x.  Of equal ones it is the last.
__device__ __forceinline__ int last_at_most(const int32_t* starts, int n, int32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// V elements of T as one load.
template <typename T, int V>
struct Vec;
template <int V>
struct Vec<__nv_bfloat16, V> {
    using Word = typename Bf16Vec<V>::Word;
};
template <>
struct Vec<float, 4> {
    using Word = float4;
};
template <>
struct Vec<float, 2> {
    using Word = float2;
};
template <>
struct Vec<float, 1> {
    using Word = float;
};
__device__ __forceinline__ void widen(const float4& w, float (&x)[4]) { x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w; }
__device__ __forceinline__ void widen(const float2& w, float (&x)[2]) { x[0] = w.x, x[1] = w.y; }
__device__ __forceinline__ void widen(const float& w, float (&x)[1]) { x[0] = w; }

}  // namespace
}  // namespace tide
