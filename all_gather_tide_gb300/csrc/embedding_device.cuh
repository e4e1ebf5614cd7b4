// Device helpers shared by the embedding lookup and its gradient.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>

#include "step_internal.h"
#include "step_launch.cuh"

namespace tide {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStatusBadId = 64;

__device__ __forceinline__ char* shard_base(const ShardPtrs& s, uint32_t d) {
    return static_cast<char*>(s.table ? s.table[d] : s.p[d]);
}

__device__ __forceinline__ int64_t load_id(const void* ids, int ids64, int64_t i) {
    return ids64 ? load_here(static_cast<const int64_t*>(ids) + i) : int64_t(load_here(static_cast<const int32_t*>(ids) + i));
}

// The table row of an id, or `rows` where the position holds no token.
__device__ __forceinline__ uint32_t row_of(int64_t id, uint32_t rows) { return id < 0 || id >= int64_t(rows) ? rows : uint32_t(id); }

// The same; ids >= rows are recorded.
__device__ __forceinline__ uint32_t row_of(const void* ids, int ids64, int64_t i, uint32_t rows, int* status) {
    const int64_t id = load_id(ids, ids64, i);
    if (id >= int64_t(rows)) atomicCAS(status, 0, kStatusBadId);
    return row_of(id, rows);
}

// V consecutive bf16 elements, widened and scaled.
template <int V>
struct Bf16Vec {
    using Word = typename std::conditional<V == 8, uint4, typename std::conditional<V == 4, uint2, typename std::conditional<V == 2, uint32_t, uint16_t>::type>::type>::type;
};

__device__ __forceinline__ float low_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void widen(const uint4& w, float (&x)[8]) {
    x[0] = low_f32(w.x), x[1] = high_f32(w.x), x[2] = low_f32(w.y), x[3] = high_f32(w.y);
    x[4] = low_f32(w.z), x[5] = high_f32(w.z), x[6] = low_f32(w.w), x[7] = high_f32(w.w);
}
__device__ __forceinline__ void widen(const uint2& w, float (&x)[4]) { x[0] = low_f32(w.x), x[1] = high_f32(w.x), x[2] = low_f32(w.y), x[3] = high_f32(w.y); }
__device__ __forceinline__ void widen(const uint32_t& w, float (&x)[2]) { x[0] = low_f32(w), x[1] = high_f32(w); }
__device__ __forceinline__ void widen(const uint16_t& w, float (&x)[1]) { x[0] = low_f32(w); }

__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void store_v8(float* p, const float (&x)[8]) {
    asm volatile("st.global.cs.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                 "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
}
__device__ __forceinline__ void load_v8(const float* p, float (&x)[8]) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void put(float* p, const float (&x)[8]) { store_v8(p, x); }
__device__ __forceinline__ void put(float* p, const float (&x)[4]) { __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3])); }
__device__ __forceinline__ void put(float* p, const float (&x)[2]) { __stcs(reinterpret_cast<float2*>(p), make_float2(x[0], x[1])); }
__device__ __forceinline__ void put(float* p, const float (&x)[1]) { *p = x[0]; }
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&x)[8]) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]), pack(x[6], x[7])));
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&x)[4]) { __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack(x[0], x[1]), pack(x[2], x[3]))); }
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&x)[2]) { *reinterpret_cast<uint32_t*>(p) = pack(x[0], x[1]); }
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&x)[1]) { *p = __float2bfloat16_rn(x[0]); }

// The aligned 16 bytes, by the warp's lanes, that hold `bytes` bytes from `from` on; what lies behind these is not
// read.  What lies before them in their first 16 is: it is of the same allocation.  bytes <= kMost, so that the
// copies are predicated and not a loop (127618 rows of 1123 columns summed in 93 us, with a loop 100).
template <uint32_t kMost>
__device__ __forceinline__ void copy_shifted(uint32_t to, uint64_t from, uint32_t bytes) {
    bytes += uint32_t(from) & 15;
    from &= ~uint64_t(15);
    const uint32_t lane16 = (threadIdx.x & 31) * 16;
#pragma unroll
    for (uint32_t i = 0; i < kMost + 15; i += 32 * 16) {
        const uint32_t at = lane16 + i;
        if (at < bytes) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + at), "l"(from + at), "r"(min(16u, bytes - at)) : "memory");
    }
}
__device__ __forceinline__ float load_shared(uint32_t at, float) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float load_shared(uint32_t at, __nv_bfloat16) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    return __uint_as_float(uint32_t(v) << 16);
}

}  // namespace
}  // namespace tide
