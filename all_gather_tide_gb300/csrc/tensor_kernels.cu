// Operators over a list of tensors: global gradient norm, clipping, AdamW (sm_103a).
//
// A work item is `chunk` consecutive elements of one tensor, and one warp takes one item at a time,
// so that thousands of small tensors spread over the GPU as well as a few large ones.  Items are cut
// on the tensor's own 8-element boundaries (32 bytes of fp32, 16 of bf16): item i covers elements
// [i*chunk - mis, (i+1)*chunk - mis) of a tensor whose first element lies mis elements past a
// boundary, so every group of 8 that lies inside the tensor is one aligned vector, and only the
// groups at the tensor's ends go element by element.  A list too short to give every warp of the GPU
// 2048 elements has shorter items, down to one group for each lane (0.85 M elements: AdamW 16.7 us with
// items of 2048 elements, 8.2 with 256).
//
// All are bound by HBM.  856 M bf16 gradients' norm: 237 us, 7.2 TB/s.  625 M fp32 gradients in 3144 pieces:
// norm 355 us (7.0 TB/s), clipping 750 us (6.6 TB/s).  AdamW over 856 M elements: 3.78 ms, 6.8 TB/s.
#include <cuda_bf16.h>

#include <algorithm>

#include "step_internal.h"
#include "step_launch.cuh"

namespace tide {
namespace {

constexpr int kWarps = kTsThreads / 32;

// Offsets are elements from the item's nominal first element, begin.
struct Item {
    int k;          // tensor
    int64_t begin;  // in the tensor
    int left;       // elements of the tensor from there on, as far as they matter to the item
    bool bf16;      // the gradient's type

    // For an array that lies mis elements past a boundary: the first element of the lane's first
    // group, the end of the item, and the least offset inside the tensor.
    __device__ __forceinline__ int first(unsigned mis) const { return int(threadIdx.x & 31) * 8 - int(mis); }
    __device__ __forceinline__ int end(unsigned mis, int chunk) const { return min(left, chunk - int(mis)); }
    __device__ __forceinline__ int least() const { return begin == 0 ? 0 : -8; }
};

__device__ __forceinline__ Item item_of(const TsList& l, int64_t c) {
    const int4 x = __ldg(reinterpret_cast<const int4*>(l.items) + c);
    return {x.x, int64_t(uint32_t(x.y)) * l.chunk, x.z, x.w != 0};
}

__device__ __forceinline__ int64_t first_item() { return int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); }
__device__ __forceinline__ int64_t item_stride() { return int64_t(gridDim.x) * kWarps; }

// Elements a pointer lies past a boundary of 8.
template <typename T>
__device__ __forceinline__ unsigned misalign(const T* p) {
    return unsigned(reinterpret_cast<uintptr_t>(p) / sizeof(T)) & 7u;
}

__device__ __forceinline__ void narrow(float* p, float v) { *p = v; }
__device__ __forceinline__ void narrow(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// 8 elements at an aligned address as they lie in memory (32-bit words), not kept in L1.
__device__ __forceinline__ void load_raw(const float* p, uint32_t (&w)[8]) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void load_raw(const __nv_bfloat16* p, uint32_t (&w)[4]) {
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void unpack(const uint32_t (&w)[8], float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[j]);
}
__device__ __forceinline__ void unpack(const uint32_t (&w)[4], float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                 "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    uint4 w;
    __nv_bfloat162 h;
    h = __floats2bfloat162_rn(x[0], x[1]), w.x = *reinterpret_cast<uint32_t*>(&h);
    h = __floats2bfloat162_rn(x[2], x[3]), w.y = *reinterpret_cast<uint32_t*>(&h);
    h = __floats2bfloat162_rn(x[4], x[5]), w.z = *reinterpret_cast<uint32_t*>(&h);
    h = __floats2bfloat162_rn(x[6], x[7]), w.w = *reinterpret_cast<uint32_t*>(&h);
    *reinterpret_cast<uint4*>(p) = w;
}

// The group of 8 elements from offset e on, as raw words: groups inside [lo, end) as a vector where
// `vec` says that the array has the alignment, else element by element; elements outside read as 0
// (and, in store_group, are not written).
__device__ __forceinline__ uint32_t bits_of(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }

template <typename T>
__device__ __forceinline__ void load_group(const T* p, int e, int lo, int end, bool vec, uint32_t (&w)[2 * sizeof(T)]) {
    if (vec && e >= lo && e + 8 <= end) {
        load_raw(p + e, w);
    } else {
        constexpr int kPer = 4 / sizeof(T);  // elements in a word
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = e + j >= lo && e + j < end ? bits_of(p[e + j]) : 0u;
            w[j / kPer] = j % kPer ? w[j / kPer] | b << 16 : b;
        }
    }
}
template <typename T>
__device__ __forceinline__ void store_group(T* p, int e, int lo, int end, bool vec, const float (&x)[8]) {
    if (vec && e >= lo && e + 8 <= end) {
        store8(p + e, x);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (e + j >= lo && e + j < end) narrow(p + e + j, x[j]);
    }
}

// Sum over the warp.
__device__ __forceinline__ double warp_sum(double v) {
    for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    return v;
}

// Sum over the CTA in a fixed order; valid in warp 0, which adds for all: a warp's fp64 addition takes the SM
// as long as 16 or more of fp32.
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double part[kTsThreads];
    part[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x >= 32) return 0.0;
    double x[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x[w] = part[threadIdx.x + 32 * w];
#pragma unroll
    for (int s = kWarps / 2; s > 0; s >>= 1)
#pragma unroll
        for (int w = 0; w < s; ++w) x[w] += x[w + s];
    return warp_sum(x[0]);
}

// The CTAs' sums of squares in a fixed order, by one warp, 16 loads of each lane in flight.
__device__ __forceinline__ double sum_partials(const double* partial, unsigned count) {
    constexpr int kAhead = 16;
    double all = 0.0;
    for (unsigned b = threadIdx.x & 31; b < count; b += 32 * kAhead) {
        double x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) x[u] = b + 32 * u < count ? load_here(&partial[b + 32 * u]) : 0.0;
#pragma unroll
        for (int s = kAhead / 2; s > 0; s >>= 1)
#pragma unroll
            for (int u = 0; u < s; ++u) x[u] += x[u + s];
        all += x[0];
    }
    return warp_sum(all);
}

// The sum of squares of 32 numbers: 32 is what a lane holds at once, and keeps fp64, whose adds the GPU
// has few of, to one for 32 elements.  In fp32 while no square can have left its range: a sum in
// [2^-100, 2^126] has lost at most 32 * 2^-150 to squares below the smallest subnormal.  Else, unless
// all are 0, in fp64 (a rare branch; NaN and infinity take it and stay what they are).
__device__ __forceinline__ double sum_squares(const float (&x)[4][8]) {
    float s[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        s[q] = x[q][0] * x[q][0];
#pragma unroll
        for (int j = 1; j < 8; ++j) s[q] = fmaf(x[q][j], x[q][j], s[q]);
    }
    const float sum = (s[0] + s[1]) + (s[2] + s[3]);
    if (sum >= 0x1p-100f && sum <= 0x1p126f) return double(sum);
    double d = 0.0;
    uint32_t any = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j) any |= __float_as_uint(x[q][j]) << 1;
    if (any)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < 8; ++j) d += double(x[q][j]) * double(x[q][j]);
    return d;
}

// Groups of 8 that a lane loads before it uses the first: 128 bytes in flight for either type.
template <typename T>
constexpr int kBatch = int(16 / sizeof(T));

template <typename T>
__device__ __forceinline__ double item_squares(const T* g, const Item& it, int chunk) {
    const unsigned mis = misalign(g);
    const int lo = it.least(), end = it.end(mis, chunk);
    g += it.begin;
    double sum = 0.0;
    for (int e = it.first(mis); e < end; e += kBatch<T> * 256) {
        uint32_t w[kBatch<T>][2 * sizeof(T)];
#pragma unroll
        for (int q = 0; q < kBatch<T>; ++q) load_group(g, e + q * 256, lo, end, true, w[q]);
#pragma unroll
        for (int q = 0; q < kBatch<T>; q += 4) {
            float x[4][8];
#pragma unroll
            for (int r = 0; r < 4; ++r) unpack(w[q + r], x[r]);
            sum += sum_squares(x);
        }
    }
    return sum;
}

// Sums of squares of the CTAs to partial; with Finish the CTA that arrives last adds them in the
// CTAs' order.
template <bool Finish>
__global__ void __launch_bounds__(kTsThreads, kTsCtasPerSm)
grad_norm_kernel(TsList l, const void* const* __restrict__ grads, double* partial, unsigned* ticket, float* norm,
                 double* sumsq) {
    wait_for_previous_kernel();
    double sum = 0.0;
    for (int64_t c = first_item(); c < l.chunks; c += item_stride()) {
        const Item it = item_of(l, c);
        const void* g = grads[it.k];
        sum += it.bf16 ? item_squares(static_cast<const __nv_bfloat16*>(g), it, l.chunk) : item_squares(static_cast<const float*>(g), it, l.chunk);
    }
    let_next_kernel_start();
    sum = block_sum(sum);
    if (!Finish) {
        if (threadIdx.x == 0) partial[blockIdx.x] = sum;
        return;
    }
    __shared__ bool last;
    if (threadIdx.x == 0) {
        partial[blockIdx.x] = sum;
        __threadfence();
        last = atomicAdd(ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last || threadIdx.x >= 32) return;
    __threadfence();
    const double all = sum_partials(partial, gridDim.x);
    if (threadIdx.x == 0) {
        norm[0] = float(sqrt(all));
        if (sumsq) sumsq[0] = all;
        *ticket = 0;
    }
}

// min(1, max_norm / (norm + 1e-6)), NaN where that is NaN.
__device__ __forceinline__ float clip_factor(float norm, float max_norm) {
    const float q = __fdiv_rn(max_norm, __fadd_rn(norm, 1e-6f));
    return q >= 1.0f ? 1.0f : q;
}

template <typename T>
__device__ __forceinline__ void scale_item(T* g, const Item& it, int chunk, float f) {
    const unsigned mis = misalign(g);
    const int lo = it.least(), end = it.end(mis, chunk);
    g += it.begin;
    for (int e = it.first(mis); e < end; e += kBatch<T> * 256) {
        uint32_t w[kBatch<T>][2 * sizeof(T)];
#pragma unroll
        for (int q = 0; q < kBatch<T>; ++q) load_group(g, e + q * 256, lo, end, true, w[q]);
#pragma unroll
        for (int q = 0; q < kBatch<T>; ++q) {
            float x[8];
            unpack(w[q], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= f;
            store_group(g, e + q * 256, lo, end, true, x);
        }
    }
}

__global__ void __launch_bounds__(kTsThreads, kTsCtasPerSm)
clip_kernel(TsList l, void* const* __restrict__ grads, float* norm, const double* partial, unsigned parts, float max_norm) {
    wait_for_previous_kernel();
    // the norm, or, straight after grad_norm_kernel<false>, what it left of it
    float n;
    if (parts) {
        __shared__ float shared_norm;
        if (threadIdx.x < 32) {
            const double all = sum_partials(partial, parts);
            if (threadIdx.x == 0) {
                shared_norm = float(sqrt(all));
                if (blockIdx.x == 0) norm[0] = shared_norm;
            }
        }
        __syncthreads();
        n = shared_norm;
    } else {
        n = *norm;
    }
    const float f = clip_factor(n, max_norm);
    if (f == 1.0f) return;
    // from the last item to the first: what the norm read last is what L2 still holds
    for (int64_t c = l.chunks - 1 - first_item(); c >= 0; c -= item_stride()) {
        const Item it = item_of(l, c);
        void* g = grads[it.k];
        if (it.bf16) scale_item(static_cast<__nv_bfloat16*>(g), it, l.chunk, f);
        else scale_item(static_cast<float*>(g), it, l.chunk, f);
    }
    let_next_kernel_start();
}

// Loshchilov and Hutter's AdamW on one item, a group of 8 elements for each lane at a time: four loads of 32
// bytes are in flight before the group's arithmetic, three stores of 32 and one of 16 follow.  Root and
// quotient are the rounded ones; there are instructions to spare (issue slots 24 % used).
template <typename T>
__device__ __forceinline__ void adamw_item(const TsList& l, const AdamwArgs& a, void* const* tables, const Item& it, float f) {
    const int64_t K = l.K;
    float* p = static_cast<float*>(tables[it.k]);
    const T* g = static_cast<const T*>(tables[K + it.k]);
    float* m = static_cast<float*>(tables[2 * K + it.k]);
    float* v = static_cast<float*>(tables[3 * K + it.k]);
    auto* w = a.write_shards ? static_cast<__nv_bfloat16*>(tables[4 * K + it.k]) : nullptr;
    const float* decay = reinterpret_cast<const float*>(tables + (a.write_shards ? 5 : 4) * K);
    const float keep = a.has_decay ? fmaf(-a.lr, __ldg(decay + it.k), 1.0f) : 1.0f;
    const unsigned mis = misalign(p);
    const bool gv = misalign(g) == mis, mv = misalign(m) == mis, vv = misalign(v) == mis, wv = misalign(w) == mis;
    const int lo = it.least(), end = it.end(mis, l.chunk);
    p += it.begin, g += it.begin, m += it.begin, v += it.begin, w += it.begin;
    for (int e = it.first(mis); e < end; e += 256) {
        uint32_t pw[8], gw[2 * sizeof(T)], mw[8], vw[8];
        load_group(p, e, lo, end, true, pw);
        load_group(g, e, lo, end, gv, gw);
        load_group(m, e, lo, end, mv, mw);
        load_group(v, e, lo, end, vv, vw);
        float pi[8], gi[8], mi[8], vi[8];
        unpack(pw, pi), unpack(gw, gi), unpack(mw, mi), unpack(vw, vi);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = gi[j] * f;
            mi[j] = a.beta1 * mi[j] + a.one_minus_beta1 * x;
            vi[j] = a.beta2 * vi[j] + a.one_minus_beta2 * x * x;
            const float den = __fsqrt_rn(vi[j]) * a.inv_sqrt_c2 + a.eps;
            pi[j] = pi[j] * keep - a.step_size * __fdiv_rn(mi[j], den);
        }
        store_group(m, e, lo, end, mv, mi);
        store_group(v, e, lo, end, vv, vi);
        store_group(p, e, lo, end, true, pi);
        if (a.write_shards) store_group(w, e, lo, end, wv, pi);
    }
}

__global__ void __launch_bounds__(kTsThreads, kAdamwCtasPerSm)
adamw_kernel(TsList l, void* const* __restrict__ tables, AdamwArgs a) {
    wait_for_previous_kernel();
    float f = 1.0f;
    if (a.norm) {
        const float n = *a.norm;
        if (a.skip_nonfinite && !isfinite(n)) return;
        f = clip_factor(n, a.max_norm);
    }
    for (int64_t c = first_item(); c < l.chunks; c += item_stride()) {
        const Item it = item_of(l, c);
        if (it.bf16) adamw_item<__nv_bfloat16>(l, a, tables, it, f);
        else adamw_item<float>(l, a, tables, it, f);
    }
    let_next_kernel_start();
}

int grid_of(const TsList& l, int ctas) { return int(std::max<int64_t>(1, std::min<int64_t>(ctas, (l.chunks + kWarps - 1) / kWarps))); }

}  // namespace

cudaError_t launch_grad_norm(const TsList& l, const void* const* grads, double* partial, unsigned* ticket, float* norm,
                             double* sumsq, int ctas, cudaStream_t stream) {
    return launch_after(grad_norm_kernel<true>, grid_of(l, ctas), kTsThreads, 0, stream, l, grads, partial, ticket, norm, sumsq);
}

cudaError_t launch_clip(const TsList& l, void* const* grads, const float* norm, float max_norm, int ctas,
                        cudaStream_t stream) {
    if (l.chunks == 0) return cudaSuccess;
    return launch_after(clip_kernel, grid_of(l, ctas), kTsThreads, 0, stream, l, grads, const_cast<float*>(norm),
                        static_cast<const double*>(nullptr), 0u, max_norm);
}

cudaError_t launch_clip_norm(const TsList& l, void* const* grads, double* partial, float* norm, float max_norm, int ctas,
                             cudaStream_t stream) {
    const int grid = grid_of(l, ctas);
    const cudaError_t e = launch_after(grad_norm_kernel<false>, grid, kTsThreads, 0, stream, l, static_cast<const void* const*>(grads), partial,
                                       static_cast<unsigned*>(nullptr), static_cast<float*>(nullptr), static_cast<double*>(nullptr));
    if (e != cudaSuccess) return e;
    return launch_after(clip_kernel, grid, kTsThreads, 0, stream, l, grads, norm, static_cast<const double*>(partial), unsigned(grid), max_norm);
}

cudaError_t launch_adamw(const TsList& l, void* const* tables, const AdamwArgs& a, int ctas, cudaStream_t stream) {
    if (l.chunks == 0) return cudaSuccess;
    return launch_after(adamw_kernel, grid_of(l, ctas), kTsThreads, 0, stream, l, tables, a);
}

}  // namespace tide
