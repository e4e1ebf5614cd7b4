// Operators over a list of tensors: global gradient norm, clipping, AdamW (sm_103a).
//
// A work item is kTsChunk elements of one tensor; one warp takes one item at a time.
#include <cuda_bf16.h>

#include <algorithm>

#include "step_internal.h"

namespace tide {
namespace {

constexpr int kWarps = kTsThreads / 32;

// Elements [lo, hi) of tensor k that work item c covers.
struct Item {
    int k;
    int64_t lo, hi;
    bool bf16;
};

__device__ __forceinline__ Item item_of(const TsList& l, int64_t c) {
    Item it;
    it.k = __ldg(&l.chunk_seg[c]);
    const TsSeg* s = l.segs + it.k;
    it.lo = (c - __ldg(&s->chunk_begin)) * kTsChunk;
    it.hi = min(__ldg(&s->elems), it.lo + kTsChunk);
    it.bf16 = __ldg(&s->bf16) != 0;
    return it;
}

__device__ __forceinline__ int64_t first_item() { return int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); }
__device__ __forceinline__ int64_t item_stride() { return int64_t(gridDim.x) * kWarps; }

__device__ __forceinline__ float load_grad(const void* p, int64_t i, bool bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

// Sum over the CTA in a fixed order; valid in thread 0.
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double part[kWarps];
    for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < kWarps; ++w) v += part[w];
    return v;
}

__global__ void __launch_bounds__(kTsThreads)
grad_norm_kernel(TsList l, const void* const* __restrict__ grads, double* partial, unsigned* ticket, float* norm,
                 double* sumsq) {
    const int lane = threadIdx.x & 31;
    double sum = 0.0;
    for (int64_t c = first_item(); c < l.chunks; c += item_stride()) {
        const Item it = item_of(l, c);
        const void* g = grads[it.k];
        for (int64_t i = it.lo + lane; i < it.hi; i += 32) {
            const float v = load_grad(g, i, it.bf16);
            sum += double(v) * double(v);
        }
    }
    sum = block_sum(sum);
    // the CTA that arrives last adds the CTAs' sums in their order
    __shared__ bool last;
    if (threadIdx.x == 0) {
        partial[blockIdx.x] = sum;
        __threadfence();
        last = atomicAdd(ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double all = 0.0;
    for (unsigned b = threadIdx.x; b < gridDim.x; b += kTsThreads) all += __ldcg(&partial[b]);
    all = block_sum(all);
    if (threadIdx.x == 0) {
        norm[0] = float(sqrt(all));
        if (sumsq) sumsq[0] = all;
        *ticket = 0;
    }
}

// min(1, max_norm / (norm + 1e-6)), NaN where that is NaN.
__device__ __forceinline__ float clip_factor(const float* norm, float max_norm) {
    const float q = __fdiv_rn(max_norm, __fadd_rn(*norm, 1e-6f));
    return q >= 1.0f ? 1.0f : q;
}

__global__ void __launch_bounds__(kTsThreads)
clip_kernel(TsList l, void* const* __restrict__ grads, const float* __restrict__ norm, float max_norm) {
    const float f = clip_factor(norm, max_norm);
    if (f == 1.0f) return;
    const int lane = threadIdx.x & 31;
    for (int64_t c = first_item(); c < l.chunks; c += item_stride()) {
        const Item it = item_of(l, c);
        void* g = grads[it.k];
        for (int64_t i = it.lo + lane; i < it.hi; i += 32) {
            const float v = load_grad(g, i, it.bf16) * f;
            if (it.bf16) static_cast<__nv_bfloat16*>(g)[i] = __float2bfloat16_rn(v);
            else static_cast<float*>(g)[i] = v;
        }
    }
}

__global__ void __launch_bounds__(kTsThreads)
adamw_kernel(TsList l, void* const* __restrict__ tables, int write_shards, AdamwArgs a) {
    float f = 1.0f;
    if (a.norm) {
        const float n = *a.norm;
        if (a.skip_nonfinite && !isfinite(n)) return;
        f = clip_factor(a.norm, a.max_norm);
    }
    const int lane = threadIdx.x & 31;
    const float* decay = reinterpret_cast<const float*>(tables + int64_t(5) * l.K);
    for (int64_t c = first_item(); c < l.chunks; c += item_stride()) {
        const Item it = item_of(l, c);
        float* p = static_cast<float*>(tables[it.k]);
        const void* g = tables[l.K + it.k];
        float* m = static_cast<float*>(tables[2 * int64_t(l.K) + it.k]);
        float* v = static_cast<float*>(tables[3 * int64_t(l.K) + it.k]);
        auto* w = static_cast<__nv_bfloat16*>(tables[4 * int64_t(l.K) + it.k]);
        const float keep = decay[it.k];
        for (int64_t i = it.lo + lane; i < it.hi; i += 32) {
            const float x = load_grad(g, i, it.bf16) * f;
            const float mi = a.beta1 * m[i] + a.one_minus_beta1 * x;
            const float vi = a.beta2 * v[i] + a.one_minus_beta2 * x * x;
            const float den = __fsqrt_rn(vi) * a.inv_sqrt_c2 + a.eps;
            const float pi = p[i] * keep - a.step_size * __fdiv_rn(mi, den);
            m[i] = mi;
            v[i] = vi;
            p[i] = pi;
            if (write_shards) w[i] = __float2bfloat16_rn(pi);
        }
    }
}

int grid_of(const TsList& l, int ctas) { return int(std::max<int64_t>(1, std::min<int64_t>(ctas, (l.chunks + kWarps - 1) / kWarps))); }

}  // namespace

cudaError_t launch_grad_norm(const TsList& l, const void* const* grads, double* partial, unsigned* ticket, float* norm,
                             double* sumsq, int ctas, cudaStream_t stream) {
    grad_norm_kernel<<<grid_of(l, ctas), kTsThreads, 0, stream>>>(l, grads, partial, ticket, norm, sumsq);
    return cudaGetLastError();
}

cudaError_t launch_clip(const TsList& l, void* const* grads, const float* norm, float max_norm, int ctas,
                        cudaStream_t stream) {
    if (l.chunks == 0) return cudaSuccess;
    clip_kernel<<<grid_of(l, ctas), kTsThreads, 0, stream>>>(l, grads, norm, max_norm);
    return cudaGetLastError();
}

cudaError_t launch_adamw(const TsList& l, void* const* tables, int write_shards, const AdamwArgs& a, int ctas,
                         cudaStream_t stream) {
    if (l.chunks == 0) return cudaSuccess;
    adamw_kernel<<<grid_of(l, ctas), kTsThreads, 0, stream>>>(l, tables, write_shards, a);
    return cudaGetLastError();
}

}  // namespace tide
