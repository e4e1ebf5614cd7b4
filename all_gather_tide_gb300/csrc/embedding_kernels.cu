// Embedding lookup over the packed dim-0 shards of a group, and its gradient (sm_103a).
//
// Row t of a table of `rows` rows split over R ranks lies on rank d = t / m, at element
// off + (t - d*m) * len of that rank's shard.  The lookup copies scale * row for every position; the
// gradient sorts the positions by row (stable, so that equal calls add in the same order) and adds
// the rows of dout that share a row of the table.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "step_internal.h"

namespace cg = cooperative_groups;

namespace tide {
namespace {

constexpr int kThreads = 256;
constexpr int kStatusBadId = 64;

__device__ __forceinline__ char* shard_base(const ShardPtrs& s, uint32_t d) {
    return static_cast<char*>(s.table ? s.table[d] : s.p[d]);
}

// The table row of an id, or `rows` where the position holds no token; ids >= rows are recorded.
__device__ __forceinline__ uint32_t row_of(const void* ids, int ids64, int64_t i, uint32_t rows, int* status) {
    const int64_t id = ids64 ? __ldg(static_cast<const long long*>(ids) + i) : int64_t(__ldg(static_cast<const int*>(ids) + i));
    if (id >= int64_t(rows)) atomicCAS(status, 0, kStatusBadId);
    return (id < 0 || id >= int64_t(rows)) ? rows : uint32_t(id);
}

template <typename Out>
__global__ void __launch_bounds__(kThreads)
embedding_kernel(const __grid_constant__ ShardPtrs shards, TableView tv, const void* __restrict__ ids, int ids64,
                 int64_t n, float scale, Out* __restrict__ out, int64_t out_stride, int* status) {
    for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
        const uint32_t t = row_of(ids, ids64, i, tv.rows, status);
        const bool held = t < tv.rows;
        const uint32_t d = held ? t / tv.m : 0;
        const auto* row = reinterpret_cast<const __nv_bfloat16*>(shard_base(shards, d)) + tv.off + int64_t(t - d * tv.m) * tv.len;
        for (int64_t j = threadIdx.x; j < tv.len; j += kThreads) {
            const float v = held ? __bfloat162float(row[j]) * scale : 0.0f;
            out[i * out_stride + j] = Out(v);
        }
    }
}

// ---- sort of positions by row -----------------------------------------------------------------

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxBits = 10;

__device__ __forceinline__ int batch_of(const Batches& b, uint32_t i) {
    int lo = 0, hi = b.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (b.start[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads)
expand_positions_kernel(const __grid_constant__ Batches b, uint32_t first, uint32_t rows, uint32_t* __restrict__ key,
                        uint64_t* __restrict__ src, int* status) {
    for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < b.start[b.count]; i += gridDim.x * kThreads) {
        const int k = batch_of(b, i);
        const uint32_t j = i - b.start[k];
        key[first + i] = row_of(b.ids[k], b.ids64, j, rows, status);
        src[first + i] = reinterpret_cast<uint64_t>(b.dout[k] + int64_t(j) * b.stride[k]);
    }
}

// Stable radix sort, least significant digit first, by one cluster: each warp owns a contiguous run
// of positions, counts its digits, and places them in order behind the digits of smaller value and
// the same digit of earlier warps and CTAs.
struct SortArgs {
    Batches b;
    uint32_t n, rows;
    int expanded, passes, bits;
    GradWorkspace w;
    int* status;
};

__global__ void __launch_bounds__(kSortThreads, 1) sort_positions_kernel(const __grid_constant__ SortArgs a) {
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t C = cluster.num_blocks(), c = cluster.block_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bins = 1 << a.bits;
    extern __shared__ uint32_t smem[];
    uint32_t* cnt = smem;                      // [kSortWarps][bins]
    uint32_t* total = cnt + kSortWarps * bins; // [bins], read by the cluster
    uint32_t* base = total + bins;             // [bins]
    __shared__ uint32_t warp_sum[kSortWarps];
    const uint32_t per = ((a.n + C * kSortWarps - 1) / (C * kSortWarps) + 31) & ~31u;
    const uint32_t lo = min(a.n, (c * kSortWarps + warp) * per), hi = min(a.n, lo + per);

    for (int pass = 0; pass < a.passes; ++pass) {
        const bool last = pass == a.passes - 1;
        const uint32_t* key_in = (pass & 1) ? a.w.key_a : a.w.key_b;
        const uint32_t* idx_in = (pass & 1) ? a.w.idx_a : a.w.idx_b;
        uint32_t* key_out = last ? a.w.keys : (pass & 1) ? a.w.key_b : a.w.key_a;
        uint32_t* idx_out = (pass & 1) ? a.w.idx_b : a.w.idx_a;
        const int shift = pass * a.bits;
        auto key_at = [&](uint32_t i) -> uint32_t {
            if (pass > 0) return __ldcg(key_in + i);
            if (a.expanded) return a.w.pre_key[i];
            const int k = batch_of(a.b, i);
            return row_of(a.b.ids[k], a.b.ids64, i - a.b.start[k], a.rows, a.status);
        };
        for (int q = threadIdx.x; q < kSortWarps * bins; q += kSortThreads) cnt[q] = 0;
        __syncthreads();
        for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
            const uint32_t i = i0 + lane;
            const uint32_t digit = i < hi ? (key_at(i) >> shift) & (bins - 1) : bins;
            const uint32_t same = __match_any_sync(0xffffffffu, digit);
            if (i < hi && lane == __ffs(same) - 1) cnt[warp * bins + digit] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        for (int q = threadIdx.x; q < bins; q += kSortThreads) {
            uint32_t run = 0;
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t v = cnt[w * bins + q];
                cnt[w * bins + q] = run;
                run += v;
            }
            total[q] = run;
        }
        cluster.sync();
        // bins <= kSortThreads: thread q owns digit q
        const int q = threadIdx.x;
        uint32_t before = 0, all = 0;
        if (q < bins)
            for (uint32_t r = 0; r < C; ++r) {
                const uint32_t v = cluster.map_shared_rank(total, r)[q];
                if (r < c) before += v;
                all += v;
            }
        uint32_t incl = all;
        for (int s = 1; s < 32; s <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl, s);
            if (lane >= s) incl += v;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        uint32_t first = 0;
        for (int w = 0; w < warp; ++w) first += warp_sum[w];
        if (q < bins) base[q] = first + incl - all + before;
        __syncthreads();
        for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
            const uint32_t i = i0 + lane;
            const uint32_t key = i < hi ? key_at(i) : 0;
            const uint32_t digit = i < hi ? (key >> shift) & (bins - 1) : bins;
            const uint32_t same = __match_any_sync(0xffffffffu, digit);
            uint32_t at = 0;
            if (i < hi) at = base[digit] + cnt[warp * bins + digit] + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (i < hi && lane == __ffs(same) - 1) cnt[warp * bins + digit] += __popc(same);
            __syncwarp();
            if (i < hi) {
                const uint32_t idx = pass > 0 ? __ldcg(idx_in + i) : i;
                key_out[at] = key;
                if (!last) {
                    idx_out[at] = idx;
                } else if (a.expanded) {
                    a.w.src[at] = a.w.pre_src[idx];
                } else {
                    const int k = batch_of(a.b, idx);
                    a.w.src[at] = reinterpret_cast<uint64_t>(a.b.dout[k] + int64_t(idx - a.b.start[k]) * a.b.stride[k]);
                }
            }
        }
        // the next pass reads what other CTAs of the cluster wrote, and no CTA may leave while
        // another still reads its totals
        __threadfence();
        cluster.sync();
    }
}

__global__ void __launch_bounds__(kThreads)
zero_table_kernel(const __grid_constant__ ShardPtrs shards, TableView tv) {
    const int64_t n = int64_t(tv.m) * tv.len;
    for (int d = 0; d < tv.R; ++d) {
        float* p = reinterpret_cast<float*>(shard_base(shards, d)) + tv.off;
        for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < n; i += int64_t(gridDim.x) * kThreads) p[i] = 0.0f;
    }
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// One warp per (first position of a row's run, 256 columns): adds the run's rows in order.
template <typename In>
__global__ void __launch_bounds__(kThreads)
sum_positions_kernel(const __grid_constant__ ShardPtrs shards, TableView tv, uint32_t n, const uint32_t* __restrict__ keys,
                     const uint64_t* __restrict__ src, float scale, int accumulate) {
    const int lane = threadIdx.x & 31;
    const int64_t segs = (tv.len + 255) / 256, items = int64_t(n) * segs;
    for (int64_t it = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += int64_t(gridDim.x) * (kThreads / 32)) {
        const uint32_t i = uint32_t(it / segs);
        const int64_t col = (it % segs) * 256 + lane;
        const uint32_t t = keys[i];
        if (t >= tv.rows || (i > 0 && keys[i - 1] == t)) continue;
        float acc[8] = {};
        for (uint32_t k = i; k < n && keys[k] == t; ++k) {
            const In* row = reinterpret_cast<const In*>(src[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col + 32 * j < tv.len) acc[j] += to_f32(row[col + 32 * j]);
        }
        const uint32_t d = t / tv.m;
        float* dst = reinterpret_cast<float*>(shard_base(shards, d)) + tv.off + int64_t(t - d * tv.m) * tv.len;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (col + 32 * j < tv.len) dst[col + 32 * j] = (accumulate ? dst[col + 32 * j] : 0.0f) + scale * acc[j];
    }
}

}  // namespace

cudaError_t launch_embedding(const ShardPtrs& shards, const TableView& tv, const void* ids, int ids64, int64_t n,
                             float scale, void* out, int out_bf16, int64_t out_stride, int ctas, int* status,
                             cudaStream_t stream) {
    if (n <= 0) return cudaSuccess;
    const int grid = int(std::min<int64_t>(n, ctas));
    if (out_bf16)
        embedding_kernel<<<grid, kThreads, 0, stream>>>(shards, tv, ids, ids64, n, scale, static_cast<__nv_bfloat16*>(out), out_stride, status);
    else
        embedding_kernel<<<grid, kThreads, 0, stream>>>(shards, tv, ids, ids64, n, scale, static_cast<float*>(out), out_stride, status);
    return cudaGetLastError();
}

size_t carve_grad_workspace(char* base, int64_t n, GradWorkspace* w) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* p = base + at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    GradWorkspace g;
    g.keys = reinterpret_cast<uint32_t*>(take(size_t(n) * 4));
    g.src = reinterpret_cast<uint64_t*>(take(size_t(n) * 8));
    g.key_a = reinterpret_cast<uint32_t*>(take(size_t(n) * 4));
    g.key_b = reinterpret_cast<uint32_t*>(take(size_t(n) * 4));
    g.idx_a = reinterpret_cast<uint32_t*>(take(size_t(n) * 4));
    g.idx_b = reinterpret_cast<uint32_t*>(take(size_t(n) * 4));
    g.pre_key = reinterpret_cast<uint32_t*>(take(size_t(n) * 4));
    g.pre_src = reinterpret_cast<uint64_t*>(take(size_t(n) * 8));
    if (w) *w = g;
    return at;
}

cudaError_t launch_expand_positions(const Batches& b, uint32_t first, uint32_t rows, const GradWorkspace& w,
                                    int* status, cudaStream_t stream) {
    const uint32_t n = b.start[b.count];
    if (n == 0) return cudaSuccess;
    const int grid = int(std::min<uint32_t>((n + kThreads - 1) / kThreads, 1024u));
    expand_positions_kernel<<<grid, kThreads, 0, stream>>>(b, first, rows, w.pre_key, w.pre_src, status);
    return cudaGetLastError();
}

cudaError_t launch_sort_positions(const Batches& b, bool expanded, uint32_t n, uint32_t rows, const GradWorkspace& w,
                                  int* status, cudaStream_t stream) {
    int bits = 0;
    while (rows >> bits) ++bits;  // keys are 0 .. rows
    SortArgs a{b, n, rows, expanded ? 1 : 0, 0, 0, w, status};
    a.passes = (bits + kSortMaxBits - 1) / kSortMaxBits;
    a.bits = (bits + a.passes - 1) / a.passes;
    const size_t smem = (size_t(kSortWarps) + 2) * (size_t(1) << a.bits) * 4;
    cudaError_t e = cudaFuncSetAttribute(sort_positions_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    sort_positions_kernel<<<1, kSortThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_zero_table(const ShardPtrs& shards, const TableView& tv, int ctas, cudaStream_t stream) {
    zero_table_kernel<<<ctas, kThreads, 0, stream>>>(shards, tv);
    return cudaGetLastError();
}

cudaError_t launch_sum_positions(const ShardPtrs& shards, const TableView& tv, uint32_t n, const GradWorkspace& w,
                                 int dout_bf16, float scale, int accumulate, int ctas, cudaStream_t stream) {
    if (n == 0) return cudaSuccess;
    const int64_t items = int64_t(n) * ((tv.len + 255) / 256);
    const int grid = int(std::min<int64_t>((items + 7) / 8, ctas));
    if (dout_bf16)
        sum_positions_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(shards, tv, n, w.keys, w.src, scale, accumulate);
    else
        sum_positions_kernel<float><<<grid, kThreads, 0, stream>>>(shards, tv, n, w.keys, w.src, scale, accumulate);
    return cudaGetLastError();
}

}  // namespace tide
