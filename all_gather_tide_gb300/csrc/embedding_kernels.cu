// Embedding lookup over the packed dim-0 shards of a group, and its gradient (sm_103a).
//
// Row t of a table of `rows` rows split over R ranks lies on rank d = t / m, at element
// off + (t - d*m) * len of that rank's shard.  The lookup copies scale * row for every position; the
// gradient sorts the positions by row (stable, so that equal calls add in the same order) and adds
// the rows of dout that share a row of the table.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

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

// The lookup.  One warp takes `tokens` positions and a stretch of columns: its lanes look up one
// position each (id, rank, shard pointer: a chain of loads and a division, paid once for all of the
// warp's positions), then the warp copies row after row, each lane Cols vectors of V elements at a
// time, with kLookupVectors<V> loads in flight before their stores.  Rows of fewer than 32 vectors go
// several at a time (tx = 1 << tx_log lanes each).
template <int V>
constexpr int kLookupVectors = V >= 4 ? 8 : 16;

template <typename Out, int V, int Cols>
__global__ void __launch_bounds__(kThreads, kLookupCtasPerSm)
embedding_kernel(const __grid_constant__ ShardPtrs shards, TableView tv, const void* __restrict__ ids, int ids64,
                 int64_t n, float scale, Out* __restrict__ out, int64_t out_stride, int tx_log, int tokens,
                 uint32_t stretches, int64_t items, int* status) {
    constexpr int Rows = kLookupVectors<V> / Cols;
    using Word = typename Bf16Vec<V>::Word;
    const int lane = threadIdx.x & 31, tx = 1 << tx_log, x = lane & (tx - 1), y = lane >> tx_log, ty = 32 >> tx_log;
    for (int64_t it = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += int64_t(gridDim.x) * (kThreads / 32)) {
        const int64_t group = it / stretches, i0 = group * tokens;
        const uint32_t col0 = (uint32_t(it - group * stretches) * (Cols * tx) + x) * V;
        const int held = int(min(int64_t(tokens), n - i0));
        // where the lane's position finds its row; 0 where it has no token
        unsigned long long at = 0;
        if (lane < held) {
            const uint32_t t = row_of(ids, ids64, i0 + lane, tv.rows, status);
            const uint32_t d = t / tv.m;
            if (t < tv.rows) at = reinterpret_cast<unsigned long long>(shard_base(shards, d)) + 2 * (tv.off + int64_t(t - d * tv.m) * tv.len);
        }
        for (int k0 = 0; k0 < held; k0 += Rows * ty) {
            Word w[Rows][Cols];
            float f[Rows];
#pragma unroll
            for (int r = 0; r < Rows; ++r) {
                const int k = k0 + r * ty + y;
                const auto* row = reinterpret_cast<const uint16_t*>(__shfl_sync(0xffffffffu, at, k & 31));
                const bool has = row && k < held;
                f[r] = has ? scale : 0.0f;  // a row of +0 where there is no token
#pragma unroll
                for (int c = 0; c < Cols; ++c) {
                    const uint32_t col = col0 + c * tx * V;
                    w[r][c] = Word{};
                    if (has && col < tv.len) w[r][c] = __ldg(reinterpret_cast<const Word*>(row + col));
                }
            }
#pragma unroll
            for (int r = 0; r < Rows; ++r) {
                const int k = k0 + r * ty + y;
                Out* o = out + (i0 + k) * out_stride;
#pragma unroll
                for (int c = 0; c < Cols; ++c) {
                    const uint32_t col = col0 + c * tx * V;
                    if (k >= held || col >= tv.len) continue;
                    float v[V];
                    widen(w[r][c], v);
#pragma unroll
                    for (int j = 0; j < V; ++j) v[j] *= f[r];
                    put(o + col, v);
                }
            }
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

namespace {

// The widest vector (8, 4, 2 or 1 elements) that every row address of the table and, of `elem` bytes
// an element, every row address of the other array allow.
int vector_of(const TableView& tv, uintptr_t shard_bits, size_t shard_elem, uintptr_t other, int64_t stride, size_t elem) {
    for (int v = 8; v > 1; v >>= 1)
        if (tv.len % v == 0 && tv.off % v == 0 && stride % v == 0 && shard_bits % (v * shard_elem) == 0 && other % (v * elem) == 0) return v;
    return 1;
}

template <typename Out, int V>
cudaError_t lookup(const ShardPtrs& shards, const TableView& tv, const void* ids, int ids64, int64_t n, float scale,
                   Out* out, int64_t out_stride, int ctas, bool overlap, int* status, cudaStream_t stream) {
    const int64_t vecs = tv.len / V;
    int tx_log = 0;
    while (tx_log < 5 && (1 << tx_log) < vecs) ++tx_log;
    const int cols = V <= 2 && vecs >= 256 ? 8 : vecs >= 128 ? 4 : vecs >= 64 ? 2 : 1;
    const int64_t stretches = (vecs + cols * (1 << tx_log) - 1) / (cols * (1 << tx_log));
    // Positions of a warp: at least 8 while that leaves each of the resident warps an item (one
    // wave), fewer below; up to 32 while there are 8 waves of items, whose ends then cost little.
    const int64_t slots = int64_t(ctas) * (kThreads / 32);
    auto count = [&](int tokens) { return (n + tokens - 1) / tokens * stretches; };
    int tokens = 32;
    while (tokens > 8 && count(tokens) < 8 * slots) tokens >>= 1;
    while (tokens > 1 && count(tokens) < slots) tokens >>= 1;
    const int64_t items = count(tokens);
    const int grid = int(std::min<int64_t>((items + kThreads / 32 - 1) / (kThreads / 32), overlap ? ctas : INT32_MAX));
    auto* kernel = cols == 8 ? embedding_kernel<Out, V, V <= 2 ? 8 : 4> : cols == 4 ? embedding_kernel<Out, V, 4> : cols == 2 ? embedding_kernel<Out, V, 2> : embedding_kernel<Out, V, 1>;
    kernel<<<grid, kThreads, 0, stream>>>(shards, tv, ids, ids64, n, scale, out, out_stride, tx_log, tokens, uint32_t(stretches), items, status);
    return cudaGetLastError();
}

template <typename Out>
cudaError_t lookup_any(const ShardPtrs& shards, const TableView& tv, const void* ids, int ids64, int64_t n, float scale,
                       Out* out, int64_t out_stride, int ctas, bool overlap, int* status, cudaStream_t stream) {
    switch (vector_of(tv, shards.bits, 2, reinterpret_cast<uintptr_t>(out), n > 1 ? out_stride : 0, sizeof(Out))) {
        case 8: return lookup<Out, 8>(shards, tv, ids, ids64, n, scale, out, out_stride, ctas, overlap, status, stream);
        case 4: return lookup<Out, 4>(shards, tv, ids, ids64, n, scale, out, out_stride, ctas, overlap, status, stream);
        case 2: return lookup<Out, 2>(shards, tv, ids, ids64, n, scale, out, out_stride, ctas, overlap, status, stream);
        default: return lookup<Out, 1>(shards, tv, ids, ids64, n, scale, out, out_stride, ctas, overlap, status, stream);
    }
}

}  // namespace

cudaError_t launch_embedding(const ShardPtrs& shards, const TableView& tv, const void* ids, int ids64, int64_t n,
                             float scale, void* out, int out_bf16, int64_t out_stride, int ctas, bool overlap, int* status,
                             cudaStream_t stream) {
    if (n <= 0) return cudaSuccess;
    if (out_bf16)
        return lookup_any(shards, tv, ids, ids64, n, scale, static_cast<__nv_bfloat16*>(out), out_stride, ctas, overlap, status, stream);
    return lookup_any(shards, tv, ids, ids64, n, scale, static_cast<float*>(out), out_stride, ctas, overlap, status, stream);
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
