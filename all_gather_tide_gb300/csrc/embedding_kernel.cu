// Embedding lookup over the packed dim-0 shards of a group (sm_103a).
//
// Row t of a table of `rows` rows split over R ranks lies on rank d = t / m, at element
// off + (t - d*m) * len of that rank's shard; out row i = scale * row ids[i].
#include <algorithm>

#include "embedding_device.cuh"

namespace tide {
namespace {

// The lookup.  One warp takes `tokens` positions and a stretch of columns: its lanes look up one
// position each (id, rank, shard pointer: a chain of loads and a division, paid once for all of the
// warp's positions), then the warp copies row after row, each lane Cols vectors of V elements at a
// time, with kLookupVectors<V> loads in flight before their stores.  Rows of fewer than 32 vectors go
// several at a time (tx = 1 << tx_log lanes each).  The product is formed in fp32 and rounded once.
//
// Bound by HBM: 65536 positions of 8192 bf16 columns out of 128000 rows take 232 us, 1.51 GB of DRAM
// traffic at 6.5 TB/s (1.40 GB needed; the rest are rows that come back after L2 dropped them).  CTAs in
// which every thread resolved its row took 272 us.
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
    wait_for_previous_kernel();
    for (int64_t it = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items; it += int64_t(gridDim.x) * kWarps) {
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
                    if (has && col < tv.len) w[r][c] = __ldcg(reinterpret_cast<const Word*>(row + col));
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
    let_next_kernel_start();
}

// The lookup of rows that no vector reaches.  A warp takes `tokens` positions as above and a stretch of `width`
// columns; the rows come to shared memory as the aligned 16 bytes that hold them, kShiftedRows in flight, and are
// read back element by element, each lane two at a time where they are written as bf16.
//
// Bound by instructions, about 10 for two elements, and for long rows by HBM: 30000 rows of 2048 columns, off by
// one element, 36 us for 0.25 GB (two-byte loads 75); 4099 of 1027 columns to fp32 5.7 us (9.1); 64000 of 129
// columns 16.3 us (19.9), but of 101 17.1 (15.3), so shorter rows go by two-byte loads.  Stretches of up to 256
// columns, 8 rows in flight, took 52 us for the first, of up to 768 with 3 rows 36, but for 30000 rows of 1001 columns
// 25.2 where 512 take 23.0.  Four-byte vectors are not worth replacing (32000 rows of 1026 columns 26.9 us both ways).
constexpr int kShiftedRows = 4;
constexpr uint32_t kShiftedLeast = 128, kShiftedMost = 512, kShiftedRow = kShiftedMost * 2 + 16;

template <typename Out>
__global__ void __launch_bounds__(kThreads, kLookupCtasPerSm)
embedding_shifted_kernel(const __grid_constant__ ShardPtrs shards, TableView tv, const void* ids, int ids64, int64_t n, float scale,
                         Out* out, int64_t out_stride, uint32_t width, int tokens, uint32_t stretches, int64_t items, int* status) {
    __shared__ __align__(16) unsigned char rings[kWarps][kShiftedRows * kShiftedRow];
    const uint32_t lane = threadIdx.x & 31, ring = uint32_t(__cvta_generic_to_shared(rings[threadIdx.x >> 5]));
    auto slot = [&](int k) { return ring + uint32_t(k) % kShiftedRows * kShiftedRow; };
    wait_for_previous_kernel();
    for (int64_t it = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items; it += int64_t(gridDim.x) * kWarps) {
        const int64_t group = it / stretches, i0 = group * tokens;
        const uint32_t first = uint32_t(it - group * stretches) * width, cols = min(width, tv.len - first);
        const int held = int(min(int64_t(tokens), n - i0));
        // where the lane's position finds its stretch; 0 where it has no token
        unsigned long long at = 0;
        if (int(lane) < held) {
            const uint32_t t = row_of(ids, ids64, i0 + lane, tv.rows, status);
            const uint32_t d = t / tv.m;
            if (t < tv.rows) at = reinterpret_cast<unsigned long long>(shard_base(shards, d)) + 2 * (tv.off + int64_t(t - d * tv.m) * tv.len + first);
        }
        auto fetch = [&](int k) {
            const unsigned long long from = __shfl_sync(0xffffffffu, at, k & 31);
            if (k < held && from) copy_shifted<kShiftedMost * 2>(slot(k), from, cols * 2);
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll 1
        for (int k = 0; k < kShiftedRows; ++k) fetch(k);
        Out* o = out + i0 * out_stride + first;
        for (int k = 0; k < held; ++k, o += out_stride) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kShiftedRows - 1) : "memory");
            __syncwarp();  // lanes read what others copied
            const unsigned long long from = __shfl_sync(0xffffffffu, at, k);
            const uint32_t row = slot(k) + (uint32_t(from) & 15);
            const float f = from ? scale : 0.0f;  // a row of +0 where there is no token
            auto value = [&](uint32_t c) { return from ? f * load_shared(row + 2 * c, __nv_bfloat16()) : 0.0f; };
            if constexpr (sizeof(Out) == 4) {
#pragma unroll 4
                for (uint32_t c = lane; c < cols; c += 32) o[c] = value(c);
            } else {
                // pairs from the first column on that lies on four bytes
                const uint32_t odd = uint32_t(reinterpret_cast<uintptr_t>(o) / 2) & 1;
                if (odd && lane == 0) o[0] = __float2bfloat16_rn(value(0));
#pragma unroll
                for (uint32_t j = 0; j < kShiftedMost / 64; j += 2) {
                    if (odd + 64 * j >= cols) break;
#pragma unroll
                    for (uint32_t q = j; q < j + 2; ++q) {
                        const uint32_t c = odd + 2 * (lane + 32 * q);
                        if (c + 1 < cols) *reinterpret_cast<uint32_t*>(o + c) = pack(value(c), value(c + 1));
                        else if (c < cols) o[c] = __float2bfloat16_rn(value(c));
                    }
                }
            }
            __syncwarp();
            fetch(k + kShiftedRows);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    }
    let_next_kernel_start();
}

// The widest vector (8, 4, 2 or 1 elements) that every row address of the table and, of `elem` bytes
// an element, every row address of the other array allow.
int vector_of(const TableView& tv, uintptr_t shard_bits, size_t shard_elem, uintptr_t other, int64_t stride, size_t elem) {
    for (int v = 8; v > 1; v >>= 1)
        if (tv.len % v == 0 && tv.off % v == 0 && stride % v == 0 && shard_bits % (v * shard_elem) == 0 && other % (v * elem) == 0) return v;
    return 1;
}

// Positions of a warp, where items(tokens) is the work items that so many make: at least 8 while that leaves each
// of the resident warps an item (one wave), fewer below; up to 32 while there are 8 waves of items, whose ends
// then cost little.  Measured with 1, 2, 4 and 8 waves as the only rule: the long case 243, 243, 238, 234 us,
// 4099 rows of 1027 10, 10, 14, 14.
template <typename F>
int tokens_of(int ctas, F&& items) {
    const int64_t slots = int64_t(ctas) * kWarps;
    int tokens = 32;
    while (tokens > 8 && items(tokens) < 8 * slots) tokens >>= 1;
    while (tokens > 1 && items(tokens) < slots) tokens >>= 1;
    return tokens;
}

template <typename Out>
cudaError_t lookup_shifted(const ShardPtrs& shards, const TableView& tv, const void* ids, int ids64, int64_t n, float scale,
                           Out* out, int64_t out_stride, int ctas, bool overlap, int* status, cudaStream_t stream) {
    // stretches of equal length, a multiple of 32
    const uint32_t even = (tv.len + kShiftedMost - 1) / kShiftedMost;
    const uint32_t width = ((tv.len + even - 1) / even + 31) / 32 * 32, stretches = (tv.len + width - 1) / width;
    auto count = [&](int tokens) { return (n + tokens - 1) / tokens * stretches; };
    const int tokens = tokens_of(ctas, count);
    const int64_t items = count(tokens);
    const int grid = int(std::min<int64_t>((items + kWarps - 1) / kWarps, overlap ? ctas : INT32_MAX));
    return launch_after(embedding_shifted_kernel<Out>, grid, kThreads, 0, stream, shards, tv, ids, ids64, n, scale, out, out_stride, width, tokens,
                        stretches, items, status);
}

template <typename Out, int V>
cudaError_t lookup(const ShardPtrs& shards, const TableView& tv, const void* ids, int ids64, int64_t n, float scale,
                   Out* out, int64_t out_stride, int ctas, bool overlap, int* status, cudaStream_t stream) {
    const int64_t vecs = tv.len / V;
    int tx_log = 0;
    while (tx_log < 5 && (1 << tx_log) < vecs) ++tx_log;
    // Vectors of a row that a lane takes at once, fewer where they would reach past the row.  Measured on
    // 67 M elements: rows of 256 columns 27 us with 1, 29 and 36 with 2 and 4; of 512, 27, 23 and 24; of
    // 4096, 34, 29 and 29.
    const int cols = V == 2 && vecs >= 256 ? 8 : vecs >= 128 ? 4 : vecs >= 64 ? 2 : 1;
    const int64_t stretches = (vecs + cols * (1 << tx_log) - 1) / (cols * (1 << tx_log));
    auto count = [&](int tokens) { return (n + tokens - 1) / tokens * stretches; };
    const int tokens = tokens_of(ctas, count);
    const int64_t items = count(tokens);
    const int grid = int(std::min<int64_t>((items + kWarps - 1) / (kWarps), overlap ? ctas : INT32_MAX));
    auto* kernel = cols == 8 ? embedding_kernel<Out, V, V == 2 ? 8 : 4> : cols == 4 ? embedding_kernel<Out, V, 4> : cols == 2 ? embedding_kernel<Out, V, 2> : embedding_kernel<Out, V, 1>;
    return launch_after(kernel, grid, kThreads, 0, stream, shards, tv, ids, ids64, n, scale, out, out_stride, tx_log, tokens,
                        uint32_t(stretches), items, status);
}

template <typename Out>
cudaError_t lookup_any(const ShardPtrs& shards, const TableView& tv, const void* ids, int ids64, int64_t n, float scale,
                       Out* out, int64_t out_stride, int ctas, bool overlap, int* status, cudaStream_t stream) {
    switch (vector_of(tv, shards.bits, 2, reinterpret_cast<uintptr_t>(out), n > 1 ? out_stride : 0, sizeof(Out))) {
        case 8: return lookup<Out, 8>(shards, tv, ids, ids64, n, scale, out, out_stride, ctas, overlap, status, stream);
        case 4: return lookup<Out, 4>(shards, tv, ids, ids64, n, scale, out, out_stride, ctas, overlap, status, stream);
        case 2: return lookup<Out, 2>(shards, tv, ids, ids64, n, scale, out, out_stride, ctas, overlap, status, stream);
        default:
            if (tv.len >= kShiftedLeast) return lookup_shifted(shards, tv, ids, ids64, n, scale, out, out_stride, ctas, overlap, status, stream);
            return lookup<Out, 1>(shards, tv, ids, ids64, n, scale, out, out_stride, ctas, overlap, status, stream);
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

}  // namespace tide
