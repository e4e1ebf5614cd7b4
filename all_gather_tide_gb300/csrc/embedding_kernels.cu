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

__device__ __forceinline__ int64_t load_id(const void* ids, int ids64, int64_t i) {
    return ids64 ? __ldg(static_cast<const long long*>(ids) + i) : int64_t(__ldg(static_cast<const int*>(ids) + i));
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
constexpr int kSortMinBits = 6, kSortMaxBits = 10;  // of a digit
constexpr uint32_t kSortMaxCtas = 16;     // of the cluster
constexpr uint32_t kSortPerCta = 2048;   // positions for which another CTA joins it
constexpr uint32_t kPieceMost = 64, kPieceLeast = 8;  // positions of a piece
constexpr int64_t kPieceWarps = 152 * 24;  // warps for which pieces are cut shorter

__device__ __forceinline__ int batch_of(const Batches& b, uint32_t i) {
    int lo = 0, hi = b.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (b.start[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads)
expand_positions_kernel(const __grid_constant__ Batches b, uint32_t first, uint32_t rows, uint4* __restrict__ to, int* status) {
    for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < b.start[b.count]; i += gridDim.x * kThreads) {
        const int k = batch_of(b, i);
        const uint32_t j = i - b.start[k];
        const uint64_t src = reinterpret_cast<uint64_t>(b.dout[k] + int64_t(j) * b.stride[k]);
        to[first + i] = make_uint4(uint32_t(src), uint32_t(src >> 32), row_of(b.ids[k], b.ids64, j, rows, status), 0);
    }
}

// Stable radix sort, least significant digit first, by one cluster: each warp owns a contiguous run
// of positions, counts its digits, and places them in order behind the digits of smaller value and
// the same digit of earlier warps and CTAs.  The counts of the CTAs meet in distributed shared
// memory.  A batch of kSortBatch rounds of 32 positions is loaded at once; a run that is one batch
// stays in registers between counting and placing.
constexpr int kSortBatch = 8;

struct SortArgs {
    Batches b;
    uint32_t n, rows;
    int expanded, passes;
    int64_t counters;
    GradWorkspace w;
    int* status;
};

template <int kBits>
__global__ void __launch_bounds__(kSortThreads, 1) sort_positions_kernel(const __grid_constant__ SortArgs a) {
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t C = cluster.num_blocks(), c = cluster.block_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int bins = 1 << kBits;
    extern __shared__ uint32_t smem[];
    uint32_t* cnt = smem;                       // [kSortWarps][bins]
    uint32_t* base = cnt + kSortWarps * bins;   // [bins]
    uint32_t* totals = base + bins;             // [C][bins], written by the cluster
    __shared__ uint32_t warp_sum[kSortWarps];
    __shared__ Batches b;  // a copy: lanes look up different batches at once
    for (int q = threadIdx.x; q < a.b.count; q += kSortThreads) {
        b.ids[q] = a.b.ids[q];
        b.dout[q] = a.b.dout[q];
        b.stride[q] = a.b.stride[q];
        b.start[q + 1] = a.b.start[q + 1];
    }
    if (threadIdx.x == 0) {
        b.start[0] = 0;
        b.count = a.b.count;
    }
    const uint32_t per = ((a.n + C * kSortWarps - 1) / (C * kSortWarps) + 31) & ~31u;
    const uint32_t lo = min(a.n, (c * kSortWarps + warp) * per), hi = min(a.n, lo + per);
    uint32_t* mine = cnt + warp * bins;

    // no CTA writes to another's shared memory before that one runs (awaited before the first such write)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

    // what the summing kernel finds cleared: its arrival counters
    for (int64_t q = c * kSortThreads + threadIdx.x; q < a.counters; q += C * kSortThreads) a.w.arrived[q] = 0;

    for (int pass = 0; pass < a.passes; ++pass) {
        const bool last = pass == a.passes - 1;
        const uint4* from = (pass & 1) ? a.w.swap_a : a.w.swap_b;
        uint4* to = last ? a.w.sorted : (pass & 1) ? a.w.swap_b : a.w.swap_a;
        const int shift = pass * kBits;
        uint32_t key[kSortBatch];
        uint64_t src[kSortBatch];  // the positions' dout rows
        auto load = [&](uint32_t i0) {
            if (pass > 0 || a.expanded) {
#pragma unroll
                for (int u = 0; u < kSortBatch; ++u) {
                    const uint32_t i = i0 + u * 32 + lane;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (i < hi) x = __ldcg((pass > 0 ? from : a.w.pre) + i);
                    key[u] = x.z;
                    src[u] = uint64_t(x.y) << 32 | x.x;
                }
                return;
            }
            // all ids before anything is done with one
            int64_t id[kSortBatch];
            int k = batch_of(b, i0);
#pragma unroll
            for (int u = 0; u < kSortBatch; ++u) {
                const uint32_t i = i0 + u * 32 + lane;
                id[u] = -1;
                if (i < hi) {
                    while (i >= b.start[k + 1]) ++k;
                    const uint32_t j = i - b.start[k];
                    id[u] = load_id(b.ids[k], a.b.ids64, j);
                    src[u] = reinterpret_cast<uint64_t>(b.dout[k] + int64_t(j) * b.stride[k]);
                }
            }
            bool bad = false;
#pragma unroll
            for (int u = 0; u < kSortBatch; ++u) {
                bad |= id[u] >= int64_t(a.rows);
                key[u] = row_of(id[u], a.rows);
            }
            if (bad) atomicCAS(a.status, 0, kStatusBadId);
        };
        for (int q = threadIdx.x; q < kSortWarps * bins; q += kSortThreads) cnt[q] = 0;
        __syncthreads();
        for (uint32_t i0 = lo; i0 < hi; i0 += kSortBatch * 32) {
            load(i0);
#pragma unroll
            for (int u = 0; u < kSortBatch; ++u)
                if (i0 + u * 32 + lane < hi) atomicAdd(&mine[(key[u] >> shift) & (bins - 1)], 1u);
        }
        __syncthreads();
        if (pass == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        for (int q = threadIdx.x; q < bins; q += kSortThreads) {
            uint32_t run = 0;
#pragma unroll 8
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t v = cnt[w * bins + q];
                cnt[w * bins + q] = run;
                run += v;
            }
            for (uint32_t r = 0; r < C; ++r) cluster.map_shared_rank(totals, r)[c * bins + q] = run;
        }
        cluster.sync();
        // bins <= kSortThreads: thread q owns digit q
        const int q = threadIdx.x;
        uint32_t before = 0, all = 0;
        if (q < bins)
#pragma unroll 4
            for (uint32_t r = 0; r < C; ++r) {
                const uint32_t v = totals[r * bins + q];
                if (r < c) before += v;
                all += v;
            }
        auto scan = [&](uint32_t v) {  // inclusive, over the warp
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, v, s);
                if (lane >= s) v += o;
            }
            return v;
        };
        const uint32_t incl = scan(all);
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        const uint32_t sums = scan(warp_sum[lane]);
        const uint32_t first = __shfl_sync(0xffffffffu, sums, (warp + 31) & 31);
        if (q < bins) base[q] = (warp ? first : 0) + incl - all + before;
        __syncthreads();
        for (uint32_t i0 = lo; i0 < hi; i0 += kSortBatch * 32) {
            if (hi - lo > kSortBatch * 32) load(i0);
#pragma unroll
            for (int u = 0; u < kSortBatch; ++u) {
                if (i0 + u * 32 >= hi) break;
                const bool in = i0 + u * 32 + lane < hi;
                const uint32_t digit = (key[u] >> shift) & (bins - 1);
                // the lanes with this digit, bit by bit: a vote each costs less than a match, which takes
                // time for every distinct value (measured: 4.5 against 8.7 us a pass on 65536 positions)
                uint32_t same = __ballot_sync(0xffffffffu, in);
#pragma unroll
                for (int bit = 0; bit < kBits; ++bit) {
                    const bool set = digit >> bit & 1;
                    const uint32_t v = __ballot_sync(0xffffffffu, set);
                    same &= set ? v : ~v;
                }
                const int lead = __ffs(same) - 1;
                uint32_t at = 0;
                if (in) at = base[digit] + mine[digit] + __popc(same & ((1u << lane) - 1u));
                __syncwarp();
                if (in && lane == lead) mine[digit] += __popc(same);
                __syncwarp();
                if (!in) continue;
                to[at] = make_uint4(uint32_t(src[u]), uint32_t(src[u] >> 32), key[u], 0);
            }
        }
        // the next pass reads what other CTAs wrote, and writes their totals again
        if (!last) {
            __threadfence();
            cluster.sync();
        }
    }
}

// ---- sums ---------------------------------------------------------------------------------------
//
// The sorted list is cut into pieces of `piece` positions; one warp sums one piece over kStretch
// columns (8 to a lane), so the work is the same whatever the texts repeat.  A row whose positions
// all lie in one piece is written at once.  One that runs over several pieces leaves a partial sum in
// each; the warp that arrives last adds them in the order of the pieces, so the result does not
// depend on who that is.  Positions without a token sort last and are not read.
constexpr uint32_t kStretch = 256;

// What a warp has in flight: groups of copies, 2 KB of dout rows each.
template <typename In>
struct Ring {
    static constexpr int kGroups = 3, kGroup = 8 / sizeof(In), kRows = kGroup * kGroups;
    static constexpr uint32_t kRow = kStretch * sizeof(In), kBytes = kRows * kRow;
};

struct SumArgs {
    ShardPtrs shards;
    TableView tv;
    uint32_t n, piece, pieces, stretches;
    GradWorkspace w;
    float scale;
    uint32_t sum_blocks;   // CTAs' worth of sums, before those that write zeros
    uint32_t zero_blocks;
    uint32_t zero_rows;    // rows of the padded table that one warp looks through for rows to zero
};

__device__ __forceinline__ float* table_row(const SumArgs& a, uint32_t t) {
    const uint32_t d = t / a.tv.m;
    return reinterpret_cast<float*>(shard_base(a.shards, d)) + a.tv.off + int64_t(t - d * a.tv.m) * a.tv.len;
}

// The table row of sorted position i (tv.rows: no token).
__device__ __forceinline__ uint32_t row_at(const SumArgs& a, uint32_t i) { return __ldg(&a.w.sorted[i].z); }

// How a warp's 256 columns lie over its lanes: every 32nd element (kSingle), or 8 consecutive ones, whose
// rows in the shard are 32-byte aligned (kWide) or not (kMixed).
enum Layout { kSingle, kMixed, kWide };

// A lane's 8 consecutive columns of a dout row, 16 or 32 bytes, copied to shared memory asynchronously:
// what is in flight takes no registers.  Each lane copies and reads its own bytes only.
template <typename In>
struct Part {
    static constexpr int kWords = sizeof(In) / 2;  // of 16 bytes
    uint4 w[kWords];

    static __device__ __forceinline__ void copy(uint32_t to, uint64_t from) {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 512), "l"(from + i * 16) : "memory");
    }
    __device__ __forceinline__ void read(uint32_t at) {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w) : "r"(at + i * 512) : "memory");
    }
    __device__ __forceinline__ void add(float (&acc)[8]) const {
        float x[8];
        if constexpr (kWords == 1) {
            widen(w[0], x);
        } else {
            x[0] = __uint_as_float(w[0].x), x[1] = __uint_as_float(w[0].y), x[2] = __uint_as_float(w[0].z), x[3] = __uint_as_float(w[0].w);
            x[4] = __uint_as_float(w[1].x), x[5] = __uint_as_float(w[1].y), x[6] = __uint_as_float(w[1].z), x[7] = __uint_as_float(w[1].w);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += x[j];
    }
};

// Every 32nd of 256 columns, for rows that have no 16-byte alignment.
template <typename In>
struct Singles {
    In x[8];
    __device__ __forceinline__ void load(uint64_t row, uint32_t col, uint32_t len) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = col + 32 * j < len ? __ldg(reinterpret_cast<const In*>(row) + col + 32 * j) : In(0.0f);
    }
    __device__ __forceinline__ void add(float (&acc)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += float(x[j]);
    }
};

// Adds without waiting for what was there: L2 reads, adds and writes.  Every element is added to once
// in a call, so the result depends on no order.
__device__ __forceinline__ void add_v1(float* p, float x) { asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(p), "f"(x) : "memory"); }

// The warp's sums to a stretch of a row, dst: `acc` as the layout spreads them over the lanes; `left`
// columns of the row lie from dst on.
template <Layout kLayout, bool Add>
__device__ __forceinline__ void write_row(const SumArgs& a, float* dst, uint32_t left, const float (&acc)[8], float* stage) {
    const int lane = threadIdx.x & 31;
    float x[8];
    if (kLayout == kWide) {
        if (lane * 8u >= left) return;
        dst += lane * 8;
        float y[8] = {};
        // read here and not ahead of need: copies of the rows made as early as dout's (or prefetches,
        // or additions in L2) took 400 to 420 us where this took 371
        if (Add) load_v8(dst, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = y[j] + a.scale * acc[j];
        store_v8(dst, x);
        return;
    }
    if (kLayout == kMixed) {  // lane * 8 + j -> lane + 32 * j, so that stores of single elements lie side by side
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) stage[lane * 9 + j] = acc[j];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int q = lane + 32 * j;
            x[j] = stage[q / 8 * 9 + q % 8];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = acc[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (lane + 32u * j < left) {
            const float v = a.scale * x[j];
            if (Add) add_v1(dst + lane + 32 * j, v);
            else dst[lane + 32 * j] = v;
        }
}

// Partial sums meet in two steps: those of up to kBlock consecutive pieces, then those of the
// blocks.  `which`: 0 for the row that a piece (block) continues, 1 for the one that starts in it.
constexpr uint32_t kBlock = 32;

__device__ __forceinline__ int64_t slot_of(const SumArgs& a, uint32_t x, int which, uint32_t stretch) {
    return (int64_t(x) * 2 + which) * a.stretches + stretch;
}
__device__ __forceinline__ float* partial_of(const SumArgs& a, uint32_t x, int which, uint32_t stretch) {
    return a.w.partial + slot_of(a, x, which, stretch) * kStretch + (threadIdx.x & 31) * 8;
}

__device__ __forceinline__ void put_partial(float* p, const float (&acc)[8]) {
    __stcg(reinterpret_cast<float4*>(p), make_float4(acc[0], acc[1], acc[2], acc[3]));
    __stcg(reinterpret_cast<float4*>(p + 4), make_float4(acc[4], acc[5], acc[6], acc[7]));
}

// Arrives at a counter with everything written so far; true, with what the others wrote visible, for
// the last of `count`.
__device__ __forceinline__ bool last_to_arrive(uint32_t* counter, uint32_t count) {
    __threadfence();
    __syncwarp();
    uint32_t earlier = 0;
    if ((threadIdx.x & 31) == 0) earlier = atomicAdd(counter, 1u);
    if (__shfl_sync(0xffffffffu, earlier, 0) != count - 1) return false;
    __threadfence();
    return true;
}

// sum += the partial sums of count pieces (blocks) from x on, of which only the first may start the row.
__device__ __forceinline__ void add_partials(const SumArgs& a, uint32_t x, uint32_t count, int first_starts, uint32_t stretch, float (&sum)[8]) {
#pragma unroll 8
    for (uint32_t k = 0; k < count; ++k) {
        const float* p = partial_of(a, x + k, k == 0 ? first_starts : 0, stretch);
        const float4 u = __ldcg(reinterpret_cast<const float4*>(p)), v = __ldcg(reinterpret_cast<const float4*>(p + 4));
        sum[0] += u.x, sum[1] += u.y, sum[2] += u.z, sum[3] += u.w, sum[4] += v.x, sum[5] += v.y, sum[6] += v.z, sum[7] += v.w;
    }
}

// After a piece has left a partial sum of row t: the last of the row's pieces in this block adds
// the block's, and the last of its blocks adds the blocks', both in order, and writes the row.
template <Layout kLayout, bool Add>
__device__ __forceinline__ void join_partials(const SumArgs& a, uint32_t t, uint32_t piece, uint32_t stretch, float* stage) {
    const uint32_t lane = threadIdx.x & 31, block = piece / kBlock, p0 = block * kBlock, y = p0 + lane;
    // the row has a position in piece y: its first or last position, or (t lying in between) both ends
    // on either side; pieces that the row crosses begin or end with it
    const bool begins = y < a.pieces && row_at(a, y * a.piece) == t;
    const bool ends = y < a.pieces && row_at(a, min(a.n, (y + 1) * a.piece) - 1) == t;
    const uint32_t in = __ballot_sync(0xffffffffu, begins || ends);
    const uint32_t from = __ffs(in) - 1, count = __popc(in);
    // the row starts in its first piece here unless that continues the one before
    const uint32_t x = p0 + from;
    const bool continued = x > 0 && row_at(a, x * a.piece - 1) == t;
    const bool starts = !continued;
    const uint32_t end = (x + count) * a.piece;
    const bool goes_on = end < a.n && row_at(a, end) == t;
    if (!last_to_arrive(&a.w.arrived[slot_of(a, x, starts, stretch)], count)) return;
    float sum[8] = {};
    add_partials(a, x, count, starts, stretch, sum);
    if (continued || goes_on) {
        // blocks are numbered after the pieces
        put_partial(partial_of(a, a.pieces + block, starts, stretch), sum);
        const uint32_t blocks = (a.pieces + kBlock - 1) / kBlock;
        uint32_t first = block, last = block;
        if (continued) {
            for (uint32_t back = 1;; back += 32) {
                const uint32_t z = back + lane;  // block - z ends with the row
                const uint32_t out = ~__ballot_sync(0xffffffffu, z <= block && row_at(a, (block - z + 1) * kBlock * a.piece - 1) == t);
                first = block - (back - 1) - (out ? __ffs(out) - 1 : 32);
                if (out) break;
            }
        }
        if (goes_on) {
            for (uint32_t ahead = 1;; ahead += 32) {
                const uint32_t z = block + ahead + lane;  // block z begins with the row
                const uint32_t out = ~__ballot_sync(0xffffffffu, z < blocks && row_at(a, z * kBlock * a.piece) == t);
                last = block + (ahead - 1) + (out ? __ffs(out) - 1 : 32);
                if (out) break;
            }
        }
        // of these blocks, the row starts in the first
        if (!last_to_arrive(&a.w.arrived[slot_of(a, a.pieces + first, 1, stretch)], last - first + 1)) return;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
        add_partials(a, a.pieces + first, last - first + 1, 1, stretch, sum);
    }
    const uint32_t col0 = stretch * kStretch;
    write_row<kLayout, Add>(a, table_row(a, t) + col0, a.tv.len - col0, sum, stage);
}

// The running sum of one piece.
template <Layout kLayout, bool Add>
struct Run {
    const SumArgs& a;
    uint32_t piece, stretch, before;
    float* stage;
    float acc[8] = {};
    uint32_t cur = ~0u;    // the row being summed
    float* dst = nullptr;  // its stretch in the shard
    bool starts = true;    // in this piece
    uint32_t head = ~0u;   // the row that an earlier piece began and this one ended

    __device__ __forceinline__ void write() { write_row<kLayout, Add>(a, dst, a.tv.len - stretch * kStretch, acc, stage); }

    // The next position's row of the table, and where it lies; what the position adds follows.
    __device__ __forceinline__ void turn_to(uint32_t t, float* to) {
        if (cur != ~0u) {
            if (starts) {
                write();
            } else {
                put_partial(partial_of(a, piece, 0, stretch), acc);
                head = cur;
            }
        }
        cur = t;
        dst = to;
        starts = t != before;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    }

    __device__ __forceinline__ void finish(uint32_t after) {
        uint32_t tail = ~0u;  // the row that a later piece ends
        if (cur != ~0u) {
            const bool ends = cur != after;
            if (starts && ends) {
                write();
            } else {
                put_partial(partial_of(a, piece, starts ? 1 : 0, stretch), acc);
                if (ends) head = cur; else tail = cur;
            }
        }
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {  // rows that run over several pieces
            const uint32_t t = side ? tail : head;
            if (t != ~0u) join_partials<kLayout, Add>(a, t, piece, stretch, stage);
        }
    }
};

template <typename In, Layout kLayout, bool Add>
__device__ __forceinline__ void sum_piece(const SumArgs& a, uint32_t piece, uint32_t stretch, float* stage, uint32_t ring) {
    const int lane = threadIdx.x & 31;
    const uint32_t lo = piece * a.piece, hi = min(a.n, lo + a.piece);
    // a lane holds positions lane and 32 + lane of the piece; those without a token come last
    static_assert(kPieceMost == 64, "two positions to a lane");
    const uint4 none = make_uint4(0, 0, a.tv.rows, 0);
    const uint4 p0 = lo + lane < hi ? __ldg(&a.w.sorted[lo + lane]) : none, p1 = lo + 32 + lane < hi ? __ldg(&a.w.sorted[lo + 32 + lane]) : none;
    const int held = __popc(__ballot_sync(0xffffffffu, p0.z < a.tv.rows)) + __popc(__ballot_sync(0xffffffffu, p1.z < a.tv.rows));
    auto of = [&](int k, auto x0, auto x1) { return __shfl_sync(0xffffffffu, k < 32 ? x0 : x1, k & 31); };
    auto row = [&](int k) { return of(k, p0.z, p1.z); };
    auto src = [&](int k) { return uint64_t(of(k, p0.y, p1.y)) << 32 | of(k, p0.x, p1.x); };
    // where their rows lie in the shards, worked out by each lane for its own
    const auto d0 = reinterpret_cast<unsigned long long>(p0.z < a.tv.rows ? table_row(a, p0.z) + stretch * kStretch : nullptr);
    const auto d1 = reinterpret_cast<unsigned long long>(p1.z < a.tv.rows ? table_row(a, p1.z) + stretch * kStretch : nullptr);
    auto place = [&](int k) { return reinterpret_cast<float*>(of(k, d0, d1)); };
    Run<kLayout, Add> run{a, piece, stretch, lo > 0 ? row_at(a, lo - 1) : ~0u, stage};
    const uint32_t after = hi < a.n ? row_at(a, hi) : ~0u;  // rows on either side of the piece
    if constexpr (kLayout == kSingle) {
        constexpr int kAhead = 4;
        const uint32_t col = stretch * kStretch + lane;
        for (int k = 0; k < held; k += kAhead) {
            Singles<In> x[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const uint64_t from = src(k + u);
                if (k + u < held) x[u].load(from, col, a.tv.len);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (k + u >= held) break;
                const uint32_t t = row(k + u);
                if (t != run.cur) run.turn_to(t, place(k + u));
                x[u].add(run.acc);
            }
        }
    } else {
        using R = Ring<In>;
        const uint32_t col = stretch * kStretch + lane * 8;
        const bool in = col < a.tv.len;
        auto slot = [&](int k) { return ring + uint32_t(k) % R::kRows * R::kRow; };
        auto fetch = [&](int k) {
#pragma unroll
            for (int u = 0; u < R::kGroup; ++u) {
                const uint64_t from = src(k + u);
                if (in && k + u < held) Part<In>::copy(slot(k + u), from + uint64_t(col) * sizeof(In));
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int k = 0; k < R::kRows; k += R::kGroup) fetch(k);
        for (int k = 0; k < held; k += R::kGroup) {
            asm volatile("cp.async.wait_group %0;" ::"n"(R::kGroups - 1) : "memory");
            Part<In> x[R::kGroup];
#pragma unroll
            for (int u = 0; u < R::kGroup; ++u) x[u].read(slot(k + u));
#pragma unroll
            for (int u = 0; u < R::kGroup; ++u) {
                if (k + u >= held) break;
                const uint32_t t = row(k + u);
                if (t != run.cur) run.turn_to(t, place(k + u));
                x[u].add(run.acc);
            }
            fetch(k + R::kRows);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    run.finish(after);
}

// Zeros from p on, n elements, by one warp: 32-byte stores between single ones at the ends.
__device__ __forceinline__ void zero_run(float* p, uint32_t n) {
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t head = min(n, (8u - (unsigned(reinterpret_cast<uintptr_t>(p) / 4) & 7u)) & 7u);
    const float z[8] = {};
    if (lane < head) p[lane] = 0.0f;
    const uint32_t vecs = (n - head) / 8;
    for (uint32_t v = lane; v < vecs; v += 32) store_v8(p + head + v * 8, z);
    for (uint32_t i = head + vecs * 8 + lane; i < n; i += 32) p[i] = 0.0f;
}

// The first sorted position in [lo, hi) whose row is >= r (hi if none), found by the whole warp, 32
// places at a time.
__device__ __forceinline__ uint32_t first_at_least(const SumArgs& a, uint32_t r, uint32_t lo, uint32_t hi) {
    const uint32_t lane = threadIdx.x & 31;
    while (lo < hi) {
        const uint32_t step = (hi - lo + 32) / 33;  // lane k looks at the last position of the k-th part
        const uint64_t x = uint64_t(lo) + uint64_t(lane + 1) * step - 1;
        const uint32_t below = __ballot_sync(0xffffffffu, x < hi && row_at(a, uint32_t(x)) < r);
        const uint32_t k = __popc(below);  // sorted: a prefix of the lanes
        const uint64_t end = uint64_t(lo) + uint64_t(k + 1) * step - 1;
        lo += k * step;
        if (end < hi) hi = uint32_t(end);
    }
    return lo;
}

// Zeros to those of the rows [r0, r0 + count) of the padded table, count <= 32, that have no token, by one
// warp.  Padding rows, from tv.rows on, never have one.
__device__ __forceinline__ void zero_rows(const SumArgs& a, uint64_t r0, uint32_t count) {
    const uint32_t lane = threadIdx.x & 31;
    uint32_t has = 0;
    if (r0 < a.tv.rows) {
        const uint32_t real = uint32_t(min(uint64_t(count), a.tv.rows - r0));
        const uint32_t lo = first_at_least(a, uint32_t(r0), 0, a.n), hi = first_at_least(a, uint32_t(r0) + real, lo, a.n);
        if (lo < hi) {  // some of them do: each lane looks for its own
            uint32_t x = lo, y = hi;
            if (lane < real)
                while (x < y) {
                    const uint32_t mid = x + (y - x) / 2;
                    if (row_at(a, mid) < uint32_t(r0) + lane) x = mid + 1; else y = mid;
                }
            has = __ballot_sync(0xffffffffu, lane < real && x < hi && row_at(a, x) == uint32_t(r0) + lane);
        }
    }
    for (uint32_t k = 0; k < count; ++k) {
        if (has >> k & 1) continue;
        const uint64_t r = r0 + k;
        const uint32_t d = uint32_t(r / a.tv.m);
        zero_run(reinterpret_cast<float*>(shard_base(a.shards, d)) + a.tv.off + int64_t(r - uint64_t(d) * a.tv.m) * a.tv.len, a.tv.len);
    }
}

template <typename In, Layout kLayout, bool Add>
__global__ void __launch_bounds__(kThreads, kSumCtasPerSm) sum_positions_kernel(const __grid_constant__ SumArgs a) {
    constexpr int kWarps = kThreads / 32;
    __shared__ float stage[kWarps][kLayout == kMixed ? 32 * 9 : 1];
    extern __shared__ __align__(16) unsigned char rings[];
    const uint32_t warp = threadIdx.x >> 5;
    // the lane's 16 bytes of the warp's ring
    const uint32_t ring = uint32_t(__cvta_generic_to_shared(rings)) + warp * Ring<In>::kBytes + (threadIdx.x & 31) * 16;
    for (uint32_t b = blockIdx.x; b < a.sum_blocks + a.zero_blocks; b += gridDim.x) {
        if (b < a.sum_blocks) {
            const uint64_t item = uint64_t(b) * kWarps + warp;
            const uint32_t piece = uint32_t(item / a.stretches);
            if (piece < a.pieces) sum_piece<In, kLayout, Add>(a, piece, uint32_t(item - uint64_t(piece) * a.stretches), stage[warp], ring);
        } else {
            const uint64_t padded = uint64_t(a.tv.m) * a.tv.R;
            const uint64_t r0 = (uint64_t(b - a.sum_blocks) * kWarps + warp) * a.zero_rows;
            if (r0 < padded) zero_rows(a, r0, uint32_t(min(uint64_t(a.zero_rows), padded - r0)));
        }
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

GradPlan plan_grad(const TableView& tv, int64_t n) {
    GradPlan g;
    g.stretches = (tv.len + kStretch - 1) / kStretch;
    // shorter pieces while they would not fill the GPU's warps once
    g.piece = kPieceMost;
    while (g.piece > kPieceLeast && (n + g.piece - 1) / g.piece * g.stretches < kPieceWarps) g.piece >>= 1;
    g.pieces = uint32_t((n + g.piece - 1) / g.piece);
    g.slots = (int64_t(g.pieces) + (g.pieces + kBlock - 1) / kBlock) * 2 * g.stretches;
    return g;
}

size_t carve_grad_workspace(char* base, const TableView& tv, int64_t n, GradWorkspace* w) {
    const GradPlan p = plan_grad(tv, n);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* q = base + at;
        at += (bytes + 255) / 256 * 256;
        return q;
    };
    GradWorkspace g;
    g.sorted = reinterpret_cast<uint4*>(take(size_t(n) * 16));
    g.swap_a = reinterpret_cast<uint4*>(take(size_t(n) * 16));
    g.swap_b = reinterpret_cast<uint4*>(take(size_t(n) * 16));
    g.pre = reinterpret_cast<uint4*>(take(size_t(n) * 16));
    g.arrived = reinterpret_cast<uint32_t*>(take(size_t(p.slots) * 4));
    g.partial = reinterpret_cast<float*>(take(size_t(p.slots) * kStretch * 4));
    if (w) *w = g;
    return at;
}

cudaError_t launch_expand_positions(const Batches& b, uint32_t first, uint32_t rows, const GradWorkspace& w,
                                    int* status, cudaStream_t stream) {
    const uint32_t n = b.start[b.count];
    if (n == 0) return cudaSuccess;
    const int grid = int(std::min<uint32_t>((n + kThreads - 1) / kThreads, 1024u));
    expand_positions_kernel<<<grid, kThreads, 0, stream>>>(b, first, rows, w.pre, status);
    return cudaGetLastError();
}

cudaError_t launch_sort_positions(const Batches& b, bool expanded, const TableView& tv, uint32_t n,
                                  const GradWorkspace& w, int* status, cudaStream_t stream) {
    int bits = 0;
    while (tv.rows >> bits) ++bits;  // keys are 0 .. rows
    const GradPlan p = plan_grad(tv, n);
    SortArgs a{b, n, tv.rows, expanded ? 1 : 0, (bits + kSortMaxBits - 1) / kSortMaxBits, p.slots, w, status};
    const int digit = std::max(kSortMinBits, (bits + a.passes - 1) / a.passes);
    static_assert(kSortMinBits == 6 && kSortMaxBits == 10, "one kernel for each digit size");
    auto* kernel = digit == 6 ? sort_positions_kernel<6> : digit == 7 ? sort_positions_kernel<7> : digit == 8 ? sort_positions_kernel<8>
                   : digit == 9 ? sort_positions_kernel<9> : sort_positions_kernel<10>;
    uint32_t c = 1;
    while (c < kSortMaxCtas && n > c * kSortPerCta) c <<= 1;
    const size_t smem = (size_t(kSortWarps) + 1 + c) * (size_t(1) << digit) * 4;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = c;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch_sum_positions(const ShardPtrs& shards, const TableView& tv, uint32_t n, const GradWorkspace& w,
                                 int dout_bf16, bool dout_vec, float scale, bool accumulate, int ctas, bool overlap,
                                 cudaStream_t stream) {
    const GradPlan p = plan_grad(tv, n);
    SumArgs a{shards, tv, n, p.piece, p.pieces, p.stretches, w, scale, 0, 0, 1};
    const int64_t sums = (int64_t(p.pieces) * p.stretches + kThreads / 32 - 1) / (kThreads / 32);
    int64_t zeros = 0;
    if (!accumulate) {
        // one row to a warp, or up to 32 that make about 32 KB of zeros
        a.zero_rows = uint32_t(std::min<int64_t>(32, std::max<int64_t>(1, 8192 / tv.len)));
        zeros = (int64_t(tv.m) * tv.R + a.zero_rows * (kThreads / 32) - 1) / (a.zero_rows * (kThreads / 32));
    }
    if (sums + zeros > INT32_MAX) return cudaErrorInvalidValue;
    if (sums + zeros == 0) return cudaSuccess;
    a.sum_blocks = uint32_t(sums);
    a.zero_blocks = uint32_t(zeros);
    const int grid = int(std::min<int64_t>(sums + zeros, overlap ? ctas : INT32_MAX));
    const bool wide = tv.len % 8 == 0 && tv.off % 8 == 0 && shards.bits % 32 == 0;
    const Layout layout = !dout_vec || tv.len % 8 ? kSingle : wide ? kWide : kMixed;
    auto launch = [&](auto* kernel, uint32_t ring) {
        const int smem = int(ring * (kThreads / 32));
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        kernel<<<grid, kThreads, smem, stream>>>(a);
        return cudaGetLastError();
    };
    auto pick = [&](auto in, auto add) {
        using In = decltype(in);
        constexpr bool kAdd = decltype(add)::value;
        if (layout == kSingle) return launch(sum_positions_kernel<In, kSingle, kAdd>, 0);
        if (layout == kMixed) return launch(sum_positions_kernel<In, kMixed, kAdd>, Ring<In>::kBytes);
        return launch(sum_positions_kernel<In, kWide, kAdd>, Ring<In>::kBytes);
    };
    if (dout_bf16) return accumulate ? pick(__nv_bfloat16(), std::true_type()) : pick(__nv_bfloat16(), std::false_type());
    return accumulate ? pick(float(), std::true_type()) : pick(float(), std::false_type());
}

}  // namespace tide
