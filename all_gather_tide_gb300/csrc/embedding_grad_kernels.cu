// Gradient of the embedding lookup, summed by token into the packed dim-0 shards (sm_103a).
//
//     grad row t (+)= scale * sum of the dout rows of the positions that hold t
//
// The positions are sorted by row (stable, so that equal calls add in the same order) and each warp adds
// one stretch of the sorted list over 256 columns; short lists are sorted by every CTA for itself.  What
// bounds it is HBM: dout is read once, and either the whole piece of every shard is written or the
// rows that have a token are read and written.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "../../include/tide.h"
#include "embedding_device.cuh"

namespace cg = cooperative_groups;

namespace tide {
namespace {

// ---- sort of positions by row -----------------------------------------------------------------

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
// Bits of a digit: as few passes as 10 bits allow (their counts take 128 KB of shared memory), and of
// equal size; below 6 a pass gets no cheaper.
constexpr int kSortMinBits = 6, kSortMaxBits = 10;
// CTAs of the cluster, and positions for which the next ones join.  131072 positions sort in 54 us on 8 CTAs
// and in 34 on 16 (before counts were pushed; 25 since); gradients of 4000 positions of 1024 columns and 6273 of 704
// take 22.0 and 22.0 us with a CTA for every 1024, 23.1 and 23.2 for every 2048, 22.3 and 22.3 for every 512.
constexpr uint32_t kSortMaxCtas = 16, kSortPerCta = 1024;

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

// Sort of up to kRankMost positions: a position's place is the number of positions that come before it, of
// smaller rows or earlier with the same row.  Every CTA has all rows in shared memory and places
// kRankPositions of them, eight lanes to a position.  n^2 comparisons, but no passes and no barriers between
// CTAs: a gradient of 257, 1024 and 2048 positions takes 10.2, 15.2 and 18.8 us with this sort and 16.8, 21.9 and
// 24.7 with the one below (rows of 4096 columns); at 4096 positions it is 26.0 against 29.6, but 24.0 against 22.4
// where rows are short, and beyond it loses.
constexpr uint32_t kRankMost = 2048;
constexpr uint32_t kRankPositions = kThreads / 8;

struct SortArgs {
    Batches b;
    uint32_t n, rows;
    int expanded, passes;
    int64_t counters;
    GradWorkspace w;
    int* status;
};

__global__ void __launch_bounds__(kThreads) rank_positions_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ __align__(16) uint32_t rank_keys[];
    const uint32_t padded = (a.n + 31) & ~31u;
    wait_for_previous_kernel();
    // what the summing kernel finds cleared: its arrival counters
    for (int64_t q = int64_t(blockIdx.x) * kThreads + threadIdx.x; q < a.counters; q += int64_t(gridDim.x) * kThreads) a.w.arrived[q] = 0;
    constexpr int kAhead = 8;  // ids loaded before one is used
    for (uint32_t j0 = threadIdx.x; j0 < padded; j0 += kAhead * kThreads) {
        int64_t id[kAhead];
        int k = a.expanded || j0 >= a.n ? 0 : batch_of(a.b, j0);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const uint32_t j = j0 + u * kThreads;
            id[u] = -1;
            if (j >= a.n) continue;
            if (a.expanded) {
                id[u] = a.w.pre[j].z;
            } else {
                while (j >= a.b.start[k + 1]) ++k;
                id[u] = load_id(a.b.ids[k], a.b.ids64, j - a.b.start[k]);
            }
        }
        bool bad = false;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const uint32_t j = j0 + u * kThreads;
            bad |= id[u] >= int64_t(a.rows);
            if (j < padded) rank_keys[j] = j < a.n ? row_of(id[u], a.rows) : ~0u;  // behind every position
        }
        if (bad && !a.expanded && blockIdx.x == 0) atomicCAS(a.status, 0, kStatusBadId);
    }
    __syncthreads();
    // as many groups of positions as CTAs, but for a launch that may have few
    for (uint32_t first = blockIdx.x * kRankPositions; first < a.n; first += gridDim.x * kRankPositions) {
        const uint32_t i = first + threadIdx.x / 8, part = threadIdx.x & 7;
        const uint32_t key = rank_keys[min(i, a.n - 1)];
        uint32_t place = 0;
        for (uint32_t v = part; v < padded / 4; v += 8) {
            const uint4 o = *reinterpret_cast<const uint4*>(&rank_keys[4 * v]);
            if (v == i / 4) {
                place += (o.x < key + (4 * v < i)) + (o.y < key + (4 * v + 1 < i)) + (o.z < key + (4 * v + 2 < i)) + (o.w < key);
            } else {
                const uint32_t below = key + (v < i / 4);  // of earlier positions, equal rows come before too
                place += (o.x < below) + (o.y < below) + (o.z < below) + (o.w < below);
            }
        }
#pragma unroll
        for (int m = 4; m > 0; m >>= 1) place += __shfl_xor_sync(0xffffffffu, place, m);
        if (part == 0 && i < a.n) {
            uint64_t src;
            if (a.expanded) {
                const uint4 x = a.w.pre[i];
                src = uint64_t(x.y) << 32 | x.x;
            } else {
                const int k = batch_of(a.b, i);
                src = reinterpret_cast<uint64_t>(a.b.dout[k] + int64_t(i - a.b.start[k]) * a.b.stride[k]);
            }
            a.w.sorted[place] = make_uint4(uint32_t(src), uint32_t(src >> 32), key, 0);
        }
    }
    let_next_kernel_start();
}

// Stable radix sort, least significant digit first, by one cluster: each warp owns a contiguous run
// of positions, counts its digits, and places them in order behind the digits of smaller value and
// the same digit of earlier warps and CTAs.  The counts of the CTAs meet in distributed shared
// memory.  A batch of kSortBatch rounds of 32 positions is loaded at once; a run that is one batch
// stays in registers between counting and placing.
//
// 131072 positions of 128000 rows (two digits of 9 bits) take 25 us, 65536 take 18 us, 12289 take 12 us.
// Bound by the placing, a scattered 16-byte store for every position and pass from 16 SMs, and by a few
// barriers a pass.
constexpr int kSortBatch = 8;

template <int kBits>
__global__ void __launch_bounds__(kSortThreads, 1) sort_positions_kernel(const __grid_constant__ SortArgs a) {
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t C = cluster.num_blocks(), c = cluster.block_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int bins = 1 << kBits;
    extern __shared__ uint32_t sort_smem[];
    uint32_t* cnt = sort_smem;                   // [kSortWarps][bins]
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

    wait_for_previous_kernel();
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
                    if (i < hi) x = load_here((pass > 0 ? from : a.w.pre) + i);
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
        if (last) let_next_kernel_start();
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
//
// Bound by HBM: 65536 positions of 8192 bf16 columns into 128000 rows, 727 us for 5.26 GB (7.2 TB/s, most of
// it zeros written); 131072 of 4096 added to 128000 rows, 330 us for 2.10 GB (6.4 TB/s, reads and writes
// mixed); 60000 bf16 rows of 1001 columns, without alignment, added to 20000 rows, 72 us.  512 or 1024 columns to
// a warp took 411 and 461 us for the second where 256 took 400.
constexpr uint32_t kStretch = 256;
// Positions of a piece (plan_grad), and the warps that they have to keep busy: those of a GB300 at three
// CTAs an SM.
constexpr uint32_t kPieceMost = 64, kPieceLeast = 8;
constexpr int64_t kPieceWarps = 152 * 24;

// What the sums go to.
struct Target {
    ShardPtrs shards;
    TableView tv;
    uint32_t stretches;
    float scale;
    uint32_t sum_blocks;   // CTAs' worth of sums, before those that write zeros
    uint32_t zero_blocks;
    uint32_t zero_rows;    // rows of the padded table that one warp looks through for rows to zero
};

struct SumArgs : Target {
    GradWorkspace w;
    uint32_t n, piece, pieces;
};

__device__ __forceinline__ float* table_row(const Target& a, uint32_t t) {
    const uint32_t d = t / a.tv.m;
    return reinterpret_cast<float*>(shard_base(a.shards, d)) + a.tv.off + int64_t(t - d * a.tv.m) * a.tv.len;
}

// The table row of sorted position i (tv.rows: no token).
__device__ __forceinline__ uint32_t row_at(const SumArgs& a, uint32_t i) { return a.w.sorted[i].z; }

// How a warp's 256 columns lie over its lanes: every 32nd element (kShifted, where dout rows have no 16-byte
// alignment), or so that 16 bytes of dout are one lane's and the next 16 the next lane's, the rows in the shard
// being 32-byte aligned (kWide) or not (kMixed).
enum Layout { kShifted, kMixed, kWide };

// A lane's 8 columns of a dout row, 16 bytes of bf16 or twice 16 bytes of fp32 (512 bytes apart, so that a
// warp's copies cover whole lines), copied to shared memory asynchronously: what is in flight takes no
// registers.  Each lane copies and reads its own bytes only.
template <typename In>
struct Part {
    static constexpr int kWords = sizeof(In) / 2;           // of 16 bytes
    static constexpr int kEach = 8 / kWords;                // columns of one
    static constexpr uint32_t kApart = 256 / kWords;        // columns from one to the next
    uint4 w[kWords];

    // The lane's j-th column of 256.
    static __device__ __forceinline__ uint32_t column(uint32_t lane, int j) { return j / kEach * kApart + lane * kEach + j % kEach; }
    // from: the lane's first column, of which, counted from it, `left` (may be negative) are the row's.
    static __device__ __forceinline__ void copy(uint32_t to, uint64_t from, int left) {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            if (int(i * kApart) < left) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 512), "l"(from + i * 512) : "memory");
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

// Rows of dout in flight for a warp: groups of copies.  A shifted row lies in the ring as it does between
// 16-byte boundaries.  Measured in us, shifted (60000 bf16 rows of 1001 columns added to 20000, and 127618 of 1123
// written to 39540): 3 groups of 4 rows 90 and 125, 4 of 2 87 and 116, 3 of 2 85 and 115, 8 of 1 84 and 115, but for
// fp32 rows 114 where 3 of 1 takes 106; loads of single elements instead 110 and 117.  Aligned (131072 rows of 4096
// added to 128000, 48042 of 1368 to 1552): 3 groups of 4 362 and 64.8, 8 of 1 361 and 63.5.
template <typename In, Layout kLayout>
struct Ring {
    static constexpr int kGroups = kLayout == kShifted ? 3 : 8, kGroup = kLayout == kShifted ? 4 / sizeof(In) : 1, kRows = kGroup * kGroups;
    static constexpr uint32_t kRow = kStretch * sizeof(In) + (kLayout == kShifted ? 16 : 0), kBytes = kRows * kRow;
};

// Adds a stretch of `count` rows of dout to acc, in order: src(k) is the k-th row's address, low(k) its low 32
// bits, and turn(k) is called before the k-th is added.  `ring`: the lane's place in the warp's shared memory.
template <typename In, Layout kLayout, typename Src, typename Low, typename Turn>
__device__ __forceinline__ void add_rows(int count, uint32_t stretch, uint32_t len, uint32_t ring, Src src, Low low, Turn turn, float (&acc)[8]) {
    using R = Ring<In, kLayout>;
    if constexpr (kLayout == kShifted) {
        const uint32_t lane = threadIdx.x & 31, first = stretch * kStretch, bytes = min(kStretch, len - first) * sizeof(In);
        ring -= lane * 16;
        auto slot = [&](int k) { return ring + uint32_t(k) % R::kRows * R::kRow; };
        auto fetch = [&](int k) {
#pragma unroll
            for (int u = 0; u < R::kGroup; ++u) {
                const uint64_t from = src(k + u);
                if (k + u < count) copy_shifted<kStretch * sizeof(In)>(slot(k + u), from + uint64_t(first) * sizeof(In), bytes);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int k = 0; k < R::kRows; k += R::kGroup) fetch(k);
        for (int k = 0; k < count; k += R::kGroup) {
            asm volatile("cp.async.wait_group %0;" ::"n"(R::kGroups - 1) : "memory");
            __syncwarp();  // lanes read what others copied
#pragma unroll
            for (int u = 0; u < R::kGroup; ++u) {
                const uint32_t at = slot(k + u) + ((low(k + u) + first * uint32_t(sizeof(In))) & 15) + lane * uint32_t(sizeof(In));
                if (k + u >= count) break;
                turn(k + u);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] += load_shared(at + 32 * j * uint32_t(sizeof(In)), In());
            }
            __syncwarp();
            fetch(k + R::kRows);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    } else {
        const uint32_t col = stretch * kStretch + Part<In>::column(threadIdx.x & 31, 0);
        const int left = int(len) - int(col);
        auto slot = [&](int k) { return ring + uint32_t(k) % R::kRows * R::kRow; };
        auto fetch = [&](int k) {
#pragma unroll
            for (int u = 0; u < R::kGroup; ++u) {
                const uint64_t from = src(k + u);
                if (k + u < count) Part<In>::copy(slot(k + u), from + uint64_t(col) * sizeof(In), left);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int k = 0; k < R::kRows; k += R::kGroup) fetch(k);
        for (int k = 0; k < count; k += R::kGroup) {
            asm volatile("cp.async.wait_group %0;" ::"n"(R::kGroups - 1) : "memory");
            Part<In> x[R::kGroup];
#pragma unroll
            for (int u = 0; u < R::kGroup; ++u) x[u].read(slot(k + u));
#pragma unroll
            for (int u = 0; u < R::kGroup; ++u) {
                if (k + u >= count) break;
                turn(k + u);
                x[u].add(acc);
            }
            fetch(k + R::kRows);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
}

// What a stretch of a row, dst, holds, as the layout spreads its columns over the lanes; `left` columns of the
// row lie from dst on.
template <typename In, Layout kLayout>
__device__ __forceinline__ void read_row(const float* dst, uint32_t left, float (&y)[8]) {
    using P = Part<In>;
    const uint32_t lane = threadIdx.x & 31;
    if constexpr (kLayout == kWide && P::kWords == 1) {
        if (lane * 8 < left) load_v8(dst + lane * 8, y);
    } else if constexpr (kLayout == kWide) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (P::column(lane, 4 * i) >= left) continue;
            const float4 v = *reinterpret_cast<const float4*>(dst + P::column(lane, 4 * i));
            y[4 * i] = v.x, y[4 * i + 1] = v.y, y[4 * i + 2] = v.z, y[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (lane + 32 * j < left) y[j] = dst[lane + 32 * j];
    }
}

// The warp's sums, scaled and added to y, to a stretch of a row: `acc` as the layout spreads them, y as read_row
// read it (or zeros).
template <typename In, Layout kLayout>
__device__ __forceinline__ void write_row(float scale, float* dst, uint32_t left, const float (&acc)[8], const float (&y)[8], float* stage) {
    using P = Part<In>;
    const uint32_t lane = threadIdx.x & 31;
    float x[8];
    if constexpr (kLayout == kMixed) {  // turned round so that stores of single elements lie side by side
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) stage[P::column(lane, j) + P::column(lane, j) / 8] = acc[j];
        __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t q = lane + 32 * j;
        x[j] = y[j] + scale * (kLayout == kMixed ? stage[q + q / 8] : acc[j]);
    }
    if constexpr (kLayout == kWide && P::kWords == 1) {
        if (lane * 8 < left) store_v8(dst + lane * 8, x);
    } else if constexpr (kLayout == kWide) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (P::column(lane, 4 * i) < left) __stcs(reinterpret_cast<float4*>(dst + P::column(lane, 4 * i)), make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (lane + 32 * j < left) dst[lane + 32 * j] = x[j];
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

// Through L2 both ways: another SM reads what one wrote.
__device__ __forceinline__ void put_partial(float* p, const float (&x)[8]) {
    asm volatile("st.global.cg.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                 "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
}
__device__ __forceinline__ void get_partial(const float* p, float (&x)[8]) {
    asm volatile("ld.global.cg.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                 : "l"(p)
                 : "memory");
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
        float y[8];
        get_partial(partial_of(a, x + k, k == 0 ? first_starts : 0, stretch), y);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += y[j];
    }
}

// After a piece has left a partial sum of row t: the last of the row's pieces in this block adds
// the block's, and the last of its blocks adds the blocks', both in order, and writes the row.
template <typename In, Layout kLayout, bool Add>
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
    const uint32_t left = a.tv.len - stretch * kStretch;
    float* dst = table_row(a, t) + stretch * kStretch;
    float old[8] = {};
    if (Add) read_row<In, kLayout>(dst, left, old);
    write_row<In, kLayout>(a.scale, dst, left, sum, old, stage);
}

// The running sum of one piece.
template <typename In, Layout kLayout, bool Add>
struct Run {
    const SumArgs& a;
    uint32_t piece, stretch, before, after;  // rows on either side of the piece
    float* stage;
    float acc[8] = {}, old[8] = {};
    uint32_t cur = ~0u;    // the row being summed
    float* dst = nullptr;  // its stretch in the shard
    bool starts = true;    // in this piece
    uint32_t head = ~0u;   // the row that an earlier piece began and this one ended

    __device__ __forceinline__ void write() { write_row<In, kLayout>(a.scale, dst, a.tv.len - stretch * kStretch, acc, old, stage); }

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
        // What this piece will write alone is read before the row's positions are awaited: 60000 rows of 1001
        // columns added 78 us, 85 if read where it is written.  Read as early as the dout rows are copied, or
        // prefetched, it takes longer (131072 rows of 4096: 400 to 420 us where reading it last took 371).
        if (Add && starts && t != after) read_row<In, kLayout>(dst, a.tv.len - stretch * kStretch, old);
    }

    __device__ __forceinline__ void finish() {
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
            if (t != ~0u) join_partials<In, kLayout, Add>(a, t, piece, stretch, stage);
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
    const uint4 p0 = lo + lane < hi ? a.w.sorted[lo + lane] : none, p1 = lo + 32 + lane < hi ? a.w.sorted[lo + 32 + lane] : none;
    const int held = __popc(__ballot_sync(0xffffffffu, p0.z < a.tv.rows)) + __popc(__ballot_sync(0xffffffffu, p1.z < a.tv.rows));
    auto of = [&](int k, auto x0, auto x1) { return __shfl_sync(0xffffffffu, k < 32 ? x0 : x1, k & 31); };
    // where their rows lie in the shards, worked out by each lane for its own
    const auto d0 = reinterpret_cast<unsigned long long>(p0.z < a.tv.rows ? table_row(a, p0.z) + stretch * kStretch : nullptr);
    const auto d1 = reinterpret_cast<unsigned long long>(p1.z < a.tv.rows ? table_row(a, p1.z) + stretch * kStretch : nullptr);
    Run<In, kLayout, Add> run{a, piece, stretch, lo > 0 ? row_at(a, lo - 1) : ~0u, hi < a.n ? row_at(a, hi) : ~0u, stage};
    add_rows<In, kLayout>(
        held, stretch, a.tv.len, ring, [&](int k) { return uint64_t(of(k, p0.y, p1.y)) << 32 | of(k, p0.x, p1.x); }, [&](int k) { return of(k, p0.x, p1.x); },
        [&](int k) {
            const uint32_t t = of(k, p0.z, p1.z);
            if (t != run.cur) run.turn_to(t, reinterpret_cast<float*>(of(k, d0, d1)));
        },
        run.acc);
    run.finish();
}

// Zeros from p on, n elements, by one warp: 32-byte stores between single ones at the ends.
__device__ __forceinline__ void zero_run(float* p, uint64_t n) {
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t head = uint32_t(min(n, uint64_t((8u - (unsigned(reinterpret_cast<uintptr_t>(p) / 4) & 7u)) & 7u)));
    const float z[8] = {};
    if (lane < head) p[lane] = 0.0f;
    const uint64_t vecs = (n - head) / 8;
    for (uint64_t v = lane; v < vecs; v += 32) store_v8(p + head + v * 8, z);
    for (uint64_t i = head + vecs * 8 + lane; i < n; i += 32) p[i] = 0.0f;
}

// The first of the sorted positions [lo, hi) whose row is >= r (hi if none), found by the whole warp, 32
// places at a time: the last positions of the first 32 of 33 parts.  The 33rd part's is not looked at, so where all
// 32 lie below r (k = 32) nothing is known of it and hi stays.
__device__ __forceinline__ uint32_t first_at_least(const uint4* sorted, uint32_t r, uint32_t lo, uint32_t hi) {
    const uint32_t lane = threadIdx.x & 31;
    while (lo < hi) {
        const uint32_t step = (hi - lo + 32) / 33;  // lane k looks at the last position of the k-th part
        const uint64_t x = uint64_t(lo) + uint64_t(lane + 1) * step - 1;
        const uint32_t below = __ballot_sync(0xffffffffu, x < hi && sorted[x].z < r);
        const uint32_t k = __popc(below);  // sorted: a prefix of the lanes
        const uint64_t end = uint64_t(lo) + uint64_t(k + 1) * step - 1;
        lo += k * step;
        if (k < 32 && end < hi) hi = uint32_t(end);
    }
    return lo;
}

// Zeros to those of the rows [r0, r0 + zero_rows) of the padded table that have none of the n sorted
// positions, by one warp.  Padding rows, from tv.rows on, never have one.
__device__ __forceinline__ void zero_rows(const Target& a, uint64_t r0, const uint4* sorted, uint32_t n) {
    const uint64_t padded = uint64_t(a.tv.m) * a.tv.R;
    if (r0 >= padded) return;
    const uint32_t lane = threadIdx.x & 31, count = uint32_t(min(uint64_t(a.zero_rows), padded - r0));
    uint32_t has = 0;
    if (r0 < a.tv.rows) {
        const uint32_t real = uint32_t(min(uint64_t(count), a.tv.rows - r0));
        const uint32_t lo = first_at_least(sorted, uint32_t(r0), 0, n), hi = first_at_least(sorted, uint32_t(r0) + real, lo, n);
        if (lo < hi) {  // some of them do: each lane looks for its own
            uint32_t x = lo, y = hi;
            if (lane < real)
                while (x < y) {
                    const uint32_t mid = x + (y - x) / 2;
                    if (sorted[mid].z < uint32_t(r0) + lane) x = mid + 1; else y = mid;
                }
            has = __ballot_sync(0xffffffffu, lane < real && x < hi && sorted[x].z == uint32_t(r0) + lane);
        }
    }
    // run after run of such rows that lie side by side in one shard, each as one: row by row, 3000 positions into
    // 128000 x 64 take 43 us instead of 26
    uint32_t left = ~has & (~0u >> (32 - count));
    while (left) {
        const uint32_t first = __ffs(left) - 1, taken = ~(left >> first);
        const uint64_t r = r0 + first;
        const uint32_t d = uint32_t(r / a.tv.m), row = uint32_t(r - uint64_t(d) * a.tv.m);
        const uint32_t run = min(taken ? __ffs(taken) - 1 : 32u, a.tv.m - row);
        zero_run(reinterpret_cast<float*>(shard_base(a.shards, d)) + a.tv.off + int64_t(row) * a.tv.len, uint64_t(run) * a.tv.len);
        left &= ~((~0u >> (32 - run)) << first);
    }
}

// Dynamic shared memory of a CTA of sums: the warps' rings, and for kMixed what write_row turns the columns
// round in.
template <typename In, Layout kLayout>
constexpr uint32_t kSumSmem = kWarps * (Ring<In, kLayout>::kBytes + (kLayout == kMixed ? 32 * 9 * 4 : 0));

template <typename In, Layout kLayout>
__device__ __forceinline__ void sum_smem(unsigned char* smem, uint32_t* ring, float** stage) {
    const uint32_t warp = threadIdx.x >> 5;
    *ring = uint32_t(__cvta_generic_to_shared(smem)) + warp * Ring<In, kLayout>::kBytes + (threadIdx.x & 31) * 16;
    *stage = reinterpret_cast<float*>(smem + kWarps * Ring<In, kLayout>::kBytes) + warp * (32 * 9);
}

// CTAs of an SM that registers leave room for: 4, except where 3 measured faster (65536 positions into
// 128000 x 8192, most of it zeros to write: 753 us with 3, 780 with 4; 131072 added to 128000 x 4096: 377
// with 3, 363 with 4; 60000 bf16 rows of 4099 columns into 128000: 462 with 3, 453 with 4).
template <Layout kLayout, bool Add>
constexpr int kSumCtas = Add || kLayout == kShifted ? kSumCtasPerSm : 3;

template <typename In, Layout kLayout, bool Add>
__global__ void __launch_bounds__(kThreads, kSumCtas<kLayout, Add>) sum_positions_kernel(const __grid_constant__ SumArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    uint32_t ring;
    float* stage;
    sum_smem<In, kLayout>(smem, &ring, &stage);
    wait_for_previous_kernel();
    for (uint32_t b = blockIdx.x; b < a.sum_blocks + a.zero_blocks; b += gridDim.x) {
        if (b < a.sum_blocks) {
            const uint64_t item = uint64_t(b) * kWarps + (threadIdx.x >> 5);
            const uint32_t piece = uint32_t(item / a.stretches);
            if (piece < a.pieces) sum_piece<In, kLayout, Add>(a, piece, uint32_t(item - uint64_t(piece) * a.stretches), stage, ring);
        } else {
            zero_rows(a, (uint64_t(b - a.sum_blocks) * kWarps + (threadIdx.x >> 5)) * a.zero_rows, a.w.sorted, a.n);
        }
    }
    let_next_kernel_start();
}

// ---- short lists ----------------------------------------------------------------------------------
//
// Up to kShortMost positions: one launch instead of two, no workspace.  Every CTA sorts the list for
// itself (each position's place is the number of positions that come before it: n^2 comparisons in
// shared memory), and one warp adds all positions of one row.  Bound by latency: 64 positions of 256
// columns 4.0 us, 256 of 256 and of 4096 columns 6.3 and 10.9 us; the two launches for 257 take 10.1 and 10.2.
constexpr uint32_t kShortMost = kThreads;

struct ShortArgs : Target {
    Batches b;
    uint32_t n;
    int* status;
};

template <typename In, Layout kLayout, bool Add>
__global__ void __launch_bounds__(kThreads, kShortCtasPerSm) sum_short_kernel(const __grid_constant__ ShortArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ __align__(16) uint32_t keys[kShortMost];
    __shared__ uint4 sorted[kShortMost];
    uint32_t ring;
    float* stage;
    sum_smem<In, kLayout>(smem, &ring, &stage);
    const uint32_t i = threadIdx.x;
    uint32_t key = ~0u;
    uint64_t src = 0;
    wait_for_previous_kernel();
    if (i < a.n) {
        const int k = batch_of(a.b, i);
        const uint32_t j = i - a.b.start[k];
        const int64_t id = load_id(a.b.ids[k], a.b.ids64, j);
        if (blockIdx.x == 0 && id >= int64_t(a.tv.rows)) atomicCAS(a.status, 0, kStatusBadId);
        key = row_of(id, a.tv.rows);
        src = reinterpret_cast<uint64_t>(a.b.dout[k] + int64_t(j) * a.b.stride[k]);
    }
    keys[i] = key;
    __syncthreads();
    uint32_t place = 0;
    for (uint32_t j = 0; j < a.n; j += 4) {
        const uint4 o = *reinterpret_cast<const uint4*>(&keys[j]);  // ~0 from n on: behind every position
        place += (o.x < key + (j < i)) + (o.y < key + (j + 1 < i)) + (o.z < key + (j + 2 < i)) + (o.w < key + (j + 3 < i));
    }
    if (i < a.n) sorted[place] = make_uint4(uint32_t(src), uint32_t(src >> 32), key, 0);
    __syncthreads();

    const uint32_t lane = threadIdx.x & 31;
    for (uint32_t b = blockIdx.x; b < a.sum_blocks + a.zero_blocks; b += gridDim.x) {
        if (b >= a.sum_blocks) {
            zero_rows(a, (uint64_t(b - a.sum_blocks) * kWarps + (threadIdx.x >> 5)) * a.zero_rows, sorted, a.n);
            continue;
        }
        const uint64_t item = uint64_t(b) * kWarps + (threadIdx.x >> 5);
        if (item >= uint64_t(a.n) * a.stretches) continue;
        const uint32_t p = uint32_t(item / a.stretches), stretch = uint32_t(item - uint64_t(p) * a.stretches);
        const uint32_t t = sorted[p].z;
        if (t >= a.tv.rows || (p > 0 && sorted[p - 1].z == t)) continue;  // the row's first position has it
        uint32_t end = p + 1;
        for (bool more = true; more;) {
            const uint32_t out = ~__ballot_sync(0xffffffffu, end + lane < a.n && sorted[end + lane].z == t);
            end += out ? __ffs(out) - 1 : 32;
            more = out == 0;
        }
        const uint32_t left = a.tv.len - stretch * kStretch;
        float* dst = table_row(a, t) + stretch * kStretch;
        float acc[8] = {}, old[8] = {};
        if (Add) read_row<In, kLayout>(dst, left, old);
        add_rows<In, kLayout>(
            int(end - p), stretch, a.tv.len, ring,
            [&](int k) {
                const uint4 x = sorted[min(p + k, a.n - 1)];
                return uint64_t(x.y) << 32 | x.x;
            },
            [&](int k) { return sorted[min(p + k, a.n - 1)].x; },
            [](int) {}, acc);
        write_row<In, kLayout>(a.scale, dst, left, acc, old, stage);
    }
    let_next_kernel_start();
}

// Sets a kernel's attributes once for each device.
template <typename F>
cudaError_t once_per_device(std::atomic<uint64_t> (&done)[4], F&& set) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    std::atomic<uint64_t>& word = done[(dev >> 6) & 3];
    if (dev < 256 && (word.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = set();
    if (e == cudaSuccess && dev < 256) word.fetch_or(bit, std::memory_order_release);
    return e;
}

template <typename In, Layout kLayout, bool Add>
cudaError_t launch_sum(const SumArgs& a, int grid, cudaStream_t stream) {
    static std::atomic<uint64_t> done[4];
    auto* kernel = sum_positions_kernel<In, kLayout, Add>;
    constexpr uint32_t smem = kSumSmem<In, kLayout>;
    cudaError_t e = once_per_device(done, [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)); });
    if (e != cudaSuccess) return e;
    return launch_after(kernel, grid, kThreads, smem, stream, a);
}

template <typename In, Layout kLayout, bool Add>
cudaError_t launch_short(const ShortArgs& a, int grid, cudaStream_t stream) {
    static std::atomic<uint64_t> done[4];
    auto* kernel = sum_short_kernel<In, kLayout, Add>;
    constexpr uint32_t smem = kSumSmem<In, kLayout>;
    cudaError_t e = once_per_device(done, [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)); });
    if (e != cudaSuccess) return e;
    return launch_after(kernel, grid, kThreads, smem, stream, a);
}

// Calls launch.template operator()<In, kLayout, Add>() for the call's types and alignments.
template <typename F>
cudaError_t with_kinds(const Target& a, int dout_bf16, bool dout_vec, bool accumulate, F&& launch) {
    const bool wide = a.tv.len % 8 == 0 && a.tv.off % 8 == 0 && a.shards.bits % 32 == 0;
    const Layout layout = !dout_vec || a.tv.len % 8 ? kShifted : wide ? kWide : kMixed;
    auto with_add = [&](auto in, auto add) {
        if (layout == kShifted) return launch(in, std::integral_constant<Layout, kShifted>(), add);
        if (layout == kMixed) return launch(in, std::integral_constant<Layout, kMixed>(), add);
        return launch(in, std::integral_constant<Layout, kWide>(), add);
    };
    if (dout_bf16) return accumulate ? with_add(__nv_bfloat16(), std::true_type()) : with_add(__nv_bfloat16(), std::false_type());
    return accumulate ? with_add(float(), std::true_type()) : with_add(float(), std::false_type());
}

// CTAs of sums and of zeros; false if they are more than a grid holds.
bool cut_blocks(Target* a, int64_t items, bool accumulate) {
    const int64_t sums = (items + kWarps - 1) / kWarps;
    int64_t zeros = 0;
    a->zero_rows = 1;
    if (!accumulate) {
        // one row to a warp, or up to 32 that make about 16 KB of zeros while the GPU's warps stay busy (12289
        // positions into 50021 x 1027: 59.2 us, with 32 KB 61.2, 64 KB 62.9, 8 KB 67.7; 277 into 118412 x 232:
        // 23.4, 30.0, 30.4, 25.7)
        const int64_t padded = int64_t(a->tv.m) * a->tv.R;
        a->zero_rows = uint32_t(std::max<int64_t>(1, std::min<int64_t>({32, 4096 / a->tv.len, padded / kPieceWarps})));
        zeros = (padded + a->zero_rows * kWarps - 1) / (a->zero_rows * kWarps);
    }
    if (sums + zeros > INT32_MAX) return false;
    a->sum_blocks = uint32_t(sums);
    a->zero_blocks = uint32_t(zeros);
    return true;
}

}  // namespace

GradPlan plan_grad(const TableView& tv, int64_t n) {
    GradPlan g;
    g.stretches = (tv.len + kStretch - 1) / kStretch;
    // Shorter pieces, which end together, while the GPU's warps go round fewer than six times; still shorter ones,
    // which leave more partial sums, only while they do not all have one, and the shortest while an SM has
    // fewer than seven.  In us with 64, 32, 16, 8 positions (warps with 32): 60000 bf16 positions of 1001 columns
    // added (7500) 84, 74, 79, 92; 20000 of 2048 written (5000) 65, 66, 70, 77; 12289 fp32 of 1027 written (1925) 69,
    // 63, 59, 59; 6000 of 4096 added (3008) -, 40, 36, 38; 6273 of 704 written (588) -, 27, 23, 25; 1024 of 4096
    // added (512) -, 19, 16, 15.
    auto items = [&] { return (n + g.piece - 1) / g.piece * g.stretches; };
    g.piece = kPieceMost;
    if (items() < 6 * kPieceWarps) g.piece = 32;
    if (items() < kPieceWarps) g.piece = 16;
    if (items() < 152 * 7) g.piece = kPieceLeast;
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

size_t grad_workspace_size(const TableView& tv, int64_t n) {
    // A size grows with n as long as the pieces keep their length, and falls where they get longer and leave fewer
    // partial sums; so the largest is that of n or of the last list with a shorter length.
    size_t most = carve_grad_workspace(nullptr, tv, n, nullptr);
    for (uint32_t piece = kPieceLeast; piece < plan_grad(tv, n).piece; piece *= 2) {
        int64_t lo = 0, hi = n;  // pieces of lo positions are this long at most, of hi longer
        while (hi - lo > 1) {
            const int64_t mid = lo + (hi - lo) / 2;
            if (plan_grad(tv, mid).piece <= piece) lo = mid; else hi = mid;
        }
        most = std::max(most, carve_grad_workspace(nullptr, tv, lo, nullptr));
    }
    return most;
}

cudaError_t launch_expand_positions(const Batches& b, uint32_t first, uint32_t rows, const GradWorkspace& w, int ctas,
                                    int* status, cudaStream_t stream) {
    const uint32_t n = b.start[b.count];
    if (n == 0) return cudaSuccess;
    const int grid = int(std::min<uint32_t>((n + kThreads - 1) / kThreads, uint32_t(ctas)));
    expand_positions_kernel<<<grid, kThreads, 0, stream>>>(b, first, rows, w.pre, status);
    return cudaGetLastError();
}

namespace {

template <int kBits>
cudaError_t launch_sort(const SortArgs& a, uint32_t ctas, cudaStream_t stream) {
    static std::atomic<uint64_t> done[4];
    auto* kernel = sort_positions_kernel<kBits>;
    auto smem = [](uint32_t c) { return (size_t(kSortWarps) + 1 + c) * (size_t(1) << kBits) * 4; };
    const cudaError_t e = once_per_device(done, [&] {
        const cudaError_t s = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem(kSortMaxCtas)));
        return s != cudaSuccess ? s : cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = smem(ctas);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_sort_positions(const Batches& b, bool expanded, const TableView& tv, uint32_t n,
                                  const GradWorkspace& w, int ctas, int* status, cudaStream_t stream) {
    int bits = 0;
    while (tv.rows >> bits) ++bits;  // keys are 0 .. rows
    SortArgs a{b, n, tv.rows, expanded ? 1 : 0, (bits + kSortMaxBits - 1) / kSortMaxBits, plan_grad(tv, n).slots, w, status};
    if (n <= kRankMost)
        return launch_after(rank_positions_kernel, std::min(int((n + kRankPositions - 1) / kRankPositions), ctas), kThreads,
                            ((size_t(n) + 31) & ~size_t(31)) * 4, stream, a);
    uint32_t cluster = 1;
    while (cluster < kSortMaxCtas && 2 * cluster <= uint32_t(ctas) && n > cluster * kSortPerCta) cluster <<= 1;
    static_assert(kSortMinBits == 6 && kSortMaxBits == 10, "one kernel for each digit size");
    switch (std::max(kSortMinBits, (bits + a.passes - 1) / a.passes)) {
        case 6: return launch_sort<6>(a, cluster, stream);
        case 7: return launch_sort<7>(a, cluster, stream);
        case 8: return launch_sort<8>(a, cluster, stream);
        case 9: return launch_sort<9>(a, cluster, stream);
        default: return launch_sort<10>(a, cluster, stream);
    }
}

cudaError_t launch_sum_positions(const ShardPtrs& shards, const TableView& tv, uint32_t n, const GradWorkspace& w,
                                 int dout_bf16, bool dout_vec, float scale, bool accumulate, int ctas, bool overlap,
                                 cudaStream_t stream) {
    const GradPlan p = plan_grad(tv, n);
    SumArgs a{{shards, tv, p.stretches, scale}, w, n, p.piece, p.pieces};
    if (!cut_blocks(&a, int64_t(p.pieces) * p.stretches, accumulate)) return cudaErrorInvalidValue;
    const int64_t blocks = int64_t(a.sum_blocks) + a.zero_blocks;
    if (blocks == 0) return cudaSuccess;
    const int grid = int(std::min<int64_t>(blocks, overlap ? ctas : INT32_MAX));
    return with_kinds(a, dout_bf16, dout_vec, accumulate, [&](auto in, auto layout, auto add) {
        return launch_sum<decltype(in), decltype(layout)::value, decltype(add)::value>(a, grid, stream);
    });
}

static_assert(kShortMost == TIDE_SHORT_POSITIONS && kInlineBatches == TIDE_SHORT_BATCHES, "what the header promises");
bool short_list(int64_t n, int32_t batches) { return n > 0 && n <= int64_t(kShortMost) && batches <= kInlineBatches; }

cudaError_t launch_sum_short(const ShardPtrs& shards, const TableView& tv, const Batches& b, uint32_t n, int dout_bf16,
                             bool dout_vec, float scale, bool accumulate, int ctas, int* status, cudaStream_t stream) {
    ShortArgs a{{shards, tv, (tv.len + kStretch - 1) / kStretch, scale}, b, n, status};
    if (!cut_blocks(&a, int64_t(n) * a.stretches, accumulate)) return cudaErrorInvalidValue;
    // no more CTAs than fit at once: each sorts the list
    const int grid = int(std::min<int64_t>(int64_t(a.sum_blocks) + a.zero_blocks, ctas));
    return with_kinds(a, dout_bf16, dout_vec, accumulate, [&](auto in, auto layout, auto add) {
        return launch_short<decltype(in), decltype(layout)::value, decltype(add)::value>(a, grid, stream);
    });
}

}  // namespace tide
