// Tokens sorted by expert and back, with the router's weights, and the gradients (sm_103a).
//
// Pair i = t*k + j is choice j of token t.  The stable order by expert puts pair i at row
//     slot[i] = offsets[id_i] + |{i' < i: id_i' = id_i}|,    offsets[e] = |{i: id_i < e}|.
#include <algorithm>

#include "experts_device.cuh"

namespace tide {
namespace {

constexpr int kSortWarps = kSortThreads / 32;
constexpr int kCtasPerSm = 4;  // of 256 threads

constexpr int kSteps = 8;  // of 32 pairs, whose ids a warp loads at once

// The experts of 32*kSteps pairs from `first` on, E where there is none.
__device__ __forceinline__ void load_experts(int (&e)[kSteps], const void* ids, int ids64, int64_t first, int64_t end, int E, int* status) {
    int64_t id[kSteps];
#pragma unroll
    for (int q = 0; q < kSteps; ++q) {
        const int64_t i = first + q * 32 + (threadIdx.x & 31);
        id[q] = i < end ? load_id(ids, ids64, i) : -1;
    }
#pragma unroll
    for (int q = 0; q < kSteps; ++q) {
        if (status && id[q] >= E) atomicCAS(status, 0, kStatusBadId);
        e[q] = int(row_of(id[q], uint32_t(E)));
    }
}

// How many pairs of its piece go to each expert, for every CTA.
__global__ void __launch_bounds__(kSortThreads) count_experts_kernel(const void* ids, int ids64, int32_t n, int32_t piece, int E, int32_t* counts, int* status) {
    __shared__ int32_t count[TIDE_MAX_EXPERTS + 1];
    for (int e = threadIdx.x; e <= E; e += kSortThreads) count[e] = 0;
    wait_for_previous_kernel();
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * piece, end = min(first + piece, int64_t(n));
    for (int64_t i = first + (threadIdx.x >> 5) * (32 * kSteps); i < end; i += kSortWarps * 32 * kSteps) {
        int e[kSteps];
        load_experts(e, ids, ids64, i, end, E, status);
#pragma unroll
        for (int q = 0; q < kSteps; ++q)
            if (e[q] < E) atomicAdd(&count[e[q]], 1);
    }
    __syncthreads();
    let_next_kernel_start();
    for (int e = threadIdx.x; e < E; e += kSortThreads) counts[int64_t(blockIdx.x) * E + e] = count[e];
}

// The rows of a piece's pairs.  Each warp has a stretch of the piece.  It first counts its pairs by expert, 32 at a time: lanes
// with the same expert find one another (match) and their first adds their number, so no atomics are needed.
// The counts of the warps before it, of the CTAs before and of all experts before give the row of its first
// pair of each expert, and a second pass over the stretch, the same way, the row of every pair. What the other CTAs have
// counted lies in their shared memory, where all are one cluster, and else in `counts`.
//
// Bound by latency, not by its 12 or 16 bytes a pair.
__global__ void __launch_bounds__(kSortThreads)
sort_experts_kernel(const void* ids, int ids64, int32_t n, int32_t piece, int k, int E, const int32_t* counts, int32_t* offsets, int32_t* slots,
                    int32_t* tokens, int* status) {
    extern __shared__ int32_t smem[];
    int32_t* base = smem;                      // [E + 1] rows before each expert
    int32_t* own = base + E + 1;               // [E] pairs of this CTA
    int32_t* before = own + E;                 // [E] pairs of the CTAs before
    int32_t* total = before + E;               // [E] pairs of all CTAs
    int32_t* warp_count = total + E;           // [kSortWarps][E + 1]
    __shared__ int32_t sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool cluster = !counts && gridDim.x > 1;
    int32_t* mine = warp_count + warp * (E + 1);
    for (int e = threadIdx.x; e < E; e += kSortThreads) before[e] = total[e] = 0;
    for (int e = lane; e <= E; e += 32) mine[e] = 0;
    wait_for_previous_kernel();
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * piece, end = min(first + piece, int64_t(n));
    const int64_t stretch = ((end - first + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const int64_t lo = min(first + warp * stretch, end), hi = min(lo + stretch, end);
    // ids past the experts are recorded once: by the counting kernel, if there was one
    int* const bad = counts ? nullptr : status;
    int e[kSteps];  // of a stretch of one batch they stay for the second pass
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kSteps) {
        load_experts(e, ids, ids64, i0, hi, E, bad);
#pragma unroll
        for (int q = 0; q < kSteps; ++q) {
            if (i0 + 32 * q >= hi) break;
            const unsigned same = __match_any_sync(kFull, e[q]);
            if ((same & ((1u << lane) - 1)) == 0) mine[e[q]] += __popc(same);
            __syncwarp();
        }
    }
    if (counts) {
        // threads in as many teams as there are, each over every so many-th CTA
        int width = 32;
        while (width < E && width < kSortThreads) width <<= 1;
        const int teams = kSortThreads / width, team = threadIdx.x / width;
        for (int x = threadIdx.x % width; x < E; x += width) {
            int32_t b = 0, t = 0;
#pragma unroll 16
            for (int c = team; c < int(gridDim.x); c += teams) {
                const int32_t v = load_here(counts + int64_t(c) * E + x);
                t += v;
                if (c < int(blockIdx.x)) b += v;
            }
            atomicAdd(&before[x], b);
            atomicAdd(&total[x], t);
        }
        __syncthreads();
    } else {
        __syncthreads();
        for (int x = threadIdx.x; x < E; x += kSortThreads) {
            int32_t t = 0;
            for (int w = 0; w < kSortWarps; ++w) t += warp_count[w * (E + 1) + x];
            own[x] = t;
            if (!cluster) total[x] = t;
        }
        if (cluster) {
            asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
            for (int x = threadIdx.x; x < E; x += kSortThreads) {
                int32_t b = 0, t = 0;
                for (uint32_t c = 0; c < gridDim.x; ++c) {
                    uint32_t at;
                    int32_t v;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(uint32_t(__cvta_generic_to_shared(own + x))), "r"(c));
                    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
                    t += v;
                    if (c < blockIdx.x) b += v;
                }
                before[x] = b, total[x] = t;
            }
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // its counterpart is at the end
        }
        __syncthreads();
    }
    exclusive_sums(base, E, sums, [&](int x) { return total[x]; });
    const int32_t held = base[E];
    if (blockIdx.x == 0)
        for (int x = threadIdx.x; x <= E; x += kSortThreads) offsets[x] = base[x];
    for (int x = threadIdx.x; x < E; x += kSortThreads) {
        int32_t at = base[x] + before[x];
        for (int w = 0; w < kSortWarps; ++w) {
            const int32_t c = warp_count[w * (E + 1) + x];
            warp_count[w * (E + 1) + x] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kSteps) {
        if (stretch > 32 * kSteps) load_experts(e, ids, ids64, i0, hi, E, nullptr);
#pragma unroll
        for (int q = 0; q < kSteps; ++q) {
            if (i0 + 32 * q >= hi) break;
            const int64_t i = i0 + 32 * q + lane;
            const unsigned same = __match_any_sync(kFull, e[q]), earlier = same & ((1u << lane) - 1);
            const int32_t row = mine[e[q]] + __popc(earlier);
            __syncwarp();
            if (earlier == 0) mine[e[q]] += __popc(same);
            __syncwarp();
            if (i < hi) {
                slots[i] = e[q] < E ? row : -1;
                if (e[q] < E) tokens[row] = int32_t(uint32_t(i) / uint32_t(k));
            }
        }
    }
    // the rows behind the last
    for (int64_t s = held + int64_t(blockIdx.x) * kSortThreads + threadIdx.x; s < n; s += int64_t(gridDim.x) * kSortThreads) tokens[s] = -1;
    let_next_kernel_start();
    __syncwarp();
    if (cluster) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the others have read this CTA's counts
}

// Which of the token's pairs, a lane each, have a row, and where.
__device__ __forceinline__ unsigned held_pairs(const int32_t* slots, int64_t t, int k, int32_t M, int lane, int32_t* slot) {
    *slot = lane < k ? load_here(slots + t * k + lane) : -1;
    return __ballot_sync(kFull, uint32_t(*slot) < uint32_t(M));
}

// The tokens' rows to where their pairs go.  A warp takes a token and a stretch of 32*U vectors of its row into
// registers and writes them once for each pair, so every row of src is read once.
//
// Bound by HBM writes: 65536 rows of 2048 bf16 values to eight places each in 357 us, 6.8 TB/s.
template <typename Word, int U>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
dispatch_kernel(const Word* src, int64_t src_stride, int64_t T, int k, int32_t M, uint32_t vecs, const int32_t* slots, Word* rows, int64_t rows_stride,
                uint32_t stretches, int64_t items) {
    const int lane = threadIdx.x & 31;
    wait_for_previous_kernel();
    for (int64_t it = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items; it += int64_t(gridDim.x) * kWarps) {
        const int64_t t = quotient(it, stretches);
        const uint32_t col = uint32_t(it - t * stretches) * (32 * U) + lane;
        Word v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (col + 32 * u < vecs) v[u] = __ldcg(src + t * src_stride + col + 32 * u);
        int32_t slot;
        unsigned held = held_pairs(slots, t, k, M, lane, &slot);
        while (held) {
            const int j = __ffs(held) - 1;
            held &= held - 1;
            Word* to = rows + int64_t(__shfl_sync(kFull, slot, j)) * rows_stride + col;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (col + 32 * u < vecs) to[32 * u] = v[u];
        }
    }
    let_next_kernel_start();
}

// The rows back at their tokens, weighted.  A warp takes a token and up to `per` stretches of 32*Cols vectors, one after the other; AtOnce
// rows are in flight before their products are added, in fp32 and in the pairs' order.
//
// Bound by HBM reads: 524288 rows of 2048 bf16 values back to 65536 tokens in 355 us, 6.8 TB/s (418 with four CTAs an SM, of whose
// registers 168 bytes spill; here 20 do).  Calls in a row find a part of the rows in L2: once it has been flushed they take 2 % longer.
constexpr int kCombineCtasPerSm = 3;
template <typename T, int V, int Cols, int AtOnce>
__global__ void __launch_bounds__(kThreads, kCombineCtasPerSm)
combine_kernel(const T* rows, int64_t rows_stride, int64_t tokens, int k, int32_t M, uint32_t len, const int32_t* slots, const float* weights, T* out,
               int64_t out_stride, uint32_t stretches, uint32_t per, uint32_t shares, int64_t items) {
    using Word = typename Vec<T, V>::Word;
    const int lane = threadIdx.x & 31;
    wait_for_previous_kernel();
    for (int64_t it = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items; it += int64_t(gridDim.x) * kWarps) {
        const int64_t t = quotient(it, shares);
        const uint32_t s0 = uint32_t(it - t * shares) * per, s1 = min(s0 + per, stretches);
        int32_t slot;
        const unsigned all = held_pairs(slots, t, k, M, lane, &slot);
        const float weight = weights && lane < k ? __ldcg(weights + t * k + lane) : 1.0f;
        for (uint32_t s = s0; s < s1; ++s) {
            const uint32_t col = (s * (32 * Cols) + lane) * V;
            float acc[Cols][V] = {};
            unsigned held = all;
            while (held) {
                Word w[AtOnce][Cols];
                float f[AtOnce];
                int many = 0;
#pragma unroll
                for (int r = 0; r < AtOnce; ++r) {
                    if (!held) break;
                    const int j = __ffs(held) - 1;
                    held &= held - 1;
                    const T* from = rows + int64_t(__shfl_sync(kFull, slot, j)) * rows_stride + col;
                    f[r] = __shfl_sync(kFull, weight, j);
                    ++many;
#pragma unroll
                    for (int c = 0; c < Cols; ++c)
                        if (col + c * 32 * V < len) w[r][c] = __ldcs(reinterpret_cast<const Word*>(from + c * 32 * V));
                }
#pragma unroll
                for (int r = 0; r < AtOnce; ++r) {
                    if (r >= many) break;
#pragma unroll
                    for (int c = 0; c < Cols; ++c) {
                        if (col + c * 32 * V >= len) continue;
                        float x[V];
                        widen(w[r][c], x);
#pragma unroll
                        for (int v = 0; v < V; ++v) acc[c][v] = weights ? fmaf(f[r], x[v], acc[c][v]) : acc[c][v] + x[v];
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < Cols; ++c)
                if (col + c * 32 * V < len) put(out + t * out_stride + col + c * 32 * V, acc[c]);
        }
    }
    let_next_kernel_start();
}

// The gradients of the weighted sum.  `team` warps take a token, a share of its columns each, and all of up to
// Pairs pairs at once: Cols vectors of dout are read once, those of the pairs' rows beside them, and each pair's
// product with its weight is written while the dot product is added up.  A lane's sums run over its columns in order, then
// over the warp's lanes and the team's warps as a tree.
//
// Bound by HBM, a row read and a row written for each pair: 262144 rows of 2048 bf16 values in 341 us, 6.7 TB/s.
template <typename T, int V, int Pairs, int Cols>
__global__ void __launch_bounds__(kThreads, 2)
combine_grad_kernel(const T* dout, int64_t dout_stride, const T* rows, int64_t rows_stride, int64_t tokens, int k, int32_t M, uint32_t len,
                    const int32_t* slots, const float* weights, T* drows, int64_t drows_stride, float* dweights, int team) {
    using Word = typename Vec<T, V>::Word;
    __shared__ float partial[kWarps][Pairs];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % team, each = kWarps / team;
    wait_for_previous_kernel();
    for (int64_t t0 = int64_t(blockIdx.x) * each; t0 < tokens; t0 += int64_t(gridDim.x) * each) {
        const int64_t t = t0 + warp / team;
        const bool here = t < tokens;
        int32_t slot = -1;
        float weight = 0.0f;
        if (here && lane < k) slot = load_here(slots + t * k + lane), weight = __ldcg(weights + t * k + lane);
        for (int j0 = 0; j0 < k; j0 += Pairs) {
            float dot[Pairs] = {}, w[Pairs];
            int32_t s[Pairs];
            unsigned any = 0;
#pragma unroll
            for (int j = 0; j < Pairs; ++j) {
                s[j] = __shfl_sync(kFull, slot, (j0 + j) & 31);
                w[j] = __shfl_sync(kFull, weight, (j0 + j) & 31);
                if (j0 + j >= k || uint32_t(s[j]) >= uint32_t(M)) s[j] = -1;
                else any = 1;
            }
            if (any) {
                for (uint32_t col = (part * 32 * Cols + lane) * V; col < len; col += team * 32 * Cols * V) {
                    Word r[Pairs][Cols], d[Cols];
#pragma unroll
                    for (int c = 0; c < Cols; ++c)
                        if (col + c * 32 * V < len) d[c] = __ldcg(reinterpret_cast<const Word*>(dout + t * dout_stride + col + c * 32 * V));
#pragma unroll
                    for (int j = 0; j < Pairs; ++j)
#pragma unroll
                        for (int c = 0; c < Cols; ++c)
                            if (s[j] >= 0 && col + c * 32 * V < len) r[j][c] = __ldcs(reinterpret_cast<const Word*>(rows + int64_t(s[j]) * rows_stride + col + c * 32 * V));
#pragma unroll
                    for (int c = 0; c < Cols; ++c) {
                        if (col + c * 32 * V >= len) continue;
                        float x[V];
                        widen(d[c], x);
#pragma unroll
                        for (int j = 0; j < Pairs; ++j) {
                            if (s[j] < 0) continue;
                            float y[V], z[V];
                            widen(r[j][c], y);
#pragma unroll
                            for (int v = 0; v < V; ++v) dot[j] = fmaf(x[v], y[v], dot[j]), z[v] = w[j] * x[v];
                            put(drows + int64_t(s[j]) * drows_stride + col + c * 32 * V, z);
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < Pairs; ++j) {
#pragma unroll
                for (int d = 16; d; d >>= 1) dot[j] += __shfl_xor_sync(kFull, dot[j], d);
            }
            if (team > 1) {
                if (lane == 0)
#pragma unroll
                    for (int j = 0; j < Pairs; ++j) partial[warp][j] = dot[j];
                __syncthreads();
                if (here && part == 0 && lane < Pairs && j0 + lane < k) {
                    float sum = 0.0f;
                    for (int p = 0; p < team; ++p) sum += partial[warp + p][lane];
                    dweights[t * k + j0 + lane] = sum;
                }
                __syncthreads();
            } else if (here) {
#pragma unroll
                for (int j = 0; j < Pairs; ++j)
                    if (lane == j && j0 + j < k) dweights[t * k + j0 + j] = dot[j];
            }
        }
    }
    let_next_kernel_start();
}

// As many CTAs as there is work where the GPU may be filled: those that come late even out the end.  65536 rows of 2048 bf16 values
// to 524288 places take 357 us so, 387 with eight CTAs an SM that go round.
int grid_of(int64_t blocks, const Ctas& c) { return int(std::max<int64_t>(1, std::min<int64_t>(blocks, c.most ? c.most : INT32_MAX))); }

// The widest vector, in bytes up to 16, that all rows of both arrays allow.
int vector_bytes(const void* a, int64_t a_stride, int64_t a_rows, const void* b, int64_t b_stride, int64_t b_rows, int64_t len, int elem) {
    const uint64_t all = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | uint64_t(len * elem) |
                         (a_rows > 1 ? uint64_t(a_stride * elem) : 0) | (b_rows > 1 ? uint64_t(b_stride * elem) : 0);
    int v = 16;
    while (v > elem && all % v) v >>= 1;
    return v;
}

template <typename Word>
cudaError_t dispatch(const RowsView& src, int elem, int64_t T, int k, int64_t len, const int32_t* slots, void* rows, int64_t rows_stride, const Ctas& c,
                     cudaStream_t stream) {
    constexpr int U = 4;
    const int per = int(sizeof(Word)) / elem;
    const uint32_t vecs = uint32_t(len / per), stretches = (vecs + 32 * U - 1) / (32 * U);
    const int64_t items = T * stretches;
    return launch_after(dispatch_kernel<Word, U>, grid_of((items + kWarps - 1) / kWarps, c), kThreads, 0, stream, static_cast<const Word*>(src.p), src.stride / per, T, k,
                        int32_t(T * k), vecs, slots, static_cast<Word*>(rows), rows_stride / per, stretches, items);
}

template <typename T, int V>
cudaError_t combine(const RowsView& rows, int64_t tokens, int k, int64_t len, const int32_t* slots, const float* weights, void* out, int64_t out_stride,
                    const Ctas& c, cudaStream_t stream) {
    auto go = [&](auto* kernel, int cols) {
        const uint32_t stretches = uint32_t((len + 32 * V * cols - 1) / (32 * V * cols));
        // a warp takes the whole row where the tokens fill the GPU four times, so that it finds their rows once (80000 rows of 1027 bf16
        // values 53 us; with eight vectors at a time 60, and a stretch a warp 76)
        const int64_t warps = 4 * int64_t(c.sms) * kCombineCtasPerSm * kWarps;
        const uint32_t shares = uint32_t(std::min<int64_t>(stretches, (warps + tokens - 1) / tokens));
        const uint32_t per = (stretches + shares - 1) / shares;
        const int64_t items = tokens * ((stretches + per - 1) / per);
        return launch_after(kernel, grid_of((items + kWarps - 1) / kWarps, c), kThreads, 0, stream, static_cast<const T*>(rows.p), rows.stride, tokens, k, int32_t(tokens * k),
                            uint32_t(len), slots, weights, static_cast<T*>(out), out_stride, stretches, per, (stretches + per - 1) / per, items);
    };
    // Short vectors go several at a time, fewer where a row has no more: 80000 rows of 1027 bf16 values take 53 us with seven of four rows; eight,
    // of which registers spill, 60; six 57; 12297 rows 12.3 us, with eight 13.9.
    constexpr int kMany = V * sizeof(T) >= 16 ? 2 : V * sizeof(T) == 8 ? 4 : 7;
    return len > 32 * V ? go(combine_kernel<T, V, kMany, 4>, kMany) : go(combine_kernel<T, V, 1, 4>, 1);
}

template <typename T, int V>
cudaError_t combine_grad(const RowsView& dout, const RowsView& rows, int64_t tokens, int k, int64_t len, const int32_t* slots, const float* weights, void* drows,
                         int64_t drows_stride, float* dweights, const Ctas& c, cudaStream_t stream) {
    auto go = [&](auto* kernel, int cols) {
        // more warps for a token while the tokens do not fill the GPU and the row has a vector for each lane
        int team = 1;
        while (team < kWarps && tokens * team < int64_t(c.sms) * 16 && len > int64_t(team) * 32 * V * cols) team *= 2;
        const int64_t blocks = (tokens + kWarps / team - 1) / (kWarps / team);
        return launch_after(kernel, grid_of(blocks, c), kThreads, 0, stream, static_cast<const T*>(dout.p), dout.stride, static_cast<const T*>(rows.p), rows.stride,
                            tokens, k, int32_t(tokens * k), uint32_t(len), slots, weights, static_cast<T*>(drows), drows_stride, dweights, team);
    };
    // Vectors of each row in flight, more where they are short and where pairs are few: 262144 rows of 2048 bf16 values, eight pairs, 341
    // us with two of 16 bytes, one 350; 12297 of 1027 fp32 values, three pairs, 17.9 with twelve, eight 18.6, four 20.7; 80000 of 1028
    // bf16 values, four pairs, 66 with eight of 8 bytes, four 70, but 48000, eight pairs, 43 with four, two 41.
    constexpr int kBytes = V * sizeof(T), kEight = kBytes >= 8 ? 2 : kBytes == 4 ? 6 : 4, kFour = kBytes >= 16 ? 4 : kBytes == 4 ? 12 : 8;
    return k > 4 ? go(combine_grad_kernel<T, V, 8, kEight>, kEight) : go(combine_grad_kernel<T, V, 4, kFour>, kFour);
}

}  // namespace

SortShape sort_shape(int64_t pairs, const Ctas& c) {
    const int64_t most = c.most ? c.most : c.sms;
    auto ctas = [&](int64_t least) { return int(std::max<int64_t>(1, std::min(most, (pairs + least - 1) / least))); };
    // one CTA, then a cluster of them, as long as each warp has at most eight steps of 32; then every SM
    if (pairs <= kSortAlone) return {1, false};
    if (pairs <= kSortCluster * kSortPiece) return {std::min(kSortCluster, ctas(kSortPiece / 2)), false};
    return {ctas(kSortPiece / 2), true};
}

cudaError_t launch_sort(const void* ids, int ids64, int64_t pairs, int k, int E, int32_t* offsets, int32_t* slots, int32_t* tokens, int32_t* counts, const Ctas& c,
                        int* status, cudaStream_t stream) {
    const size_t smem = sizeof(int32_t) * (size_t(E) + 1 + 3 * size_t(E) + size_t(kSortWarps) * (E + 1));
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(sort_experts_kernel), int(sizeof(int32_t) * (20 * (TIDE_MAX_EXPERTS + 1))), c.device, allowed);
    if (e != cudaSuccess) return e;
    const SortShape shape = sort_shape(pairs, c);
    const int32_t piece = int32_t((pairs + shape.ctas - 1) / shape.ctas);
    if (shape.counted) {
        e = launch_after(count_experts_kernel, shape.ctas, kSortThreads, 0, stream, ids, ids64, int32_t(pairs), piece, E, counts, status);
        if (e != cudaSuccess) return e;
    }
    return launch_clusters_after(sort_experts_kernel, shape.counted ? 1 : shape.ctas, shape.ctas, kSortThreads, smem, stream, ids, ids64, int32_t(pairs), piece, k, E,
                                 shape.counted ? static_cast<const int32_t*>(counts) : nullptr, offsets, slots, tokens, status);
}

cudaError_t launch_dispatch(const RowsView& src, int bf16, int64_t T, int k, int64_t len, const int32_t* slots, void* rows, int64_t rows_stride, const Ctas& c,
                            cudaStream_t stream) {
    if (T <= 0 || len <= 0) return cudaSuccess;
    const int elem = bf16 ? 2 : 4;
    switch (vector_bytes(src.p, src.stride, T, rows, rows_stride, T * k, len, elem)) {
        case 16: return dispatch<uint4>(src, elem, T, k, len, slots, rows, rows_stride, c, stream);
        case 8: return dispatch<uint2>(src, elem, T, k, len, slots, rows, rows_stride, c, stream);
        case 4: return dispatch<uint32_t>(src, elem, T, k, len, slots, rows, rows_stride, c, stream);
        default: return dispatch<uint16_t>(src, elem, T, k, len, slots, rows, rows_stride, c, stream);
    }
}

cudaError_t launch_combine(const RowsView& rows, int bf16, int64_t T, int k, int64_t len, const int32_t* slots, const float* weights, void* out, int64_t out_stride,
                           const Ctas& c, cudaStream_t stream) {
    if (T <= 0 || len <= 0) return cudaSuccess;
    const int v = vector_bytes(rows.p, rows.stride, T * k, out, out_stride, T, len, bf16 ? 2 : 4);
    if (bf16) switch (v) {
            case 16: return combine<__nv_bfloat16, 8>(rows, T, k, len, slots, weights, out, out_stride, c, stream);
            case 8: return combine<__nv_bfloat16, 4>(rows, T, k, len, slots, weights, out, out_stride, c, stream);
            case 4: return combine<__nv_bfloat16, 2>(rows, T, k, len, slots, weights, out, out_stride, c, stream);
            default: return combine<__nv_bfloat16, 1>(rows, T, k, len, slots, weights, out, out_stride, c, stream);
        }
    switch (v) {
        case 16: return combine<float, 4>(rows, T, k, len, slots, weights, out, out_stride, c, stream);
        case 8: return combine<float, 2>(rows, T, k, len, slots, weights, out, out_stride, c, stream);
        default: return combine<float, 1>(rows, T, k, len, slots, weights, out, out_stride, c, stream);
    }
}

cudaError_t launch_combine_grad(const RowsView& dout, const RowsView& rows, int bf16, int64_t T, int k, int64_t len, const int32_t* slots, const float* weights,
                                void* drows, int64_t drows_stride, float* dweights, const Ctas& c, cudaStream_t stream) {
    if (T <= 0) return cudaSuccess;
    const int elem = bf16 ? 2 : 4;
    const int v = std::min(vector_bytes(dout.p, dout.stride, T, rows.p, rows.stride, T * k, len, elem), vector_bytes(drows, drows_stride, T * k, rows.p, rows.stride, T * k, len, elem));
    if (bf16) switch (v) {
            case 16: return combine_grad<__nv_bfloat16, 8>(dout, rows, T, k, len, slots, weights, drows, drows_stride, dweights, c, stream);
            case 8: return combine_grad<__nv_bfloat16, 4>(dout, rows, T, k, len, slots, weights, drows, drows_stride, dweights, c, stream);
            case 4: return combine_grad<__nv_bfloat16, 2>(dout, rows, T, k, len, slots, weights, drows, drows_stride, dweights, c, stream);
            default: return combine_grad<__nv_bfloat16, 1>(dout, rows, T, k, len, slots, weights, drows, drows_stride, dweights, c, stream);
        }
    switch (v) {
        case 16: return combine_grad<float, 4>(dout, rows, T, k, len, slots, weights, drows, drows_stride, dweights, c, stream);
        case 8: return combine_grad<float, 2>(dout, rows, T, k, len, slots, weights, drows, drows_stride, dweights, c, stream);
        default: return combine_grad<float, 1>(dout, rows, T, k, len, slots, weights, drows, drows_stride, dweights, c, stream);
    }
}

}  // namespace tide
