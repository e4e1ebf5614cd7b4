// Values to e4m3 codes with a power-of-two scale for each block of 128: tokens' rows on their way to the experts, rows
// already there (as they are and transposed), and the experts' weights straight from the ranks' shards (sm_103a).
//
// A block whose largest magnitude is a = f * 2^e, 1 <= f < 2, gets the scale 2^(e - 8) where f <= 1.75 (448 =
// 1.75 * 2^8) and 2^(e - 7) else, so dividing by it is exact and codes have the one rounding of their conversion.
#include <algorithm>

#include "experts_device.cuh"

namespace tide {
namespace {

// The scale of a block and what its values are multiplied by.  `bits` are those of its largest magnitude as fp32;
// they order magnitudes as numbers, with NaN behind infinity.
struct Scale {
    float scale, inverse;
};
__device__ __forceinline__ Scale scale_of(uint32_t bits) {
    if (bits >= 0x7f800000u) return {__uint_as_float(0x7fffffffu), __uint_as_float(0x7fffffffu)};
    int p = max(int(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u), -126);
    if (bits == 0) p = 0;
    return {__uint_as_float(uint32_t(p + 127) << 23), __uint_as_float(uint32_t(127 - p) << 23)};
}

__device__ __forceinline__ uint32_t codes2(float a, float b) {
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(b), "f"(a));
    return h;
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) { return codes2(a, b) | codes2(c, d) << 16; }

// Eight consecutive values of a row as they lie in memory, zeros behind `left` of them.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    template <bool Vector>
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int left) {
        if constexpr (Vector) {
            zero();
            if (left > 0) w = __ldcg(reinterpret_cast<const uint4*>(p));
        } else {
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = j < left ? uint32_t(__ldcg(reinterpret_cast<const uint16_t*>(p) + j)) : 0u;
            w = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
        }
    }
    // The largest magnitude, as fp32 bits.
    __device__ __forceinline__ uint32_t largest() const {
        const uint32_t m = 0x7fff7fffu;
        const uint32_t a = __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
        return max(a << 16, a & 0xffff0000u);
    }
    __device__ __forceinline__ void values(float (&x)[8]) const { widen(w, x); }
    // Largest magnitudes of each of the eight columns so far.
    __device__ __forceinline__ void raise(const Eight& o) {
        const uint32_t m = 0x7fff7fffu;
        w = make_uint4(__vmaxu2(w.x & m, o.w.x & m), __vmaxu2(w.y & m, o.w.y & m), __vmaxu2(w.z & m, o.w.z & m), __vmaxu2(w.w & m, o.w.w & m));
    }
    __device__ __forceinline__ Eight other_half() const {
        Eight o;
        o.w = make_uint4(__shfl_xor_sync(kFull, w.x, 16), __shfl_xor_sync(kFull, w.y, 16), __shfl_xor_sync(kFull, w.z, 16), __shfl_xor_sync(kFull, w.w, 16));
        return o;
    }
};
template <>
struct Eight<float> {
    float x[8];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    }
    template <bool Vector>
    __device__ __forceinline__ void load(const float* p, int left) {
        if constexpr (Vector) {
            zero();
            if (left > 0) {
                const float4 a = __ldcg(reinterpret_cast<const float4*>(p)), b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
                x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = j < left ? __ldcg(p + j) : 0.0f;
        }
    }
    __device__ __forceinline__ uint32_t largest() const {
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(x[j]) & 0x7fffffffu);
        return a;
    }
    __device__ __forceinline__ void values(float (&y)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[j];
    }
    __device__ __forceinline__ void raise(const Eight& o) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(max(__float_as_uint(x[j]) & 0x7fffffffu, __float_as_uint(o.x[j]) & 0x7fffffffu));
    }
    __device__ __forceinline__ Eight other_half() const {
        Eight o;
#pragma unroll
        for (int j = 0; j < 8; ++j) o.x[j] = __uint_as_float(__shfl_xor_sync(kFull, __float_as_uint(x[j]), 16));
        return o;
    }
};

// ---- the tokens' rows to where their pairs go, in 8 bits ----------------------------------------
//
// A warp takes a token and 512 columns: 16 columns a lane, so that eight lanes have a block and each stores its codes as
// one vector.  The row is read and converted once and written for each pair.
//
// Bound by HBM writes.
template <typename T, bool Vector>
__global__ void __launch_bounds__(kThreads, 4)
dispatch_fp8_kernel(const T* src, int64_t src_stride, int64_t tokens, int k, int32_t M, uint32_t len, const int32_t* slots, tide_fp8_t rows, uint32_t stretches,
                    int64_t items) {
    const int lane = threadIdx.x & 31;
    wait_for_previous_kernel();
    for (int64_t it = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items; it += int64_t(gridDim.x) * kWarps) {
        const int64_t t = it / stretches;
        const uint32_t col = uint32_t(it - t * stretches) * 512 + lane * 16;
        Eight<T> a, b;
        a.template load<Vector>(src + t * src_stride + col, int(len) - int(col));
        b.template load<Vector>(src + t * src_stride + col + 8, int(len) - int(col) - 8);
        const int32_t slot = lane < k ? load_here(slots + t * k + lane) : -1;
        unsigned held = __ballot_sync(kFull, uint32_t(slot) < uint32_t(M));
        uint32_t largest = max(a.largest(), b.largest());
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) largest = max(largest, __shfl_xor_sync(kFull, largest, d));
        const Scale s = scale_of(largest);
        float x[8], y[8];
        a.values(x), b.values(y);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= s.inverse, y[j] *= s.inverse;
        const uint4 codes = make_uint4(codes4(x[0], x[1], x[2], x[3]), codes4(x[4], x[5], x[6], x[7]), codes4(y[0], y[1], y[2], y[3]), codes4(y[4], y[5], y[6], y[7]));
        while (held) {
            const int j = __ffs(held) - 1;
            held &= held - 1;
            const int64_t row = __shfl_sync(kFull, slot, j);
            if (col < len) {
                *reinterpret_cast<uint4*>(static_cast<char*>(rows.codes) + row * rows.stride + col) = codes;
                if ((lane & 7) == 0) rows.scales[row * rows.scale_stride + col / kBlock] = s.scale;
            }
        }
    }
    let_next_kernel_start();
}

// ---- tiles of 128 x 128 -------------------------------------------------------------------------
//
// A CTA of 8 warps takes 128 rows of one expert and 128 columns.  A thread has 8 consecutive rows and 8 consecutive
// columns: 16 lanes are a row, so a row's scale comes from a reduction over them, a column's from the threads' own
// eight rows, the warp's other half and the other warps.  The transposed codes are turned in shared memory, where the 8
// bytes that a thread has of a column are stored at a place rotated by its column group, so that neither the stores nor
// the loads of whole columns meet in a bank.
//
// Bound by HBM: 2 or 4 bytes read a value and 1 or 2 written.
struct TileOut {
    tide_fp8_t rows, columns;
    int has_rows, has_columns;
};

struct TileSmem {
    uint64_t row_at[kBlock];                       // where each row lies; 0: none
    __align__(16) uint32_t largest[kWarps][kBlock];  // of each column, as fp32 bits
    __align__(16) unsigned char turned[kBlock * kBlock];
};

template <typename T>
__device__ __forceinline__ void load_tile(Eight<T> (&x)[8], const TileSmem& sm, uint32_t col, uint32_t len, bool vector) {
    const int row0 = (threadIdx.x >> 4) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const T* p = reinterpret_cast<const T*>(sm.row_at[row0 + i]);
        const int left = p ? int(len) - int(col) : 0;
        if (vector) x[i].template load<true>(p + col, left);
        else x[i].template load<false>(p + col, left);
    }
}

// Codes of the tile's rows, `held` of them, at the matrix's row `first` and column `col`.
template <typename T>
__device__ __forceinline__ void put_rows(const Eight<T> (&x)[8], const float (&inverse)[8], char* codes, int64_t stride, int held, uint32_t col, uint32_t len) {
    const int row0 = (threadIdx.x >> 4) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (row0 + i >= held || col >= len) continue;
        float v[8];
        x[i].values(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= inverse[i];
        *reinterpret_cast<uint2*>(codes + int64_t(row0 + i) * stride + col) = make_uint2(codes4(v[0], v[1], v[2], v[3]), codes4(v[4], v[5], v[6], v[7]));
    }
}

// Turns the tile: codes of its columns from `col0` on, `columns` of them, each of `count` rows (a multiple of 16).
template <typename T>
__device__ __forceinline__ void put_columns(const Eight<T> (&x)[8], const float (&inverse)[8], TileSmem& sm, char* codes, int64_t stride, int columns, int count) {
    const int group = threadIdx.x & 15, rows8 = threadIdx.x >> 4;
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i].values(v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float f = inverse[j];
        const uint2 w = make_uint2(codes4(v[0][j] * f, v[1][j] * f, v[2][j] * f, v[3][j] * f), codes4(v[4][j] * f, v[5][j] * f, v[6][j] * f, v[7][j] * f));
        *reinterpret_cast<uint2*>(sm.turned + (group * 8 + j) * kBlock + ((rows8 ^ group) * 8)) = w;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int at = q * 256 + threadIdx.x, c = at >> 3, pair = at & 7, g = c >> 3;
        uint4 w = *reinterpret_cast<const uint4*>(sm.turned + c * kBlock + ((pair ^ (g >> 1)) * 16));
        if (g & 1) w = make_uint4(w.z, w.w, w.x, w.y);
        if (c < columns && pair * 16 < count) *reinterpret_cast<uint4*>(codes + int64_t(c) * stride + pair * 16) = w;
    }
}

struct QuantizeArgs {
    const void* src;
    int64_t src_stride;
    int32_t src_rows, M, E, most_blocks;
    uint32_t len;
    const int32_t* offsets;
    const int32_t* tokens;
    TileOut out;
    uint32_t across;  // tiles of a row of tiles
    int vector;
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) quantize_kernel(const __grid_constant__ QuantizeArgs a) {
    __shared__ TileSmem sm;
    __shared__ int32_t starts[TIDE_MAX_EXPERTS + 1];  // row tiles before each expert
    __shared__ int32_t sums[32];
    const int group = threadIdx.x & 15, row0 = (threadIdx.x >> 4) * 8, warp = threadIdx.x >> 5;
    wait_for_previous_kernel();
    exclusive_sums(starts, a.E, sums, [&](int e) { return (span_of(a.offsets, e, a.M).count + kBlock - 1) / kBlock; });
    const int64_t tiles = int64_t(min(starts[a.E], a.most_blocks)) * a.across;
    for (int64_t it = blockIdx.x; it < tiles; it += gridDim.x) {
        const int32_t down = int32_t(it / a.across), e = last_at_most(starts, a.E, down);
        const uint32_t col0 = uint32_t(it - int64_t(down) * a.across) * kBlock, col = col0 + group * 8;
        const Span span = span_of(a.offsets, e, a.M);
        const int32_t s0 = span.first + (down - starts[e]) * kBlock, held = min(kBlock, span.first + span.count - s0);
        __syncthreads();  // the tile before has been read
        if (threadIdx.x < kBlock) {
            uint64_t at = 0;
            if (int(threadIdx.x) < held) {
                int64_t row = s0 + threadIdx.x;
                if (a.tokens) row = load_here(a.tokens + row);
                if (row >= 0 && row < a.src_rows) at = reinterpret_cast<uint64_t>(static_cast<const T*>(a.src) + row * a.src_stride);
            }
            sm.row_at[threadIdx.x] = at;
        }
        __syncthreads();
        Eight<T> x[8];
        load_tile(x, sm, col, a.len, a.vector);
        if (a.out.has_rows) {
            float inverse[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t largest = x[i].largest();
#pragma unroll
                for (int d = 1; d < 16; d <<= 1) largest = max(largest, __shfl_xor_sync(kFull, largest, d));
                const Scale s = scale_of(largest);
                inverse[i] = s.inverse;
                if (group == i && row0 + i < held) a.out.rows.scales[int64_t(s0 + row0 + i) * a.out.rows.scale_stride + col0 / kBlock] = s.scale;
            }
            put_rows(x, inverse, static_cast<char*>(a.out.rows.codes) + int64_t(s0) * a.out.rows.stride, a.out.rows.stride, held, col, a.len);
        }
        if (a.out.has_columns) {
            Eight<T> m;
            m.zero();
#pragma unroll
            for (int i = 0; i < 8; ++i) m.raise(x[i]);
            m.raise(m.other_half());
            float v[8], inverse[8];
            m.values(v);
            if ((threadIdx.x & 16) == 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) sm.largest[warp][group * 8 + j] = __float_as_uint(v[j]);
            __syncthreads();
            uint32_t largest[8] = {};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const uint4 lo = *reinterpret_cast<const uint4*>(&sm.largest[w][group * 8]), hi = *reinterpret_cast<const uint4*>(&sm.largest[w][group * 8 + 4]);
                largest[0] = max(largest[0], lo.x), largest[1] = max(largest[1], lo.y), largest[2] = max(largest[2], lo.z), largest[3] = max(largest[3], lo.w);
                largest[4] = max(largest[4], hi.x), largest[5] = max(largest[5], hi.y), largest[6] = max(largest[6], hi.z), largest[7] = max(largest[7], hi.w);
            }
            const int64_t block = down;  // of the transposed rows: the experts' tiles lie one after the other
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const Scale s = scale_of(largest[j]);
                inverse[j] = s.inverse;
                if ((threadIdx.x >> 4) == j && col + j < a.len) a.out.columns.scales[block * a.out.columns.scale_stride + col + j] = s.scale;
            }
            put_columns(x, inverse, sm, static_cast<char*>(a.out.columns.codes) + int64_t(col0) * a.out.columns.stride + block * kBlock, a.out.columns.stride,
                        int(min(uint32_t(kBlock), a.len - col0)), kBlock);
        }
    }
    let_next_kernel_start();
}

// ---- the experts' weights from the ranks' shards --------------------------------------------------
struct GatherArgs {
    ShardPtrs shards;
    TableView tv;
    ExpertParams ps;
    tide_fp8_t w, wt;
    int has_wt;
    uint32_t across, down;  // tiles of a matrix
    int64_t tiles;
    int vector;
};

__global__ void __launch_bounds__(kThreads, 3) all_gather_fp8_kernel(const __grid_constant__ GatherArgs a) {
    __shared__ TileSmem sm;
    __shared__ uint32_t of_warp[kWarps];
    const int group = threadIdx.x & 15, warp = threadIdx.x >> 5;
    wait_for_previous_kernel();
    for (int64_t it = blockIdx.x; it < a.tiles; it += gridDim.x) {
        const uint32_t each = a.across * a.down, e = uint32_t(it / each), in = uint32_t(it - int64_t(e) * each), down = in / a.across, across = in - down * a.across;
        const uint32_t n0 = down * kBlock, col0 = across * kBlock, col = col0 + group * 8;
        const int held = int(min(uint32_t(kBlock), a.tv.rows - n0));
        __syncthreads();  // the tile before has been read
        if (threadIdx.x < kBlock) {
            uint64_t at = 0;
            if (int(threadIdx.x) < held) {
                const uint32_t n = n0 + threadIdx.x, d = n / a.tv.m;
                at = reinterpret_cast<uint64_t>(shard_base(a.shards, d)) + 2 * (a.ps.off[e] + int64_t(n - d * a.tv.m) * a.tv.len);
            }
            sm.row_at[threadIdx.x] = at;
        }
        __syncthreads();
        Eight<__nv_bfloat16> x[8];
        load_tile(x, sm, col, a.tv.len, a.vector);
        uint32_t largest = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) largest = max(largest, x[i].largest());
        largest = __reduce_max_sync(kFull, largest);
        if ((threadIdx.x & 31) == 0) of_warp[warp] = largest;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) largest = max(largest, of_warp[w]);
        const Scale s = scale_of(largest);
        if (threadIdx.x == 0) a.w.scales[int64_t(e) * a.w.scale_batch + int64_t(down) * a.w.scale_stride + across] = s.scale;
        float inverse[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) inverse[j] = s.inverse;
        put_rows(x, inverse, static_cast<char*>(a.w.codes) + int64_t(e) * a.w.batch + int64_t(n0) * a.w.stride, a.w.stride, held, col, a.tv.len);
        if (a.has_wt)
            put_columns(x, inverse, sm, static_cast<char*>(a.wt.codes) + int64_t(e) * a.wt.batch + int64_t(col0) * a.wt.stride + n0, a.wt.stride,
                        int(min(uint32_t(kBlock), a.tv.len - col0)), (held + 15) / 16 * 16);
    }
    let_next_kernel_start();
}

int grid_of(int64_t blocks, const Ctas& c, int per_sm) {
    return int(std::max<int64_t>(1, std::min<int64_t>(blocks, c.most ? c.most : int64_t(c.sms) * per_sm)));
}

// Whether eight elements can be loaded as vectors of 16 bytes from every row, at every column that is a multiple of 8.
bool vectors(uintptr_t bits, int64_t stride, int64_t rows, int64_t len, int elem) { return bits % 16 == 0 && len % 8 == 0 && (rows <= 1 || stride * elem % 16 == 0); }

template <typename T, bool Vector>
cudaError_t dispatch_fp8(const RowsView& src, int64_t tokens, int k, int64_t len, const int32_t* slots, const tide_fp8_t& rows, const Ctas& c, cudaStream_t stream) {
    const uint32_t stretches = uint32_t((len + 511) / 512);
    const int64_t items = tokens * stretches;
    return launch_after(dispatch_fp8_kernel<T, Vector>, grid_of((items + kWarps - 1) / kWarps, c, 8), kThreads, 0, stream, static_cast<const T*>(src.p), src.stride, tokens, k,
                        int32_t(tokens * k), uint32_t(len), slots, rows, stretches, items);
}

}  // namespace

cudaError_t launch_dispatch_fp8(const RowsView& src, int bf16, int64_t T, int k, int64_t len, const int32_t* slots, const tide_fp8_t& rows, const Ctas& c,
                                cudaStream_t stream) {
    if (T <= 0) return cudaSuccess;
    const bool v = vectors(reinterpret_cast<uintptr_t>(src.p), src.stride, T, len, bf16 ? 2 : 4);
    if (bf16) return (v ? dispatch_fp8<__nv_bfloat16, true> : dispatch_fp8<__nv_bfloat16, false>)(src, T, k, len, slots, rows, c, stream);
    return (v ? dispatch_fp8<float, true> : dispatch_fp8<float, false>)(src, T, k, len, slots, rows, c, stream);
}

cudaError_t launch_quantize(const RowsView& src, int bf16, int64_t src_rows, int64_t M, int64_t len, int E, const int32_t* offsets, const int32_t* tokens,
                            const tide_fp8_t* rows, const tide_fp8_t* columns, const Ctas& c, cudaStream_t stream) {
    if (M <= 0) return cudaSuccess;
    QuantizeArgs a{};
    a.src = src.p, a.src_stride = src.stride, a.src_rows = int32_t(src_rows), a.M = int32_t(M), a.E = E, a.most_blocks = int32_t(padded_blocks(M, E)), a.len = uint32_t(len);
    a.offsets = offsets, a.tokens = tokens;
    a.out.has_rows = rows != nullptr, a.out.has_columns = columns != nullptr;
    if (rows) a.out.rows = *rows;
    if (columns) a.out.columns = *columns;
    a.across = uint32_t((len + kBlock - 1) / kBlock);
    a.vector = vectors(reinterpret_cast<uintptr_t>(src.p), src.stride, src_rows, len, bf16 ? 2 : 4);
    const int64_t tiles = padded_blocks(M, E) * a.across;
    return launch_after(bf16 ? quantize_kernel<__nv_bfloat16> : quantize_kernel<float>, grid_of(tiles, c, 4), kThreads, 0, stream, a);
}

cudaError_t launch_all_gather_fp8(const ShardPtrs& shards, const TableView& tv, int E, const ExpertParams& ps, const tide_fp8_t& w, const tide_fp8_t* wt, const Ctas& c,
                                  cudaStream_t stream) {
    GatherArgs a{};
    a.shards = shards, a.tv = tv, a.ps = ps, a.w = w, a.has_wt = wt != nullptr;
    if (wt) a.wt = *wt;
    a.across = (tv.len + kBlock - 1) / kBlock, a.down = (tv.rows + kBlock - 1) / kBlock;
    a.tiles = int64_t(E) * a.across * a.down;
    a.vector = vectors(shards.bits, 0, 1, tv.len, 2);
    for (int e = 0; e < E; ++e) a.vector &= ps.off[e] % 8 == 0;
    return launch_after(all_gather_fp8_kernel, grid_of(a.tiles, c, 4), kThreads, 0, stream, a);
}

}  // namespace tide
