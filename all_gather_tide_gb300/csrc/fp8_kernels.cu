// Values to e4m3 codes with a power-of-two scale for each block of 128: tokens' rows on their way to the experts, rows
// already there (as they are and transposed), and the experts' weights straight from the ranks' shards (sm_103a).
//
// A block whose largest magnitude is a = f * 2^e, 1 <= f < 2, gets the scale 2^(e - 8) where f <= 1.75 (448 =
// 1.75 * 2^8) and 2^(e - 7) else, so dividing by it is exact and codes have the one rounding of their conversion.
#include <algorithm>

#include "copy_any.cuh"
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

// Two bf16 values times two powers of two: exact, but for values so small that their codes are zeros.
__device__ __forceinline__ uint32_t times(uint32_t w, uint32_t f) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(f));
    return r;
}

// The larger magnitudes of two pairs of bf16 values; NaN is larger than all. (As integers, by __vmaxu2, a maximum takes several
// instructions: 131072 gathered rows of 2048 took 174 us.)
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b32 x, y;\n\tabs.bf16x2 x, %1;\n\tabs.bf16x2 y, %2;\n\tmax.NaN.bf16x2 %0, x, y;\n\t}" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight consecutive values of a row as they lie in memory, zeros behind `left` of them (load: 16-byte vectors, all or none); and what a power of two, or one for
// each, times them looks like in that type.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    using Factor = uint16_t;  // a power of two, as bf16
    uint4 w;
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int left) {
        zero();
        if (left > 0) w = __ldcg(reinterpret_cast<const uint4*>(p));
    }
    // Out of the aligned 16 bytes that hold them; what lies beside the row there is of the same allocation. (Element by element 80000
    // rows of 1027 take 134 us in both forms, so 113.)
    __device__ __forceinline__ void load_shifted(const __nv_bfloat16* p, int left) {
        zero();
        if (left <= 0) return;
        const unsigned off = unsigned(reinterpret_cast<uintptr_t>(p)) & 15;
        const uint4* from = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - off);
        const uint4 a = __ldcg(from), b = off + 2 * min(left, 8) > 16 ? __ldcg(from + 1) : make_uint4(0, 0, 0, 0);
        w = off ? bytes_at(a, b, off) : a;
        if (left < 8) {
            uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = 2 * i + 1 < left ? v[i] : 2 * i < left ? v[i] & 0xffffu : 0u;
            w = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
    // The largest magnitude, as fp32 bits.
    __device__ __forceinline__ uint32_t largest() const {
        const uint32_t a = larger(larger(w.x, w.y), larger(w.z, w.w));
        return max(a << 16, a & 0xffff0000u);
    }
    // The larger magnitudes of each of the eight columns.
    __device__ __forceinline__ void raise(const Eight& o) {
        w = make_uint4(larger(w.x, o.w.x), larger(w.y, o.w.y), larger(w.z, o.w.z), larger(w.w, o.w.w));
    }
    __device__ __forceinline__ Eight other_half() const {
        Eight o;
        o.w = make_uint4(__shfl_xor_sync(kFull, w.x, 16), __shfl_xor_sync(kFull, w.y, 16), __shfl_xor_sync(kFull, w.z, 16), __shfl_xor_sync(kFull, w.w, 16));
        return o;
    }
    static __device__ __forceinline__ uint32_t magnitude(uint16_t bits) { return uint32_t(bits) << 16; }  // of a value that raise left
    using Bits = uint16_t;
    static __device__ __forceinline__ Factor factor(float f) { return uint16_t(__float_as_uint(f) >> 16); }
    __device__ __forceinline__ void scale(Factor f) {
        const uint32_t g = uint32_t(f) << 16 | f;
        w = make_uint4(times(w.x, g), times(w.y, g), times(w.z, g), times(w.w, g));
    }
    // Each by its own factor, eight in order at f.
    __device__ __forceinline__ void scale_each(const Factor* f) {
        const uint4 g = *reinterpret_cast<const uint4*>(f);
        w = make_uint4(times(w.x, g.x), times(w.y, g.y), times(w.z, g.z), times(w.w, g.w));
    }
    __device__ __forceinline__ float value(int j) const {
        const uint32_t v = j < 2 ? w.x : j < 4 ? w.y : j < 6 ? w.z : w.w;
        return j & 1 ? high_f32(v) : low_f32(v);
    }
};
template <>
struct Eight<float> {
    using Factor = float;
    float x[8];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    }
    __device__ __forceinline__ void load(const float* p, int left) {
        zero();
        if (left > 0) {
            const float4 a = __ldcg(reinterpret_cast<const float4*>(p)), b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        }
    }
    __device__ __forceinline__ void load_shifted(const float* p, int left) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = j < left ? __ldcg(p + j) : 0.0f;
    }
    __device__ __forceinline__ uint32_t largest() const {
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(x[j]) & 0x7fffffffu);
        return a;
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
    static __device__ __forceinline__ uint32_t magnitude(uint32_t bits) { return bits; }
    using Bits = uint32_t;
    static __device__ __forceinline__ Factor factor(float f) { return f; }
    __device__ __forceinline__ void scale(Factor f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= f;
    }
    __device__ __forceinline__ void scale_each(const Factor* f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= f[j];
    }
    __device__ __forceinline__ float value(int j) const { return x[j]; }
};
template <typename T>
__device__ __forceinline__ uint2 codes_of(const Eight<T>& x) {
    return make_uint2(codes4(x.value(0), x.value(1), x.value(2), x.value(3)), codes4(x.value(4), x.value(5), x.value(6), x.value(7)));
}

// ---- the tokens' rows to where their pairs go, in 8 bits ----------------------------------------
//
// A warp takes a token and 512 columns: 16 columns a lane, so that eight lanes have a block and each stores its codes as
// one vector.  The row is read and converted once and written for each pair. Rows without alignment are read as aligned words
// (20000 rows of 1027 bf16 values to four places each 32 us, element by element 39).
//
// Bound by HBM writes: 65536 rows of 2048 bf16 values to eight places each in 204 us, 6.8 TB/s with their scales (242 with eight CTAs an SM that go
// round: those that come late even out the end).
template <typename T, bool Vector>
__global__ void __launch_bounds__(kThreads, 4)
dispatch_fp8_kernel(const T* src, int64_t src_stride, int64_t tokens, int k, int32_t M, uint32_t len, const int32_t* slots, tide_fp8_t rows, uint32_t stretches,
                    int64_t items) {
    const int lane = threadIdx.x & 31;
    wait_for_previous_kernel();
    for (int64_t it = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items; it += int64_t(gridDim.x) * kWarps) {
        const int64_t t = quotient(it, stretches);
        const uint32_t col = uint32_t(it - t * stretches) * 512 + lane * 16;
        Eight<T> a, b;
        const T* from = src + t * src_stride + col;
        const int left = int(len) - int(col);
        if constexpr (Vector) a.load(from, left), b.load(from + 8, left - 8);
        else a.load_shifted(from, left), b.load_shifted(from + 8, left - 8);
        const int32_t slot = lane < k ? load_here(slots + t * k + lane) : -1;
        unsigned held = __ballot_sync(kFull, uint32_t(slot) < uint32_t(M));
        uint32_t largest = max(a.largest(), b.largest());
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) largest = max(largest, __shfl_xor_sync(kFull, largest, d));
        const Scale s = scale_of(largest);
        a.scale(Eight<T>::factor(s.inverse)), b.scale(Eight<T>::factor(s.inverse));
        const uint2 lo = codes_of(a), hi = codes_of(b);
        const uint4 codes = make_uint4(lo.x, lo.y, hi.x, hi.y);
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
// CTAs of an SM, as the registers are bounded for.
template <typename T>
constexpr int kTileCtasPerSm = sizeof(T) == 2 ? 4 : 2;

struct TileOut {
    tide_fp8_t rows, columns;
    int has_rows, has_columns;
};

template <bool Vector, typename T>
__device__ __forceinline__ void load_tile(Eight<T> (&x)[8], const uint64_t* row_at, uint32_t col, uint32_t len) {
    const int row0 = (threadIdx.x >> 4) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const T* p = reinterpret_cast<const T*>(row_at[row0 + i]);
        const int left = p ? int(len) - int(col) : 0;
        if constexpr (Vector) x[i].load(p + col, left);
        else x[i].load_shifted(p + col, left);
    }
}

// Codes of the tile's rows, scaled already, `held` of them, at the matrix's column `col`.
template <typename T>
__device__ __forceinline__ void put_row(const Eight<T>& x, int i, char* codes, int64_t stride, int held, uint32_t col, uint32_t len) {
    const int row = (threadIdx.x >> 4) * 8 + i;
    if (row < held && col < len) *reinterpret_cast<uint2*>(codes + row * stride + col) = codes_of(x);
}

// Turns the tile, scaled already: codes of `columns` of its columns, each of `count` rows (a multiple of 16).
template <typename T>
__device__ __forceinline__ void put_columns(const Eight<T> (&x)[8], unsigned char* turned, char* codes, int64_t stride, int columns, int count) {
    const int group = threadIdx.x & 15, rows8 = threadIdx.x >> 4;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint2*>(turned + (group * 8 + j) * kBlock + ((rows8 ^ group) * 8)) =
            make_uint2(codes4(x[0].value(j), x[1].value(j), x[2].value(j), x[3].value(j)), codes4(x[4].value(j), x[5].value(j), x[6].value(j), x[7].value(j)));
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int at = q * 256 + threadIdx.x, c = at >> 3, pair = at & 7, g = c >> 3;
        uint4 w = *reinterpret_cast<const uint4*>(turned + c * kBlock + ((pair ^ (g >> 1)) * 16));
        if (g & 1) w = make_uint4(w.z, w.w, w.x, w.y);
        if (c < columns && pair * 16 < count) __stcs(reinterpret_cast<uint4*>(codes + c * stride + pair * 16), w);
    }
}

// The largest magnitudes (fp32 bits) of the thread's eight rows over the 16 lanes that have them: lanes 2*i and 2*i + 1 of
// the 16 return that of row i. Each step hands half of the rows to the lanes that keep them: 8 shuffles.
__device__ __forceinline__ uint32_t largest_of_rows(const uint32_t (&a)[8]) {
    const int lane = threadIdx.x;
    uint32_t b[4], c[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t mine = lane & 8 ? a[4 + i] : a[i], theirs = lane & 8 ? a[i] : a[4 + i];
        b[i] = max(mine, __shfl_xor_sync(kFull, theirs, 8));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t mine = lane & 4 ? b[2 + i] : b[i], theirs = lane & 4 ? b[i] : b[2 + i];
        c[i] = max(mine, __shfl_xor_sync(kFull, theirs, 4));
    }
    const uint32_t mine = lane & 2 ? c[1] : c[0], theirs = lane & 2 ? c[0] : c[1];
    const uint32_t d = max(mine, __shfl_xor_sync(kFull, theirs, 2));
    return max(d, __shfl_xor_sync(kFull, d, 1));
}

struct QuantizeArgs {
    const void* src;
    int64_t src_stride;
    int32_t src_rows, M, E;
    uint32_t len;
    const int32_t* offsets;
    const int32_t* tokens;
    TileOut out;
    uint32_t across;  // tiles of a row of tiles
};

// A tile's first row, how many it has, its block of the transposed rows and its first column.
struct TilePlace {
    int32_t first, held, down;
    uint32_t col0;
};
template <typename T>
struct QuantizeSmem {
    uint64_t row_at[2][kBlock];                              // where each row of a tile lies; 0: none
    TilePlace place[2];
    int32_t sums[32];
    __align__(16) Eight<T> largest[kWarps][kBlock / 8];      // magnitudes of each column
    __align__(16) typename Eight<T>::Factor column[kBlock];  // what each column is multiplied by
    __align__(16) unsigned char turned[kBlock * kBlock];
    // and the row tiles before each expert and the first row of each, E + 1 of both
};
template <typename T>
int quantize_smem(int E) {
    return int(sizeof(QuantizeSmem<T>)) + 8 * (E + 1);
}

// While a tile is worked on, the next one's place and rows are found: 131072 gathered rows of 2048 bf16 values transposed take 110 us so,
// 125 without; 131072 of 768 in both forms 71 us, as they are 48. (To copy the next tile's values to shared memory
// as well, asynchronously, took 145 us by 16 bytes and 147 by rows: it leaves less of the memory that loads and stores pass through.)
template <typename T, bool Vector>
__global__ void __launch_bounds__(kThreads, kTileCtasPerSm<T>) quantize_kernel(const __grid_constant__ QuantizeArgs a) {
    extern __shared__ __align__(16) unsigned char dynamic_smem[];
    QuantizeSmem<T>& sm = *reinterpret_cast<QuantizeSmem<T>*>(dynamic_smem);
    int32_t* const starts = reinterpret_cast<int32_t*>(dynamic_smem + sizeof(QuantizeSmem<T>));  // [E + 1] row tiles before each expert
    int32_t* const rows = starts + a.E + 1;                                                      // [E + 1] first row of each
    const int lane = threadIdx.x & 31, group = threadIdx.x & 15, row0 = (threadIdx.x >> 4) * 8, warp = threadIdx.x >> 5;
    wait_for_previous_kernel();
    first_rows(rows, a.offsets, a.E, a.M);
    exclusive_sums(starts, a.E, sm.sums, [&](int e) { return (rows[e + 1] - rows[e] + kBlock - 1) / kBlock; });
    const int64_t tiles = int64_t(starts[a.E]) * a.across, step = gridDim.x;

    // The place of the CTA's n-th tile, and which row of src this thread of the first 128 looks for; -1: none.
    auto find = [&](int64_t it, int n) {
        int32_t row = -1;
        if (threadIdx.x < kBlock && it < tiles) {
            const int32_t down = int32_t(quotient(it, a.across));
            const int e = last_at_most(starts, a.E, down);
            const int32_t s0 = rows[e] + (down - starts[e]) * kBlock, held = min(kBlock, rows[e + 1] - s0);
            if (threadIdx.x == 0) sm.place[n & 1] = {s0, held, down, uint32_t(it - int64_t(down) * a.across) * kBlock};
            if (int(threadIdx.x) < held) row = a.tokens ? load_here(a.tokens + s0 + threadIdx.x) : s0 + int(threadIdx.x);
        }
        return row;
    };
    auto found = [&](int32_t row, int n) {
        if (threadIdx.x < kBlock) sm.row_at[n & 1][threadIdx.x] = uint32_t(row) < uint32_t(a.src_rows) ? reinterpret_cast<uint64_t>(static_cast<const T*>(a.src) + row * a.src_stride) : 0;
    };
    int n = 0;
    found(find(blockIdx.x, 0), 0);
    for (int64_t it = blockIdx.x; it < tiles; it += step, ++n) {
        Eight<T> x[8];
        __syncthreads();  // what the tile before wrote has been read, and this one's place and rows are known
        const int32_t s0 = sm.place[n & 1].first, held = sm.place[n & 1].held, down = sm.place[n & 1].down;
        const uint32_t col0 = sm.place[n & 1].col0, col = col0 + group * 8;
        load_tile<Vector>(x, sm.row_at[n & 1], col, a.len);
        const int32_t later = find(it + step, n + 1);
        if (a.out.has_rows) {
            uint32_t m[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = x[i].largest();
            const Scale s = scale_of(largest_of_rows(m));
            const int own = row0 + ((lane & 15) >> 1);
            if ((lane & 1) == 0 && own < held) a.out.rows.scales[int64_t(s0 + own) * a.out.rows.scale_stride + col0 / kBlock] = s.scale;
            char* const codes = static_cast<char*>(a.out.rows.codes) + int64_t(s0) * a.out.rows.stride;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                Eight<T> y = x[i];
                y.scale(Eight<T>::factor(__shfl_sync(kFull, s.inverse, (lane & 16) + 2 * i)));
                put_row(y, i, codes, a.out.rows.stride, held, col, a.len);
            }
        }
        if (a.out.has_columns) {
            Eight<T> m;
            m.zero();
#pragma unroll
            for (int i = 0; i < 8; ++i) m.raise(x[i]);
            m.raise(m.other_half());
            if (lane < 16) sm.largest[warp][group] = m;
            __syncthreads();
            const int64_t block = down;  // of the transposed rows: the experts' tiles lie one after the other
            if (threadIdx.x < kBlock) {
                uint32_t bits = 0;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) bits = max(bits, uint32_t(reinterpret_cast<const typename Eight<T>::Bits*>(sm.largest[w])[threadIdx.x]));
                const Scale s = scale_of(Eight<T>::magnitude(bits));
                sm.column[threadIdx.x] = Eight<T>::factor(s.inverse);
                if (col0 + threadIdx.x < a.len) a.out.columns.scales[block * a.out.columns.scale_stride + col0 + threadIdx.x] = s.scale;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i].scale_each(sm.column + group * 8);
            put_columns(x, sm.turned, static_cast<char*>(a.out.columns.codes) + int64_t(col0) * a.out.columns.stride + block * kBlock, a.out.columns.stride,
                        int(min(uint32_t(kBlock), a.len - col0)), kBlock);
        }
        found(later, n + 1);
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
};

template <bool Vector>
__global__ void __launch_bounds__(kThreads, kTileCtasPerSm<__nv_bfloat16>) all_gather_fp8_kernel(const __grid_constant__ GatherArgs a) {
    __shared__ struct {
        uint64_t row_at[kBlock];  // where each row lies; 0: none
        __align__(16) unsigned char turned[kBlock * kBlock];
    } sm;
    __shared__ uint32_t of_warp[kWarps];
    const int group = threadIdx.x & 15, warp = threadIdx.x >> 5;
    wait_for_previous_kernel();
    for (int64_t it = blockIdx.x; it < a.tiles; it += gridDim.x) {
        const uint32_t each = a.across * a.down, e = quotient(it, each), in = uint32_t(it - int64_t(e) * each), down = in / a.across, across = in - down * a.across;
        const uint32_t n0 = down * kBlock, col0 = across * kBlock, col = col0 + group * 8;
        const int held = int(min(uint32_t(kBlock), a.tv.rows - n0));
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
        load_tile<Vector>(x, sm.row_at, col, a.tv.len);
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
        char* const codes = static_cast<char*>(a.w.codes) + int64_t(e) * a.w.batch + int64_t(n0) * a.w.stride;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i].scale(Eight<__nv_bfloat16>::factor(s.inverse));
            put_row(x[i], i, codes, a.w.stride, held, col, a.tv.len);
        }
        if (a.has_wt)
            put_columns(x, sm.turned, static_cast<char*>(a.wt.codes) + int64_t(e) * a.wt.batch + int64_t(col0) * a.wt.stride + n0, a.wt.stride, int(min(uint32_t(kBlock), a.tv.len - col0)),
                        (held + 15) / 16 * 16);
        __syncthreads();  // what the next tile writes has been read
    }
    let_next_kernel_start();
}

int grid_of(int64_t blocks, const Ctas& c, int64_t most) { return int(std::max<int64_t>(1, std::min<int64_t>(blocks, c.most ? c.most : most))); }

// Whether eight elements can be loaded as vectors of 16 bytes from every row, at every column that is a multiple of 8.
bool vectors(uintptr_t bits, int64_t stride, int64_t rows, int64_t len, int elem) { return bits % 16 == 0 && len % 8 == 0 && (rows <= 1 || stride * elem % 16 == 0); }

template <typename T, bool Vector>
cudaError_t dispatch_fp8(const RowsView& src, int64_t tokens, int k, int64_t len, const int32_t* slots, const tide_fp8_t& rows, const Ctas& c, cudaStream_t stream) {
    const uint32_t stretches = uint32_t((len + 511) / 512);
    const int64_t items = tokens * stretches;
    return launch_after(dispatch_fp8_kernel<T, Vector>, grid_of((items + kWarps - 1) / kWarps, c, INT32_MAX), kThreads, 0, stream, static_cast<const T*>(src.p), src.stride, tokens, k,
                        int32_t(tokens * k), uint32_t(len), slots, rows, stretches, items);
}

template <typename T, bool Vector>
cudaError_t quantize(const QuantizeArgs& a, const Ctas& c, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(quantize_kernel<T, Vector>), quantize_smem<T>(TIDE_MAX_EXPERTS), c.device, allowed);
    if (e != cudaSuccess) return e;
    // CTAs go round with the next tile's place found beforehand; where rows are written and there are 16 tiles for each that fits, more
    // CTAs take 8 each, so that those that come late even out the end (524288 rows of 768 bf16 values 183 us, going round 209; 131072 48
    // going round, 53)
    const int64_t fit = int64_t(c.sms) * kTileCtasPerSm<T>, tiles = padded_blocks(a.M, a.E) * a.across;
    return launch_after(quantize_kernel<T, Vector>, grid_of(tiles, c, a.out.has_rows && tiles >= 16 * fit ? tiles / 8 : fit), kThreads, size_t(quantize_smem<T>(a.E)), stream, a);
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
    a.src = src.p, a.src_stride = src.stride, a.src_rows = int32_t(src_rows), a.M = int32_t(M), a.E = E, a.len = uint32_t(len);
    a.offsets = offsets, a.tokens = tokens;
    a.out.has_rows = rows != nullptr, a.out.has_columns = columns != nullptr;
    if (rows) a.out.rows = *rows;
    if (columns) a.out.columns = *columns;
    a.across = uint32_t((len + kBlock - 1) / kBlock);
    const bool v = src_rows > 0 && vectors(reinterpret_cast<uintptr_t>(src.p), src.stride, src_rows, len, bf16 ? 2 : 4);
    if (bf16) return v ? quantize<__nv_bfloat16, true>(a, c, stream) : quantize<__nv_bfloat16, false>(a, c, stream);
    return v ? quantize<float, true>(a, c, stream) : quantize<float, false>(a, c, stream);
}

cudaError_t launch_all_gather_fp8(const ShardPtrs& shards, const TableView& tv, int E, const ExpertParams& ps, const tide_fp8_t& w, const tide_fp8_t* wt, const Ctas& c,
                                  cudaStream_t stream) {
    GatherArgs a{};
    a.shards = shards, a.tv = tv, a.ps = ps, a.w = w, a.has_wt = wt != nullptr;
    if (wt) a.wt = *wt;
    a.across = (tv.len + kBlock - 1) / kBlock, a.down = (tv.rows + kBlock - 1) / kBlock;
    a.tiles = int64_t(E) * a.across * a.down;
    bool v = vectors(shards.bits, 0, 1, tv.len, 2);
    for (int e = 0; e < E; ++e) v &= ps.off[e] % 8 == 0;
    return launch_after(v ? all_gather_fp8_kernel<true> : all_gather_fp8_kernel<false>, grid_of(a.tiles, c, INT32_MAX), kThreads, 0, stream, a);
}

}  // namespace tide
