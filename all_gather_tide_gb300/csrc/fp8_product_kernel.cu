// Products of 8-bit matrices with a scale for each block of 128, an expert's rows at a time (sm_103a, tcgen05).
//
//     out[s, n] = sum over b of sa[s, b] * sw[e, n/128, b] * sum over c in block b of a[s, c] * w[e, n, c]
// and, over the rows of each expert, with a scale for every row of both operands,
//     grad_e[n, c] = sum over b of sdy[n, b] * sa[c, b] * sum over s in block b of dy[n, s] * a[c, s].
//
// Both are C = A * B^T over K in blocks of 128 bytes, one row of a 128-byte swizzled tile. One persistent CTA an SM takes
// tiles of 128 x BN: a thread issues TMA loads of A's and B's blocks into a ring of stages, another each block's four
// tcgen05.mma (K = 32 each) into Tensor Memory, and eight warps take the sums out. Two kernels differ in where the scales
// come in:
//   - scaled_product_kernel, for scales that are powers of two: the tensor cores apply them (the block-scaled form of
//     tcgen05.mma takes an exponent for each row of A and of B), so a tile's sum over all of K stays in Tensor Memory;
//   - any_scales_kernel: every block's sums go to registers, where they are scaled and added.
#include <algorithm>

#include <cuda.h>

#include "api_common.h"
#include "experts_device.cuh"

namespace tide {
namespace {

constexpr int kTileM = 128;
constexpr int kProductThreads = 384;  // a warp each for TMA and MMA, two for the scales, then eight that take the sums out
constexpr int kSumWarps = 8;
constexpr int kTmemCols = 512;
constexpr int kStatusWait = 1, kStatusScale = 2;

template <int BN>
constexpr int kTileBytes = (kTileM + BN) * kBlock;
template <int BN>
constexpr int kStages = 196608 / kTileBytes<BN>;

struct ProductArgs {
    CUtensorMap a, b;
    const float* a_scales;  // product: [row][block]; gradient: [block][row]
    const float* b_scales;  // product: [expert][column / 128][block], or transposed; gradient: [block][column]
    int64_t a_scale_stride, b_scale_stride, b_scale_batch;
    int transposed;
    const int32_t* offsets;
    int32_t M, E;
    int32_t N, K;  // columns of the result, blocks' length in all (product only)
    int32_t rows;  // rows of the result (gradient only)
    int32_t most_blocks;  // of the transposed operands (gradient only)
    void* out;
    int64_t out_stride;
    int out_vectors;  // rows of the result can be written 32 bytes at a time
    GradPtrs grads;
    int* status;
    uint64_t timeout_ns;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return uint32_t(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ uint64_t globaltimer() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ void barrier_init(uint64_t* bar, uint32_t count) { asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory"); }
__device__ __forceinline__ void barrier_arrive(uint64_t* bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory"); }
__device__ __forceinline__ void barrier_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool barrier_try(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}

// Waits of a CTA: each gives up after the limit, and then all do.
struct Waits {
    volatile int* stop;
    int* status;
    uint64_t limit;
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        if (barrier_try(bar, parity)) return true;
        const uint64_t end = globaltimer() + limit;
        while (!barrier_try(bar, parity)) {
            if (*stop) return false;
            if (globaltimer() > end) {
                atomicCAS(status, 0, kStatusWait);
                *stop = 1;
                return false;
            }
        }
        return true;
    }
};

// A position in a ring: its index and how often it has come round.
struct Cursor {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int size) {
        if (++at == size) at = 0, phase ^= 1;
    }
};

__device__ __forceinline__ void load_2d(void* to, const CUtensorMap* map, int32_t x, int32_t y, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(to)), "l"(map), "r"(x), "r"(y),
                 "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void load_3d(void* to, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(to)), "l"(map), "r"(x), "r"(y), "r"(z),
                 "r"(smem_u32(bar))
                 : "memory");
}

// A tile of rows of 128 bytes, swizzled in groups of 8 rows (1024 bytes), K along the row.
__device__ __forceinline__ uint64_t tile_descriptor(const void* tile) {
    return uint64_t((smem_u32(tile) & 0x3ffff) >> 4) | uint64_t(1) << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}
// fp32 sums of e4m3 products, both operands K-major.
template <int BN>
constexpr uint32_t kInstruction = 1u << 4 | uint32_t(BN >> 3) << 17 | uint32_t(kTileM >> 4) << 24;

__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t instruction, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(instruction),
                 "r"(uint32_t(add))
                 : "memory");
}
// The same with a power of two for each row of A and of B, whose exponents lie in Tensor Memory: row r's in lane r % 32 (and
// at the same place in each quarter), column r / 32, lowest byte.
template <int BN>
constexpr uint32_t kScaledInstruction = 1u << 23 | uint32_t(BN >> 3) << 17 | uint32_t(kTileM >> 4) << 24;
__device__ __forceinline__ void multiply_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t instruction, uint32_t a_scales, uint32_t b_scales, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\ttcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(instruction), "r"(a_scales), "r"(b_scales), "r"(uint32_t(add))
                 : "memory");
}
// 128 rows' exponents, 16 bytes for each of 32 lanes, into four columns of all quarters.
__device__ __forceinline__ void copy_exponents(uint32_t to, const void* from) {
    const uint64_t descriptor = uint64_t((smem_u32(from) & 0x3ffff) >> 4) | uint64_t(128 >> 4) << 32 | uint64_t(1) << 46;
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(to), "l"(descriptor) : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 32 columns of this warp's 32 rows.
__device__ __forceinline__ void load_sums(uint32_t (&x)[32], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, "
        "%27, %28, %29, %30, %31}, [%32];"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]),
          "=r"(x[14]), "=r"(x[15]), "=r"(x[16]), "=r"(x[17]), "=r"(x[18]), "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]), "=r"(x[24]), "=r"(x[25]), "=r"(x[26]),
          "=r"(x[27]), "=r"(x[28]), "=r"(x[29]), "=r"(x[30]), "=r"(x[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void sums_loaded() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Pairs of fp32 numbers.
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
    return v;
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t pair_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// What a CTA does next: a tile's operands, blocks and place.
struct Tile {
    int e, row0, rows_end, col0;  // rows row0.. (to rows_end) and columns col0.. of the result
    int a_row, k0, blocks;        // first row of A, first column of both operands, blocks of 128 of them
};

template <int BN, bool Grad>
struct Tiles {
    const ProductArgs& p;
    const int32_t* starts;  // [E + 1] tiles of 128 rows before each expert
    const int32_t* first;   // [E + 1] first row of each expert
    uint32_t across, down;
    // All of the block's threads call it.
    __device__ __forceinline__ Tiles(const ProductArgs& p, int32_t* starts, int32_t* first, int32_t* sums)
        : p(p), starts(starts), first(first), across(uint32_t((p.N + BN - 1) / BN)), down(uint32_t((p.rows + kTileM - 1) / kTileM)) {
        for (int e = threadIdx.x; e <= p.E; e += kProductThreads) {
            const Span s = span_of(p.offsets, min(e, p.E - 1), p.M);
            first[e] = e < p.E ? s.first : s.first + s.count;
        }
        exclusive_sums(starts, p.E, sums, [&](int e) { return (span_of(p.offsets, e, p.M).count + kTileM - 1) / kTileM; });
        if (Grad) {  // whatever the offsets hold, no tile reaches past the transposed operands
            for (int e = threadIdx.x; e <= p.E; e += kProductThreads) starts[e] = min(starts[e], p.most_blocks);
            __syncthreads();
        }
    }
    __device__ __forceinline__ int64_t count() const { return Grad ? int64_t(p.E) * across * down : int64_t(starts[p.E]) * across; }
    __device__ __forceinline__ Tile at(int64_t it) const {
        Tile t;
        if (Grad) {
            const uint32_t each = across * down;
            t.e = int(it / each);
            const uint32_t in = uint32_t(it - int64_t(t.e) * each), d = in / across;
            t.row0 = t.a_row = int(d) * kTileM, t.rows_end = p.rows, t.col0 = int(in - d * across) * BN;
            t.k0 = starts[t.e] * kBlock, t.blocks = starts[t.e + 1] - starts[t.e];
        } else {
            const int32_t d = int32_t(it / across);
            t.e = last_at_most(starts, p.E, d);
            t.row0 = t.a_row = first[t.e] + (d - starts[t.e]) * kTileM;
            t.rows_end = first[t.e + 1];
            t.col0 = int(it - int64_t(d) * across) * BN;
            t.k0 = 0, t.blocks = (p.K + kBlock - 1) / kBlock;
        }
        return t;
    }
};

// The loads of all of a CTA's tiles.
template <int BN, bool Grad>
__device__ __forceinline__ void load_tiles(const ProductArgs& p, const Tiles<BN, Grad>& tiles, int64_t count, unsigned char* ring, uint64_t* full, uint64_t* empty, const Waits& wait) {
    Cursor s;
    int64_t uses = 0;
    bool ok = true;
    for (int64_t it = blockIdx.x; ok && it < count; it += gridDim.x) {
        const Tile t = tiles.at(it);
        for (int b = 0; b < t.blocks; ++b) {
            if (!(ok = wait(&empty[s.at], s.phase ^ 1))) break;
            unsigned char* a = ring + s.at * kTileBytes<BN>;
            barrier_expect(&full[s.at], kTileBytes<BN>);
            load_2d(a, &p.a, t.k0 + b * kBlock, t.a_row, &full[s.at]);
            if (Grad) load_2d(a + kTileM * kBlock, &p.b, t.k0 + b * kBlock, t.col0, &full[s.at]);
            else load_3d(a + kTileM * kBlock, &p.b, b * kBlock, t.col0, t.e, &full[s.at]);
            s.next(kStages<BN>);
            ++uses;
        }
    }
    // no copy, and no arrival of the products that read it, is left on its way to this CTA's memory; a stopped CTA
    // waits for its copies alone
    const bool all = ok && !*wait.stop;
    for (int64_t u = max(int64_t(0), uses - kStages<BN>); u < uses; ++u) {
        const int at = int(u % kStages<BN>);
        const uint32_t parity = uint32_t(u / kStages<BN>) & 1;
        const uint64_t end = globaltimer() + (all ? p.timeout_ns : 100000000ull);
        while (!barrier_try(all ? &empty[at] : &full[at], parity) && globaltimer() < end) {
        }
    }
}

// The products on their way end before the Tensor Memory is given back.
__device__ __forceinline__ void end_products(uint64_t* ended) {
    commit(ended);
    const uint64_t end = globaltimer() + 100000000ull;
    while (!barrier_try(ended, 0) && globaltimer() < end) {
    }
}

__device__ __forceinline__ void put32(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}

// Sums of a row, of which `left` columns are there.
template <typename Out, int Count>
__device__ __forceinline__ void put_sums(Out* to, const uint32_t (&x)[Count], int left, bool vectors) {
    constexpr int kStep = 32 / sizeof(Out);
#pragma unroll
    for (int j = 0; j < Count; j += kStep) {
        if (vectors && j + kStep <= left) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (sizeof(Out) == 2) w[i] = pack(__uint_as_float(x[j + 2 * i]), __uint_as_float(x[j + 2 * i + 1]));
                else w[i] = x[j + i];
            }
            put32(to + j, w);
        } else {
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
                const float v[1] = {__uint_as_float(x[j + i])};
                if (j + i < left) put(to + j + i, v);
            }
        }
    }
}

// ---- scales that are powers of two ------------------------------------------------------------------
//
// Two warps turn the scales of A's rows and B's into exponents beside each stage's tiles, from where the MMA thread copies
// them to Tensor Memory. Two tiles' sums lie there at a time, so that one's are taken out while the next is
// multiplied; for BN = 256 they share 32 columns, as the exponents need 24 of the 512: the warps that hold the
// shared columns take these out first and the next tile begins then.
constexpr int kExponentCols = 480;  // from here on; a stage's take 4 + 8, two stages' lie there
template <int BN>
constexpr int kExponentBytes = 4 * (kTileM + BN);
template <int BN>
constexpr int kSecondTile = BN == 256 ? 224 : BN;  // column of the other tile's sums

// A scale as a power of two's exponent, biased; `count`: whether its row is there and another number is to be told of.
__device__ __forceinline__ uint32_t exponent_of(float scale, bool count, bool& bad) {
    const uint32_t bits = __float_as_uint(scale), e = bits >> 23;
    bad |= count && (((bits & 0x7fffffu) != 0 && e != 255) || e - 1 > 254);
    return e & 255;
}

template <int BN, bool Grad, typename Out>
__global__ void __launch_bounds__(kProductThreads, 1) scaled_product_kernel(const __grid_constant__ ProductArgs p) {
    constexpr int kHalf = BN / 2, kChunks = kHalf / 32, kGroups = BN / 128;
    constexpr bool kShared = kSecondTile<BN> < BN;
    extern __shared__ unsigned char dynamic_smem[];
    unsigned char* const ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dynamic_smem) + 1023) & ~uintptr_t(1023));
    unsigned char* const exponents = ring + kStages<BN> * kTileBytes<BN>;
    __shared__ __align__(8) uint64_t full[kStages<BN>], empty[kStages<BN>], ready[2], drained, ended;
    __shared__ uint32_t tmem_at;
    __shared__ int stopped;
    __shared__ int32_t starts[TIDE_MAX_EXPERTS + 1], first[TIDE_MAX_EXPERTS + 1], sums[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages<BN>; ++s) barrier_init(&full[s], 3), barrier_init(&empty[s], 1);
        barrier_init(&ready[0], 1), barrier_init(&ready[1], 1), barrier_init(&drained, kSumWarps), barrier_init(&ended, 1);
        stopped = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_at)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_at;
    wait_for_previous_kernel();
    const Tiles<BN, Grad> tiles(p, starts, first, sums);
    const int64_t count = tiles.count();
    const Waits wait{&stopped, p.status, p.timeout_ns};

    if (warp == 0 && lane == 0) {
        load_tiles<BN, Grad>(p, tiles, count, ring, full, empty, wait);
    } else if (warp == 1 && lane == 0) {
        Cursor s;
        uint32_t tile = 0, buffer = 0;
        bool ok = true;
        for (int64_t it = blockIdx.x; ok && it < count; it += gridDim.x) {
            const Tile t = tiles.at(it);
            if (t.blocks == 0) continue;
            const uint32_t to = tmem + (tile & 1) * kSecondTile<BN>;
            // where the tile before began to be taken out, the one before that has been
            if (!(ok = tile == 0 || wait(&drained, (tile - 1) & 1))) break;
            for (int b = 0; b < t.blocks; ++b) {
                if (!(ok = wait(&full[s.at], s.phase))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const unsigned char* a = ring + s.at * kTileBytes<BN>;
                const unsigned char* x = exponents + s.at * kExponentBytes<BN>;
                const uint32_t a_scales = tmem + kExponentCols + (buffer & 1) * 12, b_scales = a_scales + 4;
                ++buffer;
                copy_exponents(a_scales, x);
#pragma unroll
                for (int g = 0; g < kGroups; ++g) copy_exponents(b_scales + 4 * g, x + 512 * (1 + g));
                const uint64_t da = tile_descriptor(a), db = tile_descriptor(a + kTileM * kBlock);
#pragma unroll
                for (int k = 0; k < 4; ++k) multiply_scaled(to, da + 2 * k, db + 2 * k, kScaledInstruction<BN>, a_scales, b_scales, b > 0 || k > 0);
                commit(&empty[s.at]);
                s.next(kStages<BN>);
            }
            if (ok) commit(&ready[tile & 1]);
            ++tile;
        }
        if (!ok) end_products(&ended);
    } else if (warp == 2 || warp == 3) {
        // warp 2: A's scales, warp 3: B's; each lane has rows lane, lane + 32, ... and up to four blocks ahead
        constexpr int kAhead = 4;
        const bool of_a = warp == 2;
        const int rows = of_a ? 4 : 4 * kGroups;
        Cursor s;
        bool ok = true, bad = false;
        for (int64_t it = blockIdx.x; ok && it < count; it += gridDim.x) {
            const Tile t = tiles.at(it);
            // scale of (row i, block b) at base[i * row_step + b * step]; rows past the last read the last one's
            const int row0 = of_a ? t.row0 : t.col0, end = of_a ? t.rows_end : p.N;
            const float* base;
            int64_t row_step, step;
            if (Grad) {
                base = (of_a ? p.a_scales + t.k0 / kBlock * p.a_scale_stride : p.b_scales + t.k0 / kBlock * p.b_scale_stride);
                row_step = 1, step = of_a ? p.a_scale_stride : p.b_scale_stride;
            } else if (of_a) {
                base = p.a_scales, row_step = p.a_scale_stride, step = 1;
            } else {
                base = p.b_scales + t.e * p.b_scale_batch;
                row_step = p.transposed ? 1 : p.b_scale_stride, step = p.transposed ? p.b_scale_stride : 1;
            }
            const float* at[4 * kGroups];
#pragma unroll
            for (int i = 0; i < 4 * kGroups; ++i) {
                const int row = min(row0 + lane + 32 * i, end - 1);
                at[i] = base + int64_t(!Grad && !of_a ? row / kBlock : row) * row_step;
            }
            for (int b0 = 0; ok && b0 < t.blocks; b0 += kAhead) {
                float x[kAhead][4 * kGroups];
#pragma unroll
                for (int q = 0; q < kAhead; ++q)
#pragma unroll
                    for (int i = 0; i < 4 * kGroups; ++i)
                        if (i < rows) x[q][i] = at[i][min(b0 + q, t.blocks - 1) * step];
#pragma unroll
                for (int q = 0; q < kAhead; ++q) {
                    if (!ok || b0 + q >= t.blocks) break;
                    ok = __all_sync(kFull, wait(&empty[s.at], s.phase ^ 1));
                    if (!ok) break;
                    unsigned char* to = exponents + s.at * kExponentBytes<BN> + (of_a ? 0 : 512) + lane * 16;
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        if (4 * g >= rows) break;
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = exponent_of(x[q][4 * g + i], row0 + lane + 32 * (4 * g + i) < end, bad);
                        *reinterpret_cast<uint4*>(to + 512 * g) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) barrier_arrive(&full[s.at]);
                    s.next(kStages<BN>);
                }
            }
        }
        if (bad) atomicCAS(p.status, 0, kStatusScale);
    } else if (warp >= 4) {
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t from = tmem + (uint32_t(quarter * 32) << 16) + half * kHalf;
        uint32_t tile = 0;
        bool ok = true;
        for (int64_t it = blockIdx.x; ok && it < count; it += gridDim.x) {
            const Tile t = tiles.at(it);
            const int row = t.row0 + quarter * 32 + lane, col = t.col0 + half * kHalf;
            const bool here = row < t.rows_end;
            Out* const to = static_cast<Out*>(Grad ? p.grads.p[t.e] : p.out) + row * p.out_stride + col;
            if (t.blocks == 0) {
                const uint32_t none[32] = {};
                for (int c = 0; here && c < kChunks; ++c) put_sums(to + c * 32, none, p.N - col - c * 32, p.out_vectors);
                continue;
            }
            ok = __all_sync(kFull, wait(&ready[tile & 1], (tile >> 1) & 1));
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t at = from + (tile & 1) * kSecondTile<BN>;
            // the columns that the next tile's sums share come first: of the first buffer the last, of the second the first
            const bool backwards = kShared && !(tile & 1);
            const bool holds = kShared && half == int(backwards);
            if (!holds && lane == 0) barrier_arrive(&drained);
            uint32_t x[2][32];
            auto column = [&](int c) { return (backwards ? kChunks - 1 - c : c) * 32; };
            load_sums(x[0], at + column(0));
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                sums_loaded();
                if (c + 1 < kChunks) load_sums(x[(c + 1) & 1], at + column(c + 1));
                if (holds && c == 0) {
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    if (lane == 0) barrier_arrive(&drained);
                }
                if (here) put_sums(to + column(c), x[c & 1], p.N - col - column(c), p.out_vectors);
            }
            ++tile;
        }
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    let_next_kernel_start();
    if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// ---- any scales --------------------------------------------------------------------------------------
//
// Every block is multiplied into one of the Tensor Memory's buffers, and eight warps read the buffer's fp32 sums, multiply
// them with the block's scales and add them to the tile's sums in registers, while the next block is multiplied into another
// buffer. No sum of more than 128 products is formed before its scale is applied.
template <int BN, bool Grad, typename Out>
__global__ void __launch_bounds__(kProductThreads, 1) any_scales_kernel(const __grid_constant__ ProductArgs p) {
    constexpr int kBuffers = kTmemCols / BN, kHalf = BN / 2, kChunks = kHalf / 32;
    extern __shared__ unsigned char dynamic_smem[];
    unsigned char* const ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dynamic_smem) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full[kStages<BN>], empty[kStages<BN>], ready[kBuffers], drained[kBuffers], ended;
    __shared__ uint32_t tmem_at;
    __shared__ int stopped;
    __shared__ int32_t starts[TIDE_MAX_EXPERTS + 1], first[TIDE_MAX_EXPERTS + 1], sums[32];
    __shared__ __align__(16) float column_scales[Grad ? kSumWarps : 1][Grad ? 2 : 1][kHalf];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages<BN>; ++s) barrier_init(&full[s], 1), barrier_init(&empty[s], 1);
        for (int b = 0; b < kBuffers; ++b) barrier_init(&ready[b], 1), barrier_init(&drained[b], kSumWarps);
        barrier_init(&ended, 1);
        stopped = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_at)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_at;
    wait_for_previous_kernel();
    const Tiles<BN, Grad> tiles(p, starts, first, sums);
    const int64_t count = tiles.count();
    const Waits wait{&stopped, p.status, p.timeout_ns};

    if (warp == 0 && lane == 0) {
        load_tiles<BN, Grad>(p, tiles, count, ring, full, empty, wait);
    } else if (warp == 1 && lane == 0) {
        Cursor s, d;
        bool ok = true;
        for (int64_t it = blockIdx.x; ok && it < count; it += gridDim.x) {
            const Tile t = tiles.at(it);
            for (int b = 0; b < t.blocks; ++b) {
                if (!(ok = wait(&drained[d.at], d.phase ^ 1) && wait(&full[s.at], s.phase))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const unsigned char* a = ring + s.at * kTileBytes<BN>;
                const uint64_t da = tile_descriptor(a), db = tile_descriptor(a + kTileM * kBlock);
#pragma unroll
                for (int k = 0; k < 4; ++k) multiply(tmem + d.at * BN, da + 2 * k, db + 2 * k, kInstruction<BN>, k > 0);
                commit(&empty[s.at]);
                commit(&ready[d.at]);
                s.next(kStages<BN>), d.next(kBuffers);
            }
        }
        if (!ok) end_products(&ended);
    } else if (warp >= 4) {
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t from = tmem + (uint32_t(quarter * 32) << 16) + half * kHalf;
        Cursor d;
        bool ok = true;
        for (int64_t it = blockIdx.x; ok && it < count; it += gridDim.x) {
            const Tile t = tiles.at(it);
            const int row = t.row0 + quarter * 32 + lane, col = t.col0 + half * kHalf;
            uint64_t acc[kHalf / 2];
#pragma unroll
            for (int j = 0; j < kHalf / 2; ++j) acc[j] = 0;
            // The scales of the row and of the columns' block, one block ahead.  For a gradient, whose scales lie side by side
            // for each block, the lanes have the columns' scales between them and hand them round through shared memory.
            const int n = min(col, p.N - 1) / kBlock;
            const float* row_scales = Grad ? p.a_scales + t.k0 / kBlock * p.a_scale_stride + min(row, p.rows - 1) : p.a_scales + min(row, p.M - 1) * p.a_scale_stride;
            const float* col_scales = Grad ? p.b_scales + t.k0 / kBlock * p.b_scale_stride : p.b_scales + t.e * p.b_scale_batch + (p.transposed ? n : n * p.b_scale_stride);
            const int64_t row_step = Grad ? p.a_scale_stride : 1, col_step = Grad || p.transposed ? p.b_scale_stride : 1;
            constexpr int kColScales = Grad ? kHalf / 32 : 1;
            float next_row = 0, next_col[kColScales] = {};
            auto fetch = [&](int b) {
                if (b >= t.blocks) return;
                next_row = row_scales[b * row_step];
#pragma unroll
                for (int i = 0; i < kColScales; ++i) next_col[i] = col_scales[b * col_step + (Grad ? min(col + i * 32 + lane, p.N - 1) : 0)];
            };
            fetch(0);
            for (int b = 0; b < t.blocks; ++b) {
                const float f = Grad ? next_row : next_row * next_col[0];
                float* const mine = column_scales[Grad ? warp - 4 : 0][Grad ? b & 1 : 0];
                if (Grad) {
#pragma unroll
                    for (int i = 0; i < kColScales; ++i) mine[i * 32 + lane] = next_col[i];
                    __syncwarp();
                }
                fetch(b + 1);
                ok = wait(&ready[d.at], d.phase);
                if (!__all_sync(kFull, ok)) {
                    ok = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint64_t f2 = pair_of(__float_as_uint(f), __float_as_uint(f));
                uint32_t x[2][32];
                load_sums(x[0], from + d.at * BN);
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    sums_loaded();
                    if (c + 1 < kChunks) load_sums(x[(c + 1) & 1], from + d.at * BN + (c + 1) * 32);
                    else {
                        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                        if (lane == 0) barrier_arrive(&drained[d.at]);
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        uint64_t v = pair_of(x[c & 1][2 * j], x[c & 1][2 * j + 1]);
                        if (Grad) v = pair_mul(v, *reinterpret_cast<const uint64_t*>(mine + c * 32 + 2 * j));
                        acc[c * 16 + j] = pair_fma(v, f2, acc[c * 16 + j]);
                    }
                }
                d.next(kBuffers);
            }
            if (ok && row < t.rows_end) {
                uint32_t x[kHalf];
#pragma unroll
                for (int j = 0; j < kHalf / 2; ++j) x[2 * j] = uint32_t(acc[j]), x[2 * j + 1] = uint32_t(acc[j] >> 32);
                put_sums(static_cast<Out*>(Grad ? p.grads.p[t.e] : p.out) + row * p.out_stride + col, x, p.N - col, p.out_vectors);
            }
        }
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    let_next_kernel_start();
    if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// The driver's function that describes a matrix to the TMA unit.
int encoder(decltype(&cuTensorMapEncodeTiled)* f) {
    static std::atomic<void*> found{nullptr};
    void* at = found.load();
    if (!at) {
        cudaDriverEntryPointQueryResult result;
        TIDE_CUDA(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &at, 12000, cudaEnableDefault, &result));
        if (result != cudaDriverEntryPointSuccess || !at) return record_cuda_error(cudaErrorSymbolNotFound);
        found = at;
    }
    *f = reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(at);
    return TIDE_OK;
}

// `batches` matrices of `rows` rows of `len` codes, of which boxes of 128 columns and `box` rows are copied; what lies
// outside reads as zeros.
int describe(CUtensorMap* map, const tide_fp8_t& m, int64_t len, int64_t rows, int64_t batches, int box) {
    decltype(&cuTensorMapEncodeTiled) encode;
    const int rc = encoder(&encode);
    if (rc != TIDE_OK) return rc;
    const cuuint64_t dims[3] = {cuuint64_t(len), cuuint64_t(rows), cuuint64_t(batches)};
    const cuuint64_t strides[2] = {cuuint64_t(m.stride), cuuint64_t(batches > 1 ? m.batch : m.stride * rows)};
    const cuuint32_t boxes[3] = {kBlock, cuuint32_t(box), 1}, steps[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, batches > 0 ? 3 : 2, m.codes, dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? TIDE_OK : record_cuda_error(cudaErrorInvalidValue);
}

template <int BN, bool Grad, typename Out>
int launch(const ProductArgs& p, bool any_scales, int64_t most_tiles, const Ctas& c, cudaStream_t stream) {
    auto* kernel = any_scales ? any_scales_kernel<BN == 256 ? 128 : BN, Grad, Out> : scaled_product_kernel<BN, Grad, Out>;
    const int smem = kStages<BN> * (kTileBytes<BN> + kExponentBytes<BN>) + 1024;
    TIDE_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(most_tiles, c.most ? c.most : c.sms));
    TIDE_CUDA(launch_after(kernel, int(ctas), kProductThreads, smem, stream, p));
    return TIDE_OK;
}

bool vectors32(const void* p, int64_t stride, int64_t rows, int elem) { return aligned(p, 32) && (rows <= 1 || stride * elem % 32 == 0); }

}  // namespace

int launch_matmul(const tide_fp8_t& a, int64_t M, int E, const int32_t* offsets, const tide_fp8_t& w, uint32_t flags, int64_t N, int64_t K, void* out, int out_bf16,
                  int64_t out_stride, const Ctas& c, int* status, uint64_t timeout_ns, cudaStream_t stream) {
    if (M <= 0) return TIDE_OK;
    ProductArgs p{};
    // narrow tiles where wide ones are fewer than the SMs, and for sums in registers
    const bool any = flags & TIDE_FP8_ANY_SCALES;
    const int64_t down = padded_blocks(M, E);
    const bool narrow = any || down * ((N + 255) / 256) < c.sms;
    int rc = describe(&p.a, a, K, M, 0, kTileM);
    if (rc == TIDE_OK) rc = describe(&p.b, w, K, N, E, narrow ? 128 : 256);
    if (rc != TIDE_OK) return rc;
    p.a_scales = a.scales, p.a_scale_stride = a.scale_stride;
    p.b_scales = w.scales, p.b_scale_stride = w.scale_stride, p.b_scale_batch = w.scale_batch, p.transposed = (flags & TIDE_FP8_TRANSPOSED) != 0;
    p.offsets = offsets, p.M = int32_t(M), p.E = E, p.N = int32_t(N), p.K = int32_t(K), p.rows = 0;
    p.out = out, p.out_stride = out_stride, p.out_vectors = vectors32(out, out_stride, M, out_bf16 ? 2 : 4);
    p.status = status, p.timeout_ns = timeout_ns;
    const int64_t tiles = down * ((N + (narrow ? 127 : 255)) / (narrow ? 128 : 256));
    if (out_bf16) return narrow ? launch<128, false, __nv_bfloat16>(p, any, tiles, c, stream) : launch<256, false, __nv_bfloat16>(p, any, tiles, c, stream);
    return narrow ? launch<128, false, float>(p, any, tiles, c, stream) : launch<256, false, float>(p, any, tiles, c, stream);
}

int launch_weight_grad(const tide_fp8_t& dy, const tide_fp8_t& a, int64_t M, int E, const int32_t* offsets, uint32_t flags, int64_t N, int64_t K, const GradPtrs& grads,
                       int grad_bf16, const Ctas& c, int* status, uint64_t timeout_ns, cudaStream_t stream) {
    ProductArgs p{};
    const bool any = flags & TIDE_FP8_ANY_SCALES;
    const int64_t padded = std::max<int64_t>(1, padded_blocks(M, E)) * kBlock;
    const int64_t down = int64_t(E) * ((N + kTileM - 1) / kTileM);
    const bool narrow = any || down * ((K + 255) / 256) < c.sms;
    if (M > 0) {  // else there is nothing to sum
        int rc = describe(&p.a, dy, padded, N, 0, kTileM);
        if (rc == TIDE_OK) rc = describe(&p.b, a, padded, K, 0, narrow ? 128 : 256);
        if (rc != TIDE_OK) return rc;
    }
    p.most_blocks = int32_t(padded / kBlock);
    p.a_scales = dy.scales, p.a_scale_stride = dy.scale_stride;
    p.b_scales = a.scales, p.b_scale_stride = a.scale_stride;
    p.offsets = offsets, p.M = int32_t(M), p.E = E, p.N = int32_t(K), p.rows = int32_t(N);
    p.grads = grads, p.out_stride = K;
    p.out_vectors = 1;
    for (int e = 0; e < E; ++e) p.out_vectors &= vectors32(grads.p[e], K, N, grad_bf16 ? 2 : 4);
    p.status = status, p.timeout_ns = timeout_ns;
    const int64_t tiles = down * ((K + (narrow ? 127 : 255)) / (narrow ? 128 : 256));
    if (grad_bf16) return narrow ? launch<128, true, __nv_bfloat16>(p, any, tiles, c, stream) : launch<256, true, __nv_bfloat16>(p, any, tiles, c, stream);
    return narrow ? launch<128, true, float>(p, any, tiles, c, stream) : launch<256, true, float>(p, any, tiles, c, stream);
}

}  // namespace tide
