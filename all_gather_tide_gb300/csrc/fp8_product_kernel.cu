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
#include "copies_end.h"
#include "experts_device.cuh"

namespace tide {
namespace {

constexpr int kTileM = 128;
constexpr int kSumWarps = 8;
// A warp each for TMA and MMA, two for the scales, eight that take the sums out, two more for the scales.
constexpr int kScaledThreads = 32 * (4 + kSumWarps + 2);
constexpr int kAnyThreads = 32 * (4 + kSumWarps);
constexpr int kTmemCols = 512;
constexpr int kStatusWait = 1, kStatusScale = 2;

constexpr int kRingBytes = 196608, kMostStages = 11;

struct ProductArgs {
    CUtensorMap a, b;
    CUtensorMap result;  // boxes of 32 rows of 64 bytes, where `bulk`
    const float* a_scales;  // product: [row][block]; gradient: [block][row]
    const float* b_scales;  // product: [expert][column / 128][block], or transposed; gradient: [block][column]
    int64_t a_scale_stride, b_scale_stride, b_scale_batch;
    int transposed;
    const int32_t* offsets;
    int32_t M, E;
    int32_t a_box;  // rows of A that a copy brings, a multiple of 8: fewer than 128 where there are no more
    int32_t N, K;  // columns of the result, blocks' length in all (product only)
    int32_t rows;  // rows of the result (gradient only)
    void* out;
    int64_t out_stride;
    int scale_vectors;  // scales that lie side by side can be read four at a time
    int bulk;         // the result can be written by TMA
    int out_vectors;  // and 16 bytes of a row at a time
    WaitArgs wait;
};
// The ring of stages. A CTA's share of a stage is the rows of A that a copy brings and its part of B's BN, half of them where two CTAs
// work on one tile. Where A has few rows in all, more stages fit (products read 128 rows there all the same, those behind
// A's being B's): 8 rows of 2048 by 1536 columns of 128 experts take 9.6 us with six stages.
template <int BN, bool Pair>
struct Ring {
    int share, stages;
    __device__ __forceinline__ explicit Ring(const ProductArgs& p) {
        share = (Pair ? kTileM + BN / 2 : p.a_box + BN) * kBlock;
        stages = Pair ? kRingBytes / ((kTileM + BN / 2) * kBlock) : min(kMostStages, kRingBytes / share);
    }
    // Where B's rows begin in a stage.
    __device__ __forceinline__ int b_at(const ProductArgs& p) const { return (Pair ? kTileM : p.a_box) * kBlock; }
};
struct GradArgs : ProductArgs {
    GradPtrs grads;
};
template <bool Grad>
using ArgsOf = typename std::conditional<Grad, GradArgs, ProductArgs>::type;

// Where the result of expert e lies.
template <bool Grad>
__device__ __forceinline__ void* result_of(const ArgsOf<Grad>& p, int e) {
    if constexpr (Grad) return p.grads.p[e];
    else return p.out;
}

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
// The barrier at the same place of the pair's first CTA.
__device__ __forceinline__ uint32_t of_first_cta(uint64_t* bar) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_u32(bar)));
    return at;
}
// Arrivals at the barrier of the pair's first CTA, whose products read and write both CTAs' memory.
//
// Of Tensor Memory, whose accesses have ended (tcgen05.wait) and are fenced by tcgen05.fence on both sides: the arrival orders nothing
// else, so it is relaxed. (A release of the cluster's scope waits for all of the thread's loads and stores, here those of a tile of the
// result: 2000 cycles.)
template <bool Pair>
__device__ __forceinline__ void arrive_after_tensor_memory(uint64_t* bar) {
    if constexpr (Pair) asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(of_first_cta(bar)) : "memory");
    else barrier_arrive(bar);
}
// Of shared memory that this CTA has written: a release of the cluster's scope, by a thread without loads and stores of its own.
__device__ __forceinline__ void arrive_after_shared_memory(uint64_t* bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(of_first_cta(bar)) : "memory");
}
__device__ __forceinline__ bool barrier_try(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}
// The same where threads of the other CTA of a pair arrive too, or its products and copies do.
template <bool Pair>
__device__ __forceinline__ bool barrier_try_both(uint64_t* bar, uint32_t parity) {
    if constexpr (!Pair) return barrier_try(bar, parity);
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}

// Waits of a CTA: each gives up after the limit, and then all do.
struct Waits {
    volatile int* stop;
    int* status;
    uint64_t limit;
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        return until([&] { return barrier_try(bar, parity); });
    }
    template <bool Pair>
    __device__ __forceinline__ bool both(uint64_t* bar, uint32_t parity) const {
        return until([&] { return barrier_try_both<Pair>(bar, parity); });
    }
    template <typename Try>
    __device__ __forceinline__ bool until(Try&& done) const {
        if (done()) return true;
        const uint64_t end = globaltimer() + limit;
        while (!done()) {
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

// One lane of a whole warp. The warps that issue copies and products run as a whole up to there, so that addresses and
// descriptors stay in uniform registers: with a branch for one lane around the loop, a block's four products took 450 ns to issue.
__device__ __forceinline__ bool elected() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// A position in a ring: its index and how often it has come round.
struct Cursor {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int size) {
        if (++at == size) at = 0, phase ^= 1;
    }
};

// Boxes of codes; a pair's count at the barrier of its first CTA.
template <bool Pair>
__device__ __forceinline__ void load_2d(void* to, const CUtensorMap* map, int32_t x, int32_t y, uint64_t* bar) {
    if constexpr (Pair)
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(to)), "l"(map), "r"(x),
                     "r"(y), "r"(of_first_cta(bar))
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(to)), "l"(map), "r"(x), "r"(y),
                     "r"(smem_u32(bar))
                     : "memory");
}
template <bool Pair>
__device__ __forceinline__ void load_3d(void* to, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint64_t* bar) {
    if constexpr (Pair)
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(to)), "l"(map), "r"(x),
                     "r"(y), "r"(z), "r"(of_first_cta(bar))
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(to)), "l"(map), "r"(x), "r"(y),
                     "r"(z), "r"(smem_u32(bar))
                     : "memory");
}

// A tile of rows of 128 bytes, swizzled in groups of 8 rows (1024 bytes), K along the row.
__device__ __forceinline__ uint64_t tile_descriptor(const void* tile) {
    return uint64_t((smem_u32(tile) & 0x3ffff) >> 4) | uint64_t(1) << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}
// Instruction descriptors: fp32 sums of e4m3 products, both operands K-major, BN columns; with scales, exponents of 8 bits.
__host__ __device__ constexpr uint32_t plain_instruction(int bn) { return 1u << 4 | uint32_t(bn >> 3) << 17 | uint32_t(kTileM >> 4) << 24; }
__host__ __device__ constexpr uint32_t scaled_instruction(int bn, bool pair) { return 1u << 23 | uint32_t(bn >> 3) << 17 | uint32_t((pair ? 2 * kTileM : kTileM) >> 4) << 24; }

__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t instruction, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(instruction),
                 "r"(uint32_t(add))
                 : "memory");
}
// The same with a power of two for each row of A and of B, whose exponents lie in Tensor Memory: row r's in lane r % 32 (and
// at the same place in each quarter), column r / 32, in the byte that the instruction names.
template <bool Pair>
__device__ __forceinline__ void multiply_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t instruction, uint32_t a_scales, uint32_t b_scales, bool add) {
    if constexpr (Pair)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\ttcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(instruction), "r"(a_scales), "r"(b_scales), "r"(uint32_t(add))
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\ttcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(instruction), "r"(a_scales), "r"(b_scales), "r"(uint32_t(add))
                     : "memory");
}
// 128 rows' exponents, 16 bytes for each of 32 lanes, into four columns of all quarters; a pair's CTAs each their own.
template <bool Pair>
__device__ __forceinline__ void copy_exponents(uint32_t to, const void* from) {
    const uint64_t descriptor = uint64_t((smem_u32(from) & 0x3ffff) >> 4) | uint64_t(128 >> 4) << 32 | uint64_t(1) << 46;
    if constexpr (Pair) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(to), "l"(descriptor) : "memory");
    else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(to), "l"(descriptor) : "memory");
}
// The barrier, that of each CTA of a pair, is arrived at when all that this thread issued has ended.
template <bool Pair>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if constexpr (Pair)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)), "h"(uint16_t(3)) : "memory");
    else
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
    int e, row0, rows_end, col0;  // rows row0.. (to rows_end; of A too) and columns col0.. of the result
    int k0, blocks;               // first column of both operands, blocks of 128 of them
};

// Tiles of `Rows` rows and BN columns.
template <int Rows, int BN, bool Grad>
struct Tiles {
    const ProductArgs& p;
    const int32_t* starts;  // [E + 1] before each expert: tiles down the result, or blocks of a gradient's operands
    const int32_t* first;   // [E + 1] first row of each expert
    uint32_t across, down;
    int64_t count;
    // All of the block's threads call it.
    __device__ __forceinline__ Tiles(const ProductArgs& p, int32_t* starts, int32_t* first, int32_t* sums)
        : p(p), starts(starts), first(first), across(uint32_t((p.N + BN - 1) / BN)), down(uint32_t((p.rows + Rows - 1) / Rows)) {
        constexpr int kUnit = Grad ? kBlock : Rows;
        first_rows(first, p.offsets, p.E, p.M);
        exclusive_sums(starts, p.E, sums, [&](int e) { return (first[e + 1] - first[e] + kUnit - 1) / kUnit; });
        count = Grad ? int64_t(p.E) * across * down : int64_t(starts[p.E]) * across;
    }
    __device__ __forceinline__ Tile at(int64_t it) const {
        Tile t;
        if (Grad) {
            const uint32_t each = across * down;
            t.e = int(quotient(it, each));
            const uint32_t in = uint32_t(it - int64_t(t.e) * each), d = in / across;
            t.row0 = int(d) * Rows, t.rows_end = p.rows, t.col0 = int(in - d * across) * BN;
            t.k0 = starts[t.e] * kBlock, t.blocks = starts[t.e + 1] - starts[t.e];
        } else {
            const int32_t d = int32_t(quotient(it, across));
            t.e = last_at_most(starts, p.E, d);
            t.row0 = first[t.e] + (d - starts[t.e]) * Rows;
            t.rows_end = first[t.e + 1];
            t.col0 = int(it - int64_t(d) * across) * BN;
            t.k0 = 0, t.blocks = (p.K + kBlock - 1) / kBlock;
        }
        return t;
    }
};

// The loads of all of a CTA's tiles; a pair's CTAs each load their rows of A and their half of B's.
template <int BN, bool Pair, bool Grad, typename Tiles>
__device__ __forceinline__ void load_tiles(const ProductArgs& p, const Tiles& tiles, int rank, int64_t begin, int64_t step, unsigned char* ring, uint64_t* full, uint64_t* empty,
                                           const Waits& wait) {
    const Ring<BN, Pair> r(p);
    const int b_at = r.b_at(p);
    Cursor s;
    int64_t uses = 0;
    bool ok = true;
    if (p.wait.stall) return;
    for (int64_t it = begin; ok && it < tiles.count; it += step) {
        const Tile t = tiles.at(it);
        const int row = t.row0 + rank * kTileM, col = t.col0 + rank * (BN / 2);
        for (int b = 0; b < t.blocks; ++b) {
            if (!(ok = __all_sync(kFull, wait.both<Pair>(&empty[s.at], s.phase ^ 1)))) break;
            unsigned char* a = ring + s.at * r.share;
            if (elected()) {
                if (rank == 0) barrier_expect(&full[s.at], Pair ? 2 * (p.a_box + BN / 2) * kBlock : r.share);
                load_2d<Pair>(a, &p.a, t.k0 + b * kBlock, row, &full[s.at]);
                if (Grad) load_2d<Pair>(a + b_at, &p.b, t.k0 + b * kBlock, col, &full[s.at]);
                else load_3d<Pair>(a + b_at, &p.b, b * kBlock, col, t.e, &full[s.at]);
            }
            __syncwarp();
            s.next(r.stages);
            ++uses;
        }
    }
    // No copy, and no arrival of the products that read it, is left on its way to this CTA's memory. Copies are counted as landed
    // at the barriers of the first CTA alone.
    struct {
        uint64_t *full, *empty;
        const volatile int* stop;
        bool counts;
        __device__ __forceinline__ uint64_t now() const { return globaltimer(); }
        __device__ __forceinline__ bool stopped() const { return *stop != 0; }
        __device__ __forceinline__ bool ended(int stage, uint32_t parity) const { return barrier_try(&empty[stage], parity); }
        __device__ __forceinline__ bool landed(int stage, uint32_t parity) const { return counts && barrier_try(&full[stage], parity); }
    } const at{full, empty, wait.stop, rank == 0};
    wait_for_last_uses(uses, r.stages, !ok, p.wait.timeout_ns, at);
}

// The products on their way end before the Tensor Memory is given back.
template <bool Pair>
__device__ __forceinline__ void end_products(uint64_t* ended) {
    if (elected()) commit<Pair>(ended);
    const uint64_t end = globaltimer() + 100000000ull;
    while (!barrier_try(ended, 0) && globaltimer() < end) {
    }
}

// Sums of a row, of which `left` columns are there.
template <typename Out, int Count>
__device__ __forceinline__ void put_sums(Out* to, const uint32_t (&x)[Count], int left, bool vectors) {
    constexpr int kStep = 16 / sizeof(Out);
#pragma unroll
    for (int j = 0; j < Count; j += kStep) {
        float v[kStep];
#pragma unroll
        for (int i = 0; i < kStep; ++i) v[i] = __uint_as_float(x[j + i]);
        if (vectors && j + kStep <= left) {
            put(to + j, v);
        } else {
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
                const float one[1] = {v[i]};
                if (j + i < left) put(to + j + i, one);
            }
        }
    }
}

// A warp's 32 rows of sums go to the result by way of 2 KB of shared memory, 64 bytes of each row at a time, in which 16-byte pieces
// are swizzled as the tensor map says: whole boxes by TMA, others (an expert's last rows, rows' odd ends, results that TMA cannot
// address) row by row. A lane's own stores would reach 32 lines an instruction: those of all eight warps bounded short products, and of two
// bytes each took 10 us for a tile.
constexpr int kStagingBytes = 2048;  // a warp
template <bool Grad, typename Out>
__device__ __forceinline__ void put_staged(const ArgsOf<Grad>& p, unsigned char* staging, const uint32_t (&w)[16], int e, int row0, int rows, int col) {
    constexpr int kCols = 64 / sizeof(Out);
    const int lane = threadIdx.x & 31;
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the bytes before have been read
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(staging + lane * 64 + (i ^ (lane >> 1 & 3)) * 16) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    // TMA writes whole boxes, so all of the rows have to be there, and where it cuts a row's end it writes up to a multiple of 16 bytes
    if (p.bulk && rows >= 32 && (col + kCols <= p.N || p.N % (16 / int(sizeof(Out))) == 0)) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            if constexpr (Grad)
                asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(&p.result), "r"(col), "r"(row0), "r"(e), "r"(smem_u32(staging)) : "memory");
            else
                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(&p.result), "r"(col), "r"(row0), "r"(smem_u32(staging)) : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        return;
    }
    __syncwarp();
    Out* const to = static_cast<Out*>(result_of<Grad>(p, e)) + row0 * p.out_stride + col;
    if (p.out_vectors && col + kCols <= p.N) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 8 * i + lane / 4, piece = lane & 3;
            if (row < rows) *reinterpret_cast<uint4*>(to + row * p.out_stride + piece * (16 / sizeof(Out))) = *reinterpret_cast<const uint4*>(staging + row * 64 + (piece ^ (row >> 1 & 3)) * 16);
        }
    } else {
        // row kRows * i + r of step i; its swizzle depends on i alone
        constexpr int kRows = 32 / kCols;
        const int c = lane % kCols, r = lane / kCols, piece = c * int(sizeof(Out)) / 16;
        const unsigned char* from = staging + r * 64 + c * int(sizeof(Out)) % 16;
        const int left = col + c < p.N ? rows - r : 0;
        Out* at = to + r * p.out_stride + c;
#pragma unroll
        for (int i = 0; i < 32 / kRows; ++i, at += kRows * p.out_stride)
            if (kRows * i < left) *at = *reinterpret_cast<const Out*>(from + i * kRows * 64 + (piece ^ (kRows * i >> 1 & 3)) * 16);
    }
}
// 32 sums of each row, in that way; `rows` of the warp's rows are there.
template <bool Grad, typename Out>
__device__ __forceinline__ void put_sums_staged(const ArgsOf<Grad>& p, unsigned char* staging, const uint32_t (&x)[32], int e, int row0, int rows, int col) {
    constexpr int kCols = 64 / sizeof(Out);
    if (rows <= 0) return;
    if constexpr (sizeof(Out) == 4) {
        // 16 rows of 128 bytes at a time (64 bytes of 32 rows at a time, 120000 rows of 384 by 1203 columns take 247 us, so 170)
        if (!p.out_vectors) {
            const int lane = threadIdx.x & 31, here = min(rows, 32);
            float* to = static_cast<float*>(result_of<Grad>(p, e)) + row0 * p.out_stride + col + lane;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                __syncwarp();
                if (lane >> 4 == h)
#pragma unroll
                    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(staging + (lane & 15) * 128 + (i ^ (lane & 7)) * 16) = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                __syncwarp();
                const unsigned char* const from = staging + (lane & 3) * 4;
                const int left = col + lane < p.N ? here - 16 * h : 0;
#pragma unroll
                for (int i = 0; i < 16; ++i, to += p.out_stride)
                    if (i < left) *to = *reinterpret_cast<const float*>(from + i * 128 + (lane >> 2 ^ (i & 7)) * 16);
            }
            return;
        }
    }
#pragma unroll
    for (int c = 0; c < 32; c += kCols) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if constexpr (sizeof(Out) == 2) w[i] = pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
            else w[i] = x[c + i];
        }
        if (col + c < p.N) put_staged<Grad, Out>(p, staging, w, e, row0, min(rows, 32), col + c);
    }
}

// ---- scales that are powers of two ------------------------------------------------------------------
//
// Two warps turn the scales of A's rows and B's into exponents, four blocks' to a word, from where the MMA thread copies them
// to Tensor Memory once for those blocks. Two tiles' sums lie there at a time, so that one's are taken out while the next is
// multiplied; for BN = 256 they share 32 columns, as the exponents need 24 of the 512: the warps that hold the
// shared columns take these out first and the next tile begins then.
//
// With Pair two CTAs, on the two SMs of a cluster, work on one tile of 256 rows and BN columns: each loads 128 rows of A
// and half of B's, the first one's MMA thread multiplies for both, and each takes out its own rows. An SM's shared memory then
// takes in and gives out 32 KB each for 512 cycles of products, of the 128 bytes a cycle that it has for both; a tile of
// 128 x 256 of its own needs 48 KB each, 768 cycles.
constexpr int kAhead = 4;  // blocks in a word
// Groups of four blocks whose exponents lie there at once, and from which column on: of a wide tile 2 of 4 + 8 columns, of a narrow one,
// whose groups are short, 8 of 4 + 4.
__host__ __device__ constexpr int exponent_groups(int bn) { return bn == 256 ? 2 : 8; }
__host__ __device__ constexpr int exponent_column(int bn) { return bn == 256 ? 480 : 256; }
__host__ __device__ constexpr int exponent_words(int bn) { return (bn + 127) / 128 * 4; }  // of B for each lane
__host__ __device__ constexpr int exponent_bytes(int bn) { return 512 + 128 * exponent_words(bn); }
__host__ __device__ constexpr int second_tile(int bn) { return bn == 256 ? 224 : bn; }  // column of the other tile's sums

// Four scales' exponents, biased, a byte each.
__device__ __forceinline__ uint32_t exponents_of(float a, float b, float c, float d) {
    return (__float_as_uint(a) >> 23 & 0xffu) | (__float_as_uint(b) >> 15 & 0xff00u) | (__float_as_uint(c) >> 7 & 0xff0000u) | (__float_as_uint(d) << 1 & 0xff000000u);
}
// Whether a scale is neither a power of two from 2^-126 on nor NaN.
__device__ __forceinline__ bool no_power(float scale) {
    const uint32_t bits = __float_as_uint(scale);
    return (bits & 0x807fffffu) != 0 ? (bits & 0x7fffffffu) <= 0x7f800000u : bits == 0;
}

// The exponents of A's rows, 128 from `row0` of the tile on, or of B's BN: one warp writes every other group of four blocks, the even or
// odd ones as `which` says. What a lane loads of a group, while it writes the one before:
//   a product's A: the four blocks of rows lane, lane + 32, lane + 64 and lane + 96, v[i];
//   a product's B: the four blocks of 32 columns, which have one scale: v[0] of lane i those of columns 32*i on;
//   a gradient's: rows 4*lane to 4*lane + 3, and these + 128, of block q, v[q] and v[4 + q].
// Per group it takes 4 to 8 loads and some 60 instructions: with a load for each scale, and their addresses, the writers, not the
// products, bounded the gradient (438 us for 187).
template <int BN, bool Pair, bool Grad, bool OfA, bool Vectors, typename Tiles>
__device__ __forceinline__ void write_exponents(const ProductArgs& p, const Tiles& tiles, int row0, int which, int64_t begin, int64_t step, unsigned char* exponents, uint64_t* full,
                                                uint64_t* empty, const Waits& wait) {
    constexpr int kWords = OfA ? 4 : exponent_words(BN), kSets = kWords / 4, kLoads = Grad ? 4 * kSets : OfA ? 4 : 1;
    const int lane = threadIdx.x & 31;
    uint32_t before = 0;  // groups before the tile
    Cursor buffer;
    buffer.at = which;
    bool bad = false;
    for (int64_t it = begin; it < tiles.count; it += step) {
        const Tile t = tiles.at(it);
        const int groups = (t.blocks + kAhead - 1) / kAhead, own = (which - int(before)) & 1;
        before += groups;
        if (own >= groups) continue;
        const int from = (OfA ? t.row0 : t.col0) + row0, end = OfA ? t.rows_end : p.N;
        const int64_t stride = OfA ? p.a_scale_stride : p.b_scale_stride;
        // rows past the last read the last one's, or what lies in the same 16 bytes
        const float* at[Grad ? kSets : kLoads];
#pragma unroll
        for (int i = 0; i < (Grad ? kSets : kLoads); ++i) {
            if (Grad) at[i] = (OfA ? p.a_scales : p.b_scales) + t.k0 / kBlock * stride + min(from + 4 * lane + 128 * i, (end - 1) & ~3);
            else if (OfA) at[i] = p.a_scales + min(from + lane + 32 * i, end - 1) * stride;
            else {
                const int n = min(from + 32 * min(lane, kWords - 1), end - 1) / kBlock;
                at[i] = p.b_scales + t.e * p.b_scale_batch + (p.transposed ? n : n * stride);
            }
        }
        auto load = [&](float4 (&v)[kLoads], int g) {
            if (g >= groups) return;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                if (Grad) {
                    const float* x = at[i / 4] + min(kAhead * g + i % 4, t.blocks - 1) * stride;
                    const int left = end - 1 - min(from + 4 * lane + 128 * (i / 4), (end - 1) & ~3);
                    if constexpr (Vectors) v[i] = *reinterpret_cast<const float4*>(x);
                    else v[i] = make_float4(x[0], x[min(1, left)], x[min(2, left)], x[min(3, left)]);
                } else {
                    const int b = kAhead * g, last = t.blocks - 1;
                    const int64_t each = OfA || !p.transposed ? 1 : stride;
                    if constexpr (Vectors) v[i] = *reinterpret_cast<const float4*>(at[i] + b);
                    else v[i] = make_float4(at[i][b * each], at[i][min(b + 1, last) * each], at[i][min(b + 2, last) * each], at[i][min(b + 3, last) * each]);
                }
            }
        };
        const bool look = OfA ? t.col0 == 0 : t.row0 == (Grad ? 0 : tiles.first[t.e]);
        auto write = [&](float4 (&v)[kLoads], int g) {
            uint32_t w[kWords];
            if (Grad) {
#pragma unroll
                for (int i = 0; i < kSets; ++i) {
                    const float4 &a = v[4 * i], &b = v[4 * i + 1], &c = v[4 * i + 2], &d = v[4 * i + 3];
                    w[4 * i] = exponents_of(a.x, b.x, c.x, d.x), w[4 * i + 1] = exponents_of(a.y, b.y, c.y, d.y);
                    w[4 * i + 2] = exponents_of(a.z, b.z, c.z, d.z), w[4 * i + 3] = exponents_of(a.w, b.w, c.w, d.w);
                }
            } else if (OfA) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = exponents_of(v[i].x, v[i].y, v[i].z, v[i].w);
            } else {
                const uint32_t own_word = exponents_of(v[0].x, v[0].y, v[0].z, v[0].w);
#pragma unroll
                for (int i = 0; i < kWords; ++i) w[i] = __shfl_sync(kFull, own_word, i);
            }
            // the first tile in each row or column of tiles looks whether they are powers of two
            if (look)
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    const float x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int row = from + (Grad ? 4 * lane + 128 * (i / 4) + j : OfA ? lane + 32 * i : lane < kWords ? 32 * lane : 1 << 30), block = kAhead * g + (Grad ? i % 4 : j);
                        bad |= row < end && block < t.blocks && no_power(x[j]);
                    }
                }
            load(v, g + 2);
            if (!__all_sync(kFull, wait.both<Pair>(&empty[buffer.at], buffer.phase ^ 1))) return false;
            unsigned char* const to = exponents + buffer.at * exponent_bytes(BN);
            if (Grad) {
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    const int row = 4 * lane + (i & 3);
                    *reinterpret_cast<uint32_t*>(to + 512 * (i / 4) + (row & 31) * 16 + (row >> 5) * 4) = w[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < kWords; i += 4) *reinterpret_cast<uint4*>(to + 128 * i + lane * 16) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) barrier_arrive(&full[buffer.at]);
            buffer.next(exponent_groups(BN));
            buffer.next(exponent_groups(BN));
            return true;
        };
        float4 x[kLoads];
        load(x, own);
        for (int g = own; g < groups; g += 2)
            if (!write(x, g)) return;
    }
    if (bad) atomicCAS(p.wait.status, 0, kStatusScale);
}

// The second CTA of a pair: of each group of four blocks, its writers arrive at its own barrier, and the warp that waits there, which has no
// other loads and stores, tells the first CTA.
template <int BN, typename Tiles>
__device__ __forceinline__ void hand_over_exponents(const Tiles& tiles, int64_t begin, int64_t step, uint64_t* full, const Waits& wait) {
    Cursor g;
    for (int64_t it = begin; it < tiles.count; it += step) {
        const int blocks = tiles.at(it).blocks;
        for (int b = 0; b < blocks; b += kAhead) {
            if (!__all_sync(kFull, wait(&full[g.at], g.phase))) return;
            if (elected()) arrive_after_shared_memory(&full[g.at]);
            __syncwarp();
            g.next(exponent_groups(BN));
        }
    }
}

// All threads of the CTA, or of both of a pair.
template <bool Pair>
__device__ __forceinline__ void both_ctas() {
    __syncwarp();
    if constexpr (Pair) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else __syncthreads();
}

template <int BN, bool Pair, bool Grad, typename Out>
__global__ void __launch_bounds__(kScaledThreads, 1) scaled_product_kernel(const __grid_constant__ ArgsOf<Grad> p) {
    constexpr int kChunks = BN / 32, kFirstHalf = (kChunks + 1) / 2, kExponentGroups = exponent_groups(BN), kGroupCols = 4 + exponent_words(BN);
    constexpr int kCtas = Pair ? 2 : 1;
    constexpr bool kShared = second_tile(BN) < BN;
    extern __shared__ unsigned char dynamic_smem[];
    unsigned char* const ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dynamic_smem) + 1023) & ~uintptr_t(1023));
    unsigned char* const staging = ring + kRingBytes;
    unsigned char* const exponents = staging + kSumWarps * kStagingBytes;
    __shared__ __align__(8) uint64_t full[kMostStages], empty[kMostStages], scales_full[kExponentGroups], scales_empty[kExponentGroups], ready[2], drained[2], taken, ended;
    __shared__ uint32_t tmem_at;
    __shared__ int stopped;
    __shared__ int32_t starts[TIDE_MAX_EXPERTS + 1], first[TIDE_MAX_EXPERTS + 1], sums[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = Pair ? blockIdx.x & 1 : 0;
    const int64_t begin = blockIdx.x / kCtas, step = gridDim.x / kCtas;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMostStages; ++s) barrier_init(&full[s], 1), barrier_init(&empty[s], 1);
        for (int i = 0; i < kExponentGroups; ++i) barrier_init(&scales_full[i], Pair && rank == 0 ? 3 : 2), barrier_init(&scales_empty[i], 1);
        for (int i = 0; i < 2; ++i) barrier_init(&ready[i], 1);
        for (int i = 0; i < 2; ++i) barrier_init(&drained[i], kSumWarps * kCtas);
        barrier_init(&taken, kSumWarps / 2 * kCtas), barrier_init(&ended, 1);
        stopped = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        if constexpr (Pair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_at)), "r"(kTmemCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_at)), "r"(kTmemCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    both_ctas<Pair>();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_at;
    wait_for_previous_kernel();
    const Tiles<kCtas * kTileM, BN, Grad> tiles(p, starts, first, sums);
    const Waits wait{&stopped, p.wait.status, p.wait.timeout_ns};

    if (warp == 0) {
        load_tiles<BN, Pair, Grad>(p, tiles, rank, begin, step, ring, full, empty, wait);
    } else if (warp == 1) {
        if (rank == 0) {
            const Ring<BN, Pair> r(p);
            const int b_at = r.b_at(p);
            const uint64_t first_a = tile_descriptor(ring);
            Cursor s, g;
            uint32_t tile = 0;
            bool ok = true;
            int blocks = begin < tiles.count ? tiles.at(begin).blocks : 0, next = 0;
            for (int64_t it = begin; ok && it < tiles.count; it += step, blocks = next) {
                if (blocks == 0) {
                    next = it + step < tiles.count ? tiles.at(it + step).blocks : 0;
                    continue;
                }
                const uint32_t to = tmem + (tile & 1) * second_tile(BN);
                // the tile before the last has been taken out, and of the last the columns that it shares
                if (!(ok = tile < 2 || __all_sync(kFull, wait.both<Pair>(&drained[tile & 1], ((tile >> 1) - 1) & 1)))) break;
                if (kShared && !(ok = tile == 0 || __all_sync(kFull, wait.both<Pair>(&taken, (tile - 1) & 1)))) break;
                for (int b0 = 0; ok && b0 < blocks; b0 += kAhead) {
                    if (!(ok = __all_sync(kFull, wait.both<Pair>(&scales_full[g.at], g.phase)))) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const unsigned char* x = exponents + g.at * exponent_bytes(BN);
                    const uint32_t a_scales = tmem + exponent_column(BN) + g.at * kGroupCols, b_scales = a_scales + 4;
                    if (elected()) {
                        copy_exponents<Pair>(a_scales, x);
#pragma unroll
                        for (int i = 0; i < exponent_words(BN) / 4; ++i) copy_exponents<Pair>(b_scales + 4 * i, x + 512 * (1 + i));
                        commit<Pair>(&scales_empty[g.at]);
                    }
                    __syncwarp();
                    g.next(kExponentGroups);
#pragma unroll
                    for (int q = 0; q < kAhead; ++q) {
                        const int b = b0 + q;
                        if (b >= blocks) break;
                        if (!(ok = __all_sync(kFull, wait.both<Pair>(&full[s.at], s.phase)))) break;
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        const uint64_t da = first_a + uint32_t(s.at * r.share >> 4), db = da + uint32_t(b_at >> 4);
                        const uint32_t instruction = scaled_instruction(BN, Pair) | uint32_t(q) << 29 | uint32_t(q) << 4;
                        if (elected()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) multiply_scaled<Pair>(to, da + 2 * k, db + 2 * k, instruction, a_scales, b_scales, b > 0 || k > 0);
                            commit<Pair>(&empty[s.at]);
                            if (b + 1 == blocks) commit<Pair>(&ready[tile & 1]);
                        }
                        __syncwarp();
                        s.next(r.stages);
                    }
                    // the next tile is found while this one's products wait for their turn
                    if (b0 == 0) next = it + step < tiles.count ? tiles.at(it + step).blocks : 0;
                }
                ++tile;
            }
            if (!ok) end_products<Pair>(&ended);
        } else {
            hand_over_exponents<BN>(tiles, begin, step, scales_full, wait);
        }
    } else if (warp < 4 || warp >= 4 + kSumWarps) {
        // warps 2 and 3 write A's and B's exponents of every other group, the last two of the others
        const bool vectors = p.scale_vectors && (Grad || (warp & 1) == 0 || !p.transposed);
        if ((warp & 1) == 0) {
            if (vectors) write_exponents<BN, Pair, Grad, true, true>(p, tiles, rank * kTileM, warp >= 4, begin, step, exponents, scales_full, scales_empty, wait);
            else write_exponents<BN, Pair, Grad, true, false>(p, tiles, rank * kTileM, warp >= 4, begin, step, exponents, scales_full, scales_empty, wait);
        } else {
            if (vectors) write_exponents<BN, Pair, Grad, false, true>(p, tiles, 0, warp >= 4, begin, step, exponents + 512, scales_full, scales_empty, wait);
            else write_exponents<BN, Pair, Grad, false, false>(p, tiles, 0, warp >= 4, begin, step, exponents + 512, scales_full, scales_empty, wait);
        }
    } else {
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const int first_col = half * kFirstHalf * 32, chunks = half ? kChunks - kFirstHalf : kFirstHalf;
        const uint32_t from = tmem + (uint32_t(quarter * 32) << 16) + first_col;
        uint32_t tile = 0;
        bool ok = true;
        for (int64_t it = begin; ok && it < tiles.count; it += step) {
            const Tile t = tiles.at(it);
            const int row0 = t.row0 + rank * kTileM + quarter * 32, rows = t.rows_end - row0, col = t.col0 + first_col;
            unsigned char* const mine = staging + (warp - 4) * kStagingBytes;
            if (t.blocks == 0) {
                const uint32_t none[32] = {};
                for (int c = 0; c < chunks; ++c) put_sums_staged<Grad, Out>(p, mine, none, t.e, row0, rows, col + c * 32);
                continue;
            }
            ok = __all_sync(kFull, wait.both<Pair>(&ready[tile & 1], (tile >> 1) & 1));
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t at = from + (tile & 1) * second_tile(BN);
            // the columns that the next tile's sums share come first: of the first buffer the last, of the second the first
            const bool backwards = kShared && !(tile & 1);
            const bool holds = kShared && half == int(backwards);
            uint32_t x[32];
            auto column = [&](int c) { return (backwards ? chunks - 1 - c : c) * 32; };
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                load_sums(x, at + column(c));
                sums_loaded();
                if ((holds && c == 0) || c + 1 == chunks) {
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        if (holds && c == 0) arrive_after_tensor_memory<Pair>(&taken);
                        if (c + 1 == chunks) arrive_after_tensor_memory<Pair>(&drained[tile & 1]);
                    }
                }
                put_sums_staged<Grad, Out>(p, mine, x, t.e, row0, rows, col + column(c));
            }
            ++tile;
        }
        // what lies in shared memory has been read, and written
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    both_ctas<Pair>();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    let_next_kernel_start();
    if (warp == 2) {
        if constexpr (Pair) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// ---- any scales --------------------------------------------------------------------------------------
//
// Every block is multiplied into one of the Tensor Memory's buffers, and eight warps read the buffer's fp32 sums, multiply
// them with the block's scales and add them to the tile's sums in registers, while the next block is multiplied into another
// buffer. No sum of more than 128 products is formed before its scale is applied.
template <int BN, bool Grad, typename Out>
__global__ void __launch_bounds__(kAnyThreads, 1) any_scales_kernel(const __grid_constant__ ArgsOf<Grad> p) {
    constexpr int kBuffers = kTmemCols / BN, kHalf = BN / 2, kChunks = kHalf / 32;
    static_assert(kBuffers % 2 == 0, "a buffer's number tells whether a block is odd");
    extern __shared__ unsigned char dynamic_smem[];
    unsigned char* const ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dynamic_smem) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full[kMostStages], empty[kMostStages], ready[kBuffers], drained[kBuffers], ended;
    __shared__ uint32_t tmem_at;
    __shared__ int stopped;
    __shared__ int32_t starts[TIDE_MAX_EXPERTS + 1], first[TIDE_MAX_EXPERTS + 1], sums[32];
    __shared__ __align__(16) float column_scales[Grad ? kSumWarps : 1][Grad ? 2 : 1][kHalf];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMostStages; ++s) barrier_init(&full[s], 1), barrier_init(&empty[s], 1);
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
    const Tiles<kTileM, BN, Grad> tiles(p, starts, first, sums);
    const Waits wait{&stopped, p.wait.status, p.wait.timeout_ns};

    if (warp == 0) {
        load_tiles<BN, false, Grad>(p, tiles, 0, blockIdx.x, gridDim.x, ring, full, empty, wait);
    } else if (warp == 1) {
        const Ring<BN, false> r(p);
        const int b_at = r.b_at(p);
        Cursor s, d;
        bool ok = true;
        for (int64_t it = blockIdx.x; ok && it < tiles.count; it += gridDim.x) {
            const Tile t = tiles.at(it);
            for (int b = 0; b < t.blocks; ++b) {
                if (!(ok = __all_sync(kFull, wait(&drained[d.at], d.phase ^ 1) && wait(&full[s.at], s.phase)))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const unsigned char* a = ring + s.at * r.share;
                const uint64_t da = tile_descriptor(a), db = tile_descriptor(a + b_at);
                if (elected()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) multiply(tmem + d.at * BN, da + 2 * k, db + 2 * k, plain_instruction(BN), k > 0);
                    commit<false>(&empty[s.at]);
                    commit<false>(&ready[d.at]);
                }
                __syncwarp();
                s.next(r.stages), d.next(kBuffers);
            }
        }
        if (!ok) end_products<false>(&ended);
    } else if (warp >= 4) {
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t from = tmem + (uint32_t(quarter * 32) << 16) + half * kHalf;
        Cursor d;
        bool ok = true;
        for (int64_t it = blockIdx.x; ok && it < tiles.count; it += gridDim.x) {
            const Tile t = tiles.at(it);
            const int row = t.row0 + quarter * 32 + lane, col = t.col0 + half * kHalf;
            uint64_t acc[kHalf / 2];
#pragma unroll
            for (int j = 0; j < kHalf / 2; ++j) acc[j] = 0;
            // The scales of the row and of the columns' block, one block ahead.  For a gradient, whose scales lie side by side
            // for each block, the lanes have the columns' scales between them and hand them round through shared memory: two buffers
            // in turn, over the tiles' ends too, so that all lanes have met once between a buffer's last read and its next write.
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
                float* const mine = column_scales[Grad ? warp - 4 : 0][Grad ? d.at & 1 : 0];
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
                put_sums(static_cast<Out*>(result_of<Grad>(p, t.e)) + row * p.out_stride + col, x, p.N - col, p.out_vectors);
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

// The result for TMA: `batches` matrices (0: one) of `rows` rows of `N` elements, if they lie as it needs them.
int describe_result(ProductArgs* p, const void* at, int bf16, int64_t N, int64_t rows, int64_t stride, int64_t batches, int64_t batch_bytes) {
    const int elem = bf16 ? 2 : 4;
    p->bulk = aligned(at, 16) && stride * elem % 16 == 0 && stride * elem < int64_t(1) << 40 && (batches <= 1 || (batch_bytes > 0 && batch_bytes % 16 == 0 && batch_bytes < int64_t(1) << 40));
    if (!p->bulk) return TIDE_OK;
    decltype(&cuTensorMapEncodeTiled) encode;
    const int rc = encoder(&encode);
    if (rc != TIDE_OK) return rc;
    const cuuint64_t dims[3] = {cuuint64_t(N), cuuint64_t(rows), cuuint64_t(batches)};
    const cuuint64_t strides[2] = {cuuint64_t(stride * elem), cuuint64_t(batches > 1 ? batch_bytes : stride * elem * rows)};
    const cuuint32_t boxes[3] = {cuuint32_t(64 / elem), 32, 1}, steps[3] = {1, 1, 1};
    const CUresult r = encode(&p->result, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, batches > 0 ? 3 : 2, const_cast<void*>(at), dims, strides, boxes, steps,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? TIDE_OK : record_cuda_error(cudaErrorInvalidValue);
}

template <int BN, bool Pair, bool Grad, typename Out>
int launch(const ArgsOf<Grad>& p, bool any_scales, int64_t most_tiles, const Ctas& c, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed[2];
    void (*kernel)(ArgsOf<Grad>) = scaled_product_kernel<BN, Pair, Grad, Out>;
    if constexpr (!Pair)
        if (any_scales) kernel = any_scales_kernel<BN, Grad, Out>;
    const int smem = kRingBytes + 1024 + (any_scales ? 0 : kSumWarps * kStagingBytes + exponent_groups(BN) * exponent_bytes(BN));
    TIDE_CUDA(allow_smem(reinterpret_cast<const void*>(kernel), smem, c.device, allowed[any_scales]));
    const int64_t at_once = (c.most ? c.most : c.sms) / (Pair ? 2 : 1);
    const int64_t tiles = std::max<int64_t>(1, std::min<int64_t>(most_tiles, at_once));
    TIDE_CUDA(launch_clusters_after(kernel, Pair ? 2 : 1, int(tiles * (Pair ? 2 : 1)), any_scales ? kAnyThreads : kScaledThreads, smem, stream, p));
    return TIDE_OK;
}

bool vectors16(const void* p, int64_t stride, int64_t rows, int elem) { return aligned(p, 16) && (rows <= 1 || stride * elem % 16 == 0); }

// Whether `down` tiles of 128 rows by N columns, summed over `blocks` whole blocks (a sum of 1027 has eight), go to pairs of CTAs, in tiles of 256 x 256: where
// experts have rows enough to fill them, and these are two rounds or more, or half of a round where sums are long, whose products
// then count for more than a round that is not full (4096 rows of 2048 by 2048 columns of 4 experts 17.6 us, in tiles of 128 x 128
// 24.5; 6000 of 512 by 1024 of 5 experts 9.8 and 9.0). Else tiles are 128 x 128: also where sums go to registers, and where taking
// them out is what lasts, of up to four blocks in fp32 (131072 rows of 512 by 384 columns 46 us, by pairs 55), or eight in rows
// without alignment (6000 of 1027 by 1003 columns 16 and 18). (Pairs' tiles of
// 192 and 224 columns, whose sums share none with the next tile's, were slower at every length: 524288 rows of 2048 by 1536 columns
// 1141 and 1122 us, with 256 1083; 131072 of 768 by 2048 195 and 296, with 256 180.)
bool pairs(int64_t rows, int64_t down, int64_t N, int64_t blocks, bool bf16, bool vectors, bool any_scales, const Ctas& c) {
    const int64_t tiles = down * ((N + 255) / 256);  // of 128 x 256
    return !any_scales && c.most != 1 && rows >= 2 * kTileM && blocks > (bf16 ? -1 : vectors ? 4 : 8) && (tiles >= 2 * c.sms || (2 * tiles >= c.sms && blocks >= 8));
}

template <bool Grad>
int launch_any(const ArgsOf<Grad>& p, bool pair, bool any_scales, int64_t down, int bf16, const Ctas& c, cudaStream_t stream) {
    const int64_t tiles = down * ((p.N + (pair ? 255 : 127)) / (pair ? 256 : 128));
    if (pair) return bf16 ? launch<256, true, Grad, __nv_bfloat16>(p, false, tiles, c, stream) : launch<256, true, Grad, float>(p, false, tiles, c, stream);
    return bf16 ? launch<128, false, Grad, __nv_bfloat16>(p, any_scales, tiles, c, stream) : launch<128, false, Grad, float>(p, any_scales, tiles, c, stream);
}

}  // namespace

int launch_matmul(const tide_fp8_t& a, int64_t M, int E, const int32_t* offsets, const tide_fp8_t& w, uint32_t flags, int64_t N, int64_t K, void* out, int out_bf16,
                  int64_t out_stride, const Ctas& c, const WaitArgs& wait, cudaStream_t stream) {
    if (M <= 0) return TIDE_OK;
    ProductArgs p{};
    const bool any = flags & TIDE_FP8_ANY_SCALES;
    const int64_t down = padded_blocks(M, E);
    p.out_vectors = vectors16(out, out_stride, M, out_bf16 ? 2 : 4);
    const bool pair = pairs(M / E, down, N, K / kBlock, out_bf16, p.out_vectors, any, c);
    p.a_box = int32_t(std::min<int64_t>(kTileM, (M + 7) / 8 * 8));
    int rc = describe(&p.a, a, K, M, 0, p.a_box);
    if (rc == TIDE_OK) rc = describe(&p.b, w, K, N, E, 128);
    if (rc != TIDE_OK) return rc;
    p.a_scales = a.scales, p.a_scale_stride = a.scale_stride;
    p.b_scales = w.scales, p.b_scale_stride = w.scale_stride, p.b_scale_batch = w.scale_batch, p.transposed = (flags & TIDE_FP8_TRANSPOSED) != 0;
    // what such a vector holds behind a row's last scale is read and not used; it is of the same 16 bytes
    p.scale_vectors = aligned(a.scales, 16) && a.scale_stride % 4 == 0 && aligned(w.scales, 16) && w.scale_stride % 4 == 0 && (E == 1 || w.scale_batch % 4 == 0);
    p.offsets = offsets, p.M = int32_t(M), p.E = E, p.N = int32_t(N), p.K = int32_t(K), p.rows = 0;
    p.out = out, p.out_stride = out_stride;
    p.wait = wait;
    if ((rc = describe_result(&p, out, out_bf16, N, M, out_stride, 0, 0)) != TIDE_OK) return rc;
    // `down` counts tiles of 128 rows; of 256 there are fewer
    return launch_any<false>(p, pair, any, down, out_bf16, c, stream);
}

int launch_weight_grad(const tide_fp8_t& dy, const tide_fp8_t& a, int64_t M, int E, const int32_t* offsets, uint32_t flags, int64_t N, int64_t K, const GradPtrs& grads,
                       int grad_bf16, const Ctas& c, const WaitArgs& wait, cudaStream_t stream) {
    GradArgs p{};
    const bool any = flags & TIDE_FP8_ANY_SCALES;
    const int64_t padded = std::max<int64_t>(1, padded_blocks(M, E)) * kBlock;
    const int64_t down = int64_t(E) * ((N + kTileM - 1) / kTileM);
    p.out_vectors = 1;
    for (int e = 0; e < E; ++e) p.out_vectors &= vectors16(grads.p[e], K, N, grad_bf16 ? 2 : 4);
    const bool pair = pairs(N, down, K, M / E / kBlock, grad_bf16, p.out_vectors, any, c);
    if (M > 0) {  // else there is nothing to sum
        int rc = describe(&p.a, dy, padded, N, 0, kTileM);
        if (rc == TIDE_OK) rc = describe(&p.b, a, padded, K, 0, 128);
        if (rc != TIDE_OK) return rc;
    }
    p.a_box = kTileM;
    p.a_scales = dy.scales, p.a_scale_stride = dy.scale_stride;
    p.b_scales = a.scales, p.b_scale_stride = a.scale_stride;
    p.scale_vectors = aligned(dy.scales, 16) && dy.scale_stride % 4 == 0 && aligned(a.scales, 16) && a.scale_stride % 4 == 0;
    p.offsets = offsets, p.M = int32_t(M), p.E = E, p.N = int32_t(K), p.rows = int32_t(N);
    p.grads = grads, p.out_stride = K;
    p.wait = wait;
    // gradients at one distance from each other are one array to TMA
    const int64_t pitch = E > 1 ? static_cast<const char*>(grads.p[1]) - static_cast<const char*>(grads.p[0]) : 0;
    bool even = true;
    for (int e = 2; e < E; ++e) even &= static_cast<const char*>(grads.p[e]) - static_cast<const char*>(grads.p[e - 1]) == pitch;
    if (even) {
        const int rc = describe_result(&p, grads.p[0], grad_bf16, K, N, K, E, pitch);
        if (rc != TIDE_OK) return rc;
    }
    return launch_any<true>(p, pair, any, down, grad_bf16, c, stream);
}

}  // namespace tide
