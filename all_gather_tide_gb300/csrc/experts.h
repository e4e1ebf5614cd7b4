// The object behind tide_experts_t, and the launches of a layer of experts.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/tide.h"
#include "step_internal.h"

struct tide_experts {
    int32_t E = 0, k = 0;
    uint32_t flags = 0;
    int device = 0, sm_count = 0;
    int* d_status = nullptr;
    std::atomic<uint64_t> timeout_ns{0};
    std::atomic<uint32_t> debug{0};
};

namespace tide {

// The most pairs of a call: with 127 columns for each expert behind its own, their transposed form has columns of 31 bits.
constexpr int64_t kMaxPairs = (int64_t(1) << 31) - (int64_t(1) << 18);
constexpr int kBlock = 128;  // values that share a scale

// The device, and how many CTAs a launch may have (0: as many as it likes).
struct Ctas {
    int sms, most, device;
};

// Lets a kernel have so much shared memory, once on each device; `done` is the kernel's own.
inline cudaError_t allow_smem(const void* kernel, int bytes, int device, std::atomic<uint64_t>& done) {
    const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// ---- order, rows there and back ----
constexpr int kSortThreads = 512;
constexpr int64_t kSortAlone = 2048;   // pairs that one CTA sorts alone
constexpr int64_t kSortPiece = 4096;   // pairs of a CTA whose warps keep theirs in registers
constexpr int kSortCluster = 8;        // CTAs of a cluster
// CTAs of a sort, each of which counts and ranks a piece of the pairs, and whether a launch of its own counts (into a workspace).
struct SortShape {
    int ctas;
    bool counted;
};
SortShape sort_shape(int64_t pairs, const Ctas& c);
cudaError_t launch_sort(const void* ids, int ids64, int64_t pairs, int k, int E, int32_t* offsets, int32_t* slots,
                        int32_t* tokens, int32_t* counts, const Ctas& c, int* status, cudaStream_t stream);

struct RowsView {
    const void* p;
    int64_t stride;  // elements
};
cudaError_t launch_dispatch(const RowsView& src, int bf16, int64_t T, int k, int64_t len, const int32_t* slots, void* rows,
                            int64_t rows_stride, const Ctas& c, cudaStream_t stream);
cudaError_t launch_combine(const RowsView& rows, int bf16, int64_t T, int k, int64_t len, const int32_t* slots, const float* weights,
                           void* out, int64_t out_stride, const Ctas& c, cudaStream_t stream);
cudaError_t launch_combine_grad(const RowsView& dout, const RowsView& rows, int bf16, int64_t T, int k, int64_t len, const int32_t* slots,
                                const float* weights, void* drows, int64_t drows_stride, float* dweights, const Ctas& c, cudaStream_t stream);

// ---- 8-bit matrices ----
// Blocks of 128 columns that the transposed form of M rows of E experts takes at most.
inline int64_t padded_blocks(int64_t M, int32_t E) {
    const int64_t experts = M < E ? M : E;
    return (M + (kBlock - 1) * experts) / kBlock;
}
cudaError_t launch_dispatch_fp8(const RowsView& src, int bf16, int64_t T, int k, int64_t len, const int32_t* slots, const tide_fp8_t& rows,
                                const Ctas& c, cudaStream_t stream);
cudaError_t launch_quantize(const RowsView& src, int bf16, int64_t src_rows, int64_t M, int64_t len, int E, const int32_t* offsets,
                            const int32_t* tokens, const tide_fp8_t* rows, const tide_fp8_t* columns, const Ctas& c, cudaStream_t stream);

// Where the experts' parameters lie in the shards.
struct ExpertParams {
    int64_t off[TIDE_MAX_EXPERTS];  // o_p of each
};
cudaError_t launch_all_gather_fp8(const ShardPtrs& shards, const TableView& tv, int E, const ExpertParams& ps, const tide_fp8_t& w,
                                  const tide_fp8_t* wt, const Ctas& c, cudaStream_t stream);

// ---- products ----
struct GradPtrs {
    void* p[TIDE_MAX_EXPERTS];
};
// How long a wait lasts at most, where it tells that it did not end, and whether to let it (nothing is loaded then).
struct WaitArgs {
    int* status;
    uint64_t timeout_ns;
    bool stall;
};
// TIDE_OK or a negative status.
int launch_matmul(const tide_fp8_t& a, int64_t M, int E, const int32_t* offsets, const tide_fp8_t& w, uint32_t flags, int64_t N, int64_t K,
                  void* out, int out_bf16, int64_t out_stride, const Ctas& c, const WaitArgs& wait, cudaStream_t stream);
int launch_weight_grad(const tide_fp8_t& dy, const tide_fp8_t& a, int64_t M, int E, const int32_t* offsets, uint32_t flags, int64_t N, int64_t K,
                       const GradPtrs& grads, int grad_bf16, const Ctas& c, const WaitArgs& wait, cudaStream_t stream);

}  // namespace tide
