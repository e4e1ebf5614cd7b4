// Internal declarations of the sharded training step: embedding lookup and gradient over the shards,
// and the operators over lists of tensors.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace tide {

// ---- embedding -------------------------------------------------------------------------------
constexpr int kInlineRanks = 64;    // shard pointers that travel with a launch
constexpr int kInlineBatches = 64;  // batches that travel with a launch
// CTAs of 256 threads on an SM, as the kernels' registers are bounded for.
constexpr int kLookupCtasPerSm = 4;
constexpr int kExpandCtasPerSm = 8;
constexpr int kSumCtasPerSm = 4;
constexpr int kShortCtasPerSm = 3;

// The R shard pointers of a call: in the launch's own parameters up to kInlineRanks, else in a device
// table.
struct ShardPtrs {
    void* p[kInlineRanks];
    void* const* table;  // nullptr: use p
    uintptr_t bits;      // all addresses, or'ed: what they are all aligned to
};

// Where a parameter lies in the shards (group layout).
struct TableView {
    uint32_t rows;    // rows_p
    uint32_t m;       // m_p
    uint32_t len;     // L_p
    int64_t off;      // o_p
    int32_t R;
};

// The positions of up to kInlineBatches batches, in order.
struct Batches {
    const void* ids[kInlineBatches];
    const char* dout[kInlineBatches];
    int64_t stride[kInlineBatches];         // bytes between dout rows
    uint32_t start[kInlineBatches + 1];     // first position of every batch, and the end
    int32_t count;
    int32_t ids64;
};

cudaError_t launch_embedding(const ShardPtrs& shards, const TableView& tv, const void* ids, int ids64, int64_t n,
                             float scale, void* out, int out_bf16, int64_t out_stride, int ctas, bool overlap, int* status,
                             cudaStream_t stream);

// Workspace of the gradient, carved from the caller's buffer.
struct GradWorkspace {
    // a position: its dout row's address (x, y) and its table row (z; rows = no token)
    uint4* sorted;       // [N] by row
    uint4* swap_a;       // [N] between passes of the sort
    uint4* swap_b;
    uint4* pre;          // [N] before the sort, when there are more than kInlineBatches batches
    uint32_t* arrived;   // [slots] counts of arrivals
    float* partial;      // [slots][256] partial sums
};
// How the sorted list is summed: pieces of positions, stretches of 256 columns, and slots for partial sums.
struct GradPlan {
    uint32_t piece, pieces, stretches;
    int64_t slots;
};
GradPlan plan_grad(const TableView& tv, int64_t n);
// Carves the workspace for n positions at `base` (any pointer, also null) and returns its size.
size_t carve_grad_workspace(char* base, const TableView& tv, int64_t n, GradWorkspace* w);
// The largest size that up to n positions need.
size_t grad_workspace_size(const TableView& tv, int64_t n);

// ctas: the most that a launch may have.
cudaError_t launch_expand_positions(const Batches& b, uint32_t first, uint32_t rows, const GradWorkspace& w, int ctas,
                                    int* status, cudaStream_t stream);
cudaError_t launch_sort_positions(const Batches& b, bool expanded, const TableView& tv, uint32_t n,
                                  const GradWorkspace& w, int ctas, int* status, cudaStream_t stream);
// dout_vec: every dout row starts on a boundary of 8 elements.
cudaError_t launch_sum_positions(const ShardPtrs& shards, const TableView& tv, uint32_t n, const GradWorkspace& w,
                                 int dout_bf16, bool dout_vec, float scale, bool accumulate, int ctas, bool overlap,
                                 cudaStream_t stream);

// Whether a list goes by one launch that sorts and sums, without a workspace, and that launch.
bool short_list(int64_t n, int32_t batches);
cudaError_t launch_sum_short(const ShardPtrs& shards, const TableView& tv, const Batches& b, uint32_t n, int dout_bf16,
                             bool dout_vec, float scale, bool accumulate, int ctas, int* status, cudaStream_t stream);

// ---- lists of tensors -------------------------------------------------------------------------
constexpr int kTsChunkMost = 2048, kTsChunkLeast = 256;  // elements of one work item
constexpr int kTsThreads = 256;
// CTAs of an SM: the norm and clipping run with all the warps that their registers allow (the norm of
// 856 M bf16 values: 418, 259, 238, 236 us with 1, 2, 3, 4; norm and clipping of 625 M fp32: 1397, 1114,
// 1206, 1121 us), AdamW, whose seven streams they crowd, with two (856 M elements: 4905, 3769, 3845 us
// with 1, 2, 3).
constexpr int kTsCtasPerSm = 4;
constexpr int kAdamwCtasPerSm = 2;

// One work item: elements [i*chunk, i*chunk + left) of tensor k, left cut off at chunk + 8.
struct TsItem {
    int32_t k;
    uint32_t i;
    int32_t left;
    int32_t bf16;  // the gradient's type
};

struct AdamwArgs {
    float beta1, one_minus_beta1, beta2, one_minus_beta2, eps, step_size, inv_sqrt_c2;
    const float* norm;  // nullptr: no clipping
    float max_norm;
    float lr;
    int skip_nonfinite, write_shards, has_decay;
};

struct TsList {
    const TsItem* items;
    int64_t chunks;
    int32_t K;
    int32_t chunk;  // elements of a work item
};

cudaError_t launch_grad_norm(const TsList& l, const void* const* grads, double* partial, unsigned* ticket, float* norm,
                             double* sumsq, int ctas, cudaStream_t stream);
cudaError_t launch_clip(const TsList& l, void* const* grads, const float* norm, float max_norm, int ctas,
                        cudaStream_t stream);
// The norm and clipping by it in two launches, the second of which ends the norm's sum.
cudaError_t launch_clip_norm(const TsList& l, void* const* grads, double* partial, float* norm, float max_norm, int ctas,
                             cudaStream_t stream);
// tables: K pointers each of params, grads, exp_avg, exp_avg_sq and, where they are written, shards,
// then, where there is any, K floats of weight decay.
cudaError_t launch_adamw(const TsList& l, void* const* tables, const AdamwArgs& a, int ctas, cudaStream_t stream);

}  // namespace tide
