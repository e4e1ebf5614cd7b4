// C ABI of the embedding lookup and gradient over a group's shards, and of the placement of its parameters in 8 bits:
// argument checks and launches.
#include <algorithm>
#include <vector>

#include "api_common.h"
#include "experts.h"
#include "group.h"
#include "step_internal.h"

namespace {

using tide::aligned;
using tide::no_throw;

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 2;
constexpr int64_t kMaxRowLen = int64_t(1) << 30;
constexpr int64_t kMaxPositions = (int64_t(1) << 31) - (int64_t(1) << 16);

int table_view(const tide_group* g, int32_t p, tide::TableView* tv) {
    if (p < 0 || p >= g->plan.P) return TIDE_EINVAL;
    if (g->plan.rows[p] > kMaxRows || g->plan.row_len[p] > kMaxRowLen) return TIDE_ERANGE;
    tv->rows = uint32_t(g->plan.rows[p]);
    tv->m = uint32_t(g->plan.m[p]);
    tv->len = uint32_t(g->plan.row_len[p]);
    tv->off = g->plan.o[p];
    tv->R = g->plan.R;
    return TIDE_OK;
}

// Fills the call's shard pointers; more than kInlineRanks of them go through the group's ring (*slot >= 0
// then, to be finished after the launches that read it).
int shard_ptrs(tide_group* g, const void* const* shards, size_t elem, cudaStream_t st, tide::ShardPtrs* sp, int* slot) {
    const int R = g->plan.R;
    sp->bits = 0;
    for (int d = 0; d < R; ++d) {
        if (!shards[d] || !aligned(shards[d], elem)) return TIDE_EINVAL;
        sp->bits |= reinterpret_cast<uintptr_t>(shards[d]);
    }
    *slot = -1;
    sp->table = nullptr;
    if (R <= tide::kInlineRanks) {
        for (int d = 0; d < R; ++d) sp->p[d] = const_cast<void*>(shards[d]);
        for (int d = R; d < tide::kInlineRanks; ++d) sp->p[d] = nullptr;
        return TIDE_OK;
    }
    const int rc = tide::check_not_captured(st);
    if (rc != TIDE_OK) return rc;
    std::vector<const void*> table(shards, shards + R);
    TIDE_CUDA(g->ring.upload(table, st, slot));
    sp->table = g->ring.slots[*slot].dev;
    return TIDE_OK;
}

// Marks the ring's table, if one was used, as in use by what `st` holds, and passes on the launches' status.
int finish(tide_group* g, int slot, cudaStream_t st, int rc) {
    const cudaError_t e = slot >= 0 ? g->ring.finish(slot, st) : cudaSuccess;
    return rc != TIDE_OK ? rc : e == cudaSuccess ? TIDE_OK : tide::record_cuda_error(e);
}

// CTAs the embedding kernels may use: everything, or the few of TIDE_FLAG_OVERLAP.
bool overlap(const tide_group* g) { return (g->flags & TIDE_FLAG_OVERLAP) != 0; }
int ctas_of(const tide_group* g, int per_sm) {
    return overlap(g) ? std::max(1, g->sm_count / 9) : std::max(1, g->sm_count * per_sm);
}

size_t float_size(int32_t type) { return type == TIDE_F32 ? 4 : type == TIDE_BF16 ? 2 : 0; }
size_t id_size(int32_t type) { return type == TIDE_I32 ? 4 : type == TIDE_I64 ? 8 : 0; }

}  // namespace

extern "C" {

int tide_embedding(tide_group_t g, int32_t p, const void* const* shards, const void* ids, int32_t ids_type, int64_t n,
                   float scale, void* out, int32_t out_type, int64_t out_stride, void* stream) {
    return no_throw([&]() -> int {
        if (!g || !shards || n < 0 || !id_size(ids_type) || !float_size(out_type)) return TIDE_EINVAL;
        tide::TableView tv;
        int rc = table_view(g, p, &tv);
        if (rc != TIDE_OK) return rc;
        if (out_stride < tv.len) return TIDE_EINVAL;
        if (n > 0 && (!ids || !out || !aligned(ids, id_size(ids_type)) || !aligned(out, float_size(out_type)))) return TIDE_EINVAL;
        int64_t last;
        if (__builtin_mul_overflow(n, out_stride, &last) || __builtin_mul_overflow(last, int64_t(4), &last)) return TIDE_ERANGE;
        std::lock_guard<std::mutex> lock(g->mu);
        if ((rc = tide::check_device(g->device)) != TIDE_OK) return rc;
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        tide::ShardPtrs sp;
        int slot;
        if ((rc = shard_ptrs(g, shards, 2, st, &sp, &slot)) != TIDE_OK) return rc;
        const cudaError_t e = tide::launch_embedding(sp, tv, ids, ids_type == TIDE_I64, n, scale, out, out_type == TIDE_BF16,
                                                     out_stride, ctas_of(g, tide::kLookupCtasPerSm), overlap(g), g->d_status, st);
        return finish(g, slot, st, e == cudaSuccess ? TIDE_OK : tide::record_cuda_error(e));
    });
}

int tide_embedding_grad_workspace(tide_group_t g, int32_t p, int64_t n, int64_t* bytes) {
    if (!g || !bytes || n < 0) return TIDE_EINVAL;
    tide::TableView tv;
    const int rc = table_view(g, p, &tv);
    if (rc != TIDE_OK) return rc;
    if (n > kMaxPositions) return TIDE_ERANGE;
    *bytes = int64_t(tide::grad_workspace_size(tv, n));
    return TIDE_OK;
}

int tide_embedding_grad(tide_group_t g, int32_t p, int32_t B, const int64_t* n, const void* const* ids, int32_t ids_type,
                        const void* const* douts, const int64_t* dout_stride, int32_t dout_type, float scale,
                        int32_t accumulate, void* const* shards, void* workspace, int64_t workspace_bytes, void* stream) {
    return no_throw([&]() -> int {
        const size_t isz = id_size(ids_type), fsz = float_size(dout_type);
        if (!g || !n || !ids || !douts || !dout_stride || !shards || B < 1 || !isz || !fsz) return TIDE_EINVAL;
        if (accumulate != 0 && accumulate != 1) return TIDE_EINVAL;
        tide::TableView tv;
        int rc = table_view(g, p, &tv);
        if (rc != TIDE_OK) return rc;
        if (B > TIDE_MAX_TABLE / 8) return TIDE_ERANGE;
        int64_t total = 0;
        for (int b = 0; b < B; ++b) {
            if (n[b] < 0 || dout_stride[b] < tv.len) return TIDE_EINVAL;
            if (n[b] > kMaxPositions || (total += n[b]) > kMaxPositions) return TIDE_ERANGE;
            int64_t last;
            if (__builtin_mul_overflow(n[b], dout_stride[b], &last) || __builtin_mul_overflow(last, int64_t(4), &last)) return TIDE_ERANGE;
            if (n[b] > 0 && (!ids[b] || !douts[b] || !aligned(ids[b], isz) || !aligned(douts[b], fsz))) return TIDE_EINVAL;
        }
        // a short list goes without a workspace; one that is given has to be good all the same
        if (total > 0 && (workspace || !tide::short_list(total, B)) &&
            (!workspace || !aligned(workspace, 256) || workspace_bytes < int64_t(tide::carve_grad_workspace(nullptr, tv, total, nullptr))))
            return TIDE_EINVAL;
        std::lock_guard<std::mutex> lock(g->mu);
        if ((rc = tide::check_device(g->device)) != TIDE_OK) return rc;
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        tide::ShardPtrs sp;
        int slot;
        if ((rc = shard_ptrs(g, shards, 4, st, &sp, &slot)) != TIDE_OK) return rc;
        return finish(g, slot, st, [&]() -> int {
            tide::GradWorkspace w{};
            bool dout_vec = true;
            if (total > 0) {
                if (workspace) tide::carve_grad_workspace(static_cast<char*>(workspace), tv, total, &w);
                const bool expanded = B > tide::kInlineBatches;
                tide::Batches bt{};
                bt.ids64 = ids_type == TIDE_I64;
                // more batches than travel with one launch are expanded to rows and addresses first
                for (int32_t b0 = 0, first = 0; b0 < B; b0 += tide::kInlineBatches) {
                    bt.count = std::min(B - b0, tide::kInlineBatches);
                    bt.start[0] = 0;
                    for (int k = 0; k < bt.count; ++k) {
                        bt.ids[k] = ids[b0 + k];
                        bt.dout[k] = static_cast<const char*>(douts[b0 + k]);
                        bt.stride[k] = dout_stride[b0 + k] * int64_t(fsz);
                        bt.start[k + 1] = bt.start[k] + uint32_t(n[b0 + k]);
                        if (n[b0 + k] > 0) dout_vec &= aligned(bt.dout[k], 8 * fsz) && (n[b0 + k] == 1 || bt.stride[k] % int64_t(8 * fsz) == 0);
                    }
                    if (expanded) TIDE_CUDA(tide::launch_expand_positions(bt, uint32_t(first), tv.rows, w, ctas_of(g, tide::kExpandCtasPerSm), g->d_status, st));
                    first += int32_t(bt.start[bt.count]);
                }
                if (tide::short_list(total, B)) {
                    TIDE_CUDA(tide::launch_sum_short(sp, tv, bt, uint32_t(total), dout_type == TIDE_BF16, dout_vec, scale, accumulate != 0,
                                                     ctas_of(g, tide::kShortCtasPerSm), g->d_status, st));
                    return TIDE_OK;
                }
                TIDE_CUDA(tide::launch_sort_positions(bt, expanded, tv, uint32_t(total), w, ctas_of(g, 1), g->d_status, st));
            }
            TIDE_CUDA(tide::launch_sum_positions(sp, tv, uint32_t(total), w, dout_type == TIDE_BF16, dout_vec, scale,
                                                 accumulate != 0, ctas_of(g, tide::kSumCtasPerSm), overlap(g), st));
            return TIDE_OK;
        }());
    });
}

int tide_all_gather_fp8(tide_group_t g, int32_t E, const int32_t* ps, const void* const* shards, const tide_fp8_t* w, const tide_fp8_t* wt, void* stream) {
    return no_throw([&]() -> int {
        if (!g || !ps || !shards || !w || E < 1 || E > TIDE_MAX_EXPERTS) return TIDE_EINVAL;
        tide::TableView tv;
        tide::ExpertParams params{};
        for (int e = 0; e < E; ++e) {
            const int rc = table_view(g, ps[e], &tv);
            if (rc != TIDE_OK) return rc;
            if (g->plan.rows[ps[e]] != g->plan.rows[ps[0]] || g->plan.row_len[ps[e]] != g->plan.row_len[ps[0]]) return TIDE_EINVAL;
            params.off[e] = tv.off;
        }
        const int64_t N = tv.rows, K = tv.len;
        auto extent = [](int64_t n, int64_t each) {
            int64_t v;
            return !__builtin_mul_overflow(n, each, &v) && v < (int64_t(1) << 60);
        };
        for (const tide_fp8_t* m : {w, wt}) {
            if (!m) continue;
            const int64_t rows = m == w ? N : K, len = m == w ? K : N;
            if (!m->codes || !aligned(m->codes, 16) || m->stride % 16 != 0 || m->stride < (len + 15) / 16 * 16 || (E > 1 && (m->batch % 16 != 0 || m->batch < 0))) return TIDE_EINVAL;
            if (!extent(rows, m->stride) || !extent(E, E > 1 ? m->batch : 0)) return TIDE_ERANGE;
        }
        if (!w->scales || !aligned(w->scales, 4) || w->scale_stride < (K + tide::kBlock - 1) / tide::kBlock || (E > 1 && w->scale_batch < 0)) return TIDE_EINVAL;
        if (!extent((N + tide::kBlock - 1) / tide::kBlock, w->scale_stride) || !extent(E, E > 1 ? w->scale_batch : 0)) return TIDE_ERANGE;
        std::lock_guard<std::mutex> lock(g->mu);
        int rc = tide::check_device(g->device);
        if (rc != TIDE_OK) return rc;
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        tide::ShardPtrs sp;
        int slot;
        if ((rc = shard_ptrs(g, shards, 2, st, &sp, &slot)) != TIDE_OK) return rc;
        const cudaError_t e = tide::launch_all_gather_fp8(sp, tv, E, params, *w, wt, {g->sm_count, overlap(g) ? ctas_of(g, 1) : 0, g->device}, st);
        return finish(g, slot, st, e == cudaSuccess ? TIDE_OK : tide::record_cuda_error(e));
    });
}

}  // extern "C"
