// C ABI of the operators over lists of tensors: the list object, argument checks and launches.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <vector>

#include "api_common.h"
#include "step_internal.h"
#include "table_ring.h"

// The list behind tide_tensors_t.
struct tide_tensors {
    int32_t K = 0;
    std::vector<int64_t> elems;
    std::vector<uint8_t> bf16;
    int64_t chunks = 0;
    int32_t chunk = tide::kTsChunkMost;
    int device = 0;
    int sm_count = 0;
    char* d_block = nullptr;       // tickets, partial sums and items in one allocation
    unsigned* d_ticket = nullptr;  // one per ring slot
    double* d_partial = nullptr;   // max_ctas per ring slot
    tide::TsItem* d_items = nullptr;
    tide::TableRing ring;
    std::mutex mu;

    int max_ctas() const { return sm_count * tide::kTsCtasPerSm; }
    double* partial(int slot) const { return d_partial + int64_t(slot) * max_ctas(); }
    tide::TsList list() const { return {d_items, chunks, K, chunk}; }
};

namespace {

using tide::aligned;
using tide::no_throw;

constexpr int64_t kMaxElems = int64_t(1) << 38;
constexpr int64_t kItemsWanted = 152 * 32;  // the warps of a GB300 at four CTAs an SM

void release(tide_tensors* t) {
    t->ring.release();
    if (t->d_block) cudaFree(t->d_block);
    delete t;
}

// Checks the pointers of the tensors that have elements; elem: bytes of theirs, 0 for gradients.
bool good_pointers(const tide_tensors* t, const void* const* ptrs, size_t elem) {
    for (int k = 0; k < t->K; ++k)
        if (t->elems[k] > 0 && (!ptrs[k] || !aligned(ptrs[k], elem ? elem : t->bf16[k] ? 2 : 4))) return false;
    return true;
}

// A slot that holds the gradients' pointers.  A table that the ring holds already was checked when it
// came.
int upload_grads(tide_tensors* t, const void* const* grads, cudaStream_t st, int* slot) {
    const tide::TableRing::Part part{grads, size_t(t->K)};
    int rc = tide::check_device(t->device);
    if (rc == TIDE_OK) rc = tide::check_not_captured(st);
    if (rc != TIDE_OK) return rc;
    if ((*slot = t->ring.find(&part, 1, st)) >= 0) return TIDE_OK;
    if (!good_pointers(t, grads, 0)) return TIDE_EINVAL;
    TIDE_CUDA(t->ring.put(&part, 1, st, slot));
    return TIDE_OK;
}

// Marks the slot's table as in use by what `st` holds, and passes on the launches' status.
int finish(tide_tensors* t, int slot, cudaStream_t st, cudaError_t launched) {
    const cudaError_t e = t->ring.finish(slot, st);
    if (launched != cudaSuccess) return tide::record_cuda_error(launched);
    return e == cudaSuccess ? TIDE_OK : tide::record_cuda_error(e);
}

// A float in the first half of a table entry.
uint64_t word_of(float v) {
    uint64_t w = 0;
    std::memcpy(&w, &v, sizeof v);
    return w;
}

bool bad_max_norm(float v) { return !(v >= 0.0f); }  // NaN too

}  // namespace

extern "C" {

int tide_tensors_create(tide_tensors_t* out, int32_t K, const int64_t* elems, const int32_t* types) {
    return no_throw([&]() -> int {
        if (!out) return TIDE_EINVAL;
        *out = nullptr;
        if (!elems || K < 1) return TIDE_EINVAL;
        if (K > TIDE_MAX_TABLE / 8) return TIDE_ERANGE;
        std::vector<uint8_t> bf16(static_cast<size_t>(K));
        int64_t total = 0;
        for (int k = 0; k < K; ++k) {
            if (elems[k] < 0) return TIDE_EINVAL;
            if (types && types[k] != TIDE_F32 && types[k] != TIDE_BF16) return TIDE_EINVAL;
            if (elems[k] > kMaxElems || (total += elems[k]) > kMaxElems) return TIDE_ERANGE;
            bf16[size_t(k)] = types && types[k] == TIDE_BF16;
        }
        // short items where long ones would not give every warp of the GPU one
        int chunk = tide::kTsChunkMost;
        while (chunk > tide::kTsChunkLeast && total / chunk < kItemsWanted) chunk >>= 1;
        // one item more than the elements fill, where the first may start up to 7 before the tensor
        auto count = [&](int64_t n) { return n > 0 ? (n + 7 + chunk - 1) / chunk : 0; };
        int64_t chunks = 0;
        for (int k = 0; k < K; ++k) chunks += count(elems[k]);
        std::vector<tide::TsItem> items;
        items.reserve(size_t(chunks));
        for (int k = 0; k < K; ++k)
            for (int64_t i = 0, m = count(elems[k]); i < m; ++i)
                items.push_back({k, uint32_t(i), int32_t(std::min<int64_t>(elems[k] - i * chunk, chunk + 8)), bf16[size_t(k)]});

        tide_tensors* t = new tide_tensors();
        t->K = K;
        t->chunks = chunks;
        t->chunk = chunk;
        cudaError_t e;
        try {
            t->elems.assign(elems, elems + K);
            t->bf16 = std::move(bf16);
            e = cudaGetDevice(&t->device);
            if (e == cudaSuccess) e = cudaDeviceGetAttribute(&t->sm_count, cudaDevAttrMultiProcessorCount, t->device);
            const size_t ticket_bytes = 256, partial_bytes = size_t(tide::kSlots) * size_t(t->max_ctas()) * sizeof(double);
            const size_t item_bytes = items.size() * sizeof(tide::TsItem);
            if (e == cudaSuccess) e = cudaMalloc(&t->d_block, ticket_bytes + partial_bytes + item_bytes);
            if (e == cudaSuccess) {
                t->d_ticket = reinterpret_cast<unsigned*>(t->d_block);
                t->d_partial = reinterpret_cast<double*>(t->d_block + ticket_bytes);
                t->d_items = reinterpret_cast<tide::TsItem*>(t->d_block + ticket_bytes + partial_bytes);
                e = cudaMemset(t->d_ticket, 0, ticket_bytes);
            }
            if (e == cudaSuccess && item_bytes) e = cudaMemcpy(t->d_items, items.data(), item_bytes, cudaMemcpyHostToDevice);
            if (e == cudaSuccess) e = tide::wait_for_uploads();
            // five pointers and a factor for every tensor
            if (e == cudaSuccess) e = t->ring.create(size_t(K) * 6);
        } catch (...) {
            release(t);
            throw;
        }
        if (e != cudaSuccess) {
            release(t);
            tide::record_cuda_error(e);
            return e == cudaErrorMemoryAllocation ? TIDE_ENOMEM : TIDE_ECUDA;
        }
        *out = t;
        return TIDE_OK;
    });
}

int tide_tensors_destroy(tide_tensors_t t) {
    if (t) release(t);
    return TIDE_OK;
}

int tide_grad_norm(tide_tensors_t t, const void* const* grads, float* norm, double* sumsq, void* stream) {
    return no_throw([&]() -> int {
        if (!t || !grads || !norm || !aligned(norm, 4) || !aligned(sumsq, 8)) return TIDE_EINVAL;
        std::lock_guard<std::mutex> lock(t->mu);
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        int slot;
        const int rc = upload_grads(t, grads, st, &slot);
        if (rc != TIDE_OK) return rc;
        return finish(t, slot, st,
                      tide::launch_grad_norm(t->list(), t->ring.slots[slot].dev, t->partial(slot), t->d_ticket + slot, norm, sumsq, t->max_ctas(), st));
    });
}

int tide_clip_grads(tide_tensors_t t, void* const* grads, const float* norm, float max_norm, void* stream) {
    return no_throw([&]() -> int {
        if (!t || !grads || !norm || !aligned(norm, 4) || bad_max_norm(max_norm)) return TIDE_EINVAL;
        std::lock_guard<std::mutex> lock(t->mu);
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        int slot;
        const int rc = upload_grads(t, grads, st, &slot);
        if (rc != TIDE_OK) return rc;
        return finish(t, slot, st, tide::launch_clip(t->list(), t->ring.slots[slot].dev, norm, max_norm, t->max_ctas(), st));
    });
}

int tide_clip_grad_norm(tide_tensors_t t, void* const* grads, float max_norm, float* norm, void* stream) {
    return no_throw([&]() -> int {
        if (!t || !grads || !norm || !aligned(norm, 4) || bad_max_norm(max_norm)) return TIDE_EINVAL;
        std::lock_guard<std::mutex> lock(t->mu);
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        int slot;
        const int rc = upload_grads(t, grads, st, &slot);
        if (rc != TIDE_OK) return rc;
        return finish(t, slot, st, tide::launch_clip_norm(t->list(), t->ring.slots[slot].dev, t->partial(slot), norm, max_norm, t->max_ctas(), st));
    });
}

int tide_adamw(tide_tensors_t t, void* const* params, const void* const* grads, void* const* exp_avg,
               void* const* exp_avg_sq, void* const* shards, const float* weight_decay, double lr, double beta1,
               double beta2, double eps, int64_t step, const float* norm, float max_norm, uint32_t flags,
               void* stream) {
    return no_throw([&]() -> int {
        if (!t || !params || !grads || !exp_avg || !exp_avg_sq || (flags & ~uint32_t(TIDE_ADAMW_SKIP_NONFINITE))) return TIDE_EINVAL;
        if (!(lr >= 0) || !std::isfinite(lr) || !(eps >= 0) || !std::isfinite(eps) || step < 1) return TIDE_EINVAL;
        if (!(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1)) return TIDE_EINVAL;
        if (norm && (!aligned(norm, 4) || bad_max_norm(max_norm))) return TIDE_EINVAL;
        std::lock_guard<std::mutex> lock(t->mu);
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        int rc = tide::check_device(t->device);
        if (rc == TIDE_OK) rc = tide::check_not_captured(st);
        if (rc != TIDE_OK) return rc;
        const size_t K = size_t(t->K);
        // the weight decays as they are: two to an entry, an odd one alone
        const uint64_t odd = weight_decay && K % 2 ? word_of(weight_decay[K - 1]) : 0;
        tide::TableRing::Part parts[7];
        int count = 0;
        for (const void* p : {static_cast<const void*>(params), static_cast<const void*>(grads), static_cast<const void*>(exp_avg),
                              static_cast<const void*>(exp_avg_sq), static_cast<const void*>(shards)})
            if (p) parts[count++] = {p, K};
        if (weight_decay) {
            parts[count++] = {weight_decay, K / 2};
            parts[count++] = {&odd, K % 2};
        }
        int slot = t->ring.find(parts, count, st);
        if (slot < 0) {
            if (!good_pointers(t, params, 4) || !good_pointers(t, grads, 0) || !good_pointers(t, exp_avg, 4) ||
                !good_pointers(t, exp_avg_sq, 4) || (shards && !good_pointers(t, shards, 2)))
                return TIDE_EINVAL;
            for (size_t k = 0; weight_decay && k < K; ++k)
                if (!(weight_decay[k] >= 0) || !std::isfinite(weight_decay[k])) return TIDE_EINVAL;
            TIDE_CUDA(t->ring.put(parts, count, st, &slot));
        }
        tide::AdamwArgs a{};
        a.beta1 = float(beta1);
        a.one_minus_beta1 = float(1.0 - beta1);
        a.beta2 = float(beta2);
        a.one_minus_beta2 = float(1.0 - beta2);
        a.eps = float(eps);
        a.step_size = float(lr / (1.0 - std::pow(beta1, double(step))));
        a.inv_sqrt_c2 = float(1.0 / std::sqrt(1.0 - std::pow(beta2, double(step))));
        a.norm = norm;
        a.max_norm = max_norm;
        a.skip_nonfinite = (flags & TIDE_ADAMW_SKIP_NONFINITE) ? 1 : 0;
        a.lr = float(lr);
        a.write_shards = shards ? 1 : 0;
        a.has_decay = weight_decay ? 1 : 0;
        return finish(t, slot, st, tide::launch_adamw(t->list(), t->ring.slots[slot].dev, a, t->sm_count * tide::kAdamwCtasPerSm, st));
    });
}

}  // extern "C"
