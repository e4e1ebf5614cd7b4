// C ABI of a layer of experts: argument checks and launches.
#include <algorithm>
#include <vector>

#include "api_common.h"
#include "experts.h"

namespace {

using tide::aligned;
using tide::no_throw;

constexpr int64_t kMaxLen = int64_t(1) << 30;

size_t float_size(int32_t type) { return type == TIDE_F32 ? 4 : type == TIDE_BF16 ? 2 : 0; }
size_t id_size(int32_t type) { return type == TIDE_I32 ? 4 : type == TIDE_I64 ? 8 : 0; }

tide::Ctas ctas_of(const tide_experts* x) { return {x->sm_count, x->flags & TIDE_FLAG_OVERLAP ? std::max(1, x->sm_count / 9) : 0, x->device}; }
tide::WaitArgs wait_of(const tide_experts* x) { return {x->d_status, x->timeout_ns.load(), (x->debug.load() & TIDE_DEBUG_STALL_PRODUCER) != 0}; }

// `rows` rows of `len` elements, `stride` apart, of which an extent in bytes fits in 64 bits.
int check_extent(int64_t rows, int64_t stride, int64_t elem) {
    int64_t last;
    return __builtin_mul_overflow(rows, stride, &last) || __builtin_mul_overflow(last, elem, &last) ? TIDE_ERANGE : TIDE_OK;
}

// T tokens of k pairs each, rows of `len` elements.
int check_sizes(const tide_experts* x, int64_t T, int64_t len) {
    if (T < 0 || len < 1) return TIDE_EINVAL;
    if (T > tide::kMaxPairs / x->k || len > kMaxLen) return TIDE_ERANGE;
    return TIDE_OK;
}

// A pointer to rows that is needed only where there are any.
int check_rows(const void* p, int64_t rows, int64_t stride, int64_t len, size_t elem) {
    if (stride < len || (rows > 0 && (!p || !aligned(p, elem)))) return TIDE_EINVAL;
    return check_extent(rows, stride, int64_t(elem));
}

// An 8-bit matrix of `rows` rows of `len` codes whose scales have `scale_rows` rows of `scale_len`; `batches` of them.
int check_fp8(const tide_fp8_t& m, int64_t rows, int64_t len, int64_t scale_rows, int64_t scale_len, int64_t batches, bool scales) {
    const int64_t least = (len + 15) / 16 * 16;
    if (m.stride < least || m.stride % 16 != 0 || (scales && m.scale_stride < scale_len)) return TIDE_EINVAL;
    if (m.stride >= int64_t(1) << 40) return TIDE_ERANGE;
    int rc = check_extent(rows, m.stride, 1);
    if (rc == TIDE_OK && scales) rc = check_extent(scale_rows, m.scale_stride, 4);
    if (rc != TIDE_OK) return rc;
    if (rows > 0 && (!m.codes || !aligned(m.codes, 16) || (scales && (!m.scales || !aligned(m.scales, 4))))) return TIDE_EINVAL;
    if (batches > 1) {
        if (m.batch % 16 != 0 || m.batch < 0 || (scales && m.scale_batch < 0)) return TIDE_EINVAL;
        if (m.batch >= int64_t(1) << 40) return TIDE_ERANGE;
        rc = check_extent(batches, m.batch, 1);
        if (rc == TIDE_OK && scales) rc = check_extent(batches, m.scale_batch, 4);
        if (rc != TIDE_OK) return rc;
    }
    return TIDE_OK;
}

int64_t blocks_of(int64_t len) { return (len + tide::kBlock - 1) / tide::kBlock; }

// offsets may be left out where one expert has all rows
int check_offsets(const tide_experts* x, const int32_t* offsets) { return offsets ? (aligned(offsets, 4) ? TIDE_OK : TIDE_EINVAL) : x->E == 1 ? TIDE_OK : TIDE_EINVAL; }

}  // namespace

extern "C" {

int tide_experts_create(tide_experts_t* out, int32_t E, int32_t k, uint32_t flags) {
    if (out) *out = nullptr;
    return no_throw([&]() -> int {
        if (!out || E < 1 || E > TIDE_MAX_EXPERTS || k < 1 || k > TIDE_MAX_CHOICES || (flags & ~TIDE_FLAG_OVERLAP)) return TIDE_EINVAL;
        int dev = 0, sms = 0;
        TIDE_CUDA(cudaGetDevice(&dev));
        TIDE_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
        int* status = nullptr;
        cudaError_t e = cudaMalloc(&status, sizeof(int));
        if (e == cudaSuccess) e = cudaMemset(status, 0, sizeof(int));
        if (e == cudaSuccess) e = tide::wait_for_uploads();
        tide_experts* x = e == cudaSuccess ? new (std::nothrow) tide_experts : nullptr;
        if (!x) {
            if (status) cudaFree(status);
            if (e == cudaSuccess) return TIDE_ENOMEM;
            const int rc = tide::record_cuda_error(e);
            return e == cudaErrorMemoryAllocation ? TIDE_ENOMEM : rc;
        }
        x->E = E, x->k = k, x->flags = flags, x->device = dev, x->sm_count = sms, x->d_status = status;
        x->timeout_ns = tide::kDefaultTimeoutNs;
        *out = x;
        return TIDE_OK;
    });
}

int tide_experts_destroy(tide_experts_t x) {
    if (!x) return TIDE_OK;
    const cudaError_t e = cudaFree(x->d_status);
    delete x;
    return e == cudaSuccess ? TIDE_OK : tide::record_cuda_error(e);
}

int tide_experts_device_status(tide_experts_t x, int32_t* status) {
    if (!x || !status) return TIDE_EINVAL;
    const int rc = tide::check_device(x->device);
    if (rc != TIDE_OK) return rc;
    int v = 0;
    TIDE_CUDA(cudaMemcpy(&v, x->d_status, sizeof(int), cudaMemcpyDeviceToHost));
    if (v) {
        TIDE_CUDA(cudaMemset(x->d_status, 0, sizeof(int)));
        TIDE_CUDA(tide::wait_for_uploads());
    }
    *status = v;
    return TIDE_OK;
}

int tide_experts_set_wait_timeout(tide_experts_t x, uint64_t timeout_ns) {
    if (!x) return TIDE_EINVAL;
    // half of what 64 bits hold at most: the kernels add it to the clock
    x->timeout_ns = timeout_ns == 0 ? tide::kDefaultTimeoutNs : std::min(std::max(timeout_ns, tide::kMinTimeoutNs), UINT64_MAX / 2);
    return TIDE_OK;
}

int tide_experts_set_debug(tide_experts_t x, uint32_t flags) {
    if (!x || (flags & ~TIDE_DEBUG_STALL_PRODUCER)) return TIDE_EINVAL;
    x->debug = flags;
    return TIDE_OK;
}

int tide_experts_sort_workspace(tide_experts_t x, int64_t T, int64_t* bytes) {
    if (!x || !bytes || T < 0) return TIDE_EINVAL;
    if (T > tide::kMaxPairs / x->k) return TIDE_ERANGE;
    const tide::SortShape shape = tide::sort_shape(T * x->k, ctas_of(x));
    *bytes = shape.counted ? (int64_t(shape.ctas) * x->E * 4 + 255) / 256 * 256 : 0;
    return TIDE_OK;
}

int tide_experts_sort(tide_experts_t x, const void* ids, int32_t ids_type, int64_t T, int32_t* offsets, int32_t* slots, int32_t* tokens, void* workspace,
                      int64_t workspace_bytes, void* stream) {
    return no_throw([&]() -> int {
        if (!x || !id_size(ids_type) || !offsets || !aligned(offsets, 4)) return TIDE_EINVAL;
        int64_t bytes;
        int rc = tide_experts_sort_workspace(x, T, &bytes);
        if (rc != TIDE_OK) return rc;
        if (T > 0 && (!ids || !aligned(ids, id_size(ids_type)) || !slots || !aligned(slots, 4) || !tokens || !aligned(tokens, 4))) return TIDE_EINVAL;
        if ((workspace && !aligned(workspace, 256)) || (bytes > 0 && (!workspace || workspace_bytes < bytes))) return TIDE_EINVAL;
        if ((rc = tide::check_device(x->device)) != TIDE_OK) return rc;
        TIDE_CUDA(tide::launch_sort(ids, ids_type == TIDE_I64, T * x->k, x->k, x->E, offsets, slots, tokens, static_cast<int32_t*>(workspace), ctas_of(x), x->d_status,
                                    static_cast<cudaStream_t>(stream)));
        return TIDE_OK;
    });
}

int tide_experts_dispatch(tide_experts_t x, const void* src, int32_t type, int64_t src_stride, int64_t T, int64_t len, const int32_t* slots, void* rows,
                          int64_t rows_stride, void* stream) {
    return no_throw([&]() -> int {
        const size_t elem = float_size(type);
        if (!x || !elem) return TIDE_EINVAL;
        int rc = check_sizes(x, T, len);
        if (rc == TIDE_OK) rc = check_rows(src, T, src_stride, len, elem);
        if (rc == TIDE_OK) rc = check_rows(rows, T * x->k, rows_stride, len, elem);
        if (rc == TIDE_OK) rc = check_rows(slots, T, x->k, x->k, 4);
        if (rc == TIDE_OK) rc = tide::check_device(x->device);
        if (rc != TIDE_OK) return rc;
        TIDE_CUDA(tide::launch_dispatch({src, src_stride}, type == TIDE_BF16, T, x->k, len, slots, rows, rows_stride, ctas_of(x), static_cast<cudaStream_t>(stream)));
        return TIDE_OK;
    });
}

int tide_experts_dispatch_fp8(tide_experts_t x, const void* src, int32_t type, int64_t src_stride, int64_t T, int64_t len, const int32_t* slots, const tide_fp8_t* rows,
                              void* stream) {
    return no_throw([&]() -> int {
        const size_t elem = float_size(type);
        if (!x || !elem || !rows) return TIDE_EINVAL;
        int rc = check_sizes(x, T, len);
        if (rc == TIDE_OK) rc = check_rows(src, T, src_stride, len, elem);
        if (rc == TIDE_OK) rc = check_fp8(*rows, T * x->k, len, T * x->k, blocks_of(len), 1, true);
        if (rc == TIDE_OK) rc = check_rows(slots, T, x->k, x->k, 4);
        if (rc == TIDE_OK) rc = tide::check_device(x->device);
        if (rc != TIDE_OK) return rc;
        TIDE_CUDA(tide::launch_dispatch_fp8({src, src_stride}, type == TIDE_BF16, T, x->k, len, slots, *rows, ctas_of(x), static_cast<cudaStream_t>(stream)));
        return TIDE_OK;
    });
}

int tide_experts_combine(tide_experts_t x, const void* rows, int32_t type, int64_t rows_stride, int64_t T, int64_t len, const int32_t* slots, const float* weights,
                         void* out, int64_t out_stride, void* stream) {
    return no_throw([&]() -> int {
        const size_t elem = float_size(type);
        if (!x || !elem || !aligned(weights, 4)) return TIDE_EINVAL;
        int rc = check_sizes(x, T, len);
        if (rc == TIDE_OK) rc = check_rows(rows, T * x->k, rows_stride, len, elem);
        if (rc == TIDE_OK) rc = check_rows(out, T, out_stride, len, elem);
        if (rc == TIDE_OK) rc = check_rows(slots, T, x->k, x->k, 4);
        if (rc == TIDE_OK) rc = tide::check_device(x->device);
        if (rc != TIDE_OK) return rc;
        TIDE_CUDA(tide::launch_combine({rows, rows_stride}, type == TIDE_BF16, T, x->k, len, slots, weights, out, out_stride, ctas_of(x), static_cast<cudaStream_t>(stream)));
        return TIDE_OK;
    });
}

int tide_experts_combine_grad(tide_experts_t x, const void* dout, int32_t type, int64_t dout_stride, const void* rows, int64_t rows_stride, int64_t T, int64_t len,
                              const int32_t* slots, const float* weights, void* drows, int64_t drows_stride, float* dweights, void* stream) {
    return no_throw([&]() -> int {
        const size_t elem = float_size(type);
        if (!x || !elem) return TIDE_EINVAL;
        int rc = check_sizes(x, T, len);
        if (rc == TIDE_OK) rc = check_rows(dout, T, dout_stride, len, elem);
        if (rc == TIDE_OK) rc = check_rows(rows, T * x->k, rows_stride, len, elem);
        if (rc == TIDE_OK) rc = check_rows(drows, T * x->k, drows_stride, len, elem);
        for (const void* p : {static_cast<const void*>(slots), static_cast<const void*>(weights), static_cast<const void*>(dweights)})
            if (rc == TIDE_OK) rc = check_rows(p, T, x->k, x->k, 4);
        if (rc == TIDE_OK) rc = tide::check_device(x->device);
        if (rc != TIDE_OK) return rc;
        TIDE_CUDA(tide::launch_combine_grad({dout, dout_stride}, {rows, rows_stride}, type == TIDE_BF16, T, x->k, len, slots, weights, drows, drows_stride, dweights,
                                            ctas_of(x), static_cast<cudaStream_t>(stream)));
        return TIDE_OK;
    });
}

int tide_fp8_padded_rows(int64_t M, int32_t E, int64_t* columns) {
    if (!columns || M < 0 || E < 1 || E > TIDE_MAX_EXPERTS) return TIDE_EINVAL;
    if (M > tide::kMaxPairs) return TIDE_ERANGE;
    *columns = tide::padded_blocks(M, E) * tide::kBlock;
    return TIDE_OK;
}

int tide_experts_quantize(tide_experts_t x, const void* src, int32_t type, int64_t src_stride, int64_t src_rows, int64_t M, int64_t len, const int32_t* offsets,
                          const int32_t* tokens, const tide_fp8_t* rows, const tide_fp8_t* columns, void* stream) {
    return no_throw([&]() -> int {
        const size_t elem = float_size(type);
        if (!x || !elem || M < 0 || len < 1 || src_rows < 0 || (!tokens && src_rows < M) || !aligned(tokens, 4)) return TIDE_EINVAL;
        if (M > tide::kMaxPairs || len > kMaxLen || src_rows > tide::kMaxPairs) return TIDE_ERANGE;
        int rc = check_offsets(x, offsets);
        if (rc == TIDE_OK) rc = check_rows(src, src_rows, src_stride, len, elem);
        const int64_t blocks = tide::padded_blocks(M, x->E);
        if (rc == TIDE_OK && rows) rc = check_fp8(*rows, M, len, M, blocks_of(len), 1, true);
        if (rc == TIDE_OK && columns) rc = check_fp8(*columns, M > 0 ? len : 0, blocks * tide::kBlock, blocks, len, 1, true);
        if (rc == TIDE_OK) rc = tide::check_device(x->device);
        if (rc != TIDE_OK || (!rows && !columns)) return rc;
        TIDE_CUDA(tide::launch_quantize({src, src_stride}, type == TIDE_BF16, src_rows, M, len, x->E, offsets, tokens, rows, columns, ctas_of(x),
                                        static_cast<cudaStream_t>(stream)));
        return TIDE_OK;
    });
}

int tide_experts_matmul(tide_experts_t x, const tide_fp8_t* a, int64_t M, const int32_t* offsets, const tide_fp8_t* w, uint32_t flags, int64_t N, int64_t K, void* out,
                        int32_t out_type, int64_t out_stride, void* stream) {
    return no_throw([&]() -> int {
        const size_t elem = float_size(out_type);
        if (!x || !a || !w || !elem || M < 0 || N < 1 || K < 1 || (flags & ~(TIDE_FP8_TRANSPOSED | TIDE_FP8_ANY_SCALES))) return TIDE_EINVAL;
        if (M > tide::kMaxPairs || N > kMaxLen || K > kMaxLen) return TIDE_ERANGE;
        const bool transposed = flags & TIDE_FP8_TRANSPOSED;
        int rc = check_offsets(x, offsets);
        if (rc == TIDE_OK) rc = check_fp8(*a, M, K, M, blocks_of(K), 1, true);
        if (rc == TIDE_OK) rc = check_fp8(*w, N, K, blocks_of(transposed ? K : N), blocks_of(transposed ? N : K), x->E, true);
        if (rc == TIDE_OK) rc = check_rows(out, M, out_stride, N, elem);
        if (rc == TIDE_OK) rc = tide::check_device(x->device);
        if (rc != TIDE_OK) return rc;
        return tide::launch_matmul(*a, M, x->E, offsets, *w, flags, N, K, out, out_type == TIDE_BF16, out_stride, ctas_of(x), wait_of(x),
                                   static_cast<cudaStream_t>(stream));
    });
}

int tide_experts_weight_grad(tide_experts_t x, const tide_fp8_t* dy, const tide_fp8_t* a, int64_t M, const int32_t* offsets, uint32_t flags, int64_t N, int64_t K,
                             void* const* grads, int32_t grad_type, void* stream) {
    return no_throw([&]() -> int {
        const size_t elem = float_size(grad_type);
        if (!x || !dy || !a || !grads || !elem || M < 0 || N < 1 || K < 1 || (flags & ~TIDE_FP8_ANY_SCALES)) return TIDE_EINVAL;
        if (M > tide::kMaxPairs || N > kMaxLen || K > kMaxLen) return TIDE_ERANGE;
        int rc = check_offsets(x, offsets);
        const int64_t blocks = tide::padded_blocks(M, x->E);
        if (rc == TIDE_OK) rc = check_fp8(*dy, M > 0 ? N : 0, blocks * tide::kBlock, blocks, N, 1, true);
        if (rc == TIDE_OK) rc = check_fp8(*a, M > 0 ? K : 0, blocks * tide::kBlock, blocks, K, 1, true);
        if (rc == TIDE_OK) rc = check_extent(N, K, 4);
        if (rc != TIDE_OK) return rc;
        tide::GradPtrs ptrs{};
        for (int e = 0; e < x->E; ++e) {
            if (!grads[e] || !aligned(grads[e], elem)) return TIDE_EINVAL;
            ptrs.p[e] = grads[e];
        }
        if ((rc = tide::check_device(x->device)) != TIDE_OK) return rc;
        return tide::launch_weight_grad(*dy, *a, M, x->E, offsets, flags, N, K, ptrs, grad_type == TIDE_BF16, ctas_of(x), wait_of(x),
                                        static_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"
