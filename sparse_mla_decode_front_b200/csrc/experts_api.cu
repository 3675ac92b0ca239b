// C entry points of the routed experts (include/moe_experts.h): validation, then one
// enqueue on the caller's stream. Nothing is enqueued on an error other than MLA_ERR_CUDA.
#include <cmath>
#include <initializer_list>

#include "common.cuh"
#include "launch.h"
#include "moe_experts.h"

using namespace mla;

namespace {

static_assert(MLA_DTYPE_BF16 == kDtypeBf16 && MLA_DTYPE_FP16 == kDtypeFp16 && MLA_DTYPE_FP32 == kDtypeFp32,
              "dtype codes differ");

constexpr int kWorkspaceAlign = 256;

// Required pointers: tensors on 16 bytes, index, offset, weight and scale arrays on 4.
int check(std::initializer_list<const void*> tensors, std::initializer_list<const void*> arrays) {
    for (const void* p : tensors)
        if (!p) return MLA_ERR_NULL_POINTER;
    for (const void* p : arrays)
        if (!p) return MLA_ERR_NULL_POINTER;
    for (const void* p : tensors)
        if (reinterpret_cast<uintptr_t>(p) % 16) return MLA_ERR_MISALIGNED;
    for (const void* p : arrays)
        if (reinterpret_cast<uintptr_t>(p) % 4) return MLA_ERR_MISALIGNED;
    return MLA_OK;
}
bool misaligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }
bool dtype_ok(int dtype) { return dtype >= MLA_DTYPE_BF16 && dtype <= MLA_DTYPE_FP32; }
// A failed launch is reported here and not left behind for the caller's next CUDA check.
int done(cudaError_t e) {
    if (!cuda_call_failed(e)) return MLA_OK;
    cudaGetLastError();
    return MLA_ERR_CUDA;
}
cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

bool sort_dims_ok(int T, int K, int E) {
    return T >= 0 && K >= 1 && K <= MLA_MOE_MAX_TOP_K && E >= 1 && E <= MLA_MOE_MAX_EXPERTS &&
           (long long)T * K <= (1LL << 30);
}

// Sizes of the row movers: MLA_OK, or the refusal.
int row_dims(int T, int K, int H, int R, int dtype) {
    if (T < 0 || K < 1 || H < 1 || R < 0) return MLA_ERR_BAD_DIMS;
    if (!dtype_ok(dtype)) return MLA_ERR_BAD_ARGUMENT;
    if (K > MLA_MOE_MAX_TOP_K || H % 16 || H > (1 << 30) || (long long)T * K > (1LL << 30) || !moe_rows_fit(T, H))
        return MLA_ERR_UNSUPPORTED_DIMS;
    return MLA_OK;
}

int gemm_call(const void* x, const float* xs, const void* w, const float* ws, const int32_t* offsets, bool grouped,
              int rows, int groups, int n, int k, void* out, int dtype, int32_t* status, void* stream) {
    if (rows < 0 || groups < 1 || n < 1 || k < 1) return MLA_ERR_BAD_DIMS;
    if (!dtype_ok(dtype)) return MLA_ERR_BAD_ARGUMENT;
    if (n % 16 || k % 16 || n > (1 << 30) || k > (1 << 30) || groups > MLA_MOE_MAX_EXPERTS || !fp8_gemm_fits(rows, groups, n))
        return MLA_ERR_UNSUPPORTED_DIMS;
    if (rows == 0) return MLA_OK;
    const int rc = check({x, w, out}, {xs, ws});
    if (rc != MLA_OK) return rc;
    if (grouped && !offsets) return MLA_ERR_NULL_POINTER;
    if (misaligned(offsets, 4) || misaligned(status, 4)) return MLA_ERR_MISALIGNED;
    return done(launch_fp8_gemm(x, xs, w, ws, offsets, rows, groups, n, k, out, dtype, status, as_stream(stream)));
}

}  // namespace

extern "C" {

size_t mla_moe_sort_workspace_bytes(int n_tokens, int top_k, int n_experts) {
    return sort_dims_ok(n_tokens, top_k, n_experts) ? moe_sort_workspace_bytes(n_tokens, top_k, n_experts) : 0;
}

int mla_moe_sort(const int32_t* topk_idx, const void* affinities, int n_tokens, int top_k, int n_experts_total,
                 int first_expert, int n_experts, int normalize, float scale, int32_t* expert_offsets,
                 int32_t* row_of, int32_t* source_of, float* weights, void* workspace, size_t workspace_bytes,
                 void* stream) {
    if (n_tokens < 0 || top_k < 1 || n_experts < 1 || first_expert < 0 || (affinities && n_experts_total < 1))
        return MLA_ERR_BAD_DIMS;
    if (!std::isfinite(scale) || (normalize != 0 && normalize != 1)) return MLA_ERR_BAD_ARGUMENT;
    if (!sort_dims_ok(n_tokens, top_k, n_experts)) return MLA_ERR_UNSUPPORTED_DIMS;
    int rc = check({}, {expert_offsets});
    if (rc != MLA_OK) return rc;
    if (n_tokens > 0) {
        rc = check({}, {topk_idx, row_of, source_of});
        if (rc != MLA_OK) return rc;
        if (!affinities != !weights) return MLA_ERR_NULL_POINTER;
        if (misaligned(affinities, 16) || misaligned(weights, 4)) return MLA_ERR_MISALIGNED;
        const size_t need = moe_sort_workspace_bytes(n_tokens, top_k, n_experts);
        if (need > 0) {
            if (!workspace) return MLA_ERR_NULL_POINTER;
            if (misaligned(workspace, kWorkspaceAlign)) return MLA_ERR_MISALIGNED;
            if (workspace_bytes < need) return MLA_ERR_WORKSPACE_TOO_SMALL;
        }
    }
    return done(launch_moe_sort(topk_idx, static_cast<const bf16*>(affinities), n_tokens, top_k, n_experts_total,
                                first_expert, n_experts, normalize, scale, expert_offsets, row_of, source_of, weights,
                                workspace, as_stream(stream)));
}

int mla_moe_gather(const void* x, int dtype, const int32_t* row_of, int n_tokens, int top_k, int hidden, int n_rows,
                   void* rows, float* scales, void* stream) {
    int rc = row_dims(n_tokens, top_k, hidden, n_rows, dtype);
    if (rc != MLA_OK) return rc;
    if (n_tokens == 0 || n_rows == 0) return MLA_OK;
    rc = check({x, rows}, {row_of});
    if (rc != MLA_OK) return rc;
    if (misaligned(scales, 4)) return MLA_ERR_MISALIGNED;
    return done(launch_moe_gather(x, dtype, row_of, n_tokens, top_k, hidden, n_rows, rows, scales, as_stream(stream)));
}

int mla_moe_combine(const void* rows, int dtype, const int32_t* row_of, const float* weights, int n_tokens,
                    int top_k, int hidden, int n_rows, void* out, void* stream) {
    int rc = row_dims(n_tokens, top_k, hidden, n_rows, dtype);
    if (rc != MLA_OK) return rc;
    if (n_tokens == 0) return MLA_OK;
    rc = check({out}, {row_of});
    if (rc != MLA_OK) return rc;
    if (n_rows > 0 && !rows) return MLA_ERR_NULL_POINTER;   // without rows every output is 0
    if (misaligned(rows, 16) || misaligned(weights, 4)) return MLA_ERR_MISALIGNED;
    return done(launch_moe_combine(rows, dtype, row_of, weights, n_tokens, top_k, hidden, n_rows, out,
                                   as_stream(stream)));
}

int mla_moe_combine_backward(const void* grad_out, const void* rows, int dtype, const int32_t* row_of,
                             const float* weights, int n_tokens, int top_k, int hidden, int n_rows, void* grad_rows,
                             float* grad_weights, void* stream) {
    int rc = row_dims(n_tokens, top_k, hidden, n_rows, dtype);
    if (rc != MLA_OK) return rc;
    if (n_tokens == 0) return MLA_OK;
    rc = check({grad_out}, {row_of});
    if (rc != MLA_OK) return rc;
    if (!grad_weights && n_rows == 0) return MLA_OK;   // nothing to write (an empty tensor's address is null)
    if (!grad_weights && !grad_rows) return MLA_ERR_NULL_POINTER;
    if (grad_weights && !rows && n_rows > 0) return MLA_ERR_NULL_POINTER;
    if (misaligned(rows, 16) || misaligned(grad_rows, 16) || misaligned(weights, 4) || misaligned(grad_weights, 4))
        return MLA_ERR_MISALIGNED;
    return done(launch_moe_combine_backward(grad_out, rows, dtype, row_of, weights, n_tokens, top_k, hidden, n_rows,
                                            grad_rows, grad_weights, as_stream(stream)));
}

int mla_fp8_quantize(const void* x, int dtype, int n_rows, int cols, int gated, const int32_t* valid_rows, void* q,
                     float* scales, void* stream) {
    if (n_rows < 0 || cols < 1) return MLA_ERR_BAD_DIMS;
    if (!dtype_ok(dtype) || (gated != 0 && gated != 1)) return MLA_ERR_BAD_ARGUMENT;
    if (cols % 16 || cols > (1 << 29) || !moe_rows_fit(n_rows, cols)) return MLA_ERR_UNSUPPORTED_DIMS;
    if (n_rows == 0) return MLA_OK;
    const int rc = check({x, q}, {scales});
    if (rc != MLA_OK) return rc;
    if (misaligned(valid_rows, 4)) return MLA_ERR_MISALIGNED;
    return done(launch_fp8_quantize(x, dtype, n_rows, cols, gated, valid_rows, q, scales, as_stream(stream)));
}

int mla_fp8_matmul(const void* x, const float* x_scales, const void* w, const float* w_scales, int n_rows, int n,
                   int k, void* out, int out_dtype, int32_t* status, void* stream) {
    return gemm_call(x, x_scales, w, w_scales, nullptr, false, n_rows, 1, n, k, out, out_dtype, status, stream);
}

int mla_fp8_grouped_matmul(const void* x, const float* x_scales, const void* w, const float* w_scales,
                           const int32_t* expert_offsets, int n_rows, int n_experts, int n, int k, void* out,
                           int out_dtype, int32_t* status, void* stream) {
    return gemm_call(x, x_scales, w, w_scales, expert_offsets, true, n_rows, n_experts, n, k, out, out_dtype, status,
                     stream);
}

}  // extern "C"
