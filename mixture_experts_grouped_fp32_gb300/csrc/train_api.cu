// train_api.cu — extern "C" entry points of the training operators declared in include/moe.h: argument
// checks (before any CUDA call), device check, launches.
#include "api.cuh"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kMaxE = 256, kMaxDim = 65536;
constexpr int kPlanSms = 152;  // GB300: the split of a reduction, and so its workspace, depends on the shape alone

int check_grouped(const char* name, int mode, int M, int K, int N, int E) {
    if (mode < 0 || mode > 2) return fail(MOE_ERR_INVALID_ARG, "%s: mode = %d outside [0, 2]", name, mode);
    if (M < 0 || M > 0x7fffffff - 1024) return fail(MOE_ERR_INVALID_ARG, "%s: M = %d outside [0, 2^31 - 1025]", name, M);
    if (E < 1 || E > kMaxE) return fail(MOE_ERR_INVALID_ARG, "%s: E = %d outside [1, %d]", name, E, kMaxE);
    if (K < 8 || K > kMaxDim || K % 8) return fail(MOE_ERR_INVALID_ARG, "%s: K = %d must be a multiple of 8 in [8, %d]", name, K, kMaxDim);
    if (N < 8 || N > kMaxDim || N % 8) return fail(MOE_ERR_INVALID_ARG, "%s: N = %d must be a multiple of 8 in [8, %d]", name, N, kMaxDim);
    return MOE_OK;
}

size_t grouped_workspace(int mode, int M, int K, int N, int E) {
    const int ks = grouped_mm_ksplit(mode, M, K, N, E, kPlanSms);
    if (ks <= 1) return 0;
    const size_t rows = mode == kMmWgrad ? static_cast<size_t>(E) * K : static_cast<size_t>(M);
    return sizeof(float) * ks * rows * N;
}

int grouped_entry(const char* name, int mode, const void* a, const void* b, const int32_t* offsets, int M, int K,
                  int N, int E, void* out, int out_fp32, int accumulate, void* workspace, size_t workspace_bytes,
                  int32_t* status, moe_stream_t stream) {
    int rc = check_grouped(name, mode, M, K, N, E);
    if (rc) return rc;
    if (accumulate && !out_fp32) return fail(MOE_ERR_INVALID_ARG, "%s: accumulate needs an fp32 output", name);
    if (M == 0 && (mode != kMmWgrad || accumulate)) return ok();
    if (!out || (M > 0 && (!a || !b || !offsets))) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", name);
    if (!aligned_to(a, 16) || !aligned_to(b, 16) || !aligned_to(out, 16) || !aligned_to(workspace, 16))
        return fail(MOE_ERR_INVALID_ARG, "%s: operands and workspace must be 16-byte aligned", name);
    if (!aligned_to(offsets, 4) || !aligned_to(status, 4))
        return fail(MOE_ERR_INVALID_ARG, "%s: offsets and status must be 4-byte aligned", name);
    const size_t need = grouped_workspace(mode, M, K, N, E);
    if (workspace && workspace_bytes < need)
        return fail(MOE_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", name, workspace_bytes, need);
    int sms;
    if ((rc = check_device(&sms))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M == 0)  // the weight gradient of no rows
        return launched(cudaMemsetAsync(out, 0, static_cast<size_t>(E) * K * N * (out_fp32 ? 4 : 2), s), name);
    GroupedMmArgs g{a, b, offsets, M, K, N, E, out, out_fp32 != 0, accumulate != 0, 1, nullptr, status};
    if (workspace && need) {
        g.ksplit = grouped_mm_ksplit(mode, M, K, N, E, kPlanSms);
        g.partial = static_cast<float*>(workspace);
    }
    const char* why = "launch";
    const cudaError_t e = launch_grouped_mm(mode, g, sms, s, &why);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s (%s)", name, why, cudaGetErrorString(e));
    return ok();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grouped_mm_workspace_size(int mode, int M, int K, int N, int E) {
    if (check_grouped("moe_grouped_mm_workspace_size", mode, M, K, N, E) != MOE_OK) return 0;
    return grouped_workspace(mode, M, K, N, E);
}

int moe_grouped_mm(const void* a, const void* b, const int32_t* offsets, int M, int K, int N, int E, int transpose_b,
                   void* out, int out_fp32, void* workspace, size_t workspace_bytes, int32_t* status,
                   moe_stream_t stream) {
    return grouped_entry("moe_grouped_mm", transpose_b ? kMmTransB : kMmForward, a, b, offsets, M, K, N, E, out,
                         out_fp32, 0, workspace, workspace_bytes, status, stream);
}

int moe_grouped_mm_wgrad(const void* a, const void* g, const int32_t* offsets, int M, int K, int N, int E, void* out,
                         int out_fp32, int accumulate, void* workspace, size_t workspace_bytes, int32_t* status,
                         moe_stream_t stream) {
    return grouped_entry("moe_grouped_mm_wgrad", kMmWgrad, a, g, offsets, M, K, N, E, out, out_fp32, accumulate,
                         workspace, workspace_bytes, status, stream);
}

}  // extern "C"
