// train_api.cu — extern "C" entry points of the training operators declared in include/moe.h: argument
// checks (before any CUDA call), device check, launches.
#include <cmath>

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

// Floats of the slices of a split reduction (a multiple of 8); 0 if the shape is not split.
size_t grouped_slices(int mode, int M, int K, int N, int E) {
    const int ks = grouped_mm_ksplit(mode, M, K, N, E, kPlanSms);
    const size_t rows = mode == kMmWgrad ? static_cast<size_t>(E) * K : static_cast<size_t>(M);
    return ks > 1 ? ks * rows * N : 0;
}
// The slices, then the words that say that they are there.
size_t grouped_workspace(int mode, int M, int K, int N, int E) {
    const size_t slices = grouped_slices(mode, M, K, N, E);
    return slices ? sizeof(float) * slices + sizeof(int32_t) * kGroupedMmDone : 0;
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
    GroupedMmArgs g{a, b, offsets, M, K, N, E, out, out_fp32 != 0, accumulate != 0, 1, nullptr, inject_stall(), nullptr, status};
    if (workspace && need) {
        g.ksplit = grouped_mm_ksplit(mode, M, K, N, E, kPlanSms);
        g.partial = static_cast<float*>(workspace);
        g.done = reinterpret_cast<int32_t*>(g.partial + grouped_slices(mode, M, K, N, E));
    }
    const char* why = "launch";
    const cudaError_t e = launch_grouped_mm(mode, g, sms, s, &why);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s (%s)", name, why, cudaGetErrorString(e));
    return ok();
}

int check_rows(const char* name, int rows, const char* rows_name, int cols, const char* cols_name) {
    if (rows < 0 || rows > 0x7fffffff - 1024)
        return fail(MOE_ERR_INVALID_ARG, "%s: %s = %d outside [0, 2^31 - 1025]", name, rows_name, rows);
    if (cols < 8 || cols > kMaxDim || cols % 8)
        return fail(MOE_ERR_INVALID_ARG, "%s: %s = %d must be a multiple of 8 in [8, %d]", name, cols_name, cols, kMaxDim);
    return MOE_OK;
}

int check_norm(const char* name, const BlockNormArgs& a) {
    int rc = check_rows(name, a.T, "T", a.d, "d");
    if (rc) return rc;
    if (!(a.eps >= 0.0f) || a.eps > 3.0e38f)
        return fail(MOE_ERR_INVALID_ARG, "%s: eps must be finite and not negative", name);
    if (a.T == 0) return MOE_OK;  // tensors without rows have no address: NULL says nothing about them
    if (a.h && !a.w_post) return fail(MOE_ERR_INVALID_ARG, "%s: h needs w_post", name);
    if (!a.h && (a.w_post || a.gate || a.tgate || a.res))
        return fail(MOE_ERR_INVALID_ARG, "%s: w_post, gate, tgate and res belong to h, which is NULL", name);
    const void* ps[] = {a.x, a.h, a.w_pre, a.w_post, a.gate, a.res, a.y, a.n, a.dy, a.dn, a.dx, a.dh, a.partial};
    for (const void* p : ps)
        if (!aligned_to(p, 16)) return fail(MOE_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", name);
    const void* qs[] = {a.tgate, a.dtgate, a.dw_pre, a.dw_post, a.dgate, a.dres};
    for (const void* q : qs)
        if (!aligned_to(q, 4)) return fail(MOE_ERR_INVALID_ARG, "%s: gradients and tgate must be 4-byte aligned", name);
    return MOE_OK;
}

using bf16 = __nv_bfloat16;

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

int moe_swiglu(const void* gu, const float* w, int M, int f, void* h, moe_stream_t stream) {
    int rc = check_rows("moe_swiglu", M, "M", f, "f");
    if (rc) return rc;
    if (M == 0) return ok();
    if (!gu || !h) return fail(MOE_ERR_INVALID_ARG, "moe_swiglu: null pointer");
    if (!aligned_to(gu, 16) || !aligned_to(h, 16) || !aligned_to(w, 4))
        return fail(MOE_ERR_INVALID_ARG, "moe_swiglu: gu and h must be 16-byte aligned, w 4-byte");
    int sms;
    if ((rc = check_device(&sms))) return rc;
    return launched(launch_swiglu(static_cast<const bf16*>(gu), w, M, f, static_cast<bf16*>(h), sms,
                                  static_cast<cudaStream_t>(stream)),
                    "swiglu");
}

int moe_swiglu_backward(const void* gu, const void* dh, const float* w, int M, int f, void* dgu, float* dw, void* h,
                        moe_stream_t stream) {
    int rc = check_rows("moe_swiglu_backward", M, "M", f, "f");
    if (rc) return rc;
    if (M == 0) return ok();
    if (!gu || !dh || !dgu) return fail(MOE_ERR_INVALID_ARG, "moe_swiglu_backward: null pointer");
    if (!aligned_to(gu, 16) || !aligned_to(dh, 16) || !aligned_to(dgu, 16) || !aligned_to(h, 16) || !aligned_to(w, 4) ||
        !aligned_to(dw, 4))
        return fail(MOE_ERR_INVALID_ARG, "moe_swiglu_backward: gu, dh, dgu and h must be 16-byte aligned, w and dw 4-byte");
    int sms;
    if ((rc = check_device(&sms))) return rc;
    return launched(launch_swiglu_backward(static_cast<const bf16*>(gu), static_cast<const bf16*>(dh), w, M, f,
                                           static_cast<bf16*>(dgu), dw, static_cast<bf16*>(h), sms,
                                           static_cast<cudaStream_t>(stream)),
                    "swiglu_backward");
}

int moe_block_norm(const void* x, int x_fp32, const void* h, const float* w_pre, const float* w_post,
                   const float* gate, const float* tgate, const float* res, int T, int d, float eps, void* y, void* n,
                   moe_stream_t stream) {
    BlockNormArgs a{};
    a.x_fp32 = x_fp32 != 0;
    a.x = x;
    a.h = static_cast<const bf16*>(h);
    a.w_pre = w_pre, a.w_post = w_post, a.gate = gate, a.tgate = tgate, a.res = res;
    a.T = T, a.d = d, a.eps = eps;
    a.y = h ? y : nullptr;
    a.n = static_cast<bf16*>(n);
    int rc = check_norm("moe_block_norm", a);
    if (rc) return rc;
    if (T == 0) return ok();
    if ((w_pre == nullptr) != (n == nullptr))
        return fail(MOE_ERR_INVALID_ARG, "moe_block_norm: w_pre and n are given together or not at all");
    if (!x || (!a.y && !n)) return fail(MOE_ERR_INVALID_ARG, "moe_block_norm: null pointer");
    int sms;
    if ((rc = check_device(&sms))) return rc;
    return launched(launch_block_norm(a, false, sms, static_cast<cudaStream_t>(stream)), "block_norm");
}

size_t moe_block_norm_backward_workspace_size(int T, int d) {
    if (check_rows("moe_block_norm_backward_workspace_size", T, "T", d, "d") != MOE_OK) return 0;
    return sizeof(float) * 3 * static_cast<size_t>(d) * block_norm_blocks(T, d);
}

int moe_block_norm_backward(const void* x, int x_fp32, const void* h, const void* dy, const void* dn,
                            const float* w_pre, const float* w_post, const float* gate, const float* tgate,
                            const float* res, int T, int d, float eps, void* dx, void* dh, float* dw_pre,
                            float* dw_post, float* dgate, float* dtgate, float* dres, void* workspace,
                            size_t workspace_bytes, moe_stream_t stream) {
    const char* name = "moe_block_norm_backward";
    BlockNormArgs a{};
    a.x_fp32 = x_fp32 != 0;
    a.x = x;
    a.h = static_cast<const bf16*>(h);
    a.w_pre = w_pre, a.w_post = w_post, a.gate = gate, a.tgate = tgate, a.res = res;
    a.T = T, a.d = d, a.eps = eps;
    a.dy = dy;
    a.dn = static_cast<const bf16*>(dn);
    a.dx = dx;
    a.dh = static_cast<bf16*>(dh);
    a.dw_pre = dw_pre, a.dw_post = dw_post, a.dgate = dgate, a.dtgate = dtgate, a.dres = dres;
    a.partial = static_cast<float*>(workspace);
    int rc = check_norm(name, a);
    if (rc) return rc;
    float* sums[] = {dw_pre, dw_post, dgate, dres};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms;
    if (T == 0) {  // sums of no rows
        bool any = false;
        for (float* p : sums) any = any || p;
        if (!any) return ok();
        if ((rc = check_device(&sms))) return rc;
        for (float* p : sums)
            if (p) {
                const cudaError_t e = cudaMemsetAsync(p, 0, sizeof(float) * d, s);
                if (e != cudaSuccess) return launched(e, name);
            }
        return ok();
    }
    if (dn && !w_pre) return fail(MOE_ERR_INVALID_ARG, "%s: dn needs w_pre", name);
    if (!dn && dw_pre) return fail(MOE_ERR_INVALID_ARG, "%s: dw_pre needs dn", name);
    if (!h && (dh || dw_post || dgate || dtgate || dres))
        return fail(MOE_ERR_INVALID_ARG, "%s: dh, dw_post, dgate, dtgate and dres belong to h, which is NULL", name);
    if ((dgate && !gate) || (dtgate && !tgate) || (dres && !res))
        return fail(MOE_ERR_INVALID_ARG, "%s: the gradient of an input that is NULL", name);
    if (!x || !dx || (h && !dh) || (!dy && !dn)) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", name);
    if (!workspace || workspace_bytes < moe_block_norm_backward_workspace_size(T, d))
        return fail(MOE_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", name, workspace ? workspace_bytes : 0,
                    moe_block_norm_backward_workspace_size(T, d));
    if ((rc = check_device(&sms))) return rc;
    return launched(launch_block_norm(a, true, sms, s), "block_norm_backward");
}

int moe_adamw_step(const moe_adamw_tensor* tensors, int count, int param_bf16, int grad_bf16, int state_bits,
                   double lr, double beta1, double beta2, double eps, double weight_decay, int step,
                   const int32_t* step_dev, const float* factors, moe_stream_t stream) {
    const char* name = "moe_adamw_step";
    if (count < 0) return fail(MOE_ERR_INVALID_ARG, "%s: count = %d must be >= 0", name, count);
    if (state_bits != 8 && state_bits != 32)
        return fail(MOE_ERR_INVALID_ARG, "%s: state_bits = %d must be 8 or 32", name, state_bits);
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0))
        return fail(MOE_ERR_INVALID_ARG, "%s: betas must be in [0, 1)", name);
    if (!(eps >= 0.0) || !std::isfinite(eps) || !std::isfinite(lr) || !std::isfinite(weight_decay))
        return fail(MOE_ERR_INVALID_ARG, "%s: lr, eps and weight_decay must be finite, eps not negative", name);
    if (!step_dev && step < 1) return fail(MOE_ERR_INVALID_ARG, "%s: step = %d must be >= 1", name, step);
    if (!aligned_to(step_dev, 4) || !aligned_to(factors, 4))
        return fail(MOE_ERR_INVALID_ARG, "%s: step_dev and factors must be 4-byte aligned", name);
    if (count == 0) return ok();
    if (!tensors) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", name);
    const uintptr_t pa = param_bf16 ? 2 : 4, ga = grad_bf16 ? 2 : 4, sa = state_bits == 8 ? 1 : 4;
    for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor& t = tensors[i];
        if (t.n < 0 || t.n > (1ll << 40))
            return fail(MOE_ERR_INVALID_ARG, "%s: tensor %d: n = %lld outside [0, 2^40]", name, i, t.n);
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.m || !t.v || (state_bits == 8 && (!t.m_scale || !t.v_scale)))
            return fail(MOE_ERR_INVALID_ARG, "%s: tensor %d: null pointer", name, i);
        if (!aligned_to(t.param, pa) || !aligned_to(t.grad, ga) || !aligned_to(t.m, sa) || !aligned_to(t.v, sa) ||
            !aligned_to(t.m_scale, 4) || !aligned_to(t.v_scale, 4) || !aligned_to(t.copy, 2))
            return fail(MOE_ERR_INVALID_ARG, "%s: tensor %d: a pointer is not aligned to its element", name, i);
    }
    int rc, sms;
    if ((rc = check_device(&sms))) return rc;
    const double corr1 = 1.0 - std::pow(beta1, step), corr2 = std::sqrt(1.0 - std::pow(beta2, step));
    return launched(launch_adamw(tensors, count, param_bf16 != 0, grad_bf16 != 0, state_bits == 8, lr, beta1, beta2, eps,
                                 weight_decay, corr1, corr2, step_dev, factors, sms, static_cast<cudaStream_t>(stream)),
                    "adamw");
}

}  // extern "C"
