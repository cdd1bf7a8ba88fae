// stack_api.cu — extern "C" entry points of the operators around the blocks of a stack declared in include/moe.h
// (routing by scores, layer norm, dropout, embedding): argument checks (before any CUDA call), device check, launches.
#include <cmath>
#include <initializer_list>

#include "api.cuh"
#include "stack_ops.cuh"

namespace moe {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kMaxE = 256, kMaxK = 8, kMaxDim = 65536, kMaxRows = 0x7fffffff - 1024;

int check_rows(const char* name, int T, int d) {
    if (T < 0 || T > kMaxRows) return fail(MOE_ERR_INVALID_ARG, "%s: T = %d outside [0, 2^31 - 1025]", name, T);
    if (d < 1 || d > kMaxDim) return fail(MOE_ERR_INVALID_ARG, "%s: d = %d outside [1, %d]", name, d, kMaxDim);
    return MOE_OK;
}

// A row whose width is no multiple of 8 takes an eight more than its values fill, of the 8192 that a cluster holds.
int check_norm_rows(const char* name, int T, int d) {
    const int rc = check_rows(name, T, d);
    if (rc) return rc;
    if (d > kMaxDim - 16 && d % 8)
        return fail(MOE_ERR_INVALID_ARG, "%s: d = %d must be a multiple of 8 above %d", name, d, kMaxDim - 16);
    return MOE_OK;
}

int check_drop(const char* name, double p, uint64_t seed, int64_t offset, const int64_t* offset_dev, DropArgs* a) {
    if (!drop_args(p, seed, offset, offset_dev, a))
        return fail(MOE_ERR_INVALID_ARG, "%s: p = %g outside [0, 1 - 2^-17)", name, p);
    if (!aligned_to(offset_dev, 8)) return fail(MOE_ERR_INVALID_ARG, "%s: offset_dev must be 8-byte aligned", name);
    return MOE_OK;
}

// Tensors must be aligned to their elements; what they are aligned to beyond that decides on the kernel.
struct Operand {
    const void* p;
    uintptr_t bytes;
};
int check_aligned(const char* name, std::initializer_list<Operand> ps) {
    for (const Operand& o : ps)
        if (!aligned_to(o.p, o.bytes)) return fail(MOE_ERR_INVALID_ARG, "%s: a pointer is not aligned to its element", name);
    return MOE_OK;
}

int check_router(const char* name, int T, int E, int k, int scoring, float scale) {
    if (T < 0 || T > kMaxRows) return fail(MOE_ERR_INVALID_ARG, "%s: T = %d outside [0, 2^31 - 1025]", name, T);
    if (E < 1 || E > kMaxE) return fail(MOE_ERR_INVALID_ARG, "%s: E = %d outside [1, %d]", name, E, kMaxE);
    if (k < 1 || k > E || k > kMaxK) return fail(MOE_ERR_INVALID_ARG, "%s: top_k = %d outside [1, min(E=%d, %d)]", name, k, E, kMaxK);
    if (scoring != 0 && scoring != 1) return fail(MOE_ERR_INVALID_ARG, "%s: scoring = %d must be 0 (softmax) or 1 (sigmoid)", name, scoring);
    if (!std::isfinite(scale)) return fail(MOE_ERR_INVALID_ARG, "%s: scale must be finite", name);
    return MOE_OK;
}

int check_embed(const char* name, int T, int V, int d, float scale) {
    const int rc = check_rows(name, T, d);
    if (rc) return rc;
    if (V < 1 || V > kMaxRows) return fail(MOE_ERR_INVALID_ARG, "%s: V = %d outside [1, 2^31 - 1025]", name, V);
    if (!std::isfinite(scale)) return fail(MOE_ERR_INVALID_ARG, "%s: scale must be finite", name);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_route_scores(const void* logits, int logits_bf16, const float* bias, int T, int E, int top_k, int scoring,
                     int n_group, int topk_group, int renormalize, float scale, int32_t* idx, float* w, float* scores,
                     moe_stream_t stream) {
    const char* name = "moe_route_scores";
    int rc = check_router(name, T, E, top_k, scoring, scale);
    if (rc) return rc;
    if (n_group < 1 || n_group > 32 || E % n_group)
        return fail(MOE_ERR_INVALID_ARG, "%s: n_group = %d must divide E = %d and lie in [1, 32]", name, n_group, E);
    if (topk_group < 1 || topk_group > n_group)
        return fail(MOE_ERR_INVALID_ARG, "%s: topk_group = %d outside [1, n_group = %d]", name, topk_group, n_group);
    if (top_k > topk_group * (E / n_group))
        return fail(MOE_ERR_INVALID_ARG, "%s: top_k = %d exceeds the %d experts of the kept groups", name, top_k,
                    topk_group * (E / n_group));
    if (T == 0) return ok();
    if (!logits || !idx || !w) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", name);
    const uintptr_t l = logits_bf16 ? 2 : 4;
    if ((rc = check_aligned(name, {{logits, l}, {bias, 4}, {idx, 4}, {w, 4}, {scores, 4}}))) return rc;
    int sms;
    if ((rc = check_device(&sms))) return rc;
    return launched(launch_route_scores(logits, logits_bf16 != 0, bias, T, E, top_k, scoring == 1, n_group, topk_group,
                                        renormalize != 0, scale, idx, w, scores, static_cast<cudaStream_t>(stream)),
                    "route_scores");
}

int moe_route_scores_backward(const void* logits, int logits_bf16, const int32_t* idx, const float* dw,
                              const float* dscores, int dscores_per_token, int T, int E, int top_k, int scoring,
                              int renormalize, float scale, void* dlogits, moe_stream_t stream) {
    const char* name = "moe_route_scores_backward";
    int rc = check_router(name, T, E, top_k, scoring, scale);
    if (rc) return rc;
    if (T == 0) return ok();
    if (!logits || !dlogits || (dw && !idx)) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", name);
    const uintptr_t l = logits_bf16 ? 2 : 4;
    if ((rc = check_aligned(name, {{logits, l}, {dlogits, l}, {idx, 4}, {dw, 4}, {dscores, 4}}))) return rc;
    int sms;
    if ((rc = check_device(&sms))) return rc;
    return launched(launch_route_scores_backward(logits, logits_bf16 != 0, idx, dw, dscores, dscores_per_token != 0, T, E,
                                                 top_k, scoring == 1, renormalize != 0, scale, dlogits,
                                                 static_cast<cudaStream_t>(stream)),
                    "route_scores_backward");
}

int moe_layer_norm(const void* x, int x_fp32, const void* h, const float* weight, const float* bias, int T, int d,
                   float eps, double p, uint64_t seed, int64_t offset, const int64_t* offset_dev, void* y, void* n,
                   float* stats, moe_stream_t stream) {
    const char* name = "moe_layer_norm";
    LayerNormArgs a{};
    int rc = check_norm_rows(name, T, d);
    if (rc || (rc = check_drop(name, p, seed, offset, offset_dev, &a.drop))) return rc;
    if (!(eps >= 0.0f) || eps > 3.0e38f) return fail(MOE_ERR_INVALID_ARG, "%s: eps must be finite and not negative", name);
    if (T == 0) return ok();
    if (!h && a.drop.cut) return fail(MOE_ERR_INVALID_ARG, "%s: p belongs to h, which is NULL", name);
    if (!x || !n || !stats || (h && !y)) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", name);
    const uintptr_t sx = x_fp32 ? 4 : 2;
    if ((rc = check_aligned(name, {{x, sx}, {y, sx}, {h, 2}, {n, 2}, {weight, 4}, {bias, 4}, {stats, 8}}))) return rc;
    a.x_fp32 = x_fp32 != 0;
    a.x = x;
    a.h = static_cast<const bf16*>(h);
    a.weight = weight, a.bias = bias, a.T = T, a.d = d, a.eps = eps;
    a.y = h ? y : nullptr;
    a.n = static_cast<bf16*>(n);
    a.stats = stats;
    int sms;
    if ((rc = check_device(&sms))) return rc;
    return launched(launch_layer_norm(a, static_cast<cudaStream_t>(stream)), "layer_norm");
}

size_t moe_layer_norm_backward_workspace_size(int T, int d) {
    if (check_norm_rows("moe_layer_norm_backward_workspace_size", T, d) != MOE_OK) return 0;
    return sizeof(float) * 2 * static_cast<size_t>(layer_norm_width(d)) * layer_norm_blocks(T, d);
}

int moe_layer_norm_backward(const void* x, int x_fp32, const float* stats, const void* dn, const void* dy,
                            const float* weight, int T, int d, double p, uint64_t seed, int64_t offset,
                            const int64_t* offset_dev, void* dx, void* dh, float* dweight, float* dbias, void* workspace,
                            size_t workspace_bytes, moe_stream_t stream) {
    const char* name = "moe_layer_norm_backward";
    LayerNormArgs a{};
    int rc = check_norm_rows(name, T, d);
    if (rc || (rc = check_drop(name, p, seed, offset, offset_dev, &a.drop))) return rc;
    const uintptr_t sx = x_fp32 ? 4 : 2;
    if ((rc = check_aligned(name, {{x, sx}, {dy, sx}, {dx, sx}, {dn, 2}, {dh, 2}, {weight, 4}, {dweight, 4}, {dbias, 4}, {stats, 8}})))
        return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms;
    if (T == 0) {  // sums of no rows
        if (!dweight && !dbias) return ok();
        if ((rc = check_device(&sms))) return rc;
        for (float* g : {dweight, dbias})
            if (g) {
                const cudaError_t e = cudaMemsetAsync(g, 0, sizeof(float) * d, s);
                if (e != cudaSuccess) return launched(e, name);
            }
        return ok();
    }
    if (!x || !stats || !dn || !dx) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", name);
    if (!aligned_to(workspace, 16)) return fail(MOE_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", name);
    if (!workspace || workspace_bytes < moe_layer_norm_backward_workspace_size(T, d))
        return fail(MOE_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", name, workspace ? workspace_bytes : 0,
                    moe_layer_norm_backward_workspace_size(T, d));
    a.x_fp32 = x_fp32 != 0;
    a.x = x;
    a.stats = const_cast<float*>(stats);
    a.dn = static_cast<const bf16*>(dn);
    a.dy = dy;
    a.weight = weight, a.T = T, a.d = d;
    a.dx = dx;
    a.dh = static_cast<bf16*>(dh);
    a.dweight = dweight, a.dbias = dbias;
    a.partial = static_cast<float*>(workspace);
    if ((rc = check_device(&sms))) return rc;
    return launched(launch_layer_norm_backward(a, s), "layer_norm_backward");
}

int moe_dropout(const void* x, int x_fp32, const void* residual, int residual_fp32, long long n, double p,
                uint64_t seed, int64_t offset, const int64_t* offset_dev, void* out, moe_stream_t stream) {
    const char* name = "moe_dropout";
    DropArgs a;
    if (n < 0 || n > (1ll << 40)) return fail(MOE_ERR_INVALID_ARG, "%s: n = %lld outside [0, 2^40]", name, n);
    int rc = check_drop(name, p, seed, offset, offset_dev, &a);
    if (rc) return rc;
    if (n == 0) return ok();
    if (!x || !out) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", name);
    const uintptr_t sx = x_fp32 ? 4 : 2, sr = residual ? (residual_fp32 ? 4 : 2) : sx;
    if ((rc = check_aligned(name, {{x, sx}, {residual, sr}, {out, sr}}))) return rc;
    int sms;
    if ((rc = check_device(&sms))) return rc;
    return launched(launch_dropout(x, x_fp32 != 0, residual, residual_fp32 != 0, n, a, out, static_cast<cudaStream_t>(stream)),
                    "dropout");
}

int moe_embed(const void* ids, int ids_int64, const void* table, int table_fp32, int T, int V, int d, float scale,
              void* out, int out_fp32, int32_t* status, moe_stream_t stream) {
    const char* name = "moe_embed";
    int rc = check_embed(name, T, V, d, scale);
    if (rc) return rc;
    if (T == 0) return ok();
    if (!ids || !table || !out) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", name);
    if ((rc = check_aligned(name, {{ids, ids_int64 ? 8u : 4u}, {table, table_fp32 ? 4u : 2u}, {out, out_fp32 ? 4u : 2u}, {status, 4}})))
        return rc;
    int sms;
    if ((rc = check_device(&sms))) return rc;
    const EmbedArgs a{ids, ids_int64 != 0, table, table_fp32 != 0, T, V, d, scale, out, out_fp32 != 0, false, status};
    return launched(launch_embed(a, static_cast<cudaStream_t>(stream)), "embed");
}

size_t moe_embed_backward_workspace_size(int T, int V, int d) {
    if (check_embed("moe_embed_backward_workspace_size", T, V, d, 1.0f) != MOE_OK || T == 0) return 0;
    return embed_backward_workspace(T, V, d);
}

int moe_embed_backward(const void* ids, int ids_int64, const void* dy, int dy_fp32, int T, int V, int d, float scale,
                       void* out, int out_fp32, int accumulate, void* workspace, size_t workspace_bytes, int32_t* status,
                       moe_stream_t stream) {
    const char* name = "moe_embed_backward";
    int rc = check_embed(name, T, V, d, scale);
    if (rc) return rc;
    if (accumulate && !out_fp32) return fail(MOE_ERR_INVALID_ARG, "%s: accumulate needs an fp32 output", name);
    if (T == 0 && accumulate) return ok();
    if (!out || (T > 0 && (!ids || !dy))) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", name);
    if ((rc = check_aligned(name, {{ids, ids_int64 ? 8u : 4u}, {dy, dy_fp32 ? 4u : 2u}, {out, out_fp32 ? 4u : 2u}, {status, 4}})))
        return rc;
    if (!aligned_to(workspace, 16)) return fail(MOE_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", name);
    const size_t need = T ? embed_backward_workspace(T, V, d) : 0;
    if (T > 0 && (!workspace || workspace_bytes < need))
        return fail(MOE_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", name, workspace ? workspace_bytes : 0, need);
    int sms;
    if ((rc = check_device(&sms))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) return launched(cudaMemsetAsync(out, 0, static_cast<size_t>(V) * d * (out_fp32 ? 4 : 2), s), name);
    const EmbedArgs a{ids, ids_int64 != 0, dy, dy_fp32 != 0, T, V, d, scale, out, out_fp32 != 0, accumulate != 0, status};
    return launched(launch_embed_backward(a, workspace, s), "embed_backward");
}

}  // extern "C"
