// Entry points of the training operators (tee_train.h): argument checks, the
// context's device, one launcher call each.
#include "train_internal.cuh"

#include <stdio.h>

#include <initializer_list>

namespace {

struct Buf {
    const char* name;
    const void* p;
    int align;
};

int bad(tee_ctx* ctx, const char* op, const char* what) {
    char msg[256];
    snprintf(msg, sizeof msg, "%s: %s", op, what);
    return tee_set_error(ctx, TEE_EINVAL, msg);
}

int check_bufs(tee_ctx* ctx, const char* op, std::initializer_list<Buf> bufs) {
    char msg[160];
    for (const Buf& b : bufs) {
        if (!b.p) {
            snprintf(msg, sizeof msg, "%s is NULL", b.name);
            return bad(ctx, op, msg);
        }
        if (reinterpret_cast<uintptr_t>(b.p) % (uintptr_t)b.align) {
            snprintf(msg, sizeof msg, "%s must be %d-byte aligned", b.name, b.align);
            return bad(ctx, op, msg);
        }
    }
    return TEE_OK;
}

int check_ws(tee_ctx* ctx, const char* op, const void* ws, size_t have, size_t need) {
    if (have < need) {
        char msg[160];
        snprintf(msg, sizeof msg, "workspace of %zu bytes, %zu needed", have, need);
        return bad(ctx, op, msg);
    }
    return need ? check_bufs(ctx, op, {{"d_ws", ws, 16}}) : TEE_OK;
}

bool is_type(int t) { return t == TEE_F32 || t == TEE_BF16; }

constexpr int MAX_ROWS = 1 << 30;       // T of any operator
constexpr int MAX_EMBED_HIDDEN = 65536;

// The launch, on the context's device, bracketed by the profiling hook.
template <typename F>
int launch(tee_ctx* ctx, const char* op, int kclass, double flops, double bytes, void* stream, F&& f) {
    DeviceScope scope(ctx->device);
    if (scope.err != cudaSuccess) return tee_set_cuda_error(ctx, scope.err, "cudaSetDevice");
    cudaStream_t s = (cudaStream_t)stream;
    const int slot = prof_begin(ctx, s, kclass, flops, bytes);
    const cudaError_t e = f(s);
    prof_end(ctx, s, slot);
    return e == cudaSuccess ? TEE_OK : tee_set_cuda_error(ctx, e, op);
}

// Sizes of the vocabulary loss; the message of what is wrong with them, or NULL.
const char* vocab_sizes(int N, int V, int H) {
    if (N < 0 || N > (1 << 24)) return "N out of range";
    if (V < 1 || V > (1 << 24)) return "V out of range";
    if (H < 8 || H % 8 || H > TEE_VOCAB_MAX_HIDDEN) return "H must be a multiple of 8 within range";
    if (((long long)N + 255) / 256 * (((long long)V + 255) / 256) > (1LL << 30)) return "N times V out of range";
    return nullptr;
}

size_t type_size(int t) { return t == TEE_BF16 ? 2 : 4; }

}  // namespace

extern "C" {

int tee_op_layernorm_forward(tee_ctx* ctx, const void* d_x, int x_type, const float* d_gamma, void* d_y, int y_type,
                             float* d_stats, int T, int H, float eps, void* stream) {
    static const char* op = "layernorm_forward";
    if (!ctx) return TEE_EINVAL;
    if (!is_type(x_type) || !is_type(y_type)) return bad(ctx, op, "element types must be TEE_F32 or TEE_BF16");
    if (T < 0 || T > MAX_ROWS) return bad(ctx, op, "T out of range");
    if (H < 1 || H > TEE_LN_MAX_HIDDEN) return bad(ctx, op, "H out of range");
    if (!(eps >= 0.f)) return bad(ctx, op, "eps must be >= 0");
    if (T == 0) return TEE_OK;
    int rc = check_bufs(ctx, op, {{"d_x", d_x, 16}, {"d_gamma", d_gamma, 16}, {"d_y", d_y, 16}});
    if (rc || (d_stats && (rc = check_bufs(ctx, op, {{"d_stats", d_stats, 8}})))) return rc;
    return launch(ctx, op, TEE_K_LAYERNORM, 0, (double)T * H * (type_size(x_type) + type_size(y_type)), stream,
                  [&](cudaStream_t s) {
                      return launch_layernorm_forward(d_x, x_type == TEE_BF16, d_gamma, d_y, y_type == TEE_BF16, d_stats,
                                                      T, H, eps, s);
                  });
}

long long tee_layernorm_backward_workspace(int T, int H) {
    if (T < 0 || T > MAX_ROWS || H < 1 || H > TEE_LN_MAX_HIDDEN)
        return tee_set_global_error(TEE_EINVAL, "layernorm_backward_workspace: T or H out of range");
    return (long long)layernorm_backward_ws(T, H);
}

int tee_op_layernorm_backward(tee_ctx* ctx, const void* d_dy, int y_type, const void* d_x, int x_type,
                              const float* d_gamma, const float* d_stats, const void* d_dres, void* d_dx,
                              float* d_dgamma, int T, int H, void* d_ws, size_t ws_bytes, void* stream) {
    static const char* op = "layernorm_backward";
    if (!ctx) return TEE_EINVAL;
    if (!is_type(x_type) || !is_type(y_type)) return bad(ctx, op, "element types must be TEE_F32 or TEE_BF16");
    if (T < 0 || T > MAX_ROWS) return bad(ctx, op, "T out of range");
    if (H < 1 || H > TEE_LN_MAX_HIDDEN) return bad(ctx, op, "H out of range");
    int rc = check_bufs(ctx, op, {{"d_dgamma", d_dgamma, 16}});
    if (rc) return rc;
    if (T > 0) {
        if ((rc = check_bufs(ctx, op, {{"d_dy", d_dy, 16}, {"d_x", d_x, 16}, {"d_gamma", d_gamma, 16},
                                       {"d_stats", d_stats, 8}, {"d_dx", d_dx, 16}})))
            return rc;
        if (d_dres && (rc = check_bufs(ctx, op, {{"d_dres", d_dres, 16}}))) return rc;
        if ((rc = check_ws(ctx, op, d_ws, ws_bytes, layernorm_backward_ws(T, H)))) return rc;
    }
    return launch(ctx, op, TEE_K_LAYERNORM, 0,
                  (double)T * H * ((d_dres ? 3 : 2) * type_size(x_type) + type_size(y_type)), stream, [&](cudaStream_t s) {
                      return launch_layernorm_backward(d_dy, y_type == TEE_BF16, d_x, x_type == TEE_BF16, d_gamma, d_stats,
                                                       d_dres, d_dx, d_dgamma, T, H, d_ws, s);
                  });
}

int tee_op_embed_forward(tee_ctx* ctx, const void* d_table, int table_type, const int32_t* d_ids, void* d_y, int y_type,
                         int T, int V, int H, float scale, void* stream) {
    static const char* op = "embed_forward";
    if (!ctx) return TEE_EINVAL;
    if (!is_type(table_type) || !is_type(y_type)) return bad(ctx, op, "element types must be TEE_F32 or TEE_BF16");
    if (T < 0 || T > MAX_ROWS) return bad(ctx, op, "T out of range");
    if (V < 1) return bad(ctx, op, "V out of range");
    if (H < 1 || H > MAX_EMBED_HIDDEN) return bad(ctx, op, "H out of range");
    if (T == 0) return TEE_OK;
    int rc = check_bufs(ctx, op, {{"d_table", d_table, 16}, {"d_ids", d_ids, 4}, {"d_y", d_y, 16}});
    if (rc) return rc;
    return launch(ctx, op, TEE_K_EMBED, 0, (double)T * H * (type_size(table_type) + type_size(y_type)), stream,
                  [&](cudaStream_t s) {
                      return launch_embed_forward(d_table, table_type == TEE_BF16, d_ids, d_y, y_type == TEE_BF16, T, V, H,
                                                  scale, ctx->d_status, s);
                  });
}

long long tee_embed_backward_workspace(int T, int V, int H) {
    if (T < 0 || T > MAX_ROWS || V < 1 || H < 1 || H > MAX_EMBED_HIDDEN)
        return tee_set_global_error(TEE_EINVAL, "embed_backward_workspace: T, V or H out of range");
    return (long long)embed_backward_ws(T, V, H);
}

int tee_op_embed_backward(tee_ctx* ctx, const void* d_dy, int y_type, const int32_t* d_ids, void* d_dtable,
                          int table_type, int T, int V, int H, float scale, int accumulate, void* d_ws,
                          size_t ws_bytes, void* stream) {
    static const char* op = "embed_backward";
    if (!ctx) return TEE_EINVAL;
    if (!is_type(table_type) || !is_type(y_type)) return bad(ctx, op, "element types must be TEE_F32 or TEE_BF16");
    if (T < 0 || T > MAX_ROWS) return bad(ctx, op, "T out of range");
    if (V < 1) return bad(ctx, op, "V out of range");
    if (H < 1 || H > MAX_EMBED_HIDDEN) return bad(ctx, op, "H out of range");
    if (accumulate != 0 && accumulate != 1) return bad(ctx, op, "accumulate must be 0 or 1");
    if (T == 0 && accumulate) return TEE_OK;
    int rc = check_bufs(ctx, op, {{"d_dtable", d_dtable, 16}});
    if (rc) return rc;
    if (T > 0) {
        if ((rc = check_bufs(ctx, op, {{"d_dy", d_dy, 16}, {"d_ids", d_ids, 4}}))) return rc;
        if ((rc = check_ws(ctx, op, d_ws, ws_bytes, embed_backward_ws(T, V, H)))) return rc;
    }
    return launch(ctx, op, TEE_K_EMBED, 0,
                  (double)T * H * type_size(y_type) + (accumulate ? 0.0 : (double)V * H * type_size(table_type)), stream,
                  [&](cudaStream_t s) {
                      return launch_embed_backward(d_dy, y_type == TEE_BF16, d_ids, d_dtable, table_type == TEE_BF16, T, V,
                                                   H, scale, accumulate != 0, d_ws, ctx->d_status, s);
                  });
}

long long tee_vocab_loss_forward_workspace(int N, int V, int H) {
    if (vocab_sizes(N, V, H)) return tee_set_global_error(TEE_EINVAL, "vocab_loss_forward_workspace: N, V or H out of range");
    return N ? (long long)vocab_loss_ws(N, V, H, false) : 0;
}

int tee_op_vocab_loss_forward(tee_ctx* ctx, const void* d_x, const void* d_w, const int32_t* d_targets, float* d_loss,
                              float* d_lse, int N, int V, int H, int ignore_id, void* d_ws, size_t ws_bytes,
                              void* stream) {
    static const char* op = "vocab_loss_forward";
    if (!ctx) return TEE_EINVAL;
    if (const char* what = vocab_sizes(N, V, H)) return bad(ctx, op, what);
    if (N == 0) return TEE_OK;
    int rc = check_bufs(ctx, op, {{"d_x", d_x, 16}, {"d_w", d_w, 16}, {"d_targets", d_targets, 4}, {"d_loss", d_loss, 4},
                                  {"d_lse", d_lse, 4}});
    if (rc || (rc = check_ws(ctx, op, d_ws, ws_bytes, vocab_loss_ws(N, V, H, false)))) return rc;
    // (products and states go with the number of counted positions, which the host does not know)
    return launch(ctx, op, TEE_K_LOSS, 0, 2.0 * V * H + 12.0 * N, stream, [&](cudaStream_t s) {
        return launch_vocab_loss_forward(d_x, d_w, d_targets, d_loss, d_lse, N, V, H, ignore_id, d_ws, ctx->d_status, s);
    });
}

long long tee_vocab_loss_backward_workspace(int N, int V, int H) {
    if (vocab_sizes(N, V, H)) return tee_set_global_error(TEE_EINVAL, "vocab_loss_backward_workspace: N, V or H out of range");
    return N ? (long long)vocab_loss_ws(N, V, H, true) : 0;
}

int tee_op_vocab_loss_backward(tee_ctx* ctx, const void* d_x, const void* d_w, const int32_t* d_targets,
                               const float* d_lse, const float* d_gloss, void* d_dx, void* d_dw, int N, int V, int H,
                               int ignore_id, void* d_ws, size_t ws_bytes, void* stream) {
    static const char* op = "vocab_loss_backward";
    if (!ctx) return TEE_EINVAL;
    if (const char* what = vocab_sizes(N, V, H)) return bad(ctx, op, what);
    if (!d_dx && !d_dw) return bad(ctx, op, "d_dx and d_dw are both NULL");
    int rc = TEE_OK;
    if (d_dw && (rc = check_bufs(ctx, op, {{"d_dw", d_dw, 16}}))) return rc;
    if (N > 0) {
        if ((rc = check_bufs(ctx, op, {{"d_x", d_x, 16}, {"d_w", d_w, 16}, {"d_targets", d_targets, 4}, {"d_lse", d_lse, 4},
                                       {"d_gloss", d_gloss, 4}})))
            return rc;
        if (d_dx && (rc = check_bufs(ctx, op, {{"d_dx", d_dx, 16}}))) return rc;
        if ((rc = check_ws(ctx, op, d_ws, ws_bytes, vocab_loss_ws(N, V, H, true)))) return rc;
    }
    const double bytes = (N ? 2.0 * V * H + 12.0 * N : 0.0) + (d_dx ? 2.0 * N * H : 0.0) + (d_dw ? 2.0 * V * H : 0.0);
    return launch(ctx, op, TEE_K_LOSS, 0, bytes, stream, [&](cudaStream_t s) {
        return launch_vocab_loss_backward(d_x, d_w, d_targets, d_lse, d_gloss, d_dx, d_dw, N, V, H, ignore_id, d_ws,
                                          ctx->d_status, s);
    });
}

}  // extern "C"
