// Entry points of the training operators (tee_train.h): argument checks, the
// context's device, one launcher call each.
#include "clip_ranges.h"
#include "train_internal.cuh"

#include <float.h>
#include <stdio.h>

#include <algorithm>
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
constexpr int MAX_CLIP_TENSORS = 65536;
constexpr long long MAX_CLIP_COUNT = 1LL << 34;   // elements of one gradient
constexpr int MAX_ATTN_ROWS = 1 << 24;   // T of rotary positions and attention

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

int tee_op_rope(tee_ctx* ctx, const char* op, const void* x, int type, const int32_t* pos, void* y, int T, int n_heads,
                float base, bool backward, void* stream) {
    if (!ctx) return TEE_EINVAL;
    if (!is_type(type)) return bad(ctx, op, "element type must be TEE_F32 or TEE_BF16");
    if (T < 0 || T > MAX_ATTN_ROWS) return bad(ctx, op, "T out of range");
    if (n_heads < 1 || n_heads > TEE_ATTN_MAX_HEADS) return bad(ctx, op, "n_heads out of range");
    if (!(base > 0.f) || base > FLT_MAX) return bad(ctx, op, "base must be positive and finite");
    if (T == 0) return TEE_OK;
    const int rc = check_bufs(ctx, op, {{backward ? "d_dy" : "d_x", x, 16}, {"d_pos", pos, 4}, {backward ? "d_dx" : "d_y", y, 16}});
    if (rc) return rc;
    return launch(ctx, op, TEE_K_ELEMENTWISE, 0, 2.0 * T * 192 * n_heads * type_size(type), stream, [&](cudaStream_t s) {
        return launch_rope_train(x, type == TEE_BF16, pos, y, T, n_heads, base, backward, s);
    });
}

// Sizes of the attention operators; the message of what is wrong with them, or NULL.
const char* attention_sizes(int T, int n_texts, int n_heads) {
    if (T < 0 || T > MAX_ATTN_ROWS) return "T out of range";
    if (n_texts < 0 || n_texts > (1 << 20)) return "n_texts out of range";
    if (n_heads < 1 || n_heads > TEE_ATTN_MAX_HEADS) return "n_heads out of range";
    return nullptr;
}

const char* geglu_sizes(int T, int H, int I) {
    if (T < 0 || T > (1 << 24)) return "T out of range";
    if (H < 8 || H % 8 || H > TEE_GEGLU_MAX_HIDDEN) return "H must be a multiple of 8 within range";
    if (I < 8 || I % 8 || I > TEE_GEGLU_MAX_WIDTH) return "I must be a multiple of 8 within range";
    return nullptr;
}

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

int tee_op_rope_forward(tee_ctx* ctx, const void* d_x, int type, const int32_t* d_pos, void* d_y, int T, int n_heads,
                        float base, void* stream) {
    return tee_op_rope(ctx, "rope_forward", d_x, type, d_pos, d_y, T, n_heads, base, false, stream);
}

int tee_op_rope_backward(tee_ctx* ctx, const void* d_dy, int type, const int32_t* d_pos, void* d_dx, int T, int n_heads,
                         float base, void* stream) {
    return tee_op_rope(ctx, "rope_backward", d_dy, type, d_pos, d_dx, T, n_heads, base, true, stream);
}

long long tee_attention_forward_workspace(int T, int n_texts, int n_heads) {
    if (attention_sizes(T, n_texts, n_heads))
        return tee_set_global_error(TEE_EINVAL, "attention_forward_workspace: T, n_texts or n_heads out of range");
    return T && n_texts ? (long long)attention_train_ws(T, n_texts, n_heads, false) : 0;
}

int tee_op_attention_forward(tee_ctx* ctx, const void* d_qkv, const int32_t* d_cu, void* d_o, float* d_lse, int T,
                             int n_texts, int n_heads, int window, void* d_ws, size_t ws_bytes, void* stream) {
    static const char* op = "attention_forward";
    if (!ctx) return TEE_EINVAL;
    if (const char* what = attention_sizes(T, n_texts, n_heads)) return bad(ctx, op, what);
    if (T == 0 || n_texts == 0) return TEE_OK;
    int rc = check_bufs(ctx, op, {{"d_qkv", d_qkv, 16}, {"d_cu", d_cu, 4}, {"d_o", d_o, 16}, {"d_lse", d_lse, 4}});
    if (rc || (rc = check_ws(ctx, op, d_ws, ws_bytes, attention_train_ws(T, n_texts, n_heads, false)))) return rc;
    // (products go with the texts' lengths, which the host does not know)
    return launch(ctx, op, TEE_K_ATTENTION, 0, (512.0 + 4.0) * T * n_heads, stream, [&](cudaStream_t s) {
        return launch_attention_train_forward(d_qkv, d_cu, d_o, d_lse, T, n_texts, n_heads, std::min(window, T), d_ws,
                                              ctx->d_status, s);
    });
}

long long tee_attention_backward_workspace(int T, int n_texts, int n_heads) {
    if (attention_sizes(T, n_texts, n_heads))
        return tee_set_global_error(TEE_EINVAL, "attention_backward_workspace: T, n_texts or n_heads out of range");
    return T && n_texts ? (long long)attention_train_ws(T, n_texts, n_heads, true) : 0;
}

int tee_op_attention_backward(tee_ctx* ctx, const void* d_qkv, const int32_t* d_cu, const void* d_o, const float* d_lse,
                              const void* d_do, void* d_dqkv, int T, int n_texts, int n_heads, int window, void* d_ws,
                              size_t ws_bytes, void* stream) {
    static const char* op = "attention_backward";
    if (!ctx) return TEE_EINVAL;
    if (const char* what = attention_sizes(T, n_texts, n_heads)) return bad(ctx, op, what);
    if (T == 0 || n_texts == 0) return TEE_OK;
    int rc = check_bufs(ctx, op, {{"d_qkv", d_qkv, 16}, {"d_cu", d_cu, 4}, {"d_o", d_o, 16}, {"d_lse", d_lse, 4},
                                  {"d_do", d_do, 16}, {"d_dqkv", d_dqkv, 16}});
    if (rc || (rc = check_ws(ctx, op, d_ws, ws_bytes, attention_train_ws(T, n_texts, n_heads, true)))) return rc;
    return launch(ctx, op, TEE_K_ATTENTION, 0, (1024.0 + 4.0) * T * n_heads, stream, [&](cudaStream_t s) {
        return launch_attention_train_backward(d_qkv, d_cu, d_o, d_lse, d_do, d_dqkv, T, n_texts, n_heads,
                                               std::min(window, T), d_ws, ctx->d_status, s);
    });
}

int tee_op_geglu_forward(tee_ctx* ctx, const void* d_x, const void* d_wi, void* d_z, int T, int H, int I, void* stream) {
    static const char* op = "geglu_forward";
    if (!ctx) return TEE_EINVAL;
    if (const char* what = geglu_sizes(T, H, I)) return bad(ctx, op, what);
    if (T == 0) return TEE_OK;
    const int rc = check_bufs(ctx, op, {{"d_x", d_x, 16}, {"d_wi", d_wi, 16}, {"d_z", d_z, 16}});
    if (rc) return rc;
    return launch(ctx, op, TEE_K_GEMM, 4.0 * T * H * I, 2.0 * ((double)T * (H + I) + 2.0 * I * H), stream, [&](cudaStream_t s) {
        return launch_geglu_train_forward(d_x, d_wi, d_z, T, H, I, ctx->d_status, s);
    });
}

long long tee_geglu_backward_workspace(int T, int H, int I) {
    if (geglu_sizes(T, H, I)) return tee_set_global_error(TEE_EINVAL, "geglu_backward_workspace: T, H or I out of range");
    return T ? (long long)geglu_backward_ws(T, H, I) : 0;
}

int tee_op_geglu_backward(tee_ctx* ctx, const void* d_x, const void* d_wi, const void* d_dz, void* d_dx, void* d_dwi, int T,
                          int H, int I, void* d_ws, size_t ws_bytes, void* stream) {
    static const char* op = "geglu_backward";
    if (!ctx) return TEE_EINVAL;
    if (const char* what = geglu_sizes(T, H, I)) return bad(ctx, op, what);
    if (!d_dx && !d_dwi) return bad(ctx, op, "d_dx and d_dwi are both NULL");
    int rc = TEE_OK;
    if (d_dwi && (rc = check_bufs(ctx, op, {{"d_dwi", d_dwi, 16}}))) return rc;
    if (T > 0) {
        if ((rc = check_bufs(ctx, op, {{"d_x", d_x, 16}, {"d_wi", d_wi, 16}, {"d_dz", d_dz, 16}}))) return rc;
        if (d_dx && (rc = check_bufs(ctx, op, {{"d_dx", d_dx, 16}}))) return rc;
        if ((rc = check_ws(ctx, op, d_ws, ws_bytes, geglu_backward_ws(T, H, I)))) return rc;
    }
    const double product = 4.0 * T * H * I;
    const double bytes = 2.0 * ((double)T * (H + I) + (T ? 2.0 * I * H : 0.0) + (d_dx ? (double)T * H : 0.0) + (d_dwi ? 2.0 * I * H : 0.0));
    return launch(ctx, op, TEE_K_GEMM, product * (1 + (d_dx != nullptr) + (d_dwi != nullptr)), bytes, stream, [&](cudaStream_t s) {
        return launch_geglu_train_backward(d_x, d_wi, d_dz, d_dx, d_dwi, T, H, I, d_ws, ctx->d_status, s);
    });
}

long long tee_clip_gradients_workspace(int n_tensors) {
    if (n_tensors < 0 || n_tensors > MAX_CLIP_TENSORS)
        return tee_set_global_error(TEE_EINVAL, "clip_gradients_workspace: n_tensors out of range");
    return (long long)clip_gradients_ws(n_tensors);
}

int tee_op_clip_gradients(tee_ctx* ctx, const void* const* h_grads, const int32_t* h_types, const int64_t* h_counts,
                          void* const* h_outs, int n_tensors, float max_norm, float* d_norm, void* d_ws,
                          size_t ws_bytes, void* stream) {
    static const char* op = "clip_gradients";
    if (!ctx) return TEE_EINVAL;
    if (n_tensors < 0 || n_tensors > MAX_CLIP_TENSORS) return bad(ctx, op, "n_tensors out of range");
    if (!(max_norm >= 0.f)) return bad(ctx, op, "max_norm must be >= 0");
    if (n_tensors && (!h_grads || !h_types || !h_counts)) return bad(ctx, op, "h_grads, h_types or h_counts is NULL");
    int rc = check_bufs(ctx, op, {{"d_norm", d_norm, 4}});
    if (rc || (rc = check_ws(ctx, op, d_ws, ws_bytes, clip_gradients_ws(n_tensors)))) return rc;
    double bytes = 0;
    for (int i = 0; i < n_tensors; ++i) {
        if (!is_type(h_types[i])) return bad(ctx, op, "element types must be TEE_F32 or TEE_BF16");
        if (h_counts[i] < 0 || h_counts[i] > MAX_CLIP_COUNT) return bad(ctx, op, "a count is out of range");
        if (h_counts[i] == 0) continue;
        const int align = (int)type_size(h_types[i]);
        if ((rc = check_bufs(ctx, op, {{"a gradient", h_grads[i], align}}))) return rc;
        if (h_outs && (rc = check_bufs(ctx, op, {{"an output", h_outs[i], align}}))) return rc;
        bytes += 3.0 * h_counts[i] * align;
    }
    const int overlap = clip_overlaps(h_grads, h_counts, h_types, TEE_BF16, h_outs, n_tensors);
    if (overlap < 0) return tee_set_error(ctx, TEE_ENOMEM, "clip_gradients: host allocation failed");
    if (overlap) return bad(ctx, op, "tensors overlap");
    return launch(ctx, op, TEE_K_ELEMENTWISE, 0, bytes, stream, [&](cudaStream_t s) {
        return launch_clip_gradients(h_grads, h_types, h_counts, h_outs ? (const void* const*)h_outs : h_grads, n_tensors,
                                     max_norm, d_norm, d_ws, s);
    });
}

}  // extern "C"
