// Declarations shared by the training operators' translation units.
#pragma once

#include "tee_internal.cuh"
#include "tee_train.h"

// Sub-allocator of a caller's workspace (offsets aligned to 256 bytes from its
// base); with base == nullptr it only adds up the size.
struct WsCarve {
    char* base;
    size_t off = 0;
    explicit WsCarve(void* b) : base((char*)b) {}
    template <typename T>
    T* take(size_t count) {
        T* p = (T*)(base ? base + off : nullptr);
        off = (off + count * sizeof(T) + 255) / 256 * 256;
        return p;
    }
};

// ---- fp32 <-> stored elements ------------------------------------------------
__device__ __forceinline__ float elem_to_f32(float v) { return v; }
__device__ __forceinline__ float elem_to_f32(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void f32_to_elem(float v, float& o) { o = v; }
__device__ __forceinline__ void f32_to_elem(float v, bf16& o) { o = __float2bfloat16_rn(v); }

// W consecutive elements at an address aligned to W elements (at most 16 bytes):
// 8 bf16, or 4 or 2 of either type.  A warp whose lanes move 16 bytes each side by side
// covers whole sectors with every instruction; eight fp32 elements a lane (32
// bytes apart) would touch each sector twice (measured: 58 against 40 us for the
// lookup's gradient sums of 65536 rows of 768).
__device__ __forceinline__ void load_vec(const float* p, float (&v)[4]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}
__device__ __forceinline__ void unpack_bf16x2(uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void load_vec(const bf16* p, float (&v)[4]) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    unpack_bf16x2(q.x, v[0], v[1]);
    unpack_bf16x2(q.y, v[2], v[3]);
}
__device__ __forceinline__ void unpack_bf16x8(const uint4& q, float (&v)[8]) {
    unpack_bf16x2(q.x, v[0], v[1]);
    unpack_bf16x2(q.y, v[2], v[3]);
    unpack_bf16x2(q.z, v[4], v[5]);
    unpack_bf16x2(q.w, v[6], v[7]);
}
__device__ __forceinline__ void load_vec(const bf16* p, float (&v)[8]) {
    unpack_bf16x8(*reinterpret_cast<const uint4*>(p), v);
}
__device__ __forceinline__ void load_vec(const float* p, float (&v)[2]) {
    const float2 a = *reinterpret_cast<const float2*>(p);
    v[0] = a.x, v[1] = a.y;
}
__device__ __forceinline__ void load_vec(const bf16* p, float (&v)[2]) {
    unpack_bf16x2(*reinterpret_cast<const uint32_t*>(p), v[0], v[1]);
}
__device__ __forceinline__ void store_vec(float* p, const float (&v)[2]) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
}
__device__ __forceinline__ void store_vec(bf16* p, const float (&v)[2]) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v[0], v[1]);
}
__device__ __forceinline__ void store_vec(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_vec(bf16* p, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void store_vec(bf16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                              pack_bf16x2(v[6], v[7]));
}

// ---- values that are not finite -------------------------------------------------
template <int N>
__device__ __forceinline__ bool all_nan(const float (&v)[N]) {
    bool all = true;
#pragma unroll
    for (int i = 0; i < N; ++i) all &= v[i] != v[i];
    return all;
}
// Whether the 64 elements of a head's row all are NaN, or all are finite.
__device__ __forceinline__ bool all_nan(const bf16* row) {
    bool all = true;
#pragma unroll
    for (int c = 0; c < 64; c += 8) {
        float v[8];
        load_vec(row + c, v);
        all &= all_nan(v);
    }
    return all;
}
__device__ __forceinline__ bool all_finite(const bf16* row) {
    float z = 0.f;
#pragma unroll
    for (int c = 0; c < 64; c += 8) {
        float v[8];
        load_vec(row + c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) z = fmaf(v[i], 0.f, z);
    }
    return z == 0.f;
}
// Of sums that a warp holds in four parts, an eighth of them in each of eight lanes: whether
// `mine` holds for one part at least of each eighth.
__device__ __forceinline__ bool each_eighth_has(bool mine) {
    unsigned b = __ballot_sync(0xffffffffu, mine);
    b |= b >> 16;
    return ((b | b >> 8) & 0xffu) == 0xffu;
}

__device__ __forceinline__ float warp_sum_f32(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---- launchers (each returns the launch's error) -------------------------------
// LayerNorm over rows of any width 1 .. TEE_LN_MAX_HIDDEN.
cudaError_t launch_layernorm_forward(const void* x, bool x_bf16, const float* gamma, void* y, bool y_bf16, float* stats,
                                     int T, int H, float eps, cudaStream_t s);
cudaError_t launch_layernorm_backward(const void* dy, bool y_bf16, const void* x, bool x_bf16, const float* gamma,
                                      const float* stats, const void* dres, void* dx, float* dgamma, int T, int H,
                                      void* ws, cudaStream_t s);
size_t layernorm_backward_ws(int T, int H);

cudaError_t launch_embed_forward(const void* table, bool e_bf16, const int32_t* ids, void* y, bool y_bf16, int T, int V,
                                 int H, float scale, unsigned int* status, cudaStream_t s);
cudaError_t launch_embed_backward(const void* dy, bool y_bf16, const int32_t* ids, void* dtable, bool e_bf16, int T,
                                  int V, int H, float scale, bool accumulate, void* ws, unsigned int* status,
                                  cudaStream_t s);
size_t embed_backward_ws(int T, int V, int H);

// Softmax cross entropy over the vocabulary: x bf16[N, H], wt bf16[V, H], H % 8 == 0.
cudaError_t launch_vocab_loss_forward(const void* x, const void* wt, const int32_t* targets, float* loss, float* lse, int N,
                                      int V, int H, int ignore_id, void* ws, unsigned int* status, cudaStream_t s);
// dx and dw may each be NULL.
cudaError_t launch_vocab_loss_backward(const void* x, const void* wt, const int32_t* targets, const float* lse,
                                       const float* gloss, void* dx, void* dw, int N, int V, int H, int ignore_id, void* ws,
                                       unsigned int* status, cudaStream_t s);
size_t vocab_loss_ws(int N, int V, int H, bool backward);

// Rotary positions of packed qkv [T, 3 * 64 heads]; out may be x.
cudaError_t launch_rope_train(const void* x, bool is_bf16, const int32_t* pos, void* out, int T, int heads, float base,
                              bool backward, cudaStream_t s);

// Norm of all tensors and their scaling; the arrays are the host's.
cudaError_t launch_clip_gradients(const void* const* src, const int32_t* types, const int64_t* counts,
                                  const void* const* dst, int n_tensors, float max_norm, float* norm, void* ws, cudaStream_t s);
size_t clip_gradients_ws(int n_tensors);

// ---- attention (training) ----------------------------------------------------------
#define TEE_ATTN_MAX_TEXT TEE_ATTN_MAX_TEXT_TOKENS

// What the plan kernel leaves on the device for the attention kernels.
struct AttnPlan {
    int* n_items;       // work items in use (0 where the texts' offsets are not valid)
    int4* items;        // {q_start, q_len, k_lo, k_hi}: up to 128 rows and the keys they may see; of whole texts the longest first
    int2* row_tb;       // per token: {start, end} of its text, {0, 0} behind the last
    int* scratch;
    float* nlse2;       // backward: -lse / ln 2, [n_heads, T]
    float* ndelta;      // backward: -sum_d do o, [n_heads, T]
};

// The units of CTA c of G: one of each round of G, in turn from the first CTA on and
// from the last on.  Of whole texts they are listed the longest first, so that evens the sums
// out without the host knowing the texts; of windows they are in the order of their rows
// (nearly all alike, but for windows that are wide beside some of the texts).
__device__ __forceinline__ int attn_unit(int i, int c, int G) { return i * G + ((i & 1) ? G - 1 - c : c); }
__device__ __forceinline__ int attn_units_of(int n, int c, int G) {
    const int rounds = n / G;
    return rounds + (((rounds & 1) ? G - 1 - c : c) < n - rounds * G);
}

int attention_max_items(int T, int n_texts);
size_t attention_train_ws(int T, int n_texts, int n_heads, bool backward);
// window < 0: whole texts.
cudaError_t launch_attention_train_forward(const void* qkv, const int32_t* cu, void* o, float* lse, int T, int n_texts,
                                           int n_heads, int window, void* ws, unsigned int* status, cudaStream_t s);
cudaError_t launch_attention_train_backward(const void* qkv, const int32_t* cu, const void* o, const float* lse,
                                            const void* d_o, void* dqkv, int T, int n_texts, int n_heads, int window,
                                            void* ws, unsigned int* status, cudaStream_t s);
// The forward kernel over a plan (the attention kernel of the encoder's pass).
cudaError_t launch_attention_train_tc(const void* qkv, int T, int n_heads, int window, const AttnPlan& plan, int max_items,
                                      void* o, float* lse, unsigned int* status, cudaStream_t s);

// ---- gated feed-forward -------------------------------------------------------------
cudaError_t launch_geglu_train_forward(const void* x, const void* wi, void* z, int T, int H, int I, unsigned int* status,
                                       cudaStream_t s);
// dx and dwi may each be NULL.
cudaError_t launch_geglu_train_backward(const void* x, const void* wi, const void* dz, void* dx, void* dwi, int T, int H,
                                        int I, void* ws, unsigned int* status, cudaStream_t s);
size_t geglu_backward_ws(int T, int H, int I);
