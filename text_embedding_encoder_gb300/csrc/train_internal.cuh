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

// Eight consecutive elements at a 16-byte aligned address.
__device__ __forceinline__ void load8(const float* p, float* v) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16* p, float* v) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float* v) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(bf16* p, const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
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
