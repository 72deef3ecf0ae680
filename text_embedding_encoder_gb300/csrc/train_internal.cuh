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
__device__ __forceinline__ void load_vec(const bf16* p, float (&v)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    unpack_bf16x2(q.x, v[0], v[1]);
    unpack_bf16x2(q.y, v[2], v[3]);
    unpack_bf16x2(q.z, v[4], v[5]);
    unpack_bf16x2(q.w, v[6], v[7]);
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
