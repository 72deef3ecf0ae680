// The common norm of many gradient tensors and their scaling by it (tee_train.h has
// the formulas).
//
// Bound by memory: the norm has to be known before the first element is scaled, so the
// gradients are read twice and written once.  The second pass goes through them from
// the end, where the first left them in L2.  Measured, 151 tensors of the 310m encoder,
// 315 M elements bf16, 1.89 GB: 299 us, 6.3 TB/s (four 16-byte loads a thread together;
// two 314, eight 308; loads and stores marked for eviction in the second pass 308).
#include "train_internal.cuh"

#include <float.h>

#include <algorithm>

namespace {

constexpr int THREADS = 256;
constexpr int BLOCKS_PER_SM = 3;
// Elements of a chunk, which lies in one tensor.  (Smaller ones where the blocks have less
// than one each: 3.0 M elements 18.8 us for the two launches, 13.4 with these.)
constexpr int CHUNK = 16384;
constexpr int AT_ONCE = 4;               // 16-byte loads of a thread on their way together
constexpr int MAX_TENSORS = 256;         // of one launch
constexpr int MAX_BLOCKS = 1024;         // of one launch

struct Tensor {
    const void* src;
    void* dst;
    long long count;
    int first_chunk;                     // of this launch
    int is_bf16;
};
struct Table {
    Tensor t[MAX_TENSORS];
    int n, chunks;
};

// Calls f(tensor, first element, elements) for the block's share of the chunks, a
// contiguous run of them; from the last to the first where `reverse`.
template <typename F>
__device__ __forceinline__ void for_chunks(const Table& table, bool reverse, F&& f) {
    const int b = reverse ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
    const int lo = (int)((long long)table.chunks * b / gridDim.x), hi = (int)((long long)table.chunks * (b + 1) / gridDim.x);
    if (lo >= hi) return;
    const int start = reverse ? hi - 1 : lo;
    int i = 0, above = table.n;          // the tensor that holds chunk `start`
    while (above - i > 1) {
        const int mid = (i + above) / 2;
        if (table.t[mid].first_chunk <= start) i = mid;
        else above = mid;
    }
    for (int k = 0; k < hi - lo; ++k) {
        const int c = reverse ? hi - 1 - k : lo + k;
        if (reverse) {
            while (c < table.t[i].first_chunk) --i;
        } else {
            while (i + 1 < table.n && c >= table.t[i + 1].first_chunk) ++i;
        }
        const long long at = (long long)(c - table.t[i].first_chunk) * CHUNK;
        f(table.t[i], at, (int)min((long long)CHUNK, table.t[i].count - at));
    }
}

// Squares of a thread's elements of a chunk, summed in fp32 -- at most CHUNK / THREADS
// of them -- and whether any element is not zero.
struct Squares {
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t bits = 0;
    __device__ __forceinline__ void add(float v, int lane) {
        sum[lane & 3] = fmaf(v, v, sum[lane & 3]);
        bits |= __float_as_uint(v);
    }
    __device__ __forceinline__ void add_word(const float*, uint32_t w, int lane) { add(__uint_as_float(w), lane); }
    __device__ __forceinline__ void add_word(const bf16*, uint32_t w, int lane) {
        float a, b;
        unpack_bf16x2(w, a, b);
        add(a, lane);
        add(b, lane);
    }
    __device__ __forceinline__ float total() const { return (sum[0] + sum[1]) + (sum[2] + sum[3]); }
};

template <typename E, int W>
__device__ __forceinline__ double chunk_squares(const E* p, int n) {
    Squares q;
    const bool vec = (reinterpret_cast<uintptr_t>(p) & 15) == 0;
    const int whole = vec ? n / W : 0;
    const uint4* from = reinterpret_cast<const uint4*>(p);
    for (int i0 = threadIdx.x; i0 < whole; i0 += AT_ONCE * THREADS) {
        uint4 v[AT_ONCE];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) v[k] = i0 + k * THREADS < whole ? from[i0 + k * THREADS] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            q.add_word(p, v[k].x, 0);
            q.add_word(p, v[k].y, 1);
            q.add_word(p, v[k].z, 2);
            q.add_word(p, v[k].w, 3);
        }
    }
    for (int i = whole * W + threadIdx.x; i < n; i += THREADS) q.add(elem_to_f32(p[i]), i);
    const float s = q.total();
    // squares past fp32's range, at either end: again in 64 bits
    if ((q.bits & 0x7fffffffu) == 0) return 0.0;
    if (s > 0x1p-90f && s < 0x1p120f) return (double)s;
    double d = 0.0;
    for (int i = threadIdx.x; i < whole; i += THREADS)
        for (int j = 0; j < W; ++j) {
            const double v = elem_to_f32(p[(size_t)i * W + j]);
            d += v * v;
        }
    for (int i = whole * W + threadIdx.x; i < n; i += THREADS) {
        const double v = elem_to_f32(p[i]);
        d += v * v;
    }
    return d;
}

__device__ __forceinline__ double block_sum(double v, double* shared) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) t += shared[w];
    return t;
}

// A sum of squares per block.  The shares depend on the sizes alone, so the same
// inputs give the same bits.
__global__ void __launch_bounds__(THREADS, BLOCKS_PER_SM)
    clip_norm_kernel(const __grid_constant__ Table table, double* __restrict__ sums) {
    __shared__ double shared[THREADS / 32];
    pdl_wait();
    pdl_trigger();
    double d = 0.0;
    for_chunks(table, false, [&](const Tensor& t, long long at, int n) {
        d += t.is_bf16 ? chunk_squares<bf16, 8>((const bf16*)t.src + at, n) : chunk_squares<float, 4>((const float*)t.src + at, n);
    });
    const double s = block_sum(d, shared);
    if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

__device__ __forceinline__ uint32_t scale_word(const float*, uint32_t w, float f) { return __float_as_uint(__uint_as_float(w) * f); }
__device__ __forceinline__ uint32_t scale_word(const bf16*, uint32_t w, float f) {
    float a, b;
    unpack_bf16x2(w, a, b);
    return pack_bf16x2(a * f, b * f);
}
template <typename E, int W>
__device__ __forceinline__ void chunk_scale(const E* src, E* dst, int n, float factor) {
    const bool vec = ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15) == 0;
    const int whole = vec ? n / W : 0;
    const uint4* from = reinterpret_cast<const uint4*>(src);
    uint4* to = reinterpret_cast<uint4*>(dst);
    for (int i0 = threadIdx.x; i0 < whole; i0 += AT_ONCE * THREADS) {
        uint4 v[AT_ONCE];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k)
            if (i0 + k * THREADS < whole) v[k] = from[i0 + k * THREADS];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            if (i0 + k * THREADS >= whole) break;
            to[i0 + k * THREADS] = make_uint4(scale_word(src, v[k].x, factor), scale_word(src, v[k].y, factor),
                                              scale_word(src, v[k].z, factor), scale_word(src, v[k].w, factor));
        }
    }
    for (int i = whole * W + threadIdx.x; i < n; i += THREADS) f32_to_elem(elem_to_f32(src[i]) * factor, dst[i]);
}

template <typename U>
__device__ __forceinline__ void chunk_copy(const U* src, U* dst, int n) {
    constexpr int W = 16 / sizeof(U);
    const bool vec = ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15) == 0;
    const int whole = vec ? n / W : 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < whole; i += THREADS) reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(src)[i];
    for (int i = whole * W + threadIdx.x; i < n; i += THREADS) dst[i] = src[i];
}

// Every block adds up the blocks' sums by itself, in the same order; block 0 of the
// first launch writes the norm and the factor.
__global__ void __launch_bounds__(THREADS, BLOCKS_PER_SM)
    clip_scale_kernel(const __grid_constant__ Table table, const double* __restrict__ sums, int n_sums, float max_norm,
                      float* __restrict__ norm_out) {
    __shared__ double shared[THREADS / 32];
    pdl_wait();
    pdl_trigger();
    double d = 0.0;
    for (int i = threadIdx.x; i < n_sums; i += THREADS) d += sums[i];
    const double norm = sqrt(block_sum(d, shared));
    float factor = 1.f;                              // also where the norm is not a number or infinite
    if (norm > (double)max_norm && norm <= (double)FLT_MAX) factor = (float)((double)max_norm / norm);
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) norm_out[0] = (float)norm, norm_out[1] = factor;
    for_chunks(table, true, [&](const Tensor& t, long long at, int n) {
        if (factor == 1.f) {                         // bit by bit, NaN too
            if (t.src == t.dst) return;
            if (t.is_bf16) chunk_copy((const uint16_t*)t.src + at, (uint16_t*)t.dst + at, n);
            else chunk_copy((const uint32_t*)t.src + at, (uint32_t*)t.dst + at, n);
            return;
        }
        if (t.is_bf16) chunk_scale<bf16, 8>((const bf16*)t.src + at, (bf16*)t.dst + at, n, factor);
        else chunk_scale<float, 4>((const float*)t.src + at, (float*)t.dst + at, n, factor);
    });
}

int launches(int n_tensors) { return std::max(1, (n_tensors + MAX_TENSORS - 1) / MAX_TENSORS); }

}  // namespace

size_t clip_gradients_ws(int n_tensors) { return (size_t)launches(n_tensors) * MAX_BLOCKS * sizeof(double); }

cudaError_t launch_clip_gradients(const void* const* src, const int32_t* types, const int64_t* counts,
                                  const void* const* dst, int n_tensors, float max_norm, float* norm, void* ws, cudaStream_t s) {
    int dev = 0, num_sms = 0;
    cudaError_t e = tee_current_device(&dev, &num_sms);
    if (e != cudaSuccess) return e;
    double* sums = (double*)ws;
    int n_sums = 0;
    Table table;
    // the tensors [a, a + MAX_TENSORS); the launch's blocks
    auto fill = [&](int a) {
        table.n = table.chunks = 0;
        for (int i = a; i < std::min(n_tensors, a + MAX_TENSORS); ++i) {
            if (counts[i] == 0) continue;
            table.t[table.n++] = Tensor{src[i], const_cast<void*>(dst[i]), counts[i], table.chunks, types[i] == TEE_BF16};
            table.chunks += (int)((counts[i] + CHUNK - 1) / CHUNK);
        }
        return std::max(1, std::min(std::min(table.chunks, num_sms * BLOCKS_PER_SM), MAX_BLOCKS));
    };
    const int n_launches = launches(n_tensors);
    for (int l = 0; l < n_launches; ++l) {
        const int grid = fill(l * MAX_TENSORS);
        e = launch_pdl(clip_norm_kernel, dim3(grid), dim3(THREADS), 0, s, table, sums + n_sums);
        if (e != cudaSuccess) return e;
        n_sums += grid;
    }
    for (int l = n_launches - 1; l >= 0; --l) {
        const int grid = n_launches == 1 ? std::max(1, std::min(std::min(table.chunks, num_sms * BLOCKS_PER_SM), MAX_BLOCKS))
                                         : fill(l * MAX_TENSORS);
        e = launch_pdl(clip_scale_kernel, dim3(grid), dim3(THREADS), 0, s, table, (const double*)sums, n_sums, max_norm,
                       l == 0 ? norm : nullptr);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}
