// Rotary positions on packed qkv rows, forward and backward (tee_train.h has the
// formulas): the backward pass of a rotation is the rotation by the negated angle.
//
// Bound by memory: every element is read and written once.  Measured: 65536 rows of 12
// heads, bf16, 604 MB: 92 us, 6.5 TB/s.
#include "train_internal.cuh"

#include <math.h>

namespace {

constexpr int THREADS = 256;
constexpr int MAX_ROWS = 16;   // rows of a block
constexpr int HALF = 32;       // pairs of a head

// Turns of the 32 pairs per position: base^(-j / 32) / (2 pi).
struct Turns {
    double per_position[HALF];
};

// cos and sin of 2 pi `turns`.  Angles of far positions are thousands of turns, so
// whole turns are taken off in 64 bits; what is left goes through sincospif as fp32,
// and the part that fp32 dropped (< 2^-25 of a turn) is added by the angle-sum rule.
__device__ __forceinline__ float2 cos_sin_of_turns(double turns) {
    const double r = turns - rint(turns);
    const float hi = (float)r, lo = (float)(r - (double)hi) * 6.28318531f;
    float s, c;
    sincospif(2.f * hi, &s, &c);
    return make_float2(fmaf(-lo, s, c), fmaf(lo, c, s));
}

// A thread moves vectors of W elements, 16 bytes: one of a head's first half and the
// one it pairs with, 32 elements on.  out may be x.
template <typename E, int W>
__global__ void __launch_bounds__(THREADS)
    rope_kernel(const E* x, const int32_t* __restrict__ pos, E* out, int T, int heads, int rows, float sign,
                const __grid_constant__ Turns turns) {
    __shared__ float2 cs[MAX_ROWS][HALF];
    pdl_wait();
    pdl_trigger();
    const int row0 = blockIdx.x * rows, n = min(rows, T - row0);
    for (int i = threadIdx.x; i < n * HALF; i += THREADS) {
        float2 v = cos_sin_of_turns((double)pos[row0 + i / HALF] * turns.per_position[i % HALF]);
        v.y *= sign;
        cs[i / HALF][i % HALF] = v;
    }
    __syncthreads();
    constexpr int VECS = HALF / W;                 // vectors of half a head
    const int moved = out == x ? 2 * heads : 3 * heads;   // in place the values stay
    const int per_row = moved * VECS, items = n * per_row;
    constexpr int AT_ONCE = 3;                     // pairs of loads on their way together
    for (int i0 = threadIdx.x; i0 < items; i0 += AT_ONCE * THREADS) {
        float u[AT_ONCE][W], v[AT_ONCE][W];
        size_t at[AT_ONCE];
        int row[AT_ONCE], head[AT_ONCE], vec[AT_ONCE];
#pragma unroll
        for (int q = 0; q < AT_ONCE; ++q) {
            const int i = i0 + q * THREADS;
            if (i >= items) break;
            row[q] = i / per_row;
            const int k = i - row[q] * per_row;
            head[q] = k / VECS, vec[q] = k % VECS;
            at[q] = (size_t)(row0 + row[q]) * 3 * heads * 64 + head[q] * 64 + vec[q] * W;
            load_vec(x + at[q], u[q]);
            load_vec(x + at[q] + HALF, v[q]);
        }
#pragma unroll
        for (int q = 0; q < AT_ONCE; ++q) {
            if (i0 + q * THREADS >= items) break;
            if (head[q] < 2 * heads) {
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const float2 t = cs[row[q]][vec[q] * W + j];
                    const float a = u[q][j], b = v[q][j];
                    u[q][j] = a * t.x - b * t.y;
                    v[q][j] = b * t.x + a * t.y;
                }
            }
            store_vec(out + at[q], u[q]);
            store_vec(out + at[q] + HALF, v[q]);
        }
    }
}

}  // namespace

cudaError_t launch_rope_train(const void* x, bool is_bf16, const int32_t* pos, void* out, int T, int heads, float base,
                              bool backward, cudaStream_t s) {
    if (T == 0) return cudaSuccess;
    int dev = 0, num_sms = 0;
    cudaError_t e = tee_current_device(&dev, &num_sms);
    if (e != cudaSuccess) return e;
    Turns turns;
    for (int j = 0; j < HALF; ++j) turns.per_position[j] = pow((double)base, -j / 32.0) / 6.283185307179586476925;
    // four blocks an SM at least, as far as there are rows
    const int fit = (T + 4 * num_sms - 1) / (4 * num_sms), rows = fit < MAX_ROWS ? fit : MAX_ROWS;
    const dim3 grid((T + rows - 1) / rows);
    const float sign = backward ? -1.f : 1.f;
    if (is_bf16)
        return launch_pdl(rope_kernel<bf16, 8>, grid, dim3(THREADS), 0, s, (const bf16*)x, pos, (bf16*)out, T, heads, rows,
                          sign, turns);
    return launch_pdl(rope_kernel<float, 4>, grid, dim3(THREADS), 0, s, (const float*)x, pos, (float*)out, T, heads, rows,
                      sign, turns);
}
