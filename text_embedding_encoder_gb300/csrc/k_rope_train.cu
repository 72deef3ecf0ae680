// Rotary positions on packed qkv rows, forward and backward (tee_train.h has the
// formulas): the backward pass of a rotation is the rotation by the negated angle.
//
// Bound by memory: every element is read and written once.  Measured, 65536 rows of 12
// heads, bf16, 604 MB: 91 us, 6.6 TB/s (16 rows to a block 93, 32 100; two pairs of loads
// together 96, six 103).
#include "train_internal.cuh"

#include <math.h>

namespace {

constexpr int THREADS = 256;
constexpr int MAX_ROWS = 8;    // rows of a block
constexpr int HALF = 32;       // pairs of a head
constexpr int AT_ONCE = 3;     // pairs of loads on their way together
constexpr int BLOCKS_PER_SM = 4;

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

// 16 bytes as fp32 elements, and back.
__device__ __forceinline__ void widen(const uint4& q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void widen(const uint4& q, float (&v)[8]) {
    unpack_bf16x2(q.x, v[0], v[1]);
    unpack_bf16x2(q.y, v[2], v[3]);
    unpack_bf16x2(q.z, v[4], v[5]);
    unpack_bf16x2(q.w, v[6], v[7]);
}
__device__ __forceinline__ uint4 narrow(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 narrow(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// A thread moves vectors of W elements, 16 bytes: one of a head's first half and the one
// it pairs with, 32 elements on.  out may be x.  The first loads are on their way while
// the block makes its rows' cos and sin.
template <int W>
__global__ void __launch_bounds__(THREADS, BLOCKS_PER_SM)
    rope_kernel(const uint4* x, const int32_t* __restrict__ pos, uint4* out, int T, int heads, int rows, float sign,
                const __grid_constant__ Turns turns) {
    __shared__ float2 cs[MAX_ROWS][HALF];
    pdl_wait();
    pdl_trigger();
    const int row0 = blockIdx.x * rows, n = min(rows, T - row0);
    constexpr int VECS = HALF / W;                        // vectors of half a head
    const int moved = out == x ? 2 * heads : 3 * heads;   // in place the values stay
    const int per_row = moved * VECS, items = n * per_row;
    uint4 u[AT_ONCE], v[AT_ONCE];
    auto place = [&](int i, int& row, int& head, int& vec) {
        row = i / per_row;
        const int k = i - row * per_row;
        head = k / VECS, vec = k % VECS;
        return ((size_t)(row0 + row) * 3 * heads + head) * 2 * VECS + vec;
    };
    auto load = [&](int i0) {
#pragma unroll
        for (int q = 0; q < AT_ONCE; ++q) {
            int row, head, vec;
            if (i0 + q * THREADS >= items) break;
            const size_t at = place(i0 + q * THREADS, row, head, vec);
            u[q] = x[at];
            v[q] = x[at + VECS];
        }
    };
    int i0 = threadIdx.x;
    load(i0);
    for (int i = threadIdx.x; i < n * HALF; i += THREADS) {
        float2 t = cos_sin_of_turns((double)pos[row0 + i / HALF] * turns.per_position[i % HALF]);
        t.y *= sign;
        cs[i / HALF][i % HALF] = t;
    }
    __syncthreads();
    while (i0 < items) {
#pragma unroll
        for (int q = 0; q < AT_ONCE; ++q) {
            int row, head, vec;
            if (i0 + q * THREADS >= items) break;
            const size_t at = place(i0 + q * THREADS, row, head, vec);
            if (head < 2 * heads) {
                float a[W], b[W];
                widen(u[q], a);
                widen(v[q], b);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const float2 t = cs[row][vec * W + j];
                    const float c = a[j], d = b[j];
                    a[j] = c * t.x - d * t.y;
                    b[j] = d * t.x + c * t.y;
                }
                u[q] = narrow(a);
                v[q] = narrow(b);
            }
            out[at] = u[q];
            out[at + VECS] = v[q];
        }
        i0 += AT_ONCE * THREADS;
        load(i0);
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
    auto kernel = is_bf16 ? rope_kernel<8> : rope_kernel<4>;
    return launch_pdl(kernel, grid, dim3(THREADS), 0, s, (const uint4*)x, pos, (uint4*)out, T, heads, rows, sign, turns);
}
