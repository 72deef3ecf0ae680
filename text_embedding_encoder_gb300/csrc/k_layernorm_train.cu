// LayerNorm for training: forward with the rows' statistics, and the backward
// pass with the reduction of the gain's gradient (tee_train.h has the formulas).
//
// Both are bound by HBM: forward reads x and writes y once, backward reads x,
// dy (and the residual gradient) and writes dx once.  A row is held in the
// registers of WPR warps (with_width), so the variance is taken
// around the mean without reading the row again.
//   forward, 65536 x 768 fp32 -> bf16: 43.9 us, 6.9 TB/s.
//   backward, 32768 x 768 fp32, bf16 dy, residual: 55.5 us, 6.4 TB/s, of which 4 are
//     the second launch.
// The backward pass holds a row of x, dy and the gain and the gain's sums at once, and
// what it reaches goes with the rows in flight an SM (bwd_blocks); 210 MB of fp32
// x, bf16 dy, dx: 82 to 87 us from 256 to 4096 columns, 6.1 to 6.4 TB/s; 111 at 1001.
// A few hundred rows are launch latency (backward: two launches).
#include "train_internal.cuh"

namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
// Backward: most thread blocks, each with a partial sum of the gain's gradient
// (four per SM on 152 SMs, rounded up).
constexpr int BWD_MAX_GRID = 640;

// How a row of H elements is spread over a group of G = 32 WPR lanes, N elements
// per lane: in runs of W consecutive ones, moved as vectors, or W = 1, element by
// element; the lanes' runs side by side.  W is the largest of 8 (all types bf16),
// 4, 2 and 1 that divides H.  (Odd widths by vectors that begin where the tensor's
// alignment has them and are masked at the row's ends measured slower: forward 95
// against 58 us, backward 157 against 111, 52376 x 1001.)
template <int W, int N_, int WPR>
struct Row {
    static constexpr int G = 32 * WPR, N = N_;
    static __device__ __forceinline__ int col(int k, int lg) { return (k / W * G + lg) * W + k % W; }
    static __device__ __forceinline__ bool has(int k, int lg, int H) { return col(k / W * W, lg) < H; }
    template <typename T>
    static __device__ __forceinline__ void load(const T* row, int H, int lg, float (&v)[N]) {
#pragma unroll
        for (int k = 0; k < N; k += W) {
            if constexpr (W == 1) {
                v[k] = has(k, lg, H) ? elem_to_f32(row[col(k, lg)]) : 0.f;
            } else {
                float r[W] = {};
                if (has(k, lg, H)) load_part(row + col(k, lg), r);
#pragma unroll
                for (int j = 0; j < W; ++j) v[k + j] = r[j];
            }
        }
    }
    template <typename T>
    static __device__ __forceinline__ void store(T* row, int H, int lg, const float (&v)[N]) {
#pragma unroll
        for (int k = 0; k < N; k += W) {
            if (!has(k, lg, H)) continue;
            if constexpr (W == 1) {
                f32_to_elem(v[k], row[col(k, lg)]);
            } else {
                float r[W];
#pragma unroll
                for (int j = 0; j < W; ++j) r[j] = v[k + j];
                store_part(row + col(k, lg), r);
            }
        }
    }
    // eight fp32 elements (the gain and the partial sums of an all-bf16 norm) go as two vectors
    template <typename T, int M>
    static __device__ __forceinline__ void load_part(const T* p, float (&r)[M]) {
        if constexpr (M == 8 && sizeof(T) == 4) {
            float a[4], b[4];
            load_vec(p, a);
            load_vec(p + 4, b);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = a[j], r[4 + j] = b[j];
        } else {
            load_vec(p, r);
        }
    }
    template <typename T, int M>
    static __device__ __forceinline__ void store_part(T* p, const float (&r)[M]) {
        if constexpr (M == 8 && sizeof(T) == 4) {
            store_vec(p, {r[0], r[1], r[2], r[3]});
            store_vec(p + 4, {r[4], r[5], r[6], r[7]});
        } else {
            store_vec(p, r);
        }
    }
};

// Sum over the group's lanes; every thread of the block calls it.  `red` holds
// one slot per warp and must not be reused before the next block barrier after
// this call's own.
template <int WPR>
__device__ __forceinline__ float2 group_sum(float a, float b, float2* red) {
    a = warp_sum_f32(a);
    b = warp_sum_f32(b);
    if constexpr (WPR > 1) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) red[warp] = make_float2(a, b);
        __syncthreads();
        const int w0 = warp / WPR * WPR;
        a = b = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
            a += red[w0 + w].x;
            b += red[w0 + w].y;
        }
    }
    return make_float2(a, b);
}

template <typename TX, typename TY, int W, int N, int WPR>
__global__ void __launch_bounds__(THREADS) ln_forward_kernel(const TX* x, const float* __restrict__ gamma, TY* y,
                                                             float2* __restrict__ stats, int T, int H, float eps) {
    using R = Row<W, N, WPR>;
    pdl_wait();
    pdl_trigger();
    __shared__ float2 red[2][WARPS];
    const int lg = threadIdx.x % R::G;
    const int t = blockIdx.x * (THREADS / R::G) + threadIdx.x / R::G;
    if (WPR == 1 && t >= T) return;
    const bool live = t < T;
    const size_t base = (size_t)(live ? t : T - 1) * H;
    float v[R::N];
    R::load(x + base, H, lg, v);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < R::N; ++k) s += v[k];
    const float mean = group_sum<WPR>(s, 0.f, red[0]).x / (float)H;
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < R::N; ++k) {
        const float d = R::has(k, lg, H) ? v[k] - mean : 0.f;
        ss += d * d;
    }
    const float rstd = 1.0f / sqrtf(group_sum<WPR>(ss, 0.f, red[1]).x / (float)H + eps);
    if (!live) return;
    float g[R::N];
    R::load(gamma, H, lg, g);
#pragma unroll
    for (int k = 0; k < R::N; ++k) v[k] = (v[k] - mean) * rstd * g[k];
    R::store(y + base, H, lg, v);
    if (stats && lg == 0) stats[t] = make_float2(mean, rstd);
}

// Backward: resident blocks an SM, which give the grid: as many as the row's N
// elements a lane leave registers for.  Measured, us for 210 MB of fp32 x, bf16 dy and
// dx: N = 8, four (251 columns: 101; three 118, six 134); 16, three (1024: 83; two 94);
// 24, two (768: 87; three, with spills, 117).  With N = 32 two blocks spill and one
// leaves the loads exposed (2048 columns: 95 and 136; four warps of 16 a lane 83).
// Rows by single elements keep more addresses: 8 a lane (1001: 111; 16 a lane and
// two blocks 140, 32 and one 495), and two blocks of 16, for which three leave no registers.
template <int W, int N>
constexpr int bwd_blocks() { return N == 8 ? 4 : N == 16 && W > 1 ? 3 : 2; }
// The same as a bound on the registers.  Two blocks of 24 elements a lane fit unasked
// (asked for, two warps a row took 112 us instead of 86 at 1536 columns).
template <int W, int N, int WPR>
constexpr int bwd_min_blocks() { return N == 24 && WPR == 2 ? 1 : bwd_blocks<W, N>(); }

// Groups take rows blockIdx-strided; each lane keeps the gain's gradient of its
// columns over all its rows, the block adds its groups' sums and writes one row
// of partials, which ln_dgamma_kernel adds up in a fixed order.
template <typename TX, typename TY, int W, int N, int WPR>
__global__ void __launch_bounds__(THREADS, bwd_min_blocks<W, N, WPR>())
    ln_backward_kernel(const TY* dy, const TX* x, const float* __restrict__ gamma, const float2* __restrict__ stats,
                       const TX* dres, TX* dx, float* __restrict__ partial, int T, int H) {
    using R = Row<W, N, WPR>;
    constexpr int GROUPS = THREADS / R::G;
    extern __shared__ __align__(16) float acc[];   // GROUPS > 1: [GROUPS][H]
    pdl_wait();
    pdl_trigger();
    __shared__ float2 red[2][WARPS];
    const int lg = threadIdx.x % R::G, grp = threadIdx.x / R::G;
    const float inv_h = 1.0f / (float)H;
    float dg[R::N];
#pragma unroll
    for (int k = 0; k < R::N; ++k) dg[k] = 0.f;
    int par = 0;
    for (int t0 = blockIdx.x * GROUPS; t0 < T; t0 += gridDim.x * GROUPS, par ^= 1) {
        const int t = t0 + grp;
        if (WPR == 1 && t >= T) break;
        const size_t base = (size_t)t * H;   // WPR > 1: GROUPS rows exist whenever a block enters the loop with one
        const bool live = t < T;
        float xh[R::N], d[R::N], g[R::N];
        if (live) {
            R::load(x + base, H, lg, xh);
            R::load(dy + base, H, lg, d);
        } else {
#pragma unroll
            for (int k = 0; k < R::N; ++k) xh[k] = d[k] = 0.f;
        }
        const float2 st = live ? stats[t] : make_float2(0.f, 0.f);
        R::load(gamma, H, lg, g);
        float su = 0.f, sux = 0.f;
#pragma unroll
        for (int k = 0; k < R::N; ++k) {
            xh[k] = (xh[k] - st.x) * st.y;
            if (R::has(k, lg, H)) dg[k] += d[k] * xh[k];   // a column past H has xh = -mean rstd, d = 0
            d[k] *= g[k];
            su += d[k];
            sux += d[k] * xh[k];
        }
        const float2 sums = group_sum<WPR>(su, sux, red[par]);
        if (!live) continue;
        const float mu = sums.x * inv_h, mux = sums.y * inv_h;
#pragma unroll
        for (int k = 0; k < R::N; ++k) d[k] = st.y * (d[k] - mu - xh[k] * mux);
        if (dres) {
            R::load(dres + base, H, lg, xh);
#pragma unroll
            for (int k = 0; k < R::N; ++k) d[k] += xh[k];
        }
        R::store(dx + base, H, lg, d);
    }
    float* out = partial + (size_t)blockIdx.x * H;
    if constexpr (GROUPS == 1) {
        R::store(out, H, lg, dg);
    } else {
        R::store(acc + (size_t)grp * H, H, lg, dg);
        __syncthreads();
        for (int h = threadIdx.x; h < H; h += THREADS) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < GROUPS; ++w) s += acc[(size_t)w * H + h];
            out[h] = s;
        }
    }
}

// dgamma[h] = sum over the blocks' partials: eight columns per block, 64 slices of
// the partials, added slice by slice.  Latency alone: about 4 us for 304 partials of
// 768 columns, with 24 blocks of 32 columns as with these 96.
constexpr int DG_COLS = 8, DG_SLICES = 64;
__global__ void __launch_bounds__(DG_COLS* DG_SLICES) ln_dgamma_kernel(const float* __restrict__ partial, int n, int H,
                                                                       float* __restrict__ dgamma) {
    __shared__ float red[DG_SLICES][DG_COLS];
    pdl_wait();
    pdl_trigger();
    const int cx = threadIdx.x % DG_COLS, sl = threadIdx.x / DG_COLS;
    const int h = blockIdx.x * DG_COLS + cx;
    float s = 0.f;
    if (h < H) {
#pragma unroll 5
        for (int i = sl; i < n; i += DG_SLICES) s += partial[(size_t)i * H + h];
    }
    red[sl][cx] = s;
    __syncthreads();
    // warp w: column w, two slices per lane
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (w >= DG_COLS) return;
    const float v = warp_sum_f32(red[lane][w] + red[lane + 32][w]);
    if (lane == 0 && blockIdx.x * DG_COLS + w < H) dgamma[blockIdx.x * DG_COLS + w] = v;
}

// Warps per row in the backward pass; the layouts below are the ones that go with it.
int backward_warps(int H) {
    if (H % 2) return H <= 256 ? 1 : H <= 512 ? 2 : H <= 1024 ? 4 : 8;
    if (H <= 512) return 1;
    if (H % 4 == 0) {
        if (H <= 768) return 1;
        if (H <= 1536) return 2;
    }
    return H <= 1024 ? 2 : H <= 2048 ? 4 : 8;
}

// Calls f.template operator()<W, N, WPR>() with the row layout for H.  Forward holds
// less per element and does better with few warps a row (2048 columns, fp32 to bf16:
// 47.4 us with two, 48.0 with four); single elements want fewer a lane here too
// (1001 columns bf16: 71 us with 16 a lane, 101 with 32, 75 with 8).
template <int W, typename F>
cudaError_t with_width(int H, const F& f) {
    if (H <= 256) return f.template operator()<W, 8, 1>();
    if constexpr (W == 1) {
        if constexpr (F::BACKWARD) {
            if (H <= 512) return f.template operator()<W, 8, 2>();
            if (H <= 1024) return f.template operator()<W, 8, 4>();
            if (H <= 2048) return f.template operator()<W, 8, 8>();
        }
    }
    if constexpr (!F::BACKWARD || W > 1) {
        if (H <= 512) return f.template operator()<W, 16, 1>();
    }
    if constexpr (W >= 4) {
        if (H <= 768) return f.template operator()<W, 24, 1>();
    }
    constexpr bool SIXTEEN = F::BACKWARD || W == 1;
    if constexpr (!(F::BACKWARD && W == 1)) {
        if (H <= 1024) return f.template operator()<W, SIXTEEN ? 16 : 32, SIXTEEN ? 2 : 1>();
        if constexpr (W >= 4) {
            if (H <= 1536) return f.template operator()<W, 24, 2>();
        }
        if (H <= 2048) return f.template operator()<W, SIXTEEN ? 16 : 32, SIXTEEN ? 4 : 2>();
    }
    if (H <= 4096) return f.template operator()<W, SIXTEEN ? 16 : 32, SIXTEEN ? 8 : 4>();
    return f.template operator()<W, 32, 8>();
}
// V: widest vector for the types.
template <int V, typename F>
cudaError_t with_layout(int H, const F& f) {
    if (H % V == 0) return with_width<V>(H, f);
    if constexpr (V == 8) {
        if (H % 4 == 0) return with_width<4>(H, f);
    }
    return H % 2 == 0 ? with_width<2>(H, f) : with_width<1>(H, f);
}

template <typename TX, typename TY>
struct Forward {
    static constexpr bool BACKWARD = false;
    const void* x;
    const float* gamma;
    void* y;
    float* stats;
    int T, H;
    float eps;
    cudaStream_t s;
    template <int W, int N, int WPR>
    cudaError_t operator()() const {
        const int rows = WARPS / WPR;
        return launch_pdl(ln_forward_kernel<TX, TY, W, N, WPR>, dim3((T - 1) / rows + 1), dim3(THREADS), 0, s,
                          (const TX*)x, gamma, (TY*)y, reinterpret_cast<float2*>(stats), T, H, eps);
    }
};

template <typename TX, typename TY>
struct Backward {
    static constexpr bool BACKWARD = true;
    const void *dy, *x;
    const float *gamma, *stats;
    const void* dres;
    void* dx;
    float *dgamma, *partial;
    int T, H, num_sms;
    cudaStream_t s;
    template <int W, int N, int WPR>
    cudaError_t operator()() const {
        constexpr int GROUPS = WARPS / WPR;
        if (WPR != backward_warps(H)) return cudaErrorInvalidValue;   // the workspace is sized by it
        const int grid = min(min((T - 1) / GROUPS + 1, bwd_blocks<W, N>() * num_sms), BWD_MAX_GRID);
        const size_t smem = GROUPS > 1 ? (size_t)GROUPS * H * sizeof(float) : 0;   // at most 32 KB
        cudaError_t e = launch_pdl(ln_backward_kernel<TX, TY, W, N, WPR>, dim3(grid), dim3(THREADS), smem, s,
                                   (const TY*)dy, (const TX*)x, gamma, reinterpret_cast<const float2*>(stats),
                                   (const TX*)dres, (TX*)dx, partial, T, H);
        if (e != cudaSuccess) return e;
        return launch_pdl(ln_dgamma_kernel, dim3((H + DG_COLS - 1) / DG_COLS), dim3(DG_COLS * DG_SLICES), 0, s,
                          (const float*)partial, grid, H, dgamma);
    }
};

}  // namespace

size_t layernorm_backward_ws(int T, int H) {
    const int groups = WARPS / backward_warps(H);
    const int grid = T < 1 ? 0 : min((T - 1) / groups + 1, BWD_MAX_GRID);
    WsCarve ws(nullptr);
    ws.take<float>((size_t)grid * H);
    return ws.off;
}

cudaError_t launch_layernorm_forward(const void* x, bool x_bf16, const float* gamma, void* y, bool y_bf16, float* stats,
                                     int T, int H, float eps, cudaStream_t s) {
    if (T == 0) return cudaSuccess;
    if (x_bf16)
        return y_bf16 ? with_layout<8>(H, Forward<bf16, bf16>{x, gamma, y, stats, T, H, eps, s})
                      : with_layout<4>(H, Forward<bf16, float>{x, gamma, y, stats, T, H, eps, s});
    return y_bf16 ? with_layout<4>(H, Forward<float, bf16>{x, gamma, y, stats, T, H, eps, s})
                  : with_layout<4>(H, Forward<float, float>{x, gamma, y, stats, T, H, eps, s});
}

cudaError_t launch_layernorm_backward(const void* dy, bool y_bf16, const void* x, bool x_bf16, const float* gamma,
                                      const float* stats, const void* dres, void* dx, float* dgamma, int T, int H,
                                      void* ws, cudaStream_t s) {
    if (T == 0) return cudaMemsetAsync(dgamma, 0, (size_t)H * sizeof(float), s);
    int dev = 0, num_sms = 0;
    cudaError_t e = tee_current_device(&dev, &num_sms);
    if (e != cudaSuccess) return e;
    float* partial = (float*)ws;
    if (x_bf16)
        return y_bf16 ? with_layout<8>(H, Backward<bf16, bf16>{dy, x, gamma, stats, dres, dx, dgamma, partial, T, H, num_sms, s})
                      : with_layout<4>(H, Backward<bf16, float>{dy, x, gamma, stats, dres, dx, dgamma, partial, T, H, num_sms, s});
    return y_bf16 ? with_layout<4>(H, Backward<float, bf16>{dy, x, gamma, stats, dres, dx, dgamma, partial, T, H, num_sms, s})
                  : with_layout<4>(H, Backward<float, float>{dy, x, gamma, stats, dres, dx, dgamma, partial, T, H, num_sms, s});
}
