// Token lookup with scaling, and the table's gradient from sorted tokens
// (tee_train.h has the formulas).
//
// The gradient dE[v] = scale sum_{t: id[t] = v} dy[t] is bound by HBM: dy is
// read once and the whole table written once (most rows with zeros).  Three
// launches, all without atomics on values:
//   embed_sort_fill_kernel  one cluster of eight CTAs sorts (id, t) stably by id
//     (radix sort, at most nine bits a pass, counters in shared memory, column
//     totals exchanged through distributed shared memory); meanwhile the other
//     CTAs zero the table rows that no token has.
//   embed_sum_kernel  each warp adds the rows of 32 consecutive sorted tokens
//     for 256 columns; runs of one id inside a block of 256 tokens are joined in
//     shared memory and written, the pieces of runs that cross blocks are kept.
//   embed_join_kernel  adds the pieces of each run that crosses blocks, in order.
#include "train_internal.cuh"

#include <mutex>

#include "tc_ptx.cuh"

namespace {

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// y[t] = scale E[id[t]]; 2^lane_bits lanes per token.
template <typename TE, typename TY, bool VEC>
__global__ void __launch_bounds__(256) embed_forward_kernel(const TE* __restrict__ table, const int32_t* __restrict__ ids,
                                                            TY* __restrict__ y, int T, int V, int H, float scale,
                                                            int lane_bits, unsigned int* status) {
    pdl_wait();
    pdl_trigger();
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long t = i >> lane_bits;
    const int lane = (int)(i & ((1 << lane_bits) - 1)), step = 1 << lane_bits;
    if (t >= T) return;
    const int id = ids[t];
    const bool ok = id >= 0 && id < V;
    if (!ok && lane == 0) atomicOr(status, TEE_STATUS_BAD_ID);
    const TE* src = table + (size_t)(ok ? id : 0) * H;
    TY* dst = y + (size_t)t * H;
    if constexpr (VEC) {
#pragma unroll 4
        for (int c = lane; c < H / 8; c += step) {
            float v[8];
            load8(src + 8 * c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = ok ? v[j] * scale : 0.f;
            store8(dst + 8 * c, v);
        }
    } else {
#pragma unroll 4
        for (int c = lane; c < H; c += step) f32_to_elem(ok ? elem_to_f32(src[c]) * scale : 0.f, dst[c]);
    }
}

// ---------------------------------------------------------------------------
// backward: sort
// ---------------------------------------------------------------------------

constexpr int SORT_CTAS = 8, SORT_THREADS = 1024, SORT_WARPS = SORT_THREADS / 32;
constexpr int MAX_DIGIT_BITS = 9, MAX_BINS = 1 << MAX_DIGIT_BITS;
constexpr int TOKENS_PER_WARP = 32, SUM_WARPS = 8, TOKENS_PER_BLOCK = TOKENS_PER_WARP * SUM_WARPS;
constexpr int COLS = 256;   // columns per block of embed_sum_kernel: eight per lane
constexpr int FILL_WORDS = SORT_WARPS * MAX_BINS;   // the fill CTAs' row flags take the sort's counters

struct SortSmem {
    uint32_t hist[SORT_WARPS][MAX_BINS];   // per warp: its keys per digit, then where its next such key goes
    uint32_t total[MAX_BINS];              // this CTA's keys per digit, read by the whole cluster
    uint32_t scan[SORT_WARPS];
};
static_assert(sizeof(SortSmem) <= 80 * 1024, "shared memory");

// A sorted token: key = its id (V where the id is out of range), and its place in the batch.
typedef uint2 Pair;

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// One stable pass over digit `shift` .. `shift + bits` by the cluster's 256
// warps, each with `slice` consecutive keys.
template <bool FIRST>
__device__ void sort_pass(SortSmem& sm, const int32_t* __restrict__ ids, const Pair* in, Pair* out, int T, int V,
                          int slice, int shift, int bits, uint32_t rank, unsigned int* status) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bins = 1 << bits;
    const uint32_t mask = bins - 1;
    const long long first = (long long)(rank * SORT_WARPS + warp) * slice;
    const int lo = (int)min((long long)T, first), hi = (int)min((long long)T, first + slice);
    auto fetch = [&](int p) {
        if constexpr (FIRST) {
            const int id = ids[p];
            return make_uint2(id >= 0 && id < V ? (uint32_t)id : (uint32_t)V, (uint32_t)p);
        } else {
            return __ldcg(in + p);
        }
    };
    for (int b = lane; b < bins; b += 32) sm.hist[warp][b] = 0;
    __syncwarp();
#pragma unroll 4
    for (int p = lo + lane; p < hi; p += 32) {
        const uint32_t key = fetch(p).x;
        if (FIRST && key == (uint32_t)V) atomicOr(status, TEE_STATUS_BAD_ID);
        atomicAdd(&sm.hist[warp][(key >> shift) & mask], 1u);
    }
    __syncthreads();
    // per digit: turn the warps' counts into offsets within this CTA
    if (threadIdx.x < bins) {
        uint32_t run = 0;
#pragma unroll 8
        for (int w = 0; w < SORT_WARPS; ++w) {
            const uint32_t c = sm.hist[w][threadIdx.x];
            sm.hist[w][threadIdx.x] = run;
            run += c;
        }
        sm.total[threadIdx.x] = run;
    }
    tc::cluster_sync();
    // before the digit's keys of this CTA come all keys of smaller digits, and
    // this digit's keys in the CTAs before
    uint32_t all = 0, before = 0;
    if (threadIdx.x < bins) {
        const uint32_t mine = tc::smem_u32(&sm.total[threadIdx.x]);
#pragma unroll
        for (uint32_t r = 0; r < SORT_CTAS; ++r) {
            const uint32_t c = ld_cluster(tc::mapa_shared(mine, r));
            all += c;
            before += r < rank ? c : 0;
        }
    }
    uint32_t inc = all;   // inclusive scan over the digits
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) sm.scan[warp] = inc;
    __syncthreads();
    uint32_t base = inc - all + before;
    for (int w = 0; w < warp; ++w) base += sm.scan[w];
    if (threadIdx.x < bins) {
#pragma unroll 8
        for (int w = 0; w < SORT_WARPS; ++w) sm.hist[w][threadIdx.x] += base;
    }
    __syncthreads();
    for (int p0 = lo; p0 < hi; p0 += 32) {
        const int p = p0 + lane;
        const unsigned live = __ballot_sync(0xffffffffu, p < hi);
        if (p < hi) {
            const Pair kv = fetch(p);
            const uint32_t d = (kv.x >> shift) & mask;
            const unsigned peers = __match_any_sync(live, d);
            const uint32_t at = sm.hist[warp][d];
            __syncwarp(live);
            if (lane == 31 - __clz(peers)) sm.hist[warp][d] = at + __popc(peers);
            __syncwarp(live);
            const uint32_t to = at + __popc(peers & ((1u << lane) - 1));
            if (to < (uint32_t)T) out[to] = kv;   // always, unless another call writes to this workspace
        }
        __syncwarp();
    }
    // the next pass reads the other CTAs' keys and rewrites the totals
    tc::cluster_sync();
}

template <typename TG>
__global__ void __cluster_dims__(SORT_CTAS, 1, 1) __launch_bounds__(SORT_THREADS)
    embed_sort_fill_kernel(const int32_t* __restrict__ ids, int T, int V, int H, int key_bits, Pair* buf0, Pair* buf1,
                           TG* __restrict__ grad, unsigned int* status) {
    extern __shared__ __align__(16) uint8_t raw[];
    SortSmem& sm = *reinterpret_cast<SortSmem*>(raw);
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x < SORT_CTAS) {
        const uint32_t rank = tc::cluster_ctarank();
        const int slice = (int)(((long long)T + SORT_CTAS * SORT_WARPS * 32 - 1) / (SORT_CTAS * SORT_WARPS * 32)) * 32;
        const int passes = (key_bits + MAX_DIGIT_BITS - 1) / MAX_DIGIT_BITS;
        const int width = (key_bits + passes - 1) / passes;
        for (int p = 0; p < passes; ++p) {
            Pair* out = (p & 1) ? buf1 : buf0;
            if (p == 0) sort_pass<true>(sm, ids, nullptr, out, T, V, slice, 0, width, rank, status);
            else sort_pass<false>(sm, ids, (p & 1) ? buf0 : buf1, out, T, V, slice, p * width, width, rank, status);
        }
        return;
    }
    // fill: this CTA's share of the rows, in windows of as many flags as fit
    uint32_t* flags = reinterpret_cast<uint32_t*>(raw);
    const int fillers = gridDim.x - SORT_CTAS, me = blockIdx.x - SORT_CTAS;
    const int v_lo = (int)((long long)V * me / fillers), v_hi = (int)((long long)V * (me + 1) / fillers);
    const bool vec = ((size_t)H * sizeof(TG)) % 16 == 0;
    for (int w_lo = v_lo; w_lo < v_hi; w_lo += min(v_hi - w_lo, FILL_WORDS * 32)) {
        const int rows = min(v_hi - w_lo, FILL_WORDS * 32);
        for (int i = threadIdx.x; i < (rows + 31) / 32; i += SORT_THREADS) flags[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int t = threadIdx.x; t < T; t += SORT_THREADS) {
            const uint32_t r = (uint32_t)ids[t] - (uint32_t)w_lo;
            if (r < (uint32_t)rows) atomicOr(&flags[r >> 5], 1u << (r & 31));
        }
        __syncthreads();
        for (int r = warp; r < rows; r += SORT_WARPS) {
            if (flags[r >> 5] >> (r & 31) & 1u) continue;
            TG* row = grad + (size_t)(w_lo + r) * H;
            if (vec) {
                const int n = (int)((size_t)H * sizeof(TG) / 16);
                for (int c = lane; c < n; c += 32) reinterpret_cast<uint4*>(row)[c] = make_uint4(0, 0, 0, 0);
            } else {
                for (int c = lane; c < H; c += 32) f32_to_elem(0.f, row[c]);
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// backward: sums over runs of one id
// ---------------------------------------------------------------------------

// What a block of 256 sorted tokens leaves for embed_join_kernel.
//   head: the piece of a run that began in an earlier block: HEAD_NONE, HEAD_ENDS
//     (the run ends here) or HEAD_THROUGH (it fills the block and goes on).
//   tail_key: the id of a run that begins here and goes on, or NO_KEY.
constexpr int HEAD_NONE = 0, HEAD_ENDS = 1, HEAD_THROUGH = 2;
constexpr uint32_t NO_KEY = 0xffffffffu;
struct BlockState {
    int head;
    uint32_t tail_key;
};

template <typename TG>
__device__ __forceinline__ void put(TG* grad, size_t at, float sum, float scale, bool accumulate) {
    float v = sum * scale;
    if (accumulate) v += elem_to_f32(grad[at]);
    f32_to_elem(v, grad[at]);
}

template <typename TY, typename TG, bool VEC>
__global__ void __launch_bounds__(SUM_WARPS * 32)
    embed_sum_kernel(const TY* __restrict__ dy, const Pair* __restrict__ sorted, TG* __restrict__ grad, int T, int V, int H,
                     float scale, int accumulate, BlockState* __restrict__ state, float* __restrict__ head,
                     float* __restrict__ tail) {
    // a warp's piece of the run that reaches into it from the left (L), and of the one that leaves it to the right (R)
    __shared__ float piece[2][SUM_WARPS][COLS];
    __shared__ uint32_t key_l[SUM_WARPS], key_r[SUM_WARPS];   // NO_KEY: no such piece
    __shared__ int through[SUM_WARPS];                        // L leaves the warp to the right as well
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col0 = blockIdx.y * COLS;
    const long long first = (long long)blockIdx.x * TOKENS_PER_BLOCK + warp * TOKENS_PER_WARP;
    const int n = (int)max(0LL, min((long long)TOKENS_PER_WARP, T - first));
    auto col = [&](int j) { return VEC ? lane * 8 + j : j * 32 + lane; };   // within the block's columns
    if (lane == 0) key_l[warp] = key_r[warp] = NO_KEY, through[warp] = 0;
    if (n > 0) {
        Pair kv = make_uint2(NO_KEY, 0);
        if (lane < n) kv = sorted[first + lane];
        const uint32_t before = first > 0 ? sorted[first - 1].x : NO_KEY;
        const uint32_t after = first + n < T ? sorted[first + n].x : NO_KEY;
        float acc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
        uint32_t cur = __shfl_sync(0xffffffffu, kv.x, 0);
        bool open_left = cur == before;
        auto keep = [&](int side) {
#pragma unroll
            for (int j = 0; j < 8; ++j) piece[side][warp][col(j)] = acc[j];
        };
        auto write = [&]() {   // a run that lies within this warp
            if (cur >= (uint32_t)V) return;
            TG* row = grad + (size_t)cur * H + col0;
            if constexpr (VEC) {
                if (col0 + lane * 8 < H) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = acc[j] * scale;
                    if (accumulate) {
                        float o[8];
                        load8(row + lane * 8, o);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += o[j];
                    }
                    store8(row + lane * 8, v);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col0 + col(j) < H) put(row, col(j), acc[j], scale, accumulate);
            }
        };
        constexpr int BATCH = 8;
        for (int i0 = 0; i0 < n; i0 += BATCH) {
            float v[BATCH][8];
#pragma unroll
            for (int q = 0; q < BATCH; ++q) {
                const uint32_t k = __shfl_sync(0xffffffffu, kv.x, i0 + q), t = __shfl_sync(0xffffffffu, kv.y, i0 + q);
                const TY* row = dy + (size_t)t * H + col0;
                const bool ok = k < (uint32_t)V && t < (uint32_t)T;   // false past the end as well (NO_KEY)
                if constexpr (VEC) {
                    if (ok && col0 + lane * 8 < H) load8(row + lane * 8, v[q]);
                    else
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[q][j] = 0.f;
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[q][j] = ok && col0 + col(j) < H ? elem_to_f32(row[col(j)]) : 0.f;
                }
            }
#pragma unroll
            for (int q = 0; q < BATCH; ++q) {
                const uint32_t k = __shfl_sync(0xffffffffu, kv.x, i0 + q);
                if (i0 + q < n) {
                    if (k != cur) {
                        if (open_left) {
                            keep(0);
                            if (lane == 0) key_l[warp] = cur;
                            open_left = false;
                        } else {
                            write();
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
                        cur = k;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[j] += v[q][j];
                }
            }
        }
        const bool open_right = cur == after;
        if (open_left) {
            keep(0);
            if (lane == 0) key_l[warp] = cur, through[warp] = open_right;
        } else if (open_right) {
            keep(1);
            if (lane == 0) key_r[warp] = cur;
        } else {
            write();
        }
    }
    __syncthreads();
    // join the warps' pieces, one column per thread
    const int c = threadIdx.x;
    const bool in = col0 + c < H;
    float acc = 0.f;
    int open = 0;   // 1: a run from an earlier block, 2: one that began in this block
    int head_state = HEAD_NONE;
    uint32_t open_key = NO_KEY;
    for (int w = 0; w < SUM_WARPS; ++w) {
        if (key_l[w] != NO_KEY) {
            if (open == 0) open = 1;
            acc += piece[0][w][c];
            if (!through[w]) {
                if (open == 1) {
                    head_state = HEAD_ENDS;
                    if (in) head[(size_t)blockIdx.x * H + col0 + c] = acc;
                } else if (in && key_l[w] < (uint32_t)V) {
                    put(grad, (size_t)key_l[w] * H + col0 + c, acc, scale, accumulate);
                }
                open = 0;
                acc = 0.f;
            }
        }
        if (key_r[w] != NO_KEY) {
            open = 2;
            open_key = key_r[w];
            acc = piece[1][w][c];
        }
    }
    if (open == 1) {
        head_state = HEAD_THROUGH;
        if (in) head[(size_t)blockIdx.x * H + col0 + c] = acc;
    } else if (open == 2) {
        if (in) tail[(size_t)blockIdx.x * H + col0 + c] = acc;
    }
    if (blockIdx.y == 0 && c == 0) state[blockIdx.x] = BlockState{head_state, open == 2 ? open_key : NO_KEY};
}

// Block b adds the run that begins in block b of embed_sum_kernel and crosses
// its end: tail of b, then the heads of b + 1 .. the block where the run ends.
// Four slices of the heads, 256 columns.
template <typename TG>
__global__ void __launch_bounds__(1024)
    embed_join_kernel(const BlockState* __restrict__ state, int n_blocks, const float* __restrict__ head,
                      const float* __restrict__ tail, TG* __restrict__ grad, int V, int H, float scale, int accumulate) {
    __shared__ float red[3][COLS];
    __shared__ int end_s;
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.x;
    const uint32_t key = state[b].tail_key;
    if (key >= (uint32_t)V) return;   // NO_KEY, or the run of out-of-range ids
    if (threadIdx.x == 0) end_s = INT32_MAX;
    __syncthreads();
    // the first block after b whose head ends the run
    for (int e0 = b + 1; e0 < n_blocks; e0 += 1024) {
        const int e = e0 + threadIdx.x;
        if (e < n_blocks && state[e].head == HEAD_ENDS) atomicMin(&end_s, e);
        __syncthreads();
        const bool found = end_s != INT32_MAX;
        __syncthreads();
        if (found) break;
    }
    const int end = min(end_s, n_blocks - 1);
    const int c = threadIdx.x & (COLS - 1), sl = threadIdx.x / COLS;
    const int h = blockIdx.y * COLS + c;
    float s = 0.f;
    if (h < H) {
#pragma unroll 4
        for (int e = b + 1 + sl; e <= end; e += 4) s += head[(size_t)e * H + h];
    }
    if (sl) red[sl - 1][c] = s;
    __syncthreads();
    if (sl == 0 && h < H) put(grad, (size_t)key * H + h, (tail[(size_t)b * H + h] + s) + (red[0][c] + (red[1][c] + red[2][c])), scale, accumulate);
}

struct EmbedWs {
    Pair *buf0, *buf1;
    BlockState* state;
    float *head, *tail;
    size_t bytes;
};
EmbedWs carve_embed(int T, int H, void* base) {
    WsCarve ws(base);
    EmbedWs w;
    const size_t nb = ((size_t)T + TOKENS_PER_BLOCK - 1) / TOKENS_PER_BLOCK;
    w.buf0 = ws.take<Pair>(T);
    w.buf1 = ws.take<Pair>(T);
    w.state = ws.take<BlockState>(nb);
    w.head = ws.take<float>(nb * H);
    w.tail = ws.take<float>(nb * H);
    w.bytes = ws.off;
    return w;
}

template <typename TY, typename TG>
cudaError_t backward_t(const void* dy_, const int32_t* ids, void* grad_, int T, int V, int H, float scale, bool accumulate,
                       const EmbedWs& w, unsigned int* status, int dev, int num_sms, cudaStream_t s) {
    const TY* dy = (const TY*)dy_;
    TG* grad = (TG*)grad_;
    cudaError_t e;
    {
        static std::mutex mu;
        static bool ready[TEE_MAX_DEVICES] = {};
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[dev]) {
            e = cudaFuncSetAttribute(embed_sort_fill_kernel<TG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)sizeof(SortSmem));
            if (e != cudaSuccess) return e;
            ready[dev] = true;
        }
    }
    int key_bits = 1;
    while (key_bits < 32 && (V >> key_bits)) ++key_bits;   // keys 0 .. V
    const int passes = (key_bits + MAX_DIGIT_BITS - 1) / MAX_DIGIT_BITS;
    const int fillers = accumulate ? 0 : max(1, num_sms / SORT_CTAS - 1) * SORT_CTAS;
    if ((e = launch_pdl(embed_sort_fill_kernel<TG>, dim3(SORT_CTAS + fillers), dim3(SORT_THREADS), sizeof(SortSmem), s,
                        ids, T, V, H, key_bits, w.buf0, w.buf1, grad, status)))
        return e;
    const Pair* sorted = passes & 1 ? w.buf0 : w.buf1;
    const int nb = (T - 1) / TOKENS_PER_BLOCK + 1;
    const dim3 grid(nb, (H + COLS - 1) / COLS);
    if (H % 8 == 0)
        e = launch_pdl(embed_sum_kernel<TY, TG, true>, grid, dim3(SUM_WARPS * 32), 0, s, dy, sorted, grad, T, V, H, scale,
                       (int)accumulate, w.state, w.head, w.tail);
    else
        e = launch_pdl(embed_sum_kernel<TY, TG, false>, grid, dim3(SUM_WARPS * 32), 0, s, dy, sorted, grad, T, V, H, scale,
                       (int)accumulate, w.state, w.head, w.tail);
    if (e != cudaSuccess || nb == 1) return e;   // one block: no run crosses blocks
    return launch_pdl(embed_join_kernel<TG>, grid, dim3(1024), 0, s, (const BlockState*)w.state, nb, (const float*)w.head,
                      (const float*)w.tail, grad, V, H, scale, (int)accumulate);
}

template <typename TE, typename TY>
cudaError_t forward_t(const void* table, const int32_t* ids, void* y, int T, int V, int H, float scale,
                      unsigned int* status, cudaStream_t s) {
    const bool vec = H % 8 == 0;
    const int work = vec ? H / 8 : H;
    int lane_bits = 0;
    while (lane_bits < 5 && (1 << lane_bits) < work) ++lane_bits;
    const dim3 grid((unsigned)((((long long)T << lane_bits) + 255) / 256));
    if (vec)
        return launch_pdl(embed_forward_kernel<TE, TY, true>, grid, dim3(256), 0, s, (const TE*)table, ids, (TY*)y, T, V, H,
                          scale, lane_bits, status);
    return launch_pdl(embed_forward_kernel<TE, TY, false>, grid, dim3(256), 0, s, (const TE*)table, ids, (TY*)y, T, V, H,
                      scale, lane_bits, status);
}

}  // namespace

size_t embed_backward_ws(int T, int V, int H) {
    (void)V;
    return carve_embed(T, H, nullptr).bytes;
}

cudaError_t launch_embed_forward(const void* table, bool e_bf16, const int32_t* ids, void* y, bool y_bf16, int T, int V,
                                 int H, float scale, unsigned int* status, cudaStream_t s) {
    if (T == 0) return cudaSuccess;
    if (e_bf16)
        return y_bf16 ? forward_t<bf16, bf16>(table, ids, y, T, V, H, scale, status, s)
                      : forward_t<bf16, float>(table, ids, y, T, V, H, scale, status, s);
    return y_bf16 ? forward_t<float, bf16>(table, ids, y, T, V, H, scale, status, s)
                  : forward_t<float, float>(table, ids, y, T, V, H, scale, status, s);
}

cudaError_t launch_embed_backward(const void* dy, bool y_bf16, const int32_t* ids, void* dtable, bool e_bf16, int T,
                                  int V, int H, float scale, bool accumulate, void* ws, unsigned int* status,
                                  cudaStream_t s) {
    if (T == 0)
        return accumulate ? cudaSuccess : cudaMemsetAsync(dtable, 0, (size_t)V * H * (e_bf16 ? 2 : 4), s);
    int dev = 0, num_sms = 0;
    cudaError_t e = tee_current_device(&dev, &num_sms);
    if (e != cudaSuccess) return e;
    const EmbedWs w = carve_embed(T, H, ws);
    if (e_bf16)
        return y_bf16 ? backward_t<bf16, bf16>(dy, ids, dtable, T, V, H, scale, accumulate, w, status, dev, num_sms, s)
                      : backward_t<float, bf16>(dy, ids, dtable, T, V, H, scale, accumulate, w, status, dev, num_sms, s);
    return y_bf16 ? backward_t<bf16, float>(dy, ids, dtable, T, V, H, scale, accumulate, w, status, dev, num_sms, s)
                  : backward_t<float, float>(dy, ids, dtable, T, V, H, scale, accumulate, w, status, dev, num_sms, s);
}
