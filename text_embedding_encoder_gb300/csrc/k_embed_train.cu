// Token lookup with scaling, and the table's gradient from sorted tokens
// (tee_train.h has the formulas).
//
// The gradient dE[v] = scale sum_{t: id[t] = v} dy[t] is bound by HBM: dy is
// read once and the whole table written once (most rows with zeros).  Three
// launches, all without atomics on values:
//   embed_sort_kernel  one cluster of sixteen CTAs sorts (id, t) stably by id
//     (radix sort, at most nine bits a pass, counters in shared memory, column
//     totals exchanged through distributed shared memory); meanwhile the other
//     CTAs zero the first rows of the table, as many as the sort has time for.
//     Few tokens are sorted by counting instead (embed_rank_kernel).
//   embed_sum_kernel  each warp adds the rows of 8 or 32 consecutive sorted tokens
//     for 256 columns; runs of one id inside a block's tokens are joined in shared
//     memory and written, the pieces of runs that cross blocks are kept.  Blocks
//     behind these zero the rest of the rows that no token has.
//   embed_join_kernel  adds the pieces of each run that crosses blocks, in order.
// Measured, 102400 x 768: 2048 tokens into a bf16 table 29.7 us (157 MB of zeros
// alone take 24); 65536 tokens, 30 % of them one id, into an fp32 table 98.5 us
// (the launches one by one, caches flushed before each: sort 22, sums and zeros 70 at
// 5.8 TB/s of DRAM traffic -- a gather of the same rows by themselves runs at 5.1 --
// join 9).  The lookup forward, 32768 tokens of
// which few ids are new, bf16 -> fp32: 19.5 us, the write of its output.
#include "train_internal.cuh"

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "tc_ptx.cuh"

namespace {

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// y[t] = scale E[id[t]]; 2^lane_bits lanes per token.  (Four tokens a group, for
// more reads in flight, measured slower: 29.5 against 25.8 us at 32768 x 768.)
template <typename TE, typename TY, int W>
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
    if constexpr (W > 1) {
#pragma unroll 6
        for (int c = lane; c < H / W; c += step) {
            float v[W];
            load_vec(src + W * c, v);
#pragma unroll
            for (int j = 0; j < W; ++j) v[j] = ok ? v[j] * scale : 0.f;
            store_vec(dst + W * c, v);
        }
    } else {
#pragma unroll 4
        for (int c = lane; c < H; c += step) f32_to_elem(ok ? elem_to_f32(src[c]) * scale : 0.f, dst[c]);
    }
}

// ---------------------------------------------------------------------------
// backward: sort
// ---------------------------------------------------------------------------

constexpr int SORT_CTAS = 16, SORT_THREADS = 1024, SORT_WARPS = SORT_THREADS / 32;
constexpr int MAX_DIGIT_BITS = 9, MAX_BINS = 1 << MAX_DIGIT_BITS;
constexpr int SUM_WARPS = 8;
constexpr int COLS = 256;   // columns per block of embed_sum_kernel: eight per lane

struct SortSmem {
    uint32_t hist[SORT_WARPS][MAX_BINS];   // per warp: its keys per digit, then where its next such key goes
    uint32_t total[MAX_BINS];              // this CTA's keys per digit, read by the whole cluster
    uint32_t scan[SORT_WARPS];
};
static_assert(sizeof(SortSmem) <= 80 * 1024, "shared memory");

constexpr uint32_t NO_KEY = 0xffffffffu;

// A sorted token: key = its id (V where the id is out of range), and its place in the batch.
typedef uint2 Pair;

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

constexpr int GROUP = 8;

// One stable pass over digit `shift` .. `shift + bits` by the cluster's 512
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
    // eight keys per lane in flight at a time, here and below
    for (int p0 = lo; p0 < hi; p0 += 32 * GROUP) {
        uint32_t key[GROUP];
#pragma unroll
        for (int q = 0; q < GROUP; ++q) {
            const int p = p0 + 32 * q + lane;
            key[q] = p < hi ? fetch(p).x : 0xffffffffu;
        }
#pragma unroll
        for (int q = 0; q < GROUP; ++q) {
            if (p0 + 32 * q + lane < hi) {
                if (FIRST && key[q] == (uint32_t)V) atomicOr(status, TEE_STATUS_BAD_ID);
                atomicAdd(&sm.hist[warp][(key[q] >> shift) & mask], 1u);
            }
        }
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
    const uint32_t others = __reduce_add_sync(0xffffffffu, lane < warp ? sm.scan[lane] : 0u);
    const uint32_t base = inc - all + before + others;
    if (threadIdx.x < bins) {
#pragma unroll 8
        for (int w = 0; w < SORT_WARPS; ++w) sm.hist[w][threadIdx.x] += base;
    }
    __syncthreads();
    for (int p0 = lo; p0 < hi; p0 += 32 * GROUP) {
        Pair kv[GROUP];
#pragma unroll
        for (int q = 0; q < GROUP; ++q) {
            const int p = p0 + 32 * q + lane;
            kv[q] = p < hi ? fetch(p) : make_uint2(0, 0);
        }
#pragma unroll
        for (int q = 0; q < GROUP; ++q) {
            const int p = p0 + 32 * q + lane;
            const unsigned live = __ballot_sync(0xffffffffu, p < hi);
            if (p < hi) {
                const uint32_t d = (kv[q].x >> shift) & mask;
                const unsigned peers = __match_any_sync(live, d);
                const uint32_t at = sm.hist[warp][d];
                __syncwarp(live);
                if (lane == 31 - __clz(peers)) sm.hist[warp][d] = at + __popc(peers);
                const uint32_t to = at + __popc(peers & ((1u << lane) - 1));
                if (to < (uint32_t)T) out[to] = kv[q];   // always, unless another call writes to this workspace
            }
            __syncwarp();
        }
    }
    // the next pass reads the other CTAs' keys and rewrites the totals
    tc::cluster_sync();
}

// Zeroes n elements: pieces of ZERO_VECS vectors, dealt out to the blocks in turn.
constexpr size_t ZERO_VECS = 4096;
template <int BLOCKS, int THREADS, typename TG>
__device__ __forceinline__ void zero_span(TG* to, size_t n, int me) {
    const size_t vecs = n * sizeof(TG) / 16;
    for (size_t i0 = (size_t)me * ZERO_VECS; i0 < vecs; i0 += (size_t)BLOCKS * ZERO_VECS)
#pragma unroll
        for (size_t i = i0 + threadIdx.x; i < i0 + ZERO_VECS; i += THREADS)
            if (i < vecs) reinterpret_cast<uint4*>(to)[i] = make_uint4(0, 0, 0, 0);
    if (me == 0)
        for (size_t i = vecs * 16 / sizeof(TG) + threadIdx.x; i < n; i += THREADS) f32_to_elem(0.f, to[i]);
}

// First place in the sorted tokens whose key is not below `key`, by one warp:
// 32 probes a step.
__device__ __forceinline__ int lower_bound_warp(const Pair* __restrict__ sorted, int T, uint32_t key) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = T;
    while (hi - lo > 32) {
        const int stride = (hi - lo) / 33 + 1, pos = lo + (lane + 1) * stride - 1;
        const int c = __popc(__ballot_sync(0xffffffffu, pos < hi && sorted[pos].x < key));
        lo += c * stride;
        hi = min(hi, lo + stride - 1);
    }
    return lo + __popc(__ballot_sync(0xffffffffu, lo + lane < hi && sorted[lo + lane].x < key));
}

// Zeroes those of the rows [v_lo, v_hi) that no token has (at most 32 FLAG_WORDS
// rows): their tokens stand together in the sorted ones.
constexpr int FLAG_WORDS = 64;
template <int THREADS, typename TG>
__device__ __forceinline__ void zero_absent_rows(const Pair* __restrict__ sorted, int T, TG* grad, int H, int v_lo, int v_hi,
                                                 uint32_t* flags, int* range) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp < 2) {
        const int p = lower_bound_warp(sorted, T, (uint32_t)(warp ? v_hi : v_lo));
        if (lane == 0) range[warp] = p;
    }
    if (threadIdx.x < FLAG_WORDS) flags[threadIdx.x] = 0;
    __syncthreads();
    const int end = range[1];
#pragma unroll 4
    for (int p = range[0] + threadIdx.x; p < end; p += THREADS) {
        const uint32_t r = sorted[p].x - (uint32_t)v_lo;
        if (r < 32 * FLAG_WORDS) atomicOr(&flags[r >> 5], 1u << (r & 31));
    }
    __syncthreads();
    // a row by a warp, or by the lanes it has work for: its 16-byte pieces, and what lies beside them where rows are no
    // multiple of 16 bytes
    const size_t row_bytes = (size_t)H * sizeof(TG);
    const uint32_t vecs = max(1u, (uint32_t)(row_bytes / 16));
    const int lane_bits = vecs < 32 ? 32 - __clz(vecs - 1) : 5;   // (one: no bits)
    const uint32_t first = threadIdx.x & ((1u << lane_bits) - 1), step = 1u << lane_bits;
    for (int r = threadIdx.x >> lane_bits; r < v_hi - v_lo; r += THREADS >> lane_bits) {
        if (flags[r >> 5] >> (r & 31) & 1u) continue;
        TG* row = grad + (size_t)(v_lo + r) * H;
        if (row_bytes % 16 == 0) {
#pragma unroll 6
            for (uint32_t j = first; j < vecs; j += step) reinterpret_cast<uint4*>(row)[j] = make_uint4(0, 0, 0, 0);
            continue;
        }
        // elements up to the first piece, pieces, elements behind the last one
        const uint32_t before = min((uint32_t)H, (uint32_t)(-reinterpret_cast<uintptr_t>(row) & 15) / (uint32_t)sizeof(TG));
        const uint32_t whole = (uint32_t)((row_bytes - before * sizeof(TG)) / 16);
        TG* inner = row + before;
#pragma unroll 6
        for (uint32_t j = first; j < whole; j += step) reinterpret_cast<uint4*>(inner)[j] = make_uint4(0, 0, 0, 0);
        for (uint32_t j = first; j < before; j += step) f32_to_elem(0.f, row[j]);
        const uint32_t behind = before + whole * (16 / (uint32_t)sizeof(TG));
        for (uint32_t j = behind + first; j < (uint32_t)H; j += step) f32_to_elem(0.f, row[j]);
    }
}

// Few tokens are sorted by counting: a token's place is the number of tokens
// with a smaller id, or the same id and an earlier place.  Each warp places
// tokens of its own against all ids, held in shared memory.
constexpr int RANK_THREADS = 512, RANK_MAX_TOKENS = 4096;
__global__ void __launch_bounds__(RANK_THREADS)
    embed_rank_kernel(const int32_t* __restrict__ ids, int T, int V, Pair* __restrict__ out, unsigned int* status) {
    extern __shared__ __align__(16) uint32_t keys[];   // T rounded up to 4, padded with the largest key
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int T4 = (T + 3) / 4 * 4;
#pragma unroll 4
    for (int t = threadIdx.x; t < T4; t += RANK_THREADS) {
        const int id = t < T ? ids[t] : -1;
        const bool ok = id >= 0 && id < V;
        if (!ok && t < T && blockIdx.x == 0) atomicOr(status, TEE_STATUS_BAD_ID);
        keys[t] = ok ? (uint32_t)id : t < T ? (uint32_t)V : NO_KEY;
    }
    __syncthreads();
    for (int t = blockIdx.x * (RANK_THREADS / 32) + warp; t < T; t += gridDim.x * (RANK_THREADS / 32)) {
        const uint32_t k = keys[t];
        uint32_t n = 0;
        // up to t's group of four the same id counts as smaller; the group itself is looked at one by one
        const int g = t / 4;
#pragma unroll 4
        for (int j = lane; j < T4 / 4; j += 32) {
            const uint4 v = reinterpret_cast<const uint4*>(keys)[j];
            const uint32_t below = k + (j < g ? 1u : 0u);   // V < 2^32 - 1: no wrap
            n += (v.x < below) + (v.y < below) + (v.z < below) + (v.w < below);
        }
        if (lane < t - 4 * g) n += keys[4 * g + lane] == k;
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) out[n] = make_uint2(k, (uint32_t)t);
    }
}

constexpr int SORT_FILLERS = 512;   // fill CTAs beside the sort's: whole clusters

template <typename TG>
__global__ void __cluster_dims__(SORT_CTAS, 1, 1) __launch_bounds__(SORT_THREADS)
    embed_sort_kernel(const int32_t* __restrict__ ids, int T, int V, int H, int key_bits, Pair* buf0, Pair* buf1,
                      TG* __restrict__ grad, int fill_rows, unsigned int* status) {
    extern __shared__ __align__(16) uint8_t raw[];
    SortSmem& sm = *reinterpret_cast<SortSmem*>(raw);
    pdl_wait();
    pdl_trigger();
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
    // all of these rows: those that have tokens are written again by the sums, which wait for this kernel
    zero_span<SORT_FILLERS, SORT_THREADS>(grad, (size_t)fill_rows * H, (int)blockIdx.x - SORT_CTAS);
}

// ---------------------------------------------------------------------------
// backward: sums over runs of one id
// ---------------------------------------------------------------------------

// What a block of embed_sum_kernel leaves for embed_join_kernel.
//   head: the piece of a run that began in an earlier block: HEAD_NONE, HEAD_ENDS
//     (the run ends here) or HEAD_THROUGH (it fills the block and goes on).
//   tail_key: the id of a run that begins here and goes on, or NO_KEY.
constexpr int HEAD_NONE = 0, HEAD_ENDS = 1, HEAD_THROUGH = 2;
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

constexpr int SUM_BATCH = 4;   // rows a warp reads together

// The first sum_blocks x (column groups) blocks add, the column groups of the same
// tokens next to one another so that their rows are read together; the blocks
// behind them zero the rows fill_from .. V that no token has, chunk_rows each (one
// such block for every chunk: 256 with many chunks each took 10 us longer for 315
// MB).  Eight columns per lane in runs of W; each warp adds its tokens, and the warps' pieces of runs that
// cross warps are joined in shared memory.
template <typename TY, typename TG, int W, int TOKENS_PER_WARP>
__global__ void __launch_bounds__(SUM_WARPS * 32, 3)   // (64K tokens: 106 us for the call, 111 with two blocks an SM)
    embed_sum_kernel(const TY* __restrict__ dy, const Pair* __restrict__ sorted, TG* grad, int T, int V, int H, float scale,
                     int accumulate, int sum_blocks, int fill_from, int chunk_rows, BlockState* __restrict__ state,
                     float* __restrict__ head, float* __restrict__ tail) {
    constexpr int TOKENS_PER_BLOCK = TOKENS_PER_WARP * SUM_WARPS;
    // a warp's piece of the run that reaches into it from the left (L), and of the one that leaves it to the right (R)
    __shared__ float piece[2][SUM_WARPS][COLS];
    __shared__ uint32_t key_l[SUM_WARPS], key_r[SUM_WARPS];   // NO_KEY: no such piece
    __shared__ int through[SUM_WARPS];                        // L leaves the warp to the right as well
    pdl_wait();
    pdl_trigger();
    const int groups = (H + COLS - 1) / COLS, block = blockIdx.x / groups;
    if (block >= sum_blocks) {
        const long long lo = fill_from + (long long)((int)blockIdx.x - sum_blocks * groups) * chunk_rows;
        zero_absent_rows<SUM_WARPS * 32>(sorted, T, grad, H, (int)lo, (int)min((long long)V, lo + chunk_rows),
                                         reinterpret_cast<uint32_t*>(piece), through);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = blockIdx.x % groups, col0 = group * COLS;
    const long long first = (long long)block * TOKENS_PER_BLOCK + warp * TOKENS_PER_WARP;
    const int n = (int)max(0LL, min((long long)TOKENS_PER_WARP, T - first));
    auto col = [&](int j) { return (j / W * 32 + lane) * W + j % W; };   // within the block's columns
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
            // what is added to is read together, before anything is written
#pragma unroll
            for (int j0 = 0; j0 < 8; j0 += W) {
                float v[W] = {};
                if (accumulate && col0 + col(j0) < H) {
                    if constexpr (W == 1) v[0] = elem_to_f32(row[col(j0)]);
                    else load_vec(row + col(j0), v);
                }
#pragma unroll
                for (int j = 0; j < W; ++j) acc[j0 + j] = acc[j0 + j] * scale + v[j];
            }
#pragma unroll
            for (int j0 = 0; j0 < 8; j0 += W) {
                if (col0 + col(j0) >= H) continue;
                if constexpr (W == 1) {
                    f32_to_elem(acc[j0], row[col(j0)]);
                } else {
                    float v[W];
#pragma unroll
                    for (int j = 0; j < W; ++j) v[j] = acc[j0 + j];
                    store_vec(row + col(j0), v);
                }
            }
        };
        constexpr int BATCH = SUM_BATCH;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += BATCH) {
            float v[BATCH][8];
#pragma unroll
            for (int q = 0; q < BATCH; ++q) {
                const uint32_t k = __shfl_sync(0xffffffffu, kv.x, i0 + q), t = __shfl_sync(0xffffffffu, kv.y, i0 + q);
                const uint32_t last = i0 + q > 0 ? __shfl_sync(0xffffffffu, kv.x, (i0 + q - 1) & 31) : before;
                const TY* row = dy + (size_t)t * H + col0;
                const bool ok = k < (uint32_t)V && t < (uint32_t)T;   // false past the end as well (NO_KEY)
#pragma unroll
                for (int j0 = 0; j0 < 8; j0 += W) {
                    const bool in = ok && col0 + col(j0) < H;
                    if constexpr (W == 1) {
                        v[q][j0] = in ? elem_to_f32(row[col(j0)]) : 0.f;
                    } else {
                        float x[W] = {};
                        if (in) load_vec(row + col(j0), x);
#pragma unroll
                        for (int j = 0; j < W; ++j) v[q][j0 + j] = x[j];
                    }
                    // the row of the table that a new run will be added to, on its way while the tokens' rows are
                    if (accumulate && in && k != last)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(grad + (size_t)k * H + col0 + col(j0)));
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
                    if (in) head[(size_t)block * H + col0 + c] = acc;
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
        if (in) head[(size_t)block * H + col0 + c] = acc;
    } else if (open == 2) {
        if (in) tail[(size_t)block * H + col0 + c] = acc;
    }
    if (group == 0 && c == 0) state[block] = BlockState{head_state, open == 2 ? open_key : NO_KEY};
}

// Block b adds the run that begins in block b of embed_sum_kernel and crosses
// its end: tail of b, then the heads of b + 1 .. the block where the run ends.
// 64 threads side by side, W columns each, in four slices of the heads.
constexpr int JOIN_LANES = 64, JOIN_SLICES = 4;
template <typename TG, int W>
__global__ void __launch_bounds__(JOIN_LANES* JOIN_SLICES)
    embed_join_kernel(const BlockState* __restrict__ state, int n_blocks, const float* __restrict__ head,
                      const float* __restrict__ tail, TG* __restrict__ grad, int V, int H, float scale, int accumulate) {
    __shared__ float red[JOIN_SLICES - 1][JOIN_LANES][W];
    __shared__ int end_s;
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.x;
    const uint32_t key = state[b].tail_key;
    // the first block after b whose head ends the run
    int e = b + 1 + threadIdx.x;
    int mine = e < n_blocks ? state[e].head : HEAD_NONE;
    if (key >= (uint32_t)V) return;   // NO_KEY, or the run of out-of-range ids
    if (threadIdx.x == 0) end_s = INT32_MAX;
    __syncthreads();
    for (int e0 = b + 1; e0 < n_blocks; e0 += JOIN_LANES * JOIN_SLICES) {
        if (e0 != b + 1) {
            e = e0 + threadIdx.x;
            mine = e < n_blocks ? state[e].head : HEAD_NONE;
        }
        if (mine == HEAD_ENDS) atomicMin(&end_s, e);
        __syncthreads();
        const bool found = end_s != INT32_MAX;
        __syncthreads();
        if (found) break;
    }
    const int end = min(end_s, n_blocks - 1);
    const int c = threadIdx.x % JOIN_LANES, sl = threadIdx.x / JOIN_LANES;
    const int h = (blockIdx.y * JOIN_LANES + c) * W;
    auto load = [&](const float* p, float (&v)[W]) {
        if constexpr (W == 1) v[0] = *p;
        else load_vec(p, v);
    };
    float s[W] = {}, v[W];
    if (h < H) {
        if (sl == 0) load(tail + (size_t)b * H + h, s);
#pragma unroll 4
        for (int k = b + 1 + sl; k <= end; k += JOIN_SLICES) {
            load(head + (size_t)k * H + h, v);
#pragma unroll
            for (int j = 0; j < W; ++j) s[j] += v[j];
        }
    }
    if (sl) {
#pragma unroll
        for (int j = 0; j < W; ++j) red[sl - 1][c][j] = s[j];
    }
    __syncthreads();
    if (sl || h >= H) return;
#pragma unroll
    for (int i = 0; i < JOIN_SLICES - 1; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) s[j] += red[i][c][j];
    TG* row = grad + (size_t)key * H + h;
    if constexpr (W == 1) {
        put(row, 0, s[0], scale, accumulate);
    } else {
        float o[W] = {};
        if (accumulate) load_vec(row, o);
#pragma unroll
        for (int j = 0; j < W; ++j) o[j] = s[j] * scale + o[j];
        store_vec(row, o);
    }
}

// f(the largest of 8 (both types bf16), 4, 2 and 1 elements that divides H).
template <typename TA, typename TB, typename F>
cudaError_t with_vectors(int H, F&& f) {
    if constexpr (sizeof(TA) == 2 && sizeof(TB) == 2) {
        if (H % 8 == 0) return f(std::integral_constant<int, 8>{});
    }
    if (H % 4 == 0) return f(std::integral_constant<int, 4>{});
    return H % 2 == 0 ? f(std::integral_constant<int, 2>{}) : f(std::integral_constant<int, 1>{});
}

// Tokens per warp of embed_sum_kernel: 32 keep the pieces few; 8 spread few
// tokens over more blocks.
int tokens_per_warp(int T) { return T <= 16384 ? 8 : 32; }

struct EmbedWs {
    Pair *buf0, *buf1;
    BlockState* state;
    float *head, *tail;
    size_t bytes;
};
EmbedWs carve_embed(int T, int H, void* base) {
    WsCarve ws(base);
    EmbedWs w;
    const size_t per = (size_t)SUM_WARPS * tokens_per_warp(T), nb = (T + per - 1) / per;
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
            e = cudaFuncSetAttribute(embed_sort_kernel<TG>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            e = cudaFuncSetAttribute(embed_sort_kernel<TG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)sizeof(SortSmem));
            if (e != cudaSuccess) return e;
            ready[dev] = true;
        }
    }
    int key_bits = 1;
    while (key_bits < 32 && (V >> key_bits)) ++key_bits;   // keys 0 .. V
    const int passes = (key_bits + MAX_DIGIT_BITS - 1) / MAX_DIGIT_BITS;
    // sorting by counting takes 4 us at 2048 tokens and 25 at 8192, by digits 13 and 14
    const Pair* sorted = w.buf0;
    int fill_rows = 0;   // rows zeroed beside the sort
    if (T <= RANK_MAX_TOKENS) {
        const int blocks = std::min((T - 1) / (RANK_THREADS / 32) + 1, num_sms);
        e = launch_pdl(embed_rank_kernel, dim3(blocks), dim3(RANK_THREADS), (size_t)(T + 3) / 4 * 16, s, ids, T, V, w.buf0, status);
    } else {
        // as many as its time allows
        const double sort_us = 8.0 + (double)T * passes / 16384;
        fill_rows = accumulate ? 0 : (int)std::min((double)V, sort_us * 5e6 / ((double)H * sizeof(TG)));
        e = launch_pdl(embed_sort_kernel<TG>, dim3(SORT_CTAS + (accumulate ? 0 : SORT_FILLERS)), dim3(SORT_THREADS),
                       sizeof(SortSmem), s, ids, T, V, H, key_bits, w.buf0, w.buf1, grad, fill_rows, status);
        if (!(passes & 1)) sorted = w.buf1;
    }
    if (e != cudaSuccess) return e;
    const int per_warp = tokens_per_warp(T), nb = (T - 1) / (SUM_WARPS * per_warp) + 1;
    // chunks of 32 rows, more where they are shorter than 64 KB
    const int chunk_rows = 32 * (int)std::max<size_t>(1, std::min<size_t>(FLAG_WORDS, 2048 / ((size_t)H * sizeof(TG))));
    const int chunks = accumulate ? 0 : (int)(((long long)V - fill_rows + chunk_rows - 1) / chunk_rows);
    const dim3 grid((unsigned)((H + COLS - 1) / COLS * nb + chunks));
    auto sum = [&](auto kernel) {
        return launch_pdl(kernel, grid, dim3(SUM_WARPS * 32), 0, s, dy, sorted, grad, T, V, H, scale, (int)accumulate, nb,
                          fill_rows, chunk_rows, w.state, w.head, w.tail);
    };
    auto sums = [&](auto width) {
        constexpr int W = decltype(width)::value;
        return per_warp == 8 ? sum(embed_sum_kernel<TY, TG, W, 8>) : sum(embed_sum_kernel<TY, TG, W, 32>);
    };
    e = with_vectors<TY, TG>(H, sums);
    if (e != cudaSuccess || nb == 1) return e;   // one block: no run crosses blocks
    auto join = [&](auto kernel, int cols) {
        return launch_pdl(kernel, dim3(nb, (H + cols - 1) / cols), dim3(JOIN_LANES * JOIN_SLICES), 0, s, (const BlockState*)w.state,
                          nb, (const float*)w.head, (const float*)w.tail, grad, V, H, scale, (int)accumulate);
    };
    return H % 4 == 0 ? join(embed_join_kernel<TG, 4>, 4 * JOIN_LANES) : join(embed_join_kernel<TG, 1>, JOIN_LANES);
}

template <typename TE, typename TY>
cudaError_t forward_t(const void* table, const int32_t* ids, void* y, int T, int V, int H, float scale,
                      unsigned int* status, cudaStream_t s) {
    return with_vectors<TE, TY>(H, [&](auto width) {
        constexpr int W = decltype(width)::value;
        int lane_bits = 0;
        while (lane_bits < 5 && (1 << lane_bits) < H / W) ++lane_bits;
        const dim3 grid((unsigned)((((long long)T << lane_bits) + 255) / 256));
        return launch_pdl(embed_forward_kernel<TE, TY, W>, grid, dim3(256), 0, s, (const TE*)table, ids, (TY*)y, T, V, H, scale,
                          lane_bits, status);
    });
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
