// Attention of a training step over packed texts: the plan that both passes work by,
// and the backward pass on the 5th-generation tensor cores (sm_103a); tee_train.h has
// the formulas, k_attention_tc.cu the forward kernel.
//
// The probabilities are computed again from lse.  One kernel runs two kinds of units,
// each a tile of 128 rows of one head against all 128-row tiles that it may see:
//   rows are queries: S = Q K^T, dP = dO V^T, dQ += dS K;
//   rows are keys:    S^T = K Q^T, dP^T = V dO^T, dK += dS^T Q, dV += P^T dO,
// with P = exp2(S log2(e) / 8 - lse / ln 2) and dS = P (dP - delta).  Scores and
// probabilities are thus made twice, seven products to a pair of tiles instead of
// five: but no unit adds to another's sums, so nothing waits and nothing depends on
// an order, and dS goes from the registers to the tensor cores through tensor memory
// alone (for dQ from the key side it would cross shared memory twice, whose bandwidth
// the operands of the other products already take).
// Twelve warps: one brings the operands, three issue S, dP and the outputs' products, eight
// make P and dS of them.
// Measured, 12 heads: 8 texts of 8192 tokens 4.2 ms, where five products at the burst
// rate would take 2.09.  A pair of tiles takes 1430 cycles of each kind; the products by
// themselves, issued without a pause, take 1330 (keys) and 920 (queries), as one of K = 16
// costs 73 cycles with N = 128 and 38 with N = 64.  So the products set the pace where rows
// are keys, and the workers where rows are queries; the pipes are 63 to 67 % busy, under the
// power limit's clock of 1.76 GHz.  +-64 windows, 32768 tokens of 158 texts: 124 us, 98 of
// them in this kernel (205 + 111 MB of DRAM traffic) and 24 in the plan, which reads o and
// do (102 MB) for the deltas.
#include "gemm_tc.cuh"
#include "train_internal.cuh"

#include <limits.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "tc_ptx.cuh"

namespace {

using namespace tc;

constexpr int HD = 64;
constexpr int TILE = 128;

// ---------------------------------------------------------------------------
// the plan
// ---------------------------------------------------------------------------

constexpr int PLAN_THREADS = 512;
constexpr int PLAN_ROWS = 16;                 // rows of a row block
constexpr int PLAN_HEADS = 32;                // heads staged at once
constexpr int PLAN_SHARED_TEXTS = 2048;       // texts whose lists fit shared memory
constexpr int PLAN_BUCKETS = TEE_ATTN_MAX_TEXT / TILE + 1;

struct PlanArgs {
    const int32_t* cu;
    int T, n_texts, n_heads, window, max_items;
    AttnPlan plan;
    const bf16* o;          // backward only
    const bf16* d_o;
    const float* lse;
    unsigned int* status;
};

// The first index of cu[0 .. n] whose value is above v, n + 1 if none is.
__device__ __forceinline__ int first_above(const int32_t* cu, int n, int v) {
    int lo = 0, hi = n + 1;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (cu[mid] > v) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Block 0 lists the work items, the others prepare PLAN_ROWS rows each.
//
// Items of whole-text layers: a text of more than 128 tokens gives one per 128 rows;
// shorter ones share tiles, each the longest run of consecutive such texts that spans
// at most 128 tokens.  Where a run's tiles start depends on where the one before
// ended: with next(j) the start after one at j, the starts are what is reached from 0,
// found by doubling the steps (log2 of the number of texts).
// Items of window layers: 128 rows of the packed batch, whatever texts they are of.
// Up to PLAN_SHARED_TEXTS texts the lists are in shared memory.  For more, block 0 follows its
// links through global memory while the others have long ended: 4000 texts of 16 tokens 54 us
// (windows, which need no starts: 16), 60000 of 8 tokens 1.64 ms (0.11), 2^20 of one 39.7 ms (0.3).
__global__ void __launch_bounds__(PLAN_THREADS) attn_plan_kernel(const PlanArgs a) {
    __shared__ int lists[3 * (PLAN_SHARED_TEXTS + 1)], offsets[PLAN_SHARED_TEXTS + 1];
    __shared__ int bucket[PLAN_BUCKETS + 1];
    __shared__ int bad;
    __shared__ float stage[PLAN_HEADS][PLAN_ROWS + 1];
    // No early trigger: the attention kernel's blocks, one to an SM, would take the SMs from the
    // blocks that are still to come (window layer of 32768 tokens, backward: 200 us instead of 152).
    pdl_wait();
    const int n = a.n_texts, tid = threadIdx.x;
    // (searched out of shared memory where they fit: a search is a chain of loads)
    const bool fits = n <= PLAN_SHARED_TEXTS;
    const int32_t* cu = a.cu;
    if (fits) {
        for (int j = tid; j <= n; j += PLAN_THREADS) offsets[j] = a.cu[j];
        __syncthreads();
        cu = offsets;
    }
    if (blockIdx.x > 0) {
        const int row0 = (blockIdx.x - 1) * PLAN_ROWS;
        if (tid < PLAN_ROWS && row0 + tid < a.T) {
            const int t = row0 + tid, j = first_above(cu, n, t);
            int2 tb = make_int2(0, 0);
            if (j >= 1 && j <= n) tb = make_int2(max(cu[j - 1], 0), min(cu[j], a.T));
            a.plan.row_tb[t] = tb;
        }
        if (!a.o) return;
        // delta = sum_d do o: a head by eight lanes, eight columns each
        const int warp = tid >> 5, lane = tid & 31, H = a.n_heads * HD;
        for (int h0 = 0; h0 < a.n_heads; h0 += PLAN_HEADS) {
            const int nh = min(PLAN_HEADS, a.n_heads - h0);
            for (int r = warp; r < PLAN_ROWS && row0 + r < a.T; r += PLAN_THREADS / 32) {
                for (int g = lane >> 3; g < (nh + 3) / 4 * 4; g += 4) {
                    float s = 0.f;
                    if (g < nh) {
                        const size_t at = (size_t)(row0 + r) * H + (size_t)(h0 + g) * HD + (lane & 7) * 8;
                        float x[8], y[8];
                        load_vec(a.o + at, x);
                        load_vec(a.d_o + at, y);
#pragma unroll
                        for (int i = 0; i < 8; ++i) s = fmaf(x[i], y[i], s);
                    }
#pragma unroll
                    for (int d = 4; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                    if (g < nh && (lane & 7) == 0) stage[g][r] = -s;
                }
            }
            __syncthreads();
            for (int i = tid; i < nh * PLAN_ROWS; i += PLAN_THREADS) {
                const int g = i / PLAN_ROWS, r = i % PLAN_ROWS;
                if (row0 + r < a.T) {
                    const size_t at = (size_t)(h0 + g) * a.T + row0 + r;
                    a.plan.ndelta[at] = stage[g][r];
                    a.plan.nlse2[at] = a.lse[at] * -1.4426950408889634f;
                }
            }
            __syncthreads();
        }
        return;
    }
    if (tid == 0) bad = 0;
    for (int i = tid; i <= PLAN_BUCKETS; i += PLAN_THREADS) bucket[i] = 0;
    __syncthreads();
    int wrong = 0;
    for (int j = tid; j < n; j += PLAN_THREADS) {
        const int c0 = cu[j], c1 = cu[j + 1];
        wrong |= c0 < 0 || c1 < c0 || c1 > a.T || c1 - c0 > TEE_ATTN_MAX_TEXT || (j == 0 && c0 != 0);
    }
    if (wrong) bad = 1;
    __syncthreads();
    if (bad) {
        if (tid == 0) {
            *a.plan.n_items = 0;
            atomicOr(a.status, TEE_STATUS_BAD_ID);
        }
        return;
    }
    const int end = cu[n];
    if (a.window >= 0) {
        const int tiles = (end + TILE - 1) / TILE;
        for (int i = tid; i < tiles; i += PLAN_THREADS) {
            const int q0 = i * TILE, ql = min(TILE, end - q0);
            const int j0 = first_above(cu, n, q0), j1 = first_above(cu, n, q0 + ql - 1);   // ends of the first and last row's texts
            a.plan.items[i] = make_int4(q0, ql, max(cu[j0 - 1], q0 - a.window),
                                        (int)min((long long)cu[j1], (long long)q0 + ql + a.window));
        }
        if (tid == 0) *a.plan.n_items = tiles;
        return;
    }
    int* from = fits ? lists : a.plan.scratch;
    int* to = from + n + 1;
    int* mark = to + n + 1;
    for (int j = tid; j <= n; j += PLAN_THREADS) {
        int e = n;
        if (j < n) {
            const int c = cu[j];
            e = cu[j + 1] - c > TILE ? j + 1 : first_above(cu, n, c + TILE) - 1;
        }
        from[j] = e;
        mark[j] = j == 0;
    }
    __syncthreads();
    for (int step = 1; step < n; step *= 2) {
        for (int j = tid; j < n; j += PLAN_THREADS)
            if (mark[j]) mark[from[j]] = 1;
        __syncthreads();
        for (int j = tid; j <= n; j += PLAN_THREADS) to[j] = from[from[j]];
        __syncthreads();
        int* const x = from;
        from = to;
        to = x;
    }
    // a start's items and their keys in tiles of 128
    auto start = [&](int j, int& tiles, int& c0, int& c1) {
        if (!mark[j]) return 0;
        c0 = cu[j], c1 = cu[j + 1];
        if (c1 - c0 > TILE) {
            tiles = (c1 - c0 + TILE - 1) / TILE;
            return tiles;
        }
        c1 = cu[first_above(cu, n, c0 + TILE) - 1];
        tiles = 1;
        return c1 > c0 ? 1 : 0;
    };
    for (int j = tid; j < n; j += PLAN_THREADS) {
        int tiles, c0, c1;
        const int items = start(j, tiles, c0, c1);
        if (items) atomicAdd(&bucket[tiles], items);
    }
    __syncthreads();
    if (tid < 32) {   // where each bucket's items begin, the most keys first
        int base = 0;
        for (int i0 = PLAN_BUCKETS; i0 >= 0; i0 -= 32) {
            const int i = i0 - tid, v = i >= 0 ? bucket[i] : 0;
            int inc = v;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, inc, d);
                if (tid >= d) inc += up;
            }
            if (i >= 0) bucket[i] = base + inc - v;
            base += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (tid == 0) *a.plan.n_items = min(base, a.max_items);
    }
    __syncthreads();
    // (which of two equally long items comes first has no effect on results)
    for (int j = tid; j < n; j += PLAN_THREADS) {
        int tiles, c0, c1;
        const int items = start(j, tiles, c0, c1);
        if (!items) continue;
        const int at = atomicAdd(&bucket[tiles], items);
        for (int i = 0; i < items && at + i < a.max_items; ++i)
            a.plan.items[at + i] = make_int4(c0 + i * TILE, min(TILE, c1 - c0 - i * TILE), c0, c1);
    }
}

// ---------------------------------------------------------------------------
// the backward kernel
// ---------------------------------------------------------------------------

// (Four stages instead of boxes for the outputs: 152 us instead of 138 on the window layer.)
constexpr int STAGES = 3;
// Workers: warps 4 .. 11, two to a quarter of the rows, 64 columns each.  (8 x 8192 tokens: 16
// warps of 32 columns 4.3 to 4.5 ms; two groups of four on alternate tiles 5.8.)
constexpr int FIRST_WORKER = 4, WORKERS = 8;
constexpr int NUM_THREADS = 32 * (FIRST_WORKER + WORKERS);
constexpr uint32_t TILE_BYTES = TILE * HD * 2;                       // 16 KB
constexpr uint32_t OFF_ROWS = 0;                                     // 2 buffers of two tiles
constexpr uint32_t OFF_COLS = OFF_ROWS + 4 * TILE_BYTES;             // STAGES of two tiles
// Where columns are queries, their lse and delta come as 16 more columns of the operands:
// for S the stage's rows hold -8 lse in three bf16 that add up to it, for dP -delta in
// three, and the rows' side is ones against them.  The other columns are zeros on both
// sides: ones against lse alone, with zeros against delta beside it, would make a P of NaN
// of a delta that is.  (Read from shared memory by the workers, a column's two numbers go to
// 128 threads each: 512 bytes a warp for 16 of them, 1024 cycles a tile for what the tensor
// cores do in 128.)
// Not swizzled: 8 rows of eight columns are 128 bytes.  A stage has three such pieces for
// 8 rows, {lse, zeros, delta}, and S takes the first two, dP the last two.
constexpr uint32_t EXT_PIECES = 3 * 128, EXT_BYTES = TILE / 8 * EXT_PIECES;
constexpr uint32_t ONES_PIECES = 2 * 128, ONES_BYTES = TILE / 8 * ONES_PIECES;
constexpr uint32_t OFF_EXT = OFF_COLS + STAGES * 2 * TILE_BYTES;     // STAGES
constexpr uint32_t OFF_ONES = OFF_EXT + STAGES * EXT_BYTES;          // for S, for dP
constexpr uint32_t OFF_OUT = OFF_ONES + 2 * ONES_BYTES;              // a 4 KB box per worker warp
constexpr uint32_t OFF_BAR = OFF_OUT + WORKERS * 4096;
constexpr int B_RF = 0, B_RE = 2, B_CF = 4, B_CE = B_CF + STAGES, B_SF = B_CE + STAGES, B_XF = B_SF + STAGES,
              B_X2R = B_XF + 2, B_PF = B_X2R + 1, B_OF = B_PF + 2, B_OE = B_OF + 1, B_DONE = B_OE + 1, N_BARS = B_DONE + 1;
constexpr uint32_t SMEM_TOTAL = OFF_BAR + N_BARS * 8 + 16 + 1024;
static_assert(SMEM_TOTAL <= 227 * 1024, "shared memory");
// Tensor memory: X1 = S of even and odd tiles, X2 = dP of the current one, the outputs.
// A worker writes dS and P over columns of S that it read itself, so workers need not
// wait for one another.
constexpr uint32_t TM_X1 = 0, TM_X2 = 256, TM_O = 384, TMEM_COLS = 512;
constexpr uint32_t TILE_DESC = TILE_BYTES >> 4, PAIR_DESC = 2 * TILE_DESC;   // a tile, and two, as descriptors count
constexpr float SCALE_LOG2 = 1.4426950408889634f / 8.0f;

// Descriptor of 16 further columns: K-major, no swizzle; their two pieces of 8 rows are 128
// bytes apart, 8 rows and the next 8 `pieces`.
__device__ __forceinline__ uint64_t ext_desc(uint32_t saddr, uint32_t pieces) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 16 | (uint64_t)(pieces >> 4) << 32 |
           (uint64_t)1 << 46;
}
// v as three bf16 whose sum is within 2^-24 of it, one piece of a row; infinities as they are.
__device__ __forceinline__ uint4 three_bf16(float v) {
    bf16 o[8] = {};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        o[i] = __float2bfloat16_rn(v);
        v -= __bfloat162float(o[i]);
        if (!(v < INFINITY)) v = 0.f;
    }
    uint4 q;
    memcpy(&q, o, 16);
    return q;
}

struct BwdParams {
    AttnPlan plan;
    int T, n_heads, hidden, window;
    const bf16* qkv;
    const bf16* d_o;
    bf16* dqkv;
    unsigned int* status;
};

// How many units are the CTA's.
__device__ __forceinline__ int bwd_units(const BwdParams& p) {
    return attn_units_of(*p.plan.n_items * 2 * p.n_heads, blockIdx.x, gridDim.x);
}
// A CTA's units in turn, each read while the one before is worked on: {q_start, q_len |
// keys << 8 | head << 16, k_lo, k_hi}.  An item's rows as keys, the longer kind, for every
// head, then as queries, which finds them in L2.  From unit to unit (attn_unit) the steps
// are two in turn, so one division each does for all.
struct UnitStream {
    const BwdParams& p;
    int n, i = 0, item, head, step_item[2], step_head[2];   // (of `item` there are two for each, by kind)
    int4 ahead;
    __device__ __forceinline__ UnitStream(const BwdParams& p_, int n_) : p(p_), n(n_) {
        const int c = blockIdx.x, G = gridDim.x, heads = p.n_heads;
        item = c / heads, head = c - item * heads;
        step_item[0] = (2 * (G - c) - 1) / heads, step_head[0] = 2 * (G - c) - 1 - step_item[0] * heads;
        step_item[1] = (2 * c + 1) / heads, step_head[1] = 2 * c + 1 - step_item[1] * heads;
        read();
    }
    __device__ __forceinline__ void read() {
        ahead = make_int4(0, 0, 0, 0);
        if (i >= n) return;
        ahead = p.plan.items[item >> 1];
        ahead.y |= (~item & 1) << 8 | head << 16;
    }
    __device__ __forceinline__ int4 next() {
        const int4 it = ahead;
        item += i & 1 ? step_item[1] : step_item[0];
        head += i & 1 ? step_head[1] : step_head[0];
        if (head >= p.n_heads) head -= p.n_heads, ++item;
        ++i;
        read();
        return it;
    }
};
// Four bytes, each a byte of v's top bit over: the byte that the digit of SELECT less 8 names.
template <int SELECT>
__device__ __forceinline__ uint32_t byte_signs(uint32_t v) {
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(v), "n"(SELECT));
    return r;
}
__device__ __forceinline__ int unit_tiles(const int4& it) { return (it.w - it.z + TILE - 1) / TILE; }

// A whole warp's wait for what it has not found done; gives up as mbar_wait does.
__device__ __noinline__ bool warp_wait_longer(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    const long long t0 = clock64();
    while (true) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        const bool late = clock64() - t0 > WAIT_CYCLES;
        if (__any_sync(0xffffffffu, late || *abort_flag)) {
            *abort_flag = 1;
            return false;
        }
    }
}

// The columns that a row of a unit sees, its text being {tb.x, tb.y}: the text, and in
// window layers the window in it.
__device__ __forceinline__ void seen_columns(const BwdParams& p, const int4& it, int row, const int2& tb, int& lo, int& hi) {
    lo = max(tb.x, it.z), hi = min(tb.y, it.w);
    if (p.window >= 0) lo = max(lo, row - p.window), hi = min(hi, row + p.window + 1);
}

// dq of one row, or its dk (`first`) and dv (`second`), again, from the columns that it sees,
// outside the tensor cores, by a whole warp: four columns side by side, eight lanes to each,
// the loads of three such steps on their way together.  It ends early where nothing but NaN
// can come.
__device__ __noinline__ void bwd_row_again(const BwdParams& p, int row, int head, bool keys, int lo, int hi, bool first,
                                           bool second) {
    constexpr int AT_ONCE = 3;
    const int lane = threadIdx.x & 31, part = lane >> 3, at = head * HD + (lane & 7) * 8, H = p.hidden;
    const size_t stride = 3 * (size_t)H;
    const bf16* const qkv = p.qkv + at;
    const bf16* const d_o = p.d_o + at;
    float a1[8], a2[8], o1[8] = {}, o2[8] = {};
    load_vec(qkv + row * stride + (keys ? H : 0), a1);
    load_vec(keys ? qkv + row * stride + 2 * H : d_o + (size_t)row * H, a2);
    for (int j0 = lo; j0 < hi; j0 += 4 * AT_ONCE) {
        uint4 q1[AT_ONCE], q2[AT_ONCE];
        float nl[AT_ONCE], nd[AT_ONCE];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            const int j = min(j0 + 4 * u + part, hi - 1);
            const size_t s = (size_t)head * p.T + (keys ? j : row);
            q1[u] = *reinterpret_cast<const uint4*>(qkv + j * stride + (keys ? 0 : H));
            q2[u] = *reinterpret_cast<const uint4*>(keys ? d_o + (size_t)j * H : qkv + j * stride + 2 * H);
            nl[u] = p.plan.nlse2[s], nd[u] = p.plan.ndelta[s];
        }
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            float b1[8], b2[8], s1 = 0.f, s2 = 0.f;
            unpack_bf16x8(q1[u], b1);
            unpack_bf16x8(q2[u], b2);
#pragma unroll
            for (int i = 0; i < 8; ++i) s1 = fmaf(a1[i], b1[i], s1), s2 = fmaf(a2[i], b2[i], s2);
#pragma unroll
            for (int d = 4; d > 0; d >>= 1) {
                s1 += __shfl_xor_sync(0xffffffffu, s1, d);
                s2 += __shfl_xor_sync(0xffffffffu, s2, d);
            }
            if (j0 + 4 * u + part < hi) {
                const float e = ex2_approx(fmaf(s1, SCALE_LOG2, nl[u])), d = e * (s2 + nd[u]);
#pragma unroll
                for (int i = 0; i < 8; ++i) o1[i] = fmaf(d, b1[i], o1[i]), o2[i] = fmaf(e, b2[i], o2[i]);
            }
        }
        const bool nan1 = each_eighth_has(all_nan(o1)), nan2 = each_eighth_has(all_nan(o2));
        if ((nan1 || !first) && (nan2 || !second)) break;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int d = 8; d < 32; d *= 2) {
            o1[i] += __shfl_xor_sync(0xffffffffu, o1[i], d);
            o2[i] += __shfl_xor_sync(0xffffffffu, o2[i], d);
        }
        o1[i] *= 0.125f;
    }
    if (part) return;
    bf16* const dst = p.dqkv + row * stride + at;
    if (first) store_vec(dst + (keys ? H : 0), o1);
    if (second) store_vec(dst + 2 * H, o2);
}

// Rows whose products met NaN or infinities of rows that they do not see are computed again,
// as by the forward kernel (attn_again): once all of the CTA's units are done and no role
// waits for another any more; not those that see all of the item's columns, and not those that
// cannot have another gradient, as their own term is NaN in all of its columns: dq and dk
// of a row whose log sum or delta is NaN, dv of one whose log sum is or whose d_o is nothing else.
__device__ __noinline__ void bwd_again(const BwdParams& p) {
    const int lane = threadIdx.x & 31, units = bwd_units(p);
    for (int task = threadIdx.x >> 5; task < 4 * units; task += NUM_THREADS / 32) {
        const int unit = attn_unit(task >> 2, blockIdx.x, gridDim.x), item = unit / p.n_heads, head = unit - item * p.n_heads;
        const bool keys = !(item & 1);
        const int4 it = p.plan.items[item >> 1];
        const int r = (task & 3) * 32 + lane, row = it.x + r;
        int lo = 0, hi = 0;
        bool first = false, second = false;
        if (r < it.y) {
            seen_columns(p, it, row, p.plan.row_tb[row], lo, hi);
            const size_t s = (size_t)head * p.T + row;
            const float nl = p.plan.nlse2[s], nd = p.plan.ndelta[s];
            if ((lo > it.z || hi < it.w) && nl == nl) {
                const bf16* const out = p.dqkv + (size_t)row * 3 * p.hidden + head * HD;
                first = nd == nd && !all_finite(out + (keys ? p.hidden : 0));
                second = keys && !all_finite(out + 2 * p.hidden) && !all_nan(p.d_o + (size_t)row * p.hidden + head * HD);
            }
        }
        const unsigned firsts = __ballot_sync(0xffffffffu, first), seconds = __ballot_sync(0xffffffffu, second);
        for (unsigned again = firsts | seconds; again; again &= again - 1) {
            const int l = __ffs(again) - 1;
            bwd_row_again(p, __shfl_sync(0xffffffffu, row, l), head, keys, __shfl_sync(0xffffffffu, lo, l),
                          __shfl_sync(0xffffffffu, hi, l), firsts >> l & 1, seconds >> l & 1);
        }
    }
}

__global__ void __launch_bounds__(NUM_THREADS, 1)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap tm_qkv, const __grid_constant__ CUtensorMap tm_do,
                    const __grid_constant__ CUtensorMap tm_out,
                    const __grid_constant__ BwdParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + N_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* not_finite = abort_flag + 1;   // some output is not
    auto bar = [&](int i) { return smem_u32(bars + i); };
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(B_RF + b), 1);
            mbar_init(bar(B_RE + b), 2);          // S and dP of the unit's last tile
            mbar_init(bar(B_XF + b), 2);          // S and dP
            mbar_init(bar(B_PF + b), WORKERS);
        }
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar(B_CF + s), 1);
            mbar_init(bar(B_CE + s), 1);
            mbar_init(bar(B_SF + s), 1);
        }
        mbar_init(bar(B_X2R), WORKERS);
        mbar_init(bar(B_OF), 1);
        mbar_init(bar(B_OE), WORKERS);
        mbar_init(bar(B_DONE), 3);            // all issuers
        *abort_flag = *not_finite = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<1>(smem_u32(tmem_slot), TMEM_COLS);
    // the further columns' zeros, and ones against -lse in the first piece of 8 rows, against -delta in the second
    for (int i = threadIdx.x; i < (int)(STAGES * EXT_BYTES + 2 * ONES_BYTES) / 16; i += NUM_THREADS) {
        const int at = i * 16 - STAGES * EXT_BYTES, to = at / (int)ONES_BYTES, piece = at % (int)ONES_PIECES / 128;
        *reinterpret_cast<uint4*>(smem + OFF_EXT + 16 * i) =
            at >= 0 && piece == to ? make_uint4(0x3f803f80u, 0x00003f80u, 0, 0) : make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    const int n_units = bwd_units(p);
    // a whole warp's wait: true for all lanes, or false for all
    auto warp_wait = [&](int b, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_try_wait(bar(b), parity)) || warp_wait_longer(bar(b), parity, abort_flag);
    };

    if (warp == 0) {
        // ---------------- producer: copies, and the further columns where columns are queries ----------------
        uint32_t t = 0;
        int ui = 0;
        bool ok = true;
        UnitStream units(p, n_units);
        float v[2][4];   // of the tile to come
        auto statistics = [&](const int4& it, int kt) {
            if (!(it.y >> 8 & 1)) return;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = it.z + kt * TILE + i * 32 + lane;
                const size_t at = (size_t)(it.y >> 16) * p.T + row;
                v[0][i] = row < it.w ? p.plan.nlse2[at] : 0.f;
                v[1][i] = row < it.w ? p.plan.ndelta[at] : 0.f;
            }
        };
        if (n_units > 0) statistics(units.ahead, 0);
        for (; ui < n_units && ok; ++ui) {
            const int4 it = units.next();
            const int head = it.y >> 16, nk = unit_tiles(it), rb = ui & 1;
            const bool keys = it.y >> 8 & 1;
            const int xq = head * HD, xk = p.hidden + head * HD, xv = 2 * p.hidden + head * HD;
            if (!warp_wait(B_RE + rb, ((ui >> 1) & 1) ^ 1)) break;
            if (elect_one()) {
                mbar_expect_tx(bar(B_RF + rb), 2 * TILE_BYTES);
                const uint32_t a = sbase + OFF_ROWS + rb * 2 * TILE_BYTES;
                tma_load_2d(a, &tm_qkv, keys ? xk : xq, it.x, bar(B_RF + rb));
                tma_load_2d(a + TILE_BYTES, keys ? &tm_qkv : &tm_do, keys ? xv : xq, it.x, bar(B_RF + rb));
            }
            __syncwarp();
            for (int kt = 0; kt < nk; ++kt, ++t) {
                const int s = t % STAGES, y = it.z + kt * TILE;
                if (!warp_wait(B_CE + s, ((t / STAGES) & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    mbar_expect_tx(bar(B_CF + s), 2 * TILE_BYTES);
                    const uint32_t b = sbase + OFF_COLS + s * 2 * TILE_BYTES;
                    tma_load_2d(b, &tm_qkv, keys ? xq : xk, y, bar(B_CF + s));
                    tma_load_2d(b + TILE_BYTES, keys ? &tm_do : &tm_qkv, keys ? xq : xv, y, bar(B_CF + s));
                }
                __syncwarp();
                if (keys) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // S + 8 (-lse), of which log2(e) / 8 is the exponent
                        uint8_t* const ext =
                            smem + OFF_EXT + s * EXT_BYTES + (4 * i + (lane >> 3)) * EXT_PIECES + (lane & 7) * 16;
                        *reinterpret_cast<uint4*>(ext) = three_bf16(v[0][i] * (1.0f / SCALE_LOG2));
                        *reinterpret_cast<uint4*>(ext + 256) = three_bf16(v[1][i]);
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_SF + s));
                if (kt + 1 < nk) statistics(it, kt + 1);
                else statistics(units.ahead, 0);
            }
        }
        // no copy may still be landing in shared memory when the CTA exits
        for (int b = 0; b < 2 && b < ui; ++b) {
            const int u = (ui - 1 - b);
            mbar_wait_drain(bar(B_RF + (u & 1)), (u >> 1) & 1);
        }
        for (uint32_t s = 0; s < STAGES && s < t; ++s) {
            const uint32_t u = t - 1 - s;
            mbar_wait_drain(bar(B_CF + u % STAGES), (u / STAGES) & 1);
        }
    } else if (warp <= 2) {
        // ---------------- issuers of S (warp 1) and of dP (warp 2): the whole warp, one lane issuing ----------------
        // The tensor cores take a product when the one before is nearly done, so a warp that waits for the workers leaves
        // them idle unless another has products to issue: S, dP and the outputs have a warp each.
        constexpr uint32_t idesc = make_idesc(TILE, TILE);
        const bool is_s = warp == 1;
        const uint32_t op = is_s ? 0 : TILE_DESC;
        const uint64_t rows0 = sw128_desc(sbase + OFF_ROWS) + op, cols0 = sw128_desc(sbase + OFF_COLS) + op;
        const uint64_t ones = ext_desc(sbase + OFF_ONES + (is_s ? 0 : ONES_BYTES), ONES_PIECES);
        const uint64_t ext0 = ext_desc(sbase + OFF_EXT + (is_s ? 0 : 128), EXT_PIECES);
        uint32_t t = 0;
        bool ok = true;
        UnitStream units(p, n_units);
        for (int ui = 0; ui < n_units && ok; ++ui) {
            const int4 it = units.next();
            const int nk = unit_tiles(it), rb = ui & 1;
            const bool keys = it.y >> 8 & 1;
            if (!warp_wait(B_RF + rb, (ui >> 1) & 1)) break;
            const uint64_t a = rows0 + rb * PAIR_DESC;
            for (int kt = 0; kt < nk; ++kt, ++t) {
                const uint32_t st = t % STAGES;
                ok = warp_wait(B_CF + st, (t / STAGES) & 1);
                if (ok && keys) ok = warp_wait(B_SF + st, (t / STAGES) & 1);
                // S: the products of tile t - 2, which read this half of X1, are done; dP: the workers have read the tile before's
                if (ok && is_s && t >= 2) ok = warp_wait(B_CE + (t - 2) % STAGES, ((t - 2) / STAGES) & 1);
                if (ok && !is_s && t >= 1) ok = warp_wait(B_X2R, (t - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t b = cols0 + st * PAIR_DESC, ext = ext0 + st * (EXT_BYTES >> 4);
                const uint32_t x = tmem_base + (is_s ? TM_X1 + (t & 1) * TILE : TM_X2);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k) mma_bf16(x, a + 2 * k, b + 2 * k, idesc, k != 0);
                    if (keys) mma_bf16(x, ones, ext, idesc, 1);
                    mma_commit(bar(B_XF) + 8 * (t & 1));
                    if (kt == nk - 1) mma_commit(bar(B_RE) + 8 * rb);
                }
                __syncwarp();
            }
        }
        // every MMA issued must be finished before TMEM is freed
        if (elect_one()) mma_commit(bar(B_DONE));
        __syncwarp();
        mbar_wait_drain(bar(B_DONE), 0);
    } else if (warp == 3) {
        // ---------------- issuer of the outputs' products, of tiles whose P and dS the workers have written ----------------
        constexpr uint32_t idesc = make_idesc(TILE, HD) | IDESC_B_MN_MAJOR;
        const uint64_t cols0 = sw128_desc_mn(sbase + OFF_COLS);
        uint32_t t = 0;
        bool ok = true;
        UnitStream units(p, n_units);
        for (int ui = 0; ui < n_units && ok; ++ui) {
            const int4 it = units.next();
            const int nk = unit_tiles(it);
            const bool keys = it.y >> 8 & 1;
            for (int kt = 0; kt < nk; ++kt, ++t) {
                const uint32_t st = t % STAGES;
                ok = warp_wait(B_PF + (t & 1), (t >> 1) & 1);
                // the unit's first: the workers have read the one before
                if (ok && kt == 0) ok = warp_wait(B_OE, (ui & 1) ^ 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t x = tmem_base + TM_X1 + (t & 1) * TILE, o = tmem_base + TM_O;
                const uint64_t b = cols0 + st * PAIR_DESC;
                if (elect_one()) {
                    if (keys) {
#pragma unroll
                        for (int k = 0; k < TILE / 16; ++k) mma_bf16_ts(o, x + k * 16, b + k * 128, idesc, (kt | k) != 0);
#pragma unroll
                        for (int k = 0; k < TILE / 16; ++k)
                            mma_bf16_ts(o + HD, x + k * 16 + 8, b + TILE_DESC + k * 128, idesc, (kt | k) != 0);
                    } else {
#pragma unroll
                        for (int k = 0; k < TILE / 16; ++k)
                            mma_bf16_ts(o, x + (k >> 2) * 64 + (k & 3) * 8, b + k * 128, idesc, (kt | k) != 0);
                    }
                    mma_commit(bar(B_CE) + 8 * st);
                    if (kt == nk - 1) mma_commit(bar(B_OF));
                }
                __syncwarp();
            }
        }
        if (elect_one()) mma_commit(bar(B_DONE));
        __syncwarp();
        mbar_wait_drain(bar(B_DONE), 0);
    } else {
        // ---------------- workers: thread = row, 64 columns of each tile ----------------
        const int quad = warp & 3, chunk = (warp - FIRST_WORKER) >> 2;
        const int r = quad * 32 + lane;
        const uint32_t lanes = tmem_base + ((uint32_t)(quad * 32) << 16);
        const uint64_t sl2 = f2_pack(SCALE_LOG2, SCALE_LOG2);
        uint32_t t = 0;
        bool ok = true;

        // the text of row r of a unit, {0, 0} behind its rows
        auto text_of = [&](const int4& it) -> int2 { return r < (it.y & 0xff) ? p.plan.row_tb[it.x + r] : make_int2(0, 0); };
        // A unit's outputs, read once the next one's first tile is handed over: dq, half by
        // each warp of the two, or dk by one and dv by the other.  They leave as copies of 32
        // rows (row by row from the threads, a warp's store touches 32 lines: 1024 to 2048
        // cycles a unit for the 8 warps).
        auto finish = [&](int ui_p, const int4& it_p) -> bool {
            const int q_len_p = it_p.y & 0xff, row_p = r < q_len_p ? it_p.x + r : -1, head_p = it_p.y >> 16;
            const bool keys_p = it_p.y >> 8 & 1;
            if (!warp_wait(B_OF, ui_p & 1)) return false;
            if (lane == 0) bulk_wait_read<0>();   // the box's last copy has read it
            __syncwarp();
            tc_fence_after();
            // where rows are keys this warp's 64 columns of dk or dv, else its 32 of dq: boxes of 32
            const bool whole = quad * 32 + 32 <= q_len_p;
            const float scale = keys_p && chunk ? 1.f : 0.125f;
            float z = 0.f;   // not a number where one of the sums is not finite
            const int x = (keys_p ? (chunk + 1) * p.hidden : chunk * 32) + head_p * HD;
            const uint32_t from = lanes + TM_O + (keys_p ? HD : 32) * chunk;
            uint8_t* const box = smem + OFF_OUT + (warp - FIRST_WORKER) * 4096;
            bf16* const dst = p.dqkv + (size_t)max(row_p, 0) * 3 * p.hidden + x;
            const int boxes = keys_p ? 2 : 1;
#pragma unroll 1
            for (int h = 0; h < boxes; ++h) {
                float o[32];
                tmem_ld32(from + 32 * h, o);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t q[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float u = o[8 * c + 2 * j] * scale, v = o[8 * c + 2 * j + 1] * scale;
                        z = fmaf(u, 0.f, fmaf(v, 0.f, z));
                        q[j] = pack_bf16(u, v);
                    }
                    const uint4 piece = make_uint4(q[0], q[1], q[2], q[3]);
                    // rows of 64 bytes, swizzled: 16-byte piece c of row r at piece c ^ (r / 2 & 3)
                    if (whole) *reinterpret_cast<uint4*>(box + h * 2048 + lane * 64 + ((c ^ (lane >> 1 & 3)) << 4)) = piece;
                    else if (row_p >= 0) *reinterpret_cast<uint4*>(dst + 32 * h + 8 * c) = piece;
                }
            }
            tc_fence_before();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(B_OE));
                if (whole) {
                    for (int h = 0; h < boxes; ++h) tma_store_2d(&tm_out, smem_u32(box + h * 2048), x + 32 * h, it_p.x + quad * 32);
                    bulk_commit();
                }
            }
            if (row_p >= 0 && !(z == 0.f)) *not_finite = 1;
            return true;
        };

        // a unit's rows' texts and statistics are read while the unit before is worked on
        UnitStream units(p, n_units);
        int4 it = make_int4(0, 0, 0, 0), it_next = units.next();
        int2 tb = make_int2(0, 0), tb_next = text_of(it_next);
        float nl_next = 0.f, nd_next = 0.f;
        auto statistics = [&]() {
            if ((it_next.y >> 8 & 1) || r >= (it_next.y & 0xff)) return;
            const size_t at = (size_t)(it_next.y >> 16) * p.T + it_next.x + r;
            nl_next = p.plan.nlse2[at], nd_next = p.plan.ndelta[at];
        };
        statistics();
        for (int ui = 0; ui <= n_units && ok; ++ui) {
            const int4 it_p = it;
            it = it_next, tb = tb_next;
            const float nl = nl_next, nd = nd_next;
            it_next = units.next();
            tb_next = text_of(it_next);
            statistics();
            const int q_len = it.y & 0xff, k_lo = it.z, k_hi = it.w, nk = unit_tiles(it);
            const bool keys = it.y >> 8 & 1;
            int vis_lo, vis_hi;
            seen_columns(p, it, it.x + r, tb, vis_lo, vis_hi);
            const uint64_t nl2 = f2_pack(nl, nl), nd2 = f2_pack(nd, nd);
            // Columns that any row of the warp sees, and that all see: a row's first and last column never lie before those
            // of the row before.  A row behind the item's sees them all: what it adds up is not stored, and what it
            // multiplies is 0 behind the last column.
            const int rows = min(32, q_len - quad * 32);
            const int any_lo = rows > 0 ? __shfl_sync(0xffffffffu, vis_lo, 0) : INT_MAX;
            const int all_hi = __shfl_sync(0xffffffffu, vis_hi, 0);
            const int all_lo = __shfl_sync(0xffffffffu, vis_lo, max(rows, 1) - 1);
            const int any_hi = rows > 0 ? __shfl_sync(0xffffffffu, vis_hi, max(rows, 1) - 1) : INT_MIN;
            if (r >= q_len) vis_lo = INT_MIN / 2, vis_hi = INT_MAX / 2;
            // (a loop for each kind: one with both kinds' steps in branches takes 239 registers)
            auto tiles = [&](auto by_key, int kt, int end) {
                constexpr bool KEYS = decltype(by_key)::value;
                for (; kt < end; ++kt, ++t) {
                    const int b = t & 1, st = t % STAGES;
                    const int c0 = k_lo + kt * TILE + chunk * 64;
                    if (!warp_wait(B_XF + b, (t >> 1) & 1)) return false;
                    tc_fence_after();
                    const uint32_t xt = lanes + TM_X1 + b * TILE + chunk * 64;
                    if (c0 >= any_hi || c0 + 64 <= any_lo) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(B_X2R));
                        uint32_t zero[32] = {};
                        tmem_st32_u(xt, zero);
                        if (KEYS) tmem_st32_u(xt + 32, zero);
                    } else {
                        // 32 columns at a time: the operands of the outputs' products, as bf16 pairs over columns of S that
                        // this warp has read: dS and P in turn, 16 columns (8 words) of each; where rows are queries dS alone
                        constexpr int WORDS = KEYS ? 32 : 16;
                        auto word = [](int j) { return KEYS ? (j >> 3) * 16 + (j & 7) : j; };
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            uint32_t pk[WORDS];
                            const int c = c0 + 32 * h;
                            float x1[32], x2[32];
                            tmem_ld32_issue(lanes + TM_X2 + chunk * 64 + 32 * h, x2);
                            tmem_ld32_issue(xt + 32 * h, x1);
                            tmem_wait_ld();
                            tmem_tie32(x2);
                            tmem_tie32(x1);
                            if (h == 1) {
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(bar(B_X2R));
                            }
                            if (c >= any_hi || c + 32 <= any_lo) {   // no row of the warp sees any of them
#pragma unroll
                                for (int j = 0; j < WORDS; ++j) pk[j] = 0u;
                            } else {
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    const uint64_t s2 = f2_pack(x1[2 * j], x1[2 * j + 1]);
                                    uint64_t d2 = f2_pack(x2[2 * j], x2[2 * j + 1]);
                                    float e0, e1, s0, s1;
                                    f2_unpack(KEYS ? f2_mul(s2, sl2) : f2_fma(s2, sl2, nl2), e0, e1);
                                    if (!KEYS) d2 = f2_add(d2, nd2);
                                    e0 = ex2_approx(e0);
                                    e1 = ex2_approx(e1);
                                    f2_unpack(f2_mul(f2_pack(e0, e1), d2), s0, s1);
                                    pk[word(j)] = pack_bf16(s0, s1);
                                    if (KEYS) pk[word(j) + 8] = pack_bf16(e0, e1);
                                }
                                if (c < all_lo || c + 32 > all_hi) {   // columns that the row does not see, bit by bit: they may be NaN
                                    // bit k: column c + k is seen.  Four bits come to the tops of four bytes by a product (no two of
                                    // its terms meet), and a byte's top bit fills half a word
                                    const int from = min(max(vis_lo - c, 0), 32), to = min(max(vis_hi - c, 0), 32);
                                    const uint32_t seen_bits = ones_below(to) & ~ones_below(from);
#pragma unroll
                                    for (int j = 0; j < 16; j += 2) {
                                        const uint32_t tops = (seen_bits >> (2 * j) & 15u) * 0x10204080u;
                                        const uint32_t m0 = byte_signs<0x9988>(tops), m1 = byte_signs<0xbbaa>(tops);
                                        pk[word(j)] &= m0, pk[word(j + 1)] &= m1;
                                        if (KEYS) pk[word(j) + 8] &= m0, pk[word(j + 1) + 8] &= m1;
                                    }
                                }
                            }
                            if constexpr (KEYS) tmem_st32_issue(xt + 32 * h, pk);
                            else tmem_st16_issue(xt + 16 * h, pk);
                        }
                        tmem_wait_st();
                    }
                    // rows behind the last column's text (dS and P there are 0, and they may hold anything)
                    const int cols = k_hi - (k_lo + kt * TILE);
                    if (cols < TILE && k_hi < p.T) {
                        // (the copy's barrier has completed; waiting on it makes the tiles visible)
                        if (!warp_wait(B_CF + st, (t / STAGES) & 1)) return false;
                        uint4* v16 = reinterpret_cast<uint4*>(smem + OFF_COLS + st * 2 * TILE_BYTES);
                        for (int c = cols * 8 + (int)threadIdx.x - 32 * FIRST_WORKER; c < TILE * 8; c += 32 * WORKERS) {
                            v16[c] = make_uint4(0, 0, 0, 0);
                            v16[TILE * 8 + c] = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_PF + b));
                }
                return true;
            };
            // its first tile, the outputs of the unit before, the other tiles (the unit behind the last has none)
            for (int part = 0; part < 2 && ok; ++part) {
                const int from = part ? 1 : 0, to = part ? nk : min(nk, 1);
                ok = keys ? tiles(std::true_type{}, from, to) : tiles(std::false_type{}, from, to);
                if (ok && part == 0 && ui > 0) ok = finish(ui - 1, it_p);
            }
        }
    }

    if (warp >= FIRST_WORKER && lane == 0) bulk_wait_all();   // stores complete before the CTA exits
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<1>(tmem_base, TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort_flag) atomicOr(p.status, TEE_STATUS_TIMEOUT);
    if (*not_finite && !*abort_flag) bwd_again(p);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

size_t carve(int T, int n_texts, int n_heads, bool backward, void* base, AttnPlan* plan) {
    WsCarve ws(base);
    plan->n_items = ws.take<int>(1);
    plan->items = ws.take<int4>(attention_max_items(T, n_texts));
    plan->row_tb = ws.take<int2>(T);
    plan->scratch = n_texts > PLAN_SHARED_TEXTS ? ws.take<int>(3 * ((size_t)n_texts + 1)) : nullptr;
    plan->nlse2 = backward ? ws.take<float>((size_t)n_heads * T) : nullptr;
    plan->ndelta = backward ? ws.take<float>((size_t)n_heads * T) : nullptr;
    return ws.off;
}

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t s) {
    return launch_pdl(attn_plan_kernel, dim3(1 + (a.T + PLAN_ROWS - 1) / PLAN_ROWS), dim3(PLAN_THREADS), 0, s, a);
}

}  // namespace

// Whole texts: at most T / 128 whole tiles, and one more for each long text and each
// run of short ones.  Of those, the runs' tiles pair up to more than 128 tokens but for
// the last between two long texts.
int attention_max_items(int T, int n_texts) {
    const int tiles = T / TILE;
    return std::max(1, std::min(T, tiles + std::min(n_texts, 4 * tiles + 8) + 1));
}

size_t attention_train_ws(int T, int n_texts, int n_heads, bool backward) {
    AttnPlan plan;
    return carve(T, n_texts, n_heads, backward, nullptr, &plan);
}

cudaError_t launch_attention_train_forward(const void* qkv, const int32_t* cu, void* o, float* lse, int T, int n_texts,
                                           int n_heads, int window, void* ws, unsigned int* status, cudaStream_t s) {
    const int max_items = attention_max_items(T, n_texts);
    PlanArgs a{cu, T, n_texts, n_heads, window, max_items, {}, nullptr, nullptr, nullptr, status};
    carve(T, n_texts, n_heads, false, ws, &a.plan);
    const cudaError_t e = launch_plan(a, s);
    if (e != cudaSuccess) return e;
    return launch_attention_train_tc(qkv, T, n_heads, window, a.plan, max_items, o, lse, status, s);
}

cudaError_t launch_attention_train_backward(const void* qkv, const int32_t* cu, const void* o, const float* lse,
                                            const void* d_o, void* dqkv, int T, int n_texts, int n_heads, int window,
                                            void* ws, unsigned int* status, cudaStream_t s) {
    static std::mutex mu;
    static bool attr_set[TEE_MAX_DEVICES] = {};
    int dev = 0, num_sms = 0;
    cudaError_t e = tee_current_device(&dev, &num_sms);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!attr_set[dev]) {
            e = cudaFuncSetAttribute(attn_bwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_TOTAL);
            if (e != cudaSuccess) return e;
            attr_set[dev] = true;
        }
    }
    const int max_items = attention_max_items(T, n_texts), H = n_heads * HD;
    PlanArgs a{cu, T, n_texts, n_heads, window, max_items, {}, (const bf16*)o, (const bf16*)d_o, lse, status};
    carve(T, n_texts, n_heads, true, ws, &a.plan);
    CUtensorMap tm_qkv, tm_do, tm_out;
    if ((e = make_tensor_map_2d(&tm_qkv, false, qkv, T, 3 * (uint64_t)H, 3 * (uint64_t)H, TILE, HD)) != cudaSuccess) return e;
    if ((e = make_tensor_map_2d(&tm_do, false, d_o, T, H, H, TILE, HD)) != cudaSuccess) return e;
    if ((e = make_tensor_map_2d_64(&tm_out, dqkv, T, 3 * (uint64_t)H, 3 * (uint64_t)H, 32)) != cudaSuccess) return e;
    if ((e = launch_plan(a, s)) != cudaSuccess) return e;
    BwdParams p{a.plan, T, n_heads, H, window, (const bf16*)qkv, (const bf16*)d_o, (bf16*)dqkv, status};
    const int grid = (int)std::min<long long>(num_sms, 2LL * max_items * n_heads);
    return launch_pdl(attn_bwd_kernel, dim3(grid), dim3(NUM_THREADS), SMEM_TOTAL, s, tm_qkv, tm_do, tm_out, p);
}
