// Varlen bidirectional attention on the 5th-generation tensor cores (sm_103a).
//
// Method: tensai page "テキスト埋め込み", §何が動くか / エンコーダ and its packing
// paragraph: every query attends only to keys of its own text -- all of them on
// the global layers (layer 0 and every third), |i - j| <= 64 on the others --
// with scores q.k / sqrt(64) and a softmax over the allowed keys.
//
// Work unit = (128-query tile, head).  The host lists the query tiles with
// their key range [k_lo, k_hi): on global layers the tiles of each text (keys =
// the text), with consecutive texts that together span at most 128 tokens
// sharing one tile, longest first; on window layers the tiles of the packed
// sequence itself.  Where texts share a tile, every row is masked to its own
// text through the per-token text bounds row_tb.  The
// kernel is persistent: one CTA per SM walks its own list of units, which the
// host balances (longest first, each to the least-loaded CTA).  Ten warps:
//   warp 0 lane 0   TMA: each unit's Q tile (double-buffered, so the next
//                   unit's Q arrives early), then its K and V tiles (128 keys)
//                   into a KV_STAGES-deep ring, straight from the packed qkv
//                   rows;
//   warp 1          TMEM allocation; issues S_t = Q K_t^T (M=128, N=128,
//                   K=64) into TMEM S/P buffer t % 3, and O += P_t V_t (M=128,
//                   N=64, K=128) with P read from the first 64 columns of the
//                   same buffer (the A operand, written there by the softmax
//                   over S_t) and V from shared memory as an MN-major operand
//                   (no transpose), into the unit's TMEM O buffer (two, by
//                   unit).  P V runs two tiles behind S, across unit
//                   boundaries too, so S_{t+1} is ready when the softmax
//                   finishes tile t; the MMAs of one thread run in order, so
//                   S_{t+3} overwrites buffer t % 3 only after P_t V_t read it.
//                   The whole warp runs the loop and one lane issues, which
//                   keeps descriptors in uniform registers: eight P V MMAs
//                   take 300 cycles so, 575 from one lane's own loop (window
//                   layer of 32768 tokens 74 -> 65 us, 8 x 8192 tokens 2.34 ->
//                   1.93 ms); a barrier found done is left by one vote (1.81
//                   -> 1.79 ms);
//   warps 2-9       two threads per query row (a warp may read only its
//                   32-lane TMEM quadrant, so warps w and w+4 share one and
//                   split the 128 key columns, and the 64 output dimensions,
//                   in halves): one 64-column TMEM load of S, the mask as a
//                   per-row interval of visible keys (on window layers first
//                   decided for the whole warp per 32-column block: a block
//                   that no row sees is skipped, one that every row sees is
//                   not masked), the tile's row maximum
//                   exchanged through shared memory with a pair barrier, the
//                   softmax in fp32 with exp2 (scale folded into one FMA)
//                   against a reference maximum that moves only when a tile's
//                   maximum exceeds it by more than 2^8 (then that row of O is
//                   rescaled in TMEM), P as bf16 pairs stored into TMEM for the
//                   P V MMA (bf16 pairs written over the tile's first 64 S
//                   columns, once both warps of the pair have read theirs); a
//                   unit's O / l is read after the next unit's first P hand-off
//                   and leaves as bf16 by bulk copies of 32 whole rows (row by
//                   row from the threads a store touches 32 lines: 65 -> 59 us
//                   and 1.93 -> 1.80 ms).
// Pipeline counters run across units; every wait is bounded.
#include "gemm_tc.cuh"
#include "train_internal.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "tc_ptx.cuh"

namespace {

using namespace tc;

constexpr int BQ = 128;
constexpr int BKV = 128;
constexpr int HD = 64;
constexpr int KV_STAGES = 5;
constexpr int NUM_THREADS = 320;
constexpr int SM_THREADS = 256;   // softmax warps 2..9
constexpr uint32_t TILE_BYTES = BQ * HD * 2;        // Q, K or V tile: 16 KB
constexpr uint32_t OFF_Q = 0;                       // 2 Q buffers
constexpr uint32_t OFF_K = OFF_Q + 2 * TILE_BYTES;
constexpr uint32_t OFF_V = OFF_K + KV_STAGES * TILE_BYTES;
constexpr uint32_t OFF_BAR = OFF_V + KV_STAGES * TILE_BYTES;
// barrier indices
constexpr int SP_BUFS = 3;   // TMEM S/P buffers: tile t uses buffer t % 3
constexpr int B_QF = 0, B_QE = 2, B_KVF = 4, B_KVE = B_KVF + KV_STAGES, B_SF = B_KVE + KV_STAGES,
              B_PF = B_SF + SP_BUFS, B_OE = B_PF + SP_BUFS, B_DONE = B_OE + 2, N_BARS = B_DONE + 1;
// (behind the barriers three words: the tensor memory's address and two flags)
constexpr uint32_t OFF_RED = OFF_BAR + N_BARS * 8 + 16;       // row-maximum exchange: [2 tiles][2 halves][128 rows]
constexpr uint32_t OFF_REDL = OFF_RED + 2 * 2 * 128 * 4;       // row-sum exchange: [2 units][2 halves][128 rows]
constexpr uint32_t OFF_OUT = (OFF_REDL + 2 * 2 * 128 * 4 + 1023) / 1024 * 1024;   // a 2 KB box per softmax warp: 32 rows of 64 bytes
constexpr uint32_t SMEM_TOTAL = OFF_OUT + 8 * 2048 + 1024;
static_assert(SMEM_TOTAL <= 227 * 1024, "shared memory");
constexpr uint32_t TMEM_COLS = 512;                 // S/P: 3 x 128 columns (by tile), O: 2 x 64 (by unit)
constexpr uint32_t TM_S = 0, TM_O = SP_BUFS * BKV;

struct AttnParams {
    const int4* slots;      // {q_start, q_len | head << 16, k_lo, k_hi} per unit, CTA after CTA
    const int* slot_off;    // CTA c takes slots slot_off[c] .. slot_off[c + 1]
    const int2* row_tb;     // per token: {start, end} of its text
    int hidden;
    int window;
    float scale_log2;       // log2(e) / sqrt(64)
    bf16* o;                // [T, hidden]
    unsigned int* status;
    // TRAIN: slots holds *n_items work items without a head; every CTA takes the units
    // (item, head) that attn_unit gives it
    const int* n_items;
    int n_heads, T;
    float* lse;             // [n_heads, T]
    const bf16* qkv;
};

__device__ __forceinline__ int n_kv_tiles(const int4& it) { return (it.w - it.z + BKV - 1) / BKV; }

// Row maximum of columns [B, E) of a thread's 64 scores, as eight partial
// maxima (partial k over the columns = k mod 8; short dependency chains),
// three scores per max instruction.
template <int B, int E>
__device__ __forceinline__ void max8(const float* v, float* m8) {
    static_assert((E - B) % 16 == 0, "whole groups of two per partial");
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float m = fmaxf(v[B + k], v[B + k + 8]);
#pragma unroll
        for (int i = B + k + 16; i < E; i += 16) m = fmax3(m, v[i], v[i + 8]);
        m8[k] = m;
    }
}

// Eight partial row sums as four fp32x2 pairs: pair c & 3 takes columns 2c and
// 2c + 1, so partial k again sums the columns = k mod 8.
struct RowSum8 {
    uint64_t s[4];
    __device__ void zero() {
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] = 0ull;
    }
    __device__ float total() const {
        float a[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) f2_unpack(s[k], a[2 * k], a[2 * k + 1]);
        return ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
    }
};

// p = 2^(s * scale_log2 - m) over columns [B, E): added to the partial row
// sums and packed as bf16 pairs (pk[c] holds columns 2c, 2c + 1).
template <int B, int E>
__device__ __forceinline__ void exp_pack(float* v, uint64_t sl2x2, uint64_t negm2, RowSum8& rs, uint32_t* pk) {
#pragma unroll
    for (int c = B / 2; c < E / 2; ++c) {
        float a, b;
        f2_unpack(f2_fma(f2_pack(v[2 * c], v[2 * c + 1]), sl2x2, negm2), a, b);
        a = ex2_approx(a);
        b = ex2_approx(b);
        rs.s[c & 3] = f2_add(rs.s[c & 3], f2_pack(a, b));
        pk[c] = pack_bf16(a, b);
    }
}

template <int B, int E>
__device__ __forceinline__ void zero_pack(uint32_t* pk) {
#pragma unroll
    for (int c = B / 2; c < E / 2; ++c) pk[c] = 0u;
}

// Takes those of 32 scores out that are not of columns [lo, hi): a bit for each, one
// test instead of two comparisons (training forward, window layer of 32768 tokens: 58.7 -> 55.5 us).
__device__ __forceinline__ void mask32(float* v, int lo, int hi) {
    const uint32_t seen = ones_below(min(max(hi, 0), 32)) & ~ones_below(min(max(lo, 0), 32));
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (!(seen >> i & 1)) v[i] = -INFINITY;
}

// A CTA's units in turn, i0 .. i1 - 1; none behind the last.
template <bool TRAIN>
struct Slots {
    const AttnParams& p;
    int i, i1;
    __device__ __forceinline__ Slots(const AttnParams& p_, int i0, int i1_) : p(p_), i(i0), i1(i1_) {}
    __device__ __forceinline__ int4 next() { return i < i1 ? p.slots[i++] : make_int4(0, 0, 0, 0); }
};
// Training: from unit to unit (attn_unit) the steps are two in turn, so one division each
// does for all.
template <>
struct Slots<true> {
    const AttnParams& p;
    int i, i1, item, head, step_item[2], step_head[2];
    __device__ __forceinline__ Slots(const AttnParams& p_, int i0, int i1_) : p(p_), i(i0), i1(i1_) {
        const int c = blockIdx.x, G = gridDim.x, heads = p.n_heads;
        item = c / heads, head = c - item * heads;
        step_item[0] = (2 * (G - c) - 1) / heads, step_head[0] = 2 * (G - c) - 1 - step_item[0] * heads;
        step_item[1] = (2 * c + 1) / heads, step_head[1] = 2 * c + 1 - step_item[1] * heads;
    }
    __device__ __forceinline__ int4 next() {
        if (i >= i1) return make_int4(0, 0, 0, 0);
        int4 it = p.slots[item];
        it.y |= head << 16;
        item += i & 1 ? step_item[1] : step_item[0];
        head += i & 1 ? step_head[1] : step_head[0];
        if (head >= p.n_heads) head -= p.n_heads, ++item;
        ++i;
        return it;
    }
};

// The keys that a row of an item sees, its text being {tb.x, tb.y}: the window inside the
// text, or on global layers the text (of the item's where short texts share a tile).
template <bool WINDOW>
__device__ __forceinline__ void seen_keys(const AttnParams& p, const int4& it, int row, const int2& tb, int& lo, int& hi) {
    if constexpr (WINDOW) lo = max(tb.x, row - p.window), hi = min(tb.y, row + p.window + 1);
    else lo = max(it.z, tb.x), hi = min(it.w, tb.y);
}

// The output of one row again, from its own keys [lo, hi), outside the tensor cores, by a
// whole warp: four keys side by side, eight lanes to each, the loads of four such steps on
// their way together.  It ends early where nothing but NaN can come.
__device__ __noinline__ void attn_row_again(const AttnParams& p, int row, int head, int lo, int hi, float lse2) {
    constexpr int AT_ONCE = 4;
    const int lane = threadIdx.x & 31, part = lane >> 3, col = (lane & 7) * 8;
    const size_t stride = 3 * (size_t)p.hidden;
    const bf16* at = p.qkv + head * HD + col;
    float q[8], o[8] = {};
    load_vec(at + row * stride, q);
    for (int j0 = lo; j0 < hi; j0 += 4 * AT_ONCE) {
        uint4 k4[AT_ONCE], v4[AT_ONCE];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            const bf16* kv = at + min(j0 + 4 * u + part, hi - 1) * stride + p.hidden;
            k4[u] = *reinterpret_cast<const uint4*>(kv);
            v4[u] = *reinterpret_cast<const uint4*>(kv + p.hidden);
        }
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            float k[8], v[8], s = 0.f;
            unpack_bf16x8(k4[u], k);
            unpack_bf16x8(v4[u], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
            for (int d = 4; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (j0 + 4 * u + part < hi) {
                const float e = ex2_approx(fmaf(s, p.scale_log2, -lse2));
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = fmaf(e, v[i], o[i]);
            }
        }
        if (each_eighth_has(all_nan(o))) break;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        o[i] += __shfl_xor_sync(0xffffffffu, o[i], 8);
        o[i] += __shfl_xor_sync(0xffffffffu, o[i], 16);
    }
    if (part == 0) store_vec(p.o + (size_t)row * p.hidden + head * HD + col, o);
}

// Rows whose products met NaN or infinities of keys that they do not see (their probability
// is 0, but 0 x NaN is NaN) are computed again, once all of the CTA's units are done and no
// role waits for another any more: 131072 keys for each of a tile's rows would come near the
// bound of the waits.  Every warp goes through a quarter of every few units, a lane to a row:
// not rows that see all of the item's keys, whose NaN are their own, and not those that
// cannot have another output: NaN in the log sum (or -infinity, as of scores that are all
// that), or a value row that is nothing but NaN.
template <bool WINDOW>
__device__ __noinline__ void attn_again(const AttnParams& p, int units) {
    const int lane = threadIdx.x & 31;
    for (int task = threadIdx.x >> 5; task < 4 * units; task += NUM_THREADS / 32) {
        const int unit = attn_unit(task >> 2, blockIdx.x, gridDim.x), head = unit % p.n_heads;
        const int4 it = p.slots[unit / p.n_heads];
        const int r = (task & 3) * 32 + lane, row = it.x + r;
        int lo = 0, hi = 0;
        float lse2 = 0.f;
        bool mine = r < it.y;
        if (mine) {
            seen_keys<WINDOW>(p, it, row, p.row_tb[row], lo, hi);
            lse2 = p.lse[(size_t)head * p.T + row] * 1.4426950408889634f;
            mine = (lo > it.z || hi < it.w) && lse2 > -INFINITY;
        }
        if (mine) mine = !all_finite(p.o + (size_t)row * p.hidden + head * HD);
        if (mine) mine = !all_nan(p.qkv + (size_t)row * 3 * p.hidden + 2 * p.hidden + head * HD);
        for (unsigned again = __ballot_sync(0xffffffffu, mine); again; again &= again - 1) {
            const int l = __ffs(again) - 1;
            attn_row_again(p, __shfl_sync(0xffffffffu, row, l), head, __shfl_sync(0xffffffffu, lo, l),
                           __shfl_sync(0xffffffffu, hi, l), __shfl_sync(0xffffffffu, lse2, l));
        }
    }
}

// WINDOW: the ±window layers (per-row text bounds, 32-column block skipping);
// otherwise the global layers, whose rows all see the same keys.
// TRAIN: the training operator (tee_train.h): work items planned on the device, the
// rows' log sums written beside their outputs, and rows that see no trace of what lies
// outside their text: rows of V behind the item's keys are zeroed in shared memory
// (they may be anything, also behind the last text), and a row that is not finite, in
// items whose rows see different keys, is computed again from its own (attn_again).
template <bool WINDOW, bool TRAIN>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm_o,
                   const __grid_constant__ AttnParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + N_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* not_finite = abort_flag + 1;   // TRAIN: some output is not
    auto bar = [&](int i) { return smem_u32(bars + i); };

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(B_QF + b), 1);
            mbar_init(bar(B_QE + b), 1);
            mbar_init(bar(B_OE + b), SM_THREADS);
        }
        for (int b = 0; b < SP_BUFS; ++b) {
            mbar_init(bar(B_SF + b), 1);
            mbar_init(bar(B_PF + b), SM_THREADS);
        }
        for (int s = 0; s < KV_STAGES; ++s) {
            mbar_init(bar(B_KVF + s), 1);
            mbar_init(bar(B_KVE + s), 1);
        }
        mbar_init(bar(B_DONE), 1);
        *abort_flag = 0;
        if constexpr (TRAIN) *not_finite = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm)) : "memory");
    }
    if (warp == 1) tmem_alloc<1>(smem_u32(tmem_slot), TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // the prologue above may overlap the previous kernel; global memory only after it completes
    pdl_wait();
    pdl_trigger();

    // this CTA's units
    int i0 = 0, i1;
    if constexpr (TRAIN) {
        i1 = attn_units_of(*p.n_items * p.n_heads, blockIdx.x, gridDim.x);
    } else {
        i0 = p.slot_off[blockIdx.x], i1 = p.slot_off[blockIdx.x + 1];
    }

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        if (lane == 0) {
            bool q_armed[2] = {false, false}, kv_armed[KV_STAGES] = {};
            uint32_t q_par[2] = {0, 0}, kv_par[KV_STAGES] = {};
            uint32_t g = 0;   // KV tiles issued
            int ui = 0;
            bool ok = true;
            Slots<TRAIN> slots(p, i0, i1);
            int4 it_next = slots.next();   // units are read one ahead
            for (int i = i0; i < i1 && ok; ++i, ++ui) {
                const int4 it = it_next;
                it_next = slots.next();
                const int head = it.y >> 16;
                const int nk = n_kv_tiles(it);
                const int qb = ui & 1;
                if (!mbar_wait(bar(B_QE + qb), ((ui >> 1) & 1) ^ 1, abort_flag)) break;
                mbar_expect_tx(bar(B_QF + qb), TILE_BYTES);
                tma_load_2d(sbase + OFF_Q + qb * TILE_BYTES, &tm, head * HD, it.x, bar(B_QF + qb));
                q_armed[qb] = true;
                q_par[qb] = (ui >> 1) & 1;
                const int xk = p.hidden + head * HD, xv = 2 * p.hidden + head * HD;
                for (int kt = 0; kt < nk; ++kt, ++g) {
                    const int s = g % KV_STAGES;
                    const uint32_t r = g / KV_STAGES;
                    if (!mbar_wait(bar(B_KVE + s), (r & 1) ^ 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const int y = it.z + kt * BKV;
                    mbar_expect_tx(bar(B_KVF + s), 2 * TILE_BYTES);
                    tma_load_2d(sbase + OFF_K + s * TILE_BYTES, &tm, xk, y, bar(B_KVF + s));
                    tma_load_2d(sbase + OFF_V + s * TILE_BYTES, &tm, xv, y, bar(B_KVF + s));
                    kv_armed[s] = true;
                    kv_par[s] = r & 1;
                }
            }
            for (int b = 0; b < 2; ++b)
                if (q_armed[b]) mbar_wait_drain(bar(B_QF + b), q_par[b]);
            for (int s = 0; s < KV_STAGES; ++s)
                if (kv_armed[s]) mbar_wait_drain(bar(B_KVF + s), kv_par[s]);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issuer (the whole warp, one lane issuing: addresses and descriptors stay uniform) ----------------
        constexpr uint32_t idesc_s = make_idesc(BQ, BKV);
        constexpr uint32_t idesc_pv = make_idesc(BQ, HD) | IDESC_B_MN_MAJOR;
        const uint64_t q0desc = sw128_desc(sbase + OFF_Q), k0desc = sw128_desc(sbase + OFF_K);
        const uint64_t v0desc = sw128_desc_mn(sbase + OFF_V);
        constexpr uint32_t TILE_DESC = TILE_BYTES >> 4;
        auto wait = [&](int b, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_try_wait(bar(b), parity)) ||
                   __all_sync(0xffffffffu, mbar_wait(bar(b), parity, abort_flag));
        };
        // P_tt V_tt accumulated into the unit's TMEM O buffer; the first
        // tile of a unit overwrites it once the softmax warps have read the
        // unit two back out of that buffer
        auto issue_pv = [&](uint32_t tt, bool first, int ub, uint32_t uuse) -> bool {
            const uint32_t sb = tt % SP_BUFS, st = tt % KV_STAGES;
            if (!wait(B_PF + sb, (tt / SP_BUFS) & 1)) return false;
            if (first && !wait(B_OE + ub, (uuse & 1) ^ 1)) return false;
            tc_fence_after();
            const uint32_t pbase = tmem_base + TM_S + sb * BKV, obase = tmem_base + TM_O + ub * HD;
            const uint64_t vdesc = v0desc + st * TILE_DESC;
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < BKV / 16; ++s)
                    mma_bf16_ts(obase, pbase + 8 * s, vdesc + s * 128, idesc_pv, !(first && s == 0));
                // one commit frees the K/V stage and tells the softmax warps
                // that P_tt V_tt is in O
                mma_commit(bar(B_KVE) + 8 * st);
            }
            __syncwarp();
            return true;
        };
        struct Pend {
            uint32_t t, use;
            bool first;
            int ub;
        };
        Pend q0{}, q1{};         // tiles whose S is issued and whose P V is not (at most two)
        int nq = 0;
        uint32_t t = 0;          // tiles whose S has been issued (global)
        bool ok = true;
        int ui = 0;
        Slots<TRAIN> slots(p, i0, i1);
        int4 it_next = slots.next();
        for (int i = i0; i < i1 && ok; ++i, ++ui) {
            const int nk = n_kv_tiles(it_next);
            it_next = slots.next();
            const int qb = ui & 1;
            if (!wait(B_QF + qb, (ui >> 1) & 1)) break;
            const uint64_t qdesc = q0desc + qb * TILE_DESC;
            for (int kt = 0; kt < nk; ++kt, ++t) {
                // buffer t % 3 last held tile t - 3, whose P V was issued
                // before this S (and runs before it): no wait for it here
                const uint32_t st = t % KV_STAGES, sb = t % SP_BUFS;
                if (!wait(B_KVF + st, (t / KV_STAGES) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t kdesc = k0desc + st * TILE_DESC;
                const uint32_t sbuf = tmem_base + TM_S + sb * BKV;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k) mma_bf16(sbuf, qdesc + 2 * k, kdesc + 2 * k, idesc_s, k != 0);
                    mma_commit(bar(B_SF) + 8 * sb);
                    if (kt == nk - 1) mma_commit(bar(B_QE) + 8 * qb);   // Q buffer free once these S MMAs finish
                }
                __syncwarp();
                const Pend cur{t, (uint32_t)ui >> 1, kt == 0, ui & 1};
                if (nq == 2) {   // P V two tiles behind S
                    if (!issue_pv(q0.t, q0.first, q0.ub, q0.use)) {
                        ok = false;
                        break;
                    }
                    q0 = q1;
                    q1 = cur;
                } else if (nq == 1) {
                    q1 = cur;
                    nq = 2;
                } else {
                    q0 = cur;
                    nq = 1;
                }
            }
        }
        if (ok && nq >= 1) ok = issue_pv(q0.t, q0.first, q0.ub, q0.use);
        if (ok && nq == 2) ok = issue_pv(q1.t, q1.first, q1.ub, q1.use);
        if (elect_one()) mma_commit(bar(B_DONE));
        __syncwarp();
        mbar_wait_drain(bar(B_DONE), 0);
    } else {
        // ---------------- softmax / output (warps 2..9) ----------------
        // Warps w and w + 4 share a TMEM lane quadrant (rows 32*quad ..) and
        // split each tile's 128 key columns; the tile's row maximum is exchanged
        // through shared memory.  P V accumulates in TMEM across the unit's key
        // tiles against a reference maximum m_ref that moves only when a tile's
        // maximum exceeds it by more than RESCALE_LOG2 (then the row of O is
        // rescaled in TMEM), so most tiles touch no O at all.
        constexpr float RESCALE_LOG2 = 8.0f;
        const int quad = warp & 3;
        const int half = (warp - 2) >> 2;               // key columns [64*half, +64), O columns [32*half, +32)
        const int r = quad * 32 + lane;                 // query row of the tile
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        float* red = reinterpret_cast<float*>(smem + OFF_RED);   // [2][2][128]
        float* red_l = reinterpret_cast<float*>(smem + OFF_REDL);   // [2][2][128]
        const uint32_t pair_bar = 1 + quad;             // named barrier of warps (w, w + 4)
        const float sl2 = p.scale_log2;
        const uint64_t sl2x2 = f2_pack(sl2, sl2);
        uint32_t t = 0;
        bool ok = true;

        auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory"); };
        // P_tt V_tt is in O once tile tt's K/V stage is released (the commit
        // after that P V).  The wait's parity cannot alias: it is asked for
        // after the S of tile tt was seen ready, and that S was issued after
        // the P V of tile tt - 3, so the stage's previous phase (tile tt - 5)
        // is complete; its next phase needs the P of tile tt + 5, which these
        // warps have not yet written.
        auto pv_done = [&](uint32_t tt) -> bool {
            return mbar_wait(bar(B_KVE + tt % KV_STAGES), (tt / KV_STAGES) & 1, abort_flag);
        };

        // The previous unit's output, deferred past the next unit's first
        // softmax: wait for its last P V, read this warp's 32 columns of O,
        // release the buffer, store O / l.  The pair's two halves of the row
        // sum l travel with the next unit's first row-maximum exchange (slot
        // by the unit's O buffer, so a slot is rewritten only after both warps
        // have passed a later exchange); the last unit exchanges them itself.
        bool pend = false;
        float l_p = 0.f, l_tot_p = 0.f;
        uint32_t t_p = 0;
        int ub_p = 0;
        bool row_is_p = false;                // the unit has the row
        int row_p = 0, head_p = 0, q_len_p = 0;
        float m_p = 0.f;                      // TRAIN: the unit's reference maximum
        uint8_t* const box = smem + OFF_OUT + (warp - 2) * 2048;
        auto finalize = [&](bool exchanged) -> bool {
            if (!pv_done(t_p)) return false;
            tc_fence_after();
            float o[32];
            tmem_ld32(tmem_base + lane_off + TM_O + ub_p * HD + half * 32, o);
            tc_fence_before();
            mbar_arrive(bar(B_OE + ub_p));
            if (!exchanged) {
                red_l[(ub_p * 2 + half) * 128 + r] = l_p;
                pair_sync();
                l_tot_p = l_p + red_l[(ub_p * 2 + (half ^ 1)) * 128 + r];
            }
            const float inv = 1.0f / l_tot_p;
#pragma unroll
            for (int d = 0; d < 32; ++d) o[d] *= inv;
            // 32 whole rows leave as one bulk copy (row by row from the threads, each store touches 32 lines)
            if (quad * 32 + 32 <= q_len_p) {
                if (lane == 0) bulk_wait_read<0>();   // the box's last copy has read it
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 4; ++c) {         // 64-byte swizzle: 16-byte piece c of row r at piece c ^ (r / 2 & 3)
                    uint4 q;
                    q.x = pack_bf16(o[8 * c + 0], o[8 * c + 1]);
                    q.y = pack_bf16(o[8 * c + 2], o[8 * c + 3]);
                    q.z = pack_bf16(o[8 * c + 4], o[8 * c + 5]);
                    q.w = pack_bf16(o[8 * c + 6], o[8 * c + 7]);
                    *reinterpret_cast<uint4*>(box + lane * 64 + ((c ^ (lane >> 1 & 3)) << 4)) = q;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(&tm_o, smem_u32(box), head_p * HD + half * 32, row_p);
                    bulk_commit();
                }
            } else if (row_is_p) {
                store_bf16x32(p.o + (size_t)row_p * p.hidden + head_p * HD + half * 32, o);
            }
            if constexpr (TRAIN) {
                const float lse2 = m_p + log2f(l_tot_p);
                if (row_is_p && half == 0) p.lse[(size_t)head_p * p.T + row_p] = lse2 * 0.69314718055994531f;
                float z = 0.f;                // not a number where one of the row's outputs is not finite
#pragma unroll
                for (int d = 0; d < 32; ++d) z = fmaf(o[d], 0.f, z);
                if (row_is_p && !(z == 0.f)) *not_finite = 1;
            }
            pend = false;
            return true;
        };

        // Work items are read two units ahead and the row's text bounds one
        // unit ahead, so neither load's latency lands on a unit's first tile.
        auto row_bounds = [&](const int4& x) -> int2 {
            return r < (x.y & 0xffff) ? p.row_tb[x.x + r] : make_int2(0, 0);
        };
        int ui = 0;
        Slots<TRAIN> slots(p, i0, i1);
        int4 it_next = slots.next(), it_next2 = slots.next();
        int2 tb_next = row_bounds(it_next);
        for (int i = i0; i < i1 && ok; ++i, ++ui) {
            const int4 it = it_next;
            const int2 tb = tb_next;
            it_next = it_next2;
            if (i + 1 < i1) tb_next = row_bounds(it_next);
            it_next2 = slots.next();
            const int head = it.y >> 16;
            const int q_start = it.x, q_len = it.y & 0xffff, k_lo = it.z, k_hi = it.w;
            const int nk = n_kv_tiles(it);
            const int qg = q_start + r;
            const int ub = ui & 1;
            // keys visible to this row: [vis_lo, vis_hi) -- the row's text on
            // global layers, the window inside the row's own text otherwise
            // (nothing for window rows past the end of the sequence).  As seen_keys says
            // it; called here, 8 x 8192 tokens take 1.777 ms instead of 1.771
            int vis_lo = k_lo, vis_hi = k_hi;
            if constexpr (WINDOW) {
                if (r < q_len) {
                    vis_lo = max(tb.x, qg - p.window);
                    vis_hi = min(tb.y, qg + p.window + 1);
                } else {
                    vis_hi = vis_lo;
                }
            } else if (r < q_len) {   // a tile shared by short texts: the row's own text
                vis_lo = max(k_lo, tb.x);
                vis_hi = min(k_hi, tb.y);
            }
            float m_ref = -INFINITY, l = 0.f;
            for (int kt = 0; kt < nk; ++kt, ++t) {
                const int sb = t % SP_BUFS;
                const int key0 = k_lo + kt * BKV + half * 64;
                const int lo = vis_lo - key0, hi = vis_hi - key0;   // visible columns [lo, hi)
                // Window layers: the warp's 64 columns as two 32-column blocks,
                // each decided for the whole warp (before S is ready: the
                // decision needs no score): no row sees a key of it (skipped:
                // no maximum, no exponentials, P = 0), every row sees all of it
                // (no mask), or a mixed block (masked per element).  The band
                // crosses one mixed block per pair of warps and tile.  Global
                // layers: every block counts as seen (a tile past the text's
                // end is masked per element).
                bool any0 = true, any1 = true, all0 = true, all1 = true;
                if constexpr (WINDOW) {
                    any0 = __any_sync(0xffffffffu, lo < hi && lo < 32 && hi > 0);
                    any1 = __any_sync(0xffffffffu, lo < hi && lo < 64 && hi > 32);
                    all0 = __all_sync(0xffffffffu, lo <= 0 && hi >= 32);
                    all1 = __all_sync(0xffffffffu, lo <= 32 && hi >= 64);
                }
                if (!mbar_wait(bar(B_SF + sb), (t / SP_BUFS) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                float v[64];
                tmem_ld64(tmem_base + lane_off + TM_S + sb * BKV + half * 64, v);
                if constexpr (WINDOW) {
                    if (any0 && !all0) {
                        mask32(v + 0, lo - 0, hi - 0);
                    }
                    if (any1 && !all1) {
                        mask32(v + 32, lo - 32, hi - 32);
                    }
                } else if (lo > 0 || hi < 64) {
                    mask32(v, lo, hi);
                    mask32(v + 32, lo - 32, hi - 32);
                }
                // row maximum and (below) row sum over eight independent
                // partials: short dependency chains for the latency-bound warps
                float m8[8];
                if (any0 && any1) {
                    max8<0, 64>(v, m8);
                } else if (any0) {
                    max8<0, 32>(v, m8);
                } else if (any1) {
                    max8<32, 64>(v, m8);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) m8[k] = -INFINITY;
                }
                float mx = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
                float* red_t = red + (t & 1) * 256;
                red_t[half * 128 + r] = mx;
                const bool carry_l = kt == 0 && pend;   // the previous unit's row sum rides along
                if (carry_l) red_l[(ub_p * 2 + half) * 128 + r] = l_p;
                pair_sync();
                mx = fmaxf(mx, red_t[(half ^ 1) * 128 + r]) * sl2;
                if (carry_l) l_tot_p = l_p + red_l[(ub_p * 2 + (half ^ 1)) * 128 + r];
                if (kt == 0) {
                    m_ref = mx;
                } else {
                    // both warps of the pair see the same row maxima, so they
                    // agree on which rows (and so whether the warp) rescale
                    const bool need = mx > m_ref + RESCALE_LOG2;
                    if (__any_sync(0xffffffffu, need)) {
                        const float corr = need ? ex2_approx(m_ref - mx) : 1.0f;
                        // P V of the previous tile must be in O before it is rescaled
                        if (!pv_done(t - 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        float o[32];
                        const uint32_t oaddr = tmem_base + lane_off + TM_O + ub * HD + half * 32;
                        tmem_ld32(oaddr, o);
#pragma unroll
                        for (int d = 0; d < 32; ++d) o[d] *= corr;
                        tmem_st32(oaddr, o);
                        tc_fence_before();
                        if (need) {
                            l *= corr;
                            m_ref = mx;
                        }
                    }
                }
                const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
                const uint64_t negm2 = f2_pack(-m_use, -m_use);
                RowSum8 rs;
                rs.zero();
                // P as bf16 pairs over the tile's first 64 S columns (the A
                // operand of P V): this half's 64 keys are columns [32 * half,
                // +32).  Both warps of the pair have read their S (the row
                // maximum exchange above), so overwriting the other half's S
                // columns is safe.
                uint32_t pk[32];
                if (any0 && any1) {   // one loop over all 64 columns: the common case on global layers
                    exp_pack<0, 64>(v, sl2x2, negm2, rs, pk);
                } else {
                    if (any0) exp_pack<0, 32>(v, sl2x2, negm2, rs, pk);
                    else zero_pack<0, 32>(pk);
                    if (any1) exp_pack<32, 64>(v, sl2x2, negm2, rs, pk);
                    else zero_pack<32, 64>(pk);
                }
                const float sum = rs.total();
                if constexpr (TRAIN) {
                    // rows of V behind the keys (P there is 0, and they may hold anything): whole 128-byte rows of the tile.
                    // The copy's barrier has completed (S was made from the same stage); waiting on it makes V visible.
                    const int keys = k_hi - (k_lo + kt * BKV);
                    if (keys < BKV && k_hi < p.T) {
                        const int st = t % KV_STAGES;
                        if (!mbar_wait(bar(B_KVF + st), (t / KV_STAGES) & 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        uint4* v16 = reinterpret_cast<uint4*>(smem + OFF_V + st * TILE_BYTES);
                        for (int c = keys * 8 + (int)threadIdx.x - 64; c < BKV * 8; c += SM_THREADS) v16[c] = make_uint4(0, 0, 0, 0);
                        fence_proxy_async_smem();
                    }
                }
                tmem_st32_u(tmem_base + lane_off + TM_S + sb * BKV + half * 32, pk);
                tc_fence_before();
                mbar_arrive(bar(B_PF + sb));
                l += sum;
                // the previous unit's output, once this tile's P is handed over
                if (kt == 0 && pend && !finalize(true)) {
                    ok = false;
                    break;
                }
            }
            if (!ok) break;
            l_p = l;
            t_p = t - 1;
            ub_p = ub;
            row_is_p = r < q_len;
            row_p = qg, head_p = head, q_len_p = q_len;
            if constexpr (TRAIN) {
                m_p = m_ref;
            }
            pend = true;
        }
        if (ok && pend) ok = finalize(false);
        // A warp that gave up on a bounded wait leaves with one arrival on its
        // pair barrier, so a partner already waiting there is released (and
        // next sees the abort flag at its next, bounded, wait: every path
        // between two pair barriers passes one).  Unawaited, it is harmless.
        if (!ok) asm volatile("bar.arrive %0, 64;" ::"r"(pair_bar) : "memory");
        if (lane == 0) bulk_wait_all();   // stores complete before the CTA exits
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<1>(tmem_base, TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort_flag && p.status) atomicOr(p.status, TEE_STATUS_TIMEOUT);
    if constexpr (TRAIN) {
        if (*not_finite && !*abort_flag) attn_again<WINDOW>(p, i1);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_once;
cudaError_t g_init_err = cudaSuccess;
std::mutex g_attr_mu;
bool g_attr_set[TEE_MAX_DEVICES] = {};   // the kernel's shared-memory attribute, per device

void init_once() {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn) {
        g_init_err = e != cudaSuccess ? e : cudaErrorNotSupported;
        return;
    }
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
}

}  // namespace

namespace {

// Tensor map and attributes of a launch on the current device.
cudaError_t prepare_launch(const void* qkv, int T, int H, const void* o, CUtensorMap* tm, CUtensorMap* tm_o, int* num_sms) {
    std::call_once(g_once, init_once);
    if (g_init_err != cudaSuccess) return g_init_err;
    if ((reinterpret_cast<uintptr_t>(qkv) & 15) || (reinterpret_cast<uintptr_t>(o) & 15)) return cudaErrorInvalidValue;
    cuuint64_t dims[2] = {(cuuint64_t)3 * H, (cuuint64_t)T};
    cuuint64_t strides[1] = {(cuuint64_t)3 * H * 2};
    cuuint32_t box[2] = {(cuuint32_t)HD, (cuuint32_t)BQ};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = g_encode(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(qkv), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
    cudaError_t e = make_tensor_map_2d_64(tm_o, o, T, H, H, 32);
    if (e != cudaSuccess) return e;
    int dev = 0;
    e = tee_current_device(&dev, num_sms);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_attr_mu);
    if (!g_attr_set[dev]) {
        for (auto kernel : {attn_tc_kernel<true, false>, attn_tc_kernel<false, false>, attn_tc_kernel<true, true>,
                            attn_tc_kernel<false, true>}) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_TOTAL);
            if (e != cudaSuccess) return e;
        }
        g_attr_set[dev] = true;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_attention_tc(const void* qkv, int T, int H, int n_heads, const int4* d_slots,
                                const int32_t* d_slot_off, int grid, bool is_global, int window, const int2* row_tb,
                                void* o, unsigned int* status, cudaStream_t s) {
    if (grid == 0 || T == 0) return cudaSuccess;
    if (H != n_heads * HD) return cudaErrorInvalidValue;
    if (!row_tb || !d_slots || !d_slot_off || grid < 0) return cudaErrorInvalidValue;
    CUtensorMap tm, tm_o;
    int num_sms = 0;
    cudaError_t e = prepare_launch(qkv, T, H, o, &tm, &tm_o, &num_sms);
    if (e != cudaSuccess) return e;
    AttnParams p{d_slots, d_slot_off, row_tb, H, window, 1.4426950408889634f / 8.0f, (bf16*)o, status, nullptr, 0, 0, nullptr,
                 nullptr};
    e = is_global ? launch_pdl(attn_tc_kernel<false, false>, dim3(grid), dim3(NUM_THREADS), SMEM_TOTAL, s, tm, tm_o, p)
                  : launch_pdl(attn_tc_kernel<true, false>, dim3(grid), dim3(NUM_THREADS), SMEM_TOTAL, s, tm, tm_o, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

cudaError_t launch_attention_train_tc(const void* qkv, int T, int n_heads, int window, const AttnPlan& plan, int max_items,
                                      void* o, float* lse, unsigned int* status, cudaStream_t s) {
    const int H = n_heads * HD;
    CUtensorMap tm, tm_o;
    int num_sms = 0;
    cudaError_t e = prepare_launch(qkv, T, H, o, &tm, &tm_o, &num_sms);
    if (e != cudaSuccess) return e;
    const int grid = (int)std::min<long long>(num_sms, (long long)max_items * n_heads);
    AttnParams p{plan.items, nullptr, plan.row_tb, H, window, 1.4426950408889634f / 8.0f, (bf16*)o, status,
                 plan.n_items, n_heads, T, lse, (const bf16*)qkv};
    return window < 0 ? launch_pdl(attn_tc_kernel<false, true>, dim3(grid), dim3(NUM_THREADS), SMEM_TOTAL, s, tm, tm_o, p)
                      : launch_pdl(attn_tc_kernel<true, true>, dim3(grid), dim3(NUM_THREADS), SMEM_TOTAL, s, tm, tm_o, p);
}
