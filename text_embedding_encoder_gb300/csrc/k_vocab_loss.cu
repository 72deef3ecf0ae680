// Softmax cross entropy over a large vocabulary, and its gradients, on the
// 5th-generation tensor cores (tcgen05, sm_103a); tee_train.h has the formulas.
//
// The logits X W^T (X the counted positions' states, W the token table) are
// never kept.  Forward reduces each 256 x 256 tile of them, as it lies in tensor
// memory, to one (reference exponent, sum of exponentials) pair per row.
// Backward takes the vocabulary in pieces: the logits of a piece are computed
// again and become D = ratio (exp(logit - lse) - [target]) in bf16, from which
// the next launch adds D W to dX (fp32) and writes that piece's D^T X to dW.
// Work: 2 n V H flops forward, 6 n V H backward, n the counted positions.  Both
// are bound by the tensor cores.  Measured at n = 9830 of 32768, V = 102400, H = 768:
//   forward 0.80 to 0.92 ms, 1680 to 1930 TFLOP/s, the tensor pipes 95 to 97 % busy:
//     the clock, under the power limit, sets the time.
//   backward 3.0 to 3.25 ms, 1430 to 1550 TFLOP/s; the pipes 79 % busy.  A piece's
//     launch takes 107 to 111 us: products at 0.29 to 0.33 us a K step (0.27 is the pipes' rate at
//     1.9 GHz), logits 4.0 us a tile instead of 3.3 -- their operands' way through
//     shared memory, in and out again, already takes its whole bandwidth, and D's
//     adds to it --, and 5 us from one launch's last store to the next one's first.
// n = 315 of 1051: backward 0.18 to 0.19 ms.  One piece; DRAM moves 0.6 GB (the table
// twice, D three times, dW), and the second tile of 256 rows holds 59.
// Far from their floors, of whole row tiles and launches one after the other: one
// position 151 us backward and 54 forward (the table's bytes: 47 and 24); and of a
// small table, whose few tiles of D^T X leave CTA pairs idle: 16384 positions against
// 1000 rows 152 us (products: 38).
//
//   * Positions that are not counted cost nothing: vocab_rows_kernel lists the
//     others in order and copies their states together, and every later kernel
//     takes their number from device memory, so nothing waits on the host.
//   * One persistent kernel of CTA pairs (tcgen05 cta_group::2, 256 x 256 tiles,
//     K steps of 64, TMA-fed ring) runs every product.  The transposed operands
//     (W in D W, both in D^T X) are read as they lie, as MN-major tiles.
//   * A backward launch holds three kinds of independent tiles: D^T X and D W of
//     one piece and the logits of the next, shared out among the CTA pairs by
//     their length (make_shares); D is double-buffered.
//   * D is rounded to bf16 for the tensor cores, as the states and the table are.
//     The upstream gradients enter it divided by their largest magnitude (put
//     back in fp32 at the end), so that a gradient that all positions share does
//     not round every entry the same way.
#include "gemm_tc.cuh"
#include "train_internal.cuh"

#include <float.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "tc_ptx.cuh"

namespace {

using namespace tc;

constexpr int TILE = 256;              // rows and columns of a tile (a CTA holds 128 of the rows)
constexpr int BK = 64;
// A set of epilogue warps has two per quarter of the accumulator's rows, 128 columns
// each.  Forward has two sets, for every other tile each, so that one's loads and
// maxima run beside the other's exponentials: below 400 columns the epilogue is the
// longer part (9830 x 102400: H = 128 281 us with two sets, 411 with one; 384 451
// and 480; 768 820 and 814).  Backward measured no better with two: a box for each warp
// costs a stage of the operands (H = 768: 3.03 ms with two, 2.97 with one; 384 1.85
// and 1.89).
constexpr int EPI_WARPS = 8;
constexpr int epi_sets(bool bwd) { return bwd ? 1 : 2; }
constexpr int num_threads(bool bwd) { return 64 + 32 * EPI_WARPS * epi_sets(bwd); }
constexpr int MAX_PAIRS = 128;         // CTA pairs of a launch
constexpr uint32_t HALF_BYTES = 128 * BK * 2;          // this CTA's half of one operand's K step
constexpr uint32_t STAGE_BYTES = 2 * HALF_BYTES;
constexpr int STAGES = 6;
constexpr uint32_t OUT_OFF = STAGES * STAGE_BYTES;     // a 4 KB staging box per epilogue warp
constexpr uint32_t BAR_OFF = OUT_OFF + EPI_WARPS * 4096;
constexpr int N_BARS = 2 * STAGES + 5 + 16;
constexpr uint32_t SMEM_BYTES = BAR_OFF + N_BARS * 8 + 16 + 1024;   // + alignment slack
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
constexpr uint32_t TMEM_COLS = 512;    // two accumulators of 256 columns
constexpr float LOG2E = 1.4426950408889634f;
// A tile's epilogue, in K steps of products (2.4 us; 6 measured 196 us where this
// takes 183, 10 and 12 the same).
constexpr int EPILOGUE_K_STEPS = 8;

// Up to so many counted positions are listed twice in the backward pass, once in
// each half of the only row tile: the first gives D rounded to bf16, the second what
// that left over.  The products of the logits and of D W stay the same; D^T X walks up
// to four K steps instead of two, and D is written and read twice (102400 x 768: 128
// positions 171 us, 129, which are listed once, 147).  With many positions the roundings of D
// average out; with few, one of them (the target's entry, up to 2^-8 off) could be
// most of the error of a row of dW.
constexpr int FEW_ROWS = 128;

// What vocab_rows_kernel prepares, and the kernels after it read.
struct Rows {
    int* count;             // rows of x in use: the counted positions, and 128 more where `twice` is set
    int* twice;             // (backward) see FEW_ROWS
    float* gmax;            // largest finite magnitude of their upstream gradients, 1 if that is 0 (backward)
    int32_t* list;          // [N] their positions, ascending
    int32_t* index;         // [N] a position's place in the list, or -1 (backward)
    bf16* x;                // [Np, H] their states; rows up to the next multiple of 256 are zero
    int32_t* target;        // [Np]
    float* lse2;            // [Np] lse / ln 2 (backward)
    float* ratio;           // [Np] upstream gradient / gmax (backward)
    double* target_dot;     // [Np] x . w[target], summed outside the tensor cores (forward)
    float* target_d;        // [Np] ratio (exp(target_dot - lse) - 1), the target's entry of D (backward)
};

// ---------------------------------------------------------------------------
// the products
// ---------------------------------------------------------------------------

enum Kind { LOGITS, DX, DW };

struct Maps {
    CUtensorMap x, w;               // K-major operands of the logits: boxes of 64 columns x 128 rows
    CUtensorMap d;                  // D of the piece being multiplied, K-major (D W)
    CUtensorMap w_mn, d_mn, x_mn;   // MN-major operands: boxes of 64 columns x 64 rows
    CUtensorMap d_out, dx_acc, dw;  // outputs: boxes of 32 rows x 128 bytes (dw: of the table's gradient or its fp32 sums)
};

struct Share;

struct Params {
    Rows r;
    int V, H, Np;
    // logits: columns [v_log, v_log + n_log) of the vocabulary
    int v_log, n_log;
    // forward
    float2* part;                   // [tiles][Np] {reference exponent, sum}
    float* target_logit;            // [Np]
    // products of D: columns [v_mul, v_mul + n_mul)
    int v_mul, n_mul;
    int want_dx, want_dw;
    int acc_rows;                   // rows of the dX accumulators
    int first;                      // dX is written, not added to
    int dw_sum;                     // 0: dW is written rounded; else its fp32 sums, 1: written, 2: added to
    const Share* shares;            // the pairs' shares of this launch (backward)
    unsigned int* status;
};

// How many slices of a piece's columns the tiles of D W are split into, each
// with accumulators of its own: as many as give every CTA pair at most one
// tile, as far as the accumulators reach and a slice has at least four K steps.
__device__ __forceinline__ int dx_slices(int mt, int ht, int pairs, int acc_rows, int n_mul) {
    return max(1, min(min(pairs / (mt * ht), acc_rows / (mt * TILE)), n_mul / (4 * BK)));
}

struct Unit {
    int kind, m, n, k0, num_k, slice;   // tile (m, n); K steps k0 .. k0 + num_k
};

// The tiles of one launch.
struct Tiles {
    int mt, ht, n_dw, n_dx, n_log, k_slice, k_rows, k_mul, kh;
    static __device__ __forceinline__ Tiles of(int count, int H, int n_log, int n_mul, bool want_dx, bool want_dw, int pairs,
                                               int acc_rows) {
        Tiles q;
        q.mt = (count + TILE - 1) / TILE;
        q.ht = (H + TILE - 1) / TILE;
        q.kh = (H + BK - 1) / BK;
        q.n_log = q.mt * ((n_log + TILE - 1) / TILE);
        q.k_rows = (count + BK - 1) / BK;
        q.k_mul = (n_mul + BK - 1) / BK;
        q.n_dw = want_dw ? (n_mul + TILE - 1) / TILE * q.ht : 0;
        q.n_dx = q.k_slice = 0;
        if (want_dx && n_mul && q.mt) {
            const int slices = dx_slices(q.mt, q.ht, pairs, acc_rows, n_mul);
            q.k_slice = (q.k_mul + slices - 1) / slices;
            q.n_dx = q.mt * q.ht * slices;
        }
        return q;
    }
    __device__ __forceinline__ Unit unit(int kind, int u) const {
        if (kind == LOGITS) return Unit{LOGITS, u % mt, u / mt, 0, kh, 0};
        const int n = u % ht, rest = u / ht;
        if (kind == DW) return Unit{DW, rest, n, 0, k_rows, 0};
        const int s = rest / mt, k0 = s * k_slice;
        return Unit{DX, rest % mt, n, k0, max(0, min(k_slice, k_mul - k0)), s};
    }
};

// A CTA pair's share of a backward launch: of each kind the units [first, first + n).
struct Share {
    int first[3], n[3];   // by Kind
};

// The units a CTA pair takes, in the order it takes them: D W and D^T X, the
// longer of them first, then logits.  Forward: every pairs-th tile.
template <bool BWD>
struct Walk {
    int pos, end, step;
    Share share;
    int order[3];
    __device__ __forceinline__ Walk(const Tiles& t, const Share* shares, int pair, int pairs) {
        if constexpr (BWD) {
            share = shares[pair];
            const int units[3] = {t.n_log, t.n_dx, t.n_dw};
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                share.first[k] = min(max(share.first[k], 0), units[k]);
                share.n[k] = min(max(share.n[k], 0), units[k] - share.first[k]);
            }
            const bool dx_first = t.k_slice > t.k_rows;
            order[0] = dx_first ? DX : DW;
            order[1] = dx_first ? DW : DX;
            order[2] = LOGITS;
            pos = 0, step = 1, end = share.n[0] + share.n[1] + share.n[2];
        } else {
            pos = pair, step = pairs, end = t.n_log;
        }
    }
    __device__ __forceinline__ bool done() const { return pos >= end; }
    __device__ __forceinline__ Unit next(const Tiles& t) {
        int u = pos;
        pos += step;
        if constexpr (BWD) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int k = order[i], n = k == DX ? share.n[DX] : share.n[DW];
                if (u < n) return t.unit(k, (k == DX ? share.first[DX] : share.first[DW]) + u);
                u -= n;
            }
            return t.unit(LOGITS, share.first[LOGITS] + u);
        } else {
            return t.unit(LOGITS, u);
        }
    }
};

// The pairs' shares of backward launch i, by one warp: launch i computes the logits
// of piece i and multiplies D of piece i - 1.  Kind by kind, the longest units
// first, each unit goes to the pair with the least work so far -- computed for
// all units of a kind at once: the level X is searched up to which the pairs
// fill (a pair takes units while its work is below X), and what is left goes to
// pairs that stand at X exactly.
struct ShareArgs {
    int piece, pieces, want_dx, want_dw, pairs, acc_rows;
    Share* shares;   // [pieces + 1][pairs]
};
__device__ void make_shares(const ShareArgs& a, int count, int V, int H, int i) {
    constexpr int PER = MAX_PAIRS / 32;   // pair j * 32 + lane
    const int lane = threadIdx.x & 31, pairs = a.pairs;
    const int n_log = i < a.pieces ? min(a.piece, V - i * a.piece) : 0;
    const int n_mul = i > 0 ? min(a.piece, V - (i - 1) * a.piece) : 0;
    const Tiles t = Tiles::of(count, H, n_log, n_mul, a.want_dx, a.want_dw, pairs, a.acc_rows);
    const bool dx_first = t.k_slice > t.k_rows;
    int load[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) load[j] = j * 32 + lane < pairs ? 0 : INT32_MAX;
    auto sum = [](int v) { return __reduce_add_sync(0xffffffffu, v); };
#pragma unroll 1
    for (int q = 0; q < 3; ++q) {
        const int kind = q == 2 ? LOGITS : (q == 0) == dx_first ? DX : DW;
        const int units = kind == LOGITS ? t.n_log : kind == DX ? t.n_dx : t.n_dw;
        // a unit's time in K steps: its products, or its epilogue where that is longer
        const int cost = max(kind == LOGITS ? t.kh : kind == DX ? t.k_slice : t.k_rows, EPILOGUE_K_STEPS);
        auto taken = [&](int x, int j) { return load[j] < x ? (x - load[j] + cost - 1) / cost : 0; };
        int top = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) top = max(top, load[j] == INT32_MAX ? 0 : load[j]);
        top = __reduce_max_sync(0xffffffffu, top);
        // at lo the pairs take at most `units` units, at hi more; first the range in
        // which X lies where no pair's work is above it
        auto taken_by_all = [&](int x) {
            int f = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j) f += taken(x, j);
            return sum(f);
        };
        int before = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) before += load[j] == INT32_MAX ? 0 : load[j];
        const int even = (int)((sum(before) + (long long)units * cost) / pairs);
        long long lo = max(0, even - cost - 1), hi = (long long)even + 1;
        if (taken_by_all((int)lo) > units) lo = 0;
        if (taken_by_all((int)hi) <= units) hi = (long long)top + (long long)(units / pairs + 1) * cost + 1;
        while (hi - lo > 1) {
            const int mid = (int)((lo + hi) / 2);
            if (taken_by_all(mid) <= units) lo = mid;
            else hi = mid;
        }
        int k[PER], f = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) f += k[j] = taken((int)lo, j);
        int left = units - sum(f);
        int first = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const bool at = load[j] != INT32_MAX && load[j] + k[j] * cost == (int)lo;
            const unsigned m = __ballot_sync(0xffffffffu, at);
            if (at && __popc(m & ((1u << lane) - 1)) < left) ++k[j];
            left -= min(left, __popc(m));
            int inc = k[j];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += up;
            }
            if (j * 32 + lane < pairs) {
                Share& s = a.shares[i * pairs + j * 32 + lane];
                s.first[kind] = first + inc - k[j];
                s.n[kind] = k[j];
                load[j] += k[j] * cost;
            }
            first += __shfl_sync(0xffffffffu, inc, 31);
        }
    }
}

// ---------------------------------------------------------------------------
// before the products
// ---------------------------------------------------------------------------

// Lists the counted positions and copies their states together.  Each block has
// a slice of the positions; it counts what is counted before its slice by
// itself, so that no block waits for another (the targets are a few hundred KB
// out of L2).  The last slice's block also writes their number and zeroes the
// rest of the last tile; backward has a block more for each product launch's
// shares.  Both take the target's logit by a sum of their own; forward (gloss
// NULL) zeroes the outputs of the positions that are not counted, backward divides
// the upstream gradients by the largest and makes the target's entry of D: with a
// logit that is low by 2^-20 of itself (768 columns; 2^-18 at 2048), as the tensor
// cores' sums are, nothing would be left of exp(logit - lse) - 1 where the target
// is nearly certain.
constexpr int ROWS_THREADS = 512, ROWS_WARPS = ROWS_THREADS / 32;

// A sum of products of bf16 pairs, each exact in fp32, that keeps beside the fp32
// sum what its additions round off (Knuth's two-sum).
struct Dot {
    float sum = 0.f, rest = 0.f;
    __device__ __forceinline__ void add(float p) {
        const float t = sum + p, z = t - sum;
        rest += (sum - (t - z)) + (p - z);
        sum = t;
    }
    __device__ __forceinline__ void add8(const uint4& a, const uint4& b) {
        const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x0, x1, y0, y1;
            unpack_bf16x2(x[i], x0, x1);
            unpack_bf16x2(y[i], y0, y1);
            add(x0 * y0);
            add(x1 * y1);
        }
    }
    // over the warp's lanes (64-bit additions here cost 9 us for 9830 rows)
    __device__ __forceinline__ void over_warp() {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float s = __shfl_xor_sync(0xffffffffu, sum, o), r = __shfl_xor_sync(0xffffffffu, rest, o);
            rest += r;
            add(s);
        }
    }
    // an infinite sum leaves a rest that is not a number
    __device__ __forceinline__ double value() const { return (double)sum + (fabsf(rest) <= FLT_MAX ? (double)rest : 0.0); }
};

__global__ void __launch_bounds__(ROWS_THREADS, 2)
    vocab_rows_kernel(const bf16* __restrict__ x, const bf16* __restrict__ wt, const int32_t* __restrict__ targets,
                      const float* __restrict__ lse_in, const float* __restrict__ gloss, int N, int V, int H, int ignore_id,
                      int slice, float* loss, float* lse,
                      Rows r, ShareArgs shares, unsigned int* status) {
    __shared__ int warp_n[ROWS_WARPS], warp_all[ROWS_WARPS], from_s[ROWS_THREADS], to_s[ROWS_THREADS];
    __shared__ float warp_g[ROWS_WARPS];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lo = blockIdx.x * slice, hi = min(N, lo + slice);
    auto counted = [&](int t) { return t >= 0 && t < V && t != ignore_id; };
    // the counted positions before the slice, and (backward) all of them and their largest gradient
    int n = 0, all = 0;
    float g = 0.f;
    const int upto = gloss ? N : lo;
#pragma unroll 8
    for (int i = threadIdx.x; i < upto; i += ROWS_THREADS) {
        const bool live = counted(targets[i]);
        n += live && i < lo;
        all += live;
        if (gloss) {
            const float a = fabsf(gloss[i]);
            if (live && a < INFINITY) g = fmaxf(g, a);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        n += __shfl_xor_sync(0xffffffffu, n, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
        g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    }
    if (lane == 0) warp_n[warp] = n, warp_all[warp] = all, warp_g[warp] = g;
    __syncthreads();
    int at = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < ROWS_WARPS; ++w) at += warp_n[w], all += warp_all[w], g = fmaxf(g, warp_g[w]);
    const bool twice = gloss && all > 0 && all <= FEW_ROWS;
    if (lo >= N) {   // the blocks behind the slices: a launch's shares each
        if (warp == 0) make_shares(shares, twice ? FEW_ROWS + all : all, V, H, (int)blockIdx.x - (N - 1) / slice - 1);
        return;
    }
    const float gmax = g > 0.f ? g : 1.f;
    __syncthreads();
    for (int i0 = lo; i0 < hi; i0 += ROWS_THREADS) {   // (uniform: the block's barriers are inside)
        const int i = i0 + threadIdx.x;
        const int t = i < hi ? targets[i] : ignore_id;
        const bool live = counted(t);
        if (!live && t != ignore_id) atomicOr(status, TEE_STATUS_BAD_ID);
        const unsigned m = __ballot_sync(0xffffffffu, live);
        if (lane == 0) warp_n[warp] = __popc(m);
        __syncthreads();
        const int chunk0 = at;
        int place = at + __popc(m & ((1u << lane) - 1));
#pragma unroll
        for (int w = 0; w < ROWS_WARPS; ++w) {
            place += w < warp ? warp_n[w] : 0;
            at += warp_n[w];
        }
        if (live) {
            r.list[place] = i;
            for (int c = place; c <= place + (twice ? FEW_ROWS : 0); c += FEW_ROWS) {
                r.target[c] = t;
                if (gloss) {
                    r.lse2[c] = lse_in[i] * LOG2E;
                    r.ratio[c] = gloss[i] / gmax;
                }
            }
        }
        if (i < hi) {
            if (gloss) r.index[i] = live ? place : -1;
            else if (!live) loss[i] = lse[i] = 0.f;
        }
        if (live) {
            const int j = place - chunk0;
            from_s[j] = i;
            to_s[j] = t;
        }
        __syncthreads();
        // the block's warps copy the states, two rows at a time
        const int rows = at - chunk0;
        for (int j = 2 * warp; j < rows; j += 2 * ROWS_WARPS) {
            const bool two = j + 1 < rows;
            const uint4* src[2] = {reinterpret_cast<const uint4*>(x + (size_t)from_s[j] * H),
                                   reinterpret_cast<const uint4*>(x + (size_t)from_s[two ? j + 1 : j] * H)};
            uint4* dst = reinterpret_cast<uint4*>(r.x + (size_t)(chunk0 + j) * H);
            const int row = H / 8, half = row * FEW_ROWS;   // (in vectors)
            const uint4* to[2] = {reinterpret_cast<const uint4*>(wt + (size_t)to_s[j] * H),
                                  reinterpret_cast<const uint4*>(wt + (size_t)to_s[two ? j + 1 : j] * H)};
            Dot dot[2];
#pragma unroll 3
            for (int k = lane; k < row; k += 32) {
                const uint4 v[2] = {src[0][k], src[1][k]};
#pragma unroll
                for (int q = 0; q < 2; ++q) dot[q].add8(v[q], to[q][k]);
                dst[k] = v[0];
                if (two) dst[row + k] = v[1];
                if (twice) {
                    dst[half + k] = v[0];
                    if (two) dst[half + row + k] = v[1];
                }
            }
            dot[0].over_warp();
            dot[1].over_warp();
            if (lane < (two ? 2 : 1)) {   // a row by a lane
                const int c = chunk0 + j + lane, i = from_s[j + lane];
                const double logit = (lane ? dot[1] : dot[0]).value();
                if (gloss) {
                    const float e = gloss[i] / gmax * expm1f((float)(logit - (double)lse_in[i]));
                    r.target_d[c] = e;
                    if (twice) r.target_d[c + FEW_ROWS] = e;
                } else {
                    r.target_dot[c] = logit;
                }
            }
        }
        __syncthreads();
    }
    if (hi != N) return;
    if (threadIdx.x == 0) {
        *r.count = twice ? FEW_ROWS + at : at;
        if (gloss) *r.gmax = gmax, *r.twice = twice;
    }
    const int end = (at + TILE - 1) / TILE * TILE;
    for (int c = at + warp; c < end; c += ROWS_WARPS) {
        if (twice && c >= FEW_ROWS && c < FEW_ROWS + at) continue;
        for (int k = lane; k < H / 8; k += 32) reinterpret_cast<uint4*>(r.x + (size_t)c * H)[k] = make_uint4(0, 0, 0, 0);
        if (lane == 0) {
            r.target[c] = -1;
            if (gloss) r.lse2[c] = r.ratio[c] = r.target_d[c] = 0.f;
        }
    }
}

// ---------------------------------------------------------------------------
// the product kernel
// ---------------------------------------------------------------------------

template <bool BWD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(num_threads(BWD), 1)
    vocab_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_OFF);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + N_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    auto bar = [&](int i) { return smem_u32(bars + i); };
    constexpr int FULL = 0, EMPTY = STAGES, TFULL = 2 * STAGES, TEMPTY = 2 * STAGES + 2, MMA_DONE = 2 * STAGES + 4,
                  JOIN = 2 * STAGES + 5;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank();
    // the even CTA's barriers, which both signal
    const uint32_t full0 = mapa_shared(bar(FULL), 0), tempty0 = mapa_shared(bar(TEMPTY), 0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar(FULL + s), 1);
            mbar_init(bar(EMPTY + s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar(TFULL + a), 1);
            mbar_init(bar(TEMPTY + a), 2 * EPI_WARPS);   // every epilogue warp of both CTAs
        }
        mbar_init(bar(MMA_DONE), 1);
        for (int j = 0; j < 16; ++j) mbar_init(bar(JOIN + j), 32);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<2>(smem_u32(tmem_slot), TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // the peer's copies and commits may target these barriers only after init
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    // (what comes out of the workspace is kept within its arrays, so that a
    // workspace that another call writes to gives wrong numbers and no stray access)
    const int count = min(max(__ldcg(p.r.count), 0), p.Np);
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const Tiles tiles = Tiles::of(count, p.H, p.n_log, p.n_mul, p.want_dx, p.want_dw, pairs, p.acc_rows);
    Walk<BWD> walk(tiles, p.shares, pair, pairs);

    // a wait that gives up does so for the whole warp
    auto all = [](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };

    if (warp == 0) {
        // ---------------- TMA producer (the whole warp, one lane issuing) ----------------
        uint32_t s = 0, phase = 0, loaded = 0;
        bool ok = true;
        // one K step: both CTAs' halves land on the even CTA's barrier, which expects both
        auto step = [&](auto&& loads) {
            if (!all(mbar_wait(bar(EMPTY) + 8 * s, phase ^ 1, abort_flag))) return false;
            if (elect_one()) {
                if (crank == 0) mbar_expect_tx(bar(FULL) + 8 * s, 2 * STAGE_BYTES);
                const uint32_t sa = sbase + s * STAGE_BYTES;
                loads(sa, sa + HALF_BYTES, full0 + 8 * s);
            }
            __syncwarp();
            ++loaded;
            if (++s == STAGES) s = 0, phase ^= 1;
            return true;
        };
        while (ok && !walk.done()) {
            const Unit w = walk.next(tiles);
            const int a0 = w.m * TILE + (int)crank * 128, b0 = w.n * TILE + (int)crank * 128;
            const int k_end = (w.k0 + w.num_k) * BK;
            if (!BWD || w.kind == LOGITS) {
                for (int k = 0; k < k_end && ok; k += BK)
                    ok = step([&](uint32_t sa, uint32_t sb, uint32_t full) {
                        tma_load_2d_pair(sa, &maps.x, k, a0, full);
                        tma_load_2d_pair(sb, &maps.w, k, p.v_log + b0, full);
                    });
            } else if (w.kind == DX) {
                for (int k = w.k0 * BK; k < k_end && ok; k += BK)
                    ok = step([&](uint32_t sa, uint32_t sb, uint32_t full) {
                        tma_load_2d_pair(sa, &maps.d, k, a0, full);
                        tma_load_2d_pair(sb, &maps.w_mn, b0, p.v_mul + k, full);
                        tma_load_2d_pair(sb + HALF_BYTES / 2, &maps.w_mn, b0 + 64, p.v_mul + k, full);
                    });
            } else {
                for (int k = 0; k < k_end && ok; k += BK)
                    ok = step([&](uint32_t sa, uint32_t sb, uint32_t full) {
                        tma_load_2d_pair(sa, &maps.d_mn, a0, k, full);
                        tma_load_2d_pair(sa + HALF_BYTES / 2, &maps.d_mn, a0 + 64, k, full);
                        tma_load_2d_pair(sb, &maps.x_mn, b0, k, full);
                        tma_load_2d_pair(sb + HALF_BYTES / 2, &maps.x_mn, b0 + 64, k, full);
                    });
            }
        }
        // no copy may still be landing in shared memory when the CTA exits (the
        // even CTA's barriers complete with both CTAs' copies)
        if (crank == 0)
            for (uint32_t left = loaded < STAGES ? loaded : STAGES; left > 0; --left) {
                if (s == 0) s = STAGES, phase ^= 1;
                --s;
                mbar_wait_drain(bar(FULL) + 8 * s, phase);
            }
    } else if (warp == 1) {
        // ---------------- MMA issuer (the even CTA's, for both; the whole warp, one lane issuing) ----------------
        if (crank == 0) {
            uint32_t s = 0, phase = 0;
            bool ok = true;
            // the products of one unit; a K step of 16 is 32 bytes along a K-major
            // row, or 16 rows of 128 bytes of an MN-major group
            auto products = [&](auto a_mn, auto b_mn, uint32_t d_tmem, int num_k) {
                constexpr bool A_MN = decltype(a_mn)::value, B_MN = decltype(b_mn)::value;
                constexpr uint32_t idesc =
                    make_idesc(2 * 128, TILE) | (A_MN ? IDESC_A_MN_MAJOR : 0) | (B_MN ? IDESC_B_MN_MAJOR : 0);
                constexpr uint32_t a_step = A_MN ? 128 : 2, b_step = B_MN ? 128 : 2;
                const uint64_t a0 = A_MN ? sw128_desc_mn_groups(sbase, HALF_BYTES / 2) : sw128_desc(sbase);
                const uint64_t b0 = B_MN ? sw128_desc_mn_groups(sbase + HALF_BYTES, HALF_BYTES / 2)
                                         : sw128_desc(sbase + HALF_BYTES);
                for (int kb = 0; kb < num_k; ++kb) {
                    if (!all(mbar_wait_cluster(bar(FULL) + 8 * s, phase, abort_flag))) return false;
                    tc_fence_after();
                    const uint64_t ad = a0 + s * (STAGE_BYTES >> 4), bd = b0 + s * (STAGE_BYTES >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < BK / 16; ++k)
                            mma_bf16_pair(d_tmem, ad + k * a_step, bd + k * b_step, idesc, (kb | k) != 0);
                        mma_commit_pair(bar(EMPTY) + 8 * s, 0x3);   // both CTAs' stage s
                    }
                    __syncwarp();
                    if (++s == STAGES) s = 0, phase ^= 1;
                }
                return true;
            };
            constexpr std::integral_constant<bool, true> mn{};
            constexpr std::integral_constant<bool, false> kmajor{};
            for (int it = 0; ok && !walk.done(); ++it) {
                const Unit w = walk.next(tiles);
                const int acc = it & 1, use = it >> 1;
                if (!all(mbar_wait_cluster(bar(TEMPTY + acc), (use & 1) ^ 1, abort_flag))) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * TILE;
                if (!BWD || w.kind == LOGITS) ok = products(kmajor, kmajor, d_tmem, w.num_k);
                else if (w.kind == DX) ok = products(kmajor, mn, d_tmem, w.num_k);
                else ok = products(mn, mn, d_tmem, w.num_k);
                if (ok && elect_one()) mma_commit_pair(bar(TFULL + acc), 0x3);   // both CTAs' accumulator halves
                __syncwarp();
            }
            // every MMA issued must be finished before TMEM is freed
            if (elect_one()) mma_commit_pair(bar(MMA_DONE), 0x1);
            __syncwarp();
            mbar_wait_drain(bar(MMA_DONE), 0);
        }
    } else {
        // ---------------- epilogue: thread = row, warps 2..5 columns 0..127, 6..9 the others (10..17 as 2..9) ----------------
        const int quad = warp & 3, half = (warp - 2) >> 2 & 1, set = (warp - 2) / EPI_WARPS;
        uint8_t* stage = smem + OUT_OFF + (warp - 2) % EPI_WARPS * 4096;   // (backward) this warp's staging box
        auto box_free = [&]() {   // the box's last store has read it
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
        };
        auto send = [&](auto&& issue) {   // lane 0 stores the box just written
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                issue(smem_u32(stage));
                bulk_commit();
            }
        };
        const float gmax = BWD ? __ldcg(p.r.gmax) : 0.f;
        const bool left_over = BWD && crank == 1 && __ldcg(p.r.twice);   // this CTA's rows: what the even CTA's rounding left
        for (int it = 0; !walk.done(); ++it) {
            const Unit w = walk.next(tiles);
            const int acc = it & 1, use = it >> 1;
            if (!BWD && acc != set) continue;
            const int row0 = w.m * TILE + (int)crank * 128 + quad * 32, row = row0 + lane;
            const int col0 = w.n * TILE + half * 128;          // this warp's first column of the output
            const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + acc * TILE + half * 128;
            // what the row needs, fetched while the products run
            float lse2 = 0.f, ratio = 0.f, target_d = 0.f;
            int target = -1;
            bool counted = false;
            if (!BWD || w.kind == LOGITS) {
                target = p.r.target[row];
                counted = target >= 0;
                target -= p.v_log + col0;                      // within this warp's columns, if it is there
                if (BWD) lse2 = p.r.lse2[row], ratio = p.r.ratio[row], target_d = p.r.target_d[row];
            }
            if (!all(mbar_wait(bar(TFULL + acc), use & 1, abort_flag))) break;
            tc_fence_after();
            if constexpr (!BWD) {
                // 64 columns at a time, to a reference exponent and a sum
                float ref = -INFINITY, sum = 0.f;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v[64];
                    tmem_ld64(taddr + 64 * c, v);
                    if (c) {   // the accumulator is free
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * acc);
                    }
                    if (col0 + 64 * c + 64 > p.V) {
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (col0 + 64 * c + j >= p.V) v[j] = -INFINITY;
                    }
                    const int tj = target - 64 * c;
                    if (__any_sync(0xffffffffu, tj >= 0 && tj < 64)) {
                        float tv = 0.f;
#pragma unroll
                        for (int j = 0; j < 64; ++j) tv = j == tj ? v[j] : tv;
                        if (tj >= 0 && tj < 64) p.target_logit[row] = tv;
                    }
                    float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                    for (int j = 4; j < 64; j += 8)   // (the last step's upper half repeats its lower one)
#pragma unroll
                        for (int q = 0; q < 4; ++q) mx[q] = fmax3(mx[q], v[j + q], v[j + 4 < 64 ? j + 4 + q : j + q]);
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    // exponentials are taken against the maximum so far, kept finite (infinity against infinity would give NaN)
                    const float mine = top == -INFINITY ? -INFINITY : fminf(fmaxf(top * LOG2E, -FLT_MAX), FLT_MAX);
                    const float both = fmaxf(ref, mine), to = both == -INFINITY ? 0.f : both;
                    float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < 64; ++j) s4[j & 3] += ex2_approx(fmaf(v[j], LOG2E, -to));
                    const float s1 = (s4[0] + s4[1]) + (s4[2] + s4[3]);
                    sum = c && both != -INFINITY ? fmaf(sum, ex2_approx(ref - both), s1) : sum + s1;
                    ref = both;
                }
                // the two warps of a row join through shared memory.  Four slots: a
                // slot comes round again after its tile's fourth successor has been
                // multiplied, which waits for this row's warps to have left the second
                const int slot = it & 3, joined = JOIN + quad * 4 + slot;
                float2* other = reinterpret_cast<float2*>(smem + OUT_OFF) + slot * 128 + quad * 32 + lane;
                if (half) {
                    *other = make_float2(ref, sum);
                    mbar_arrive(bar(joined));
                } else {
                    if (!all(mbar_wait(bar(joined), (it >> 2) & 1, abort_flag))) break;
                    const float2 o = *other;
                    const float both = fmaxf(ref, o.x);
                    if (both != -INFINITY) sum = sum * ex2_approx(ref - both) + o.y * ex2_approx(o.x - both);
                    else sum += o.y;
                    if (row < count) p.part[(size_t)w.n * p.Np + row] = make_float2(both, sum);
                }
                continue;
            }
            // the accumulator is free once both loads are in registers
            float v[2][64];
            tmem_ld64_issue(taddr, v[0]);
            tmem_ld64_issue(taddr + 64, v[1]);
            tmem_wait_ld();
            tmem_tie64(v[0]);
            tmem_tie64(v[1]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * acc);
            if (w.kind == LOGITS) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int j = 0; j < 64; ++j) v[c][j] = ex2_approx(fmaf(v[c][j], LOG2E, -lse2));
                    // rows of padding are zero whatever the table holds
#pragma unroll
                    for (int j = 0; j < 64; ++j) v[c][j] = counted ? v[c][j] * ratio : 0.f;
                    // and so are columns behind the table, where logits of 0 against an lse far below give infinities
                    if (col0 + 64 * c + 64 > p.n_log) {
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (col0 + 64 * c + j >= p.n_log) v[c][j] = 0.f;
                    }
                    const int tj = target - 64 * c;
                    if (__any_sync(0xffffffffu, tj >= 0 && tj < 64)) {
#pragma unroll
                        for (int j = 0; j < 64; ++j) v[c][j] = j == tj ? target_d : v[c][j];
                    }
                    if (left_over) {
#pragma unroll
                        for (int j = 0; j < 64; ++j) v[c][j] -= __bfloat162float(__float2bfloat16_rn(v[c][j]));
                    }
                    // rows that D^T X does not reach; in D W they only reach themselves
                    if (row0 >= tiles.k_rows * BK) continue;
                    box_free();
                    stage_row_bf16x64(stage, lane, v[c]);
                    send([&](uint32_t src) { tma_store_2d(&maps.d_out, src, col0 + 64 * c, row0); });
                }
            } else if (w.kind == DX || p.dw_sum) {
                // fp32 sums.  Each element is added to once a launch: the order of the sums is fixed
                const bool is_dx = w.kind == DX, write = is_dx ? p.first != 0 : p.dw_sum == 1;
                const CUtensorMap* map = is_dx ? &maps.dx_acc : &maps.dw;
                const int y = is_dx ? w.slice * tiles.mt * TILE + row0 : p.v_mul + row0;
                const float scale = is_dx ? 1.f : gmax;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int x = col0 + 32 * c;
                    if (x < p.H && (is_dx || y < p.V)) {
                        const float* a = v[c >> 1] + 32 * (c & 1);
                        box_free();
                        uint8_t* b = stage + lane * 128;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            *reinterpret_cast<float4*>(b + ((k ^ (lane & 7)) << 4)) =
                                w.num_k ? make_float4(a[4 * k] * scale, a[4 * k + 1] * scale, a[4 * k + 2] * scale,
                                                      a[4 * k + 3] * scale)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
                        send([&](uint32_t src) {
                            if (write) tma_store_2d(map, src, x, y);
                            else tma_reduce_add_2d(map, src, x, y);
                        });
                    }
                }
            } else {
                const int y = p.v_mul + row0;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int x = col0 + 64 * c;
                    if (x < p.H && y < p.V) {
#pragma unroll
                        for (int j = 0; j < 64; ++j) v[c][j] = w.num_k ? v[c][j] * gmax : 0.f;
                        box_free();
                        stage_row_bf16x64(stage, lane, v[c]);
                        send([&](uint32_t src) { tma_store_2d(&maps.dw, src, x, y); });
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_all();   // stores complete before the CTA exits
    }

    tc_fence_before();
    __syncthreads();
    // the even CTA's MMAs (which write both CTAs' tensor memory) have drained before either CTA frees it
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<2>(tmem_base, TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort_flag) atomicOr(p.status, TEE_STATUS_TIMEOUT);
    // the peer's last copies, commits and arrivals target this CTA's barriers: leave together
    cluster_sync();
}

// ---------------------------------------------------------------------------
// after the products
// ---------------------------------------------------------------------------

// lse and loss of the counted positions from the tiles' pairs: 32 rows by 16
// slices of the tiles per block; the last step in 64 bits.
__global__ void __launch_bounds__(512)
    vocab_finish_kernel(const float2* __restrict__ part, const float* __restrict__ target_logit, Rows r, int tiles, int N,
                        int Np, float* __restrict__ loss, float* __restrict__ lse) {
    __shared__ float2 red[16][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int row = blockIdx.x * 32 + lane, n = min(*r.count, N);
    if (blockIdx.x * 32 >= n) return;
    float2 a = make_float2(-INFINITY, 0.f);
    auto join = [](float2 a, float2 b) {
        const float to = fmaxf(a.x, b.x);
        if (to == -INFINITY) return make_float2(-INFINITY, a.y + b.y);
        return make_float2(to, a.y * exp2f(a.x - to) + b.y * exp2f(b.x - to));
    };
    if (row < n) {
        constexpr int AT_ONCE = 9;   // pairs on their way together
        for (int t0 = sl; t0 < tiles; t0 += 16 * AT_ONCE) {
            float2 v[AT_ONCE];
#pragma unroll
            for (int q = 0; q < AT_ONCE; ++q)
                v[q] = t0 + 16 * q < tiles ? part[(size_t)(t0 + 16 * q) * Np + row] : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int q = 0; q < AT_ONCE; ++q) a = join(a, v[q]);
        }
    }
    red[sl][lane] = a;
    __syncthreads();
    if (sl || row >= n) return;
    for (int s = 1; s < 16; ++s) a = join(a, red[s][lane]);
    const double l = ((double)a.x + log2((double)a.y)) * 0.69314718055994530942;
    const int i = r.list[row];
    if ((unsigned)i >= (unsigned)N) return;
    // The tensor cores' sums of H products are off by a few 2^-24 of the logit.
    // The target's logit counts most, alone and, where it is likely, in lse: both
    // take the sum of its own instead, lse by exchanging the one term (H = 768: the
    // losses are 0.8e-7 off; 6.5e-7 without this, 2.7e-7 with fp32 products).
    const double mma = target_logit[row], dot = r.target_dot[row];
    const double shift = exp(mma - l) * expm1(dot - mma);
    const double fixed = shift > -0.5 && shift < 1e3 ? l + log1p(shift) : l;   // (not with infinities or NaN)
    lse[i] = (float)fixed;
    loss[i] = (float)(fixed - dot);
}

// dX of every position: gmax times the sum of its accumulators, or zeros; four
// columns per thread.  n_mul: the columns of the first piece, whose products wrote
// every slice.  What the rounding of D left of the target's entry, mostly the
// largest by far, is added here in fp32, where D holds one half only: dx is then
// as exact as its type (H = 768: 1.66e-3 of the norm; 1.97e-3 without).
__global__ void __launch_bounds__(256)
    vocab_scatter_kernel(const float* __restrict__ acc, const bf16* __restrict__ wt, const int32_t* __restrict__ targets,
                         Rows r, int N, int Np, int V, int H, int n_mul, int acc_rows, int pairs, bf16* __restrict__ dx) {
    pdl_wait();
    pdl_trigger();
    const size_t at4 = (size_t)blockIdx.x * 256 + threadIdx.x;
    const int quads = H / 4, i = (int)(at4 / quads), k = (int)(at4 - (size_t)i * quads);
    if (at4 >= (size_t)N * quads) return;
    const int target = targets[i];
    const float gmax = *r.gmax;
    const int n = min(max(*r.count, 0), Np), mt = (n + TILE - 1) / TILE;
    const int at = min(r.index[i], n - 1), more = *r.twice ? FEW_ROWS : 0;
    float v[4] = {};
    if (at >= 0) {
        float w[4];
        load_vec(wt + (size_t)min(max(target, 0), V - 1) * H + 4 * k, w);
        const float d = r.target_d[at];
        const int slices = dx_slices(mt, (H + TILE - 1) / TILE, pairs, acc_rows, n_mul);
        const float* from = acc + (size_t)at * H + 4 * k;
#pragma unroll 4
        for (int s = 0; s < slices; ++s) {
            float a[4];
            load_vec(from + (size_t)s * mt * TILE * H, a);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += a[j];
        }
        if (!more) {
            const float rest = d - __bfloat162float(__float2bfloat16_rn(d));
            if (fabsf(rest) <= FLT_MAX) {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = fmaf(rest, w[j], v[j]);
            }
        } else {
            from = acc + (size_t)((at + more) % TILE) * H + 4 * k;
            for (int s = 0; s < slices; ++s) {
                float a[4];
                load_vec(from + (size_t)s * mt * TILE * H, a);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] += a[j];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= gmax;
    }
    store_vec(dx + (size_t)i * H + 4 * k, v);
}

// dW from its fp32 sums, eight elements a thread.
__global__ void __launch_bounds__(256) vocab_round_kernel(const float* __restrict__ sums, size_t n8, bf16* __restrict__ dw) {
    pdl_wait();
    pdl_trigger();
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8) return;
    float a[4], b[4];
    load_vec(sums + 8 * i, a);
    load_vec(sums + 8 * i + 4, b);
    store_vec(dw + 8 * i, {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Backward takes the positions in parts of at most so many, the parts' dW added in
// fp32 in order.  The tensor cores drop part of the last bit of a sum at every step
// of 16 terms: a dW of 65536 positions whose terms all have one sign is 2e-4 low,
// which its rounding to bf16 covers; of 2^20 in one sum 0.7 %, of 2^24 10 %.
constexpr int PART_ROWS = 65536;

int round_up(int v, int a) { return (int)(((long long)v + a - 1) / a * a); }

// Positions of each of the parts but the last: equal ones, whole tiles.
int part_rows(int N) {
    const int parts = (N + PART_ROWS - 1) / PART_ROWS;
    return round_up((N + parts - 1) / parts, TILE);
}

// Columns of a backward piece: D at most 256 MB for as many rows as there are
// positions, 2048 columns at least.  Smaller pieces keep D in L2 but their launches
// cost more than that saves (128 MB: 3.2 against 3.1 ms at 32768 positions, 0.19
// against 0.18 at 1051); 512 MB measured the same as 256.
int piece_columns(int Np, int V) {
    const long long fit = (256LL << 20) / (2LL * Np) / TILE * TILE;
    return (int)std::min<long long>(std::max<long long>(fit, 2048), round_up(V, TILE));
}

// Rows of the dX accumulators: every position once, or enough for two slices per
// CTA pair of 80 where there are few positions.
int accumulator_rows(int Np, int H) { return std::max(Np, 160 / ((H + TILE - 1) / TILE) * TILE); }

struct LossWs {
    Rows r{};
    float2* part = nullptr;
    float* target_logit = nullptr;
    bf16* d[2] = {nullptr, nullptr};
    float* acc = nullptr;
    Share* shares = nullptr;
    float* dw_sum = nullptr;
    size_t bytes = 0;
};
// (backward: of a part)
LossWs carve_loss(int N, int V, int H, bool backward, void* base) {
    WsCarve ws(base);
    LossWs w;
    if (backward && N > PART_ROWS) {
        w.dw_sum = ws.take<float>((size_t)V * H);
        N = part_rows(N);
    }
    const int Np = round_up(N, TILE);
    w.r.count = ws.take<int>(1);
    w.r.gmax = ws.take<float>(1);
    w.r.twice = ws.take<int>(1);
    w.r.list = ws.take<int32_t>(N);
    w.r.x = ws.take<bf16>((size_t)Np * H);
    w.r.target = ws.take<int32_t>(Np);
    if (!backward) {
        w.target_logit = ws.take<float>(Np);
        w.r.target_dot = ws.take<double>(Np);
        w.part = ws.take<float2>((size_t)Np * ((V + TILE - 1) / TILE));
    } else {
        w.r.index = ws.take<int32_t>(N);
        w.r.lse2 = ws.take<float>(Np);
        w.r.ratio = ws.take<float>(Np);
        w.r.target_d = ws.take<float>(Np);
        const int vc = piece_columns(Np, V);
        for (int b = 0; b < (vc < V ? 2 : 1); ++b) w.d[b] = ws.take<bf16>((size_t)Np * vc);
        w.acc = ws.take<float>((size_t)accumulator_rows(Np, H) * H);
        w.shares = ws.take<Share>((size_t)((V + vc - 1) / vc + 1) * MAX_PAIRS);
    }
    w.bytes = ws.off;
    return w;
}

template <bool BWD>
cudaError_t max_pairs(int dev, int num_sms, int* pairs) {
    static std::mutex mu;
    static int of[TEE_MAX_DEVICES] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (!of[dev]) {
        cudaError_t e = cudaFuncSetAttribute(vocab_kernel<BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(num_sms / 2 * 2);
        cfg.blockDim = dim3(num_threads(BWD));
        cfg.dynamicSmemBytes = SMEM_BYTES;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, vocab_kernel<BWD>, &cfg);
        if (e != cudaSuccess) return e;
        of[dev] = std::min(std::max(1, n), MAX_PAIRS);
    }
    *pairs = of[dev];
    return cudaSuccess;
}

#define TRY(call)                           \
    do {                                    \
        const cudaError_t e_ = (call);      \
        if (e_ != cudaSuccess) return e_;   \
    } while (0)

cudaError_t prepare_rows(const void* x, const void* wt, const int32_t* targets, const float* lse_in, const float* gloss,
                         float* loss, float* lse, int N, int V, int H, int ignore_id, const LossWs& w,
                         const ShareArgs& shares, unsigned int* status, cudaStream_t s) {
    // a slice for each of 296 blocks, about two an SM, of 32 positions at least (16384 counted positions against 1000
    // rows, backward: 152 us, with 148 blocks 158; few positions take the same)
    const int slice = round_up(std::max(1, (N + 295) / 296), 32);
    const int blocks = (N + slice - 1) / slice + (shares.pairs ? shares.pieces + 1 : 0);
    return launch_pdl(vocab_rows_kernel, dim3(blocks), dim3(ROWS_THREADS), 0, s, (const bf16*)x, (const bf16*)wt, targets,
                      lse_in, gloss, N, V, H, ignore_id, slice, loss, lse, w.r, shares, status);
}

}  // namespace

size_t vocab_loss_ws(int N, int V, int H, bool backward) { return carve_loss(N, V, H, backward, nullptr).bytes; }

cudaError_t launch_vocab_loss_forward(const void* x, const void* wt, const int32_t* targets, float* loss, float* lse, int N,
                                      int V, int H, int ignore_id, void* ws, unsigned int* status, cudaStream_t s) {
    if (N == 0) return cudaSuccess;
    int dev = 0, num_sms = 0, pairs = 0;
    TRY(tee_current_device(&dev, &num_sms));
    TRY(max_pairs<false>(dev, num_sms, &pairs));
    const int Np = round_up(N, TILE), tiles = (V + TILE - 1) / TILE;
    const LossWs w = carve_loss(N, V, H, false, ws);
    Maps maps{};
    TRY(make_tensor_map_2d(&maps.x, false, w.r.x, Np, H, H, 128, 64));
    TRY(make_tensor_map_2d(&maps.w, false, wt, V, H, H, 128, 64));
    Params p{};
    p.r = w.r;
    p.V = V, p.H = H, p.Np = Np;
    p.n_log = V;
    p.part = w.part;
    p.target_logit = w.target_logit;
    p.status = status;
    TRY(prepare_rows(x, wt, targets, nullptr, nullptr, loss, lse, N, V, H, ignore_id, w, ShareArgs{}, status, s));
    const int grid = 2 * std::min(pairs, Np / TILE * tiles);
    TRY(launch_pdl(vocab_kernel<false>, dim3(grid), dim3(num_threads(false)), SMEM_BYTES, s, maps, p));
    return launch_pdl(vocab_finish_kernel, dim3(round_up(N, 32) / 32), dim3(512), 0, s, (const float2*)w.part,
                      (const float*)w.target_logit, w.r, tiles, N, Np, loss, lse);
}

cudaError_t launch_vocab_loss_backward(const void* x, const void* wt, const int32_t* targets, const float* lse,
                                       const float* gloss, void* dx, void* dw, int N, int V, int H, int ignore_id, void* ws,
                                       unsigned int* status, cudaStream_t s) {
    if (N == 0) return dw ? cudaMemsetAsync(dw, 0, (size_t)V * H * sizeof(bf16), s) : cudaSuccess;
    int dev = 0, num_sms = 0, pairs = 0;
    TRY(tee_current_device(&dev, &num_sms));
    TRY(max_pairs<true>(dev, num_sms, &pairs));
    const bool parts = N > PART_ROWS;
    const int part = parts ? part_rows(N) : N, Np = round_up(part, TILE), vc = piece_columns(Np, V);
    const LossWs w = carve_loss(N, V, H, true, ws);
    Maps maps{};
    TRY(make_tensor_map_2d(&maps.x, false, w.r.x, Np, H, H, 128, 64));
    TRY(make_tensor_map_2d(&maps.w, false, wt, V, H, H, 128, 64));
    TRY(make_tensor_map_2d(&maps.w_mn, false, wt, V, H, H, 64, 64));
    TRY(make_tensor_map_2d(&maps.x_mn, false, w.r.x, Np, H, H, 64, 64));
    const int acc_rows = accumulator_rows(Np, H);
    TRY(make_tensor_map_2d(&maps.dx_acc, true, w.acc, acc_rows, H, H, 32, 32));
    if (dw && parts) TRY(make_tensor_map_2d(&maps.dw, true, w.dw_sum, V, H, H, 32, 32));
    else if (dw) TRY(make_tensor_map_2d(&maps.dw, false, dw, V, H, H, 32, 64));
    CUtensorMap d_in[2], d_mn[2], d_out[2];
    for (int b = 0; b < (vc < V ? 2 : 1); ++b) {
        TRY(make_tensor_map_2d(&d_in[b], false, w.d[b], Np, vc, vc, 128, 64));
        TRY(make_tensor_map_2d(&d_mn[b], false, w.d[b], Np, vc, vc, 64, 64));
        TRY(make_tensor_map_2d(&d_out[b], false, w.d[b], Np, vc, vc, 32, 64));
    }
    Params p{};
    p.r = w.r;
    p.V = V, p.H = H, p.Np = Np;
    p.want_dx = dx != nullptr, p.want_dw = dw != nullptr;
    p.acc_rows = acc_rows;
    p.status = status;
    const int pieces = (V + vc - 1) / vc;
    const ShareArgs shares{vc, pieces, p.want_dx, p.want_dw, pairs, acc_rows, w.shares};
    for (int at = 0; at < N; at += part) {
        const int n = std::min(part, N - at);
        TRY(prepare_rows((const bf16*)x + (size_t)at * H, wt, targets + at, lse + at, gloss + at, nullptr, nullptr, n, V, H,
                         ignore_id, w, shares, status, s));
        p.dw_sum = !parts ? 0 : at == 0 ? 1 : 2;
        for (int i = 0; i <= pieces; ++i) {
            // logits of piece i into one buffer, products of piece i - 1 out of the other
            p.v_log = i < pieces ? i * vc : 0;
            p.n_log = i < pieces ? std::min(vc, V - p.v_log) : 0;
            p.v_mul = i > 0 ? (i - 1) * vc : 0;
            p.n_mul = i > 0 ? std::min(vc, V - p.v_mul) : 0;
            p.first = i == 1;
            p.shares = w.shares + (size_t)i * pairs;
            if (i < pieces) maps.d_out = d_out[i & 1];
            if (i > 0) maps.d = d_in[(i - 1) & 1], maps.d_mn = d_mn[(i - 1) & 1];
            TRY(launch_pdl(vocab_kernel<true>, dim3(2 * pairs), dim3(num_threads(true)), SMEM_BYTES, s, maps, p));
        }
        if (!dx) continue;
        const unsigned blocks = (unsigned)(((size_t)n * (H / 4) + 255) / 256);
        TRY(launch_pdl(vocab_scatter_kernel, dim3(blocks), dim3(256), 0, s, (const float*)w.acc, (const bf16*)wt,
                       targets + at, w.r, n, Np, V, H, std::min(vc, V), acc_rows, pairs, (bf16*)dx + (size_t)at * H));
    }
    if (!parts || !dw) return cudaSuccess;
    const size_t n8 = (size_t)V * H / 8;
    return launch_pdl(vocab_round_kernel, dim3((unsigned)((n8 + 255) / 256)), dim3(256), 0, s, (const float*)w.dw_sum, n8,
                      (bf16*)dw);
}
