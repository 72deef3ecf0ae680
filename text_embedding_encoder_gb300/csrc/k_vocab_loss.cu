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
// are bound by the tensor cores.
//
//   * Positions that are not counted cost nothing: their rows are left out first
//     (vocab_rows_kernel lists the others in order, vocab_gather_kernel copies
//     them together), and every later kernel takes their number from device
//     memory, so nothing waits on the host.
//   * One persistent kernel of CTA pairs (tcgen05 cta_group::2, 256 x 256 tiles,
//     K steps of 64, TMA-fed ring) runs every product.  The transposed operands
//     (W in D W, both in D^T X) are read as they lie, as MN-major tiles.
//   * A backward launch holds three kinds of independent tiles: D^T X and D W of
//     one piece and the logits of the next, so there are always tiles to fill
//     the SMs with; D is double-buffered.
//   * D is rounded to bf16 for the tensor cores, as the states and the table are.
//     The upstream gradients enter it divided by their largest magnitude (put
//     back in fp32 at the end), so that a gradient that all positions share does
//     not round every entry the same way.
#include "gemm_tc.cuh"
#include "train_internal.cuh"

#include <algorithm>
#include <mutex>

#include "tc_ptx.cuh"

namespace {

using namespace tc;

constexpr int TILE = 256;              // rows and columns of a tile (a CTA holds 128 of the rows)
constexpr int BK = 64;
constexpr int NUM_THREADS = 192;
constexpr uint32_t HALF_BYTES = 128 * BK * 2;          // this CTA's half of one operand's K step
constexpr uint32_t STAGE_BYTES = 2 * HALF_BYTES;
constexpr int STAGES = 6;
constexpr uint32_t OUT_OFF = STAGES * STAGE_BYTES;     // two 4 KB staging boxes per epilogue warp
constexpr uint32_t BAR_OFF = OUT_OFF + 4 * 2 * 4096;
constexpr int N_BARS = 2 * STAGES + 5;
constexpr uint32_t SMEM_BYTES = BAR_OFF + N_BARS * 8 + 16 + 1024;   // + alignment slack
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
constexpr uint32_t TMEM_COLS = 512;    // two accumulators of 256 columns
constexpr float LOG2E = 1.4426950408889634f;

// What the rows and gather kernels prepare, and the kernels after them read.
struct Rows {
    int* count;             // counted positions
    float* gmax;            // largest finite magnitude of their upstream gradients, 1 if that is 0 (backward)
    int32_t* list;          // [N] their positions, ascending
    int32_t* index;         // [N] a position's place in the list, or -1 (backward)
    bf16* x;                // [Np, H] their states; rows up to the next multiple of 256 are zero
    int32_t* target;        // [Np]
    float* lse2;            // [Np] lse / ln 2 (backward)
    float* ratio;           // [Np] upstream gradient / gmax (backward)
};

// ---------------------------------------------------------------------------
// before the products
// ---------------------------------------------------------------------------

// Lists the counted positions.  One block: each warp counts its slice, then
// writes it behind the slices before it.  Forward (gloss NULL) also zeroes the
// outputs of the positions that are not counted.
__global__ void __launch_bounds__(1024) vocab_rows_kernel(const int32_t* __restrict__ targets, int N, int V, int ignore_id,
                                                          const float* __restrict__ gloss, float* loss, float* lse, Rows r,
                                                          unsigned int* status) {
    __shared__ int warp_n[32];
    __shared__ float warp_g[32];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slice = ((N + 1023) / 1024) * 32;
    const int lo = min(N, warp * slice), hi = min(N, lo + slice);
    int n = 0;
    float g = 0.f;
    bool out_of_range = false;
#pragma unroll 4
    for (int i = lo + lane; i < hi; i += 32) {
        const int t = targets[i];
        const bool live = t >= 0 && t < V && t != ignore_id;
        out_of_range |= !live && t != ignore_id;
        n += live;
        if (live && gloss) {
            const float a = fabsf(gloss[i]);
            if (a < INFINITY) g = fmaxf(g, a);
        }
    }
    if (out_of_range) atomicOr(status, TEE_STATUS_BAD_ID);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        n += __shfl_xor_sync(0xffffffffu, n, o);
        g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    }
    if (lane == 0) warp_n[warp] = n, warp_g[warp] = g;
    __syncthreads();
    int at = 0;
    for (int w = 0; w < warp; ++w) at += warp_n[w];
    if (threadIdx.x == 1023) *r.count = at + n;
    if (threadIdx.x == 0 && gloss) {
        for (int w = 0; w < 32; ++w) g = fmaxf(g, warp_g[w]);
        *r.gmax = g > 0.f ? g : 1.f;
    }
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        const int t = i < hi ? targets[i] : ignore_id;
        const bool live = i < hi && t >= 0 && t < V && t != ignore_id;
        const unsigned m = __ballot_sync(0xffffffffu, live);
        const int place = at + __popc(m & ((1u << lane) - 1));
        if (live) r.list[place] = i;
        if (gloss) {
            if (i < hi) r.index[i] = live ? place : -1;
        } else if (i < hi && !live) {
            loss[i] = 0.f;
            lse[i] = 0.f;
        }
        at += __popc(m);
    }
}

// Copies the listed rows together, one warp per row, and zeroes the rest of the last tile.
__global__ void __launch_bounds__(256) vocab_gather_kernel(const bf16* __restrict__ x, const int32_t* __restrict__ targets,
                                                           const float* __restrict__ lse, const float* __restrict__ gloss,
                                                           int H, Rows r) {
    pdl_wait();
    pdl_trigger();
    const int c = (blockIdx.x * 256 + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    const int n = *r.count;
    if (c >= (n + TILE - 1) / TILE * TILE) return;
    const bool live = c < n;
    const int i = live ? r.list[c] : 0;
    const uint4* src = reinterpret_cast<const uint4*>(x + (size_t)i * H);
    uint4* dst = reinterpret_cast<uint4*>(r.x + (size_t)c * H);
#pragma unroll 4
    for (int k = lane; k < H / 8; k += 32) dst[k] = live ? src[k] : make_uint4(0, 0, 0, 0);
    if (lane == 0) {
        r.target[c] = live ? targets[i] : -1;
        if (gloss) {
            r.lse2[c] = live ? lse[i] * LOG2E : 0.f;
            r.ratio[c] = live ? gloss[i] / *r.gmax : 0.f;
        }
    }
}

// ---------------------------------------------------------------------------
// the products
// ---------------------------------------------------------------------------

enum Kind { LOGITS, DX, DW };

struct Maps {
    CUtensorMap x, w;               // K-major operands of the logits: boxes of 64 columns x 128 rows
    CUtensorMap d;                  // D of the piece being multiplied, K-major (D W)
    CUtensorMap w_mn, d_mn, x_mn;   // MN-major operands: boxes of 64 columns x 64 rows
    CUtensorMap d_out, dx_acc, dw;  // outputs: boxes of 32 rows x 128 bytes
};

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
    unsigned int* status;
};

// How many slices of a piece's columns the tiles of D W are split into, each
// with accumulators of its own: enough tiles for two per CTA pair, as far as the
// accumulators reach and a slice has at least four K steps.
__device__ __forceinline__ int dx_slices(int mt, int ht, int pairs, int acc_rows, int n_mul) {
    const int want = (2 * pairs + mt * ht - 1) / (mt * ht);
    return max(1, min(min(want, acc_rows / (mt * TILE)), n_mul / (4 * BK)));
}

struct Unit {
    int kind, m, n, k0, num_k, slice;   // tile (m, n); K steps k0 .. k0 + num_k
};

// The launch's units: D^T X and D W (the longer first), then the logits, whose
// short tiles even out what the long ones leave.
struct Plan {
    int mt, ht, n_dw, n_dx, n_log, slices, k_slice, k_rows, k_mul, kh;
    bool dx_first;
    template <bool BWD>
    static __device__ __forceinline__ Plan make(const Params& p, int count, int pairs) {
        Plan q;
        q.mt = (count + TILE - 1) / TILE;
        q.ht = (p.H + TILE - 1) / TILE;
        q.kh = (p.H + BK - 1) / BK;
        q.n_log = q.mt * ((p.n_log + TILE - 1) / TILE);
        q.n_dw = q.n_dx = 0;
        q.slices = 1;
        q.k_slice = q.k_rows = q.k_mul = 0;
        q.dx_first = false;
        if (BWD && p.n_mul) {
            q.k_rows = (count + BK - 1) / BK;
            q.k_mul = (p.n_mul + BK - 1) / BK;
            if (p.want_dw) q.n_dw = (p.n_mul + TILE - 1) / TILE * q.ht;
            if (p.want_dx && q.mt) {
                q.slices = dx_slices(q.mt, q.ht, pairs, p.acc_rows, p.n_mul);
                q.k_slice = (q.k_mul + q.slices - 1) / q.slices;
                q.n_dx = q.mt * q.ht * q.slices;
            }
            q.dx_first = q.k_slice > q.k_rows;
        }
        return q;
    }
    __device__ __forceinline__ int units() const { return n_dw + n_dx + n_log; }
    template <bool BWD>
    __device__ __forceinline__ Unit unit(int u) const {
        if constexpr (BWD) {
            const int a = dx_first ? n_dx : n_dw;
            if (u < n_dw + n_dx) {
                const bool dx = (u < a) == dx_first;
                if (u >= a) u -= a;
                const int n = u % ht, rest = u / ht;
                if (!dx) return Unit{DW, rest, n, 0, k_rows, 0};
                const int s = rest / mt, k0 = s * k_slice;
                return Unit{DX, rest % mt, n, k0, max(0, min(k_slice, k_mul - k0)), s};
            }
            u -= n_dw + n_dx;
        }
        return Unit{LOGITS, u % mt, u / mt, 0, kh, 0};
    }
};

template <bool BWD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
    vocab_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_OFF);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + N_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    auto bar = [&](int i) { return smem_u32(bars + i); };
    constexpr int FULL = 0, EMPTY = STAGES, TFULL = 2 * STAGES, TEMPTY = 2 * STAGES + 2, MMA_DONE = 2 * STAGES + 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank();
    auto lead_bar = [&](int i) { return mapa_shared(bar(i), 0); };   // the even CTA's, which both CTAs signal

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar(FULL + s), 1);
            mbar_init(bar(EMPTY + s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar(TFULL + a), 1);
            mbar_init(bar(TEMPTY + a), 256);   // every epilogue thread of both CTAs
        }
        mbar_init(bar(MMA_DONE), 1);
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

    const int count = __ldcg(p.r.count);
    const int unit0 = blockIdx.x / 2, ustride = gridDim.x / 2;
    const Plan plan = Plan::make<BWD>(p, count, ustride);
    const int num_units = plan.units();

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        if (lane == 0) {
            uint32_t g = 0;
            bool armed[STAGES], ok = true;
            uint32_t armed_parity[STAGES];
            for (int s = 0; s < STAGES; ++s) armed[s] = false, armed_parity[s] = 0;
            for (int u = unit0; u < num_units && ok; u += ustride) {
                const Unit w = plan.unit<BWD>(u);
                const int a0 = w.m * TILE + (int)crank * 128, b0 = w.n * TILE + (int)crank * 128;
                for (int kb = 0; kb < w.num_k; ++kb, ++g) {
                    const int s = g % STAGES;
                    const uint32_t r = g / STAGES;
                    if (!mbar_wait(bar(EMPTY + s), (r & 1) ^ 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = sbase + s * STAGE_BYTES, sb = sa + HALF_BYTES;
                    const int k = (w.k0 + kb) * BK;
                    const uint32_t full = lead_bar(FULL + s);
                    if (crank == 0) {   // its barrier expects both CTAs' halves
                        mbar_expect_tx(bar(FULL + s), 2 * STAGE_BYTES);
                        armed[s] = true;
                        armed_parity[s] = r & 1;
                    }
                    if (!BWD || w.kind == LOGITS) {
                        tma_load_2d_pair(sa, &maps.x, k, a0, full);
                        tma_load_2d_pair(sb, &maps.w, k, p.v_log + b0, full);
                    } else if (w.kind == DX) {
                        tma_load_2d_pair(sa, &maps.d, k, a0, full);
                        tma_load_2d_pair(sb, &maps.w_mn, b0, p.v_mul + k, full);
                        tma_load_2d_pair(sb + HALF_BYTES / 2, &maps.w_mn, b0 + 64, p.v_mul + k, full);
                    } else {
                        tma_load_2d_pair(sa, &maps.d_mn, a0, k, full);
                        tma_load_2d_pair(sa + HALF_BYTES / 2, &maps.d_mn, a0 + 64, k, full);
                        tma_load_2d_pair(sb, &maps.x_mn, b0, k, full);
                        tma_load_2d_pair(sb + HALF_BYTES / 2, &maps.x_mn, b0 + 64, k, full);
                    }
                }
            }
            // no copy may still be landing in shared memory when the CTA exits
            for (int s = 0; s < STAGES; ++s)
                if (armed[s]) mbar_wait_drain(bar(FULL + s), armed_parity[s]);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issuer (the even CTA's, for both) ----------------
        if (lane == 0 && crank == 0) {
            uint32_t g = 0;
            int it = 0;
            bool ok = true;
            for (int u = unit0; u < num_units && ok; u += ustride, ++it) {
                const Unit w = plan.unit<BWD>(u);
                const int acc = it & 1, use = it >> 1;
                if (!mbar_wait_cluster(bar(TEMPTY + acc), (use & 1) ^ 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * TILE;
                const bool a_mn = BWD && w.kind == DW, b_mn = BWD && w.kind != LOGITS;
                const uint32_t idesc = make_idesc(2 * 128, TILE) | (a_mn ? IDESC_A_MN_MAJOR : 0) | (b_mn ? IDESC_B_MN_MAJOR : 0);
                // a K step of 16: 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major group
                const uint32_t a_step = a_mn ? 128 : 2, b_step = b_mn ? 128 : 2;
                for (int kb = 0; kb < w.num_k; ++kb, ++g) {
                    const int s = g % STAGES;
                    if (!mbar_wait_cluster(bar(FULL + s), (g / STAGES) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = sbase + s * STAGE_BYTES, sb = sa + HALF_BYTES;
                    const uint64_t ad = a_mn ? sw128_desc_mn_groups(sa, HALF_BYTES / 2) : sw128_desc(sa);
                    const uint64_t bd = b_mn ? sw128_desc_mn_groups(sb, HALF_BYTES / 2) : sw128_desc(sb);
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k)
                        mma_bf16_pair(d_tmem, ad + k * a_step, bd + k * b_step, idesc, (kb | k) != 0);
                    mma_commit_pair(bar(EMPTY + s), 0x3);   // both CTAs' stage s
                }
                if (!ok) break;
                mma_commit_pair(bar(TFULL + acc), 0x3);     // both CTAs' accumulator halves
            }
            // every MMA issued must be finished before TMEM is freed
            mma_commit_pair(bar(MMA_DONE), 0x1);
            mbar_wait_drain(bar(MMA_DONE), 0);
        }
        __syncwarp();
    } else {
        // ---------------- epilogue (warps 2..5): thread = row of the accumulator ----------------
        const int quad = warp & 3;
        uint8_t* stage = smem + OUT_OFF + (warp - 2) * 8192;   // this warp's two staging boxes
        uint32_t n_stores = 0;
        auto box = [&]() {   // the next box, free to be written
            if (lane == 0 && n_stores >= 2) bulk_wait_read<1>();
            __syncwarp();
            return stage + (n_stores & 1) * 4096;
        };
        auto send = [&](auto&& issue) {   // lane 0 stores the box just written
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                issue(smem_u32(stage + (n_stores & 1) * 4096));
                bulk_commit();
            }
            ++n_stores;
        };
        const float gmax = BWD ? __ldcg(p.r.gmax) : 0.f;
        int it = 0;
        for (int u = unit0; u < num_units; u += ustride, ++it) {
            const Unit w = plan.unit<BWD>(u);
            const int acc = it & 1, use = it >> 1;
            const int row0 = w.m * TILE + (int)crank * 128 + quad * 32, row = row0 + lane;
            const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + acc * TILE;
            if constexpr (!BWD) {
                const int target = p.r.target[row] - w.n * TILE;   // within this tile's columns, if it is there
                if (!mbar_wait(bar(TFULL + acc), use & 1, abort_flag)) break;
                tc_fence_after();
                float top = -INFINITY, ref = -INFINITY, sum = 0.f;
#pragma unroll 1
                for (int c = 0; c < TILE; c += 64) {
                    float v[64];
                    tmem_ld64(taddr + c, v);
                    if (w.n * TILE + c + 64 > p.V) {
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (w.n * TILE + c + j >= p.V) v[j] = -INFINITY;
                    }
                    const int tj = target - c;
                    if (__any_sync(0xffffffffu, tj >= 0 && tj < 64)) {
                        float tv = 0.f;
#pragma unroll
                        for (int j = 0; j < 64; ++j) tv = j == tj ? v[j] : tv;
                        if (tj >= 0 && tj < 64) p.target_logit[row] = tv;
                    }
                    float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                    for (int j = 4; j < 64; ++j) mx[j & 3] = fmaxf(mx[j & 3], v[j]);
                    top = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                    // exponentials are taken against the running maximum; one that is
                    // infinite would give NaN where the sum is 0 or infinite
                    const float to = isinf(top) ? 0.f : top * LOG2E;
                    sum *= ex2_approx(ref - to);
                    float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < 64; ++j) s4[j & 3] += ex2_approx(fmaf(v[j], LOG2E, -to));
                    sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
                    ref = top == -INFINITY ? -INFINITY : to;
                }
                if (row < count) p.part[(size_t)w.n * p.Np + row] = make_float2(ref, sum);
            } else if (w.kind == LOGITS) {
                const float lse2 = p.r.lse2[row], ratio = p.r.ratio[row];
                const int target = p.r.target[row] - p.v_log - w.n * TILE;
                if (!mbar_wait(bar(TFULL + acc), use & 1, abort_flag)) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < TILE; c += 64) {
                    float v[64];
                    tmem_ld64(taddr + c, v);
#pragma unroll
                    for (int j = 0; j < 64; ++j) v[j] = ex2_approx(fmaf(v[j], LOG2E, -lse2));
                    const int tj = target - c;
                    if (__any_sync(0xffffffffu, tj >= 0 && tj < 64)) {
#pragma unroll
                        for (int j = 0; j < 64; ++j) v[j] -= j == tj ? 1.f : 0.f;
                    }
                    // rows of padding are zero whatever the table holds
#pragma unroll
                    for (int j = 0; j < 64; ++j) v[j] = row < count ? v[j] * ratio : 0.f;
                    stage_row_bf16x64(box(), lane, v);
                    send([&](uint32_t src) { tma_store_2d(&maps.d_out, src, w.n * TILE + c, row0); });
                }
            } else if (w.kind == DX) {
                if (!mbar_wait(bar(TFULL + acc), use & 1, abort_flag)) break;
                tc_fence_after();
                const int y = w.slice * plan.mt * TILE + row0;
#pragma unroll 1
                for (int c = 0; c < TILE; c += 32) {
                    const int x = w.n * TILE + c;
                    if (x >= p.H) break;
                    float v[32];
                    tmem_ld32(taddr + c, v);
                    uint8_t* b = box() + lane * 128;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<float4*>(b + ((k ^ (lane & 7)) << 4)) =
                            w.num_k ? make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
                    // each element is added to once a launch: the order of the sums is fixed
                    send([&](uint32_t src) {
                        if (p.first) tma_store_2d(&maps.dx_acc, src, x, y);
                        else tma_reduce_add_2d(&maps.dx_acc, src, x, y);
                    });
                }
            } else {
                if (!mbar_wait(bar(TFULL + acc), use & 1, abort_flag)) break;
                tc_fence_after();
                const int y = p.v_mul + row0;
#pragma unroll 1
                for (int c = 0; c < TILE; c += 64) {
                    const int x = w.n * TILE + c;
                    if (x >= p.H) break;
                    float v[64];
                    tmem_ld64(taddr + c, v);
#pragma unroll
                    for (int j = 0; j < 64; ++j) v[j] = w.num_k ? v[j] * gmax : 0.f;
                    stage_row_bf16x64(box(), lane, v);
                    if (y < p.V) send([&](uint32_t src) { tma_store_2d(&maps.dw, src, x, y); });
                }
            }
            tc_fence_before();
            mbar_arrive_cluster(lead_bar(TEMPTY + acc));
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
__global__ void __launch_bounds__(512) vocab_finish_kernel(const float2* __restrict__ part, const float* __restrict__ target_logit,
                                                           Rows r, int tiles, int Np, float* __restrict__ loss,
                                                           float* __restrict__ lse) {
    __shared__ float2 red[16][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int row = blockIdx.x * 32 + lane, n = *r.count;
    if (blockIdx.x * 32 >= n) return;
    float2 a = make_float2(-INFINITY, 0.f);
    auto join = [](float2 a, float2 b) {
        const float to = fmaxf(a.x, b.x);
        if (to == -INFINITY) return make_float2(-INFINITY, a.y + b.y);
        return make_float2(to, a.y * exp2f(a.x - to) + b.y * exp2f(b.x - to));
    };
    if (row < n) {
#pragma unroll 4
        for (int t = sl; t < tiles; t += 16) a = join(a, part[(size_t)t * Np + row]);
    }
    red[sl][lane] = a;
    __syncthreads();
    if (sl || row >= n) return;
    for (int s = 1; s < 16; ++s) a = join(a, red[s][lane]);
    const double l = ((double)a.x + log2((double)a.y)) * 0.69314718055994530942;
    const int i = r.list[row];
    lse[i] = (float)l;
    loss[i] = (float)(l - (double)target_logit[row]);
}

// dX of every position: gmax times the sum of its accumulators, or zeros.
// n_mul: the columns of the first piece, whose products wrote every slice.
__global__ void __launch_bounds__(256) vocab_scatter_kernel(const float* __restrict__ acc, Rows r, int N, int H, int n_mul,
                                                            int acc_rows, int pairs, bf16* __restrict__ dx) {
    pdl_wait();
    pdl_trigger();
    const int i = (blockIdx.x * 256 + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    if (i >= N) return;
    const int at = r.index[i];
    const float gmax = *r.gmax;
    const int mt = (*r.count + TILE - 1) / TILE;
    const int slices = at < 0 ? 0 : dx_slices(mt, (H + TILE - 1) / TILE, pairs, acc_rows, n_mul);
    for (int k = lane; k < H / 8; k += 32) {
        float v[8] = {};
        for (int s = 0; s < slices; ++s) {
            float a[8];
            load8(acc + ((size_t)s * mt * TILE + at) * H + 8 * k, a);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += a[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= slices ? gmax : 0.f;
        store8(dx + (size_t)i * H + 8 * k, v);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

int round_up(int v, int a) { return (int)(((long long)v + a - 1) / a * a); }

// Columns of a backward piece: D at most 256 MB for as many rows as there are
// positions, 2048 columns at least.
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
    size_t bytes = 0;
};
LossWs carve_loss(int N, int V, int H, bool backward, void* base) {
    WsCarve ws(base);
    LossWs w;
    const int Np = round_up(N, TILE);
    w.r.count = ws.take<int>(1);
    w.r.gmax = ws.take<float>(1);
    w.r.list = ws.take<int32_t>(N);
    w.r.x = ws.take<bf16>((size_t)Np * H);
    w.r.target = ws.take<int32_t>(Np);
    if (!backward) {
        w.target_logit = ws.take<float>(Np);
        w.part = ws.take<float2>((size_t)Np * ((V + TILE - 1) / TILE));
    } else {
        w.r.index = ws.take<int32_t>(N);
        w.r.lse2 = ws.take<float>(Np);
        w.r.ratio = ws.take<float>(Np);
        const int vc = piece_columns(Np, V);
        for (int b = 0; b < (vc < V ? 2 : 1); ++b) w.d[b] = ws.take<bf16>((size_t)Np * vc);
        w.acc = ws.take<float>((size_t)accumulator_rows(Np, H) * H);
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
        cfg.blockDim = dim3(NUM_THREADS);
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
        of[dev] = std::max(1, n);
    }
    *pairs = of[dev];
    return cudaSuccess;
}

#define TRY(call)                           \
    do {                                    \
        const cudaError_t e_ = (call);      \
        if (e_ != cudaSuccess) return e_;   \
    } while (0)

cudaError_t prepare_rows(const void* x, const int32_t* targets, const float* lse_in, const float* gloss, float* loss,
                         float* lse, int N, int V, int H, int ignore_id, const LossWs& w, unsigned int* status, cudaStream_t s) {
    TRY(launch_pdl(vocab_rows_kernel, dim3(1), dim3(1024), 0, s, targets, N, V, ignore_id, gloss, loss, lse, w.r, status));
    return launch_pdl(vocab_gather_kernel, dim3(round_up(N, TILE) / 8), dim3(256), 0, s, (const bf16*)x, targets, lse_in, gloss,
                      H, w.r);
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
    TRY(prepare_rows(x, targets, nullptr, nullptr, loss, lse, N, V, H, ignore_id, w, status, s));
    const int grid = 2 * std::min(pairs, Np / TILE * tiles);
    TRY(launch_pdl(vocab_kernel<false>, dim3(grid), dim3(NUM_THREADS), SMEM_BYTES, s, maps, p));
    return launch_pdl(vocab_finish_kernel, dim3(round_up(N, 32) / 32), dim3(512), 0, s, (const float2*)w.part,
                      (const float*)w.target_logit, w.r, tiles, Np, loss, lse);
}

cudaError_t launch_vocab_loss_backward(const void* x, const void* wt, const int32_t* targets, const float* lse,
                                       const float* gloss, void* dx, void* dw, int N, int V, int H, int ignore_id, void* ws,
                                       unsigned int* status, cudaStream_t s) {
    if (N == 0) return dw ? cudaMemsetAsync(dw, 0, (size_t)V * H * sizeof(bf16), s) : cudaSuccess;
    int dev = 0, num_sms = 0, pairs = 0;
    TRY(tee_current_device(&dev, &num_sms));
    TRY(max_pairs<true>(dev, num_sms, &pairs));
    const int Np = round_up(N, TILE), vc = piece_columns(Np, V);
    const LossWs w = carve_loss(N, V, H, true, ws);
    Maps maps{};
    TRY(make_tensor_map_2d(&maps.x, false, w.r.x, Np, H, H, 128, 64));
    TRY(make_tensor_map_2d(&maps.w, false, wt, V, H, H, 128, 64));
    TRY(make_tensor_map_2d(&maps.w_mn, false, wt, V, H, H, 64, 64));
    TRY(make_tensor_map_2d(&maps.x_mn, false, w.r.x, Np, H, H, 64, 64));
    const int acc_rows = accumulator_rows(Np, H);
    TRY(make_tensor_map_2d(&maps.dx_acc, true, w.acc, acc_rows, H, H, 32, 32));
    if (dw) TRY(make_tensor_map_2d(&maps.dw, false, dw, V, H, H, 32, 64));
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
    TRY(prepare_rows(x, targets, lse, gloss, nullptr, nullptr, N, V, H, ignore_id, w, status, s));
    const int pieces = (V + vc - 1) / vc;
    for (int i = 0; i <= pieces; ++i) {
        // logits of piece i into one buffer, products of piece i - 1 out of the other
        p.v_log = i < pieces ? i * vc : 0;
        p.n_log = i < pieces ? std::min(vc, V - p.v_log) : 0;
        p.v_mul = i > 0 ? (i - 1) * vc : 0;
        p.n_mul = i > 0 ? std::min(vc, V - p.v_mul) : 0;
        p.first = i == 1;
        if (i < pieces) maps.d_out = d_out[i & 1];
        if (i > 0) maps.d = d_in[(i - 1) & 1], maps.d_mn = d_mn[(i - 1) & 1];
        TRY(launch_pdl(vocab_kernel<true>, dim3(2 * pairs), dim3(NUM_THREADS), SMEM_BYTES, s, maps, p));
    }
    if (!dx) return cudaSuccess;
    return launch_pdl(vocab_scatter_kernel, dim3(round_up(N, 8) / 8), dim3(256), 0, s, (const float*)w.acc, w.r, N, H,
                      std::min(vc, V), acc_rows, pairs, (bf16*)dx);
}
