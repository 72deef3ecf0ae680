// The gated half of the feed-forward block, z = GELU(x Wa^T) (x Wg^T), and its
// gradients, on the 5th-generation tensor cores (tcgen05, sm_103a); tee_train.h has the
// formulas.
//
// One persistent kernel of CTA pairs (tcgen05 cta_group::2, 256 x 256 tiles, K steps
// of 64, TMA-fed ring) runs every product.
//   * Both projections lie in one accumulator: the even CTA brings 128 rows of Wa, the
//     odd one the same 128 rows of Wg, so that each has a and g of its 128 rows of x
//     side by side, and the activation and the product are taken as they leave tensor
//     memory.
//   * Backward keeps nothing of the forward pass but x: a and g are computed again,
//     and dU = [da | dg] is written in bf16, from which dX = dU Wi and dWi = dU^T X are
//     made with the transposed operands read as they lie, as MN-major tiles.
//   * Rows are taken in parts: a launch multiplies the dU of one part and makes that of
//     the next, its tiles shared out among the CTA pairs by their length.
// Work: 4 T I H flops forward, 12 T I H backward; both are bound by the tensor cores and
// their power.  Measured at 32768 x 768 x 3072: forward 192 us, 1610 TFLOP/s (pipes 87 %
// busy); backward 625 to 640 us, 1450 to 1480 TFLOP/s: dU 224 us with the pipes 62 % busy --
// operands, dz, da and dg all cross shared memory, 7500 cycles of it a tile by the bytes
// where the products are 6144; 9900 are measured --, its products 332 us and 88 %.
// 1051 rows: backward 40 us of GPU time in three launches, two rounds of tiles in the first.
#include "gemm_tc.cuh"
#include "train_internal.cuh"

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "tc_ptx.cuh"

namespace {

using namespace tc;

constexpr int TILE = 256;              // rows and columns of a tile (a CTA holds 128 of the rows)
constexpr int HALF = 128;              // columns of z in a tile
constexpr int BK = 64;
constexpr int EPI_WARPS = 8;           // two per quarter of the accumulator's rows
constexpr int NUM_THREADS = 64 + 32 * EPI_WARPS;
constexpr int MAX_PAIRS = 128;
constexpr uint32_t HALF_BYTES = 128 * BK * 2;
constexpr uint32_t STAGE_BYTES = 2 * HALF_BYTES;
// Stages of operands, and 4 KB boxes of each epilogue warp: one for stores, backward
// another that dz comes in.  (Read by the threads from their rows instead, dz comes 2.7
// times out of DRAM: 16 bytes of a sector each, and hardly any L1 beside this much shared
// memory.)
template <bool BWD>
struct Smem {
    static constexpr int STAGES = BWD ? 5 : 6, BOXES = BWD ? 2 : 1;
    static constexpr uint32_t OUT_OFF = STAGES * STAGE_BYTES;
    static constexpr uint32_t BAR_OFF = OUT_OFF + EPI_WARPS * BOXES * 4096;
    static constexpr int N_BARS = 2 * STAGES + 5 + EPI_WARPS;
    static constexpr uint32_t BYTES = BAR_OFF + N_BARS * 8 + 16 + 1024;
};
static_assert(Smem<true>::BYTES <= 227 * 1024 && Smem<false>::BYTES <= 227 * 1024, "shared memory");
constexpr uint32_t TMEM_COLS = 512;    // two accumulators of 256 columns
constexpr int EPILOGUE_K_STEPS = 8;    // a tile's epilogue, in K steps of products
// Slices of a sum: tiles that are too few for all CTA pairs are split along K, into so
// many tiles of fp32 sums at most.
constexpr int ACC_TILES = MAX_PAIRS;
constexpr int SLICE_K_STEPS = 4;       // at least

enum Kind { UP, DX, DW };

struct Maps {
    CUtensorMap x, wi;                  // K-major operands of the projections: boxes of 64 columns x 128 rows
    CUtensorMap du;                     // dU of the part being multiplied, K-major
    CUtensorMap wi_mn, du_mn, x_mn;     // MN-major operands: boxes of 64 columns x 64 rows
    CUtensorMap z;                      // z, or da of the part being made (backward): boxes of 32 rows x 64 columns
    CUtensorMap dz;                     // boxes of 32 rows x 64 columns
    CUtensorMap dg, dx, dw;             // outputs (dx and dw: bf16, or the slices' fp32 sums in boxes of 32 columns)
};

// The CTA pairs' shares of a launch: of each kind so many units.  A pair's r-th unit is
// taken in round r: the kind's units go to the pairs that have one in the round in turn,
// so that pairs running at the same time share operands in L2.
struct Shares {
    int n[3][MAX_PAIRS];   // by Kind
};

struct Params {
    int H, I;
    // part being made: rows [up0, up0 + up_rows); being multiplied: rows [mul0, mul0 + mul_rows)
    int up0, up_rows, mul0, mul_rows;
    int dx_slices, dw_slices, dx_steps, dw_steps;   // slices, and K steps of each
    int dx_f32, dw_f32, dw_add;         // sums in fp32; dw added to what is there
    unsigned int* status;
    Shares shares;
};

struct Unit {
    int kind, m, n, k0, num_k, slice;   // tile (m, n); K steps k0 .. k0 + num_k
};

__host__ __device__ __forceinline__ int tiles_of(int v, int tile) { return (v + tile - 1) / tile; }

struct Tiles {
    int nt_up, ht, kh, mt_mul, it, k_rows, k_cols, dx_steps, dw_steps;
    __device__ __forceinline__ Tiles(const Params& p) {
        nt_up = tiles_of(p.I, HALF);
        ht = tiles_of(p.H, TILE);
        kh = tiles_of(p.H, BK);
        mt_mul = tiles_of(p.mul_rows, TILE);
        it = tiles_of(2 * p.I, TILE);
        k_rows = tiles_of(p.mul_rows, BK);
        k_cols = tiles_of(2 * p.I, BK);
        dx_steps = p.dx_steps, dw_steps = p.dw_steps;
    }
    __device__ __forceinline__ Unit unit(int kind, int u) const {
        if (kind == UP) return Unit{UP, u / nt_up, u % nt_up, 0, kh, 0};
        const int n = u % ht, rest = u / ht;
        if (kind == DX) {
            const int s = rest / mt_mul, k0 = s * dx_steps;
            return Unit{DX, rest % mt_mul, n, k0, max(0, min(dx_steps, k_cols - k0)), s};
        }
        const int s = rest / it, k0 = s * dw_steps;
        return Unit{DW, rest % it, n, k0, max(0, min(dw_steps, k_rows - k0)), s};
    }
};

// The units a CTA pair takes, in the order it takes them (by a whole warp).
template <bool BWD>
struct Walk {
    const Params& p;
    int pair, pairs, kind, round;
    __device__ __forceinline__ Walk(const Params& p_, int pair_, int pairs_)
        : p(p_), pair(pair_), pairs(pairs_), kind(BWD ? (int)DW : (int)UP), round(0) { skip(); }
    __device__ __forceinline__ void skip() {
        while (BWD && kind > UP && round >= p.shares.n[kind][pair]) --kind, round = 0;   // DW, DX, UP
    }
    __device__ __forceinline__ bool done() const { return kind == UP && round >= p.shares.n[UP][pair]; }
    __device__ __forceinline__ Unit next(const Tiles& t) {
        int u = 0;   // units of the rounds before, and of this round for the pairs before
        for (int q = threadIdx.x & 31; q < pairs; q += 32) {
            const int n = p.shares.n[kind][q];
            u += min(n, round) + (q < pair && n > round);
        }
        const Unit w = t.unit(kind, __reduce_add_sync(0xffffffffu, u));
        ++round;
        skip();
        return w;
    }
};

// da and dg of two elements.  GELU(a) = a Phi(a) and GELU'(a) = Phi(a) + a phi(a); Phi by
// the rational approximation of erf of Abramowitz & Stegun, formula 7.1.26, as in
// gelu_as, whose exponential is phi's too: with q = t (a1 + t (a2 + ...)) exp(-a^2 / 2),
// t = 1 / (1 + p |a| / sqrt 2), Phi(-|a|) = q / 2 (error below 1e-7).  On the packed fp32x2
// instructions.
__device__ __forceinline__ void geglu_grad2(float& a0, float& a1, float& g0, float& g1, float z0, float z1) {
    constexpr float P = 0.3275911f * 0.70710678118654752f;
    constexpr float H1 = 0.5f * 0.254829592f, H2 = 0.5f * -0.284496736f, H3 = 0.5f * 1.421413741f,
                    H4 = 0.5f * -1.453152027f, H5 = 0.5f * 1.061405429f;
    constexpr float NEG_HALF_LOG2E = -0.72134752044448170f, INV_SQRT_2PI = 0.39894228040143268f;
    auto both = [](float v) { return f2_pack(v, v); };
    float x0, x1, y0, y1;
    const uint64_t A = f2_pack(a0, a1), Z = f2_pack(z0, z1);
    f2_unpack(f2_fma(f2_pack(fabsf(a0), fabsf(a1)), both(P), both(1.0f)), x0, x1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(x0) : "f"(x0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(x1) : "f"(x1));
    const uint64_t T = f2_pack(x0, x1);
    f2_unpack(f2_mul(f2_mul(A, A), both(NEG_HALF_LOG2E)), y0, y1);
    const uint64_t E = f2_pack(ex2_approx(y0), ex2_approx(y1));
    uint64_t q = f2_fma(T, both(H5), both(H4));
    q = f2_fma(T, q, both(H3));
    q = f2_fma(T, q, both(H2));
    q = f2_fma(T, q, both(H1));
    q = f2_mul(f2_mul(T, q), E);
    float q0, q1;
    f2_unpack(q, q0, q1);
    const uint64_t phi = f2_pack(a0 < 0.f ? q0 : 1.f - q0, a1 < 0.f ? q1 : 1.f - q1);
    const uint64_t u = f2_mul(Z, A);
    const uint64_t da = f2_mul(f2_pack(g0, g1), f2_fma(f2_mul(u, both(INV_SQRT_2PI)), E, f2_mul(Z, phi)));
    f2_unpack(f2_mul(u, phi), g0, g1);
    f2_unpack(da, a0, a1);
}

template <bool BWD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
    geglu_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    using S = Smem<BWD>;
    constexpr int STAGES = S::STAGES;
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BAR_OFF);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + S::N_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    auto bar = [&](int i) { return smem_u32(bars + i); };
    constexpr int FULL = 0, EMPTY = STAGES, TFULL = 2 * STAGES, TEMPTY = 2 * STAGES + 2, MMA_DONE = 2 * STAGES + 4,
                  DZ = 2 * STAGES + 5;
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
        for (int w = 0; w < EPI_WARPS; ++w) mbar_init(bar(DZ + w), 1);
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

    const Tiles tiles(p);
    Walk<BWD> walk(p, blockIdx.x / 2, gridDim.x / 2);
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
            if (!BWD || w.kind == UP) {
                const int wrow = (crank ? p.I : 0) + w.n * HALF;
                for (int k = 0; k < k_end && ok; k += BK)
                    ok = step([&](uint32_t sa, uint32_t sb, uint32_t full) {
                        tma_load_2d_pair(sa, &maps.x, k, p.up0 + a0, full);
                        tma_load_2d_pair(sb, &maps.wi, k, wrow, full);
                    });
            } else if (w.kind == DX) {
                for (int k = w.k0 * BK; k < k_end && ok; k += BK)
                    ok = step([&](uint32_t sa, uint32_t sb, uint32_t full) {
                        tma_load_2d_pair(sa, &maps.du, k, a0, full);
                        tma_load_2d_pair(sb, &maps.wi_mn, b0, k, full);
                        tma_load_2d_pair(sb + HALF_BYTES / 2, &maps.wi_mn, b0 + 64, k, full);
                    });
            } else {
                for (int k = w.k0 * BK; k < k_end && ok; k += BK)
                    ok = step([&](uint32_t sa, uint32_t sb, uint32_t full) {
                        tma_load_2d_pair(sa, &maps.du_mn, a0, k, full);
                        tma_load_2d_pair(sa + HALF_BYTES / 2, &maps.du_mn, a0 + 64, k, full);
                        tma_load_2d_pair(sb, &maps.x_mn, b0, p.mul0 + k, full);
                        tma_load_2d_pair(sb + HALF_BYTES / 2, &maps.x_mn, b0 + 64, p.mul0 + k, full);
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
                if (!BWD || w.kind == UP) ok = products(kmajor, kmajor, d_tmem, w.num_k);
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
        // ---------------- epilogue: thread = row; of each tile half its columns ----------------
        const int quad = warp & 3, half = (warp - 2) >> 2;
        uint8_t* const stage = smem + S::OUT_OFF + (warp - 2) * S::BOXES * 4096;   // this warp's staging box
        uint8_t* const dz_box = stage + 4096;                  // (backward) dz comes here, and dg leaves
        const uint32_t dz_bar = bar(DZ + warp - 2);
        int dz_asked = 0, dz_taken = 0;                        // boxes of dz
        auto ask_dz = [&](const Unit& w) {                     // of the warp's rows and columns of a tile
            const int x = w.n * HALF + half * 64, y = w.m * TILE + (int)crank * 128 + quad * 32;
            if (x >= p.I || y >= p.up_rows) return;
            if (lane == 0) {
                bulk_wait_read<0>();
                mbar_expect_tx(dz_bar, 4096);
                tma_load_2d(smem_u32(dz_box), &maps.dz, x, p.up0 + y, dz_bar);
            }
            ++dz_asked;
            __syncwarp();
        };
        auto send = [&](auto&& write, auto&& issue) {
            if (lane == 0) bulk_wait_read<0>();                // the box's last store has read it
            __syncwarp();
            write();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                issue(smem_u32(stage));
                bulk_commit();
            }
        };
        for (int it = 0; !walk.done(); ++it) {
            const Unit w = walk.next(tiles);
            if (BWD && w.kind == UP) ask_dz(w);
            const int acc = it & 1, use = it >> 1;
            const int row0 = w.m * TILE + (int)crank * 128 + quad * 32, row = row0 + lane;
            const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + acc * TILE;
            if (!BWD || w.kind == UP) {
                const int col = w.n * HALF + half * 64;        // of z
                if (!all(mbar_wait(bar(TFULL + acc), use & 1, abort_flag))) break;
                tc_fence_after();
                // 16 columns of a and g at a time, the next on their way while these are worked on: beside the products a
                // load takes 1000 cycles and more
                const bool used = col < p.I && row0 < p.up_rows;
                if (used) {
                    if (BWD) {
                        if (!all(mbar_wait(dz_bar, dz_taken & 1, abort_flag))) break;
                        ++dz_taken;
                        // (asking for dz waited until the stores from both boxes had read them)
                    } else {
                        if (lane == 0) bulk_wait_read<0>();
                        __syncwarp();
                    }
                    float a[2][16], g[2][16];
                    tmem_ld16_issue(taddr + half * 64, a[0]);
                    tmem_ld16_issue(taddr + HALF + half * 64, g[0]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float(&ca)[16] = a[c & 1], (&cg)[16] = g[c & 1];
                        tmem_wait_ld();
                        tmem_tie16(ca);
                        tmem_tie16(cg);
                        if (c < 3) {
                            tmem_ld16_issue(taddr + half * 64 + 16 * (c + 1), a[(c + 1) & 1]);
                            tmem_ld16_issue(taddr + HALF + half * 64 + 16 * (c + 1), g[(c + 1) & 1]);
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {   // eight columns, a 16-byte piece of a box's row
                            const uint32_t at = lane * 128 + ((2 * c + h) ^ (lane & 7)) * 16;
                            uint32_t x[4], y[4];
                            if constexpr (BWD) {
                                const uint4 q = *reinterpret_cast<const uint4*>(dz_box + at);
                                const uint32_t d[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const int k = 8 * h + 2 * j;
                                    float d0, d1;
                                    unpack_bf16x2(d[j], d0, d1);
                                    geglu_grad2(ca[k], ca[k + 1], cg[k], cg[k + 1], d0, d1);
                                    x[j] = pack_bf16(ca[k], ca[k + 1]);
                                    y[j] = pack_bf16(cg[k], cg[k + 1]);
                                }
                                *reinterpret_cast<uint4*>(dz_box + at) = make_uint4(y[0], y[1], y[2], y[3]);
                            } else {
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const int k = 8 * h + 2 * j;
                                    float z0, z1;
                                    gelu_mul2(ca[k], ca[k + 1], cg[k], cg[k + 1], z0, z1);
                                    x[j] = pack_bf16(z0, z1);
                                }
                            }
                            *reinterpret_cast<uint4*>(stage + at) = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * acc);
                if (used) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&maps.z, smem_u32(stage), col, row0);
                        if (BWD) tma_store_2d(&maps.dg, smem_u32(dz_box), col, row0);
                        bulk_commit();
                    }
                }
                continue;
            }
            if constexpr (BWD) {
                const int col0 = w.n * TILE + half * 128;
                if (!all(mbar_wait(bar(TFULL + acc), use & 1, abort_flag))) break;
                tc_fence_after();
                // the accumulator is free once both loads are in registers
                float v[2][64];
                tmem_ld64_issue(taddr + half * 128, v[0]);
                tmem_ld64_issue(taddr + half * 128 + 64, v[1]);
                tmem_wait_ld();
                tmem_tie64(v[0]);
                tmem_tie64(v[1]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * acc);
                const bool is_dx = w.kind == DX, f32 = is_dx ? p.dx_f32 != 0 : p.dw_f32 != 0;
                const CUtensorMap* map = is_dx ? &maps.dx : &maps.dw;
                const int rows = is_dx ? p.mul_rows : 2 * p.I;
                if (row0 >= rows) continue;
                if (!f32) {
                    const int y = (is_dx ? p.mul0 : 0) + row0;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        if (col0 + 64 * c < p.H)
                            send([&]() { stage_row_bf16x64(stage, lane, v[c]); },
                                 [&](uint32_t src) { tma_store_2d(map, src, col0 + 64 * c, y); });
                } else {
                    // fp32 sums.  Each element is added to once a launch: the order of the sums is fixed
                    const int y = w.slice * (is_dx ? tiles.mt_mul : tiles.it) * TILE + row0;
                    const bool add = !is_dx && p.dw_add;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int x = col0 + 32 * c;
                        if (x >= p.H) continue;
                        const float* f = v[c >> 1] + 32 * (c & 1);
                        send(
                            [&]() {
                                uint8_t* b = stage + lane * 128;
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    *reinterpret_cast<float4*>(b + ((k ^ (lane & 7)) << 4)) =
                                        make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
                            },
                            [&](uint32_t src) {
                                if (add) tma_reduce_add_2d(map, src, x, y);
                                else tma_store_2d(map, src, x, y);
                            });
                    }
                }
            }
        }
        if (dz_asked > dz_taken) mbar_wait_drain(dz_bar, dz_taken & 1);   // no copy may still be landing
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

// Sums of slices, rounded: out[i] = sum_s acc[s * stride + i], eight elements a thread; two of them in one launch.
struct Sum {
    const float* acc;
    bf16* out;
    size_t n8, stride;      // eights of elements, elements from slice to slice
    int slices;
};
__global__ void __launch_bounds__(256) geglu_sum_kernel(Sum a, Sum b) {
    pdl_wait();
    pdl_trigger();
    size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    const bool second = i >= a.n8;
    if (second) i -= a.n8;
    const Sum& q = second ? b : a;
    if (i >= q.n8) return;
    float v[8] = {};
#pragma unroll 2
    for (int s = 0; s < q.slices; ++s) {
        float x[4], y[4];
        load_vec(q.acc + s * q.stride + 8 * i, x);
        load_vec(q.acc + s * q.stride + 8 * i + 4, y);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += x[j], v[4 + j] += y[j];
    }
    store_vec(q.out + 8 * i, v);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Rows of a part.  The dW of more rows than that is added up in fp32 from part to part:
// the tensor cores drop part of the last bit of a sum at every step of 16 terms, 2e-4 of
// a sum of 65536 rows whose terms have one sign.
constexpr int PART_ROWS = 65536;

int part_rows(int T) {
    const int parts = tiles_of(T, PART_ROWS);
    return tiles_of(tiles_of(T, parts), TILE) * TILE;
}

// The most slices of `tiles` tiles of `steps` K steps.
int max_slices(int tiles, int steps) { return std::max(1, std::min(ACC_TILES / std::max(tiles, 1), steps / SLICE_K_STEPS)); }

struct GegluWs {
    bf16* du[2] = {nullptr, nullptr};
    float* dx_acc = nullptr;
    float* dw_acc = nullptr;
    size_t bytes = 0;
};
GegluWs carve_geglu(int T, int H, int I, void* base) {
    WsCarve ws(base);
    GegluWs w;
    const int part = part_rows(T), parts = tiles_of(T, part), rows = std::min(part, T);
    const int ht = tiles_of(H, TILE), mt = tiles_of(rows, TILE), it = tiles_of(2 * I, TILE);
    for (int b = 0; b < std::min(parts, 2); ++b) w.du[b] = ws.take<bf16>((size_t)rows * 2 * I);
    const int sx = max_slices(mt * ht, tiles_of(2 * I, BK)), sw = max_slices(it * ht, tiles_of(rows, BK));
    if (sx > 1) w.dx_acc = ws.take<float>((size_t)sx * mt * TILE * H);
    if (sw > 1 || parts > 1) w.dw_acc = ws.take<float>((size_t)(parts > 1 ? 1 : sw) * it * TILE * H);
    w.bytes = ws.off;
    return w;
}

// Shares of a launch: kind by kind, the longest units first, each unit goes to the pair
// with the least work so far -- for all units of a kind at once: the level is searched
// up to which the pairs fill (a pair takes units while its work is below it), and what
// is left goes to pairs that stand at the level exactly.
void make_shares(const int (&units)[3], const int (&steps)[3], int pairs, Shares& sh) {
    int order[3] = {DW, DX, UP};
    std::stable_sort(order, order + 3, [&](int a, int b) { return steps[a] > steps[b]; });
    long long load[MAX_PAIRS] = {};
    for (int kind : order) {
        const long long cost = std::max(steps[kind], EPILOGUE_K_STEPS);
        auto taken = [&](long long x, int p) { return load[p] < x ? (x - load[p] + cost - 1) / cost : 0; };
        auto taken_by_all = [&](long long x) {
            long long f = 0;
            for (int p = 0; p < pairs; ++p) f += taken(x, p);
            return f;
        };
        long long lo = 0, hi = *std::max_element(load, load + pairs) + (units[kind] / pairs + 1) * cost + 1;
        while (hi - lo > 1) {
            const long long mid = (lo + hi) / 2;
            if (taken_by_all(mid) <= units[kind]) lo = mid;
            else hi = mid;
        }
        long long left = units[kind] - taken_by_all(lo);
        for (int p = 0; p < pairs; ++p) {
            long long k = taken(lo, p);
            if (left > 0 && load[p] + k * cost == lo) ++k, --left;
            sh.n[kind][p] = (int)k;
            load[p] += k * cost;
        }
    }
}

template <bool BWD>
cudaError_t max_pairs(int dev, int num_sms, int* pairs) {
    static std::mutex mu;
    static int of[TEE_MAX_DEVICES] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (!of[dev]) {
        cudaError_t e = cudaFuncSetAttribute(geglu_kernel<BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Smem<BWD>::BYTES);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(num_sms / 2 * 2);
        cfg.blockDim = dim3(NUM_THREADS);
        cfg.dynamicSmemBytes = Smem<BWD>::BYTES;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, geglu_kernel<BWD>, &cfg);
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

}  // namespace

size_t geglu_backward_ws(int T, int H, int I) { return carve_geglu(T, H, I, nullptr).bytes; }

cudaError_t launch_geglu_train_forward(const void* x, const void* wi, void* z, int T, int H, int I, unsigned int* status,
                                       cudaStream_t s) {
    if (T == 0) return cudaSuccess;
    int dev = 0, num_sms = 0, pairs = 0;
    TRY(tee_current_device(&dev, &num_sms));
    TRY(max_pairs<false>(dev, num_sms, &pairs));
    Maps maps{};
    TRY(make_tensor_map_2d(&maps.x, false, x, T, H, H, 128, 64));
    TRY(make_tensor_map_2d(&maps.wi, false, wi, 2 * (uint64_t)I, H, H, 128, 64));
    TRY(make_tensor_map_2d(&maps.z, false, z, T, I, I, 32, 64));
    Params p{};
    p.H = H, p.I = I;
    p.up_rows = T;
    p.status = status;
    const int units = tiles_of(T, TILE) * tiles_of(I, HALF);
    pairs = std::min(pairs, units);
    make_shares({units, 0, 0}, {tiles_of(H, BK), 0, 0}, pairs, p.shares);
    return launch_pdl(geglu_kernel<false>, dim3(2 * pairs), dim3(NUM_THREADS), Smem<false>::BYTES, s, maps, p);
}

cudaError_t launch_geglu_train_backward(const void* x, const void* wi, const void* dz, void* dx, void* dwi, int T, int H,
                                        int I, void* ws, unsigned int* status, cudaStream_t s) {
    if (T == 0) return dwi ? cudaMemsetAsync(dwi, 0, 2 * (size_t)I * H * sizeof(bf16), s) : cudaSuccess;
    int dev = 0, num_sms = 0, pairs = 0;
    TRY(tee_current_device(&dev, &num_sms));
    TRY(max_pairs<true>(dev, num_sms, &pairs));
    const GegluWs w = carve_geglu(T, H, I, ws);
    const int part = part_rows(T), parts = tiles_of(T, part);
    const int ht = tiles_of(H, TILE), it = tiles_of(2 * I, TILE), k_cols = tiles_of(2 * I, BK);
    Maps maps{};
    TRY(make_tensor_map_2d(&maps.x, false, x, T, H, H, 128, 64));
    TRY(make_tensor_map_2d(&maps.wi, false, wi, 2 * (uint64_t)I, H, H, 128, 64));
    TRY(make_tensor_map_2d(&maps.wi_mn, false, wi, 2 * (uint64_t)I, H, H, 64, 64));
    TRY(make_tensor_map_2d(&maps.x_mn, false, x, T, H, H, 64, 64));
    Params p{};
    p.H = H, p.I = I;
    TRY(make_tensor_map_2d(&maps.dz, false, dz, T, I, I, 32, 64));
    p.status = status;
    Sum sum_dx{}, sum_dw{};
    for (int i = 0; i <= parts; ++i) {
        // dU of part i into one buffer, the products of part i - 1 out of the other
        p.up0 = i < parts ? i * part : 0;
        p.up_rows = i < parts ? std::min(part, T - p.up0) : 0;
        p.mul0 = i > 0 ? (i - 1) * part : 0;
        p.mul_rows = i > 0 ? std::min(part, T - p.mul0) : 0;
        int units[3] = {tiles_of(p.up_rows, TILE) * tiles_of(I, HALF), 0, 0}, steps[3] = {tiles_of(H, BK), 0, 0};
        if (i < parts) {
            bf16* du = w.du[i & 1];
            TRY(make_tensor_map_2d(&maps.z, false, du, p.up_rows, I, 2 * (uint64_t)I, 32, 64));
            TRY(make_tensor_map_2d(&maps.dg, false, du + I, p.up_rows, I, 2 * (uint64_t)I, 32, 64));
        }
        if (i > 0) {
            const bf16* du = w.du[(i - 1) & 1];
            TRY(make_tensor_map_2d(&maps.du, false, du, p.mul_rows, 2 * (uint64_t)I, 2 * (uint64_t)I, 128, 64));
            TRY(make_tensor_map_2d(&maps.du_mn, false, du, p.mul_rows, 2 * (uint64_t)I, 2 * (uint64_t)I, 64, 64));
            const int mt = tiles_of(p.mul_rows, TILE), k_rows = tiles_of(p.mul_rows, BK);
            auto slices = [&](int tiles, int k) { return std::min(max_slices(tiles, k), std::max(1, pairs / tiles)); };
            if (dx) {
                p.dx_slices = parts > 1 ? 1 : slices(mt * ht, k_cols);
                p.dx_steps = tiles_of(k_cols, p.dx_slices);
                p.dx_slices = tiles_of(k_cols, p.dx_steps);
                p.dx_f32 = p.dx_slices > 1;
                units[DX] = mt * ht * p.dx_slices, steps[DX] = p.dx_steps;
                if (p.dx_f32) {
                    const size_t rows = (size_t)mt * TILE;
                    TRY(make_tensor_map_2d(&maps.dx, true, w.dx_acc, p.dx_slices * rows, H, H, 32, 32));
                    sum_dx = Sum{w.dx_acc, (bf16*)dx, (size_t)T * H / 8, rows * H, p.dx_slices};
                } else {
                    TRY(make_tensor_map_2d(&maps.dx, false, dx, T, H, H, 32, 64));
                }
            }
            if (dwi) {
                p.dw_slices = parts > 1 ? 1 : slices(it * ht, k_rows);
                p.dw_steps = tiles_of(k_rows, p.dw_slices);
                p.dw_slices = tiles_of(k_rows, p.dw_steps);
                p.dw_f32 = p.dw_slices > 1 || parts > 1;
                p.dw_add = i > 1;
                units[DW] = it * ht * p.dw_slices, steps[DW] = p.dw_steps;
                if (p.dw_f32) {
                    const size_t rows = (size_t)it * TILE;
                    TRY(make_tensor_map_2d(&maps.dw, true, w.dw_acc, p.dw_slices * rows, H, H, 32, 32));
                    sum_dw = Sum{w.dw_acc, (bf16*)dwi, 2 * (size_t)I * H / 8, rows * H, p.dw_slices};
                } else {
                    TRY(make_tensor_map_2d(&maps.dw, false, dwi, 2 * (uint64_t)I, H, H, 32, 64));
                }
            }
        }
        make_shares(units, steps, pairs, p.shares);
        TRY(launch_pdl(geglu_kernel<true>, dim3(2 * pairs), dim3(NUM_THREADS), Smem<true>::BYTES, s, maps, p));
    }
    const size_t n8 = sum_dx.n8 + sum_dw.n8;
    if (!n8) return cudaSuccess;
    return launch_pdl(geglu_sum_kernel, dim3((unsigned)((n8 + 255) / 256)), dim3(256), 0, s, sum_dx, sum_dw);
}
