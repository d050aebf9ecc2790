// hq_gemm_fp8.cu -- e4m3 tensor-core GEMM with a scale for each block of 128 (tcgen05 MMA, TMEM
// accumulators, TMA operand loads).
//
//   Y[m, n] = sum_t sa[t, m] sw[t, n / 128] S_{m,n,t},  S_{m,n,t} = sum_{k in block t} A[m, k] W[n, k]
//
// A [M, K] carries one scale per row and 128 columns, W [N, K] one per 128 x 128 block.  A block's sum
// S is one accumulation of four MMAs (K = 32 each) in TMEM; the scales differ from block to block,
// so the epilogue warps take every block's sums out and add them, scaled, in binary32 registers:
// acc = fma(S, sa sw, acc) over t in order.
//
// Persistent CTAs (one per SM) walk the 128 x GN tiles of Y (GN = 128 columns; 64 or 32 where the
// 128-wide tiles are too few to occupy the SMs): warp 0 streams 128-byte wide boxes of A and W into a
// ring with TMA (128-byte swizzle; rows and columns outside the matrices read as zeros), warp 1
// issues the MMAs of a block into one of 512 / GN accumulator slots, the epilogue warps (warpgroups of
// 32 columns each) read each finished slot, release it and scale.  Every wait is bounded: on a
// timeout the kernel records HQ_ERR_TIMEOUT and winds down.
//
// 4096 x 11008 x 4096, in pairs of CTAs: 200 us, 1.85 PFLOP/s.  The scaling epilogue (each block's sums
// through the FP32 pipe) bounds it; without it the operands' stream from L2 takes 149 us.  333 x 1000 x
// 1460: 6.0 us, twelve blocks one behind the other.
#include <cuda.h>
#include <cuda_runtime.h>

#include "hq_fp8.cuh"
#include "hq_launch.h"
#include "hq_tc.cuh"
#ifdef HQ_TEST_HOOKS
#include "../../include/hq_test.h"
#endif

namespace hq {
namespace {

constexpr int GM = 128, GK = 128;  // CTA tile rows and K block

template <int GN>
struct F8Cfg {
    static constexpr int STAGES = GN == 128 ? 6 : 8;  // operand ring
    static constexpr int ACC = 512 / GN;              // accumulator slots
    static constexpr int EPI = GN / 8;                // epilogue warps: GN / 32 warpgroups of 32 columns
    static constexpr int THREADS = 64 + 32 * EPI;
    static constexpr uint32_t IDESC = idesc_f8(GM, GN);
};

template <int GN>
struct F8Smem {
    using C = F8Cfg<GN>;
    alignas(1024) uint8_t a[C::STAGES][GM * GK];
    alignas(1024) uint8_t b[C::STAGES][GN * GK];
    alignas(8) uint64_t full[C::STAGES];
    uint64_t empty[C::STAGES];
    uint64_t acc_full[C::ACC];
    uint64_t acc_empty[C::ACC];
    uint64_t drain;  // the MMAs
    uint32_t tmem_base;
    uint32_t status;
};

struct F8Args {
    int64_t M, N, K;
    const float* sa;
    const float* sw;
    void* Y;
    int bf16, vec;
    int box_m;  // rows of A's boxes: fewer than the tile's 128 where A has fewer (the rest of the stage is never stored)
    WsHeader* ws;
    // read only by the test build (HQ_TEST_HOOKS): the block of every CTA whose MMAs are withheld, so that the
    // waits behind it run out, and (NULL: no block is) three words a CTA: boxes asked for, boxes awaited, MMAs awaited at the end
    int test_silent;
    uint32_t* test_log;
};

__device__ __forceinline__ bool test_withheld(const F8Args& a, int it)
{
#ifdef HQ_TEST_HOOKS
    return a.test_log && it == a.test_silent;
#else
    return false;
#endif
}
__device__ __forceinline__ void test_boxes(const F8Args& a, int issued, int awaited)
{
#ifdef HQ_TEST_HOOKS
    if (!a.test_log) return;
    a.test_log[3 * blockIdx.x] = issued;
    a.test_log[3 * blockIdx.x + 1] = awaited;
#endif
}
__device__ __forceinline__ void test_drained(const F8Args& a, bool done)
{
#ifdef HQ_TEST_HOOKS
    if (a.test_log) a.test_log[3 * blockIdx.x + 2] = done;
#endif
}

// No copy may be in flight when a block leaves, whatever ended its work: waits for the last boxes of a ring
// of which `issued` were asked for.
template <int STAGES>
__device__ __forceinline__ void await_boxes(const F8Args& a, uint64_t* full, int issued)
{
    int landed = 0;
    for (int it = max(0, issued - STAGES); it < issued; ++it) landed += mbar_wait_sleep(&full[it % STAGES], (uint32_t)((it / STAGES) & 1));
    test_boxes(a, issued, landed);
}

// columns n0 .. n0 + 31 of row m
__device__ __forceinline__ void store_row32(const F8Args& a, int64_t m, int64_t n0, const float2 (&acc)[16])
{
    if (n0 >= a.N) return;
    const int left = (int)(a.N - n0 < 32 ? a.N - n0 : 32);
    if (a.bf16) {
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.Y) + m * a.N + n0;
        if (a.vec && left == 32) {
#pragma unroll
            for (int c = 0; c < 16; c += 4) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __nv_bfloat162 x = __floats2bfloat162_rn(acc[c + j].x, acc[c + j].y);
                    w[j] = *reinterpret_cast<const uint32_t*>(&x);
                }
                *reinterpret_cast<uint4*>(y + 2 * c) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                if (2 * c < left) y[2 * c] = __float2bfloat16_rn(acc[c].x);
                if (2 * c + 1 < left) y[2 * c + 1] = __float2bfloat16_rn(acc[c].y);
            }
        }
    } else {
        float* y = static_cast<float*>(a.Y) + m * a.N + n0;
        if (a.vec && left == 32) {
#pragma unroll
            for (int c = 0; c < 16; c += 2)
                *reinterpret_cast<float4*>(y + 2 * c) = make_float4(acc[c].x, acc[c].y, acc[c + 1].x, acc[c + 1].y);
        } else {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                if (2 * c < left) y[2 * c] = acc[c].x;
                if (2 * c + 1 < left) y[2 * c + 1] = acc[c].y;
            }
        }
    }
}

template <int GN>
__global__ void __launch_bounds__(F8Cfg<GN>::THREADS, 1)
    gemm_fp8_kernel(const F8Args a, const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tB)
{
    using C = F8Cfg<GN>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    F8Smem<GN>& sm = *reinterpret_cast<F8Smem<GN>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int KB = (int)((a.K + GK - 1) / GK);
    const int NT = (int)((a.N + GN - 1) / GN);
    const int64_t tiles = ((a.M + GM - 1) / GM) * NT;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int s = 0; s < C::ACC; ++s) {
            mbar_init(&sm.acc_full[s], 1);
            mbar_init(&sm.acc_empty[s], C::EPI);
        }
        mbar_init(&sm.drain, 1);
        sm.status = 0u;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(&sm.tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = sm.tmem_base;

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            bool alive = true;
            for (int64_t tile = blockIdx.x; alive && tile < tiles; tile += gridDim.x) {
                const int m0 = (int)(tile / NT) * GM, n0 = (int)(tile % NT) * GN;
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const int s = it % C::STAGES;
                    if (it >= C::STAGES && !mbar_wait_sleep(&sm.empty[s], (uint32_t)((it / C::STAGES - 1) & 1))) {
                        atomicOr(&sm.status, kStTimeout);
                        alive = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&sm.full[s], (uint32_t)(a.box_m * GK + GN * GK));
                    tma_load_2d(sm.a[s], &tA, kb * GK, m0, &sm.full[s]);
                    tma_load_2d(sm.b[s], &tB, kb * GK, n0, &sm.full[s]);
                }
            }
            await_boxes<C::STAGES>(a, sm.full, it);
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint64_t ad0 = sw128_desc(sm.a[0]), bd0 = sw128_desc(sm.b[0]);
        const uint32_t tb = __shfl_sync(0xFFFFFFFFu, tbase, 0), leader = elect_lane();
        int it = 0;
        bool alive = true;
        for (int64_t tile = blockIdx.x; alive && tile < tiles; tile += gridDim.x) {
            for (int kb = 0; kb < KB; ++kb, ++it) {
                if (test_withheld(a, it)) {
                    alive = false;
                    break;
                }
                const int s = it % C::STAGES, slot = it % C::ACC;
                const bool got = (it < C::ACC || mbar_wait_sleep(&sm.acc_empty[slot], (uint32_t)((it / C::ACC - 1) & 1))) &&
                                 mbar_wait_sleep(&sm.full[s], (uint32_t)((it / C::STAGES) & 1));
                if (!__all_sync(0xFFFFFFFFu, got)) {
                    if (lane == 0) atomicOr(&sm.status, kStTimeout);
                    alive = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < GK / 32; ++kk)  // K 32 per MMA: the start address moves 32 bytes
                    mma_f8(tb + (uint32_t)(slot * GN), ad0 + (uint64_t)(s * (GM * GK / 16) + 2 * kk),
                           bd0 + (uint64_t)(s * (GN * GK / 16) + 2 * kk), C::IDESC, kk > 0 ? 1u : 0u, leader);
                mma_commit_warp(&sm.empty[s], leader);
                mma_commit_warp(&sm.acc_full[slot], leader);
            }
        }
        // after a timeout the epilogue may not have waited for the last MMAs: none may be under way when the
        // tensor memory is given back
        mma_commit_warp(&sm.drain, leader);
        test_drained(a, mbar_wait_sleep(&sm.drain, 0));
    } else {
        // warpgroup h takes columns 32 h .. 32 h + 31 of each slot; a warp reads the TMEM lane quarter
        // warp % 4, one row of the tile per thread
        const int q = warp & 3, h = (warp - 2) >> 2, row = q * 32 + lane;
        const int64_t NB = (a.N + 127) / 128;
        int it = 0;
        bool alive = true;
        for (int64_t tile = blockIdx.x; alive && tile < tiles; tile += gridDim.x) {
            const int64_t m = (tile / NT) * GM + row, n0 = (tile % NT) * GN + 32 * h;
            const float* sa = a.sa + (m < a.M ? m : 0);
            const float* sw = a.sw + n0 / 128;
            const bool some = n0 < a.N;  // the last tile's warpgroups may lie past N
            float2 acc[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) acc[c] = make_float2(0.0f, 0.0f);
            float f = some ? __ldg(sa) * __ldg(sw) : 0.0f;
            for (int kb = 0; kb < KB; ++kb, ++it) {
                const int slot = it % C::ACC;
                // the next block's scales are on their way while this block's sums are awaited
                const float nsa = some && kb + 1 < KB ? __ldg(sa + (int64_t)(kb + 1) * a.M) : 0.0f;
                const float nsw = some && kb + 1 < KB ? __ldg(sw + (int64_t)(kb + 1) * NB) : 0.0f;
                const bool got = mbar_wait_sleep(&sm.acc_full[slot], (uint32_t)((it / C::ACC) & 1));
                __syncwarp();
                if (!__all_sync(0xFFFFFFFFu, got)) {
                    if (lane == 0) atomicOr(&sm.status, kStTimeout);
                    alive = false;
                    break;
                }
                tc_fence_after();
                uint32_t S[32];
                tmem_ld32_nowait(tbase + ((uint32_t)(q * 32) << 16) + (uint32_t)(slot * GN + 32 * h), S);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.acc_empty[slot]);
                const float2 ff = make_float2(f, f);
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    acc[c] = __ffma2_rn(make_float2(__uint_as_float(S[2 * c]), __uint_as_float(S[2 * c + 1])), ff, acc[c]);
                f = nsa * nsw;
            }
            if (alive && m < a.M) store_row32(a, m, n0, acc);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tbase, 512);
    if (threadIdx.x == 0) slot_write(a.ws, gridDim.x, blockIdx.x, sm.status, 0u);
}

// ------------------------------------------------------------------------------------------------
// The same product on pairs of CTAs, for outputs of many tiles: one MMA makes 256 x 256 of Y, each CTA
// holding 128 rows of A, 128 rows of W and 128 x 256 sums, so an operand byte brought from L2 feeds
// twice the multiplications of the 128 x 128 tile, whose operand stream (32 KB a block and CTA) is
// what bounds it.  Eight epilogue warps of 128 columns each keep their sums in registers.
// ------------------------------------------------------------------------------------------------
constexpr int PN = 256, PSTAGES = 5, PACC = 2, PEPI = 8, PTHREADS = 128 + 32 * PEPI;
// registers a thread: 384 threads start with 168; the first warpgroup (producer, MMA issuer, two idle
// warps) gives 144 each back, which the epilogue warpgroups take 72 each of (sums 128, a TMEM load 32)
constexpr int PREGS_LOW = 24, PREGS_HIGH = 240;

struct PairSmem {
    alignas(1024) uint8_t a[PSTAGES][GM * GK];
    alignas(1024) uint8_t b[PSTAGES][GM * GK];
    alignas(128) uint8_t out[PEPI][32 * 128];  // 128 bytes of each of a warp's rows on their way to Y
    alignas(8) uint64_t full[PSTAGES];
    uint64_t empty[PSTAGES];
    uint64_t acc_full[PACC];
    uint64_t acc_empty[PACC];
    uint64_t drain;  // the MMAs
    uint64_t peer_done;    // even CTA: the odd one has asked for its last box,
    uint32_t peer_issued;  // of so many
    uint32_t tmem_base;
    uint32_t status;
};

// Tiles in bands of PBAND rows of tiles, down each band's columns: the pairs at work share about as many
// rows of A as of W, instead of one row of A and all of W
constexpr int PBAND = 8;
struct PairTile {
    int m, n;
};
__device__ __forceinline__ PairTile pair_tile(int64_t tile, int MT, int NT)
{
    const int band = (int)(tile / ((int64_t)PBAND * NT)), rows = min(PBAND, MT - band * PBAND);
    const int at = (int)(tile - (int64_t)band * PBAND * NT);
    return PairTile{band * PBAND + at % rows, at / rows};
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PTHREADS, 1)
    gemm_fp8_pair_kernel(const F8Args a, const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tB)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    PairSmem& sm = *reinterpret_cast<PairSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int KB = (int)((a.K + GK - 1) / GK);
    const int NT = (int)((a.N + PN - 1) / PN);
    const int MT = (int)((a.M + 2 * GM - 1) / (2 * GM));
    const int64_t tiles = (int64_t)MT * NT;
    const int64_t tile0 = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < PSTAGES; ++s) {
            mbar_init(&sm.full[s], 1);   // even CTA: its own arrival and both CTAs' bytes
            mbar_init(&sm.empty[s], 1);  // the MMAs' commit, in both CTAs
        }
        for (int s = 0; s < PACC; ++s) {
            mbar_init(&sm.acc_full[s], 1);
            mbar_init(&sm.acc_empty[s], 2 * PEPI);  // even CTA: both CTAs' epilogue warps
        }
        mbar_init(&sm.peer_done, 1);
        mbar_init(&sm.drain, 1);
        sm.status = 0u;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc2(&sm.tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tbase = sm.tmem_base;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PREGS_LOW));
        if (warp == 0 && lane == 0) {
            int it = 0;
            bool alive = true;
            for (int64_t tile = tile0; alive && tile < tiles; tile += step) {
                const PairTile at = pair_tile(tile, MT, NT);
                const int m0 = at.m * 2 * GM + (int)rank * GM, n0 = at.n * PN + (int)rank * GM;
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const int s = it % PSTAGES;
                    if (rank == 0 && test_withheld(a, it - PSTAGES + 2)) {  // the test build: two boxes less than the odd CTA
                        alive = false;
                        break;
                    }
                    if (it >= PSTAGES && !mbar_wait_sleep(&sm.empty[s], (uint32_t)((it / PSTAGES - 1) & 1))) {
                        atomicOr(&sm.status, kStTimeout);
                        alive = false;
                        break;
                    }
                    const uint32_t bar = peer_addr(&sm.full[s], 0);
                    if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 4u * GM * GK);
                    tma_load_2d_pair(sm.a[s], &tA, kb * GK, m0, bar);
                    tma_load_2d_pair(sm.b[s], &tB, kb * GK, n0, bar);
                }
            }
            // The odd CTA's boxes complete on the even one's barriers.  Where one of them ran out of time, the
            // other may have asked for more boxes: the even CTA waits for the boxes of both.
            if (rank == 1) {
                st_cluster(peer_addr(&sm.peer_issued, 0), (uint32_t)it);
                mbar_arrive_release(peer_addr(&sm.peer_done, 0));
            } else {
                const int peer = mbar_wait_acquire(&sm.peer_done, 0) ? (int)sm.peer_issued : it;
                for (int j = it; j < peer; ++j) mbar_arrive_expect_tx(&sm.full[j % PSTAGES], 2u * GM * GK);
                await_boxes<PSTAGES>(a, sm.full, max(it, peer));
            }
        } else if (warp == 1 && rank == 0) {
            const uint64_t ad0 = sw128_desc(sm.a[0]), bd0 = sw128_desc(sm.b[0]);
            const uint32_t tb = __shfl_sync(0xFFFFFFFFu, tbase, 0), leader = elect_lane();
            int it = 0;
            bool alive = true;
            for (int64_t tile = tile0; alive && tile < tiles; tile += step) {
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    if (test_withheld(a, it)) {
                        alive = false;
                        break;
                    }
                    const int s = it % PSTAGES, slot = it % PACC;
                    const bool got = (it < PACC || mbar_wait_sleep(&sm.acc_empty[slot], (uint32_t)((it / PACC - 1) & 1))) &&
                                     mbar_wait_sleep(&sm.full[s], (uint32_t)((it / PSTAGES) & 1));
                    if (!__all_sync(0xFFFFFFFFu, got)) {
                        if (lane == 0) atomicOr(&sm.status, kStTimeout);
                        alive = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < GK / 32; ++kk)
                        mma_f8_pair(tb + (uint32_t)(slot * PN), ad0 + (uint64_t)(s * (GM * GK / 16) + 2 * kk),
                                    bd0 + (uint64_t)(s * (GM * GK / 16) + 2 * kk), idesc_f8(2 * GM, PN), kk > 0 ? 1u : 0u, leader);
                    mma_commit_pair(&sm.empty[s], leader);
                    mma_commit_pair(&sm.acc_full[slot], leader);
                }
            }
            mma_commit_pair(&sm.drain, leader, 1);  // as in the kernel above
            test_drained(a, mbar_wait_sleep(&sm.drain, 0));
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PREGS_HIGH));
        // warpgroup h takes columns 128 h .. 128 h + 127 of each slot: one scale of W
        const int q = warp & 3, h = (warp - 4) >> 2, row = q * 32 + lane;
        const int64_t NB = (a.N + 127) / 128;
        int it = 0;
        bool alive = true;
        for (int64_t tile = tile0; alive && tile < tiles; tile += step) {
            const PairTile at = pair_tile(tile, MT, NT);
            const int64_t m = (int64_t)at.m * 2 * GM + rank * GM + row, n0 = (int64_t)at.n * PN + 128 * h;
            const float* sa = a.sa + (m < a.M ? m : 0);
            const float* sw = a.sw + n0 / 128;
            const bool some = n0 < a.N;
            float2 acc[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) acc[c] = make_float2(0.0f, 0.0f);
            float f = some ? __ldg(sa) * __ldg(sw) : 0.0f;
            const uint32_t ta = tbase + ((uint32_t)(q * 32) << 16) + (uint32_t)(128 * h);
            // 32 columns are on their way from TMEM while the 32 before them are scaled, across blocks too
            uint32_t S[2][32];
            auto await_block = [&](int i) {
                const bool got = mbar_wait_sleep(&sm.acc_full[i % PACC], (uint32_t)((i / PACC) & 1));
                __syncwarp();
                if (__all_sync(0xFFFFFFFFu, got)) {
                    tc_fence_after();
                    tmem_ld32_nowait(ta + (uint32_t)((i % PACC) * PN), S[0]);
                    return true;
                }
                if (lane == 0) atomicOr(&sm.status, kStTimeout);
                return false;
            };
            alive = await_block(it);
            for (int kb = 0; alive && kb < KB; ++kb, ++it) {
                const int slot = it % PACC;
                const float nsa = some && kb + 1 < KB ? __ldg(sa + (int64_t)(kb + 1) * a.M) : 0.0f;
                const float nsw = some && kb + 1 < KB ? __ldg(sw + (int64_t)(kb + 1) * NB) : 0.0f;
                const float2 ff = make_float2(f, f);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    tmem_wait_ld();
                    if (p < 3) {
                        tmem_ld32_nowait(ta + (uint32_t)(slot * PN + 32 * (p + 1)), S[(p + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(peer_addr(&sm.acc_empty[slot], 0));
                        if (kb + 1 < KB) alive = await_block(it + 1);
                    }
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        acc[16 * p + c] = __ffma2_rn(
                            make_float2(__uint_as_float(S[p & 1][2 * c]), __uint_as_float(S[p & 1][2 * c + 1])), ff, acc[16 * p + c]);
                }
                f = nsa * nsw;
            }
            if (!alive) continue;
            if (a.vec && n0 + 128 <= a.N) {
                // through shared memory, so that a warp stores 128 contiguous bytes of four rows at a time
                uint8_t* out = sm.out[warp - 4];
                const int es = a.bf16 ? 2 : 4;
                const int64_t r0 = m - lane;
                uint8_t* y = static_cast<uint8_t*>(a.Y) + (r0 * a.N + n0) * es;
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    if (a.bf16 && (p & 1)) continue;
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint4 w;
                        if (a.bf16) {
                            const float2* v = &acc[16 * (p & 2) + 4 * j];
                            const __nv_bfloat162 x0 = __floats2bfloat162_rn(v[0].x, v[0].y), x1 = __floats2bfloat162_rn(v[1].x, v[1].y);
                            const __nv_bfloat162 x2 = __floats2bfloat162_rn(v[2].x, v[2].y), x3 = __floats2bfloat162_rn(v[3].x, v[3].y);
                            w = make_uint4(*reinterpret_cast<const uint32_t*>(&x0), *reinterpret_cast<const uint32_t*>(&x1),
                                           *reinterpret_cast<const uint32_t*>(&x2), *reinterpret_cast<const uint32_t*>(&x3));
                        } else {
                            const float2* v = &acc[16 * p + 2 * j];
                            w = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                                           __float_as_uint(v[1].y));
                        }
                        *reinterpret_cast<uint4*>(out + swz(lane, j)) = w;
                    }
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int r = 4 * k + (lane >> 3);
                        if (r0 + r < a.M)
                            *reinterpret_cast<uint4*>(y + (int64_t)r * a.N * es + 32 * p * es + (lane & 7) * 16) =
                                *reinterpret_cast<const uint4*>(out + swz(r, lane & 7));
                    }
                }
                continue;
            }
            if (m >= a.M) continue;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float2(&part)[16] = *reinterpret_cast<const float2(*)[16]>(&acc[16 * p]);
                store_row32(a, m, n0 + 32 * p, part);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other's MMAs, commits or arrivals may reach it
    tc_fence_after();
    if (warp == 1) tmem_dealloc2(tbase, 512);
    if (threadIdx.x == 0) slot_write(a.ws, gridDim.x, blockIdx.x, sm.status, 0u);
}

cudaError_t launch_gemm_fp8_pair(const F8Args& a, const CUtensorMap& ta, const CUtensorMap& tb, cudaStream_t st)
{
    const size_t smem = sizeof(PairSmem) + 1024;
    cudaError_t e = cudaFuncSetAttribute(gemm_fp8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = ((a.M + 2 * GM - 1) / (2 * GM)) * ((a.N + PN - 1) / PN);
    const int pairs = (int)(tiles < num_sms() / 2 ? tiles : num_sms() / 2);
    gemm_fp8_pair_kernel<<<2 * pairs, PTHREADS, smem, st>>>(a, ta, tb);
    return cudaGetLastError();
}

// ------------------------------------------------------------------------------------------------
// The same product for up to sixteen rows of A and a long K: bound by the bytes of W, which want many loads
// under way on every SM from the first moment.  The weights take the MMA's 128 rows and A's rows its NT
// columns (16; with 32 and 64 the sums sent between CTAs made it slower than the tiles: 12.1 and 18.8 us
// against 10.9 for 4096 x 4096), and a cluster of up to eight CTAs divides the blocks of one 128-row slab of W, so that
// a 4096 x 4096 weight is one ring fill on 128 SMs (8.7 us, the bytes alone 2.6).  Each CTA's scaled sums (binary32) meet over
// distributed shared memory: CTA c of the cluster adds, in the order of the ranks, the columns
// c NT / size .. of all of them and stores those.
// ------------------------------------------------------------------------------------------------
template <int NT>
struct FewCfg {
    static constexpr int STAGES = 8;
    static constexpr int ACC = 256 / NT;  // accumulator slots in 256 TMEM columns
};
constexpr int kFewThreads = 192;  // producer, MMA issue, four epilogue warps
constexpr int kFewChunk = 8;      // blocks whose scales are fetched at a time

template <int NT>
struct FewSmem {
    using C = FewCfg<NT>;
    alignas(1024) uint8_t w[C::STAGES][GM * GK];
    alignas(1024) uint8_t a[C::STAGES][NT * GK];
    alignas(16) float red[NT * GM];      // [source rank][column of this CTA's share][row of W]
    alignas(16) float factor[2][kFewChunk][NT];  // sa sw of the columns, for a chunk of blocks and the next
    alignas(8) uint64_t full[C::STAGES];
    uint64_t empty[C::STAGES];
    uint64_t acc_full[C::ACC];
    uint64_t acc_empty[C::ACC];
    uint64_t drain;  // the MMAs
    uint32_t tmem_base;
    uint32_t status;
};

template <int NT>
__global__ void __launch_bounds__(kFewThreads, 1)
    gemm_fp8_few_kernel(const F8Args a, const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tW, int parts)
{
    using C = FewCfg<NT>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    FewSmem<NT>& sm = *reinterpret_cast<FewSmem<NT>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int KB = (int)((a.K + GK - 1) / GK);
    const int k0 = (int)((int64_t)KB * rank / parts), k1 = (int)((int64_t)KB * (rank + 1) / parts);
    const int n0 = (int)(blockIdx.x / (uint32_t)parts) * GM;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int s = 0; s < C::ACC; ++s) {
            mbar_init(&sm.acc_full[s], 1);
            mbar_init(&sm.acc_empty[s], 4);
        }
        mbar_init(&sm.drain, 1);
        sm.status = 0u;
        fence_mbar_init();
        // the first loads need none of the other warps
        for (int kb = k0; kb < k1 && kb < k0 + C::STAGES; ++kb) {
            const int s = kb - k0;
            mbar_arrive_expect_tx(&sm.full[s], (uint32_t)(GM * GK + NT * GK));
            tma_load_2d(sm.w[s], &tW, kb * GK, n0, &sm.full[s]);
            tma_load_2d(sm.a[s], &tA, kb * GK, 0, &sm.full[s]);
        }
    }
    if (warp == 1) tmem_alloc(&sm.tmem_base, 256);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = sm.tmem_base;

    if (warp == 0) {
        if (lane == 0) {
            int it = min(k1 - k0, C::STAGES);
            for (; it < k1 - k0; ++it) {
                const int s = it % C::STAGES, kb = k0 + it;
                if (!mbar_wait_sleep(&sm.empty[s], (uint32_t)((it / C::STAGES - 1) & 1))) {
                    atomicOr(&sm.status, kStTimeout);
                    break;
                }
                mbar_arrive_expect_tx(&sm.full[s], (uint32_t)(GM * GK + NT * GK));
                tma_load_2d(sm.w[s], &tW, kb * GK, n0, &sm.full[s]);
                tma_load_2d(sm.a[s], &tA, kb * GK, 0, &sm.full[s]);
            }
            await_boxes<C::STAGES>(a, sm.full, it);
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint64_t wd0 = sw128_desc(sm.w[0]), ad0 = sw128_desc(sm.a[0]);
        const uint32_t tb = __shfl_sync(0xFFFFFFFFu, tbase, 0), leader = elect_lane();
        for (int it = 0; it < k1 - k0; ++it) {
            if (test_withheld(a, it)) break;
            const int s = it % C::STAGES, slot = it % C::ACC;
            const bool got = (it < C::ACC || mbar_wait_sleep(&sm.acc_empty[slot], (uint32_t)((it / C::ACC - 1) & 1))) &&
                             mbar_wait_sleep(&sm.full[s], (uint32_t)((it / C::STAGES) & 1));
            if (!__all_sync(0xFFFFFFFFu, got)) {
                if (lane == 0) atomicOr(&sm.status, kStTimeout);
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < GK / 32; ++kk)
                mma_f8(tb + (uint32_t)(slot * NT), wd0 + (uint64_t)(s * (GM * GK / 16) + 2 * kk),
                       ad0 + (uint64_t)(s * (NT * GK / 16) + 2 * kk), idesc_f8(GM, NT), kk > 0 ? 1u : 0u, leader);
            mma_commit_warp(&sm.empty[s], leader);
            mma_commit_warp(&sm.acc_full[slot], leader);
        }
        mma_commit_warp(&sm.drain, leader);  // as in the kernels above
        test_drained(a, mbar_wait_sleep(&sm.drain, 0));
    }
    float2 acc[NT / 2];
    const int q = warp & 3, row = q * 32 + lane;
    if (warp >= 2) {
        // One row of W per thread.  The columns' factors sa sw go through shared memory, a chunk of blocks at
        // a time with the next chunk's under way: a block takes less time than fetching its scales.
        const int64_t NB = (a.N + 127) / 128;
        const float* sw = a.sw + n0 / 128;
#pragma unroll
        for (int c = 0; c < NT / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
        constexpr int PER = kFewChunk * NT / 128;
        float next[PER];
        const int et = (int)threadIdx.x - 64;
        auto fetch = [&](int kb0) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int m = (et + 128 * i) % NT, kb = kb0 + (et + 128 * i) / NT;
                next[i] = m < a.M && kb < k1 ? __ldg(a.sa + (int64_t)kb * a.M + m) * __ldg(sw + (int64_t)kb * NB) : 0.0f;
            }
        };
        fetch(k0);
        bool alive = true;  // after a timeout a warp only walks on, so that all reach the named barrier
        for (int it = 0; it < k1 - k0; ++it) {
            const int slot = it % C::ACC, chunk = it / kFewChunk;
            if (it % kFewChunk == 0) {
#pragma unroll
                for (int i = 0; i < PER; ++i) sm.factor[chunk & 1][0][et + 128 * i] = next[i];
                named_sync(1, 128);
                fetch(k0 + it + kFewChunk);
            }
            if (!alive) continue;
            const float* factor = sm.factor[chunk & 1][it % kFewChunk];
            const bool got = mbar_wait_sleep(&sm.acc_full[slot], (uint32_t)((it / C::ACC) & 1));
            __syncwarp();
            if (!__all_sync(0xFFFFFFFFu, got)) {
                if (lane == 0) atomicOr(&sm.status, kStTimeout);
                alive = false;
                continue;
            }
            tc_fence_after();
            uint32_t S[NT];
            tmem_ld_columns<NT>(tbase + ((uint32_t)(q * 32) << 16) + (uint32_t)(slot * NT), S);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.acc_empty[slot]);
#pragma unroll
            for (int c = 0; c < NT / 4; ++c) {
                const float4 f = *reinterpret_cast<const float4*>(factor + 4 * c);
                acc[2 * c] = __ffma2_rn(make_float2(__uint_as_float(S[4 * c]), __uint_as_float(S[4 * c + 1])), make_float2(f.x, f.y), acc[2 * c]);
                acc[2 * c + 1] = __ffma2_rn(make_float2(__uint_as_float(S[4 * c + 2]), __uint_as_float(S[4 * c + 3])), make_float2(f.z, f.w),
                                            acc[2 * c + 1]);
            }
        }
    }
    // the parts' sums: column c to the CTA that owns it
    const int share = NT / parts;
    if (parts > 1) cluster_sync();  // every CTA of the cluster is up (an arrival at the start and a wait here: slower)
    if (warp >= 2) {
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            const float x = c & 1 ? acc[c / 2].y : acc[c / 2].x;
            const int owner = c / share;
            float* to = &sm.red[(rank * share + c - owner * share) * GM + row];
            if (parts > 1) st_cluster(peer_addr(to, (uint32_t)owner), __float_as_uint(x));
            else *to = x;
        }
    }
    tc_fence_before();
    if (parts > 1) cluster_sync();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tbase, 256);
    if (warp >= 2 && n0 + row < a.N) {
        for (int c = 0; c < share; ++c) {
            const int m = rank * share + c;
            if (m >= a.M) break;
            float x = sm.red[c * GM + row];
            for (int p = 1; p < parts; ++p) x += sm.red[(p * share + c) * GM + row];
            const int64_t at = (int64_t)m * a.N + n0 + row;
            if (a.bf16) static_cast<__nv_bfloat16*>(a.Y)[at] = __float2bfloat16_rn(x);
            else static_cast<float*>(a.Y)[at] = x;
        }
    }
    if (threadIdx.x == 0) slot_write(a.ws, gridDim.x, blockIdx.x, sm.status, 0u);
}

template <int NT>
cudaError_t launch_gemm_fp8_few(const F8Args& a, const CUtensorMap& ta, const CUtensorMap& tw, int parts, cudaStream_t st)
{
    const size_t smem = sizeof(FewSmem<NT>) + 1024;
    cudaError_t e = cudaFuncSetAttribute(gemm_fp8_few_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)((a.N + GM - 1) / GM) * (unsigned)parts);
    c.blockDim = dim3(kFewThreads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)parts;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, gemm_fp8_few_kernel<NT>, a, ta, tw, parts);
}

template <int GN>
cudaError_t launch_gemm_fp8(const F8Args& a, const CUtensorMap& ta, const CUtensorMap& tb, cudaStream_t st)
{
    const size_t smem = sizeof(F8Smem<GN>) + 1024;
    cudaError_t e = cudaFuncSetAttribute(gemm_fp8_kernel<GN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = ((a.M + GM - 1) / GM) * ((a.N + GN - 1) / GN);
    const int grid = (int)(tiles < num_sms() ? tiles : num_sms());
    gemm_fp8_kernel<GN><<<grid, F8Cfg<GN>::THREADS, smem, st>>>(a, ta, tb);
    return cudaGetLastError();
}

hq_status_t gemm_fp8(const uint8_t* A, int64_t lda, const float* sa, int64_t M, const uint8_t* W, int64_t ldw, const float* sw,
                     int64_t N, int64_t K, void* Y, hq_dtype_t ydtype, void* ws, size_t ws_bytes, void* stream, int test_silent,
                     uint32_t* test_log)
{
    if (!A || !sa || !W || !sw || !Y || M < 1 || N < 1 || K < 1 || lda < K || ldw < K || lda % 16 || ldw % 16) return HQ_ERR_ARG;
    if (ydtype != HQ_BF16 && ydtype != HQ_F32) return HQ_ERR_ARG;
    if (M > ((int64_t)1 << 30) || N > ((int64_t)1 << 30) || K > ((int64_t)1 << 20)) return HQ_ERR_UNSUPPORTED;
    const uintptr_t es = ydtype == HQ_BF16 ? 2 : 4, y = reinterpret_cast<uintptr_t>(Y);
    if ((reinterpret_cast<uintptr_t>(A) | reinterpret_cast<uintptr_t>(W)) & 15u) return HQ_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(sa) | reinterpret_cast<uintptr_t>(sw)) & 3u || y % es) return HQ_ERR_ARG;
    if (ws && (ws_bytes < kSlotBytes || (reinterpret_cast<uintptr_t>(ws) & 15u))) return HQ_ERR_ARG;
    DeviceGuard dev(A);
    if (!dev.ok) return HQ_ERR_ARG;
    const int64_t sms = num_sms(), mt = (M + GM - 1) / GM, kbs = (K + GK - 1) / GK, slabs = (N + GM - 1) / GM;
    F8Args a{M, N, K, sa, sw, Y, ydtype == HQ_BF16, ((y | (uintptr_t)N * es) & 15u) == 0, GM,
             static_cast<WsHeader*>(ws), test_silent, test_log};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    CUtensorMap ta, tb;
    // A block of the tiled kernel takes about 0.25 us (a TMA round trip is hidden by the ring, the issue of its
    // MMAs and commits is not) and half as much again at 128 columns; so the width with the fewest rounds of
    // the SMs, weighed by that.  4096 columns and blocks of one row of tiles: 32 columns 11 us, 128: 19.
    auto rounds = [&](int64_t width) { return (mt * ((N + width - 1) / width) + sms - 1) / sms; };
    int gn = 128;
    for (int w = 64; w >= 32; w /= 2)
        if (rounds(w) * (128 + w) < rounds(gn) * (128 + gn)) gn = w;
    // Up to sixteen rows: K in parts over a cluster, whose barriers cost about as much as fourteen blocks (3.5 us).
    // 8 x 4096 x 4096: 8.7 us against 10.5 tiled; 8 x 11008 x 4096: 16.4, 22.8; 8 x 1024 x 4096: 7.1, 10.5; but
    // 8 x 4096 x 2048: 7.4, 6.4; 8 x 1000 x 500: 6.3, 3.5.  Clusters of eight only where they leave half the
    // SMs free (8 x 2048 x 2048 as 128 CTAs in eights: 11.4 us, twice the tiled time).
    int parts = 1;
    while (parts < 8 && slabs * parts * 2 <= (parts == 4 ? sms / 2 : sms) && kbs >= parts * 2) parts *= 2;
    if (M <= 16 && slabs * parts <= kMaxSlots && rounds(32) * kbs > kbs / parts + 14) {
        if (!tensor_map_bytes(&ta, A, M, K, lda, 16) || !tensor_map_bytes(&tb, W, N, K, ldw, GM)) return HQ_ERR_CUDA;
        return launch_gemm_fp8_few<16>(a, ta, tb, parts, st) == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
    }
    // Pairs of CTAs from a quarter of the SMs' number of 256 x 256 tiles on: 48 tiles (768 x 4096 x 4096) 23.7 us
    // against 28.2, 72 tiles 26.8 against 30.3, but 32 tiles (1024 x 2048 x 4096) 22.9 against 16.7.
    const bool pair = ((M + 2 * GM - 1) / (2 * GM)) * ((N + PN - 1) / PN) >= sms / 4;
    // K blocks over all tiles of a CTA are counted in 31 bits
    if ((mt * ((N + gn - 1) / gn) / sms + 1) * ((K + GK - 1) / GK) > ((int64_t)1 << 30)) return HQ_ERR_UNSUPPORTED;
    if (!pair && M < GM) a.box_m = (int)((M + 7) / 8 * 8);
    if (!tensor_map_bytes(&ta, A, M, K, lda, a.box_m) || !tensor_map_bytes(&tb, W, N, K, ldw, pair ? GM : gn)) return HQ_ERR_CUDA;
    const cudaError_t e = pair        ? launch_gemm_fp8_pair(a, ta, tb, st)
                          : gn == 128 ? launch_gemm_fp8<128>(a, ta, tb, st)
                                    : (gn == 64 ? launch_gemm_fp8<64>(a, ta, tb, st) : launch_gemm_fp8<32>(a, ta, tb, st));
    return e == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

}  // namespace
}  // namespace hq

using namespace hq;

extern "C" hq_status_t hq_gemm_fp8(const uint8_t* A, int64_t lda, const float* sa, int64_t M, const uint8_t* W, int64_t ldw,
                                   const float* sw, int64_t N, int64_t K, void* Y, hq_dtype_t ydtype, void* ws,
                                   size_t ws_bytes, void* stream)
{
    return gemm_fp8(A, lda, sa, M, W, ldw, sw, N, K, Y, ydtype, ws, ws_bytes, stream, -1, nullptr);
}

#ifdef HQ_TEST_HOOKS
// only in the test library (libhq_test.so): the product library does not export it
extern "C" hq_status_t hq_test_gemm_fp8_silent_block(const uint8_t* A, int64_t lda, const float* sa, int64_t M, const uint8_t* W,
                                                     int64_t ldw, const float* sw, int64_t N, int64_t K, void* Y, hq_dtype_t ydtype,
                                                     void* ws, size_t ws_bytes, int32_t silent_block, uint32_t* log, void* stream)
{
    if (silent_block < 0 || !log) return HQ_ERR_ARG;
    return gemm_fp8(A, lda, sa, M, W, ldw, sw, N, K, Y, ydtype, ws, ws_bytes, stream, silent_block, log);
}
#endif
