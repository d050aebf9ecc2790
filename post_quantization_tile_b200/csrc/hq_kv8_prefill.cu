// hq_kv8_prefill.cu -- attention of many query rows over the e4m3 KV cache (prompt chunks, long
// speculative runs): both products on tcgen05 with TMEM accumulators.
//
// A unit is 256 rows of one (sequence, key head), two tiles of 128, against tiles of 128 slots.  Per step
// of 64 slots and row tile: S = Q K^T (MMAs M 128, N 64, K 16) into one of two TMEM buffers, softmax by
// 128 threads with one row each, P as binary16 back into the same buffer, O += P V (P from TMEM).  The
// scores of a step are there two steps ahead, so the softmax warps need not wait for the tensor cores;
// keys and values are read from the cache and converted to binary16 in shared memory once for both
// row tiles.
//
// Warps: 0-3 and 4-7 softmax of the two row tiles, 8-11 conversion, 12 MMA issue.
//
// 2 x 512 queries x 32 heads over 8192 slots: 183 us, 0.75 PFLOP/s, tensor pipe 39% and issue slots 41%
// busy.  In this arrangement, one warpgroup for both score buffers of a row tile, the chain of a step takes the
// time (scores out of TMEM, maximum, exponentials, P back, P V): with half of the score MMAs, without the conversion
// or without the exponentials it stayed within 6%.
//
// Numerics as in the kernel for few rows (hq_kv8_attend.cu).  One accumulator serves pages of unlike scales, so
// value codes enter binary16 times 2^-15 .. 2^7, their page's scale (up to the next power of two) over the
// accumulator's unit: exact, since the last bit of e4m3 is 2^-9, of binary16 2^-24.  A segment whose pages' value
// scales span more than these 22 octaves is walked once for each window of 22, the quietest first, with the
// values outside the window as zeros and the accumulator brought to the next window's unit in between; four
// windows hold 2^-40 .. 2^40.  What a scale lacks to a power of two multiplies the probabilities of its slots.
#include <cuda.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "hq_kv8_attend.cuh"
#include "hq_tc.cuh"

namespace hq {
namespace {

constexpr int kThreadsP = 512;
constexpr int kTok = 128;     // slots of a tile
constexpr int kStep = 64;     // slots of one step of the softmax: a row tile has two buffers of scores
constexpr int kScaleRing = 4;  // tiles whose key scales are kept: the converter is at most two ahead
constexpr int kWindows = 4;    // value scales: windows of a segment at most
constexpr float kWindow = 4194304.0f, kWindowTop = 128.0f;  // their width, and their largest scale over the unit

// the power of two at or above a positive scale, and the reciprocal of a power of two
__device__ __forceinline__ float pow2_above(float x) { return __uint_as_float((__float_as_uint(x) + 0x7FFFFFu) & 0x7F800000u); }
__device__ __forceinline__ float pow2_inverse(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }

// units of 256 rows; a unit's tiles end with the last slot that any of its rows sees
struct ManyRows {
    static constexpr int R = kManyRows, TILE = kTok;
    static __device__ __forceinline__ int row_tiles(const AttendArgs& a, int m) { return (m * a.G + R - 1) / R; }
    static __device__ __forceinline__ int end(const AttendArgs& a, const SeqLen& s, int rt)
    {
        return sees(a, s.n, s.m, min(rt * R + R - 1, s.m * a.G - 1) / a.G);
    }
    static __device__ __forceinline__ uint32_t tiles(const AttendArgs& a, const SeqLen& s, int rt)
    {
        return (uint32_t)((end(a, s, rt) + TILE - 1) / TILE);
    }
    static __device__ __forceinline__ uint32_t up_to(const AttendArgs& a, const SeqLen& s, int rts)
    {
        if (!a.causal) return (uint32_t)rts * (uint32_t)((s.n + TILE - 1) / TILE);
        uint32_t n = 0;
        for (int rt = 0; rt < rts; ++rt) n += tiles(a, s, rt);
        return n;
    }
    static __device__ __forceinline__ uint32_t of_sequence(const AttendArgs& a, const SeqLen& s)
    {
        return (uint32_t)a.c.heads * up_to(a, s, row_tiles(a, s.m));
    }
    static __device__ __forceinline__ uint32_t before(const AttendArgs& a, const SeqLen& s, int h, int rt)
    {
        return (uint32_t)h * up_to(a, s, row_tiles(a, s.m)) + up_to(a, s, rt);
    }
    static __device__ __forceinline__ void find(const AttendArgs& a, const SeqLen& s, uint32_t of_head, uint32_t at, Segment& g)
    {
        g.h = at / of_head;
        at -= g.h * of_head;
        for (g.rt = 0; at >= (g.tiles = tiles(a, s, g.rt)); ++g.rt) at -= g.tiles;
        g.t0 = at;
    }
};

template <int D>
struct PrefillSmem {
    static constexpr int HALF = 128 * 128;  // bytes of 64 dims of 128 rows: one run of swizzled 128-byte rows
    alignas(1024) unsigned char q[2][D / 64][HALF];
    alignas(1024) unsigned char k[2][D / 64][HALF];
    alignas(1024) unsigned char v[2][D / 64][HALF];
    alignas(16) float ks[kScaleRing][8];  // key scale of each sixteen slots; negative: no such page
    alignas(16) float vm[kScaleRing][8];  // their value scale over the power of two above it
    int2 seg[4];                          // by segment: windows, whether a value scale is no power of two
    float vref[4];                        // by window: the accumulator's unit
    float cut[kWindows + 1], top[kWindows];  // the converter's: a segment's windows (cut[i], cut[i + 1]], their largest scales
    alignas(16) uint32_t red[4][4];
    float sum[256];                       // by row: the first window's
    alignas(8) uint64_t k_full[2];
    uint64_t k_empty[2], v_full[2], v_empty[2];
    uint64_t s_full[2][2], p_ready[2][2];  // by row tile and score buffer
    uint64_t pv_done[2], o_full[2];        // by row tile
    uint64_t q_ready[2], drain;
    uint32_t tmem_base;
    uint32_t status;
    uint64_t scan[kThreadsP / 32];
};

// sixteen codes of a row (16-byte chunk c of 64) as binary16, times r2, into a swizzled operand run.  The
// lanes of a store are eight rows by four chunks, which meet in no bank.
template <bool SCALE>
__device__ __forceinline__ void put_codes(unsigned char* run, int row, int c, uint4 x, uint32_t r2)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[2 * i] = e4m3x2_to_f16x2(w[i] & 0xFFFFu);
        h[2 * i + 1] = e4m3x2_to_f16x2(w[i] >> 16);
    }
    if (SCALE)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&h[i]), *reinterpret_cast<const __half2*>(&r2));
            h[i] = *reinterpret_cast<const uint32_t*>(&y);
        }
    *reinterpret_cast<uint4*>(run + swz(row, 2 * c)) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(run + swz(row, 2 * c + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
}

// this thread's row of an accumulator times f
template <int D>
__device__ __forceinline__ void scale_row(uint32_t to, float f)
{
#pragma unroll 1
    for (int p = 0; p < D / 32; ++p) {
        uint32_t o[32];
        tmem_ld32_nowait(to + 32 * p, o);
        tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
        tmem_st32(to + 32 * p, o);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreadsP, 1) kv8_prefill_kernel(const AttendArgs a)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    using Smem = PrefillSmem<D>;
    Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint32_t* pre = reinterpret_cast<uint32_t*>(&sm + 1);
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.k_full[i], 4);
            mbar_init(&sm.k_empty[i], 1);
            mbar_init(&sm.v_full[i], 4);
            mbar_init(&sm.v_empty[i], 1);
            for (int j = 0; j < 2; ++j) {
                mbar_init(&sm.s_full[i][j], 1);
                mbar_init(&sm.p_ready[i][j], 4);
            }
            mbar_init(&sm.pv_done[i], 1);
            mbar_init(&sm.o_full[i], 1);
            mbar_init(&sm.q_ready[i], 4);
        }
        mbar_init(&sm.drain, 1);
        sm.status = 0u;
        fence_mbar_init();
    }
    if (warp == 12) tmem_alloc(&sm.tmem_base, 512);
    tc_fence_before();
    const bool odd_len = share_prefix<ManyRows, kThreadsP>(a, pre, sm.scan);  // two block barriers
    tc_fence_after();
    if (odd_len && blockIdx.x == 0) atomicOr(&sm.status, kStRange);
    after_me();
    const uint32_t tbase = sm.tmem_base;
    const uint32_t W = pre[a.B];
    const uint32_t shares = pre[a.B + 1];
    uint32_t w0 = blockIdx.x < shares ? (uint32_t)((uint64_t)blockIdx.x * W / shares) : 0u;
    const uint32_t w1 = blockIdx.x < shares ? (uint32_t)((uint64_t)(blockIdx.x + 1) * W / shares) : 0u;
    // After a wait that ran out a warp only walks its loops, without waiting or working.
    bool alive = true;
    auto wait = [&](uint64_t* bar, uint32_t n) {
        if (alive && !__all_sync(0xFFFFFFFFu, mbar_wait_sleep(bar, n & 1))) {
            alive = false;
            if (lane == 0) atomicOr(&sm.status, kStTimeout);
        }
    };

    if (warp < 8) {
        // ---------------- softmax: row tile t, one row per thread ----------------
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lanes = tbase + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = lanes + 128 * t, to = lanes + 256 + 128 * t;
        // segments, windows and slot tiles, and those and the steps of this row tile
        uint32_t seg_n = 0, win_n = 0, tile_n = 0, s_n = 0, pv_n = 0;
        while (w0 < w1) {
            const Segment g = segment_at<ManyRows>(a, pre, w0, w1);
            const int row = g.rt * kManyRows + t * 128 + r, i = row / a.G;
            const bool is = i < g.s.m, active = g.rt * kManyRows + t * 128 < g.s.m * a.G;
            const int end = is ? sees(a, g.s.n, g.s.m, i) : 0x7FFFFFFF;
            float c = 1.0f;
            if (active) {
                uint4 x[D / 8];
                uint32_t top = 0;
                const __nv_bfloat16* q = a.q + g.b * a.qb + (int64_t)(g.h * a.G + (is ? row - i * a.G : 0)) * a.qh + (int64_t)(is ? i : 0) * a.qs;
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    x[j] = is ? __ldg(reinterpret_cast<const uint4*>(q) + j) : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) top = max(top, max((w[y] << 16) & 0x7FFF0000u, w[y] & 0x7FFF0000u));
                }
                // a power of two brings the row's largest to [2^14, 2^15); a negative scale goes into the
                // queries, so that the factors of the scores are not negative
                const int e = top ? min(126, 14 + 127 - (int)(top >> 23)) : 0;
                const float up = a.scale < 0.0f ? -exp2_int(e) : exp2_int(e);
                c = exp2_int(-e) * fabsf(a.scale) * kLog2e;
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                    uint32_t h[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) h[y] = pack_f16(bf16lo_to_f32(w[y]) * up, bf16hi_to_f32(w[y]) * up);
                    *reinterpret_cast<uint4*>(&sm.q[t][j >> 3][swz(r, j & 7)]) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.q_ready[t]);
            const int full_end = (int)__reduce_min_sync(0xFFFFFFFFu, (uint32_t)end);
            float m = -INFINITY, l = 0.0f, vref = 1.0f;
            const int T = (int)(g.t1 - g.t0);
            int windows = 1;
            if (active) {
#pragma unroll 1
                for (int win = 0; win < windows; ++win) {
                    bool odd = false;
                    wait(&sm.s_full[t][0], s_n);  // the window's first scores, and with them what the converter says of it
                    if (alive) {
                        const int2 of_seg = sm.seg[seg_n & 3];
                        const float unit = sm.vref[win_n & 3];
                        windows = of_seg.x;
                        odd = of_seg.y != 0;
                        if (win > 0) {
                            wait(&sm.pv_done[t], pv_n - 1);
                            tc_fence_after();
                            if (alive) scale_row<D>(to, vref / unit);
                        }
                        vref = unit;
                    }
                    ++win_n;
                    auto steps = [&](auto with_factors) {
                        constexpr bool ODD = decltype(with_factors)::value;
#pragma unroll 1
                        for (int i2 = 0; i2 < 2 * T; ++i2) {
                            const int tok = (int)g.t0 * kTok + i2 * kStep, buf = i2 & 1;
                            const uint32_t tb = ts + kStep * buf;
                            wait(&sm.s_full[t][buf], s_n + (i2 >> 1));
                            if (!alive) continue;
                            tc_fence_after();
                            uint32_t S[2][32];
                            tmem_ld32_nowait(tb, S[0]);
                            tmem_ld32_nowait(tb + 32, S[1]);
                            const float4 ks = *reinterpret_cast<const float4*>(&sm.ks[(tile_n + (i2 >> 1)) % kScaleRing][4 * buf]);
                            tmem_wait_ld();
                            if (tok + kStep > full_end || fminf(fminf(ks.x, ks.y), fminf(ks.z, ks.w)) < 0.0f) {
                                // slots that some row does not see, or whose page is missing
                                const int left = end - tok;
#pragma unroll
                                for (int y = 0; y < kStep; ++y)
                                    if (y >= left || (y < 16 ? ks.x : (y < 32 ? ks.y : (y < 48 ? ks.z : ks.w))) < 0.0f) S[y >> 5][y & 31] = 0xFF800000u;
                            }
                            // the scores' factors, positive: a masked score times zero would be NaN (products of codes
                            // and queries stay below 2^31, so that scores times 1e-30 are zeros all the same)
                            const float cg[4] = {fmaxf(c * fabsf(ks.x), 1e-30f), fmaxf(c * fabsf(ks.y), 1e-30f),
                                                 fmaxf(c * fabsf(ks.z), 1e-30f), fmaxf(c * fabsf(ks.w), 1e-30f)};
                            float x[8];
#pragma unroll
                            for (int z = 0; z < 8; ++z) x[z] = __uint_as_float(S[z >> 2][(z & 3) * 8]);
#pragma unroll
                            for (int y = 1; y < 8; ++y)
#pragma unroll
                                for (int z = 0; z < 8; ++z) x[z] = fmaxf(x[z], __uint_as_float(S[z >> 2][(z & 3) * 8 + y]));
                            const float top = fmaxf(fmaxf(fmaxf(x[0], x[1]) * cg[0], fmaxf(x[2], x[3]) * cg[1]),
                                                    fmaxf(fmaxf(x[4], x[5]) * cg[2], fmaxf(x[6], x[7]) * cg[3]));
                            const bool moves = top > m + kSlack;
                            if (__any_sync(0xFFFFFFFFu, moves)) {  // in the first window only: the others see the same scores
                                const float next = moves ? top : m, f = m == -INFINITY ? 1.0f : ex2(m - next);
                                l *= f;
                                m = next;
                                if (i2 > 0) {  // once the products before this step's are done
                                    wait(&sm.pv_done[t], pv_n + i2 - 1);
                                    if (!alive) continue;
                                    tc_fence_after();
                                    scale_row<D>(to, f);
                                }
                            }
                            const float sub = m == -INFINITY ? 0.0f : m - kBoost;
                            const float2 nsub = make_float2(-sub, -sub);
                            float2 sum = make_float2(0.0f, 0.0f);
                            const float4 vm = ODD ? *reinterpret_cast<const float4*>(&sm.vm[(tile_n + (i2 >> 1)) % kScaleRing][4 * buf])
                                                  : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                            const float vg[4] = {vm.x, vm.y, vm.z, vm.w};
#pragma unroll
                            for (int p = 0; p < 2; ++p) {
                                uint32_t P[16];
#pragma unroll
                                for (int y = 0; y < 16; ++y) {
                                    const float cq = cg[2 * p + (y >> 3)];
                                    float2 e = __ffma2_rn(make_float2(__uint_as_float(S[p][2 * y]), __uint_as_float(S[p][2 * y + 1])),
                                                          make_float2(cq, cq), nsub);
                                    e = make_float2(ex2(e.x), ex2(e.y));
                                    sum = f2add(sum, e);
                                    if (ODD) e = f2mul(e, make_float2(vg[2 * p + (y >> 3)], vg[2 * p + (y >> 3)]));
                                    P[y] = pack_f16(e.x, e.y);
                                }
                                tmem_st16(tb + 16 * p, P);
                            }
                            l += sum.x + sum.y;
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sm.p_ready[t][buf]);
                        }
                    };
                    if (odd) steps(std::true_type{});
                    else steps(std::false_type{});
                    if (win == 0 && windows > 1) sm.sum[tid] = l;
                    s_n += T;
                    pv_n += 2 * T;
                    tile_n += T;
                }
                if (windows > 1) l = sm.sum[tid];  // once for all windows
                // the segment's accumulator
                wait(&sm.o_full[t], seg_n);
                if (alive) {
                    tc_fence_after();
                    const bool whole = g.t0 == 0 && g.t1 == g.tiles;
                    const int slot = 2 * blockIdx.x + (g.t0 == 0 ? 1 : 0);
                    const float f = whole ? (l == 0.0f ? 0.0f : vref / l) : vref;
                    int head, iq;
                    row_place(a, g.h, row, head, iq);
                    __nv_bfloat16* out = a.out + g.b * a.ob + head * a.oh + (int64_t)iq * a.os;
                    float* part = a.part_o + ((int64_t)slot * kManyRows + t * 128 + r) * D;
                    if (is) {
                        if (whole) write_lse(a, g.b, g.h, row, m, l);
                        else a.part_ml[slot * kManyRows + t * 128 + r] = make_float2(m, l);
                    }
#pragma unroll
                    for (int p = 0; p < D / 32; ++p) {
                        uint32_t o[32];
                        tmem_ld32_nowait(to + 32 * p, o);
                        tmem_wait_ld();
                        if (!is) continue;
                        if (whole) {
#pragma unroll
                            for (int y = 0; y < 32; y += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int z = 0; z < 4; ++z) {
                                    const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(o[y + 2 * z]) * f, __uint_as_float(o[y + 2 * z + 1]) * f);
                                    w[z] = *reinterpret_cast<const uint32_t*>(&x);
                                }
                                *reinterpret_cast<uint4*>(out + 32 * p + y) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        } else {
#pragma unroll
                            for (int y = 0; y < 32; y += 4)
                                *reinterpret_cast<float4*>(part + 32 * p + y) =
                                    make_float4(__uint_as_float(o[y]) * f, __uint_as_float(o[y + 1]) * f, __uint_as_float(o[y + 2]) * f,
                                                __uint_as_float(o[y + 3]) * f);
                        }
                    }
                    tc_fence_before();
                }
            } else {
                wait(&sm.o_full[t], seg_n);  // without rows: keep step with the others, one segment at a time
                if (alive) windows = sm.seg[seg_n & 3].x;
                win_n += windows;
                tile_n += T * windows;
            }
            ++seg_n;
            w0 += T;
        }
    } else if (warp < 12) {
        // ---------------- conversion: codes from the cache to binary16 operand tiles ----------------
        // a pass: 32 rows by 64 dims; a warp's eight rows lie in one group of sixteen slots
        constexpr int RUNS = D / 64, PASSES = 4 * RUNS;
        const int ct = tid - 256, c = ct & 3, row0 = ct >> 2, half = ct >> 6;
        uint32_t seg_n = 0, win_n = 0, tile_n = 0;
        while (w0 < w1) {
            const Segment g = segment_at<ManyRows>(a, pre, w0, w1);
            const int32_t* table = a.table + g.b * a.table_stride;
            const int end = min((int)g.t1 * kTok, ManyRows::end(a, g.s, g.rt)), T = (int)(g.t1 - g.t0);
            // of the value scales of the segment's pages: the largest up to `cut`, the smallest above it, the
            // largest of all, and whether one is no power of two (positive floats order like their bit patterns)
            auto scales = [&](float cut, float& under, float& above, float& top) {
                uint32_t u = 0u, o = 0x7F800000u, m = 0u, odd = 0u;
                for (int tok = ((int)g.t0 * kTok / a.c.page + ct) * a.c.page; tok < end; tok += 128 * a.c.page) {
                    const int32_t id = __ldg(table + (tok >> a.page_shift));
                    if (id >= 0 && id < a.c.pages) {
                        const float vs = __ldg(a.c.v_scale + (int64_t)id * a.c.heads + g.h);
                        const uint32_t w = __float_as_uint(vs);
                        if (!(vs > 0.0f)) continue;
                        if (vs > cut) o = min(o, w);
                        else u = max(u, w);
                        m = max(m, w);
                        odd |= w & 0x7FFFFFu;
                    } else {
                        atomicOr(&sm.status, kStRange);
                    }
                }
                u = __reduce_max_sync(0xFFFFFFFFu, u);
                o = __reduce_min_sync(0xFFFFFFFFu, o);
                m = __reduce_max_sync(0xFFFFFFFFu, m);
                odd = __reduce_or_sync(0xFFFFFFFFu, odd);
                named_sync(1, 128);  // what the last call left is read
                if (lane == 0) *reinterpret_cast<uint4*>(sm.red[warp - 8]) = make_uint4(u, o, m, odd);
                named_sync(1, 128);
                for (int w = 0; w < 4; ++w) {
                    u = max(u, sm.red[w][0]);
                    o = min(o, sm.red[w][1]);
                    m = max(m, sm.red[w][2]);
                    odd |= sm.red[w][3];
                }
                under = __uint_as_float(u);
                above = __uint_as_float(o);
                top = __uint_as_float(m);
                return odd != 0u;
            };
            float under, low, vmax, cut_lo = 0.0f, cut_hi = INFINITY;
            const bool odd = scales(0.0f, under, low, vmax);
            int windows = 1;
            if (vmax > low * kWindow) {
                float from = 0.0f;
                for (windows = 0; windows < kWindows; ++windows) {
                    const bool last = windows == kWindows - 1 || vmax <= low * kWindow;
                    const float to = last ? INFINITY : low * kWindow;
                    if (!last) scales(to, under, low, vmax);
                    if (ct == 0) sm.cut[windows] = from, sm.cut[windows + 1] = to, sm.top[windows] = last ? vmax : under;
                    from = to;
                    if (last) break;
                }
                ++windows;
                named_sync(1, 128);
            }
            // the groups of sixteen slots of a tile: lane y < 8 knows the page (two tiles ahead of the codes),
            // the first cache row and the scales (one ahead) of group y; the keys of the next tile and the
            // values of this one are on their way while the tile before is stored
            const int gy = lane & 7, stop = T * kTok;
            int g_id = -1, g_row = -1;
            float2 g_scale = make_float2(-1.0f, 0.0f);
            const int tok0 = (int)g.t0 * kTok;
            auto find_pages = [&](int j) {
                const int at = j * kTok + 16 * gy;
                g_id = at < stop && tok0 + at < end ? __ldg(table + ((tok0 + at) >> a.page_shift)) : -2;
            };
            auto find_rows = [&](int j) {
                const bool ok = g_id >= 0 && g_id < a.c.pages;
                const int ph = ok ? g_id * a.c.heads + g.h : 0;
                g_row = ok ? (ph << a.page_shift) + ((tok0 + j * kTok + 16 * gy) & (a.c.page - 1)) : -1;
                // -2, behind the segment's last slot: hidden by the rows' ends, any positive key scale will do
                g_scale = ok ? make_float2(__ldg(a.c.k_scale + ph), __ldg(a.c.v_scale + ph)) : make_float2(g_id == -2 ? 1.0f : -1.0f, 0.0f);
            };
            // rows of a missing group come from the pool's first page; the values are cleared below
            auto fetch = [&](uint4 (&x)[PASSES], const uint8_t* codes) {
#pragma unroll
                for (int p = 0; p < PASSES; ++p) {
                    const int row = __shfl_sync(0xFFFFFFFFu, g_row, 2 * (p / RUNS) + half);
                    x[p] = __ldg(reinterpret_cast<const uint4*>(codes + (int64_t)(max(row, 0) + (row0 & 15)) * D + (p % RUNS) * 64) + c);
                }
            };
            uint4 xk[PASSES], xv[PASSES];
#pragma unroll 1
            for (int win = 0; win < windows; ++win, ++win_n) {
                if (windows > 1) cut_lo = sm.cut[win], cut_hi = sm.cut[win + 1], vmax = sm.top[win];
                const float vref = vmax > 0.0f ? pow2_above(vmax) * (1.0f / kWindowTop) : 1.0f, inv = pow2_inverse(vref);
                find_pages(0);
                find_rows(0);
                find_pages(1);
                fetch(xk, a.c.k);
#pragma unroll 1
                for (int j = 0; j < T; ++j, ++tile_n) {
                    const int st = tile_n & 1;
                    fetch(xv, a.c.v);
                    const float ks = g_scale.x, v2 = pow2_above(g_scale.y), vm = g_scale.y * pow2_inverse(v2);
                    const float vr = g_scale.y > cut_lo && g_scale.y <= cut_hi ? v2 * inv : 0.0f;
                    const uint32_t vr2 = pack_f16(vr, vr);
                    // values that nobody may see are zeros: behind the last slot, and of missing pages
                    const uint32_t gone = __ballot_sync(0xFFFFFFFFu, g_row < 0) & 0xFFu;
                    const bool edge = gone != 0u || tok0 + (j + 1) * kTok > end;
                    find_rows(j + 1);
                    find_pages(j + 2);
                    if (tile_n >= 2) wait(&sm.k_empty[st], tile_n / 2 - 1);
                    if (ct < 8) sm.ks[tile_n % kScaleRing][ct] = ks, sm.vm[tile_n % kScaleRing][ct] = vm;
                    if (ct == 0 && j == 0) sm.seg[seg_n & 3] = make_int2(windows, odd), sm.vref[win_n & 3] = vref;
#pragma unroll
                    for (int p = 0; p < PASSES; ++p) put_codes<false>(sm.k[st][p % RUNS], (p / RUNS) * 32 + row0, c, xk[p], 0u);
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.k_full[st]);
                    fetch(xk, a.c.k);
                    if (tile_n >= 2) wait(&sm.v_empty[st], tile_n / 2 - 1);
                    if (edge)
#pragma unroll
                        for (int p = 0; p < PASSES; ++p) {
                            const int r = (p / RUNS) * 32 + row0;
                            if ((gone >> (r >> 4) & 1u) || tok0 + j * kTok + r >= end) xv[p] = make_uint4(0u, 0u, 0u, 0u);
                        }
#pragma unroll
                    for (int p = 0; p < PASSES; ++p)
                        put_codes<true>(sm.v[st][p % RUNS], (p / RUNS) * 32 + row0, c, xv[p],
                                        __shfl_sync(0xFFFFFFFFu, vr2, 2 * (p / RUNS) + half));
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.v_full[st]);
                }
            }
            ++seg_n;
            w0 += T;
        }
    } else {
        if (warp == 12) {
            // ---------------- MMA issue ----------------
            constexpr uint32_t IDS = idesc_f16(128, kStep, false), IDO = idesc_f16(128, D, true);
            uint32_t seg_n = 0, tile_n = 0, s_n[2] = {0, 0};
            // operand tiles follow one another: descriptors differ by their distance in 16-byte units
            constexpr uint64_t RUN = Smem::HALF >> 4, TILE = (D / 64) * RUN;
            const uint64_t dq = sw128_desc(sm.q[0][0]), dk = sw128_desc(sm.k[0][0]), dv = sw128_desc_mn(sm.v[0][0], Smem::HALF);
            const uint32_t tb = __shfl_sync(0xFFFFFFFFu, tbase, 0), leader = elect_lane();
            // step i of the segment, half `i & 1` of slot tile `st`, into score buffer i & 1
            constexpr uint64_t HALFTILE = (kStep * 128) >> 4;
            auto score = [&](int t, int st, int buf) {
                const uint64_t ad = dq + (t ? TILE : 0), bd = dk + (st ? TILE : 0) + (buf ? HALFTILE : 0);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_f16_ss(tb + 128 * t + kStep * buf, ad + (kk >> 2) * RUN + 2 * (kk & 3), bd + (kk >> 2) * RUN + 2 * (kk & 3), IDS, kk > 0, leader);
                mma_commit_warp(&sm.s_full[t][buf], leader);
            };
            while (w0 < w1) {
                const Segment g = segment_at<ManyRows>(a, pre, w0, w1);
                const int T = __shfl_sync(0xFFFFFFFFu, (int)(g.t1 - g.t0), 0);
                const int nt = __shfl_sync(0xFFFFFFFFu, g.rt * kManyRows + 128 < g.s.m * a.G ? 2 : 1, 0);  // row tiles with rows
                wait(&sm.q_ready[0], seg_n);
                wait(&sm.q_ready[1], seg_n);
                wait(&sm.k_full[tile_n & 1], tile_n / 2);
                tc_fence_after();
                const int tiles = T * (alive ? __shfl_sync(0xFFFFFFFFu, sm.seg[seg_n & 3].x, 0) : 1);  // of all windows
                if (alive) {
#pragma unroll
                    for (int buf = 0; buf < 2; ++buf)
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            if (t < nt) score(t, tile_n & 1, buf);
                    mma_commit_warp(&sm.k_empty[tile_n & 1], leader);
                }
#pragma unroll 1
                for (int j = 0; j < tiles; ++j, ++tile_n) {
                    const int st = tile_n & 1, next = st ^ 1;
                    wait(&sm.v_full[st], tile_n / 2);
                    if (j + 1 < tiles) wait(&sm.k_full[next], (tile_n + 1) / 2);
#pragma unroll
                    for (int buf = 0; buf < 2; ++buf)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (t >= nt) continue;
                            wait(&sm.p_ready[t][buf], s_n[t]);
                            tc_fence_after();
                            if (!alive) continue;
#pragma unroll
                            for (int kk = 0; kk < kStep / 16; ++kk)
                                mma_f16_ts(tb + 256 + 128 * t, tb + 128 * t + kStep * buf + 8 * kk,
                                           dv + (st ? TILE : 0) + (buf ? HALFTILE : 0) + (uint64_t)(128 * kk), IDO, j > 0 || buf > 0 || kk > 0, leader);
                            mma_commit_warp(&sm.pv_done[t], leader);
                            if (buf && t == nt - 1) mma_commit_warp(&sm.v_empty[st], leader);
                            if (j + 1 < tiles) {  // the scores of two steps on take this step's buffer
                                score(t, next, buf);
                                if (buf && t == nt - 1) mma_commit_warp(&sm.k_empty[next], leader);
                            } else if (buf) {
                                mma_commit_warp(&sm.o_full[t], leader);
                                if (nt == 1) mma_commit_warp(&sm.o_full[1], leader);
                            }
                        }
                    ++s_n[0];
                    if (nt == 2) ++s_n[1];
                }
                ++seg_n;
                w0 += T;
            }
            // nothing may be under way when the tensor memory is given back
            mma_commit_warp(&sm.drain, leader);
            mbar_wait_sleep(&sm.drain, 0);
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(tbase, 512);
    if (tid == 0) slot_write(a.ws, gridDim.x, blockIdx.x, sm.status, 0u);
}

template <int D>
cudaError_t launch_many(const AttendArgs& a, int grid, cudaStream_t st)
{
    const size_t smem = 1024 + sizeof(PrefillSmem<D>) + share_bytes(a.B);
    cudaError_t e = cudaFuncSetAttribute(kv8_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kv8_prefill_kernel<D><<<grid, kThreadsP, smem, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int rts = (a.Sq * a.G + 15) / 16;
    return launch_after(kv8_join_kernel<D, ManyRows>, dim3((unsigned)(a.B * a.c.heads * rts)), kJoinThreads<D, kManyRows>, 0, st, a, rts);
}

}  // namespace

cudaError_t launch_attend_many(const AttendArgs& a, int grid, cudaStream_t st)
{
    return a.c.dim == 64 ? launch_many<64>(a, grid, st) : launch_many<128>(a, grid, st);
}

}  // namespace hq
