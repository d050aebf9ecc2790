// hq_kv8_prefill.cu -- attention of many query rows over the e4m3 KV cache (prompt chunks, long
// speculative runs): both products on tcgen05 with TMEM accumulators.
//
// A unit is 256 rows of one (sequence, key head), two tiles of 128, against tiles of 128 slots.  Per slot
// tile and row tile: S = Q K^T (eight MMAs M 128, N 128, K 16) into TMEM, softmax by 128 threads with
// one row each, P as binary16 back into the same TMEM columns, O += P V (P from TMEM).  The two row
// tiles alternate, so the tensor cores work on one while the other's softmax runs; keys and values
// are read from the cache and converted to binary16 in shared memory once for both.
//
// Warps: 0-3 and 4-7 softmax of the two row tiles, 8-11 conversion, 12 MMA issue.  The time of a slot
// tile is bound by three units that are nearly even: the MMAs (4 x 512 cycles), the 32768
// exponentials (16 a cycle), and shared memory (operand reads of the first product, 64 KB written).
//
// Numerics as in the kernel for few rows (hq_kv8_attend.cu), except that value codes enter binary16
// multiplied by their page's scale over the largest scale of the segment: exact for power-of-two
// scales down to 2^-24 of that largest scale.
#include <cuda.h>
#include <cuda_runtime.h>

#include "hq_kv8_attend.cuh"
#include "hq_tc.cuh"

namespace hq {
namespace {

constexpr int kThreadsP = 512;
constexpr int kTok = 128;     // slots of a tile
constexpr int kScaleRing = 4;  // tiles whose key scales are kept: the converter is at most two ahead

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
    float vref[4];                        // by segment
    float red[4];
    alignas(8) uint64_t k_full[2];
    uint64_t k_empty[2], v_full[2], v_empty[2];
    uint64_t s_full[2], p_ready[2], o_full[2];  // by row tile
    uint64_t q_ready[2], drain;
    uint32_t tmem_base;
    uint32_t status;
    uint32_t scan[kThreadsP / 32];
};

// sixteen codes of one row (16-byte chunk c of it) as binary16, times r, into a swizzled operand tile
template <int D, bool SCALE>
__device__ __forceinline__ void put_codes(unsigned char (*tile)[PrefillSmem<D>::HALF], int row, int c, uint4 x, uint32_t r2)
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
    // chunks 4 .. 7 go to the second run, whose banks are the first one's: those lanes store their second
    // half first, so that eight lanes of a row meet in no bank
    unsigned char* to = tile[c >> 2];
    const int cc = (c & 3) * 2;
    const bool odd = c >= 4;
    const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
    *reinterpret_cast<uint4*>(to + swz(row, cc + odd)) = odd ? hi : lo;
    *reinterpret_cast<uint4*>(to + swz(row, cc + !odd)) = odd ? lo : hi;
}

template <int D>
__global__ void __launch_bounds__(kThreadsP, 1) kv8_prefill_kernel(const AttendArgs a)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    using Smem = PrefillSmem<D>;
    Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint32_t* pre = reinterpret_cast<uint32_t*>(&sm + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.k_full[i], 4);
            mbar_init(&sm.k_empty[i], 1);
            mbar_init(&sm.v_full[i], 4);
            mbar_init(&sm.v_empty[i], 1);
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_ready[i], 4);
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
    const uint32_t tbase = sm.tmem_base;
    const uint32_t W = pre[a.B];
    const uint32_t shares = min(W, gridDim.x);  // none is empty: the join walks a unit's shares one by one
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
        uint32_t seg_n = 0, tile_n = 0, s_n = 0;  // segments, slot tiles, and this row tile's scores so far
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
                // queries, a zero one becomes tiny, so that the factors of the scores are positive
                const int e = top ? min(126, 14 + 127 - (int)(top >> 23)) : 0;
                const float up = a.scale < 0.0f ? -exp2_int(e) : exp2_int(e);
                c = fmaxf(exp2_int(-e) * fabsf(a.scale) * kLog2e, 1e-37f);
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
            float m = -INFINITY, l = 0.0f;
            const int T = (int)(g.t1 - g.t0);
            if (active) {
#pragma unroll 1
                for (int j = 0; j < T; ++j) {
                    const int tok = (int)(g.t0 + j) * kTok;
                    wait(&sm.s_full[t], s_n + j);
                    if (!alive) continue;
                    tc_fence_after();
                    // twice over the scores, 32 at a time with the next 32 on their way: keeping all 128 would
                    // take the registers of a third warpgroup
                    uint32_t S[2][32];
                    tmem_ld32_nowait(ts, S[0]);
                    const float* ks = sm.ks[(tile_n + j) % kScaleRing];
                    const bool edge = tok + kTok > full_end || __any_sync(0xFFFFFFFFu, ks[lane & 7] < 0.0f);
                    // slots that this row does not see, or whose page is missing
                    auto hide = [&](uint32_t (&x)[32], int p, float k0, float k1) {
                        if (edge)
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                if (tok + 32 * p + y >= end || (y < 16 ? k0 : k1) < 0.0f) x[y] = 0xFF800000u;  // -infinity
                    };
                    float top = -INFINITY;
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        tmem_wait_ld();
                        tmem_ld32_nowait(ts + 32 * ((p + 1) & 3), S[(p + 1) & 1]);
                        const float k0 = ks[2 * p], k1 = ks[2 * p + 1];
                        hide(S[p & 1], p, k0, k1);
                        float x0 = __uint_as_float(S[p & 1][0]), x1 = __uint_as_float(S[p & 1][16]);
#pragma unroll
                        for (int y = 1; y < 16; ++y) {
                            x0 = fmaxf(x0, __uint_as_float(S[p & 1][y]));
                            x1 = fmaxf(x1, __uint_as_float(S[p & 1][16 + y]));
                        }
                        top = fmaxf(top, fmaxf(x0 * (c * fabsf(k0)), x1 * (c * fabsf(k1))));
                    }
                    const bool moves = top > m + kSlack;
                    if (__any_sync(0xFFFFFFFFu, moves)) {
                        const float next = moves ? top : m, f = m == -INFINITY ? 1.0f : ex2(m - next);
                        l *= f;
                        m = next;
                        if (j > 0) {  // the accumulator's products so far are done: this tile's scores came after them
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
                    }
                    const float sub = m == -INFINITY ? 0.0f : m - kBoost;
                    const float2 nsub = make_float2(-sub, -sub);
                    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        tmem_wait_ld();
                        if (p < 3) tmem_ld32_nowait(ts + 32 * (p + 1), S[(p + 1) & 1]);
                        const float k0 = ks[2 * p], k1 = ks[2 * p + 1];
                        hide(S[p & 1], p, k0, k1);
                        const float c0 = c * fabsf(k0), c1 = c * fabsf(k1);
                        uint32_t P[16];
#pragma unroll
                        for (int y = 0; y < 16; ++y) {
                            const float cq = y < 8 ? c0 : c1;
                            float2 x = __ffma2_rn(make_float2(__uint_as_float(S[p & 1][2 * y]), __uint_as_float(S[p & 1][2 * y + 1])),
                                                  make_float2(cq, cq), nsub);
                            x.x = ex2(x.x);
                            x.y = ex2(x.y);
                            sum = f2add(sum, x);
                            P[y] = pack_f16(x.x, x.y);
                        }
                        tmem_st16(ts + 16 * p, P);
                    }
                    l += sum.x + sum.y;
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.p_ready[t]);
                }
                // the segment's accumulator
                wait(&sm.o_full[t], seg_n);
                if (alive) {
                    tc_fence_after();
                    const float vref = sm.vref[seg_n & 3];
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
                s_n += T;
            } else {
                wait(&sm.o_full[t], seg_n);  // without rows: keep step with the others, one segment at a time
            }
            tile_n += T;
            ++seg_n;
            w0 += T;
        }
    } else if (warp < 12) {
        // ---------------- conversion: codes from the cache to binary16 operand tiles ----------------
        constexpr int CPR = D / 16, RPP = 128 / CPR, PASSES = 128 / RPP;  // chunks of a row, rows of a pass
        const int ct = tid - 256, c = ct % CPR, row0 = ct / CPR;
        uint32_t seg_n = 0, tile_n = 0;
        while (w0 < w1) {
            const Segment g = segment_at<ManyRows>(a, pre, w0, w1);
            const int32_t* table = a.table + g.b * a.table_stride;
            const int end = min((int)g.t1 * kTok, ManyRows::end(a, g.s, g.rt)), T = (int)(g.t1 - g.t0);
            // the largest value scale of the segment's pages
            float vmax = 0.0f;
            for (int tok = ((int)g.t0 * kTok / a.c.page + ct) * a.c.page; tok < end; tok += 128 * a.c.page) {
                const int32_t id = __ldg(table + (tok >> a.page_shift));
                if (id >= 0 && id < a.c.pages) vmax = fmaxf(vmax, __ldg(a.c.v_scale + (int64_t)id * a.c.heads + g.h));
                else atomicOr(&sm.status, kStRange);
            }
            vmax = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(vmax)));
            named_sync(1, 128);  // the last segment's maximum is read
            if (lane == 0) sm.red[warp - 8] = vmax;
            named_sync(1, 128);
            vmax = fmaxf(fmaxf(sm.red[0], sm.red[1]), fmaxf(sm.red[2], sm.red[3]));
            const float vref = vmax > 0.0f ? vmax : 1.0f;
            // the groups of sixteen slots of a tile: lane y < 8 knows the first cache row and the scales of
            // group y, one tile ahead of the codes; the keys of the next tile and the values of this one are
            // on their way while the tile before is stored
            int g_row = -1;
            float2 g_scale = make_float2(-1.0f, 0.0f);
            auto find_groups = [&](int j) {
                const int tok = (int)(g.t0 + j) * kTok + 16 * (lane & 7);
                g_row = j < T && tok < end ? locate(a, table, g.h, tok) : -1;
                g_scale = j < T && tok < end ? make_float2(-1.0f, 0.0f) : make_float2(1.0f, 0.0f);
                if (g_row >= 0) {
                    const int ph = g_row >> a.page_shift;
                    g_scale = make_float2(__ldg(a.c.k_scale + ph), __ldg(a.c.v_scale + ph));
                }
            };
            auto fetch = [&](uint4 (&x)[PASSES], const uint8_t* codes, int j) {
#pragma unroll
                for (int p = 0; p < PASSES; ++p) {
                    const int tk = p * RPP + row0, row = __shfl_sync(0xFFFFFFFFu, g_row, tk >> 4);
                    x[p] = row >= 0 && (int)(g.t0 + j) * kTok + tk < end
                               ? __ldg(reinterpret_cast<const uint4*>(codes + (int64_t)(row + (tk & 15)) * D) + c)
                               : make_uint4(0u, 0u, 0u, 0u);
                }
            };
            uint4 xk[PASSES], xv[PASSES];
            find_groups(0);
            fetch(xk, a.c.k, 0);
#pragma unroll 1
            for (int j = 0; j < T; ++j, ++tile_n) {
                const int st = tile_n & 1;
                fetch(xv, a.c.v, j);
                const float ks = g_scale.x, vr = g_scale.y / vref;
                const uint32_t vr2 = pack_f16(vr, vr);
                find_groups(j + 1);
                if (tile_n >= 2) wait(&sm.k_empty[st], tile_n / 2 - 1);
                if (ct < 8) sm.ks[tile_n % kScaleRing][ct] = ks;
                if (ct == 0 && j == 0) sm.vref[seg_n & 3] = vref;
#pragma unroll
                for (int p = 0; p < PASSES; ++p) put_codes<D, false>(sm.k[st], p * RPP + row0, c, xk[p], 0u);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.k_full[st]);
                if (j + 1 < T) fetch(xk, a.c.k, j + 1);
                if (tile_n >= 2) wait(&sm.v_empty[st], tile_n / 2 - 1);
#pragma unroll
                for (int p = 0; p < PASSES; ++p)
                    put_codes<D, true>(sm.v[st], p * RPP + row0, c, xv[p], __shfl_sync(0xFFFFFFFFu, vr2, (p * RPP + row0) >> 4));
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.v_full[st]);
            }
            ++seg_n;
            w0 += T;
        }
    } else {
        if (warp == 12) {
            // ---------------- MMA issue (one lane; the whole warp walks along for the waits) ----------------
            constexpr uint32_t IDS = idesc_f16(128, 128, false), IDO = idesc_f16(128, D, true);
            uint32_t seg_n = 0, tile_n = 0, s_n[2] = {0, 0};
            auto score = [&](int t, int st) {
                if (lane == 0) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t ad = sw128_desc(sm.q[t][kk >> 2]) + (uint64_t)(2 * (kk & 3));
                        const uint64_t bd = sw128_desc(sm.k[st][kk >> 2]) + (uint64_t)(2 * (kk & 3));
                        mma_f16_ss(tbase + 128 * t, ad, bd, IDS, kk > 0);
                    }
                    mma_commit(&sm.s_full[t]);
                }
                __syncwarp();
            };
            while (w0 < w1) {
                const Segment g = segment_at<ManyRows>(a, pre, w0, w1);
                const int T = (int)(g.t1 - g.t0);
                const int nt = g.rt * kManyRows + 128 < g.s.m * a.G ? 2 : 1;  // row tiles with rows
                wait(&sm.q_ready[0], seg_n);
                wait(&sm.q_ready[1], seg_n);
                wait(&sm.k_full[tile_n & 1], tile_n / 2);
                tc_fence_after();
                if (alive) {
                    for (int t = 0; t < nt; ++t) score(t, tile_n & 1);
                    if (lane == 0) mma_commit(&sm.k_empty[tile_n & 1]);
                    __syncwarp();
                }
#pragma unroll 1
                for (int j = 0; j < T; ++j, ++tile_n) {
                    const int st = tile_n & 1, next = st ^ 1;
                    wait(&sm.v_full[st], tile_n / 2);
                    for (int t = 0; t < nt; ++t) {
                        wait(&sm.p_ready[t], s_n[t]++);
                        if (t == 0 && j + 1 < T) wait(&sm.k_full[next], (tile_n + 1) / 2);
                        tc_fence_after();
                        if (!alive) continue;
                        if (lane == 0) {
#pragma unroll
                            for (int kk = 0; kk < kTok / 16; ++kk)
                                mma_f16_ts(tbase + 256 + 128 * t, tbase + 128 * t + 8 * kk,
                                           sw128_desc_mn(sm.v[st][0], Smem::HALF) + (uint64_t)(128 * kk), IDO, j > 0 || kk > 0);
                            if (t == nt - 1) mma_commit(&sm.v_empty[st]);
                            if (j + 1 == T) mma_commit(&sm.o_full[t]);
                            if (j + 1 == T && nt == 1) mma_commit(&sm.o_full[1]);
                        }
                        __syncwarp();
                        if (j + 1 < T) {
                            score(t, next);
                            if (t == nt - 1 && lane == 0) mma_commit(&sm.k_empty[next]);
                            __syncwarp();
                        }
                    }
                }
                ++seg_n;
                w0 += T;
            }
            // nothing may be under way when the tensor memory is given back
            if (lane == 0) {
                mma_commit(&sm.drain);
                mbar_wait_sleep(&sm.drain, 0);
            }
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
    const size_t smem = 1024 + sizeof(PrefillSmem<D>) + sizeof(uint32_t) * (size_t)(a.B + 1);
    cudaError_t e = cudaFuncSetAttribute(kv8_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kv8_prefill_kernel<D><<<grid, kThreadsP, smem, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int rts = (a.Sq * a.G + 15) / 16;
    kv8_join_kernel<D, ManyRows><<<(unsigned)(a.B * a.c.heads * rts), 128, 0, st>>>(a, rts, grid);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_many(const AttendArgs& a, int grid, cudaStream_t st)
{
    return a.c.dim == 64 ? launch_many<64>(a, grid, st) : launch_many<128>(a, grid, st);
}

}  // namespace hq
