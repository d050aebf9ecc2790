// hq_kv8_attend.cu -- attention of bf16 queries over the e4m3 KV cache.
//
//   s_rj = scale q_r . k_j,  out_r = sum_j exp(s_rj) v_j / sum_j exp(s_rj) over the visible slots j
//
// One pass over the keys and values with a running reference and sum.  The rows r of one (sequence,
// key head) are its queries times the query heads of the group; eight or sixteen of them make one
// unit, and all of them share the keys and values that a warp loads.  The units' slots, in tiles of 64, are
// laid end to end and cut into equal shares, one per resident thread block, so ragged batches and
// single long sequences fill the GPU alike; where a unit is cut, the parts leave their reference, sum and
// accumulator in the workspace and a second small kernel joins them.
//
// Codes become binary16 in registers (one conversion instruction for two codes, exact) and both
// products run on the matrix instruction m16n8k16 with binary32 accumulators, keys and values on the
// wide side: S^T = K Q^T (sixteen slots by eight rows), O^T += V^T P^T.  Sixteen slots of one head are
// contiguous (a page holds a multiple of sixteen), so every warp streams its groups of sixteen keys
// and values with two TMA boxes each into a ring of its own, without any barrier between warps.  The
// order of the contraction and of the output is free: every lane reads 16 contiguous bytes of a key or
// value row as the fragments it needs, the boxes' swizzle keeps those reads free of bank conflicts, and
// nothing is transposed but byte pairs of two value rows and the 8 x 8 tiles of probabilities
// (movmatrix).  Bound by the codes' bytes on long caches (5.7 TB/s); below some 10 MB by the latency of
// this kernel and the join (and the weights): 3 x 8 heads x 1500 slots, ten rows, weights: 17.9 us.
//   - queries become binary16 after a power-of-two scaling per row (bf16's 8 bits fit exactly, elements
//     below 2^-31 of the row's largest lose bits);
//   - probabilities become binary16 at 2^7 times their value relative to a running reference, which
//     moves up to the maximum when that is more than 2^8 larger: 11 bits, at most 2^15, and weights
//     down to 2^-31 of the largest still count.  The lanes look for a maximum only when one of them
//     meets a score beyond that;
//   - key scales multiply the scores, value scales stay out of the products: the accumulator is kept in
//     units of the last value scale and multiplied by the (power-of-two) ratio when that changes.
#include <cuda_runtime.h>

#include <algorithm>

#include "hq_kv8_attend.cuh"

namespace hq {
namespace {

constexpr int kWarps = 4, kThreadsA = 32 * kWarps;

// Rows of a unit, thread blocks of an SM and groups in a warp's ring.  Eight rows take half the registers
// of sixteen, so twelve warps are resident instead of eight, each with 12 KB of keys and values under
// way (dim 128): 8 sequences x 32 heads x 8192 slots, one row each, 94 us (5.7 TB/s, 87% of the copy rate)
// against 123 in units of sixteen.
template <int ROWS>
struct FewCfg {
    static constexpr int NT = ROWS / 8;                 // row tiles of the matrix instruction
    static constexpr int BLOCKS = ROWS == 8 ? 3 : 2;
    static constexpr int STAGES = ROWS == 8 ? 3 : 4;
};

// units of ROWS rows in tiles of 64 slots; slots that only later rows of a sequence see are part of
// every unit's tiles (at most its queries: few) and skipped
template <int ROWS>
struct FewRows {
    static constexpr int R = ROWS, TILE = 64;
    static __device__ __forceinline__ int row_tiles(const AttendArgs& a, int m) { return (m * a.G + R - 1) / R; }
    static __device__ __forceinline__ uint32_t tiles(const AttendArgs&, const SeqLen& s, int) { return (uint32_t)((s.n + TILE - 1) / TILE); }
    static __device__ __forceinline__ uint32_t of_sequence(const AttendArgs& a, const SeqLen& s)
    {
        return (uint32_t)(a.c.heads * row_tiles(a, s.m)) * tiles(a, s, 0);
    }
    static __device__ __forceinline__ uint32_t before(const AttendArgs& a, const SeqLen& s, int h, int rt)
    {
        return (uint32_t)(h * row_tiles(a, s.m) + rt) * tiles(a, s, 0);
    }
    static __device__ __forceinline__ void find(const AttendArgs& a, const SeqLen& s, uint32_t, uint32_t at, Segment& g)
    {
        const int rts = row_tiles(a, s.m);
        g.tiles = tiles(a, s, 0);
        const uint32_t unit = at / g.tiles;
        g.t0 = at - unit * g.tiles;
        g.h = unit / rts;
        g.rt = unit - g.h * rts;
    }
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, const uint32_t (&b)[2])
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
}
// transposes an 8 x 8 tile of binary16 pairs across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// 8 NT query rows as the B fragments of the score product; for the rows 8 i + 2 t + e of this lane's
// scores, their factor and the slots they see
template <int D, int NT>
struct QueryRows {
    uint32_t f[NT][D / 16][2];
    float c[NT][2];
    int end[NT][2];  // 0: no such row
    int full;        // slots that all rows see

    __device__ __forceinline__ void load(const AttendArgs& a, int b, int h, int rt, const SeqLen& s)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        full = 0x7FFFFFFF;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = (rt * NT + n) * 8 + g, i = r / a.G;
            const bool is = i < s.m;
            const __nv_bfloat16* q = a.q + b * a.qb + (int64_t)(h * a.G + (is ? r - i * a.G : 0)) * a.qh + (is ? i : 0) * a.qs;
            uint2 w[D / 16];
            uint32_t m = 0;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                w[kk] = is ? __ldg(reinterpret_cast<const uint2*>(q + t * (D / 4) + kk * 4)) : make_uint2(0u, 0u);
                m = max(m, max(max((w[kk].x << 16) & 0x7FFF0000u, w[kk].x & 0x7FFF0000u),
                               max((w[kk].y << 16) & 0x7FFF0000u, w[kk].y & 0x7FFF0000u)));
            }
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            const int e = m ? min(126, 14 + 127 - (int)(m >> 23)) : 0;
            const float up = exp2_int(e), factor = exp2_int(-e) * a.scale * kLog2e;
            const int sees_r = is ? sees(a, s.n, s.m, i) : 0;
            full = min(full, (int)__reduce_min_sync(0xFFFFFFFFu, is ? (uint32_t)sees_r : 0x7FFFFFFFu));
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                c[n][y] = __shfl_sync(0xFFFFFFFFu, factor, 4 * (2 * t + y));
                end[n][y] = __shfl_sync(0xFFFFFFFFu, sees_r, 4 * (2 * t + y));
            }
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                f[n][kk][0] = pack_f16(bf16lo_to_f32(w[kk].x) * up, bf16hi_to_f32(w[kk].x) * up);
                f[n][kk][1] = pack_f16(bf16lo_to_f32(w[kk].y) * up, bf16hi_to_f32(w[kk].y) * up);
            }
        }
    }
};

// byte offset of 16-byte chunk c of row r in a swizzled TMA box of D-byte rows
template <int D>
__device__ __forceinline__ uint32_t swz_row(int r, int c)
{
    return (uint32_t)(r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4));
}

// sixteen slots' keys: lane (g, t) holds dims t D/4 .. of slots g and g + 8, the rows of its score tile
template <int D>
struct KeyGroup {
    uint4 w[2][D / 64];

    __device__ __forceinline__ void load(const unsigned char* box)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                w[i][j] = *reinterpret_cast<const uint4*>(box + swz_row<D>(g + 8 * i, t * (D / 64) + j));
    }
    __device__ __forceinline__ void load_global(const uint8_t* k, bool ok)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                w[i][j] = ok ? __ldg(reinterpret_cast<const uint4*>(k + (g + 8 * i) * D + t * (D / 4) + j * 16))
                             : make_uint4(0u, 0u, 0u, 0u);
    }
    // s[n]: rows 8 n + 2 t, + 1 against slot g, then against slot g + 8
    template <int NT>
    __device__ __forceinline__ void scores(const QueryRows<D, NT>& q, float (&s)[NT][4]) const
    {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            const uint32_t x[4] = {w[0][j].x, w[0][j].y, w[0][j].z, w[0][j].w}, y[4] = {w[1][j].x, w[1][j].y, w[1][j].z, w[1][j].w};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const uint32_t a0 = e4m3x2_to_f16x2(x[z] & 0xFFFFu), a1 = e4m3x2_to_f16x2(y[z] & 0xFFFFu);
                const uint32_t a2 = e4m3x2_to_f16x2(x[z] >> 16), a3 = e4m3x2_to_f16x2(y[z] >> 16);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816(s[n], a0, a1, a2, a3, q.f[n][4 * j + z]);
            }
        }
    }
};

// sixteen slots' values: lane (g, t) holds dims g D/8 .. of slots 2 t, 2 t + 1, 2 t + 8 and 2 t + 9
template <int D>
struct ValueGroup {
    uint32_t w[4][D / 32];

    __device__ __forceinline__ void load(const unsigned char* box, int left)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 2 * t + (i & 1) + 8 * (i >> 1);
            if (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4*>(box + swz_row<D>(r, g));
                w[i][0] = x.x, w[i][1] = x.y, w[i][D / 32 - 2] = x.z, w[i][D / 32 - 1] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(box + swz_row<D>(r, g >> 1) + (g & 1) * 8);
                w[i][0] = x.x, w[i][1] = x.y;
            }
        }
        if (left < 16) {  // slots nobody sees may hold anything: zero times NaN
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (2 * t + (i & 1) + 8 * (i >> 1) >= left)
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) w[i][j] = 0u;
        }
    }
    // o[n][i]: rows 8 n + 2 t, + 1 of dim g D/8 + 2 i, then of dim g D/8 + 2 i + 1
    template <int NT>
    __device__ __forceinline__ void accumulate(const uint32_t (&p)[NT][2], float (&o)[NT][D / 16][4]) const
    {
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            const uint32_t x[2] = {__byte_perm(w[0][j], w[1][j], 0x5140), __byte_perm(w[0][j], w[1][j], 0x7362)};
            const uint32_t y[2] = {__byte_perm(w[2][j], w[3][j], 0x5140), __byte_perm(w[2][j], w[3][j], 0x7362)};
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const uint32_t a0 = e4m3x2_to_f16x2(x[z] & 0xFFFFu), a1 = e4m3x2_to_f16x2(x[z] >> 16);
                const uint32_t a2 = e4m3x2_to_f16x2(y[z] & 0xFFFFu), a3 = e4m3x2_to_f16x2(y[z] >> 16);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816(o[n][2 * j + z], a0, a1, a2, a3, p[n]);
            }
        }
    }
};

template <int D, int ROWS>
struct AttendSmem {
    static constexpr int STAGES = FewCfg<ROWS>::STAGES;
    unsigned char ring[kWarps][STAGES][2][16 * D];  // keys, values of a group (TMA boxes: 1024-byte aligned)
    float o[kWarps][ROWS][D + 4];
    float m[kWarps][ROWS], l[kWarps][ROWS];
    float2 scale[kWarps][STAGES];  // of the group's keys and values; values < 0: no such page
    uint64_t full[kWarps][STAGES];
    uint64_t scan[kWarps];
    uint32_t status;
};

constexpr float kNoReference = -3e38f;  // below every score: the first visible one moves it

template <int D, int ROWS>
__global__ void __launch_bounds__(kThreadsA, FewCfg<ROWS>::BLOCKS)
    kv8_attend_kernel(const AttendArgs a, const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv)
{
    constexpr int NT = FewCfg<ROWS>::NT, STAGES = FewCfg<ROWS>::STAGES;
    using U = FewRows<ROWS>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    using Smem = AttendSmem<D, ROWS>;
    Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint32_t* pre = reinterpret_cast<uint32_t*>(&sm + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    if (tid == 0) {
        sm.status = 0u;
        for (int w = 0; w < kWarps; ++w)
            for (int i = 0; i < STAGES; ++i) mbar_init(&sm.full[w][i], 1);
        fence_mbar_init();
    }
    if (share_prefix<U, kThreadsA>(a, pre, sm.scan) && blockIdx.x == 0) atomicOr(&sm.status, kStRange);
    after_me();
    const uint32_t W = pre[a.B];
    const uint32_t shares = pre[a.B + 1];
    uint32_t w0 = blockIdx.x < shares ? (uint32_t)((uint64_t)blockIdx.x * W / shares) : 0u;
    const uint32_t w1 = blockIdx.x < shares ? (uint32_t)((uint64_t)(blockIdx.x + 1) * W / shares) : 0u;
    uint32_t status = 0u;
    bool dead = false;  // after a timeout a warp only walks the loops, so that all reach the barriers
    uint32_t stage = 0, parity = 0;  // of the next group this warp waits for
    while (w0 < w1) {
        const Segment seg = segment_at<U>(a, pre, w0, w1);
        const SeqLen s = seg.s;
        const int b = seg.b, h = seg.h, rt = seg.rt;
        const uint32_t t0 = seg.t0, t1 = seg.t1, tiles = seg.tiles;
        const int last_row = min(rt * ROWS + ROWS - 1, s.m * a.G - 1);
        const int end = min((int)t1 * U::TILE, sees(a, s.n, s.m, last_row / a.G));
        const int groups = (end + 15) / 16;  // sixteen-slot groups up to the last visible slot
        const int32_t* table = a.table + b * a.table_stride;

        // this warp's groups: every kWarps-th; their page rows and scales are fetched 32 at a time, one
        // per lane, and the boxes of STAGES groups are under way at any time
        const int gr0 = (int)t0 * (U::TILE / 16) + warp, count = gr0 < groups && !dead ? (groups - gr0 + kWarps - 1) / kWarps : 0;
        int my_row = -1;
        float2 my_scale = make_float2(0.0f, -1.0f);
        auto issue = [&](int i, uint32_t st) {
            if ((i & 31) == 0) {
                my_row = i + lane < count ? locate(a, table, h, (gr0 + (i + lane) * kWarps) * 16) : -1;
                my_scale.y = -1.0f;
                if (my_row >= 0) {
                    const int ph = my_row >> a.page_shift;
                    my_scale = make_float2(__ldg(a.c.k_scale + ph), __ldg(a.c.v_scale + ph));
                } else if (i + lane < count) {
                    status |= kStRange;
                }
            }
            if (lane == (i & 31)) {  // the lane that knows the group issues it
                if (my_row >= 0) {
                    mbar_arrive_expect_tx(&sm.full[warp][st], 32 * D);
                    tma_load_2d(sm.ring[warp][st][0], &tk, 0, my_row, &sm.full[warp][st]);
                    tma_load_2d(sm.ring[warp][st][1], &tv, 0, my_row, &sm.full[warp][st]);
                } else {
                    mbar_arrive(&sm.full[warp][st]);
                }
                sm.scale[warp][st] = my_scale;  // may still be on its way when the boxes are asked for
            }
        };
        {
            uint32_t st = stage;
            for (int i = 0; i < STAGES && i < count; ++i) {
                issue(i, st);
                st = st + 1 == STAGES ? 0 : st + 1;
            }
        }
        QueryRows<D, NT> q;
        q.load(a, b, h, rt, s);
        float o[NT][D / 16][4], sub[NT][2], l[NT][2], vref = 1.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.0f;
            sub[n][0] = sub[n][1] = kNoReference;
            l[n][0] = l[n][1] = 0.0f;
        }
        __syncwarp();
        for (int i = 0; i < count; ++i) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sm.full[warp][stage], parity))) {
                status |= kStTimeout;
                for (int j = i; j < count && j < i + STAGES; ++j) {  // the copies under way land first, if they ever do
                    mbar_wait(&sm.full[warp][stage], parity);
                    stage = stage + 1 == STAGES ? 0 : stage + 1;
                    parity ^= stage == 0;
                }
                dead = true;
                break;
            }
            const int tok = (gr0 + i * kWarps) * 16;
            const float ks = sm.scale[warp][stage].x, vs = sm.scale[warp][stage].y;
            KeyGroup<D> k;
            ValueGroup<D> v;
            k.load(sm.ring[warp][stage][0]);
            v.load(sm.ring[warp][stage][1], end - tok);
            // The stage is filled again by the asynchronous proxy, which does not wait for loads from shared
            // memory that are merely issued: without the fence a group now and then read the next one's bytes.
            fence_proxy_async();
            __syncwarp();
            if (i + STAGES < count) issue(i + STAGES, stage);
            stage = stage + 1 == STAGES ? 0 : stage + 1;
            parity ^= stage == 0;
            if (vs < 0.0f) continue;
            float x[NT][4], y[NT][4];
            k.scores(q, y);
            const bool edge = tok + 16 > q.full;
            float top = -INFINITY;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[n][e] *= q.c[n][e & 1] * ks;
                    if (edge && tok + g + 8 * (e >> 1) >= q.end[n][e & 1]) y[n][e] = -INFINITY;
                    x[n][e] = y[n][e] - sub[n][e & 1];
                    top = fmaxf(top, x[n][e]);
                }
            // a reference that moves or another value scale changes the accumulator's units
            if (__any_sync(0xFFFFFFFFu, top > kBoost + kSlack || vs != vref)) {
                const float vr = __fdiv_rn(vref, vs);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float best = fmaxf(y[n][e], y[n][e + 2]);
#pragma unroll
                        for (int z = 4; z < 32; z <<= 1) best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, z));
                        const float next = best - kBoost > sub[n][e] + kSlack ? best - kBoost : sub[n][e];
                        const float f = ex2(sub[n][e] - next);
                        sub[n][e] = next;
                        l[n][e] *= f;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            o[n][j][e] *= f * vr;
                            o[n][j][e + 2] *= f * vr;
                        }
                        x[n][e] = y[n][e] - next;
                        x[n][e + 2] = y[n][e + 2] - next;
                    }
                vref = vs;
            }
            uint32_t p[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[n][e] = ex2(x[n][e]);
                    l[n][e & 1] += x[n][e];
                }
                p[n][0] = transpose8(pack_f16(x[n][0], x[n][1]));
                p[n][1] = transpose8(pack_f16(x[n][2], x[n][3]));
            }
            v.accumulate(p, o);
        }

        // join the warps: their accumulators through shared memory, each at the common reference
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * n + 2 * t + e;
#pragma unroll
                for (int z = 4; z < 32; z <<= 1) l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], z);
                if (g == 0) {
                    sm.m[warp][r] = sub[n][e] == kNoReference ? -INFINITY : sub[n][e] + kBoost;
                    sm.l[warp][r] = l[n][e];
                }
#pragma unroll
                for (int j = 0; j < D / 16; j += 2)
                    *reinterpret_cast<float4*>(&sm.o[warp][r][g * (D / 8) + 2 * j]) =
                        make_float4(o[n][j][e] * vref, o[n][j][e + 2] * vref, o[n][j + 1][e] * vref, o[n][j + 1][e + 2] * vref);
            }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == tiles;
        const int slot = 2 * blockIdx.x + (t0 == 0 ? 1 : 0);
        constexpr int TPR = kThreadsA / ROWS, DPT = D / TPR;  // threads of a row, dims of a thread
        const int r = tid / TPR, d0 = (tid % TPR) * DPT;
        float M = -INFINITY, f[kWarps], L = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.m[w][r]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            f[w] = sm.m[w][r] == -INFINITY ? 1.0f : ex2(sm.m[w][r] - M);
            L += sm.l[w][r] * f[w];
        }
        const int rr = rt * ROWS + r;
        if (!whole || rr < s.m * a.G) {
            const float inv = whole ? (L == 0.0f ? 0.0f : 1.0f / L) : 1.0f;
            int head, i;
            row_place(a, h, rr, head, i);
            __nv_bfloat16* out = a.out + b * a.ob + head * a.oh + (int64_t)i * a.os;
            if (d0 == 0) {
                if (whole) write_lse(a, b, h, rr, M, L);
                else a.part_ml[slot * ROWS + r] = make_float2(M, L);
            }
#pragma unroll
            for (int d = 0; d < DPT; d += 4) {
                float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][r][d0 + d]);
                    y.x = fmaf(x.x, f[w], y.x), y.y = fmaf(x.y, f[w], y.y), y.z = fmaf(x.z, f[w], y.z), y.w = fmaf(x.w, f[w], y.w);
                }
                if (whole) {
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x * inv, y.y * inv), hi = __floats2bfloat162_rn(y.z * inv, y.w * inv);
                    *reinterpret_cast<uint2*>(out + d0 + d) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                } else {
                    *reinterpret_cast<float4*>(a.part_o + ((int64_t)slot * ROWS + r) * D + d0 + d) = y;
                }
            }
        }
        __syncthreads();
        w0 += t1 - t0;
    }
    if (status) atomicOr(&sm.status, status);
    __syncthreads();
    if (tid == 0) slot_write(a.ws, gridDim.x, blockIdx.x, sm.status, 0u);
}

// The weight each cached slot received, summed over a key head's rows: with the rows' sums known,
// exp(s - lse) is recomputed from the keys.  One warp takes sixteen slots and walks the rows sixteen at a
// time, so every slot is summed by four lanes in a fixed order.  Reads the keys once more, half the bytes of
// the attention itself, and converts the queries again for every sixteen slots: one row over 8 x 32 heads x
// 8192 slots 327 us with weights, 92 without; 2 x 512 queries x 32 heads over 8192 slots 1.63 ms and 0.18.
template <int D>
__global__ void __launch_bounds__(kThreadsA, 2) kv8_weights_kernel(const AttendArgs a)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int h = blockIdx.y, b = blockIdx.z;
    const int tok = (blockIdx.x * kWarps + warp) * 16;
    wait_before_me();  // in every block, so that this grid never ends before those it follows
    const int2 len = a.len[b];
    const SeqLen s{len.x, len.y, false};
    const int n = (int)min((int64_t)s.n, a.L);
    if (tok >= n) return;
    const int row = locate(a, a.table + b * a.table_stride, h, tok);
    const bool ok = row >= 0;
    KeyGroup<D> k;
    k.load_global(a.c.k + (int64_t)(ok ? row : 0) * D, ok);
    const float ks = ok ? __ldg(a.c.k_scale + (row >> a.page_shift)) : 0.0f;
    float sum[2] = {0.0f, 0.0f};
    const float* lse2 = a.lse2 + ((int64_t)b * a.c.heads + h) * a.G * a.Sq;
    const int rows = s.m * a.G;
    for (int rt = 0; rt * 16 < rows && ok; ++rt) {
        QueryRows<D, 2> q;
        q.load(a, b, h, rt, s);
        float x[2][4];
        k.scores(q, x);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = rt * 16 + 8 * i + 2 * t + (e & 1);
                if (tok + g + 8 * (e >> 1) < q.end[i][e & 1]) sum[e >> 1] += ex2(x[i][e] * (q.c[i][e & 1] * ks) - lse2[r]);
            }
    }
    const float* win = a.win ? a.win + b * a.wib + h * a.wih : nullptr;
    float* w = a.w + b * a.wb + h * a.wh;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float x = sum[i];
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
        const int j = tok + g + 8 * i;
        if (t == 0 && j < n) w[j] = win ? win[j] + x : x;
    }
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// The kernel for many rows (tensor memory, units of 256 rows) reads the cache once for all of them; this
// one once for every sixteen, the second time from L2, but with far more of it under way.  8 heads of 4096
// slots, dim 128, four sequences: 32 rows 29.0 us here against 32.9 there, 64 rows 39.9 against 34.2; sixteen
// sequences: 63.8 against 80.9 and 111.5 against 85.4.
bool many_rows(int64_t rows) { return rows > 32; }
constexpr int kMaxGridFew = 3 * 148, kMaxGridMany = 148;  // thread blocks: residents of an SM times SMs, at most

struct AttendLayout {
    size_t prefix, len, part_o, part_ml, lse2, bytes;
};
// slots: of a sequence's table.  Parts: two of a unit's rows for each share, and a share has two tiles at least
// (share_count).
AttendLayout attend_layout(int64_t B, int64_t heads, int64_t Hq, int64_t Sq, int64_t D, int64_t slots, bool weights)
{
    const int64_t rows = Sq * (Hq / heads);
    const bool many = many_rows(rows);
    const int64_t unit = many ? kManyRows : (rows <= 8 ? 8 : 16), grid = many ? kMaxGridMany : kMaxGridFew;
    const int64_t tile = many ? 128 : 64, units = B * heads * ((rows + unit - 1) / unit), tiles = (slots + tile - 1) / tile;
    const int64_t shares = tiles > 2 * grid || units > 2 * grid ? grid : std::min(grid, (units * tiles + 1) / 2);
    const size_t parts = (size_t)(2 * shares * unit);
    AttendLayout l;
    l.prefix = align256(kSlotBytes);
    l.len = l.prefix + align256(sizeof(uint32_t) * (size_t)(B + 2));
    l.part_o = l.len + align256(sizeof(int2) * (size_t)B);
    l.part_ml = l.part_o + parts * (size_t)D * sizeof(float);
    l.lse2 = l.part_ml + parts * sizeof(float2);
    l.bytes = l.lse2 + (weights ? align256(sizeof(float) * (size_t)(B * Hq * Sq)) : 0);
    return l;
}

template <int D, int ROWS>
cudaError_t launch_few(const AttendArgs& a, cudaStream_t st)
{
    CUtensorMap tk, tv;
    const int64_t rows = a.c.pages * a.c.heads * a.c.page;
    if (!tensor_map_kv8(&tk, a.c.k, rows, D, 16) || !tensor_map_kv8(&tv, a.c.v, rows, D, 16)) return cudaErrorInvalidValue;
    const size_t smem = 1024 + sizeof(AttendSmem<D, ROWS>) + share_bytes(a.B);
    cudaError_t e = cudaFuncSetAttribute(kv8_attend_kernel<D, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int grid = min(FewCfg<ROWS>::BLOCKS * num_sms(), kMaxGridFew);
    kv8_attend_kernel<D, ROWS><<<grid, kThreadsA, smem, st>>>(a, tk, tv);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int rts = (a.Sq * a.G + ROWS - 1) / ROWS;
    return launch_after(kv8_join_kernel<D, FewRows<ROWS>>, dim3((unsigned)(a.B * a.c.heads * rts)), kJoinThreads<D, ROWS>, 0, st, a, rts);
}

template <int D>
cudaError_t launch_attend(const AttendArgs& a, bool many, cudaStream_t st)
{
    cudaError_t e;
    if (many) e = launch_attend_many(a, min(num_sms(), kMaxGridMany), st);
    else e = a.Sq * a.G <= 8 ? launch_few<D, 8>(a, st) : launch_few<D, 16>(a, st);
    if (e != cudaSuccess) return e;
    if (a.w) {
        const int64_t most = a.slots < a.L ? a.slots : a.L;
        const dim3 wg((unsigned)((most + 16 * kWarps - 1) / (16 * kWarps)), (unsigned)a.c.heads, (unsigned)a.B);
        e = launch_after(kv8_weights_kernel<D>, wg, kThreadsA, 0, st, a);
    }
    return e;
}

}  // namespace
}  // namespace hq

using namespace hq;

extern "C" size_t hq_kv8_attend_workspace_bytes(int64_t B, int32_t heads, int64_t Hq, int64_t Sq, int32_t D, int32_t weights)
{
    if (B < 1 || B > kMaxBatch || heads < 1 || Hq < heads || Hq % heads || Sq < 1 || (D != 64 && D != 128) || Hq > 65535 ||
        Sq > ((int64_t)1 << 24))
        return 0;
    return attend_layout(B, heads, Hq, Sq, D, (int64_t)1 << 30, weights != 0).bytes;
}

extern "C" size_t hq_kv8_attend_workspace_need(const hq_kv8_attend_t* p)
{
    if (!p || p->max_pages < 1 || p->max_pages > ((int64_t)1 << 24) || !kv8_shape_supported(&p->cache) ||
        !hq_kv8_attend_workspace_bytes(p->B, p->cache.heads, p->Hq, p->Sq, p->cache.dim, 0))
        return 0;
    return attend_layout(p->B, p->cache.heads, p->Hq, p->Sq, p->cache.dim, p->max_pages * p->cache.page, p->weights != nullptr).bytes;
}

extern "C" hq_status_t hq_kv8_attend(const hq_kv8_attend_t* p, void* ws, size_t ws_bytes, void* stream)
{
    if (!p || !kv8_cache_ok(&p->cache) || !p->q || !p->out || !p->table || !p->lens || !ws) return HQ_ERR_ARG;
    if (!kv8_shape_supported(&p->cache)) return HQ_ERR_UNSUPPORTED;
    const int64_t H = p->cache.heads, page = p->cache.page;
    if (p->B < 1 || p->Sq < 1 || p->Hq < H || p->Hq % H || p->max_pages < 1 || p->table_stride < p->max_pages) return HQ_ERR_ARG;
    if (!(p->scale == p->scale) || p->scale - p->scale != 0.0f) return HQ_ERR_ARG;
    if (p->B > kMaxBatch || p->Hq > 65535 || p->Sq > ((int64_t)1 << 24) || p->max_pages > ((int64_t)1 << 24)) return HQ_ERR_UNSUPPORTED;
    const int64_t G = p->Hq / H, rts = (p->Sq * G + 7) / 8, slots = p->max_pages * page;
    if (p->cache.pages * H > (((int64_t)1 << 31) - 1) / page) return HQ_ERR_UNSUPPORTED;  // cache rows in 31 bits
    // share units and thread blocks are counted in 31 bits, slots of a sequence too
    if (slots > ((int64_t)1 << 30) || p->Sq * G > ((int64_t)1 << 26) || p->B * H > ((int64_t)1 << 26) ||
        p->B * H * rts > ((int64_t)1 << 31) / ((slots + FewRows<16>::TILE - 1) / FewRows<16>::TILE))
        return HQ_ERR_UNSUPPORTED;
    const int64_t qs = p->q_stride[0] | p->q_stride[1] | p->q_stride[2];
    const int64_t os = p->out_stride[0] | p->out_stride[1] | p->out_stride[2];
    if ((qs | os) & 7) return HQ_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(p->q) | reinterpret_cast<uintptr_t>(p->out)) & 15u) return HQ_ERR_ARG;
    const uintptr_t al = reinterpret_cast<uintptr_t>(p->table) | reinterpret_cast<uintptr_t>(p->lens) |
                         reinterpret_cast<uintptr_t>(p->q_lens) | reinterpret_cast<uintptr_t>(p->lse) |
                         reinterpret_cast<uintptr_t>(p->weights) | reinterpret_cast<uintptr_t>(p->weights_in);
    if ((al & 3u) || (reinterpret_cast<uintptr_t>(ws) & 255u)) return HQ_ERR_ARG;
    if (p->weights && p->L < 1) return HQ_ERR_ARG;
    if ((p->weights_in && !p->weights) || p->out == p->q) return HQ_ERR_ARG;
    if (expanded(p->out_stride, {p->B, p->Hq, p->Sq}) || (p->lse && expanded(p->lse_stride, {p->B, p->Hq})) ||
        (p->weights && expanded(p->w_stride, {p->B, H})))
        return HQ_ERR_ARG;
    if (p->weights && p->B > 65535) return HQ_ERR_UNSUPPORTED;
    const bool many = many_rows(p->Sq * G);
    const AttendLayout l = attend_layout(p->B, H, p->Hq, p->Sq, p->cache.dim, slots, p->weights != nullptr);
    if (ws_bytes < l.bytes) return HQ_ERR_ARG;
    DeviceGuard dev(p->cache.k);
    if (!dev.ok) return HQ_ERR_ARG;
    AttendArgs a;
    a.c = p->cache;
    a.q = static_cast<const __nv_bfloat16*>(p->q);
    a.qb = p->q_stride[0];
    a.qh = p->q_stride[1];
    a.qs = p->q_stride[2];
    a.out = static_cast<__nv_bfloat16*>(p->out);
    a.ob = p->out_stride[0];
    a.oh = p->out_stride[1];
    a.os = p->out_stride[2];
    a.B = (int)p->B;
    a.Hq = (int)p->Hq;
    a.Sq = (int)p->Sq;
    a.G = (int)G;
    a.page_shift = page_shift_of(p->cache.page);
    a.table = p->table;
    a.table_stride = p->table_stride;
    a.slots = slots;
    a.lens = p->lens;
    a.q_lens = p->q_lens;
    a.scale = p->scale;
    a.causal = p->causal;
    a.lse = p->lse;
    a.lb = p->lse_stride[0];
    a.lh = p->lse_stride[1];
    a.win = p->weights_in;
    a.w = p->weights;
    a.wib = p->win_stride[0];
    a.wih = p->win_stride[1];
    a.wb = p->w_stride[0];
    a.wh = p->w_stride[1];
    a.L = p->L;
    char* base = static_cast<char*>(ws);
    a.prefix = reinterpret_cast<uint32_t*>(base + l.prefix);
    a.len = reinterpret_cast<int2*>(base + l.len);
    a.part_o = reinterpret_cast<float*>(base + l.part_o);
    a.part_ml = reinterpret_cast<float2*>(base + l.part_ml);
    a.lse2 = p->weights ? reinterpret_cast<float*>(base + l.lse2) : nullptr;
    a.ws = static_cast<WsHeader*>(ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = p->cache.dim == 64 ? launch_attend<64>(a, many, st) : launch_attend<128>(a, many, st);
    return e == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}
