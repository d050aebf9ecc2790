// hq_kv8_attend.cuh -- what the two attention kernels over the e4m3 KV cache share: arguments, lengths
// and masks, the division of the work into equal shares, and the join of the parts.
#pragma once
#include "hq_kv8.cuh"

namespace hq {

constexpr int kMaxBatch = 2048;   // sequences of one call (their prefix sums live in shared memory)
constexpr float kBoost = 7.0f;    // probabilities are held times 2^7, and up to 2^8 times that
constexpr float kSlack = 8.0f;    // before a larger maximum moves the reference they are relative to
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttendArgs {
    hq_kv8_t c;
    const __nv_bfloat16* q;
    int64_t qb, qh, qs;
    __nv_bfloat16* out;
    int64_t ob, oh, os;
    int B, Hq, Sq, G, page_shift;
    const int32_t* table;
    int64_t table_stride;
    int64_t slots;  // max_pages * page
    const int32_t* lens;
    const int32_t* q_lens;
    float scale;
    int causal;
    float* lse;
    int64_t lb, lh;
    const float* win;
    float* w;
    int64_t wib, wih, wb, wh, L;
    uint32_t* prefix;  // [B + 2] tiles before each sequence, of all, and the number of shares
    int2* len;         // [B] the lengths (slots, queries) that the first block read
    float* part_o;     // [2 grid][rows of a unit][D]
    float2* part_ml;   // [2 grid][rows of a unit]
    float* lse2;       // [B][heads][G Sq] binary logarithm of the sums (weights only)
    WsHeader* ws;
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// lengths of sequence b: cached slots and queries, inside what the call's shapes allow
struct SeqLen {
    int n, m;
    bool odd;
};
__device__ __forceinline__ SeqLen seq_len(const AttendArgs& a, int b)
{
    SeqLen s;
    const int n = a.lens[b], m = a.q_lens ? a.q_lens[b] : a.Sq;
    s.n = (int)max((int64_t)0, min((int64_t)n, a.slots));
    s.m = max(0, min(m, a.Sq));
    s.odd = n != s.n || m != s.m || (a.w && s.n > a.L);
    return s;
}
// slots that query i of m sees, of n
__device__ __forceinline__ int sees(const AttendArgs& a, int n, int m, int i)
{
    return a.causal ? max(0, n - m + i + 1) : n;
}

// first cache row (of [page][head][token]) of sixteen tokens from slot `tok`; -1 if their page is
// outside the pool.  The entry points keep the number of rows below 2^31.
__device__ __forceinline__ int locate(const AttendArgs& a, const int32_t* table, int h, int tok)
{
    const int32_t id = __ldg(table + (tok >> a.page_shift));
    return id >= 0 && id < a.c.pages ? (int)(((uint32_t)id * a.c.heads + h) << a.page_shift) + (tok & (a.c.page - 1)) : -1;
}

// a finished row r of a unit: the output, the logarithm of its sum
__device__ __forceinline__ void row_place(const AttendArgs& a, int h, int r, int& head, int& i)
{
    i = r / a.G;
    head = h * a.G + (r - i * a.G);
}
__device__ __forceinline__ void write_lse(const AttendArgs& a, int b, int h, int r, float M, float l)
{
    int head, i;
    row_place(a, h, r, head, i);
    const float l2 = l > 0.0f ? M - kBoost + log2f(l) : (l == 0.0f ? -INFINITY : l);  // a NaN sum stays one
    if (a.lse) a.lse[b * a.lb + head * a.lh + i] = l2 * kLn2;
    if (a.lse2) a.lse2[((int64_t)b * a.c.heads + h) * a.G * a.Sq + r] = l2;
}

// ------------------------------------------------------------------------------------------------
// Shares.  A unit is U::R rows of one (sequence, key head) against their visible slots, in tiles of
// U::TILE slots.  All units' tiles are laid end to end (sequences, then heads, then row tiles) and cut
// into equal shares, one per thread block.
// ------------------------------------------------------------------------------------------------
// Number of shares of W tiles in `units` units over `grid` thread blocks.  None is empty (the join walks a
// unit's shares one by one).  Few tiles are cut into fewer shares than thread blocks: a share of n tiles
// takes time with n, a unit of T tiles is joined in time with T / n, so n is about the root of T (8192
// slots of two heads: 26.9 us with shares of 2 tiles, 16.7 with 8; 1000 slots of eight heads: 10.6, 12.8).
__device__ __forceinline__ uint32_t share_count(uint32_t W, uint32_t units, uint32_t grid)
{
    const uint32_t n = max(2u, (uint32_t)sqrtf((float)W / (float)max(units, 1u)));
    return min((W + n - 1) / n, grid);
}

// Prefix sums of the sequences' tiles into `pre` [B + 1] (shared memory), the number of shares into
// pre[B + 1], the lengths behind them; block 0 also leaves all of it for the kernels that follow.  Lengths
// are read here and nowhere else: were they changed meanwhile, the results would be wrong, but every
// warp still walks the same units.  `scan` holds one value per warp.  Returns whether this thread met
// a length out of range.
__host__ __device__ constexpr size_t share_bytes(int64_t B) { return sizeof(uint32_t) * (size_t)((B + 3) / 2 * 2) + sizeof(int2) * (size_t)B; }
__device__ __forceinline__ int2* share_lens(uint32_t* pre, int B) { return reinterpret_cast<int2*>(pre + (B + 3) / 2 * 2); }
__device__ __forceinline__ const int2* share_lens(const uint32_t* pre, int B) { return reinterpret_cast<const int2*>(pre + (B + 3) / 2 * 2); }

template <class U, int THREADS>
__device__ __forceinline__ bool share_prefix(const AttendArgs& a, uint32_t* pre, uint64_t* scan)
{
    int2* len = share_lens(pre, a.B);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int run = (a.B + THREADS - 1) / THREADS, b0 = min(a.B, tid * run), b1 = min(a.B, b0 + run);
    uint64_t mine = 0;  // units (high word) and tiles
    uint32_t last = 0;
    bool odd = false;
    for (int b = b0; b < b1; ++b) {
        const SeqLen s = seq_len(a, b);
        odd |= s.odd;
        len[b] = make_int2(s.n, s.m);
        last = U::of_sequence(a, s);
        mine += last + ((uint64_t)(last ? a.c.heads * U::row_tiles(a, s.m) : 0) << 32);
    }
    uint64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    uint64_t before = inc - mine;
    for (int i = 0; i < warp; ++i) before += scan[i];
    uint32_t at = (uint32_t)before;
    for (int b = b0; b < b1; ++b) {
        pre[b] = at;
        at += b1 - b0 == 1 ? last : U::of_sequence(a, SeqLen{len[b].x, len[b].y, false});
    }
    if (tid == THREADS - 1) {
        pre[a.B] = at;
        pre[a.B + 1] = share_count(at, (uint32_t)((before + mine) >> 32), gridDim.x);
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int b = tid; b <= a.B + 1; b += THREADS) a.prefix[b] = pre[b];
        for (int b = tid; b < a.B; b += THREADS) a.len[b] = len[b];
    }
    return odd;
}

// the part of a thread block's share [w0, w1) that lies in the unit of tile w0
struct Segment {
    int b, h, rt;
    uint32_t t0, t1, tiles;  // tiles [t0, t1) of the unit's
    SeqLen s;
};
template <class U>
__device__ __forceinline__ Segment segment_at(const AttendArgs& a, const uint32_t* pre, uint32_t w0, uint32_t w1)
{
    Segment g;
    g.b = 0;
    for (int hi = a.B; hi - g.b > 1;) {
        const int mid = (g.b + hi) >> 1;
        if (pre[mid] <= w0) g.b = mid;
        else hi = mid;
    }
    const int2 len = share_lens(pre, a.B)[g.b];
    g.s = SeqLen{len.x, len.y, false};
    U::find(a, g.s, (pre[g.b + 1] - pre[g.b]) / a.c.heads, w0 - pre[g.b], g);
    g.t1 = min(g.tiles, g.t0 + (w1 - w0));
    return g;
}

// Joins the parts of the units that were cut, up to sixteen rows a thread block, and writes zeros where a
// row sees nothing.  A row's threads take four dims each; first they find the row's reference
// together.  U: how the attention kernel makes units (U::R rows each) and lays them end to end.
template <int ROWS>
constexpr int kJoinRows = ROWS < 16 ? ROWS : 16;
template <int D, int ROWS>
constexpr int kJoinThreads = D / 4 * kJoinRows<ROWS>;

template <int D, class U>
__global__ void __launch_bounds__((kJoinThreads<D, U::R>)) kv8_join_kernel(const AttendArgs a, int row_tiles_max)
{
    constexpr int JR = kJoinRows<U::R>, TPR = D / 4;
    const int jr = blockIdx.x % row_tiles_max, bh = blockIdx.x / row_tiles_max;
    const int h = bh % a.c.heads, b = bh / a.c.heads, rt = jr / (U::R / JR), sub = jr % (U::R / JR) * JR;
    after_me();
    wait_before_me();  // in every block, so that this grid never ends before the one it joins
    const int2 len = a.len[b];
    const SeqLen s{len.x, len.y, false};
    if (jr * JR >= s.m * a.G) return;
    __shared__ uint32_t s_tiles, s_before;
    if (threadIdx.x == 0) {  // sums over row tiles: one thread's work
        s_tiles = U::tiles(a, s, rt);
        s_before = U::before(a, s, h, rt);
    }
    __syncthreads();
    const uint32_t tiles = s_tiles, W = a.prefix[a.B], w0 = a.prefix[b] + s_before, w1 = w0 + tiles;
    // the share that holds tile w: the smallest c with w < floor((c + 1) W / shares)
    const uint32_t shares = a.prefix[a.B + 1];
    const int c0 = tiles ? (int)(((uint64_t)(w0 + 1) * shares - 1) / W) : 0;
    const int c1 = tiles ? (int)(((uint64_t)w1 * shares - 1) / W) : -1;
    if (tiles && c0 == c1) return;  // whole: written already
    const int r = sub + threadIdx.x / TPR, lane = threadIdx.x % TPR, rr = rt * U::R + r;
    if (rr >= s.m * a.G) return;  // a row's threads are whole halves of warps: the shuffles below stay inside
    const uint32_t mask = TPR == 32 ? 0xFFFFFFFFu : 0xFFFFu << (threadIdx.x & 16);
    auto at = [&](int c) { return (int64_t)(2 * c + (c == c0)) * U::R + r; };
    float M = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += TPR) M = fmaxf(M, a.part_ml[at(c)].x);
#pragma unroll
    for (int o = TPR / 2; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(mask, M, o));
    float L = 0.0f;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int c = c0; c <= c1; ++c) {
        const float2 ml = a.part_ml[at(c)];
        const float4 x = *reinterpret_cast<const float4*>(a.part_o + at(c) * D + 4 * lane);
        const float f = ml.x == -INFINITY ? 1.0f : ex2(ml.x - M);
        L = fmaf(ml.y, f, L);
        y.x = fmaf(x.x, f, y.x), y.y = fmaf(x.y, f, y.y), y.z = fmaf(x.z, f, y.z), y.w = fmaf(x.w, f, y.w);
    }
    if (lane == 0) write_lse(a, b, h, rr, M, L);
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    int head, i;
    row_place(a, h, rr, head, i);
    const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x * inv, y.y * inv), hi = __floats2bfloat162_rn(y.z * inv, y.w * inv);
    *reinterpret_cast<uint2*>(a.out + b * a.ob + head * a.oh + (int64_t)i * a.os + 4 * lane) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// what the attention entry point needs of the kernel for many rows (hq_kv8_prefill.cu)
constexpr int kManyRows = 256;  // rows of its units
cudaError_t launch_attend_many(const AttendArgs& a, int grid, cudaStream_t st);

}  // namespace hq
