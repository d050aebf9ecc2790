// hq_kv8.cu -- writing to the e4m3 KV cache: new tokens behind each sequence (append), and the tokens
// worth keeping moved to other pages (evict).
#include <cuda_runtime.h>

#include "hq_kv8.cuh"

namespace hq {
namespace {

// ------------------------------------------------------------------------------------------------
// Append.  A page's scale is the largest that any of its tokens asked for.  One thread block takes the keys
// and values of one (sequence, head, page that new tokens touch): it reads the new rows once into
// registers, reduces their maximum, joins it with the page's scale if the page held tokens before,
// codes the new rows and, only where the scale grew, the older rows again (exact in e4m3 but for
// codes that become subnormal).  Bound by the rows read and the codes written: 8 prompts of up to 2048 tokens,
// 32 heads, dim 128, 44.6 us, 4.5 TB/s (69% of the copy rate; a page's loads, maximum and stores follow each
// other); a step of one token by its launch and two dependent loads, 3.8 us.  The heads of a page follow
// one another, so that the blocks at work read whole tokens and write whole pages (46.4 us against 49.2).
// ------------------------------------------------------------------------------------------------
constexpr int kAThreads = 256;

struct AppendArgs {
    hq_kv8_t c;
    const void* x[2];  // keys, values
    int64_t sb[2], sh[2], ss[2];
    int64_t S;
    const int32_t* table;
    int64_t table_stride, max_pages;
    const int32_t* lens;
    const int32_t* n_new;
    uint32_t span, units;  // pages a sequence's new tokens can touch; B * heads * span
    WsHeader* ws;
};

// PASSES: row passes over a page.  Five blocks an SM where the rows of one fit 48 registers a thread (four:
// 46.4 us, six: 47.1).
template <typename T, int D, int PASSES>
__global__ void __launch_bounds__(kAThreads, sizeof(T) == 2 && PASSES <= 4 ? 5 : 1) kv8_append_kernel(const AppendArgs a)
{
    constexpr int LPR = D / 8;                // lanes of one row
    constexpr int RPP = kAThreads / LPR;      // rows of one pass
    // by turns, so that one barrier a unit (between the maxima and their use) suffices
    __shared__ uint32_t warp_max[2][2][kAThreads / 32];
    __shared__ uint32_t s_status, s_nonfinite;
    const int sub = threadIdx.x % LPR, row = threadIdx.x / LPR;
    if (threadIdx.x == 0) s_status = 0u, s_nonfinite = 0u;
    const int page = a.c.page;
    __syncthreads();
    int turn = 0;
    for (uint32_t u = blockIdx.x; u < a.units; u += gridDim.x, turn ^= 1) {
        const uint32_t bs = u / (uint32_t)a.c.heads;
        const int h = (int)(u - bs * (uint32_t)a.c.heads), b = (int)(bs / a.span);
        const uint32_t sp = bs - (uint32_t)b * a.span;
        // Every thread reaches the unit's one barrier, whatever the lengths and the table it read, and touches
        // only what they allow.
        const int64_t first = a.lens[b];
        int64_t n = a.n_new ? (int64_t)a.n_new[b] : a.S;
        const bool odd = first < 0 || n < 0 || n > a.S || first + n > a.max_pages * page;
        if (odd && threadIdx.x == 0 && sp == 0) atomicOr(&s_status, kStRange);
        n = min(n, a.S);
        const int64_t at = first < 0 ? a.max_pages : first / page + sp;  // page of the sequence
        const int64_t lo64 = max(first, at * page), hi64 = min(first + n, (at + 1) * page);
        const bool some = at < a.max_pages && lo64 < hi64;
        const int lo = some ? (int)(lo64 - at * page) : 0, hi = some ? (int)(hi64 - at * page) : 0;
        const int32_t id = some ? a.table[b * a.table_stride + at] : -1;
        // the new rows are on their way before the page is known
        Raw8<T> v[2][PASSES];
        if (!__any_sync(0xFFFFFFFFu, some)) {
            __syncthreads();
            continue;
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const T* x = static_cast<const T*>(a.x[kv]) + b * a.sb[kv] + h * a.sh[kv] + (at * page - first) * a.ss[kv];
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int r = p * RPP + row;
                v[kv][p].zero();
                if (r >= lo && r < hi) v[kv][p].load(x + r * a.ss[kv] + sub * 8);
            }
        }
        const bool good = id >= 0 && id < a.c.pages;
        if (some && !good && threadIdx.x == 0) atomicOr(&s_status, kStRange);
        const int64_t ph = good ? (int64_t)id * a.c.heads + h : 0;
        const float s_old[2] = {good && lo > 0 ? a.c.k_scale[ph] : 0.0f, good && lo > 0 ? a.c.v_scale[ph] : 0.0f};
        uint32_t top[2] = {0u, 0u};
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                uint32_t m = v[kv][p].amax_bits();
#pragma unroll
                for (int o = LPR / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                if (m > kFiniteMax) {  // a token with NaN or infinity is kept as zeros
                    v[kv][p].zero();
                    if (sub == 0) atomicOr(&s_status, kStNonfinite), atomicAdd(&s_nonfinite, 1u);
                    m = 0;
                }
                top[kv] = max(top[kv], m);
            }
            top[kv] = __reduce_max_sync(0xFFFFFFFFu, top[kv]);
            if ((threadIdx.x & 31) == 0) warp_max[turn][kv][threadIdx.x >> 5] = top[kv];
        }
        __syncthreads();  // also: every thread has read the old scales
        if (!good) continue;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
            for (int w = 0; w < kAThreads / 32; ++w) top[kv] = max(top[kv], warp_max[turn][kv][w]);
            if (top[kv] > kAmaxLimit && threadIdx.x == 0) atomicOr(&s_status, kStRange);
            const float s_new = fmaxf(s_old[kv], exp2_int(scale_exp(top[kv])));
            if (threadIdx.x == 0 && s_new != s_old[kv]) (kv ? a.c.v_scale : a.c.k_scale)[ph] = s_new;
            uint8_t* codes = (kv ? a.c.v : a.c.k) + ph * page * D + sub * 8;
            const float inv = __fdiv_rn(1.0f, s_new);
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int r = p * RPP + row;
                if (r >= lo && r < hi) *reinterpret_cast<uint2*>(codes + r * D) = encode8(v[kv][p], inv);
            }
            if (lo > 0 && s_new != s_old[kv]) {
                const float ratio = __fdiv_rn(s_old[kv], s_new);
                for (int r = row; r < lo; r += RPP) {
                    uint2* q = reinterpret_cast<uint2*>(codes + r * D);
                    const uint2 w = *q;
                    *q = make_uint2(rescale4(w.x, ratio), rescale4(w.y, ratio));
                }
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) slot_write(a.ws, gridDim.x, blockIdx.x, s_status, s_nonfinite);
}

// ------------------------------------------------------------------------------------------------
// Evict, first step: which slots of a (sequence, head) stay.  The last `recent` do; of the others the
// budget - recent with the largest weights, the lower slot first among equals.  One thread block reads
// the weights once and finds the one that divides them digit by digit over order-preserving keys:
// histograms of 11, 11 and 10 bits, each with a scan from the largest digit down.  Then every thread
// takes a run of consecutive slots, counts, and writes its kept ones behind those of the threads before
// it, so the kept slots come out in order.  Up to 8192 slots stay in registers; bound by instructions and,
// where half of the weights share an exponent, by the histogram's conflicts.
// ------------------------------------------------------------------------------------------------
constexpr int kEBins = 2048;
constexpr int64_t kEHeld = 40 * 1024;  // weights held in shared memory at most (160 KB)
constexpr int64_t kEPages = 4096;      // pages whose first rows are held there, if a sequence has no more

struct EvictArgs {
    hq_kv8_t c;
    const int32_t* table;
    int64_t table_stride, max_pages;
    const int32_t* lens;
    const float* w;
    int64_t wb, wh, L;
    int64_t budget, recent;
    const int32_t* to;
    int64_t to_stride;
    int32_t* out_lens;
    float* out_w;
    int64_t ob, oh;
    int32_t* idx;  // [B * heads, budget] cache rows of the kept slots, -1 on a page outside the pool
    uint32_t to_pages, units;
    int page_shift, held, pages;  // weights and pages held in shared memory
    WsHeader* ws;
};

// unsigned key in the order of the weights; -0 equals 0 and NaN sorts below everything
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (!(w == w)) return 0u;
    const uint32_t b = __float_as_uint(w + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int64_t kept_len(const EvictArgs& a, int64_t b, bool& odd)
{
    const int64_t most = min(a.L, a.max_pages << a.page_shift);
    const int64_t n = a.lens[b];
    odd = n < 0 || n > most;
    return max((int64_t)0, min(n, most));
}

// exclusive prefix sum of x over the thread block in thread order; `sums` holds one value per warp and is
// free again after the caller's next barrier
__device__ __forceinline__ uint32_t block_before(uint32_t x, uint32_t* sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += t;
    }
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    return s - x + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sums[lane] : 0u);
}

// E > 0: up to E * T weights, every thread's run of E consecutive ones as keys in its registers (E divides
// a page's sixteen slots, so the run lies on one page); E = 0: any number, from shared or global memory in
// every pass (the keys are made anew each time).
template <int T, int E>
__global__ void __launch_bounds__(T, T == 512 ? 2 : 1) kv8_select_kernel(const EvictArgs a)
{
    constexpr int OWN = kEBins / T;  // bins of a thread
    extern __shared__ float held_w[];
    int32_t* held_row = reinterpret_cast<int32_t*>(held_w + a.held);
    __shared__ alignas(16) uint32_t hist[kEBins];
    __shared__ uint32_t s_digit, s_need;
    __shared__ uint32_t sums[2][32];
    const int h = blockIdx.x % a.c.heads;
    const int64_t b = blockIdx.x / a.c.heads;
    __shared__ int s_n;
    if (threadIdx.x == 0) {  // read once: the whole block takes the same way
        bool odd;
        s_n = (int)kept_len(a, b, odd);
    }
    for (int i = threadIdx.x; i < kEBins; i += T) hist[i] = 0u;
    __syncthreads();
    const int n = s_n, keep = (int)min((int64_t)n, a.budget);
    const float* w = a.w + b * a.wb + h * a.wh;
    float* out_w = a.out_w ? a.out_w + b * a.ob + h * a.oh : nullptr;
    int32_t* idx = a.idx + (int64_t)blockIdx.x * a.budget;
    const int32_t* table = a.table + b * a.table_stride;
    // first cache row of a page of the sequence, -1 outside the pool
    auto first_row = [&](int pg) {
        const int32_t id = __ldg(table + pg);
        return id >= 0 && id < a.c.pages ? (int)(((uint32_t)id * a.c.heads + h) << a.page_shift) : -1;
    };
    for (int pg = threadIdx.x; pg < a.pages && pg << a.page_shift < n; pg += T) held_row[pg] = first_row(pg);
    auto row_of = [&](int slot) {
        const int row = a.pages ? held_row[slot >> a.page_shift] : first_row(slot >> a.page_shift);
        return row < 0 ? -1 : row + (slot & (a.c.page - 1));
    };
    after_me();
    if (n <= a.budget) {
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += T) {
            idx[i] = row_of(i);
            if (out_w) out_w[i] = w[i];
        }
        return;
    }
    const int recent = (int)min(a.recent, (int64_t)keep);
    const int old = n - recent, held = min(old, a.held);
    const int run = E ? E : (old + T - 1) / T;
    const int i0 = min(old, (int)threadIdx.x * run), i1 = min(old, i0 + run);
    uint32_t mine_k[E ? E : 1];
    if (E) {
        float x[E ? E : 1];
        if (E >= 4 && (reinterpret_cast<uintptr_t>(w) & 15u) == 0 && i0 + E <= i1) {
#pragma unroll
            for (int y = 0; y + 4 <= E; y += 4) {
                const float4 four = *reinterpret_cast<const float4*>(w + i0 + y);
                x[y] = four.x, x[y + 1] = four.y, x[y + 2] = four.z, x[y + 3] = four.w;
            }
        } else {
#pragma unroll
            for (int y = 0; y < E; ++y) x[y] = i0 + y < i1 ? w[i0 + y] : 0.0f;
        }
#pragma unroll
        for (int y = 0; y < E; ++y) mine_k[y] = weight_key(x[y]);
    } else {
#pragma unroll 4
        for (int i = threadIdx.x; i < held; i += T) held_w[i] = w[i];
    }
    auto weight_at = [&](int i) { return i < held ? held_w[i] : w[i]; };
    uint32_t need = (uint32_t)(keep - recent);  // still to find at or below the digits fixed so far
    uint32_t key = 0xFFFFFFFFu;                 // need 0: nothing lies above, none is taken at it
    __syncthreads();
    if (need > 0) {
        key = 0;
        uint32_t mask = 0;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
            const uint32_t digits = pass == 2 ? 1023u : 2047u;
            if (E) {
#pragma unroll
                for (int y = 0; y < E; ++y)
                    if (i0 + y < i1 && (mine_k[y] & mask) == key) atomicAdd(&hist[(mine_k[y] >> shift) & digits], 1u);
            } else {
                for (int i = threadIdx.x; i < old; i += T) {
                    const uint32_t k = weight_key(weight_at(i));
                    if ((k & mask) == key) atomicAdd(&hist[(k >> shift) & digits], 1u);
                }
            }
            __syncthreads();
            // thread t owns the OWN digits from kEBins - 1 - OWN t down: the scan runs from the largest
            const uint32_t low = kEBins - OWN * (threadIdx.x + 1);
            uint32_t c[OWN], sum = 0;
#pragma unroll
            for (int y = 0; y < OWN; ++y) sum += c[y] = hist[low + y];
            uint32_t above = block_before(sum, sums[0]);
            if (above < need && need <= above + sum) {
#pragma unroll
                for (int y = OWN - 1; y >= 0; --y) {
                    if (above < need && need <= above + c[y]) {
                        s_digit = low + y;
                        s_need = need - above;
                    }
                    above += c[y];
                }
            }
#pragma unroll
            for (int y = 0; y < OWN; ++y) hist[low + y] = 0u;
            __syncthreads();
            key |= s_digit << shift;
            mask |= digits << shift;
            need = s_need;
        }
    }
    // this thread's slots above the dividing key and at it
    uint32_t over = 0, same = 0;
    if (E) {
#pragma unroll
        for (int y = 0; y < E; ++y) {
            over += i0 + y < i1 && mine_k[y] > key;
            same += i0 + y < i1 && mine_k[y] == key;
        }
    } else {
        for (int i = i0; i < i1; ++i) {
            const uint32_t k = weight_key(weight_at(i));
            over += k > key;
            same += k == key;
        }
    }
    uint32_t above = block_before(over, sums[0]), at = block_before(same, sums[1]);
    auto keep_slot = [&](int i, int row, uint32_t k) {
        if (k > key || (k == key && at < need)) {
            const uint32_t pos = above + min(at, need);
            idx[pos] = row;
            if (out_w) out_w[pos] = w[i];
        }
        above += k > key;
        at += k == key;
    };
    if (over | same) {
        if (E) {
            const int row = row_of(i0);
#pragma unroll
            for (int y = 0; y < E; ++y)
                if (i0 + y < i1) keep_slot(i0 + y, row < 0 ? -1 : row + y, mine_k[y]);
        } else {
            for (int i = i0; i < i1; ++i) keep_slot(i, row_of(i), weight_key(weight_at(i)));
        }
    }
    for (int i = threadIdx.x; i < recent; i += T) {
        idx[keep - recent + i] = row_of(old + i);
        if (out_w) out_w[keep - recent + i] = w[old + i];
    }
}

// Second step: one thread block per (sequence, head, new page) gathers its rows of keys and values.  A page's
// scale is the largest of its rows' old scales; a row with a smaller one is coded again.  Every thread
// has all its 16-byte loads under way, beside the scales', before the first is stored.  Bound by the
// rows' bytes: 8 x 32 heads, 2048 of 8192 slots, 45 us of the operator's 63, 6.0 TB/s (91% of the copy rate);
// rows looked up one unit ahead made the registers cost residents (87 against 77 us then).
constexpr int kMThreads = 256;

template <int D, int PASSES>
__global__ void __launch_bounds__(kMThreads, PASSES > 2 ? 4 : 8) kv8_move_kernel(const EvictArgs a)
{
    constexpr int LPR = D / 16, RPP = kMThreads / LPR;
    __shared__ float s_ks[128], s_vs[128];
    __shared__ uint32_t s_top[2], s_status;
    __shared__ int64_t s_n;
    const int page = a.c.page;
    const int sub = threadIdx.x % LPR, row = threadIdx.x / LPR;
    const int32_t all_rows = (int32_t)((a.c.pages * a.c.heads) << a.page_shift);
    if (threadIdx.x == 0) s_status = 0u;
    wait_before_me();  // the kept rows
    for (uint32_t u = blockIdx.x; u < a.units; u += gridDim.x) {
        const uint32_t bh = u / a.to_pages, pg = u - bh * a.to_pages;
        const int b = (int)(bh / (uint32_t)a.c.heads), h = (int)(bh - (uint32_t)b * a.c.heads);
        __syncthreads();
        if (threadIdx.x == 0) {  // read once: the whole block takes the same way
            bool odd;
            s_n = min(kept_len(a, b, odd), a.budget);
            s_top[0] = s_top[1] = 0u;
            if (odd) s_status |= kStRange;
            // out_lens may be lens itself: every reader takes min(lens, budget), the value written here
            if (pg == 0 && h == 0) a.out_lens[b] = (int32_t)s_n;
        }
        __syncthreads();
        const int64_t n = s_n;
        const int rows = (int)min((int64_t)page, n - (int64_t)pg * page);
        if (rows <= 0) continue;
        const int32_t id = a.to[b * a.to_stride + pg];
        const int32_t* from = a.idx + (int64_t)bh * a.budget + (int64_t)pg * page;
        const int mine = (int)threadIdx.x < rows ? from[threadIdx.x] : 0;
        uint4 q[2][PASSES];
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int r = p * RPP + row, at = r < rows ? from[r] : -1;
            if (at >= 0 && at < all_rows) {
                q[0][p] = *reinterpret_cast<const uint4*>(a.c.k + (int64_t)at * D + sub * 16);
                q[1][p] = *reinterpret_cast<const uint4*>(a.c.v + (int64_t)at * D + sub * 16);
            }
        }
        uint32_t ktop = 0, vtop = 0;  // positive floats order like their bit patterns
        const bool good = mine >= 0 && mine < all_rows;  // a row that the selection wrote, on a page of the pool
        if ((int)threadIdx.x < rows && good) {
            const float ks = a.c.k_scale[mine >> a.page_shift], vs = a.c.v_scale[mine >> a.page_shift];
            s_ks[threadIdx.x] = ks;
            s_vs[threadIdx.x] = vs;
            ktop = __float_as_uint(ks);
            vtop = __float_as_uint(vs);
        }
        ktop = __reduce_max_sync(0xFFFFFFFFu, ktop);
        vtop = __reduce_max_sync(0xFFFFFFFFu, vtop);
        if ((threadIdx.x & 31) == 0 && (ktop | vtop)) atomicMax(&s_top[0], ktop), atomicMax(&s_top[1], vtop);
        if (__syncthreads_or(!good || id < 0 || id >= a.c.pages)) {  // a page outside the pool: left as it was
            if (threadIdx.x == 0) s_status |= kStRange;
            continue;
        }
        const float kto = __uint_as_float(s_top[0]), vto = __uint_as_float(s_top[1]);
        const int64_t to = (int64_t)id * a.c.heads + h;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int r = p * RPP + row;
            if (r < rows) {
                const int64_t at = ((to << a.page_shift) + r) * D + sub * 16;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const float s = kv ? s_vs[r] : s_ks[r], t = kv ? vto : kto;
                    uint4 x = q[kv][p];
                    if (s != t) {
                        const float ratio = __fdiv_rn(s, t);
                        x = make_uint4(rescale4(x.x, ratio), rescale4(x.y, ratio), rescale4(x.z, ratio), rescale4(x.w, ratio));
                    }
                    *reinterpret_cast<uint4*>((kv ? a.c.v : a.c.k) + at) = x;
                }
            }
        }
        if (threadIdx.x == 0) a.c.k_scale[to] = kto, a.c.v_scale[to] = vto;
    }
    __syncthreads();
    if (threadIdx.x == 0) slot_write(a.ws, gridDim.x, blockIdx.x, s_status, 0u);
}

template <int D>
cudaError_t launch_move(const EvictArgs& a, int grid, cudaStream_t st)
{
    constexpr int RPP = kMThreads / (D / 16);
    const int passes = (a.c.page + RPP - 1) / RPP;
    if (passes == 1) return launch_after(kv8_move_kernel<D, 1>, dim3((unsigned)grid), kMThreads, 0, st, a);
    if (passes == 2) return launch_after(kv8_move_kernel<D, 2>, dim3((unsigned)grid), kMThreads, 0, st, a);
    return launch_after(kv8_move_kernel<D, 128 / RPP>, dim3((unsigned)grid), kMThreads, 0, st, a);
}

template <typename T, int D>
void launch_append_dim(const AppendArgs& a, int grid, cudaStream_t st)
{
    constexpr int RPP = kAThreads / (D / 8);
    const int passes = (a.c.page + RPP - 1) / RPP;
    if (passes == 1) kv8_append_kernel<T, D, 1><<<grid, kAThreads, 0, st>>>(a);
    else if (passes == 2) kv8_append_kernel<T, D, 2><<<grid, kAThreads, 0, st>>>(a);
    else if (passes == 4) kv8_append_kernel<T, D, 4><<<grid, kAThreads, 0, st>>>(a);
    else kv8_append_kernel<T, D, 128 / RPP><<<grid, kAThreads, 0, st>>>(a);
}
template <typename T>
void launch_append(const AppendArgs& a, int grid, cudaStream_t st)
{
    if (a.c.dim == 64) launch_append_dim<T, 64>(a, grid, st);
    else launch_append_dim<T, 128>(a, grid, st);
}

int slots_grid(int64_t units) { return (int)(units < kMaxSlots ? units : kMaxSlots); }

}  // namespace
}  // namespace hq

using namespace hq;

extern "C" hq_status_t hq_kv8_append(const hq_kv8_append_t* p, void* ws, size_t ws_bytes, void* stream)
{
    if (!p || !kv8_cache_ok(&p->cache) || !p->k || !p->v || !p->table || !p->lens) return HQ_ERR_ARG;
    if (p->dtype != HQ_BF16 && p->dtype != HQ_F32) return HQ_ERR_ARG;
    if (!kv8_shape_supported(&p->cache)) return HQ_ERR_UNSUPPORTED;
    if (p->B < 1 || p->S < 1 || p->max_pages < 1 || p->table_stride < p->max_pages) return HQ_ERR_ARG;
    if (p->B > ((int64_t)1 << 24) || p->S > ((int64_t)1 << 31) - 1 || p->max_pages > ((int64_t)1 << 24)) return HQ_ERR_ARG;
    const int64_t es = p->dtype == HQ_BF16 ? 2 : 4;
    const int64_t strides = p->k_stride[0] | p->k_stride[1] | p->k_stride[2] | p->v_stride[0] | p->v_stride[1] | p->v_stride[2];
    const uintptr_t bases = reinterpret_cast<uintptr_t>(p->k) | reinterpret_cast<uintptr_t>(p->v);
    if ((strides * es) % 16 || (bases & 15u)) return HQ_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(p->table) | reinterpret_cast<uintptr_t>(p->lens) | reinterpret_cast<uintptr_t>(p->n_new)) & 3u)
        return HQ_ERR_ARG;
    if (ws && (ws_bytes < kSlotBytes || (reinterpret_cast<uintptr_t>(ws) & 15u))) return HQ_ERR_ARG;
    DeviceGuard dev(p->cache.k);
    if (!dev.ok) return HQ_ERR_ARG;
    AppendArgs a;
    a.c = p->cache;
    a.x[0] = p->k;
    a.x[1] = p->v;
    for (int i = 0; i < 2; ++i) {
        const int64_t* s = i ? p->v_stride : p->k_stride;
        a.sb[i] = s[0];
        a.sh[i] = s[1];
        a.ss[i] = s[2];
    }
    a.S = p->S;
    a.table = p->table;
    a.table_stride = p->table_stride;
    a.max_pages = p->max_pages;
    a.lens = p->lens;
    a.n_new = p->n_new;
    const int64_t span = (p->S + p->cache.page - 2) / p->cache.page + 1;
    if (span > (((int64_t)1 << 31) - 1) / p->cache.heads / p->B) return HQ_ERR_UNSUPPORTED;
    a.span = (uint32_t)span;
    a.units = (uint32_t)(p->B * p->cache.heads * span);
    a.ws = static_cast<WsHeader*>(ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int grid = slots_grid(a.units);
    if (p->dtype == HQ_BF16) launch_append<__nv_bfloat16>(a, grid, st);
    else launch_append<float>(a, grid, st);
    return cudaGetLastError() == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

extern "C" size_t hq_kv8_evict_workspace_bytes(int64_t B, int32_t heads, int64_t budget)
{
    if (B < 1 || heads < 1 || budget < 1 || B > ((int64_t)1 << 24) || budget > ((int64_t)1 << 31) - 1) return 0;
    return kSlotBytes + (size_t)B * (size_t)heads * (size_t)budget * sizeof(int32_t);
}

extern "C" hq_status_t hq_kv8_evict(const hq_kv8_evict_t* p, void* ws, size_t ws_bytes, void* stream)
{
    if (!p || !kv8_cache_ok(&p->cache) || !p->table || !p->lens || !p->weights || !p->to_table || !p->out_lens || !ws)
        return HQ_ERR_ARG;
    if (!kv8_shape_supported(&p->cache)) return HQ_ERR_UNSUPPORTED;
    const int64_t page = p->cache.page;
    if (p->B < 1 || p->max_pages < 1 || p->table_stride < p->max_pages || p->L < 1 || p->budget < 1 || p->recent < 0)
        return HQ_ERR_ARG;
    if (p->L > ((int64_t)1 << 31) - 1 || p->max_pages > ((int64_t)1 << 24) || p->budget > ((int64_t)1 << 31) - 1 ||
        p->B > ((int64_t)1 << 24) || p->B * p->cache.heads > ((int64_t)1 << 31) - 1)
        return HQ_ERR_ARG;
    const int64_t to_pages = (p->budget + page - 1) / page;
    if (p->to_pages < to_pages || p->to_stride < p->to_pages) return HQ_ERR_ARG;
    const uintptr_t al = reinterpret_cast<uintptr_t>(p->table) | reinterpret_cast<uintptr_t>(p->lens) |
                         reinterpret_cast<uintptr_t>(p->weights) | reinterpret_cast<uintptr_t>(p->to_table) |
                         reinterpret_cast<uintptr_t>(p->out_lens) | reinterpret_cast<uintptr_t>(p->out_weights);
    if ((al & 3u) || (reinterpret_cast<uintptr_t>(ws) & 15u) || p->out_weights == p->weights) return HQ_ERR_ARG;
    if (p->out_weights && expanded(p->ow_stride, {p->B, p->cache.heads})) return HQ_ERR_ARG;
    if (ws_bytes < hq_kv8_evict_workspace_bytes(p->B, p->cache.heads, p->budget)) return HQ_ERR_ARG;
    DeviceGuard dev(p->cache.k);
    if (!dev.ok) return HQ_ERR_ARG;
    EvictArgs a;
    a.c = p->cache;
    a.table = p->table;
    a.table_stride = p->table_stride;
    a.max_pages = p->max_pages;
    a.lens = p->lens;
    a.w = p->weights;
    a.wb = p->w_stride[0];
    a.wh = p->w_stride[1];
    a.L = p->L;
    a.budget = p->budget;
    a.recent = p->recent;
    a.to = p->to_table;
    a.to_stride = p->to_stride;
    a.out_lens = p->out_lens;
    a.out_w = p->out_weights;
    a.ob = p->ow_stride[0];
    a.oh = p->ow_stride[1];
    a.idx = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kSlotBytes);
    if (p->B * p->cache.heads > (((int64_t)1 << 31) - 1) / to_pages) return HQ_ERR_UNSUPPORTED;
    if (p->cache.pages * p->cache.heads > (((int64_t)1 << 31) - 1) / page) return HQ_ERR_UNSUPPORTED;  // cache rows in 31 bits
    a.to_pages = (uint32_t)to_pages;
    a.units = (uint32_t)(p->B * p->cache.heads * to_pages);
    a.page_shift = page_shift_of(p->cache.page);
    const int64_t most = p->L < p->max_pages * page ? p->L : p->max_pages * page;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned blocks = (unsigned)(p->B * p->cache.heads);
    // Weights in registers up to 8192.  Blocks of 1024 threads where every head has an SM of its own, else
    // blocks of 512, two on an SM: 8 heads of 8192 slots 11.5 us (both steps) with 1024 threads, 13.4 with 512;
    // 256 heads 50.6 and 47.7; 4000 slots 8.9, 9.6 and 24.1, 20.6.  Up to 1024 slots 512 threads either way:
    // 6.8 against 7.1 us, 256 heads 10.6 against 13.9.  From shared memory: 16.0 and 56.5 at 8192 slots.
    const bool wide = most > 1024 && blocks <= (unsigned)num_sms();
    const int runs = most <= 1024 ? 2 : (most <= 4096 ? 8 : (most <= 8192 ? 16 : 0));  // of 512 threads
    a.held = runs ? 0 : (int)(most < kEHeld ? most : kEHeld);
    a.pages = p->max_pages <= kEPages ? (int)p->max_pages : 0;
    a.ws = static_cast<WsHeader*>(ws);
    const size_t smem = 4 * (size_t)(a.held + a.pages);
    if (runs == 2) kv8_select_kernel<512, 2><<<blocks, 512, smem, st>>>(a);
    else if (runs == 8 && wide) kv8_select_kernel<1024, 4><<<blocks, 1024, smem, st>>>(a);
    else if (runs == 8) kv8_select_kernel<512, 8><<<blocks, 512, smem, st>>>(a);
    else if (runs == 16 && wide) kv8_select_kernel<1024, 8><<<blocks, 1024, smem, st>>>(a);
    else if (runs == 16) kv8_select_kernel<512, 16><<<blocks, 512, smem, st>>>(a);
    else {
        // set on every call: the attribute belongs to the current device's context
        if (cudaFuncSetAttribute(kv8_select_kernel<1024, 0>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(4 * (kEHeld + kEPages))) != cudaSuccess)
            return HQ_ERR_CUDA;
        kv8_select_kernel<1024, 0><<<blocks, 1024, smem, st>>>(a);
    }
    if (cudaGetLastError() != cudaSuccess) return HQ_ERR_CUDA;
    const int grid = slots_grid(a.units);
    const cudaError_t e = p->cache.dim == 64 ? launch_move<64>(a, grid, st) : launch_move<128>(a, grid, st);
    return e == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}
