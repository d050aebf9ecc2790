// hq_kv8.cu -- writing to the e4m3 KV cache: new tokens behind each sequence (append), and the tokens
// worth keeping moved to other pages (evict).
#include <cuda_runtime.h>

#include "hq_kv8.cuh"

namespace hq {
namespace {

// ------------------------------------------------------------------------------------------------
// Append.  A page's scale is the largest that any of its tokens asked for.  One thread block takes one
// (sequence, head, page that new tokens touch) of keys or values: it reads the new rows once into
// registers, reduces their maximum, joins it with the page's scale if the page held tokens before,
// codes the new rows and, only where the scale grew, the older rows again (exact in e4m3 but for
// codes that become subnormal).  Bound by the rows read and the codes written; a step of one token
// by its launch.
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
    int64_t span, units;  // pages a sequence's new tokens can touch; 2 * B * heads * span
    WsHeader* ws;
};

template <typename T, int D>
__global__ void __launch_bounds__(kAThreads) kv8_append_kernel(const AppendArgs a)
{
    constexpr int LPR = D / 8;                // lanes of one row
    constexpr int RPP = kAThreads / LPR;      // rows of one pass
    constexpr int PASSES = 128 / RPP;         // passes of the largest page
    __shared__ uint32_t warp_max[kAThreads / 32];
    __shared__ uint32_t s_status, s_nonfinite;
    const int sub = threadIdx.x % LPR, row = threadIdx.x / LPR;
    if (threadIdx.x == 0) s_status = 0u, s_nonfinite = 0u;
    __syncthreads();
    const int page = a.c.page;
    for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
        const int64_t sp = u % a.span;
        const int kv = (int)(u / a.span % 2);
        const int h = (int)(u / (2 * a.span) % a.c.heads);
        const int64_t b = u / (2 * a.span * a.c.heads);
        int64_t first = a.lens[b];
        int64_t n = a.n_new ? (int64_t)a.n_new[b] : a.S;
        const bool odd = first < 0 || n < 0 || n > a.S || first + n > a.max_pages * page;
        if (odd && threadIdx.x == 0 && sp == 0) atomicOr(&s_status, kStRange);
        n = min(n, a.S);
        if (first < 0 || n <= 0) continue;
        const int64_t at = first / page + sp;             // page of the sequence
        const int64_t lo64 = max(first, at * page), hi64 = min(first + n, (at + 1) * page);
        if (at >= a.max_pages || lo64 >= hi64) continue;
        const int lo = (int)(lo64 - at * page), hi = (int)(hi64 - at * page);
        const int32_t id = a.table[b * a.table_stride + at];
        if (id < 0 || id >= a.c.pages) {
            if (threadIdx.x == 0) atomicOr(&s_status, kStRange);
            continue;
        }
        const T* x = static_cast<const T*>(a.x[kv]) + b * a.sb[kv] + h * a.sh[kv] + (at * page - first) * a.ss[kv];
        const int64_t ph = (int64_t)id * a.c.heads + h;
        uint8_t* codes = (kv ? a.c.v : a.c.k) + ph * page * D;
        float* scale = (kv ? a.c.v_scale : a.c.k_scale) + ph;
        const float s_old = lo > 0 ? *scale : 0.0f;
        float v[PASSES][8];
        uint32_t top = 0;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int r = p * RPP + row;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
            if (r >= lo && r < hi) load8(x + r * a.ss[kv] + sub * 8, v[p]);
            uint32_t m = amax_bits8(v[p]);
#pragma unroll
            for (int o = LPR / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            if (m > kFiniteMax) {  // a token with NaN or infinity is kept as zeros
#pragma unroll
                for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
                if (sub == 0) atomicOr(&s_status, kStNonfinite), atomicAdd(&s_nonfinite, 1u);
                m = 0;
            }
            top = max(top, m);
        }
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = top;
        __syncthreads();  // also: every thread has read the old scale
#pragma unroll
        for (int w = 0; w < kAThreads / 32; ++w) top = max(top, warp_max[w]);
        if (top > kAmaxLimit && threadIdx.x == 0) atomicOr(&s_status, kStRange);
        const float s_new = fmaxf(s_old, exp2_int(scale_exp(top)));
        if (threadIdx.x == 0 && s_new != s_old) *scale = s_new;
        const float inv = __fdiv_rn(1.0f, s_new);
        const bool grown = lo > 0 && s_new != s_old;
        const float ratio = __fdiv_rn(s_old, s_new);
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int r = p * RPP + row;
            uint2* q = reinterpret_cast<uint2*>(codes + r * D + sub * 8);
            if (r >= lo && r < hi) {
                *q = encode8(v[p], inv);
            } else if (grown && r < lo) {
                const uint2 w = *q;
                *q = make_uint2(rescale4(w.x, ratio), rescale4(w.y, ratio));
            }
        }
        __syncthreads();  // warp_max is written again by the next unit
    }
    __syncthreads();
    if (threadIdx.x == 0) slot_write(a.ws, gridDim.x, blockIdx.x, s_status, s_nonfinite);
}

// ------------------------------------------------------------------------------------------------
// Evict, first step: which slots of a (sequence, head) stay.  The last `recent` do; of the others the
// budget - recent with the largest weights, the lower slot first among equals.  The weight that
// divides them is found digit by digit (four histograms of 8 bits over order-preserving keys), then
// every thread takes a run of consecutive slots, counts, and writes its kept ones behind those of the
// threads before it, so the kept slots come out in order.
// ------------------------------------------------------------------------------------------------
constexpr int kEThreads = 1024;

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
    int32_t* idx;  // [B * heads, budget] kept slots
    int64_t to_pages, units;
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
    const int64_t most = min(a.L, a.max_pages * a.c.page);
    const int64_t n = a.lens[b];
    odd = n < 0 || n > most;
    return max((int64_t)0, min(n, most));
}

__global__ void __launch_bounds__(kEThreads) kv8_select_kernel(const EvictArgs a)
{
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_digit, s_need;
    __shared__ uint64_t warp_sum[32];
    const int h = blockIdx.x % a.c.heads;
    const int64_t b = blockIdx.x / a.c.heads;
    bool odd;
    const int n = (int)kept_len(a, b, odd);
    const int keep = (int)min((int64_t)n, a.budget);
    const float* w = a.w + b * a.wb + h * a.wh;
    float* out_w = a.out_w ? a.out_w + b * a.ob + h * a.oh : nullptr;
    int32_t* idx = a.idx + (int64_t)blockIdx.x * a.budget;
    if (n <= a.budget) {
        for (int i = threadIdx.x; i < n; i += kEThreads) {
            idx[i] = i;
            if (out_w) out_w[i] = w[i];
        }
        return;
    }
    const int recent = (int)min(a.recent, (int64_t)keep);
    const int old = n - recent;
    uint32_t need = (uint32_t)(keep - recent);  // still to find at or below the digits fixed so far
    uint32_t key = 0, mask = 0;
    if (need > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (threadIdx.x < 256) hist[threadIdx.x] = 0u;
            __syncthreads();
            for (int i = threadIdx.x; i < old; i += kEThreads) {
                const uint32_t k = weight_key(w[i]);
                if ((k & mask) == key) atomicAdd(&hist[(k >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (threadIdx.x == 0) {  // from the largest digit down
                uint32_t left = need;
                int d = 255;
                while (d > 0 && hist[d] < left) left -= hist[d--];
                s_digit = (uint32_t)d;
                s_need = left;
            }
            __syncthreads();
            key |= s_digit << shift;
            mask |= 255u << shift;
            need = s_need;
        }
    } else {
        key = 0xFFFFFFFFu;  // nothing above, none taken at
    }
    // counts of this thread's run: slots above the dividing key (high word), at it (low word)
    const int run = (old + kEThreads - 1) / kEThreads;
    const int i0 = min(old, (int)threadIdx.x * run), i1 = min(old, i0 + run);
    uint64_t mine = 0;
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = weight_key(w[i]);
        mine += k > key ? (1ull << 32) : (k == key ? 1ull : 0ull);
    }
    uint64_t before = mine;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t t = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before += t;
    }
    if (lane == 31) warp_sum[warp] = before;
    __syncthreads();
    before -= mine;
    for (int i = 0; i < warp; ++i) before += warp_sum[i];
    uint32_t above = (uint32_t)(before >> 32), at = (uint32_t)before;
    for (int i = i0; i < i1; ++i) {
        const uint32_t k = weight_key(w[i]);
        const bool take = k > key || (k == key && at < need);
        if (take) {
            const uint32_t pos = above + min(at, need);
            idx[pos] = i;
            if (out_w) out_w[pos] = w[i];
        }
        above += k > key;
        at += k == key;
    }
    for (int i = threadIdx.x; i < recent; i += kEThreads) {
        idx[keep - recent + i] = old + i;
        if (out_w) out_w[keep - recent + i] = w[old + i];
    }
}

// Second step: one thread block per (sequence, head, new page) of keys or values gathers its rows.  The
// page's scale is the largest of its rows' old scales; a row with a smaller one is coded again.
constexpr int kMThreads = 256;

template <int D>
__global__ void __launch_bounds__(kMThreads) kv8_move_kernel(const EvictArgs a)
{
    constexpr int LPR = D / 16, RPP = kMThreads / LPR;
    __shared__ uint32_t s_top, s_status;
    const int page = a.c.page;
    const int sub = threadIdx.x % LPR, row = threadIdx.x / LPR;
    if (threadIdx.x == 0) s_status = 0u, s_top = 0u;
    __syncthreads();
    for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
        const int64_t pg = u % a.to_pages;
        const int kv = (int)(u / a.to_pages % 2);
        const int h = (int)(u / (2 * a.to_pages) % a.c.heads);
        const int64_t b = u / (2 * a.to_pages * a.c.heads);
        bool odd;
        const int64_t n = min(kept_len(a, b, odd), a.budget);
        if (odd && threadIdx.x == 0) atomicOr(&s_status, kStRange);
        // out_lens may be lens itself: every reader takes min(lens, budget), the value written here
        if (pg == 0 && kv == 0 && h == 0 && threadIdx.x == 0) a.out_lens[b] = (int32_t)n;
        const int rows = (int)min((int64_t)page, n - pg * page);
        if (rows <= 0) continue;
        const int32_t* idx = a.idx + (b * a.c.heads + h) * a.budget + pg * page;
        const int32_t* table = a.table + b * a.table_stride;
        const int32_t id = a.to[b * a.to_stride + pg];
        const uint8_t* src = kv ? a.c.v : a.c.k;
        float* scales = kv ? a.c.v_scale : a.c.k_scale;
        bool bad = id < 0 || id >= a.c.pages;
        uint32_t top = 0;  // positive floats order like their bit patterns
        for (int r = threadIdx.x; r < rows; r += kMThreads) {
            const int32_t from = table[idx[r] / page];
            if (from < 0 || from >= a.c.pages) bad = true;
            else top = max(top, __float_as_uint(scales[(int64_t)from * a.c.heads + h]));
        }
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if ((threadIdx.x & 31) == 0 && top) atomicMax(&s_top, top);
        if (__syncthreads_or(bad)) {  // a page outside the pool: this page is left as it was
            if (threadIdx.x == 0) atomicOr(&s_status, kStRange), s_top = 0u;
            __syncthreads();
            continue;
        }
        const float s_to = __uint_as_float(s_top);
        const int64_t to = ((int64_t)id * a.c.heads + h);
        for (int r = row; r < rows; r += RPP) {
            const int slot = idx[r];
            const int64_t from = (int64_t)table[slot / page] * a.c.heads + h;
            const float ratio = __fdiv_rn(scales[from], s_to);
            uint4 q = *reinterpret_cast<const uint4*>(src + (from * page + slot % page) * D + sub * 16);
            if (ratio != 1.0f)
                q = make_uint4(rescale4(q.x, ratio), rescale4(q.y, ratio), rescale4(q.z, ratio), rescale4(q.w, ratio));
            *reinterpret_cast<uint4*>((kv ? a.c.v : a.c.k) + (to * page + r) * D + sub * 16) = q;
        }
        if (threadIdx.x == 0) scales[to] = s_to;
        __syncthreads();
        if (threadIdx.x == 0) s_top = 0u;
        __syncthreads();
    }
    __syncthreads();
    if (threadIdx.x == 0) slot_write(a.ws, gridDim.x, blockIdx.x, s_status, 0u);
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
    if (p->B > ((int64_t)1 << 24) || p->S > ((int64_t)1 << 31) || p->max_pages > ((int64_t)1 << 24)) return HQ_ERR_ARG;
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
    a.span = (p->S + p->cache.page - 2) / p->cache.page + 1;
    a.units = 2 * p->B * p->cache.heads * a.span;
    a.ws = static_cast<WsHeader*>(ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int grid = slots_grid(a.units);
    if (p->dtype == HQ_BF16) {
        if (p->cache.dim == 64) kv8_append_kernel<__nv_bfloat16, 64><<<grid, kAThreads, 0, st>>>(a);
        else kv8_append_kernel<__nv_bfloat16, 128><<<grid, kAThreads, 0, st>>>(a);
    } else {
        if (p->cache.dim == 64) kv8_append_kernel<float, 64><<<grid, kAThreads, 0, st>>>(a);
        else kv8_append_kernel<float, 128><<<grid, kAThreads, 0, st>>>(a);
    }
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
    a.to_pages = to_pages;
    a.units = 2 * p->B * p->cache.heads * to_pages;
    a.ws = static_cast<WsHeader*>(ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    kv8_select_kernel<<<(unsigned)(p->B * p->cache.heads), kEThreads, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return HQ_ERR_CUDA;
    const int grid = slots_grid(a.units);
    if (p->cache.dim == 64) kv8_move_kernel<64><<<grid, kMThreads, 0, st>>>(a);
    else kv8_move_kernel<128><<<grid, kMThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}
