// hq_fp8.cu -- quantization to e4m3 with a power-of-two scale for each block of 1 x 128 (activations)
// or 128 x 128 (weights).
//
//   s[t, rb] = 2^e, the smallest with max |x| over the block <= 448 s;  q = e4m3(x / s)
//
// One pass: a block's elements stay in registers between its maximum and its codes, so x is read
// once and q written once; the operator is bound by that traffic.  Sixteen lanes take one row of a
// block, eight elements (one or two 16-byte loads, one 8-byte store) each, so a warp's loads are
// two whole rows of the block.  Blocks of 1 x 128 reduce over their sixteen lanes, blocks of
// 128 x 128 over the thread block that holds one of them.
//
// 11008 x 4096 bf16 in blocks of 128 x 128: 27.0 us, 5.0 TB/s, 76% of the copy rate (a block does not load
// while it reduces and stores; streaming loads take 24.9 when replayed, but 30.7 against 28.8 in a
// loop of calls); 8 x 4096 in blocks of 1 x 128: 1.7 us, a launch.
#include <cuda_runtime.h>

#include "hq_fp8.cuh"
#include "hq_launch.h"

namespace hq {
namespace {

// threads of a block and row passes over its tile: 32 rows x 128 columns for blocks of 1 x 128, the
// 128 x 128 block itself otherwise
template <int BLOCK>
struct QuantCfg {
    static constexpr int THREADS = BLOCK == 128 ? 512 : 256;
    static constexpr int ROWS = THREADS / 16;  // rows of one pass
    static constexpr int PASSES = BLOCK == 128 ? 4 : 2;
    static constexpr int TILE = ROWS * PASSES;
};

struct QuantArgs {
    const void* x;
    int64_t rows, cols, ldx, ldq;
    uint8_t* q;
    float* scale;
    int64_t tiles_r, tiles;  // row tiles, all tiles
    WsHeader* ws;
};

// BLOCK: rows of a scale block (1 or the whole tile of 128); VEC: rows of x start on 16 bytes
template <typename T, int BLOCK, bool VEC>
__global__ void __launch_bounds__(QuantCfg<BLOCK>::THREADS, sizeof(T) == 2 ? 2048 / QuantCfg<BLOCK>::THREADS - 1 : 1024 / QuantCfg<BLOCK>::THREADS)
    fp8_quantize_kernel(const QuantArgs a)
{
    constexpr int kQThreads = QuantCfg<BLOCK>::THREADS, kQRows = QuantCfg<BLOCK>::ROWS;
    constexpr int PASSES = QuantCfg<BLOCK>::PASSES, TILE = QuantCfg<BLOCK>::TILE;
    __shared__ uint32_t warp_max[kQThreads / 32];
    __shared__ uint32_t s_status, s_nonfinite;
    const int sub = threadIdx.x & 15, row16 = threadIdx.x >> 4;
    if (threadIdx.x == 0) s_status = 0u, s_nonfinite = 0u;
    __syncthreads();
    const T* x = static_cast<const T*>(a.x);
    for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const int64_t r0 = (tile % a.tiles_r) * TILE;
        const int64_t kb = tile / a.tiles_r;
        const int64_t c = kb * 128 + sub * 8;  // this lane's first column
        Raw8<T> v[PASSES];
        uint32_t m[PASSES];
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int64_t r = r0 + p * kQRows + row16;
            v[p].zero();
            if (r < a.rows) {
                const T* at = x + r * a.ldx + c;
                if (VEC && c + 8 <= a.cols) v[p].load(at);
                else v[p].load_part(at, a.cols - c);
            }
        }
#pragma unroll
        for (int p = 0; p < PASSES; ++p) m[p] = v[p].amax_bits();
        if (BLOCK == 1) {
#pragma unroll
            for (int p = 0; p < PASSES; ++p)
#pragma unroll
                for (int o = 8; o; o >>= 1) m[p] = max(m[p], __shfl_xor_sync(0xFFFFFFFFu, m[p], o));
        } else {
            uint32_t top = 0;
#pragma unroll
            for (int p = 0; p < PASSES; ++p) top = max(top, m[p]);
            top = __reduce_max_sync(0xFFFFFFFFu, top);
            if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kQThreads / 32; ++w) top = max(top, warp_max[w]);
#pragma unroll
            for (int p = 0; p < PASSES; ++p) m[p] = top;
            __syncthreads();
        }
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int64_t r = r0 + p * kQRows + row16;
            if (r >= a.rows) continue;
            const bool bad = m[p] > kFiniteMax;  // a block with NaN or infinity is coded as zeros
            const int e = scale_exp(bad ? 0u : m[p]);
            const bool first = sub == 0 && (BLOCK == 1 || (p == 0 && row16 == 0));
            if (first) {
                a.scale[kb * (BLOCK == 1 ? a.rows : a.tiles_r) + (BLOCK == 1 ? r : r0 / TILE)] = exp2_int(e);
                if (bad) {
                    atomicOr(&s_status, kStNonfinite);
                    atomicAdd(&s_nonfinite, 1u);
                } else if (m[p] > kAmaxLimit) {
                    atomicOr(&s_status, kStRange);
                }
            }
            if (c < a.ldq) {  // columns cols .. ldq - 1 are zeros already in v; ldq is a multiple of 16
                const uint2 w = bad ? make_uint2(0u, 0u) : encode8(v[p], exp2_int(-e));
                *reinterpret_cast<uint2*>(a.q + r * a.ldq + c) = w;
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) slot_write(a.ws, gridDim.x, blockIdx.x, s_status, s_nonfinite);
}

template <typename T, int BLOCK>
cudaError_t launch_quantize(const QuantArgs& a, bool vec, cudaStream_t st)
{
    const int64_t most = kMaxSlots;
    const int grid = (int)(a.tiles < most ? a.tiles : most);
    if (vec) fp8_quantize_kernel<T, BLOCK, true><<<grid, QuantCfg<BLOCK>::THREADS, 0, st>>>(a);
    else fp8_quantize_kernel<T, BLOCK, false><<<grid, QuantCfg<BLOCK>::THREADS, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace
}  // namespace hq

using namespace hq;

extern "C" size_t hq_fp8_workspace_bytes(void) { return kSlotBytes; }

extern "C" hq_status_t hq_fp8_quantize(const void* x, hq_dtype_t dtype, int64_t rows, int64_t cols, int64_t ldx,
                                       int32_t block, uint8_t* q, int64_t ldq, float* scale, void* ws, size_t ws_bytes,
                                       void* stream)
{
    const int64_t most = (int64_t)1 << 31;
    if (!x || !q || !scale || rows < 1 || cols < 1 || rows > most || cols > most || ldx < cols) return HQ_ERR_ARG;
    if (dtype != HQ_BF16 && dtype != HQ_F32) return HQ_ERR_ARG;
    if (block != 1 && block != 128) return HQ_ERR_UNSUPPORTED;
    if (ldq != (cols + 15) / 16 * 16) return HQ_ERR_ARG;
    const uintptr_t es = dtype == HQ_BF16 ? 2 : 4;
    if ((reinterpret_cast<uintptr_t>(q) & 15u) || (reinterpret_cast<uintptr_t>(scale) & 3u) ||
        reinterpret_cast<uintptr_t>(x) % es)
        return HQ_ERR_ARG;
    if (ws && (ws_bytes < kSlotBytes || (reinterpret_cast<uintptr_t>(ws) & 15u))) return HQ_ERR_ARG;
    DeviceGuard dev(x);
    if (!dev.ok) return HQ_ERR_ARG;
    QuantArgs a;
    a.x = x;
    a.rows = rows;
    a.cols = cols;
    a.ldx = ldx;
    a.ldq = ldq;
    a.q = q;
    a.scale = scale;
    a.tiles_r = block == 128 ? (rows + 127) / 128 : (rows + QuantCfg<1>::TILE - 1) / QuantCfg<1>::TILE;
    a.tiles = a.tiles_r * ((cols + 127) / 128);
    a.ws = static_cast<WsHeader*>(ws);
    const bool vec = ((reinterpret_cast<uintptr_t>(x) | (uintptr_t)ldx * es) & 15u) == 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == HQ_BF16)
        e = block == 1 ? launch_quantize<__nv_bfloat16, 1>(a, vec, st) : launch_quantize<__nv_bfloat16, 128>(a, vec, st);
    else
        e = block == 1 ? launch_quantize<float, 1>(a, vec, st) : launch_quantize<float, 128>(a, vec, st);
    return e == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}
