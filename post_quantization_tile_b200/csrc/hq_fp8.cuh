// hq_fp8.cuh -- helpers shared by the 8-bit floating-point kernels: e4m3 conversions, the
// power-of-two scale of a block, and the status slots of the workspace.
#pragma once
#include <cuda_fp16.h>

#include "hq_common.cuh"

namespace hq {

// ------------------------------------------------------------------------------------------------
// Status without a clearing launch: every block of a grid owns one slot and writes it in any case;
// block 0 writes the header with their number, and hq_status_read merges them.  `ws` may be NULL
// (nothing is recorded then).  The grids are at most kMaxSlots blocks (each walks its share).
// ------------------------------------------------------------------------------------------------
struct StatusSlot {
    uint32_t status;
    uint32_t nonfinite;
};
constexpr int kMaxSlots = 4096;
constexpr size_t kSlotBytes = sizeof(WsHeader) + sizeof(StatusSlot) * kMaxSlots;

__device__ __forceinline__ void slot_write(WsHeader* ws, uint32_t slots, uint32_t slot, uint32_t status, uint32_t nonfinite)
{
    if (!ws) return;
    StatusSlot* s = reinterpret_cast<StatusSlot*>(ws + 1);
    s[slot] = StatusSlot{status, nonfinite};
    if (slot == 0) {
        WsHeader h{};
        h.slots = slots;
        *ws = h;
    }
}

// ------------------------------------------------------------------------------------------------
// Kernels of one call that follow one another: the first lets the second's blocks come up while it
// still runs (after_me), the second waits for its results before it touches them (wait_before_me).
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ void after_me() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_before_me() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// launches a kernel that starts with wait_before_me()
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args)
{
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

// ------------------------------------------------------------------------------------------------
// e4m3
// ------------------------------------------------------------------------------------------------
// two binary32 -> two e4m3 codes (lo in the low byte), nearest even, saturating at 448
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// two e4m3 codes (the low 16 bits of w) -> binary16 pair, exact
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
    return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t w)
{
    const uint32_t h = e4m3x2_to_f16x2(w);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// the four codes of w times r (a power of two unless the scales came from elsewhere), coded again
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r)
{
    const float2 a = e4m3x2_to_float2(w & 0xFFFFu), b = e4m3x2_to_float2(w >> 16);
    return e4m3x4(__fmul_rn(a.x, r), __fmul_rn(a.y, r), __fmul_rn(b.x, r), __fmul_rn(b.y, r));
}

// Exponent e of a block's scale 2^e from the bit pattern of its largest magnitude: the smallest e
// in [-40, 40] with amax <= 448 * 2^e (448 = 1.75 * 2^8, the largest e4m3 number).  A power of two
// costs e4m3 nothing but the place of its subnormals, and makes x / 2^e, and the codes of a block
// whose scale grows, exact.  The range keeps the ratio of any two scales inside binary32.
constexpr int kScaleExpMin = -40, kScaleExpMax = 40;
__device__ __forceinline__ int scale_exp(uint32_t amax_bits)
{
    const int e = (int)(amax_bits >> 23) - 127 - ((amax_bits & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
    return max(kScaleExpMin, min(kScaleExpMax, e));
}
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((127 + e) << 23); }
// the largest magnitude the largest scale can hold (448 * 2^40), as a bit pattern
constexpr uint32_t kAmaxLimit = ((127u + 48u) << 23) | 0x600000u;

// eight elements of a row as they lie in memory (bf16: four words, fp32: eight), kept so between their
// maximum and their codes
template <typename T>
struct Raw8;

template <>
struct Raw8<__nv_bfloat16> {
    uint32_t w[4];
    __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
    __device__ __forceinline__ void load(const __nv_bfloat16* p)  // 16-byte aligned
    {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    }
    __device__ __forceinline__ void load_part(const __nv_bfloat16* p, int64_t left)  // any alignment, `left` elements
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) w[i >> 1] |= (uint32_t)__bfloat16_as_ushort(p[i]) << (16 * (i & 1));
    }
    // bit pattern (binary32) of the largest magnitude: above kFiniteMax where an element is infinite or NaN
    __device__ __forceinline__ uint32_t amax_bits() const
    {
        __nv_bfloat162 m = __habs2(at(0));
#pragma unroll
        for (int i = 1; i < 4; ++i) m = __hmax2_nan(m, __habs2(at(i)));
        const uint32_t b = *reinterpret_cast<const uint32_t*>(&m) & 0x7FFF7FFFu;
        return max(b & 0xFFFF0000u, b << 16);
    }
    __device__ __forceinline__ float2 get(int i) const { return make_float2(bf16lo_to_f32(w[i]), bf16hi_to_f32(w[i])); }
    __device__ __forceinline__ __nv_bfloat162 at(int i) const { return *reinterpret_cast<const __nv_bfloat162*>(&w[i]); }
};

template <>
struct Raw8<float> {
    float v[8];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
    __device__ __forceinline__ void load(const float* p)
    {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    __device__ __forceinline__ void load_part(const float* p, int64_t left)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) v[i] = p[i];
    }
    __device__ __forceinline__ uint32_t amax_bits() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        return m;
    }
    __device__ __forceinline__ float2 get(int i) const { return make_float2(v[2 * i], v[2 * i + 1]); }
};

constexpr uint32_t kFiniteMax = 0x7F7FFFFFu;

// the codes of eight elements, inv = 1 / scale
template <typename T>
__device__ __forceinline__ uint2 encode8(const Raw8<T>& x, float inv)
{
    const float2 i2 = make_float2(inv, inv);
    const float2 a = f2mul(x.get(0), i2), b = f2mul(x.get(1), i2), c = f2mul(x.get(2), i2), d = f2mul(x.get(3), i2);
    return make_uint2(e4m3x4(a.x, a.y, b.x, b.y), e4m3x4(c.x, c.y, d.x, d.y));
}

}  // namespace hq
