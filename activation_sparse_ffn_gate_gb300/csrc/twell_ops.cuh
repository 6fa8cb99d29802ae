// twell_ops.cuh -- helpers shared by the operators around the FFN (norm, key-value cache, attention
// over it, 4-bit products): 8-element loads and stores, the 8-bit rounding with its scale, and on the host their
// workspaces' sizes and the shared memory of their kernels.
#pragma once

#include <algorithm>
#include <atomic>

#include "twell_common.cuh"

namespace twell {

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&o)[8])
{
    unpack16(*reinterpret_cast<const uint4*>(p), o, static_cast<__nv_bfloat16*>(nullptr));
}
__device__ __forceinline__ void load8(const float* p, float (&o)[8])
{
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w;
    o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&o)[8])
{
    *reinterpret_cast<uint4*>(p) = pack16(o, static_cast<__nv_bfloat16*>(nullptr));
}
__device__ __forceinline__ void store8(float* p, const float (&o)[8])
{
    *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(o[4], o[5], o[6], o[7]);
}

// Two fp32 numbers in one register pair, for the instructions that work on both.
struct F2 {
    unsigned long long v;
    __device__ __forceinline__ static F2 of(float a, float b)
    {
        F2 r;
        asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
        return r;
    }
    __device__ __forceinline__ void get(float& a, float& b) const
    {
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
    }
};
__device__ __forceinline__ F2 operator*(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ void to_f2(const float (&v)[8], F2 (&o)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = F2::of(v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void from_f2(const F2 (&v)[4], float (&o)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i].get(o[2 * i], o[2 * i + 1]);
}
template <typename E>
__device__ __forceinline__ void load8(const E* p, F2 (&o)[4])
{
    float v[8];
    load8(p, v);
    to_f2(v, o);
}
template <typename E>
__device__ __forceinline__ void store8(E* p, const F2 (&v)[4])
{
    float o[8];
    from_f2(v, o);
    store8(p, o);
}

// 8-bit rounding of values whose largest magnitude is `top`: code = e4m3(v * (448 / a)) to nearest
// even, a = max(top, 2^-60), so that 448 / a stays finite and a row of zeros has codes 0; the code
// stands for code * scale, scale = a / 448. A row that holds an infinity has an infinite scale and
// codes 0 or NaN; a NaN element has the code NaN and does not count toward `top`.
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxMin = 8.6736173798840355e-19f;  // 2^-60

struct Scale8 {
    float a, mul;
    // The factor is rounded once: with a reciprocal to 2^-23 2% to 10% more codes would fall to the other side of a tie
    // (30000 x 1024 then takes 25.3 us, so 26.4; 27.3 with the scale's own quotient).
    __device__ __forceinline__ static Scale8 of(float top)
    {
        const float a = fmaxf(top, kAmaxMin);
        return {a, kE4m3Max / a};
    }
    // Once a group, by the thread that writes it.
    __device__ __forceinline__ float scale() const { return a / kE4m3Max; }
    // two codes, the first in the low byte
    __device__ __forceinline__ static uint32_t round2(float a, float b)
    {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
        return r;
    }
    __device__ __forceinline__ uint32_t pack2(float a, float b) const { return round2(a * mul, b * mul); }
    __device__ __forceinline__ uint2 pack8(const F2 (&v)[4]) const
    {
        const F2 m = F2::of(mul, mul);
        F2 s[4];
        float o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = v[i] * m;
        from_f2(s, o);
        return make_uint2(round2(o[0], o[1]) | (round2(o[2], o[3]) << 16), round2(o[4], o[5]) | (round2(o[6], o[7]) << 16));
    }
    __device__ __forceinline__ uint2 pack8(const float (&v)[8]) const
    {
        return make_uint2(pack2(v[0], v[1]) | (pack2(v[2], v[3]) << 16), pack2(v[4], v[5]) | (pack2(v[6], v[7]) << 16));
    }
};

// Two e4m3 codes (low byte first) as an fp16 pair; every e4m3 value is exact in fp16.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t v)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}
// Four codes as two fp16 pairs.
__device__ __forceinline__ void e4m3x4_f16(uint32_t v, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}
__device__ __forceinline__ float2 e4m3x2_f32(uint16_t v)
{
    const uint32_t h = e4m3x2_f16x2(v);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace twell

namespace twell_host {

// Bytes of the workspaces of twell_add_rmsnorm_bwd (twell_norm.cu) and twell_paged_attn_decode (twell_attn.cu).
size_t norm_bwd_ws_bytes(int N, int d);
size_t paged_attn_ws_bytes(int B, int hd);

// Allow `kern` up to `bytes` of dynamic shared memory, the most that any of its launches takes, on the current
// device. `done` is the caller's, one for each kernel: a bit for each device it has been allowed on, so that a
// kernel launched often is asked about once.
template <typename K>
twell_status allow_smem(K kern, size_t bytes, std::atomic<uint64_t>& done)
{
    DevInfo d;
    if (dev_info(&d) != TWELL_OK) return TWELL_ERR_CUDA;
    const uint64_t bit = 1ull << d.device;
    if (done.load(std::memory_order_relaxed) & bit) return TWELL_OK;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess)
        return TWELL_ERR_CUDA;
    done.fetch_or(bit, std::memory_order_relaxed);
    return TWELL_OK;
}

}  // namespace twell_host
