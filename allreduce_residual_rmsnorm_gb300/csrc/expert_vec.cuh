// Element access shared by the expert-layer kernels: single elements, and
// vectors of 8 at 16-byte aligned addresses (fp32: two 128-bit accesses, so
// that 16 bytes of alignment are enough for every element type).
#pragma once

#include "ar_common.cuh"

namespace arf {

template <class D>
__device__ __forceinline__ float load1(const void* p, uint64_t i)
{
    if constexpr (D::bytes == 4)
        return static_cast<const float*>(p)[i];
    else if constexpr (D::id == AR_DT_BF16)
        return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    else
        return __half2float(static_cast<const __half*>(p)[i]);
}

// 8 consecutive elements as loaded, read once
template <class D>
__device__ __forceinline__ typename D::Vec load8_raw(const uint8_t* p)
{
    if constexpr (D::bytes == 4) {
        V32 v;
        v.lo = ld_stream(p);
        v.hi = ld_stream(p + 16);
        return v;
    } else {
        return ld_stream(p);
    }
}

template <class D>
__device__ __forceinline__ void store8(uint8_t* p, const float (&f)[8])
{
    const typename D::Vec v = pack8<D>(f);
    if constexpr (D::bytes == 4) {
        *reinterpret_cast<uint4*>(p) = v.lo;
        *reinterpret_cast<uint4*>(p + 16) = v.hi;
    } else {
        *reinterpret_cast<uint4*>(p) = v;
    }
}

// ----------------------------------------------------- packed fp32 pairs
//
// Two fp32 values in a 64-bit register; each half is rounded as by the scalar
// instruction.

__device__ __forceinline__ uint64_t pack_pair(uint32_t lo, uint32_t hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ uint64_t pair_of(float lo, float hi)
{
    return pack_pair(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float2 unpack_pair(uint64_t v)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma3_pair(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// acc = d * s + acc
__device__ __forceinline__ void fma_pair(uint64_t& acc, uint64_t d, uint64_t s)
{
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(d), "l"(s));
}

}  // namespace arf
