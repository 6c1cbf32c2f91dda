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

}  // namespace arf
