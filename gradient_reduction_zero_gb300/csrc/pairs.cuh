// Two floats in one register pair, for the paired fp32 operations (sm_100 and later): each
// half is rounded as the single operation rounds it, and one instruction is issued
// instead of two.
#pragma once

#include <cstdint>

namespace dpz {

using F2 = uint64_t;
__device__ __forceinline__ F2 pack2(float lo, float hi)
{
    F2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float lo2(F2 a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float hi2(F2 a) { return __uint_as_float((uint32_t)(a >> 32)); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ F2 swap2(F2 a) { return a << 32 | a >> 32; }

}  // namespace dpz
