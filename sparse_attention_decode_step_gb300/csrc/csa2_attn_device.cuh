// csa2_attn_device.cuh -- device helpers shared by the attention kernels:
// FP4 and bf16 to f16, the 128-byte-swizzled tile layout, TMEM stores and warp
// reductions.
#pragma once
#include "csa2_device.cuh"

namespace csa2 {

__device__ __forceinline__ void fence_async_smem()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// 8 E2M1 codes (one 32-bit word, channel 2i in the low nibble of byte i) ->
// 4 x f16x2, multiplied by the f16x2 scale pair {s, s}.
__device__ __forceinline__ uint4 fp4x8_to_f16(uint32_t w, uint32_t s2)
{
    uint32_t o0, o1, o2, o3;
    asm("{\n"
        ".reg .b8 b0, b1, b2, b3;\n"
        "mov.b32 {b0, b1, b2, b3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n"
        "}\n"
        : "=r"(o0), "=r"(o1), "=r"(o2), "=r"(o3)
        : "r"(w));
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(o0) : "r"(s2));
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(o1) : "r"(s2));
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(o2) : "r"(s2));
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(o3) : "r"(s2));
    return make_uint4(o0, o1, o2, o3);
}

// two E4M3 bytes -> f16x2
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t bytes)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)bytes));
    return r;
}

// E4M3 scale byte -> f16x2 {s, s}
__device__ __forceinline__ uint32_t scale_pair(uint32_t byte)
{
    uint32_t r;
    const uint16_t two = (uint16_t)(byte | (byte << 8));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(two));
    return r;
}

// two bf16 (one 32-bit word) -> f16x2
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w)
{
    const float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xFFFF0000u);
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// byte offset of the 16-byte chunk c (0..7) of row r inside a 128-byte-swizzled atom column
__device__ __forceinline__ uint32_t sw128(uint32_t r, uint32_t c)
{
    return r * 128u + ((c ^ (r & 7u)) << 4);
}

__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 2^x (hardware approximation, relative error near 2^-22; 2^-inf = 0)
__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16])
{
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

// Transposed warp reduction of 16 values per lane: afterwards lanes l and
// l + 16 hold, in v[0], the reduction over all 32 lanes of value l & 15.
template <bool kMax>
__device__ __forceinline__ void warp_reduce16(float (&v)[16], int lane)
{
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float recv = __shfl_xor_sync(0xffffffffu, v[i], 16);
        v[i] = kMax ? fmaxf(v[i], recv) : v[i] + recv;
    }
#pragma unroll
    for (int n = 16, o = 8; n > 1; n >>= 1, o >>= 1) {
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float send = upper ? v[i] : v[i + n / 2];
            const float keep = upper ? v[i + n / 2] : v[i];
            const float recv = __shfl_xor_sync(0xffffffffu, send, o);
            v[i] = kMax ? fmaxf(keep, recv) : keep + recv;
        }
    }
}

// 4 x 4 transpose within each group of 4 lanes: lane 4g + j holds a[i] =
// element (row j, column i) before and element (row i, column j) after.
__device__ __forceinline__ void transpose4(float (&a)[4], int lane)
{
    const bool b0 = (lane & 1) != 0, b1 = (lane & 2) != 0;
    float x0 = b0 ? a[0] : a[1], x1 = b0 ? a[2] : a[3];
    float r0 = __shfl_xor_sync(0xffffffffu, x0, 1), r1 = __shfl_xor_sync(0xffffffffu, x1, 1);
    if (b0) { a[0] = r0; a[2] = r1; } else { a[1] = r0; a[3] = r1; }
    x0 = b1 ? a[0] : a[2];
    x1 = b1 ? a[1] : a[3];
    r0 = __shfl_xor_sync(0xffffffffu, x0, 2);
    r1 = __shfl_xor_sync(0xffffffffu, x1, 2);
    if (b1) { a[0] = r0; a[1] = r1; } else { a[2] = r0; a[3] = r1; }
}

}  // namespace csa2
