// csa2_rows.cu -- cache rows by number: latents (and indexer keys) quantised
// into given rows, and rows read back as the values they hold.
//
// Write, per row: 16 channels at a time, scale s = the smallest E4M3 with
// 6 s >= max |x|, codes = the nearest of s {0, .5, 1, 1.5, 2, 3, 4, 6} (ties to
// the even code); key: s = the smallest 2^e with 448 2^e >= max |k|, bytes =
// E4M3(k / s).  The same encode as the append's.  Read: value = E2M1 code x
// E4M3 scale, at most 6 significant bits in [2^-10, 2688], so exact in fp32,
// bf16 and f16 alike; key = E4M3 byte x scale in fp32.
//
// Both are bound by memory traffic: a row is 1 KB of bf16 against 288 B of
// cache.  A warp takes a whole row.  A write's lane takes one 16-channel group, so that a
// scale is found once; a read's lane takes 16 bytes of every 512, so that a warp's
// stores are contiguous (fp32 rows with 32 bytes a lane: 65,536 in 33.0 us instead
// of 25.2).  With seven comparisons per value (the append's form) the write of bf16
// rows was bound by its instructions, at 50 us for 65,536 rows, and that of fp32
// rows at 38; see fp4_codes16.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "csa2_attn_device.cuh"
#include "csa2_internal.h"

namespace csa2 {

// A call has at most 2^31 rows of strides below 2^31: 32-bit counts, so that an
// address is one wide multiplication.
constexpr int kRowThreads = 256;

// kWords consecutive words (4 k of them 16-byte aligned, 2 or 1 aligned to their size)
template <int kWords>
__device__ __forceinline__ void load_words(const void *src, uint32_t (&w)[kWords])
{
    if constexpr (kWords >= 4) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 v = __ldg(static_cast<const uint4 *>(src) + i);
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
    } else if constexpr (kWords == 2) {
        const uint2 v = __ldg(static_cast<const uint2 *>(src));
        w[0] = v.x; w[1] = v.y;
    } else {
        w[0] = __ldg(static_cast<const uint32_t *>(src));
    }
}

// words of T elements as fp32
template <typename T, int kWords, int N>
__device__ __forceinline__ void words_as_f32(const uint32_t (&w)[kWords], float (&x)[N])
{
    static_assert(N * sizeof(T) == kWords * 4, "whole words");
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        if constexpr (__is_same(T, float)) {
            x[i] = __uint_as_float(w[i]);
        } else if constexpr (__is_same(T, __half)) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x; x[2 * i + 1] = f.y;
        } else {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

// two values to E4M3 bytes (the first in the low byte), nearest even, saturating
__device__ __forceinline__ uint32_t e4m3x2_near(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// fp4_scale_byte by the hardware's E4M3 rounding: the nearest E4M3 to amax / 6,
// or the next one up when that is too small (6 s is exact).
__device__ __forceinline__ uint32_t fp4_scale_near(float amax, float *s)
{
    uint32_t b = e4m3x2_near(amax * (1.0f / 6.0f), 0.f);
    auto value = [](uint32_t byte) {
        const uint32_t h = e4m3x2_to_f16x2(byte);
        return __half2float(*reinterpret_cast<const __half *>(&h));
    };
    *s = value(b);
    if (6.0f * *s < amax && b < 0x7Eu) *s = value(++b);
    return b;
}

// E2M1 codes (nearest even, saturating) of 8 values; one that rounds to zero has code 0
__device__ __forceinline__ uint32_t e2m1x8_near(const float (&q)[8])
{
    uint32_t w;
    asm("{\n"
        ".reg .b8 b0, b1, b2, b3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        "mov.b32 %0, {b0, b1, b2, b3};\n"
        "}\n"
        : "=r"(w)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    const uint32_t mag = w & 0x77777777u;
    return mag | (w & ((mag + 0x77777777u) & 0x88888888u));
}

// E2M1 codes of 16 values under scale s, two at a time.  With the hardware's
// reciprocal r of s (off by at most one step), x r is within 2^-23 (relative) of x / s.
//  * 16-bit x (kSplit false): x has at most 11 significant bits and a midpoint m s (m
//    of .25, .75, 1.25, 1.75, 2.5, 3.5, 5) at most 7, so x / s is either exactly m
//    or at least 2^-11 of itself away, which is 2^-14 or more.  768 + x r has steps
//    of 2^-14 (while |x r| < 256): rounded to them, x r becomes exactly m in the first
//    case and stays on its side in the second, and the hardware's
//    round-to-nearest-even then decides as the exact quotient would.
//  * fp32 x: x / s lies between x r (1 - 2^-20) and x r (1 + 2^-20); where both have
//    the same code it is that one's (rounding is monotonic), else (one value in
//    some 2^17) the values are compared with the midpoints, which are exact.
// (65,536 bf16 rows with keys: 19.2 us with three instructions a value, 18.0 so.)
template <bool kSplit>
__device__ __forceinline__ uint2 fp4_codes16(const float (&x)[16], float s)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float q[8];
        if constexpr (kSplit) {
            float t[8];
            const float2 lo = make_float2(r * (1.0f - 0x1p-20f), r * (1.0f - 0x1p-20f));
            const float2 hi = make_float2(r * (1.0f + 0x1p-20f), r * (1.0f + 0x1p-20f));
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 v = make_float2(x[8 * h + i], x[8 * h + i + 1]);
                const float2 a = fma_f32x2(v, lo, make_float2(0.f, 0.f)), b = fma_f32x2(v, hi, make_float2(0.f, 0.f));
                q[i] = a.x; q[i + 1] = a.y;
                t[i] = b.x; t[i + 1] = b.y;
            }
            w[h] = e2m1x8_near(q);
            if (w[h] != e2m1x8_near(t)) {
                w[h] = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) w[h] |= fp4_code(x[8 * h + i], s) << (4 * i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 v = make_float2(x[8 * h + i], x[8 * h + i + 1]);
                const float2 y = fma_f32x2(v, make_float2(r, r), make_float2(768.f, 768.f));
                const float2 a = fma_f32x2(y, make_float2(1.f, 1.f), make_float2(-768.f, -768.f));
                q[i] = a.x; q[i + 1] = a.y;
            }
            w[h] = e2m1x8_near(q);
        }
    }
    return make_uint2(w[0], w[1]);
}

// Neither kernel lets the next one in before its blocks end: a waiting block takes
// registers that a block of this kernel could have (5,003 bf16 rows written and
// read back: 6.0 us with an early trigger in both, 4.2 without).

// A warp goes from row to row, the next row's loads on their way while this one is
// encoded (65,536 bf16 rows with keys: 21.4 us with a row per warp, 19.2 so).  fp32 rows hold
// twice the words: four blocks to an SM with 64 registers a thread, not five with
// 48 and spills (65,536 rows 32.5 -> 24.2 us).
template <typename T>
constexpr int kWriteResident = sizeof(T) == 4 ? 4 : 5;

template <typename T>
__global__ void __launch_bounds__(kRowThreads, kWriteResident<T>) cache_write_kernel(csa2_cache cache, const int64_t *__restrict__ rows,
                                                          uint32_t n, const T *__restrict__ x, uint32_t ld_x,
                                                          const T *__restrict__ key, uint32_t ld_key,
                                                          uint32_t *counters)
{
    pdl_wait();
    constexpr int kX = 16 * sizeof(T) / 4, kK = sizeof(T);          // words of a lane's latents, of up to 4 key components
    const uint32_t step = gridDim.x * (kRowThreads / 32);
    const int lane = threadIdx.x & 31;
    uint32_t next = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    uint32_t xw[kX], kw[kK] = {};
    int64_t next_row = -1;
    auto load = [&]() {
        next_row = __ldg(rows + next);
        load_words(x + (uint64_t)next * ld_x + 16 * lane, xw);
        if (key != nullptr) {
            if (cache.d_idx == 128) {
                load_words(key + (uint64_t)next * ld_key + 4 * lane, kw);
            } else {
                uint32_t half[kK / 2];
                load_words(key + (uint64_t)next * ld_key + 2 * lane, half);
#pragma unroll
                for (int c = 0; c < kK; ++c) kw[c] = c < kK / 2 ? half[c] : 0u;
            }
        }
    };
    if (next < n) load();
    while (next < n) {
        const int64_t row = next_row;
        float v[16], k[4];
        words_as_f32<T>(xw, v);
        words_as_f32<T>(kw, k);
        next += step;
        if (next < n) load();
        if (row < 0) continue;                    // padding
        if (row >= cache.cap) {
            if (lane == 0) count_event(counters, CSA2_CNT_BAD_INPUT);
            continue;
        }
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < 16; ++c) amax = fmaxf(amax, fabsf(v[c]));
        uint32_t sb = 0;
        uint2 codes = make_uint2(0u, 0u);
        if (amax > 0.f) {
            if (amax > 2688.f) count_event(counters, CSA2_CNT_FP4_SATURATED);
            float s;
            sb = fp4_scale_near(amax, &s);
            codes = fp4_codes16<sizeof(T) == 4>(v, s);
        }
        *reinterpret_cast<uint2 *>(cache.codes + row * CSA2_CODE_BYTES + 8 * lane) = codes;
        cache.scales[row * CSA2_SCALE_BYTES + lane] = (uint8_t)sb;
        if (key == nullptr) continue;
        float a = fmaxf(fmaxf(fabsf(k[0]), fabsf(k[1])), fmaxf(fabsf(k[2]), fabsf(k[3])));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        const float s = fp8_pow2_scale(a);
        // 1 / s by its exponent: s = 2^e with -126 <= e <= 120, so k / s is k times a power of two
        const float r = __uint_as_float((254u << 23) - __float_as_uint(s));
        uint32_t w = e4m3x2_near(k[0] * r, k[1] * r) | (e4m3x2_near(k[2] * r, k[3] * r) << 16);
        // a negative value that rounds to zero is byte 0
        const uint32_t mag = w & 0x7F7F7F7Fu;
        w = mag | (w & ((mag + 0x7F7F7F7Fu) & 0x80808080u));
        if (cache.d_idx == 128)
            *reinterpret_cast<uint32_t *>(cache.kidx + row * 128 + lane * 4) = w;
        else
            *reinterpret_cast<uint16_t *>(cache.kidx + row * 64 + lane * 2) = (uint16_t)w;
        if (lane == 0) cache.kscale[row] = s;
    }
}

// 16 bytes of T, 16-byte aligned, from f16 values (exact): 8 of them, or for fp32 the first 4
template <typename T>
__device__ __forceinline__ void store16(T *dst, uint4 h)
{
    if constexpr (__is_same(T, __half)) {
        __stcs(reinterpret_cast<uint4 *>(dst), h);
    } else {
        const uint32_t w[4] = {h.x, h.y, h.z, h.w};
        float2 f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
        if constexpr (__is_same(T, float)) {
            __stcs(reinterpret_cast<float4 *>(dst), make_float4(f[0].x, f[0].y, f[1].x, f[1].y));
        } else {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[j]) : "f"(f[j].y), "f"(f[j].x));
            __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
}

// A warp reads kReadRows rows, their loads all on the way before the first store
// (200,003 rows with keys: 64.6 us one row at a time, 61.0 two, 62 four; the
// stores are not read back soon and are marked so).
constexpr int kReadRows = 2;

template <typename T>
__global__ void __launch_bounds__(256) cache_read_kernel(csa2_cache cache, const int64_t *__restrict__ rows,
                                                         uint32_t n, T *__restrict__ x, uint32_t ld_x,
                                                         float *__restrict__ key, uint32_t ld_key,
                                                         uint32_t *counters)
{
    pdl_wait();
    const uint32_t i0 = (blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * kReadRows;
    const int lane = threadIdx.x & 31;
    const int per = cache.d_idx / 32;
    // part h of a row: 32 lanes' 16 bytes, channels kE (32 h + lane) ..
    constexpr int kE = 16 / sizeof(T), kParts = CSA2_D / (32 * kE);
    using Codes = std::conditional_t<kE == 8, uint32_t, uint16_t>;
    int64_t row[kReadRows];
    uint32_t w[kReadRows][kParts], sc[kReadRows][kParts], kb[kReadRows];
    float ks[kReadRows];
#pragma unroll
    for (int j = 0; j < kReadRows; ++j) row[j] = i0 + j < n ? __ldg(rows + i0 + j) : -1;
#pragma unroll
    for (int j = 0; j < kReadRows; ++j) {
        if (row[j] >= cache.cap) {
            if (lane == 0) count_event(counters, CSA2_CNT_BAD_INPUT);
            row[j] = -1;
        }
        if (row[j] >= 0) {
#pragma unroll
            for (int h = 0; h < kParts; ++h) {
                w[j][h] = __ldg(reinterpret_cast<const Codes *>(cache.codes + row[j] * CSA2_CODE_BYTES) + 32 * h + lane);
                sc[j][h] = __ldg(cache.scales + row[j] * CSA2_SCALE_BYTES + 2 * kE * h + lane * kE / 16);
            }
            if (key != nullptr) {
                ks[j] = __ldg(cache.kscale + row[j]);
                kb[j] = per == 4 ? __ldg(reinterpret_cast<const uint32_t *>(cache.kidx + row[j] * 128 + 4 * lane))
                                 : __ldg(reinterpret_cast<const uint16_t *>(cache.kidx + row[j] * 64 + 2 * lane));
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kReadRows; ++j) {
        if (row[j] < 0) continue;
        const uint32_t i = i0 + j;
#pragma unroll
        for (int h = 0; h < kParts; ++h)
            store16(x + (uint64_t)i * ld_x + kE * (32 * h + lane), fp4x8_to_f16(w[j][h], scale_pair(sc[j][h])));
        if (key == nullptr) continue;
        const uint32_t lo = e4m3x2_to_f16x2(kb[j] & 0xFFFFu), hi = e4m3x2_to_f16x2(kb[j] >> 16);
        const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
        const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
        float *dst = key + (uint64_t)i * ld_key + per * lane;
        const float s = ks[j];
        if (per == 4)
            __stcs(reinterpret_cast<float4 *>(dst), make_float4(f0.x * s, f0.y * s, f1.x * s, f1.y * s));
        else
            __stcs(reinterpret_cast<float2 *>(dst), make_float2(f0.x * s, f0.y * s));
    }
}

// blocks for n rows, `per` to a warp
static unsigned row_blocks(int64_t n, int per)
{
    const int64_t k = kRowThreads / 32 * per;
    return (unsigned)((n + k - 1) / k);
}

cudaError_t launch_cache_write(const csa2_cache &c, const int64_t *rows, int64_t n, const void *x, int x_type,
                               int64_t ld_x, const void *key, int64_t ld_key, uint32_t *counters,
                               cudaStream_t st)
{
    auto go = [&](auto tag) {
        using T = decltype(tag);
        // (twice the resident blocks: 65,536 bf16 rows with keys in 19.3 us, once: 19.7)
        const unsigned blocks = std::min(row_blocks(n, 1), (unsigned)(device_sm_count() * 2 * kWriteResident<T>));
        return launch_k(cache_write_kernel<T>, dim3(blocks), dim3(kRowThreads), 0, st, 0, c, rows, (uint32_t)n,
                        static_cast<const T *>(x), (uint32_t)ld_x, static_cast<const T *>(key), (uint32_t)ld_key,
                        counters);
    };
    const cudaError_t e = x_type == CSA2_F32 ? go(float{}) : x_type == CSA2_BF16 ? go(__nv_bfloat16{}) : go(__half{});
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_cache_read(const csa2_cache &c, const int64_t *rows, int64_t n, void *x, int x_type, int64_t ld_x,
                              float *key, int64_t ld_key, uint32_t *counters, cudaStream_t st)
{
    auto go = [&](auto tag) {
        using T = decltype(tag);
        return launch_k(cache_read_kernel<T>, dim3(row_blocks(n, kReadRows)), dim3(kRowThreads), 0, st, 0, c, rows, (uint32_t)n,
                        static_cast<T *>(x), (uint32_t)ld_x, key, (uint32_t)ld_key, counters);
    };
    const cudaError_t e = x_type == CSA2_F32 ? go(float{}) : x_type == CSA2_BF16 ? go(__nv_bfloat16{}) : go(__half{});
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa2
