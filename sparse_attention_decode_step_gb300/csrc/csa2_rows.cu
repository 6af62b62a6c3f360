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
// cache.  One warp per row.
#include <cuda_fp16.h>

#include "csa2_attn_device.cuh"
#include "csa2_internal.h"

namespace csa2 {

// 16 consecutive elements of a row as fp32 (src 16-byte aligned)
template <typename T>
__device__ __forceinline__ void load16(const T *src, float (&x)[16])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(src) + i);
            x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src) + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 f;
                if constexpr (sizeof(T) == 2 && __is_same(T, __half))
                    f = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
                else
                    f = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
                x[8 * i + 2 * j] = f.x;
                x[8 * i + 2 * j + 1] = f.y;
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ float as_float(T v)
{
    if constexpr (__is_same(T, float)) return v;
    else if constexpr (__is_same(T, __half)) return __half2float(v);
    else return __bfloat162float(v);
}

template <typename T>
__global__ void __launch_bounds__(256) cache_write_kernel(csa2_cache cache, const int64_t *__restrict__ rows,
                                                          int64_t n, const T *__restrict__ x, int64_t ld_x,
                                                          const T *__restrict__ key, int64_t ld_key,
                                                          uint32_t *counters)
{
    pdl_wait();
    pdl_trigger();
    const int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (i >= n) return;
    const int64_t row = rows[i];
    if (row < 0) return;                          // padding
    if (row >= cache.cap) {
        if (lane == 0) count_event(counters, CSA2_CNT_BAD_INPUT);
        return;
    }
    float v[16];
    load16(x + i * ld_x + 16 * lane, v);
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < 16; ++c) amax = fmaxf(amax, fabsf(v[c]));
    uint32_t sb = 0, packed[2] = {0u, 0u};
    if (amax > 0.f) {
        bool sat = false;
        sb = fp4_scale_byte(amax, &sat);
        if (sat) count_event(counters, CSA2_CNT_FP4_SATURATED);
        const float s = e4m3_pos_value(sb);
#pragma unroll
        for (int c = 0; c < 16; ++c) packed[c >> 3] |= fp4_code(v[c], s) << (4 * (c & 7));
    }
    *reinterpret_cast<uint2 *>(cache.codes + row * CSA2_CODE_BYTES + lane * 8) =
        make_uint2(packed[0], packed[1]);
    cache.scales[row * CSA2_SCALE_BYTES + lane] = (uint8_t)sb;
    if (key == nullptr) return;
    const T *kr = key + i * ld_key;
    const int per = cache.d_idx / 32;             // 2 or 4 components per lane
    float k[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (c < per) k[c] = as_float(kr[per * lane + c]);
    float a = fmaxf(fmaxf(fabsf(k[0]), fabsf(k[1])), fmaxf(fabsf(k[2]), fabsf(k[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    const float s = fp8_pow2_scale(a);
    const uint32_t w = e4m3_byte(k[0] / s) | (e4m3_byte(k[1] / s) << 8) | (e4m3_byte(k[2] / s) << 16) |
                       (e4m3_byte(k[3] / s) << 24);
    if (per == 4)
        *reinterpret_cast<uint32_t *>(cache.kidx + row * 128 + lane * 4) = w;
    else
        *reinterpret_cast<uint16_t *>(cache.kidx + row * 64 + lane * 2) = (uint16_t)w;
    if (lane == 0) cache.kscale[row] = s;
}

// 8 values (4 x f16x2, exact) stored as T, 16-byte aligned
template <typename T>
__device__ __forceinline__ void store8(T *dst, uint4 h)
{
    if constexpr (__is_same(T, __half)) {
        *reinterpret_cast<uint4 *>(dst) = h;
    } else {
        const uint32_t w[4] = {h.x, h.y, h.z, h.w};
        float2 f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
        if constexpr (__is_same(T, float)) {
            reinterpret_cast<float4 *>(dst)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
            reinterpret_cast<float4 *>(dst)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
        } else {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[j]) : "f"(f[j].y), "f"(f[j].x));
            *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// Lane l takes channels 8 l .. 8 l + 7 and 256 + 8 l ..: a warp reads 128
// contiguous code bytes and writes 32 contiguous 16-byte words at a time.
template <typename T>
__global__ void __launch_bounds__(256) cache_read_kernel(csa2_cache cache, const int64_t *__restrict__ rows,
                                                         int64_t n, T *__restrict__ x, int64_t ld_x,
                                                         float *__restrict__ key, int64_t ld_key,
                                                         uint32_t *counters)
{
    pdl_wait();
    pdl_trigger();
    const int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (i >= n) return;
    const int64_t row = rows[i];
    if (row < 0) return;                          // padding
    if (row >= cache.cap) {
        if (lane == 0) count_event(counters, CSA2_CNT_BAD_INPUT);
        return;
    }
    uint32_t w[2], sc[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        w[h] = *reinterpret_cast<const uint32_t *>(cache.codes + row * CSA2_CODE_BYTES + 128 * h + 4 * lane);
        sc[h] = cache.scales[row * CSA2_SCALE_BYTES + 16 * h + (lane >> 1)];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        store8(x + i * ld_x + 256 * h + 8 * lane, fp4x8_to_f16(w[h], scale_pair(sc[h])));
    if (key == nullptr) return;
    const float s = cache.kscale[row];
    const int per = cache.d_idx / 32;
    const uint32_t b = per == 4 ? *reinterpret_cast<const uint32_t *>(cache.kidx + row * 128 + 4 * lane)
                                : *reinterpret_cast<const uint16_t *>(cache.kidx + row * 64 + 2 * lane);
    const uint32_t lo = e4m3x2_to_f16x2(b & 0xFFFFu), hi = e4m3x2_to_f16x2(b >> 16);
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    float *dst = key + i * ld_key + per * lane;
    if (per == 4)
        *reinterpret_cast<float4 *>(dst) = make_float4(f0.x * s, f0.y * s, f1.x * s, f1.y * s);
    else
        *reinterpret_cast<float2 *>(dst) = make_float2(f0.x * s, f0.y * s);
}

constexpr int kRowThreads = 256;

static unsigned row_blocks(int64_t n) { return (unsigned)((n + kRowThreads / 32 - 1) / (kRowThreads / 32)); }

cudaError_t launch_cache_write(const csa2_cache &c, const int64_t *rows, int64_t n, const void *x, int x_type,
                               int64_t ld_x, const void *key, int64_t ld_key, uint32_t *counters,
                               cudaStream_t st)
{
    auto go = [&](auto tag) {
        using T = decltype(tag);
        return launch_k(cache_write_kernel<T>, dim3(row_blocks(n)), dim3(kRowThreads), 0, st, 0, c, rows, n,
                        static_cast<const T *>(x), ld_x, static_cast<const T *>(key), ld_key, counters);
    };
    const cudaError_t e = x_type == CSA2_F32 ? go(float{}) : x_type == CSA2_BF16 ? go(__nv_bfloat16{}) : go(__half{});
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_cache_read(const csa2_cache &c, const int64_t *rows, int64_t n, void *x, int x_type, int64_t ld_x,
                              float *key, int64_t ld_key, uint32_t *counters, cudaStream_t st)
{
    auto go = [&](auto tag) {
        using T = decltype(tag);
        return launch_k(cache_read_kernel<T>, dim3(row_blocks(n)), dim3(kRowThreads), 0, st, 0, c, rows, n,
                        static_cast<T *>(x), ld_x, key, ld_key, counters);
    };
    const cudaError_t e = x_type == CSA2_F32 ? go(float{}) : x_type == CSA2_BF16 ? go(__nv_bfloat16{}) : go(__half{});
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa2
