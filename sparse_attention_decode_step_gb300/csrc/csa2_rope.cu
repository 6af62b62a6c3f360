// csa2_rope.cu -- RMS norm of 512-wide rows and the rotation of their last channels
// by the position of their token, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * weight;  pairs (u, v) of the last rot channels:
//   (u cos a - v sin a, u sin a + v cos a),  a = pos * inv_freq[p].
//
// Bound by memory traffic: a row is read and written once, 2 KB in bf16.  A warp
// takes a whole row, so that the sum of squares is five shuffles and nothing leaves
// the registers in between; a lane holds channels 8 lane .. and 256 + 8 lane .., 16
// bytes each in 16-bit types, so that loads and stores are whole lines.
//
// The heads of a token turn by the same angles: a warp works on several heads of a
// token in a row and finds the cosines once, lane by lane, into its own part of shared
// memory.  The angle is kept in turns: inv_freq / 2 pi as 64-bit fixed point (made
// once per block in fp64), times pos mod 2^64, is the fraction of a turn exactly,
// however far the position; the top 32 bits of it are half-turns for sincospif.
#include <cuda_fp16.h>

#include <algorithm>

#include "csa2_attn_device.cuh"
#include "csa2_internal.h"

namespace csa2 {

namespace {

constexpr int kWarps = 8;
constexpr int kResident = 3;                  // blocks to an SM, of 80 registers (4, of 64 and spills: 93.1 us where 3 took 92.4)

// Rows of x on their way to a warp, each in a slot of shared memory.  A lane copies the
// 16 bytes 512 i + 16 lane of a row, so that a copy is of whole lines; of 16-bit types these
// are its own channels, so that no other thread is waited for.
// (4,096 x 64 bf16 rows: 115 us with one row ahead in registers, 104 with three here;
// 90 now, 88 % of the measured copy.)
template <typename T>
constexpr int kSlots = sizeof(T) == 2 ? 4 : 2;

template <typename T>
constexpr uint32_t kPieces = 2 * sizeof(T) / 2;             // of a lane: 16 bytes of 16-bit types are eight channels

template <typename T>
__device__ __forceinline__ void copy_row(uint32_t slot, const T *src, int lane, bool in)
{
    if (in) {
#pragma unroll
        for (int i = 0; i < (int)kPieces<T>; ++i) {
            const T *const from = src + (32 * i + lane) * (16 / (int)sizeof(T));
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + 512 * i + 16 * lane), "l"(from) : "memory");
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <typename T>
__device__ __forceinline__ void read_row(uint32_t slot, int lane, float (&x)[16])
{
#pragma unroll
    for (int i = 0; i < (int)kPieces<T>; ++i) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(sizeof(T) == 2 ? slot + 512 * i + 16 * lane : slot + 1024 * (i >> 1) + 32 * lane + 16 * (i & 1))
                     : "memory");
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (__is_same(T, float)) {
                x[4 * i + k] = __uint_as_float(w[k]);
            } else if constexpr (__is_same(T, __half)) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
                x[8 * i + 2 * k] = f.x; x[8 * i + 2 * k + 1] = f.y;
            } else {
                x[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
                x[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *dst, const float *x)
{
    if constexpr (__is_same(T, float)) {
        reinterpret_cast<float4 *>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (__is_same(T, __half)) w[i] = f32x2_to_f16x2(x[2 * i], x[2 * i + 1]);
            else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        }
        *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// `per` heads of a token to a warp, `parts` warps to a token.
template <typename T, typename O, bool kWeight>
__global__ void __launch_bounds__(32 * kWarps, kResident) norm_rope_kernel(RopeParams p, uint32_t per, uint32_t parts)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pairs = p.rot / 2;
    extern __shared__ __align__(16) uint8_t smem[];
    const uint32_t slots = smem_u32(smem) + warp * (kSlots<T> * CSA2_D * (uint32_t)sizeof(T));       // [slots][row]
    uint64_t *const sTurn = reinterpret_cast<uint64_t *>(smem + kWarps * kSlots<T> * CSA2_D * sizeof(T));
    float4 *const sCs = reinterpret_cast<float4 *>(sTurn + pairs) + warp * (pairs / 2);           // (cos, sin) of two pairs
    float4 *const sY = reinterpret_cast<float4 *>(sTurn + pairs) + (kWarps + warp) * (pairs / 2); // the rotated part of a row (halves)
    pdl_wait();
    if ((int)threadIdx.x < pairs) {
        // f / 2 pi in two parts, of which only the fraction of a turn counts
        const double f = p.inv_freq[threadIdx.x];
        const double hi = f * 0.15915494309189535, lo = fma(f, 0.15915494309189535, -hi) + f * -9.839338337591243e-18;
        const double frac = hi - floor(hi);
        sTurn[threadIdx.x] = (uint64_t)(frac * 0x1p64) + (uint64_t)(int64_t)(lo * 0x1p64);
    }
    float w[kWeight ? 16 : 1];
    if constexpr (kWeight) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = *reinterpret_cast<const float4 *>(p.weight + 256 * (i >> 1) + 8 * lane + 4 * (i & 1));
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
    }
    __syncthreads();
    // where a lane's two groups of eight channels lie in the rotated part (negative: before it)
    const int at[2] = {8 * lane - (CSA2_D - p.rot), 256 + 8 * lane - (CSA2_D - p.rot)};
    const T *const x = static_cast<const T *>(p.x);
    O *const out = static_cast<O *>(p.out);
    const uint32_t units = p.n * parts, step = gridDim.x * kWarps;
    // a warp's rows in order
    struct Place {
        uint32_t u, token, head, left;
        __device__ __forceinline__ void start(uint32_t at, uint32_t per, uint32_t parts, uint32_t H)
        {
            u = at;
            token = u / parts;
            head = (u - token * parts) * per;
            left = min(per, H - head);
        }
        __device__ __forceinline__ bool next(uint32_t step, uint32_t per, uint32_t parts, uint32_t H)      // true: another unit
        {
            if (--left > 0) { ++head; return false; }
            start(u + step, per, parts, H);
            return true;
        }
    };
    Place now, ahead;
    now.start(blockIdx.x * kWarps + warp, per, parts, p.H);
    ahead = now;
    auto load = [&](uint32_t slot) {
        copy_row(slots + slot * (uint32_t)(CSA2_D * sizeof(T)), x + (uint64_t)ahead.token * p.ld_x + ahead.head * CSA2_D, lane, ahead.u < units);
        if (ahead.u < units) ahead.next(step, per, parts, p.H);
    };
#pragma unroll
    for (int i = 0; i < kSlots<T> - 1; ++i) load(i);
    bool turn = true;                                    // a new token's angles are due
    for (uint32_t slot = 0; now.u < units; slot = (slot + 1) % kSlots<T>) {
        load((slot + kSlots<T> - 1) % kSlots<T>);              // (the row before was read from there)
        asm volatile("cp.async.wait_group %0;" ::"n"(kSlots<T> - 1) : "memory");
        if constexpr (sizeof(T) == 4) __syncwarp();      // (the row before is read: its sum came from every lane)
        float v[16];
        read_row<T>(slots + slot * (uint32_t)(CSA2_D * sizeof(T)), lane, v);
        O *const dst = out + (uint64_t)now.token * p.ld_out + now.head * CSA2_D + 8 * lane;
        const bool due = turn;
        const uint32_t token = now.token;
        turn = now.next(step, per, parts, p.H);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum = fmaf(v[i], v[i], sum);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float r = rsqrtf(fmaf(sum, 1.0f / CSA2_D, p.eps));
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= kWeight ? r * w[kWeight ? i : 0] : r;
        if (pairs > 0) {
            if (due) {
                const int64_t pos = p.pos[token];
                __syncwarp();                            // (the last token's are read)
                for (int i = lane; i < pairs; i += 32) {
                    float s, c;
                    sincospif((float)(int32_t)(((uint64_t)pos * sTurn[i]) >> 32) * 0x1p-31f, &s, &c);
                    reinterpret_cast<float2 *>(sCs)[i] = make_float2(c, s);
                }
                __syncwarp();
            }
            if (!p.halves) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (at[h] >= 0) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float4 cs = sCs[at[h] / 4 + i];
                            float *const y = v + 8 * h + 4 * i;
                            const float a = y[0], b = y[1], c = y[2], d = y[3];
                            y[0] = a * cs.x - b * cs.y; y[1] = a * cs.y + b * cs.x;
                            y[2] = c * cs.z - d * cs.w; y[3] = c * cs.w + d * cs.z;
                        }
                    }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (at[h] >= 0) {
                        sY[at[h] / 4] = make_float4(v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3]);
                        sY[at[h] / 4 + 1] = make_float4(v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]);
                    }
                __syncwarp();
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (at[h] >= 0) {
                        const bool second = at[h] >= pairs;          // (a group lies in one half: pairs is a multiple of 8)
                        const int pair = at[h] - (second ? pairs : 0), other = pair + (second ? 0 : pairs);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float4 o = sY[other / 4 + i];
                            const float4 c0 = sCs[pair / 2 + 2 * i], c1 = sCs[pair / 2 + 2 * i + 1];
                            const float oo[4] = {o.x, o.y, o.z, o.w}, c[4] = {c0.x, c0.z, c1.x, c1.z}, s[4] = {c0.y, c0.w, c1.y, c1.w};
                            float *const y = v + 8 * h + 4 * i;
#pragma unroll
                            for (int k = 0; k < 4; ++k) y[k] = y[k] * c[k] + (second ? oo[k] : -oo[k]) * s[k];
                        }
                    }
                __syncwarp();                            // (the next row's part goes there)
            }
        }
        store8(dst, v);
        store8(dst + 256, v + 8);
    }
}

}  // namespace

template <typename T, typename O, bool kWeight>
static cudaError_t launch_rope_as(const RopeParams &p, cudaStream_t st)
{
    // as many heads (a power of two) to a unit as leave each warp of a full GPU four units or
    // more (eight: 92.4 us instead of 90.2 for 4,096 x 64 rows, more cosines; a share of all
    // rows each, which need not divide evenly: 104).  Below some 58,000 rows that is one or two, and
    // the angles of a token are made by every warp that has a head of it: 500 x 64 rows 11.5 us,
    // 9.6 by their bytes; 160 x 64 5.7 us, 3.1 by theirs.
    const uint64_t rows = (uint64_t)p.n * p.H, warps = (uint64_t)device_sm_count() * kResident * kWarps;
    uint32_t per = 1;
    while (2 * per <= p.H && 2 * per * 4 * warps <= rows) per *= 2;
    const uint32_t parts = (p.H + per - 1) / per;
    const uint64_t blocks = ((uint64_t)p.n * parts + kWarps - 1) / kWarps;
    // slots, turns, and for each warp (cos, sin) and, for halves, a row's rotated part
    const size_t smem = kWarps * kSlots<T> * CSA2_D * sizeof(T) + (size_t)p.rot / 2 * 8 + (size_t)kWarps * p.rot * 4 * (p.halves ? 2 : 1);
    cudaError_t e = cudaSuccess;
    if (smem > 48 * 1024) e = cudaFuncSetAttribute(norm_rope_kernel<T, O, kWeight>, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024);
    if (e == cudaSuccess)
        e = launch_k(norm_rope_kernel<T, O, kWeight>, dim3((unsigned)std::min<uint64_t>(blocks, warps / kWarps)), dim3(32 * kWarps), smem, st, 0, p, per, parts);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_norm_rope(const RopeParams &p, int type, int out_type, cudaStream_t st)
{
    auto as = [&](auto from, auto to) {
        using T = decltype(from);
        using O = decltype(to);
        return p.weight != nullptr ? launch_rope_as<T, O, true>(p, st) : launch_rope_as<T, O, false>(p, st);
    };
    auto to = [&](auto from) {
        return out_type == CSA2_F32 ? as(from, float{}) : out_type == CSA2_BF16 ? as(from, __nv_bfloat16{}) : as(from, __half{});
    };
    return type == CSA2_F32 ? to(float{}) : type == CSA2_BF16 ? to(__nv_bfloat16{}) : to(__half{});
}

}  // namespace csa2
