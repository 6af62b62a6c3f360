// csa2_device.cuh -- device helpers shared by the CSA2 kernels (sm_103a):
// mbarrier, TMA and tcgen05 wrappers in inline PTX, bounded waits, number
// formats.  Host code never includes this file.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "csa2.h"

namespace csa2 {

// ------------------------------------------------------------------ basics
__device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void count_event(uint32_t *counters, int slot, uint32_t n = 1)
{
    if (counters != nullptr && n != 0) atomicAdd(counters + slot, n);
}

// Order-preserving map fp32 -> uint32 (larger float -> larger key); -0 and +0
// map to the same key. A NaN with a clear sign bit lies above +infinity (the eviction
// marks what stays in any case by one).
__device__ __forceinline__ uint32_t score_key(float f)
{
    // (-0 + 0 is +0; the rest by bits: with comparisons of floats a NaN lay elsewhere, and
    // 128 x 262,144 scores took 61.1 us instead of 46.8)
    const uint32_t b = __float_as_uint(__fadd_rn(f, 0.0f));
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// ------------------------------------------------------------------ mbarrier
// Waits give up after kWaitNs nanoseconds of wall time (read from %globaltimer)
// or kSpinLimit polls, whichever comes first, so a broken pipeline returns
// with an error count instead of hanging the GPU.
constexpr uint32_t kSpinLimit = 1u << 24;
constexpr uint64_t kWaitNs = 2000000000ull;   // 2 s

__device__ __forceinline__ uint64_t global_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
}

__device__ __forceinline__ void fence_barrier_init()
{
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(
                     smem_u32(bar)),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// The same with a suspend-time hint: the thread may sleep up to `ns`
// nanoseconds (or until the phase completes) instead of returning at once, so
// that a waiting warp takes fewer issue slots from the warps that are working.
__device__ __forceinline__ bool mbar_try_wait_sleep(uint64_t *bar, uint32_t parity, uint32_t ns)
{
    uint32_t ok;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(ns)
        : "memory");
    return ok != 0;
}

constexpr uint32_t kSleepHintNs = 20000;   // 64 polls: at most ~1.3 ms between limit checks

// Returns false when the wait gave up (time or poll limit reached, or *abort set).
// kSleep: poll with the suspend-time hint.
template <bool kSleep = false>
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity,
                                          volatile int *abort_flag)
{
    auto poll = [&]() {
        return kSleep ? mbar_try_wait_sleep(bar, parity, kSleepHintNs) : mbar_try_wait(bar, parity);
    };
    if (poll()) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 1; i < kSpinLimit; ++i) {
        if (poll()) return true;
        if ((i & 63u) == 0u) {
            if (*abort_flag) return false;
            if (global_ns() - t0 > kWaitNs) return false;
        }
    }
    return false;
}

// ------------------------------------------------------------------ TMA / bulk copies
__device__ __forceinline__ void tma_load_2d(void *smem_dst, const void *tmap, int32_t x,
                                            int32_t y, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// L2 policy for data read once (a streamed key cache): its lines are the first
// to be evicted, so that what is written meanwhile (scores) stays in L2.
__device__ __forceinline__ uint64_t l2_evict_first_policy()
{
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

// tma_load_2d with an L2 cache policy
__device__ __forceinline__ void tma_load_2d_hint(void *smem_dst, const void *tmap, int32_t x,
                                                 int32_t y, uint64_t *bar, uint64_t pol)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(smem_u32(bar)), "l"(pol)
        : "memory");
}

// bulk_load (below) with an L2 cache policy
__device__ __forceinline__ void bulk_load_hint(void *smem_dst, const void *gsrc, uint32_t bytes,
                                               uint64_t *bar, uint64_t pol)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(smem_dst)),
        "l"(gsrc), "r"(bytes), "r"(smem_u32(bar)), "l"(pol)
        : "memory");
}

// Plain bulk copy global -> shared (16-byte aligned addresses, size % 16 == 0).
__device__ __forceinline__ void bulk_load(void *smem_dst, const void *gsrc, uint32_t bytes,
                                          uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(smem_u32(smem_dst)),
        "l"(gsrc), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// Programmatic dependent launch.  Every kernel of the library is launched so
// that it may start while the previous kernel of the stream is finishing; it
// calls pdl_wait() before its first access to global memory that an earlier
// kernel may write (the wait returns once every earlier kernel has completed
// and its writes are visible), and pdl_trigger() right after, which lets the
// next kernel be scheduled as this one's CTAs retire.  Only set-up that reads
// no such memory (barrier init, TMEM allocation, descriptor prefetch) runs
// before the wait.
__device__ __forceinline__ void pdl_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void pdl_trigger()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void prefetch_tmap(const void *tmap)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tmap)) : "memory");
}

// ------------------------------------------------------------------ tcgen05
// Shared-memory matrix descriptor (tcgen05 form): start address, leading and
// stride byte offsets (all >> 4), version bit 46 = 1, layout type in 61..63.
enum : uint32_t { kLayoutNone = 0, kLayoutSW128 = 2, kLayoutSW64 = 4, kLayoutSW32 = 6 };

__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo_bytes,
                                              uint32_t sbo_bytes, uint32_t layout)
{
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)((lbo_bytes >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)((sbo_bytes >> 4) & 0x3FFFu) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)(layout & 7u) << 61;
    return d;
}

// Instruction descriptor for kind::f16 / kind::f8f6f4 with fp32 accumulate.
// a_fmt/b_fmt: kind::f16 -> 0 f16, 1 bf16; kind::f8f6f4 -> 0 e4m3.
// a_mn/b_mn: 0 = K-major, 1 = MN-major.
__host__ __device__ constexpr uint32_t instr_desc(uint32_t M, uint32_t N, uint32_t a_fmt,
                                                  uint32_t b_fmt, uint32_t a_mn, uint32_t b_mn)
{
    return (1u << 4) | (a_fmt << 7) | (b_fmt << 10) | (a_mn << 15) | (b_mn << 16) |
           ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ void tmem_alloc(uint32_t *smem_result, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(smem_result)),
                 "r"(ncols)
                 : "memory");
}

__device__ __forceinline__ void tmem_relinquish()
{
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void mma_f8f6f4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrives on `bar` once every earlier tcgen05.mma of this thread completed.
__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// 32 lanes x 32 bit, 16 consecutive columns per thread.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32])
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// c + a * b on two fp32 lanes at once (one packed f32x2 FMA, round to nearest)
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c)
{
    uint64_t d;
    asm("{\n"
        ".reg .b64 ra, rb, rc;\n"
        "mov.b64 ra, {%1, %2};\n"
        "mov.b64 rb, {%3, %4};\n"
        "mov.b64 rc, {%5, %6};\n"
        "fma.rn.f32x2 %0, ra, rb, rc;\n"
        "}\n"
        : "=l"(d)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return make_float2(__uint_as_float((uint32_t)d), __uint_as_float((uint32_t)(d >> 32)));
}

// ------------------------------------------------------------------ formats
// Value of a positive E4M3 byte b in 1..126 (exact in fp32).
__device__ __forceinline__ float e4m3_pos_value(uint32_t b)
{
    uint32_t e = b >> 3, mt = b & 7u;
    if (e == 0) return (float)mt * 0x1p-9f;
    return __uint_as_float(((e + 120u) << 23) | (mt << 20));
}

// Power-of-two FP8 scale of a vector: smallest 2^e with 448 * 2^e >= amax
// (amax > 0, normal fp32).  448 = 1.75 * 2^8.
__device__ __forceinline__ float fp8_pow2_scale(float amax)
{
    if (!(amax > 0.0f)) return 1.0f;
    uint32_t bits = __float_as_uint(amax);
    int ea = (int)((bits >> 23) & 0xFF) - 127;
    uint32_t mant = bits & 0x7FFFFFu;          // 1.75 -> 0x600000
    int e = (mant <= 0x600000u) ? ea - 8 : ea - 7;
    if (e < -126) e = -126;                    // subnormal amax: out of contract
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// E4M3 byte of y (|y| <= 448), round to nearest even, zero -> 0x00.
__device__ __forceinline__ uint32_t e4m3_byte(float y)
{
    uint32_t b = (uint32_t)__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
    return ((b & 0x7Fu) == 0) ? 0u : b;
}

// Smallest positive E4M3 byte b with 6 * value(b) >= amax (amax > 0); 0x7E and
// *sat when even 6 * 448 is too small.
__device__ __forceinline__ uint32_t fp4_scale_byte(float amax, bool *sat)
{
    if (6.0f * 448.0f < amax) { *sat = true; return 0x7Eu; }
    uint32_t lo = 0, hi = 0x7E;       // value(hi) * 6 >= amax, value(lo) * 6 < amax (lo = 0 -> 0)
    while (hi - lo > 1) {
        uint32_t mid = (lo + hi) >> 1;
        if (6.0f * e4m3_pos_value(mid) >= amax) hi = mid; else lo = mid;
    }
    return hi;
}

// E2M1 code of x under scale s: round to nearest, ties to the even code.
// Midpoints between magnitudes {0, .5, 1, 1.5, 2, 3, 4, 6} are {.25, .75,
// 1.25, 1.75, 2.5, 3.5, 5}; at a tie with midpoint k the result goes up when
// code k + 1 is even (k odd).  Every m_k * s is exact in fp32.
__device__ __forceinline__ uint32_t fp4_code(float x, float s)
{
    float a = fabsf(x);
    uint32_t c = 0;
    c += (a > 0.25f * s);
    c += (a >= 0.75f * s);
    c += (a > 1.25f * s);
    c += (a >= 1.75f * s);
    c += (a > 2.5f * s);
    c += (a >= 3.5f * s);
    c += (a > 5.0f * s);
    if (c != 0 && x < 0.0f) c |= 8u;
    return c;
}

// Value of E2M1 code `code` (sign bit 3) under scale s: magnitudes 0, 0.5, 1,
// 1.5, 2, 3, 4, 6 built as fp32 bit patterns (index i >= 2: exponent
// 126 + i / 2, mantissa bit i & 1; index 1: 0.5).
__device__ __forceinline__ float fp4_value(uint32_t code, float s)
{
    const uint32_t i = code & 7u;
    const uint32_t bits = (i >= 2u) ? (((126u + (i >> 1)) << 23) | ((i & 1u) << 22))
                                    : (i == 1u ? (126u << 23) : 0u);
    const float v = __uint_as_float(bits) * s;
    return (code & 8u) ? -v : v;
}

}  // namespace csa2
