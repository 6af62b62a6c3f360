// csa2_mass.cu -- attention weights by entry: how much weight the queries of a group
// gave to each entry of its sequence, from the log sums that the attention left.
//
//     mass[j] = decay prev[j] + sum over rows r (query, head) that see j of
//               2^(l2s q_r . v_j - lse2_r),   l2s = sm_scale log2 e, lse2 = lse log2 e.
//
// The sum is over rows, so entries lie along the tensor core's M: one CTA takes 128
// entries at a time against a block of up to 128 rows, 64 of them in one pass,
//     S [128 entries x 64 rows] = K [128 x 512] . Q^T          (M 128, N 16 .. 64)
// and a thread of the epilogue, which holds one entry's row of S in TMEM, sums over
// its columns alone: no value crosses threads.  The block's queries stay in shared
// memory (128 KB) while the entries go by.  Their codes and scales come by TMA, as they
// are stored (36 KB a tile); dequantised (E2M1 x E4M3 is exact in f16), they go straight
// to TMEM, from where the MMAs read them: through shared memory, writing and reading
// them would take 256 KB a tile and with the queries' reads more of its 128 bytes a
// cycle than there are (32 x 64 heads over 65,536 entries: 245 us so, 162 now; and an
// MMA of N = 64 takes 33 cycles with A in TMEM, 50 with both operands in shared memory).
//
// What bounds it: no unit.  A tile takes some 3,000 cycles, the tensor pipe 1,020 of them
// (2,040 for 128 rows), HBM 1,360 (621 MB in 162 us: 56 % of the measured copy).  The rest
// are waits, commits and hand-overs between loader, producers, issuer and epilogue: with the
// arithmetic of all of them taken out it was 144 us, with three quarters of the loads out as
// well 116.  TMEM holds one tile of K beside two buffers of S, so that what lies between a
// half's last MMA and its next first one is not hidden.
//
// S is summed in two parts of 256 channels, which the epilogue adds: the tensor core's
// additions to an fp32 sum are cut off, not rounded, each by up to 2^-23 of the sum so
// far, and with two sums half as large the loss is half.
//
// A weight is computed as r 2^(l2s x - m), with m = lse2 rounded to a whole number and
// r = 2^(m - lse2): the exponents that matter lie near zero then, and lse2's own
// rounding (2^-20 at 20) does not come in.  Sums are fp32.
//
// Groups of up to 64 rows write mass themselves.  The blocks of larger ones leave the
// sums of each 64 rows side by side in the workspace, which a second kernel adds in order: no atomics,
// results do not depend on the run.  A first kernel lays out the blocks; the work,
// counted in tiles of entries over all blocks, is divided into equal runs.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "csa2_attn_device.cuh"
#include "csa2_internal.h"

namespace csa2 {

namespace {

// Warp 0 issues the MMAs, warp 1 the loads (the first ones: of the warps that could issue, a
// scheduler seems to take the first, and these two hold up all others), 2 and 3 are
// idle, so that a warp's TMEM lanes go by its number mod 4.
constexpr int kWarpMma = 0, kWarpLoad = 1, kWarpEpi = 4, kWarpsEpi = 8, kWarpProd = 12, kWarpsProd = 8;
constexpr int kThreads = 32 * (kWarpProd + kWarpsProd);
constexpr int kRows = kMassRows, kEnt = kMassEntries;
constexpr uint32_t kPass = 64;                             // rows of a pass
constexpr int kUnits = 4, kScaleUnits = 3;            // codes: half tiles (256 channels), scales: tiles
constexpr uint32_t kUnit = kEnt * 128, kScaleUnit = kEnt * CSA2_SCALE_BYTES;
constexpr uint32_t kQBytes = kRows * CSA2_D * 2;      // [8 atoms of 64 channels][128 rows][128 B]
constexpr uint32_t kQAtom = kRows * 128;
constexpr uint32_t kColS = 256;                       // TMEM: K in columns 0 .. 255 (two halves), S from here
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPlanThreads = 1024;
constexpr int kFinishThreads = 256;

// A block of rows.
struct Block {
    int64_t first;       // tiles of the blocks before
    int seq;
    int n;               // entries that it adds to (all of the group's if it is alone)
    int row0, rows;      // (query, head) rows of q
    int k0;              // of the group: row0 is row k0 of its own
    int pos;             // token position of the group's first query
    int n_group;
    int base;            // cache row of entry 0 (without pages)
    int alone;           // the group's only block, of one pass: it writes mass itself
    int causal;
};

// The workspace: blocks (and one behind the last), each group's first block (and the
// total), owner of each sequence, parts.
struct Space {
    Block *blocks;
    int *group_first;
    int *owner;
    float *parts;
};

__host__ __device__ __forceinline__ Space space_of(const MassParams &p)
{
    Space s;
    s.blocks = reinterpret_cast<Block *>(p.ws);
    s.group_first = reinterpret_cast<int *>(p.ws + p.plan.off_groups);
    s.owner = s.group_first + p.ng + 1;
    s.parts = reinterpret_cast<float *>(p.ws + p.plan.off_parts);
    return s;
}

__device__ __forceinline__ int tiles_of(int n) { return n / kEnt + (n % kEnt != 0); }

// Entries that the k-th query of a group sees.
__device__ __forceinline__ int sees(const MassParams &p, bool causal, int pos, int n, int k)
{
    if (!causal) return n;
    const int64_t t = (int64_t)pos + k + 1;            // (under 2^32)
    return t <= 0 ? 0 : (int)min((uint32_t)t / (uint32_t)p.m, (uint32_t)n);
}

// ------------------------------------------------------------------ plan
// One CTA.  A group's blocks are its rows 0 .. 127, 128 .. 255 and so on (one without
// rows for a group without queries: its mass decays).
struct GroupArgs { int seq, n, a, e, base; bool bad; };

__device__ __forceinline__ GroupArgs args_of(const MassParams &p, int g)
{
    GroupArgs r{};
    r.seq = p.g_seq[g];
    r.a = p.g_off[g];
    r.e = p.g_off[g + 1];
    r.bad = r.seq < 0 || r.seq >= p.batch || r.a < 0 || r.e < r.a || r.e > p.nq;
    if (r.bad) return r;
    const int64_t len = p.seq_len[r.seq], n = p.g_len ? (int64_t)p.g_len[g] : len;
    r.bad = n < 0 || n > len || n > p.max_n;
    if (p.pages.table != nullptr) {
        r.bad = r.bad || n > p.pages.ld << p.pages.log;
    } else {
        const int64_t base = p.seq_base[r.seq];
        r.bad = r.bad || base < 0 || base + n > p.cap;
        r.base = (int)base;
    }
    r.n = (int)n;
    return r;
}

// Sum over the block's threads before this one, and over all.
__device__ __forceinline__ int64_t scan(int64_t v, int64_t *s_warp, int64_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t upto = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
    }
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int i = 0; i < kPlanThreads / 32; ++i) {
        if (i == warp) before = all;
        all += s_warp[i];
    }
    __syncthreads();
    *total = all;
    return before + upto - v;
}

// Block i of a group's.
__device__ __forceinline__ Block block_of(const MassParams &p, const GroupArgs &a, int pos, int blocks, int i)
{
    Block r{};
    r.seq = a.seq;
    r.n_group = a.n;
    r.base = a.base;
    r.alone = blocks == 1 && (a.e - a.a) * p.H <= (int)kPass;
    r.causal = p.pos != nullptr;
    r.pos = pos;
    r.k0 = i * kRows;
    r.rows = min(kRows, (a.e - a.a) * p.H - r.k0);
    r.row0 = a.a * p.H + r.k0;
    r.n = r.alone ? a.n : sees(p, r.causal, r.pos, a.n, (r.k0 + r.rows - 1) / p.H);
    return r;
}

__device__ __forceinline__ int blocks_of(const MassParams &p, const GroupArgs &a) { return max(1, ((a.e - a.a) * p.H + kRows - 1) / kRows); }

constexpr int kFewGroups = 128;

__global__ void __launch_bounds__(kPlanThreads) mass_plan_kernel(MassParams p)
{
    __shared__ int64_t s_warp[kPlanThreads / 32];
    __shared__ int s_fall;
    __shared__ GroupArgs s_args[kFewGroups];
    __shared__ int s_pos[kFewGroups], s_first[kFewGroups + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Space ws = space_of(p);
    pdl_wait();
    pdl_trigger();                             // (one block: those of the next kernel find room beside it)
    // ---- few groups of few blocks, as a decode step has: a thread to a group, then to a
    // block, every array read once (3 x 1 x 16 rows over 1,000 entries 10.7 us, by the general
    // way below 12.2)
    if (p.ng <= kFewGroups) {
        int mine = 0;
        if (tid == 0) s_fall = p.ng;
        __syncthreads();
        if (tid < p.ng) {
            if (p.pos) s_pos[tid] = p.pos[tid];
            else s_pos[tid] = 0;
            s_args[tid] = args_of(p, tid);
            if (s_args[tid].e < s_args[tid].a) atomicMin(&s_fall, tid);
        }
        __syncthreads();
        if (tid < p.ng) {
            bool bad = s_args[tid].bad || tid >= s_fall;
            for (int g = 0; g < tid && !bad; ++g) bad = s_args[g].seq == s_args[tid].seq && !s_args[g].bad;
            if (bad) count_event(p.counters, CSA2_CNT_BAD_INPUT);
            else mine = blocks_of(p, s_args[tid]);
        }
        int64_t blocks;
        const int64_t before = scan(mine, s_warp, &blocks);
        if (tid <= p.ng) s_first[tid] = ws.group_first[tid] = (int)before;       // (thread ng: all of them)
        __syncthreads();
        if (blocks <= kPlanThreads) {
            Block r{};
            if (tid < blocks) {
                int g = 0;                     // the group whose blocks tid is among: the last that begins at it or before
                for (int step = kFewGroups / 2; step > 0; step >>= 1)
                    if (g + step < p.ng && s_first[g + step] <= tid) g += step;
                r = block_of(p, s_args[g], s_pos[g], s_first[g + 1] - s_first[g], tid - s_first[g]);
            }
            int64_t tiles;
            r.first = scan(tid < blocks ? tiles_of(r.n) : 0, s_warp, &tiles);
            if (tid < blocks) ws.blocks[tid] = r;
            if (tid == 0) ws.blocks[blocks].first = tiles;
            return;
        }
    }
    // ---- any number
    if (tid == 0) s_fall = p.ng;
    for (int b = tid; b < p.batch; b += kPlanThreads) ws.owner[b] = p.ng;
    __syncthreads();
    for (int g = tid; g < p.ng; g += kPlanThreads)
        if (p.g_off[g + 1] < p.g_off[g]) atomicMin(&s_fall, g);
    __syncthreads();
    // (groups from the first whose offsets fall on may share queries with those before)
    const int fall = s_fall;
    for (int g = tid; g < fall; g += kPlanThreads) {
        const GroupArgs a = args_of(p, g);
        if (!a.bad) atomicMin(&ws.owner[a.seq], g);
    }
    __syncthreads();
    int64_t blocks = 0;
    for (int g0 = 0; g0 < p.ng; g0 += kPlanThreads) {
        const int g = g0 + tid;
        int mine = 0;
        if (g < p.ng) {
            const GroupArgs a = args_of(p, g);
            if (g < fall && !a.bad && ws.owner[a.seq] == g) mine = blocks_of(p, a);
            else if (p.ng > kFewGroups) count_event(p.counters, CSA2_CNT_BAD_INPUT);     // (few: counted above)
        }
        int64_t total;
        const int64_t before = scan(mine, s_warp, &total);
        if (g < p.ng) ws.group_first[g] = (int)(blocks + before);
        blocks += total;
    }
    if (tid == 0) ws.group_first[p.ng] = (int)blocks;
    __syncthreads();
    for (int g = warp; g < p.ng; g += kPlanThreads / 32) {
        const int b0 = ws.group_first[g], nb = ws.group_first[g + 1] - b0;
        if (nb == 0) continue;
        const GroupArgs a = args_of(p, g);
        const int pos = p.pos ? p.pos[g] : 0;
        for (int i = lane; i < nb; i += 32) ws.blocks[b0 + i] = block_of(p, a, pos, nb, i);
    }
    __syncthreads();
    int64_t tiles = 0;
    for (int64_t b0 = 0; b0 < blocks; b0 += kPlanThreads) {
        const int64_t b = b0 + tid;
        int64_t total;
        const int64_t before = scan(b < blocks ? tiles_of(ws.blocks[b].n) : 0, s_warp, &total);
        if (b < blocks) ws.blocks[b].first = tiles + before;
        tiles += total;
    }
    if (tid == 0) ws.blocks[blocks].first = tiles;
}

// ------------------------------------------------------------------ weights
// A CTA's pieces of work in order: tiles k0 .. k1 of a block.  (A role takes what it
// needs of the block into registers itself.)
struct Work {
    int b;
    int k0, k1;
    int64_t left;        // tiles after this piece

    __device__ __forceinline__ void take(const Space &ws, int at, int64_t tiles)
    {
        k0 = at;
        k1 = (int)min((int64_t)tiles_of(ws.blocks[b].n), at + tiles);
        left = tiles - (k1 - k0);
    }
    __device__ __forceinline__ bool next(const Space &ws)
    {
        if (left <= 0) return false;
        do { ++b; } while (ws.blocks[b].n == 0);       // (ends: tiles are left)
        take(ws, 0, left);
        return true;
    }
};

// Columns of S that a block of rows takes.
__device__ __forceinline__ int columns(int rows) { return max(16, (rows + 15) & ~15); }

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarpsEpi) : "memory"); }

// Whether any thread of the epilogue says so (a barrier of them all).
__device__ __forceinline__ bool epi_any(bool v)
{
    uint32_t r;
    asm volatile(
        "{\n"
        ".reg .pred pin, pout;\n"
        "setp.ne.u32 pin, %1, 0;\n"
        "bar.red.or.pred pout, 1, %2, pin;\n"
        "selp.u32 %0, 1, 0, pout;\n"
        "}\n"
        : "=r"(r)
        : "r"((uint32_t)v), "n"(32 * kWarpsEpi)
        : "memory");
    return r != 0;
}

// An arrival that hands nothing over in memory.  (With release it waits for the warp's
// global loads and stores on their way: 2,500 cycles a tile in the epilogue.)
__device__ __forceinline__ void arrive_relaxed(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A row without weight: its log sum is infinite.
__device__ __forceinline__ bool no_weight(float lse) { return fabsf(lse) > 0x1p29f; }

// D (TMEM) += A (TMEM, K-major) . B (shared memory)
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 lanes x 32 columns
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// 16 columns of both parts of S; wait_s: they are there.
__device__ __forceinline__ void load_s(uint32_t tS, float (&x)[2][16])
{
    tmem_ld16(tS, x[0]);
    tmem_ld16(tS + 64, x[1]);
}

__device__ __forceinline__ void wait_s(float (&x)[2][16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+f"(x[0][i]), "+f"(x[1][i]));      // (what is done with them stays behind the wait)
}

// Adds an entry's weights of `cols` rows (a multiple of 16).  kPlain: all of them see the
// entry and one m serves them all; else a NaN of a row that does not see it stays out.
template <bool kPlain>
__device__ __forceinline__ void weigh(uint32_t tS, int cols, const float *r, const float *m, const int *see, int e, float l2s, float m_all,
                                      float (&sum)[4])
{
    auto add = [&](int c0, const float (&x)[2][16]) {
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
            const float4 row = *reinterpret_cast<const float4 *>(r + c0 + c);
            float4 mm = make_float4(m_all, m_all, m_all, m_all);
            if (!kPlain) mm = *reinterpret_cast<const float4 *>(m + c0 + c);
            const float2 y = fma_f32x2(make_float2(x[0][c] + x[1][c], x[0][c + 1] + x[1][c + 1]), make_float2(l2s, l2s), make_float2(-mm.x, -mm.y));
            const float2 z = fma_f32x2(make_float2(x[0][c + 2] + x[1][c + 2], x[0][c + 3] + x[1][c + 3]), make_float2(l2s, l2s),
                                       make_float2(-mm.z, -mm.w));
            const float s0 = fmaf(fast_exp2(y.x), row.x, sum[0]), s1 = fmaf(fast_exp2(y.y), row.y, sum[1]);
            const float s2 = fmaf(fast_exp2(z.x), row.z, sum[2]), s3 = fmaf(fast_exp2(z.y), row.w, sum[3]);
            if (kPlain) {
                sum[0] = s0; sum[1] = s1; sum[2] = s2; sum[3] = s3;
            } else {
                const int4 v = *reinterpret_cast<const int4 *>(see + c0 + c);
                if (e < v.x) sum[0] = s0;
                if (e < v.y) sum[1] = s1;
                if (e < v.z) sum[2] = s2;
                if (e < v.w) sum[3] = s3;
            }
        }
    };
    if (kPlain && cols == (int)kPass) {                     // the next columns on their way
        float x[2][2][16];
        load_s(tS, x[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            wait_s(x[i & 1]);
            if (i < 3) load_s(tS + 16 * (i + 1), x[(i + 1) & 1]);
            add(16 * i, x[i & 1]);
        }
    } else {
        for (int c0 = 0; c0 < cols; c0 += 16) {
            float x[2][16];
            load_s(tS + c0, x);
            wait_s(x);
            add(c0, x);
        }
    }
}

// Blocks b0 .. b1 - 1 of the plan (b1 may lie behind the last).
__global__ void __launch_bounds__(kThreads, 1) mass_kernel(const __grid_constant__ CUtensorMap codes, const __grid_constant__ CUtensorMap scales,
                                                           MassParams p, int b0, int b1, int run_log)
{
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *sQ = smem;
    uint8_t *sCodes = sQ + kQBytes;                                  // [4][128 entries][128 B], swizzled
    uint8_t *sScales = sCodes + kUnits * kUnit;                      // [3][128 entries][32 B]
    float *sM = reinterpret_cast<float *>(sScales + kScaleUnits * kScaleUnit);       // [128] m and r of a row
    float *sR = sM + kRows;
    int *sSees = reinterpret_cast<int *>(sR + kRows);                // [128]
    float *sTop = reinterpret_cast<float *>(sSees + kRows);          // [8] largest and smallest lse2 of four warps
    uint64_t *bar_raw = reinterpret_cast<uint64_t *>(sTop + 8);      // [4] half tile loaded
    uint64_t *bar_read = bar_raw + kUnits;                           // [4] half tile dequantised
    uint64_t *bar_sc = bar_read + kUnits;                            // [3] scales loaded
    uint64_t *bar_scread = bar_sc + kScaleUnits;                     // [3] scales read
    uint64_t *bar_k = bar_scread + kScaleUnits;                      // [2] half of K stored
    uint64_t *bar_kfree = bar_k + 2;                                 // [2] its MMAs done
    uint64_t *bar_s = bar_kfree + 2;                                 // [2] S complete
    uint64_t *bar_sfree = bar_s + 2;                                 // [2] S read
    uint64_t *bar_q = bar_sfree + 2;                                 // queries stored
    uint64_t *bar_piece = bar_q + 1;                                 // a piece's MMAs done
    int *sFlag = reinterpret_cast<int *>(bar_piece + 1);             // [0] abort, [1] first block
    uint32_t *sTmem = reinterpret_cast<uint32_t *>(sFlag + 2);
    volatile int *abort_flag = sFlag;
    if (tid == 0) {
        for (int i = 0; i < kUnits; ++i) { mbar_init(&bar_raw[i], 1); mbar_init(&bar_read[i], kWarpsProd / 2); }   // (half a tile: four warps)
        for (int i = 0; i < kScaleUnits; ++i) { mbar_init(&bar_sc[i], 1); mbar_init(&bar_scread[i], kWarpsProd); }
        for (int i = 0; i < 2; ++i) { mbar_init(&bar_k[i], kWarpsProd / 2); mbar_init(&bar_kfree[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&bar_s[i], 1); mbar_init(&bar_sfree[i], kWarpsEpi / 2); }
        mbar_init(bar_q, kWarpsProd);
        mbar_init(bar_piece, 1);
        sFlag[0] = 0;
        fence_barrier_init();
        prefetch_tmap(&codes);
        prefetch_tmap(&scales);
    }
    if (warp == kWarpMma) {
        tmem_alloc(sTmem, 512);
        tmem_relinquish();
    }
    pdl_wait();
    const Space ws = space_of(p);
    b1 = min(b1, ws.group_first[p.ng]);
    int64_t u0 = 0, run = 0;
    if (b0 < b1) {
        const int64_t first = ws.blocks[b0].first, units = ws.blocks[b1].first - first;
        const int64_t each = (units + gridDim.x - 1) / gridDim.x;
        u0 = first + min(blockIdx.x * each, units);
        run = min(each, first + units - u0);
        if (run > 0)
            for (int b = b0 + tid; b < b1; b += kThreads)
                if (ws.blocks[b].first <= u0 && u0 < ws.blocks[b + 1].first) sFlag[1] = b;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *sTmem;
    Work w{};
    bool more = run > 0;
    if (more) {
        w.b = sFlag[1];
        w.take(ws, (int)(u0 - ws.blocks[w.b].first), run);
    }
    bool ok = true;

    if (warp == kWarpMma) {
        // ============================================== MMA issuer (the whole warp runs the loop, one lane issues)
        // Buffers, halves and passes are unrolled, so that every address and descriptor is
        // an immediate away from two registers: the MMAs take theirs from uniform
        // registers, and moving five of them there for each costs 55 cycles, 33 being its own.
        // K comes in two halves, not more: a wait or a commit costs the warp some 100
        // cycles (four stages: 178 us instead of 163 for 32 x 64 rows over 65,536 entries).
        uint32_t elected;
        asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(elected));
        const uint32_t q0 = __shfl_sync(0xffffffffu, smem_u32(sQ), 0), t0 = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dq = smem_desc(q0, 16, 1024, kLayoutSW128);
        uint32_t tile = 0, pieces = 0, used[2] = {1, 1};       // parities of the waits
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
            tc_fence_after();
        };
        // a pass over the rows kR .. (the first waits for K) into buffer kBuf; last: K is not used again
        auto pass_as = [&](auto buf, auto r, uint32_t id, bool last) {
            constexpr uint32_t kBuf = decltype(buf)::value, kR = decltype(r)::value;
            wait(&bar_sfree[kBuf], used[kBuf]);
            used[kBuf] ^= 1;
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) {
                if (kR == 0) wait(&bar_k[h], tile & 1);
                if (!ok) break;
                if (elected) {
#pragma unroll
                    for (uint32_t ks = 0; ks < 16; ++ks)
                        mma_f16_ts(t0 + (kColS + 128 * kBuf + 64 * h), t0 + (128 * h + 8 * ks),
                                   dq + (kR * 128 / 16 + (4 * h + (ks >> 2)) * (kQAtom >> 4) + 2 * (ks & 3)), id, ks > 0 ? 1u : 0u);
                    if (last) mma_commit(&bar_kfree[h]);
                    if (h == 1) mma_commit(&bar_s[kBuf]);
                }
                __syncwarp();
            }
        };
        constexpr uint32_t id64 = instr_desc(128, kPass, 0, 0, 0, 0);
        using B0 = std::integral_constant<uint32_t, 0>;
        using B1 = std::integral_constant<uint32_t, 1>;
        using R1 = std::integral_constant<uint32_t, kPass>;
        for (; more && ok; more = w.next(ws), ++pieces) {
            const uint32_t n = (uint32_t)columns(ws.blocks[w.b].rows), rest = n > kPass ? n - kPass : n;
            const uint32_t id = instr_desc(128, 0, 0, 0, 0, 0) | ((rest >> 3) << 17);
            wait(bar_q, pieces & 1);
            for (int t = w.k0; t < w.k1 && ok; ++t, ++tile) {
                if (n > kPass) {
                    pass_as(B0{}, B0{}, id64, false);
                    if (rest == kPass) pass_as(B1{}, R1{}, id64, true);
                    else pass_as(B1{}, R1{}, id, true);
                } else if (tile & 1) {
                    if (rest == kPass) pass_as(B1{}, B0{}, id64, true);
                    else pass_as(B1{}, B0{}, id, true);
                } else {
                    if (rest == kPass) pass_as(B0{}, B0{}, id64, true);
                    else pass_as(B0{}, B0{}, id, true);
                }
            }
            if (ok && elected) mma_commit(bar_piece);
            __syncwarp();
        }
        // every MMA has completed before TMEM and shared memory go back
        if (!ok) {
            volatile int no_abort = 0;
            if (elected) mma_commit(bar_piece);
            __syncwarp();
            mbar_wait<true>(bar_piece, (pieces - 1) & 1, &no_abort);       // (the piece that gave up is counted)
        } else if (pieces > 0) {
            wait(bar_piece, (pieces - 1) & 1);
        }
    } else if (warp == kWarpLoad) {
        // ============================================== loads: lane i has the entries run i .. of a tile
        // (One copy for as many entries as lie in one page, 128 at most; the warp goes through
        // them together, since a copy that lanes issue apart takes the place of several.)
        uint32_t unit = 0, sc_loads = 0;
        uint32_t elected;
        asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(elected));
        for (; more && ok; more = w.next(ws)) {
            const bool paged = p.pages.table != nullptr;
            const int n = ws.blocks[w.b].n, base = ws.blocks[w.b].base;
            const int32_t *const table = p.pages.table + (int64_t)ws.blocks[w.b].seq * p.pages.ld;      // (if paged)
            auto entry = [&](int t) { return t * kEnt + (lane << run_log); };
            auto there = [&](int t) { return lane < kEnt >> run_log && t < w.k1 && entry(t) < n; };
            auto page_of = [&](int t) { return paged && there(t) ? __ldg(table + (entry(t) >> p.pages.log)) : 0; };
            int page = page_of(w.k0);
            for (int t = w.k0; t < w.k1 && ok; ++t) {
                bool in = there(t);
                const int e = entry(t);
                int row = base + e;
                if (paged) {
                    if (in && (uint32_t)page >= p.pages.pages) {           // no page of the cache: nothing is read
                        count_event(p.counters, CSA2_CNT_BAD_INPUT);
                        in = false;
                    }
                    row = (int)((uint32_t)page << p.pages.log) + (e & ((1 << p.pages.log) - 1));
                    page = page_of(t + 1);
                }
                const uint32_t loads = __ballot_sync(0xffffffffu, in), tile = unit / 2, s = tile % kScaleUnits;
                // the tile's copies of `bytes` a row to `to`, once what was there is read
                auto load = [&](uint64_t *read, uint32_t parity, uint64_t *full, const CUtensorMap *map, uint8_t *to, int x, uint32_t bytes) {
                    ok = ok && __all_sync(0xffffffffu, mbar_wait<true>(read, parity, abort_flag));
                    if (!ok) return;
                    if (elected) mbar_arrive_expect_tx(full, __popc(loads) * (bytes << run_log));
                    __syncwarp();
                    for (uint32_t left = loads; left; left &= left - 1) {
                        const int i = __ffs(left) - 1, r = __shfl_sync(0xffffffffu, row, i);
                        if (elected) tma_load_2d(to + i * (bytes << run_log), map, x, r, full);
                        __syncwarp();
                    }
                };
                load(&bar_scread[s], ((tile / kScaleUnits) & 1) ^ 1, &bar_sc[s], &scales, sScales + s * kScaleUnit, 0, CSA2_SCALE_BYTES);
                if (ok) sc_loads = tile + 1;
                for (int h = 0; h < 2; ++h) {
                    const uint32_t u = unit % kUnits;
                    load(&bar_read[u], ((unit / kUnits) & 1) ^ 1, &bar_raw[u], &codes, sCodes + u * kUnit, 128 * h, 128);
                    if (ok) ++unit;
                }
            }
        }
        // (copies on their way end before the CTA does)
        if (!ok) {
            volatile int no_abort = 0;
            for (uint32_t i = unit > kUnits ? unit - kUnits : 0; i < unit; ++i) mbar_wait<true>(&bar_raw[i % kUnits], (i / kUnits) & 1, &no_abort);
            for (uint32_t i = sc_loads > kScaleUnits ? sc_loads - kScaleUnits : 0; i < sc_loads; ++i)
                mbar_wait<true>(&bar_sc[i % kScaleUnits], (i / kScaleUnits) & 1, &no_abort);
        }
    } else if (warp >= kWarpProd) {
        // ============================================== producers
        // A warp dequantises the 32 entries of its TMEM lanes, an entry a lane, in one
        // half of the channels: 128 bytes of codes, 128 TMEM columns.
        const int pw = warp - kWarpProd, quarter = warp & 3, half = pw >> 2;
        const int row = 32 * quarter + lane;
        const uint32_t to = tmem + 128 * half + ((uint32_t)(32 * quarter) << 16);
        uint32_t tile = 0, pieces = 0;
        for (; more && ok; more = w.next(ws), ++pieces) {
            // ---- the block's queries, once the last block's products are done
            if (pieces > 0) ok = __all_sync(0xffffffffu, mbar_wait<true>(bar_piece, (pieces - 1) & 1, abort_flag));
            if (!ok) break;
            const int rows = ws.blocks[w.b].rows, row0 = ws.blocks[w.b].row0, n = columns(rows);
            const uint4 *const q = reinterpret_cast<const uint4 *>(p.q) + (int64_t)row0 * (CSA2_D / 8);
            for (int i0 = 32 * pw + lane; i0 < n * 64; i0 += 4 * 32 * kWarpsProd) {
                uint4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = i0 + k * 32 * kWarpsProd;
                    // (zeros for a row without weight: whatever its query holds stays out)
                    const bool in = i < rows * 64 && !no_weight(__ldg(p.lse + row0 + (i >> 6)));
                    v[k] = in ? __ldg(q + i) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = i0 + k * 32 * kWarpsProd, r = i >> 6, c = i & 63;
                    if (i >= n * 64) break;
                    if (p.q_type == CSA2_BF16)
                        v[k] = make_uint4(bf16x2_to_f16x2(v[k].x), bf16x2_to_f16x2(v[k].y), bf16x2_to_f16x2(v[k].z), bf16x2_to_f16x2(v[k].w));
                    *reinterpret_cast<uint4 *>(sQ + (c >> 3) * kQAtom + sw128(r, c & 7)) = v[k];
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_q);
            for (int t = w.k0; t < w.k1 && ok; ++t, ++tile) {
                const uint32_t unit = 2 * tile + half, u = unit % kUnits, s = tile % kScaleUnits;
                ok = __all_sync(0xffffffffu, mbar_wait<true>(&bar_sc[s], (tile / kScaleUnits) & 1, abort_flag) &&
                                                 mbar_wait<true>(&bar_raw[u], (unit / kUnits) & 1, abort_flag));
                if (!ok) break;
                const uint8_t *const src = sCodes + u * kUnit;
                const uint4 sc = *reinterpret_cast<const uint4 *>(sScales + s * kScaleUnit + row * CSA2_SCALE_BYTES + 16 * half);
                const uint32_t scale[4] = {sc.x, sc.y, sc.z, sc.w};
                // (in registers at once, so that the next load of the unit is under way early)
                uint4 c[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) c[i] = *reinterpret_cast<const uint4 *>(src + sw128(row, i));
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar_read[u]);
                    mbar_arrive(&bar_scread[s]);
                }
                ok = __all_sync(0xffffffffu, mbar_wait<true>(&bar_kfree[half], (tile & 1) ^ 1, abort_flag));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t r[32];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint4 v = c[2 * i + k];
                        const uint32_t s2 = e4m3x2_to_f16x2(scale[i] >> (16 * k));
                        const uint32_t lo = __byte_perm(s2, 0, 0x1010), hi = __byte_perm(s2, 0, 0x3232);
                        const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint4 o = fp4x8_to_f16(in[x], x < 2 ? lo : hi);
                            uint32_t *const at = r + 16 * k + 4 * x;
                            at[0] = o.x; at[1] = o.y; at[2] = o.z; at[3] = o.w;
                        }
                    }
                    tmem_st32u(to + 32 * i, r);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_k[half]);
            }
        }
    } else if (warp >= kWarpEpi) {
        // ============================================== epilogue: a thread has an entry
        // Two sets of four warps, each with an S buffer of its own: of up to 64 rows they take
        // tiles in turn, of more each takes its half of the rows.  What a tile costs in
        // latency (S read, exponentials, prev) then has two passes' time.
        const float l2s = p.sm_scale * kLog2e;
        const int at = tid - 32 * kWarpEpi, ent = at & (kEnt - 1), set = at / kEnt;
        const uint32_t tS = tmem + kColS + 128 * set + ((uint32_t)(32 * (warp & 3)) << 16);
        uint32_t tile = 0, used = 0;           // parity of the next wait
        for (; more && ok; more = w.next(ws)) {
            const Block &blk = ws.blocks[w.b];
            const int rows = blk.rows, n = columns(rows), n_ent = blk.n;
            const bool alone = blk.alone;
            // Where the rows' lse2 lie within 2^64 of each other, one m in the middle serves them all:
            // a weight is 2^(l2s x - m) times up to 2^32, so that what the exponential flushes
            // to zero below 2^-126 is below 2^-94 (with the largest it was 2^-62).
            float lse2 = NAN;                  // (a row without weight, or past the block's)
            int s = 0;
            if (at < rows) {
                const float lse = p.lse[blk.row0 + at];
                if (!no_weight(lse)) lse2 = lse * kLog2e;
                s = sees(p, blk.causal, blk.pos, blk.n_group, (blk.k0 + at) / p.H);
            }
            float top = lse2, low = lse2;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
            }
            if (at < kRows && lane == 0) { sTop[at >> 5] = top; sTop[4 + (at >> 5)] = low; }
            epi_sync();
            top = fmaxf(fmaxf(sTop[0], sTop[1]), fmaxf(sTop[2], sTop[3]));
            low = fminf(fminf(sTop[4], sTop[5]), fminf(sTop[6], sTop[7]));
            const float m_all = rintf(0.5f * (top + low));
            // (false without any weight; below 2^-96 a column without a row, whose S is 0, would not stay finite)
            const bool near = top - low < 64.f && m_all > -96.f;
            if (at < kRows) {
                const float m = near ? m_all : lse2 == lse2 ? rintf(lse2) : 0.f;
                sM[at] = m;
                // (a NaN lse stays one)
                float r = 0.f;
                if (at < rows && !no_weight(p.lse[blk.row0 + at])) r = exp2f(-fmaf(p.lse[blk.row0 + at], kLog2e, -m));
                sR[at] = r;
                sSees[at] = s;
            }
            const bool halves = n > (int)kPass;
            float *const to = alone ? p.mass + (int64_t)blk.seq * p.ld_mass : ws.parts + (2 * (int64_t)(w.b - b0) + (halves ? set : 0)) * p.max_n;
            const float *const prev = alone && p.prev ? p.prev + (int64_t)blk.seq * p.ld_mass : nullptr;
            epi_sync();
            const int r0 = halves ? set * (int)kPass : 0, cols = min(n - r0, (int)kPass);
            const int all = near && r0 < rows ? sSees[r0] : 0;    // entries that every row sees
            for (int t = w.k0; t < w.k1 && ok; ++t, ++tile) {
                if (!halves && (int)(tile & 1) != set) continue;
                const int e = t * kEnt + ent;
                const float before = prev && e < n_ent ? prev[e] : 0.f;     // (on its way while S is made)
                ok = __all_sync(0xffffffffu, mbar_wait<true>(&bar_s[set], used, abort_flag));
                tc_fence_after();
                if (!ok) break;
                used ^= 1;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                if ((t + 1) * kEnt <= all) weigh<true>(tS, cols, sR + r0, sM + r0, sSees + r0, e, l2s, m_all, sum);
                else weigh<false>(tS, cols, sR + r0, sM + r0, sSees + r0, e, l2s, m_all, sum);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_relaxed(&bar_sfree[set]);
                if (e >= n_ent) continue;
                const float s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
                to[e] = prev ? fmaf(p.decay, before, s) : s;
            }
            // (all leave together if a wait gave up; else the block's rows are read)
            ok = !epi_any(!ok);
        }
    }
    if (!ok && lane == 0) *abort_flag = 1;
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) count_event(p.counters, CSA2_CNT_TIMEOUT);
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ sums over a group's blocks
// The first blocks of a group come with its decayed mass, later ones are added to it.
__global__ void __launch_bounds__(kFinishThreads) mass_finish_kernel(MassParams p, int b0, int b1)
{
    pdl_wait();
    const Space ws = space_of(p);
    const int64_t chunks = (p.max_n + kFinishThreads - 1) / kFinishThreads;
    for (int64_t item = blockIdx.x; item < p.ng * chunks; item += gridDim.x) {
        const int g = (int)(item / chunks), f = ws.group_first[g], l = ws.group_first[g + 1];
        const int lo = max(f, b0), hi = min(l, b1);
        if (lo >= hi || ws.blocks[f].alone) continue;
        const int64_t e = (item - g * chunks) * kFinishThreads + threadIdx.x;
        const Block &any = ws.blocks[f];
        if (e >= any.n_group) continue;
        float *const at = p.mass + any.seq * p.ld_mass + e;
        float s = 0.f;
        for (int b = lo; b < hi; ++b)
            if (e < ws.blocks[b].n) {
                const float *const part = ws.parts + 2 * (int64_t)(b - b0) * p.max_n + e;
                s += part[0];
                if (ws.blocks[b].rows > (int)kPass) s += part[p.max_n];
            }
        if (lo > f) *at += s;
        else *at = p.prev ? fmaf(p.decay, p.prev[any.seq * p.ld_mass + e], s) : s;
    }
}

}  // namespace

// Parts, two to a block, are kept for 32 blocks or, up to a million entries, as many as take
// 256 MB; more blocks go in turns.  Which blocks leave parts (those of groups of more than 64
// rows) only the device knows, so that all are counted: with single tokens of 64 heads, which leave
// none, a call has their memory and their turns all the same (64 of them over a million entries: 256 MB
// and three turns instead of one).
MassPlan mass_plan(int batch, int ng, int nq, int H, int64_t max_n)
{
    MassPlan pl{};
    const int64_t blocks = ((int64_t)nq * H + kRows - 1) / kRows + ng;
    pl.parts = std::max<int64_t>(32, (256ll << 20) / 8 / std::max<int64_t>(1, max_n));
    pl.blocks = blocks;
    const int64_t units = blocks * ((max_n + kEnt - 1) / kEnt);
    pl.ctas = (int)std::max<int64_t>(1, std::min<int64_t>(device_sm_count(), units));
    pl.off_groups = align_up((size_t)(blocks + 1) * sizeof(Block), 256);
    pl.off_parts = pl.off_groups + align_up(((size_t)ng + 1 + batch) * 4, 256);
    // (a group of one pass has no parts)
    const bool any = (int64_t)nq * H > (int64_t)kPass;
    pl.total = pl.off_parts + (any ? (size_t)std::min(pl.parts, blocks) * max_n * 8 : 0);
    return pl;
}

cudaError_t launch_mass(const MassParams &p, cudaStream_t st)
{
    constexpr size_t smem = 1024 + kQBytes + kUnits * kUnit + kScaleUnits * kScaleUnit + kRows * 12 + 32 + (2 * kUnits + 2 * kScaleUnits + 10) * 8 + 16;
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    // the shared-memory attribute is set once per device (a bit each; setting it twice does no harm)
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if ((done.load(std::memory_order_acquire) & bit) == 0) {
        e = cudaFuncSetAttribute(mass_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_release);
    }
    static_assert(kEnt == 128, "seven bits");
    const int run_log = p.pages.table != nullptr ? std::min(p.pages.log, 7) : 7;
    CUtensorMap codes, scales;
    e = make_tmap_rows_u8(&codes, p.codes, p.cap, CSA2_CODE_BYTES, 1 << run_log, 128, 128);
    if (e == cudaSuccess) e = make_tmap_rows_u8(&scales, p.scales, p.cap, CSA2_SCALE_BYTES, 1 << run_log, 0);
    if (e != cudaSuccess) return e;
    e = launch_k(mass_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, 0, p);
    const int64_t items = p.ng * ((p.max_n + kFinishThreads - 1) / kFinishThreads);
    for (int64_t b0 = 0; b0 < p.plan.blocks && e == cudaSuccess; b0 += p.plan.parts) {
        const int b1 = (int)std::min(b0 + p.plan.parts, p.plan.blocks);
        e = launch_k(mass_kernel, dim3(p.plan.ctas), dim3(kThreads), smem, st, 0, codes, scales, p, (int)b0, b1, run_log);
        if (e == cudaSuccess && (int64_t)p.nq * p.H > (int64_t)kPass && items > 0)
            e = launch_k(mass_finish_kernel, dim3((unsigned)std::min<int64_t>(items, device_sm_count() * 8)), dim3(kFinishThreads), 0, st, 0,
                         p, (int)b0, b1);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa2
