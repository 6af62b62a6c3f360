// csa2_dense.cu -- attention of groups of queries over whole sequences of the
// FP4 latent cache: a prompt that many sequences share (read once for all of
// them), or an encoder's entries attended by a decoder sequence's queries.
//
// Every row (query, head) of group g sees the entries j < n_g of one sequence:
//     x_j = sm_scale q . v_j,   M = max(max_j x_j, lse_prev),
//     out = (sum_j e^(x_j - M) v_j + e^(lse_prev - M) out_prev) / L,
//     lse = M + log L,  L = the same sum without v_j and out_prev.
//
// A pair of CTAs (one cluster) works on a tile of 128 rows, 64 in each CTA, and
// 256 entries at a time, with both SMs' tensor cores as one (cta_group::2):
//     S [128 rows x 256 entries]  = Q [128 x 512] . K^T          (M 128, N 256)
//     O [128 rows x 512 channels] += P [128 x 256] . V           (M 128, 2 x N 256)
// An SM then holds 64 rows' O (256 TMEM columns) and two S buffers (2 x 128),
// and an MMA reads 6 KB of its shared memory for 64 cycles of products
// (measured: 4,056 MAC per cycle and SM; M = 128 entries x N = 64 rows, the
// layout of the sparse attention, also reads 6 KB, for 32 cycles of products,
// and runs at 2,705).  Each CTA dequantises its half of both operands (E2M1 x
// E4M3 is exact in f16): as K, its 128 entries x all channels; as V, all 256
// entries x its 256 channels.  Beside Q (64 KB) and P (32 KB) there is room for
// 128 KB of them: a ring of two 64 KB stages, each 128 entries x 256 channels and
// 16 MMAs, read as K-major K or as MN-major V.
//
// Warps of a CTA: 0..7 softmax (two per TMEM lane quarter), 8..15 producers, 16
// issues the MMAs (the first CTA of the pair only).  S is double buffered: the
// product of tile i + 1's scores runs while tile i's softmax does, so the order on
// the tensor pipe is S(0) S(1) O(0) S(2) O(1) ...  All sums are fp32; P is
// rounded to f16.  A row's reference lies 7 below a maximum already seen (log2
// units) and moves whenever a logit exceeds it by 15, O being rescaled in TMEM then:
// P is at most 2^15, the row's largest weight so far at least 2^7, and a weight is off
// by 2^-11 of itself or, below f16's normals, by 2^-25, which is 2^-32 of that largest
// one (with the reference at the maximum it was 2^-25, and what lay below it, such as
// 65,535 entries at 2^-26 of one, was lost from out but not from the sum).
//
// Work is counted over all groups, and each pair takes an equal run of it
// whatever the groups' sizes.  A pair whose run begins or ends inside a row tile
// leaves that tile's sums in the workspace (at most two such pieces per pair); a
// second kernel joins the pieces in a fixed order, so results do not depend on
// timing.
//
// Measured: 32 queries x 64 heads over 65,536 entries (275 GFLOP) in 179 to 184 us
// (in a graph), 1,494 to 1,537 TFLOP/s.  What bounds a long run is the refilling of
// the ring.  With cycle counters around the waits (they add about a tenth to the
// call), of 6,240 cycles a tile the issuer waits 3,890 for filled stages and 400 for P;
// a producer waits only 700 for an empty one and takes 3,970 to convert and store, the
// rest for its loads; a softmax warp waits 2,170.  The MMAs alone are 4,134.  No
// counted unit is at its limit (16 queries: tensor pipe 60 %, LSU data pipe 58 % of
// the active cycles, issue 54 %): which of the producers' steps to shorten, or whether
// more stages would do, has not been told apart.  What bounds a short run is the chain of a piece, in cycles with a single tile: work
// found 4,700, first scores 5,900, softmax 3,400, O 2,700, epilogue 3,000 to 4,000;
// and the join (about 4 us).
#include <cuda_fp16.h>

#include <atomic>

#include "csa2_attn_device.cuh"
#include "csa2_internal.h"

namespace csa2 {

namespace {

constexpr int kWarpsSoft = 8, kWarpsProd = 8;
constexpr int kThreads = 32 * (kWarpsSoft + kWarpsProd + 1);
constexpr int kSoft = 32 * kWarpsSoft;
constexpr int kRowsPair = kDenseRows;          // rows per pair of CTAs
constexpr int kRowsCta = kRowsPair / 2;
constexpr int kEnt = kDenseEntries;            // entries per tile
constexpr int kStages = 2;
constexpr uint32_t kStage = 65536;
constexpr uint32_t kQBytes = kRowsCta * CSA2_D * 2;     // 64 KB: [8 atoms][64 rows][128 B]
constexpr uint32_t kQAtom = kRowsCta * 128;
constexpr uint32_t kPBytes = kRowsCta * kEnt * 2;       // 32 KB: [4 atoms][64 rows][128 B]
constexpr uint32_t kAtom = 128 * 128;                   // stage: [4 atoms of 64 channels][128 entries][128 B]
constexpr uint32_t kColS = 256;                // TMEM: O in columns 0 .. 255, S buffer b from 256 + 128 b
constexpr int kJoinThreads = 512;
constexpr int kSetup = kDenseSetup;
constexpr float kLazy = 8.0f;                  // log2 units
constexpr float kHead = 7.0f;                  // log2 units that a reference lies below its maximum
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

static_assert(kRowsPair == 128 && kEnt == 256, "lane and column maps below");

// ------------------------------------------------------------------ groups and work
// What a group asks for.  bad: its arguments are out of contract and its rows
// are left as they are.
struct Group {
    int base;            // cache row of entry 0 (a cache has under 2^31 rows)
    int row0;            // first row (query * H, under 2^30)
    int rows;
    int n;
    bool bad;
    bool falls;          // its offsets do
};

__device__ __forceinline__ Group group_of(const DenseParams &p, int g)
{
    Group r{};
    const int b = p.g_seq[g], a = p.g_off[g], e = p.g_off[g + 1];
    r.falls = e < a;
    r.bad = b < 0 || b >= p.batch || a < 0 || e < a || e > p.nq;
    if (r.bad) return r;
    const int64_t len = p.seq_len[b];
    const int64_t n = p.g_len ? (int64_t)p.g_len[g] : len;
    const int64_t base = p.seq_base[b];
    r.bad = n < 0 || n > len || n > p.max_n || base < 0 || base + n > p.cap;
    if (r.bad) return r;
    r.base = (int)base;
    r.n = (int)n;
    r.row0 = a * p.H;
    r.rows = (e - a) * p.H;
    return r;
}

__device__ __forceinline__ int row_tiles(const Group &g) { return (g.rows + kRowsPair - 1) / kRowsPair; }
__device__ __forceinline__ int ent_tiles(const Group &g) { return g.n / kEnt + (g.n % kEnt != 0); }

// Work is counted in units: a tile of entries is one, and each row tile has
// kSetup more in front for what a piece costs besides (queries, first scores,
// epilogue: about as long as a tile).  A run that ends in those has no piece there.
// (Without them 61 queries over five prompts of 1 to 20,011 entries take 36.5 us
// instead of 26.0, four chunks of queries 49.3 instead of 37.8.)
__device__ __forceinline__ int row_units(const Group &g) { return g.n > 0 ? ent_tiles(g) + kSetup : 0; }
__device__ __forceinline__ int64_t units(const Group &g) { return (int64_t)row_tiles(g) * row_units(g); }   // (bad: 0)

// a / b of non-negative numbers (a 32-bit division where it serves)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

// Units in a pair's run: ceil(U / pairs) each, so that the last pairs may have
// none (no more pairs, and no more split row tiles, than the longest run needs).
__device__ __forceinline__ int64_t run_units(const DenseParams &p, int64_t U) { return quotient(U + p.pairs - 1, p.pairs); }

// One pair's pieces of work in order: entries k0 .. k1 (in tiles) of a row tile.
// find() sets up the first piece.
struct Work {
    Group gr;
    int g;
    int rt;              // row tile of the group
    int kt;              // tiles of entries of the group
    int k0, k1;
    int at;              // the run's first unit within its row tile
    int64_t left;        // units left after this piece

    // From unit `at` of a row tile on, with `units` left; false: no piece.
    __device__ __forceinline__ bool take(int at, int64_t units)
    {
        kt = ent_tiles(gr);
        const int n = (int)min((int64_t)(kt + kSetup - at), units);
        k0 = max(0, at - kSetup);
        k1 = max(0, at + n - kSetup);
        left = units - n;
        return k1 > k0;
    }
    __device__ __forceinline__ bool next(const DenseParams &p)
    {
        if (left <= 0) return false;
        if (++rt == row_tiles(gr)) {
            do { gr = group_of(p, ++g); } while (units(gr) == 0);      // (ends: units are left)
            rt = 0;
        }
        return take(0, left);
    }
};

constexpr int kMaxPieces = 96;                 // of a row tile: one more than the pairs at most, three per lane of a warp
static_assert(kDensePairsMax < kMaxPieces && kMaxPieces == 96, "join's weights");
static_assert(kJoinThreads == 512 && CSA2_D == 4 * 128, "join's shifts");

// What a pair works on.
struct Found {
    Work w;
    int64_t run;         // units of a pair's run
    int64_t u0;          // this pair's first
    int work;            // whether it has a piece
    int empty;           // some group has rows but no entries
    int groups;          // groups before the first whose offsets fall: those behind it may share rows with them
};

// Found by the whole CTA: thread t < 512 takes ceil(ng / 512) groups, whose units
// are summed over the warps (totals in `sums`, kFindWarps of them); the thread that
// holds unit u0 sets up the work.  Up to 32 groups are one warp's alone (0.7 us
// less than with the others waiting for it).  Where offsets fall, the units of the
// groups from there on are taken out and the sums made again.  Ends without a barrier.
constexpr int kFindWarps = 16;

__device__ __forceinline__ void find(const DenseParams &p, int pair, int tid, bool count_bad, int64_t *sums, Found *out)
{
    const int lane = tid & 31, warp = tid >> 5;
    const bool few = p.ng <= 32;
    if (few && warp != 0) return;
    const int each = (p.ng + 32 * kFindWarps - 1) / (32 * kFindWarps);
    const int g0 = warp < kFindWarps ? min(tid * each, p.ng) : p.ng, g1 = min(g0 + each, p.ng);
    Group gr{};
    int64_t mine = 0;
    int empty = 0, fall = p.ng;
    for (int g = g0; g < g1; ++g) {
        gr = group_of(p, g);
        if (gr.falls) fall = min(fall, g);
        if (gr.bad && count_bad) count_event(p.counters, CSA2_CNT_BAD_INPUT);
        if (!gr.bad && gr.n == 0 && gr.rows > 0) empty = 1;
        mine += units(gr);
    }
    int groups = p.ng;                         // in contract as far as their offsets go
    auto drop = [&](int from) {                // the groups from `from` on count no more
        groups = from;
        for (int g = max(g0, from); g < g1; ++g) {
            const Group x = group_of(p, g);
            if (!x.bad && count_bad) count_event(p.counters, CSA2_CNT_BAD_INPUT);
            mine -= units(x);
        }
    };
    auto warp_sum = [&]() {                    // inclusive
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        return upto;
    };
    int64_t before, total = 0;
    if (few) {
        empty = __any_sync(0xffffffffu, empty);
        fall = __reduce_min_sync(0xffffffffu, fall);
        if (fall < groups) drop(fall);
        const int64_t upto = warp_sum();
        before = upto - mine;
        total = __shfl_sync(0xffffffffu, upto, 31);
    } else {
        int *const falls = reinterpret_cast<int *>(sums + kFindWarps);
        fall = __reduce_min_sync(0xffffffffu, fall);
        for (;;) {                             // (twice at most)
            const int64_t upto = warp_sum();
            if (lane == 31 && warp < kFindWarps) { sums[warp] = upto; falls[warp] = fall; }
            empty = __syncthreads_or(empty);
            before = upto - mine;
            total = 0;
            int first = p.ng;
#pragma unroll
            for (int i = 0; i < kFindWarps; ++i) {
                const int64_t v = sums[i];
                if (i < warp) before += v;
                total += v;
                first = min(first, falls[i]);
            }
            if (first == groups) break;
            drop(first);
            __syncthreads();                   // the sums are read
        }
    }
    const int64_t run = run_units(p, total), u0 = min(pair * run, total), left = min(run, total - u0);
    if (left > 0 ? u0 >= before && u0 < before + mine : tid == 0) {
        out->run = run;
        out->u0 = u0;
        out->empty = empty;
        out->groups = groups;
        out->work = 0;
        if (left > 0) {
            int g = g0;
            if (each > 1) {
                for (gr = group_of(p, g); u0 >= before + units(gr); gr = group_of(p, ++g)) before += units(gr);
            }
            Work &w = out->w;
            w.gr = gr;
            w.g = g;
            w.rt = (int)quotient(u0 - before, row_units(gr));
            w.at = (int)(u0 - before - (int64_t)w.rt * row_units(gr));
            out->work = w.take(w.at, left);
        }
    }
}

// ------------------------------------------------------------------ pairs of CTAs
__device__ __forceinline__ uint32_t cta_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t in_cta(uint32_t saddr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}

// Arrives on a barrier of either CTA.  What the arrival announces is written to
// this CTA's own shared memory or TMEM and read by this SM's tensor core (the
// proxy fence before it orders that), so CTA scope is enough; at cluster scope
// the release waits for the warp's outstanding loads and an acquire drops L1
// (with 16 KB stages, 823 us instead of 404 at 32 x 64 heads x 65,536 entries).
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Every wait of both CTAs ends: the flag of each is raised (before this CTA can
// arrive at the last barrier).
__device__ __forceinline__ void raise_abort(int *flag)
{
    const uint32_t a = smem_u32(flag);
    for (uint32_t r = 0; r < 2; ++r)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(in_cta(a, r)), "r"(1) : "memory");
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
}

__device__ __forceinline__ void mma2(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrives on `bar` of both CTAs once every earlier MMA of this thread completed.
__device__ __forceinline__ void commit2(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoft) : "memory"); }

__device__ __forceinline__ bool soft_any(bool v)
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
        : "r"((uint32_t)v), "n"(kSoft)
        : "memory");
    return r != 0;
}

// 16 bytes global -> shared, zeros when !in
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b)
{
    uint64_t d;
    asm("{\n"
        ".reg .b64 ra, rb;\n"
        "mov.b64 ra, {%1, %2};\n"
        "mov.b64 rb, {%3, %4};\n"
        "add.rn.f32x2 %0, ra, rb;\n"
        "}\n"
        : "=l"(d)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return make_float2(__uint_as_float((uint32_t)d), __uint_as_float((uint32_t)(d >> 32)));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32])
{
    float a[16], b[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) { a[i] = v[i]; b[i] = v[16 + i]; }
    tmem_st16(taddr, a);
    tmem_st16(taddr + 16, b);
}

// ------------------------------------------------------------------ results
template <int kOut>
__device__ __forceinline__ void store4(void *out, int64_t at, float a, float b, float c, float d)
{
    if constexpr (kOut == CSA2_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + at) = make_float4(a, b, c, d);
    } else if constexpr (kOut == CSA2_BF16) {
        uint32_t lo, hi;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(d), "f"(c));
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(out) + at) = make_uint2(lo, hi);
    } else {
        *reinterpret_cast<uint2 *>(static_cast<__half *>(out) + at) =
            make_uint2(f32x2_to_f16x2(a, b), f32x2_to_f16x2(c, d));
    }
}

// A row's softmax (its reference m in log2 units and l = sum 2^(x - m)) joined with
// the caller's partial result: the weights of the two, and the joint lse.
struct Joined { float own, prev, lse; };

__device__ __forceinline__ Joined join_prev(float m, float l, bool any_prev, float prev_lse)
{
    const float pm = any_prev ? prev_lse * kLog2e : -INFINITY;
    const bool has = m > -INFINITY, hasp = pm > -INFINITY || pm != pm;
    Joined j;
    const float M = has ? (hasp ? fmaxf(m, pm) : m) : pm;
    const float a = has ? fast_exp2(m - M) : 0.f, b = hasp ? fast_exp2(pm - M) : 0.f;
    const float L = fmaf(l, a, b);
    const float inv = (has || hasp) ? 1.f / L : 0.f;
    j.own = a * inv;
    j.prev = hasp ? b * inv : 0.f;      // (a NaN sum does not make a missing partial result count)
    j.lse = (has || hasp) ? (M + log2f(L)) * kLn2 : -INFINITY;
    return j;
}

// 64 rows of Q as f16 into the swizzled sQ (rows from n_rows on are zero), by
// the 256 threads t of eight warps: warp w takes rows w + 8 i, all 16 copies of a
// thread on their way at once, and converts what it copied where it lies, the
// first 256 channels first: the scores' first stage needs no others (that takes
// 0.7 us off every first piece).
__device__ __forceinline__ void issue_q(const DenseParams &p, uint8_t *sQ, int64_t row0, int n_rows, int t)
{
    const int c8 = t & 31;
    const uint8_t *src = reinterpret_cast<const uint8_t *>(p.q + row0 * CSA2_D);
    const uint32_t dst = smem_u32(sQ) + (c8 >> 3) * kQAtom;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = (t >> 5) + 8 * i;
            cp_async16(dst + h * 4 * kQAtom + sw128(r, c8 & 7), r < n_rows ? src + r * 1024 + h * 512 + c8 * 16 : src, r < n_rows);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
}

// Half h of them, then one arrival per warp on q_bar[h].
template <int h>
__device__ __forceinline__ void finish_q(const DenseParams &p, uint8_t *sQ, int t, uint32_t q_bar)
{
    const int c8 = t & 31;
    asm volatile("cp.async.wait_group %0;" ::"n"(1 - h) : "memory");
    if (p.q_type == CSA2_BF16) {
#pragma unroll 4
        for (int i = 0; i < 8; ++i) {
            uint4 *const at = reinterpret_cast<uint4 *>(sQ + (4 * h + (c8 >> 3)) * kQAtom + sw128((t >> 5) + 8 * i, c8 & 7));
            const uint4 v = *at;
            *at = make_uint4(bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y), bf16x2_to_f16x2(v.z), bf16x2_to_f16x2(v.w));
        }
    }
    fence_async_smem();
    __syncwarp();
    if ((t & 31) == 0) arrive_at(q_bar + 8 * h);
}

// Rows of a group without entries: the caller's partial result, or nothing.
template <int kOut>
__device__ __forceinline__ void empty_rows(const DenseParams &p, const Group &gr, int first, int step)
{
    for (int64_t i = first; i < (int64_t)gr.rows * (CSA2_D / 4); i += step) {
        const int64_t row = gr.row0 + i / (CSA2_D / 4);
        const int c = (int)(i % (CSA2_D / 4)) * 4;
        const float pl = p.prev_out ? p.prev_lse[row] : -INFINITY;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (pl > -INFINITY || pl != pl) v = *reinterpret_cast<const float4 *>(p.prev_out + row * CSA2_D + c);
        store4<kOut>(p.out, row * CSA2_D + c, v.x, v.y, v.z, v.w);
        if (c == 0 && p.lse) p.lse[row] = pl;
    }
}

template <int kOut>
__global__ void __launch_bounds__(kThreads, 1) dense_attn_kernel(DenseParams p)
{
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t rank = cta_rank();
    const int pair = (int)(blockIdx.x >> 1);

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *sRing = smem;                     // [2 stages][64 KB]
    uint8_t *sQ = sRing + kStages * kStage;
    uint8_t *sP = sQ + kQBytes;
    float *sRed = reinterpret_cast<float *>(sP + kPBytes);   // [4 threads of a row][64 rows]
    float *sM = sRed + 4 * kRowsCta;           // reference per row: kHead below a maximum (log2 units)
    float *sAlpha = sM + kRowsCta;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sAlpha + kRowsCta);
    uint64_t *bar_full = bars;                 // [2] (first CTA's) stage filled by both CTAs
    uint64_t *bar_empty = bars + 8;            // [2] stage's MMAs done
    uint64_t *bar_s = bars + 16;               // [2] S buffer complete
    uint64_t *bar_p = bars + 18;               // (first CTA's) P stored by both CTAs
    uint64_t *bar_o = bars + 19;               // a tile's O products done
    uint64_t *bar_q = bars + 20;               // [2] (first CTA's) a half of Q's channels stored by both CTAs
    uint64_t *bar_done = bars + 22;            // (first CTA's) every MMA done
    int *sFlag = reinterpret_cast<int *>(bars + 23);         // [0] abort
    uint32_t *sTmem = reinterpret_cast<uint32_t *>(sFlag + 1);
    Found *sFound = reinterpret_cast<Found *>(bars + 24);
    volatile int *abort_flag = sFlag;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bar_full[i], 2 * kWarpsProd);
            mbar_init(&bar_empty[i], 1);
        }
        mbar_init(&bar_s[0], 1);
        mbar_init(&bar_s[1], 1);
        mbar_init(bar_p, 2 * kWarpsSoft);
        mbar_init(bar_o, 1);
        mbar_init(&bar_q[0], 2 * 8);           // eight warps of each CTA, of either kind
        mbar_init(&bar_q[1], 2 * 8);
        mbar_init(bar_done, 1);
        sFlag[0] = 0;
        fence_barrier_init();
    }
    if (warp == kWarpsSoft + kWarpsProd) {     // (warp 0 is looking for its work)
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(sTmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    // (the other CTA's barriers are used only once it has arrived here)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    pdl_wait();
    find(p, pair, tid, blockIdx.x == 0, reinterpret_cast<int64_t *>(sRing), sFound);
    tc_fence_before();
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    tc_fence_after();
    const uint32_t tmem = *sTmem;
    Work w = sFound->w;
    if (tid == 32 * (kWarpsSoft + kWarpsProd) && rank == 0) {
        // for the join: the row tile that this pair begins in
        DenseBegin d{};
        if (sFound->work) {
            d.first = sFound->u0 - w.at + kSetup;
            d.last = d.first + w.kt;
            d.run = sFound->run;
            d.row0 = w.gr.row0 + w.rt * kRowsPair;
            d.rows = min(kRowsPair, w.gr.rows - w.rt * kRowsPair);
        }
        p.begin[pair] = d;
    }
    bool more = sFound->work != 0;
    // A row tile's rows are halved between the CTAs: the first of this one's, in the tile
    auto row_split = [&](const Work &x) { return (int)rank * ((min(kRowsPair, x.gr.rows - x.rt * kRowsPair) + 1) >> 1); };
    auto row_count = [&](const Work &x) {
        const int n = min(kRowsPair, x.gr.rows - x.rt * kRowsPair);
        return rank == 0 ? (n + 1) >> 1 : n >> 1;
    };

    if (warp == kWarpsSoft + kWarpsProd) {
        // ============================================== MMA issuer
        // The whole warp runs the loop and one elected lane issues: descriptors and
        // waits then stay in uniform registers.  (Measured for a wait, four MMAs and
        // a commit: 258 cycles, the MMAs' own time; with a branch on lane 0 around
        // the loop 404 to 483.)  The loop over stages stays rolled, or its
        // descriptors are kept in registers and spilled.
        if (rank == 0) {
            uint32_t elected;
            asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(elected));
            constexpr uint32_t id_s = instr_desc(128, 256, 0, 0, 0, 0);
            constexpr uint32_t id_o = instr_desc(128, 256, 0, 0, 0, 1);
            const uint32_t ring = __shfl_sync(0xffffffffu, smem_u32(sRing), 0);
            const uint32_t t0 = __shfl_sync(0xffffffffu, tmem, 0);
            const uint64_t dq = smem_desc(ring + kStages * kStage, 16, 1024, kLayoutSW128);
            const uint64_t dp = smem_desc(ring + kStages * kStage + kQBytes, 16, 1024, kLayoutSW128);
            const uint64_t dk = smem_desc(ring, 16, 1024, kLayoutSW128);
            const uint64_t dv = smem_desc(ring, kAtom, 1024, kLayoutSW128);
            uint32_t fills = 0;                // parity of the ring's fill (all stages at a time)
            uint32_t tile = 0, pieces = 0;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
                tc_fence_after();
            };
            auto scores = [&](uint32_t buf, bool first) {
                const uint32_t d = t0 + kColS + 128 * buf;
#pragma unroll 1
                for (uint32_t j = 0; j < kStages; ++j) {
                    if (first) wait(&bar_q[j], pieces & 1);
                    wait(&bar_full[j], fills);
                    if (!ok) return;
                    if (elected) {
#pragma unroll
                        for (int ks = 0; ks < 16; ++ks)
                            mma2(d, dq + (j * (4 * kQAtom >> 4) + (ks >> 2) * (kQAtom >> 4) + 2 * (ks & 3)),
                                 dk + (j * (kStage >> 4) + (ks >> 2) * (kAtom >> 4) + 2 * (ks & 3)), id_s, ks > 0 ? 1u : j);
                        commit2(&bar_empty[j]);
                        if (j == kStages - 1) commit2(&bar_s[buf]);
                    }
                    __syncwarp();
                }
                fills ^= 1;
            };
            for (; more && ok; more = w.next(p), ++pieces) {
                const int n_tiles = w.k1 - w.k0;
                scores(tile & 1, true);
                for (int i = 0; i < n_tiles && ok; ++i, ++tile) {
                    if (i + 1 < n_tiles) scores((tile + 1) & 1, false);
                    wait(bar_p, tile & 1);
                    if (!ok) break;
#pragma unroll 1
                    for (uint32_t j = 0; j < kStages; ++j) {
                        wait(&bar_full[j], fills);
                        if (!ok) break;
                        if (elected) {
#pragma unroll
                            for (int ks = 0; ks < 8; ++ks) {
                                const uint64_t a = dp + (j * (2 * kQAtom >> 4) + (ks >> 2) * (kQAtom >> 4) + 2 * (ks & 3));
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    mma2(t0 + 128 * c, a, dv + (j * (kStage >> 4) + ((c * 2 * kAtom + ks * 2048) >> 4)), id_o,
                                         ks > 0 ? 1u : (uint32_t)i | j);
                            }
                            commit2(&bar_empty[j]);
                            if (j == kStages - 1) commit2(bar_o);
                        }
                        __syncwarp();
                    }
                    fills ^= 1;
                }
            }
            // every MMA has completed before the pair gives its TMEM and shared memory back
            volatile int no_abort = 0;
            if (elected)
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                                 smem_u32(bar_done))
                             : "memory");
            __syncwarp();
            if (!mbar_wait<true>(bar_done, 0, &no_abort)) ok = false;
            if (!ok && elected) raise_abort(sFlag);
        }
    } else if (warp >= kWarpsSoft) {
        // ============================================== producers
        // A stage is 1,024 units of 32 channels of one entry (16 code bytes, 2
        // scales), four per lane of the eight warps.  Eight lanes read one entry's
        // 128 code bytes, a whole line (with 64 or 32 bytes of an entry per eight lanes
        // it took 298 and 323 us at 32 x 64 heads x 65,536 entries, so 248).  Those eight
        // lanes write their four 16-byte pieces each in an order turned by 0 .. 3, so
        // that they hit eight bank groups at every store.  Codes are loaded a whole
        // ring (two stages) ahead.
        const int pw = warp - kWarpsSoft;
        const int half = lane & 1, atom = (lane >> 1) & 3, e4 = lane >> 3;
        const bool turn1 = (atom & 1) != 0, turn2 = (atom & 2) != 0;
        const uint32_t full0 = in_cta(smem_u32(bar_full), 0);
        uint32_t piece[4];                     // the four stores of an entry e4 mod 8; of e4 + 4 mod 8: ^ 64
#pragma unroll
        for (int i = 0; i < 4; ++i)
            piece[i] = smem_u32(sRing) + atom * kAtom + (16 * pw + e4) * 128u +
                       (uint32_t)(((4 * half + ((i + atom) & 3)) ^ e4) << 4);
        uint32_t fills = 1;                    // parity of the next wait on "empty": the first pass is free
        const uint32_t q_full = in_cta(smem_u32(bar_q), 0);
        uint32_t tiles = 0;                    // of the pieces before
        bool ok = true;
        uint4 gc[4 * kStages];
        uint32_t gs[4 * kStages];
        for (; more && ok; more = w.next(p)) {
            const int n_tiles = w.k1 - w.k0, n_blocks = 2 * n_tiles;
            const int n_left = w.gr.n - w.k0 * kEnt;                     // entries from the piece's first on
            const int64_t first = (int64_t)w.gr.base + w.k0 * kEnt;
            const uint8_t *const codes = p.codes + first * CSA2_CODE_BYTES;
            const uint8_t *const scales = p.scales + first * CSA2_SCALE_BYTES;
            // The blocks of two stages: S(0) S(1) O(0) S(2) O(1) ... O(last).  Unit u of
            // stage s is, for S, entry 16 pw + 4 u + e4 of this CTA's 128, channels
            // 256 s + ..; for O, that entry of the tile's s-th 128, channels 256 rank + ..
            const uint8_t *c0 = nullptr, *s0 = nullptr;
            int c_step = 0, s_step = 0, left = 0, left_s = 0;
            bool inside = true;                // the whole tile lies inside the sequence
            auto begin = [&](int b) {
                const bool k = b == 0 || ((b & 1) != 0 && b != n_blocks - 1);
                const int tile = b == 0 ? 0 : b == n_blocks - 1 ? n_tiles - 1 : (b & 1) ? (b + 1) >> 1 : (b >> 1) - 1;
                const int e = tile * kEnt + e4 + 16 * pw + (k ? 128 * (int)rank : 0);
                const int ch = 64 * atom + 32 * half + (k ? 0 : 256 * (int)rank);
                inside = (tile + 1) * kEnt <= n_left;
                left = n_left - e;
                c0 = codes + (int64_t)e * CSA2_CODE_BYTES + (ch >> 1);
                s0 = scales + (int64_t)e * CSA2_SCALE_BYTES + (ch >> 4);
                c_step = k ? 128 : 128 * CSA2_CODE_BYTES;
                s_step = k ? 16 : 128 * CSA2_SCALE_BYTES;
                left_s = k ? 0 : 128;
            };
            auto load = [&](int s) {
                const uint8_t *c = c0 + s * c_step, *sc = s0 + s * s_step;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    uint32_t t = 0;
                    if (inside || left_s * s + 4 * u < left) {
                        v = __ldg(reinterpret_cast<const uint4 *>(c + 4 * u * CSA2_CODE_BYTES));
                        t = __ldg(reinterpret_cast<const uint16_t *>(sc + 4 * u * CSA2_SCALE_BYTES));
                    }
                    gc[4 * s + u] = v;
                    gs[4 * s + u] = t;
                }
            };
            begin(0);
            load(0);
            // ---- Q, once the last piece's scores are done (the first piece's comes from
            // the softmax warps, which have nothing else to do then)
            if (tiles > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait<true>(&bar_s[(tiles - 1) & 1], ((tiles - 1) >> 1) & 1, abort_flag));
                if (!ok) break;
                const int r0 = w.rt * kRowsPair + row_split(w);
                const int n_rows = row_count(w);
                issue_q(p, sQ, (int64_t)(w.gr.row0 + r0), n_rows, 32 * pw + lane);
                load(1);
                finish_q<0>(p, sQ, 32 * pw + lane, q_full);
                finish_q<1>(p, sQ, 32 * pw + lane, q_full);
            } else {
                load(1);
            }
            tiles += n_tiles;
            for (int b = 0; b < n_blocks && ok; ++b) {
                const bool ahead = b + 1 < n_blocks;
                if (ahead) begin(b + 1);
#pragma unroll
                for (int s = 0; s < kStages; ++s) {
                    ok = ok && __all_sync(0xffffffffu, mbar_wait<true>(&bar_empty[s], fills, abort_flag));
                    if (!ok) break;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t sc = e4m3x2_to_f16x2(gs[4 * s + u]);
                        const uint32_t p0 = __byte_perm(sc, 0, 0x1010), p1 = __byte_perm(sc, 0, 0x3232);
                        uint4 c = gc[4 * s + u];
                        if (turn1) c = make_uint4(c.y, c.z, c.w, c.x);
                        if (turn2) c = make_uint4(c.z, c.w, c.x, c.y);
                        const uint32_t q0 = turn2 ? p1 : p0, q1 = turn1 != turn2 ? p1 : p0;
                        const uint32_t q2 = turn2 ? p0 : p1, q3 = turn1 != turn2 ? p0 : p1;
                        const uint32_t d = s * kStage + 4 * u * 128, x = (u & 1) * 64;
                        st_shared16((piece[0] ^ x) + d, fp4x8_to_f16(c.x, q0));
                        st_shared16((piece[1] ^ x) + d, fp4x8_to_f16(c.y, q1));
                        st_shared16((piece[2] ^ x) + d, fp4x8_to_f16(c.z, q2));
                        st_shared16((piece[3] ^ x) + d, fp4x8_to_f16(c.w, q3));
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive_at(full0 + 8 * s);
                    if (ahead) load(s);
                }
                fills ^= 1;
            }
        }
        if (!ok && lane == 0) raise_abort(sFlag);
    } else {
        // ============================================== softmax
        // TMEM lane l < 64 of a buffer holds row l, entries 0 .. 127 of the tile
        // (O: the first 128 channels of each 256), lane 64 + l the rest.
        const int quarter = warp & 3, ch = warp >> 2;              // ch: which half of the columns
        const uint32_t lane_q = (uint32_t)(quarter * 32) << 16;
        const int row = 32 * (quarter & 1) + lane;
        const int ent0 = 128 * (quarter >> 1) + 64 * ch;           // its 64 entries of a tile
        const int which = 2 * (quarter >> 1) + ch;                 // of the row's four threads
        const uint32_t p_bar = in_cta(smem_u32(bar_p), 0);
        uint8_t *p_row = sP + which * kQAtom;
        const float l2s = p.sm_scale * kLog2e;
        const float worst = l2s >= 0.f ? -INFINITY : INFINITY;     // a score that never is the largest logit
        uint32_t tile = 0;
        bool ok = true;
        for (; more && ok; more = w.next(p)) {
            const int r_tile = row_split(w);                     // of the tile's 128
            const int r0 = w.rt * kRowsPair + r_tile;
            const int n_rows = row_count(w);
            const int64_t row0 = w.gr.row0 + r0;
            if (tile == 0) {
                issue_q(p, sQ, row0, n_rows, tid);
                finish_q<0>(p, sQ, tid, in_cta(smem_u32(bar_q), 0));
                finish_q<1>(p, sQ, tid, in_cta(smem_u32(bar_q), 0));
            }
            if (tid < kRowsCta) sM[tid] = -INFINITY;
            soft_sync();
            float l = 0.f;
            const int n_tiles = w.k1 - w.k0;
            const int n_left = w.gr.n - w.k0 * kEnt;              // entries from the piece's first on
            for (int i = 0; i < n_tiles; ++i, ++tile) {
                const uint32_t tS = tmem + kColS + 128 * (tile & 1) + 64 * ch + lane_q;
                bool got = mbar_wait<true>(&bar_s[tile & 1], (tile >> 1) & 1, abort_flag);
                tc_fence_after();
                const int left = n_left - i * kEnt - ent0;        // entries of this thread's 64
                float m = sM[row];
                // the largest logit: of the scores if sm_scale >= 0, else of their negatives
                float hi = -INFINITY;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x[32];
                    tmem_ld32(tS + 32 * h, x);
                    tmem_wait_ld();
                    if (left < 64) {
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (32 * h + c >= left) x[c] = worst;
                    }
                    if (l2s >= 0.f) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) hi = fmaxf(hi, x[c]);
                    } else {
#pragma unroll
                        for (int c = 0; c < 32; ++c) hi = fmaxf(hi, -x[c]);
                    }
                }
                // (rounded up, and compared by its exact difference, so that P stays below 2^15
                // however far apart fp32's values are at these logits)
                const float top = hi == -INFINITY ? hi : __fmaf_ru(hi, fabsf(l2s), -kHead);
                // (a wait that gave up takes the same path, and the vote makes every thread
                // leave together)
                if (soft_any(top - m > kLazy || !got)) {
                    sRed[which * kRowsCta + row] = top;
                    ok = !soft_any(!got || *abort_flag);
                    if (!ok) break;
                    if (tid < kRowsCta) {
                        const float t = fmaxf(fmaxf(sRed[tid], sRed[kRowsCta + tid]),
                                              fmaxf(sRed[2 * kRowsCta + tid], sRed[3 * kRowsCta + tid]));
                        const float old = sM[tid];
                        const bool moves = t - old > kLazy;
                        sAlpha[tid] = !moves ? 1.f : old == -INFINITY ? 0.f : fast_exp2(old - t);
                        if (moves) sM[tid] = t;
                    }
                    soft_sync();
                    m = sM[row];
                    const float alpha = sAlpha[row];
                    if (i > 0) {
                        l *= alpha;
                        // O *= alpha, once the previous tile's products have completed
                        const bool done = __all_sync(0xffffffffu, mbar_wait<true>(bar_o, (tile - 1) & 1, abort_flag));
                        const bool moved = __any_sync(0xffffffffu, alpha != 1.f);
                        tc_fence_after();
                        if (done && moved) {
#pragma unroll 1
                            for (int c = 0; c < 4; ++c) {
                                float o[32];
                                const uint32_t ta = tmem + 128 * ch + 32 * c + lane_q;
                                tmem_ld32(ta, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] *= alpha;
                                tmem_st32(ta, o);
                            }
                            tmem_wait_st();
                        }
                        if (!done) raise_abort(sFlag);
                    }
                }
                // P is free once the previous tile's products have completed
                if (tile > 0 && !mbar_wait<true>(bar_o, (tile - 1) & 1, abort_flag)) raise_abort(sFlag);
                const float mref = m == -INFINITY ? 0.f : m;    // (no finite logit yet: e^-inf = 0, a NaN stays one)
                // (a warp whose 32 rows are all past the tile's leaves their P as it is: no row's O
                // depends on another's P)
                const int halves = 32 * (quarter & 1) < n_rows ? 2 : 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h >= halves) break;
                    float x[32];
                    tmem_ld32(tS + 32 * h, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const float2 y = fma_f32x2(make_float2(x[c], x[c + 1]), make_float2(l2s, l2s), make_float2(-mref, -mref));
                        x[c] = fast_exp2(y.x);
                        x[c + 1] = fast_exp2(y.y);
                    }
                    if (left < 64) {
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (32 * h + c >= left) x[c] = 0.f;
                    }
                    float2 sum[2] = {make_float2(x[0], x[1]), make_float2(x[2], x[3])};
#pragma unroll
                    for (int c = 4; c < 32; c += 4) {
                        sum[0] = add_f32x2(sum[0], make_float2(x[c], x[c + 1]));
                        sum[1] = add_f32x2(sum[1], make_float2(x[c + 2], x[c + 3]));
                    }
                    const float2 s2 = add_f32x2(sum[0], sum[1]);
                    l += s2.x + s2.y;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        *reinterpret_cast<uint4 *>(p_row + sw128((uint32_t)row, (uint32_t)(4 * h + c))) =
                            make_uint4(f32x2_to_f16x2(x[8 * c], x[8 * c + 1]), f32x2_to_f16x2(x[8 * c + 2], x[8 * c + 3]),
                                       f32x2_to_f16x2(x[8 * c + 4], x[8 * c + 5]),
                                       f32x2_to_f16x2(x[8 * c + 6], x[8 * c + 7]));
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_at(p_bar);
            }
            if (!ok) break;
            // ---- the piece's sums: complete rows are finished, others left for the join
            const bool whole = w.k0 == 0 && w.k1 == w.kt;
            const bool done = mbar_wait<true>(bar_o, (tile - 1) & 1, abort_flag);
            tc_fence_after();
            sRed[which * kRowsCta + row] = l;
            ok = !soft_any(!done || *abort_flag);
            if (!ok) break;
            l = (sRed[row] + sRed[kRowsCta + row]) + (sRed[2 * kRowsCta + row] + sRed[3 * kRowsCta + row]);
            const float m = l != l ? 0.f : sM[row];             // (a NaN row is not an empty one)
            const int chan = 256 * (quarter >> 1) + 128 * ch;
            const int64_t piece = 2 * (int64_t)pair + (w.k0 == 0 ? 1 : 0);
            Joined j{1.f, 0.f, 0.f};
            if (whole && row < n_rows)
                j = join_prev(m, l, p.prev_out != nullptr, p.prev_out ? p.prev_lse[row0 + row] : 0.f);
            soft_sync();                       // (sRed is read, and prev_lse, which may be lse itself)
            if (which == 0) {
                sRed[row] = j.prev;
                if (whole) {
                    if (row < n_rows && p.lse) p.lse[row0 + row] = j.lse;
                } else if (row < n_rows) {
                    float *ml = p.part_ml + piece * 2 * kRowsPair + r_tile + row;
                    ml[0] = m;
                    ml[kRowsPair] = l;
                }
            }
            soft_sync();
            // O goes through the warp's 4 KB of the (now free) P buffer, so that 8 lanes
            // read and write 32 consecutive channels of a row
            uint8_t *turn = sP + warp * 4096;
            const int r_base = 32 * (quarter & 1) + (lane >> 3), c_lane = chan + 4 * (lane & 7);
            const int mine = (n_rows - r_base + 3) / 4;       // of this lane's 8 rows r_base + 4 i
            const int64_t out0 = (row0 + r_base) * CSA2_D + c_lane;
            float *const part0 = p.part_o + (piece * kRowsPair + r_tile + r_base) * CSA2_D + c_lane;
            const int chunks = 32 * (quarter & 1) < n_rows ? 4 : 0;
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                float o[32];
                tmem_ld32(tmem + 128 * ch + 32 * c + lane_q, o);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<float4 *>(turn + sw128((uint32_t)lane, (uint32_t)k)) =
                        make_float4(o[4 * k] * j.own, o[4 * k + 1] * j.own, o[4 * k + 2] * j.own, o[4 * k + 3] * j.own);
                __syncwarp();
                float4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = *reinterpret_cast<const float4 *>(
                        turn + sw128((uint32_t)((lane >> 3) + 4 * i), (uint32_t)(lane & 7)));
                __syncwarp();
                if (whole) {
                    if (p.prev_out != nullptr) {
                        float4 pv[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)    // (a row without a partial result: weight 0, prev_out not read)
                            pv[i] = i < mine && sRed[r_base + 4 * i] != 0.f
                                        ? *reinterpret_cast<const float4 *>(p.prev_out + out0 + 4 * i * CSA2_D + 32 * c)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float pw = sRed[r_base + 4 * i];
                            v[i].x = fmaf(pv[i].x, pw, v[i].x); v[i].y = fmaf(pv[i].y, pw, v[i].y);
                            v[i].z = fmaf(pv[i].z, pw, v[i].z); v[i].w = fmaf(pv[i].w, pw, v[i].w);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < mine) store4<kOut>(p.out, out0 + 4 * i * CSA2_D + 32 * c, v[i].x, v[i].y, v[i].z, v[i].w);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < mine) *reinterpret_cast<float4 *>(part0 + 4 * i * CSA2_D + 32 * c) = v[i];
                }
            }
            tc_fence_before();
            soft_sync();                       // sRed, sM and O are read
        }
        // (the join is let in this late because its blocks fill whichever SMs end first, and
        // its first blocks would wait there two to an SM: 22.8 us instead of 21.8 for
        // 61 queries over five prompts when let in before the epilogue)
        pdl_trigger();
        if (!ok && lane == 0) raise_abort(sFlag);
    }
    // groups without entries
    if (sFound->empty && warp != kWarpsSoft + kWarpsProd)
        for (int g = pair; g < sFound->groups; g += p.pairs) {
            const Group gr = group_of(p, g);
            if (!gr.bad && gr.n == 0)
                empty_rows<kOut>(p, gr, (int)rank * 32 * (kWarpsSoft + kWarpsProd) + tid, 2 * 32 * (kWarpsSoft + kWarpsProd));
        }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) count_event(p.counters, CSA2_CNT_TIMEOUT);
    __syncwarp();
    // Neither CTA leaves (or gives TMEM back) while the other's tensor core may use
    // it; nothing is handed over in memory, so the arrival need not wait for the
    // stores on their way (release: 0.1 to 0.2 us more).
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
    if (warp == kWarpsSoft + kWarpsProd) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// Joins the pieces of the row tiles that lie in several pairs' runs, in the
// pairs' order, and the caller's partial result.  Pair c >= 1 answers for a
// tile when it is the first to begin inside it; its pieces are the second slot
// of pair c - 1 and the first of c, c + 1, ...  A thread takes 4 channels of a
// row; the pieces of a tile are dealt to `parts` threads each (1, 2 or 4), whose
// sums are added in order.  A block's item is 4 / parts whole rows, so that lse
// may be prev_lse itself.
template <int kOut>
__global__ void __launch_bounds__(kJoinThreads, 2) dense_join_kernel(DenseParams p)
{
    struct Tile { int c, pieces, row0, rows, item; };
    __shared__ Tile sTile[kDensePairsMax];
    __shared__ int sWarp[2][kJoinThreads / 32];
    __shared__ float sW[4][kMaxPieces];
    __shared__ float4 sO[kJoinThreads];
    __shared__ Joined sJ[4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // (the next kernel of the stream is let in only as these blocks finish: one of
    // this library's attention CTAs takes a whole SM, and waiting there it would
    // keep the SM from the blocks it waits for)
    pdl_wait();
    // the tiles to join (in order) and their work items; every thread looks at one pair
    auto log_parts = [](int pieces) { return pieces <= 4 ? 0 : pieces <= 8 ? 1 : 2; };
    Tile mine{};
    int items = 0;
    if (tid > 0 && tid < p.pairs) {
        const DenseBegin d = p.begin[tid];
        const int64_t b0 = tid * d.run;
        if (d.rows > 0 && b0 > d.first && b0 - d.run <= d.first) {
            // pair tid - 1's piece, and one of each pair that begins before d.last
            mine.c = tid;
            mine.pieces = (int)quotient(d.last + d.run - 1, d.run) - tid + 1;
            mine.row0 = d.row0;
            mine.rows = d.rows;
            items = ((d.rows << log_parts(mine.pieces)) + 3) >> 2;         // 4 / parts rows each
        }
    }
    const uint32_t has = __ballot_sync(0xffffffffu, items > 0);
    int upto = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) { sWarp[0][warp] = upto; sWarp[1][warp] = __popc(has); }
    __syncthreads();
    int before = 0, n = 0, total = 0, tiles = 0;
#pragma unroll
    for (int i = 0; i < (kDensePairsMax + 31) / 32; ++i) {
        const int a = sWarp[0][i], b = sWarp[1][i];
        if (i < warp) { before += a; n += b; }
        total += a;
        tiles += b;
    }
    if (items > 0) {
        mine.item = before + upto - items;
        sTile[n + __popc(has & ((1u << lane) - 1))] = mine;
    }
    __syncthreads();
    int at = 0;
    for (int item = blockIdx.x; item < total; item += gridDim.x) {
        while (at + 1 < tiles && sTile[at + 1].item <= item) ++at;
        const Tile t = sTile[at];
        const int lp = log_parts(t.pieces), parts = 1 << lp;
        const int part = tid >> (9 - lp);             // of the 512 >> lp threads (of 4 channels) side by side
        const int r0 = (item - t.item) << (2 - lp);   // the item's rows: r0 .. r0 + 4 / parts - 1
        const int r = r0 + ((tid & ((512 >> lp) - 1)) >> 7), ch = 4 * (tid & 127);
        const bool in = r < t.rows;
        const int64_t out_at = (int64_t)(t.row0 + r) * CSA2_D + ch;
        // piece i's slot: 2 (c - 1) + 1 for the first, 2 (c - 1 + i) for the others
        const uint32_t slot0 = 2u * (t.c - 1);
        auto slot = [&](int i) { return slot0 + (i == 0 ? 1u : 2u * i); };
        const float *src = p.part_o + r * CSA2_D + ch;
        auto load = [&](int i) {
            return in && i < t.pieces ? *reinterpret_cast<const float4 *>(src + slot(i) * (uint32_t)(kRowsPair * CSA2_D))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        // the first pieces and the caller's part are on their way before the weights
        // are known (without a partial result prev_out may hold anything: weight 0)
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = load(part + (k << lp));
        float4 pv = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.prev_out != nullptr && part == 0 && in) pv = *reinterpret_cast<const float4 *>(p.prev_out + out_at);
        __syncthreads();                              // (the last item's shared values are read)
        if (warp < (4 >> lp) && r0 + warp < t.rows) {
            const float prev = p.prev_out != nullptr ? p.prev_lse[t.row0 + r0 + warp] : 0.f;
            float m[3], l[3];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const int i = lane + 32 * k;
                const float *ml = p.part_ml + slot(i) * (2u * kRowsPair) + r0 + warp;
                m[k] = i < t.pieces ? ml[0] : -INFINITY;
                l[k] = i < t.pieces ? ml[kRowsPair] : 0.f;
            }
            float top = fmaxf(fmaxf(m[0], m[1]), m[2]), sum = 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const float wgt = m[k] == -INFINITY ? 0.f : fast_exp2(m[k] - top);
                sW[warp][lane + 32 * k] = wgt;
                sum = fmaf(l[k], wgt, sum);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) sJ[warp] = join_prev(top, sum, p.prev_out != nullptr, prev);
        }
        __syncthreads();
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        const float *const w = sW[r - r0];
        for (int i0 = part; i0 < t.pieces; i0 += 4 << lp) {
            if (i0 != part) {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = load(i0 + (k << lp));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + (k << lp);
                const float wgt = i < t.pieces ? w[i] : 0.f;
                o.x = fmaf(v[k].x, wgt, o.x); o.y = fmaf(v[k].y, wgt, o.y);
                o.z = fmaf(v[k].z, wgt, o.z); o.w = fmaf(v[k].w, wgt, o.w);
            }
        }
        if (lp > 0) {
            sO[tid] = o;
            __syncthreads();
            if (part == 0)
                for (int i = 1; i < parts; ++i) {
                    const float4 u = sO[(i << (9 - lp)) + tid];
                    o.x += u.x; o.y += u.y; o.z += u.z; o.w += u.w;
                }
        }
        if (part == 0 && in) {
            const Joined j = sJ[r - r0];
            if (j.prev == 0.f) pv = make_float4(0.f, 0.f, 0.f, 0.f);
            store4<kOut>(p.out, out_at, fmaf(pv.x, j.prev, o.x * j.own), fmaf(pv.y, j.prev, o.y * j.own),
                         fmaf(pv.z, j.prev, o.z * j.own), fmaf(pv.w, j.prev, o.w * j.own));
        }
        if (p.lse && tid < (4 >> lp) && r0 + tid < t.rows) p.lse[t.row0 + r0 + tid] = sJ[tid].lse;
    }
}

}  // namespace

template <int kOut>
static cudaError_t launch_dense_as(const DenseParams &p, cudaStream_t st)
{
    constexpr size_t smem = 1024 + kStages * kStage + kQBytes + kPBytes + 6 * kRowsCta * 4 + 24 * 8 + sizeof(Found);
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    // the shared-memory attribute is set once per device (a bit each; setting it twice does no harm)
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if ((done.load(std::memory_order_acquire) & bit) == 0) {
        e = cudaFuncSetAttribute(dense_attn_kernel<kOut>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_release);
    }
    e = launch_k(dense_attn_kernel<kOut>, dim3(2 * p.pairs), dim3(kThreads), smem, st, 2, p);
    if (e == cudaSuccess && p.pairs > 1)
        e = launch_k(dense_join_kernel<kOut>, dim3(4 * p.pairs), dim3(kJoinThreads), 0, st, 0, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_dense(const DenseParams &p, int out_type, cudaStream_t st)
{
    return out_type == CSA2_F32    ? launch_dense_as<CSA2_F32>(p, st)
           : out_type == CSA2_BF16 ? launch_dense_as<CSA2_BF16>(p, st)
                                   : launch_dense_as<CSA2_F16>(p, st);
}

}  // namespace csa2
