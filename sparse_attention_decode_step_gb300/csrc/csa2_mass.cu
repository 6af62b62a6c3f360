// csa2_mass.cu -- attention weights by entry: how much weight the queries of a group
// gave to each entry of its sequence, from the log sums that the attention left.
//
//     mass[j] = decay prev[j] + sum over rows r (query, head) that see j of
//               2^(l2s q_r . v_j - lse2_r),   l2s = sm_scale log2 e, lse2 = lse log2 e.
//
// The sum is over rows, so entries lie along the tensor core's M: one CTA takes 128
// entries at a time against a block of up to 128 rows,
//     S [128 entries x N rows] = K [128 x 512] . Q^T          (M 128, N 16 .. 128)
// and a thread of the epilogue, which holds one entry's row of S in TMEM, sums over
// its columns alone: no value crosses threads.  The block's queries stay in shared
// memory (128 KB) while the entries go by, dequantised (E2M1 x E4M3 is exact in f16)
// into a ring of 32 KB stages of 128 entries x 128 channels, four to a tile.  Which
// channels a stage holds is free as long as queries and entries agree: those that a
// lane of a producer has at once, so that every load is of whole 128-byte lines
// and still every lane works on every stage (see slot()).
//
// A weight is computed as r 2^(l2s x - m), with m = lse2 rounded to a whole number and
// r = 2^(m - lse2): the exponents that matter lie near zero then, and lse2's own
// rounding (2^-20 at 20) does not come in.  Sums are fp32.
//
// Groups of one block write mass themselves.  The blocks of larger ones leave their
// sums side by side in the workspace, which a second kernel adds in order: no atomics,
// results do not depend on the run.  A first kernel lays out the blocks; the work,
// counted in tiles of entries over all blocks, is divided into equal runs.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "csa2_attn_device.cuh"
#include "csa2_internal.h"

namespace csa2 {

namespace {

constexpr int kWarpsEpi = 4, kWarpsProd = 8;
constexpr int kThreads = 32 * (kWarpsEpi + kWarpsProd + 1);
constexpr int kRows = kMassRows, kEnt = kMassEntries;
constexpr int kStages = 3;
constexpr uint32_t kStage = 32768;                    // [2 atoms of 64 channels][128 entries][128 B]
constexpr uint32_t kAtom = 128 * 128;
constexpr uint32_t kQBytes = kRows * CSA2_D * 2;      // [4 stages][2 atoms][N rows][128 B]
constexpr int kBufs = 4;                              // S buffers of 128 TMEM columns
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
    int alone;           // the group's only block
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

__global__ void __launch_bounds__(kPlanThreads) mass_plan_kernel(MassParams p)
{
    __shared__ int64_t s_warp[kPlanThreads / 32];
    __shared__ int s_fall;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Space ws = space_of(p);
    pdl_wait();
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
            if (g >= fall || a.bad || ws.owner[a.seq] != g)
                count_event(p.counters, CSA2_CNT_BAD_INPUT);
            else
                mine = max(1, ((a.e - a.a) * p.H + kRows - 1) / kRows);
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
        Block r{};
        r.seq = a.seq;
        r.n_group = a.n;
        r.base = a.base;
        r.alone = nb == 1;
        r.causal = p.pos != nullptr;
        r.pos = r.causal ? p.pos[g] : 0;
        for (int i = lane; i < nb; i += 32) {
            r.k0 = i * kRows;
            r.rows = min(kRows, (a.e - a.a) * p.H - r.k0);
            r.row0 = a.a * p.H + r.k0;
            r.n = r.alone ? a.n : sees(p, r.causal, r.pos, a.n, (r.k0 + r.rows - 1) / p.H);
            ws.blocks[b0 + i] = r;
        }
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
// The 16 bytes (8 channels) c of a row of 64 lie in stage slot_stage(c), there in the
// 64-channel atom slot_atom(c), 16-byte piece slot_piece(c): lane l = 0 .. 7 of an
// entry's 128 bytes of codes (256 channels, half h) holds the pieces 4 l .. 4 l + 3 of that
// half; its first two go to stage 2 h, the others to 2 h + 1, as channels 16 l ..
__device__ __forceinline__ int slot_stage(int c) { return 2 * (c >> 5) + ((c >> 1) & 1); }
__device__ __forceinline__ int slot_atom(int c) { return (c >> 4) & 1; }
__device__ __forceinline__ int slot_piece(int c) { return 2 * ((c >> 2) & 3) + (c & 1); }

// A CTA's pieces of work in order: tiles k0 .. k1 of a block.
struct Work {
    Block blk;
    int b;
    int k0, k1;
    int64_t left;        // tiles after this piece

    __device__ __forceinline__ void take(const Space &ws, int at, int64_t tiles)
    {
        blk = ws.blocks[b];
        k0 = at;
        k1 = (int)min((int64_t)tiles_of(blk.n), at + tiles);
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

// A row without weight: its log sum is infinite.
__device__ __forceinline__ bool no_weight(float lse) { return fabsf(lse) > 0x1p29f; }

__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

// Blocks b0 .. b1 - 1 of the plan (b1 may lie behind the last).
__global__ void __launch_bounds__(kThreads, 1) mass_kernel(MassParams p, int b0, int b1)
{
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *sRing = smem;
    uint8_t *sQ = sRing + kStages * kStage;
    float2 *sRow = reinterpret_cast<float2 *>(sQ + kQBytes);         // [128] (m, r) of a row
    int *sSees = reinterpret_cast<int *>(sRow + kRows);              // [128]
    uint64_t *bar_full = reinterpret_cast<uint64_t *>(sSees + kRows);   // [3] stage filled
    uint64_t *bar_empty = bar_full + kStages;                        // [3] stage's MMAs done
    uint64_t *bar_s = bar_empty + kStages;                           // [4] S buffer complete
    uint64_t *bar_free = bar_s + kBufs;                              // [4] S buffer read
    uint64_t *bar_q = bar_free + kBufs;                              // queries stored
    uint64_t *bar_done = bar_q + 1;                                  // every MMA done
    int *sFlag = reinterpret_cast<int *>(bar_done + 1);              // [0] abort, [1] first block
    uint32_t *sTmem = reinterpret_cast<uint32_t *>(sFlag + 2);
    volatile int *abort_flag = sFlag;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) { mbar_init(&bar_full[i], kWarpsProd); mbar_init(&bar_empty[i], 1); }
        for (int i = 0; i < kBufs; ++i) { mbar_init(&bar_s[i], 1); mbar_init(&bar_free[i], kWarpsEpi); }
        mbar_init(bar_q, kWarpsProd);
        mbar_init(bar_done, 1);
        sFlag[0] = 0;
        fence_barrier_init();
    }
    if (warp == kWarpsEpi + kWarpsProd) {
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
    auto columns = [](const Block &b) { return max(16, (b.rows + 15) & ~15); };
    bool ok = true;

    if (warp == kWarpsEpi + kWarpsProd) {
        // ============================================== MMA issuer (the whole warp runs the loop, one lane issues)
        uint32_t elected;
        asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(elected));
        const uint32_t ring = __shfl_sync(0xffffffffu, smem_u32(sRing), 0), t0 = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dk = smem_desc(ring, 16, 1024, kLayoutSW128), dq = smem_desc(ring + kStages * kStage, 16, 1024, kLayoutSW128);
        uint32_t stage = 0, phase = 0, tile = 0, pieces = 0;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
            tc_fence_after();
        };
        for (; more && ok; more = w.next(ws), ++pieces) {
            const uint32_t n = (uint32_t)columns(w.blk), id = instr_desc(128, 0, 0, 0, 0, 0) | ((n >> 3) << 17);
            wait(bar_q, pieces & 1);
            for (int t = w.k0; t < w.k1 && ok; ++t, ++tile) {
                const uint32_t buf = tile % kBufs;
                if (tile >= kBufs) wait(&bar_free[buf], (tile / kBufs - 1) & 1);
#pragma unroll 1
                for (uint32_t j = 0; j < 4; ++j) {
                    wait(&bar_full[stage], phase);
                    if (!ok) break;
                    if (elected) {
#pragma unroll
                        for (uint32_t ks = 0; ks < 8; ++ks)
                            mma_f16(t0 + 128 * buf, dk + (stage * (kStage >> 4) + (ks >> 2) * (kAtom >> 4) + 2 * (ks & 3)),
                                    dq + ((2 * j + (ks >> 2)) * (n * 128 >> 4) + 2 * (ks & 3)), id, ks > 0 ? 1u : j);
                        mma_commit(&bar_empty[stage]);
                        if (j == 3) mma_commit(&bar_s[buf]);
                    }
                    __syncwarp();
                    if (++stage == kStages) { stage = 0; phase ^= 1; }
                }
            }
        }
        // every MMA has completed before TMEM and shared memory go back
        volatile int no_abort = 0;
        if (elected) mma_commit(bar_done);
        __syncwarp();
        if (!mbar_wait<true>(bar_done, 0, &no_abort)) ok = false;
    } else if (warp >= kWarpsEpi) {
        // ============================================== producers
        // Warp pw dequantises the entries 16 pw .. 16 pw + 15 of a tile, four at a time
        // (e4), eight lanes to an entry.  A lane's 16 code bytes feed two stages; the next
        // tile's are loaded as soon as their registers are free.
        const int pw = warp - kWarpsEpi, l = lane & 7, e4 = lane >> 3;
        const bool turn = l >= 4;              // (its atom's stores go in the other order: eight bank groups at every store)
        const int row = 16 * pw + e4;          // of entry u: row + 4 u
        uint32_t piece[2];                     // of entry u: ^ 64 where u is odd, + 512 u
#pragma unroll
        for (int j = 0; j < 2; ++j)
            piece[j] = smem_u32(sRing) + (l >> 2) * kAtom + row * 128u + (uint32_t)(((2 * (l & 3) + (j ^ (int)turn)) ^ (row & 7)) << 4);
        uint32_t stage = 0, phase = 1, tile = 0;
        uint4 gc[2][4];
        uint32_t gs[2][4];
        const bool paged = p.pages.table != nullptr;
        for (; more && ok; more = w.next(ws)) {
            const int32_t *const table = p.pages.table + (int64_t)w.blk.seq * p.pages.ld;      // (if paged)
            // a warp's 16 entries lie in one page
            auto page_of = [&](int t) {
                const int e = t * kEnt + 16 * pw;
                return paged && t < w.k1 && e < w.blk.n ? __ldg(table + (e >> p.pages.log)) : 0;
            };
            int page = page_of(w.k0);
            int left = 0;                      // entries from the lane's first on
            const uint8_t *c0 = nullptr, *s0 = nullptr;
            auto begin = [&](int t) {
                const int e = t * kEnt + 16 * pw;
                left = t < w.k1 ? w.blk.n - e - e4 : 0;
                int64_t r = (int64_t)w.blk.base + e;
                if (paged) {
                    if ((uint32_t)page >= p.pages.pages) {     // no page of the cache: nothing is read
                        if (lane == 0 && left > 0) count_event(p.counters, CSA2_CNT_BAD_INPUT);
                        left = 0;
                    }
                    r = ((int64_t)page << p.pages.log) + (e & ((1 << p.pages.log) - 1));
                    page = page_of(t + 1);
                }
                c0 = p.codes + (r + e4) * CSA2_CODE_BYTES + 16 * l;
                s0 = p.scales + (r + e4) * CSA2_SCALE_BYTES + 2 * l;
            };
            auto load = [&](int h) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    gc[h][u] = make_uint4(0, 0, 0, 0);
                    gs[h][u] = 0;
                    if (4 * u < left) {
                        gc[h][u] = __ldg(reinterpret_cast<const uint4 *>(c0 + 4 * u * CSA2_CODE_BYTES + 128 * h));
                        gs[h][u] = __ldg(reinterpret_cast<const uint16_t *>(s0 + 4 * u * CSA2_SCALE_BYTES + 16 * h));
                    }
                }
            };
            begin(w.k0);
            load(0);
            load(1);
            // ---- the block's queries, once the last block's products are done
            if (tile > 0) ok = __all_sync(0xffffffffu, mbar_wait<true>(&bar_s[(tile - 1) % kBufs], ((tile - 1) / kBufs) & 1, abort_flag));
            if (!ok) break;
            const int n = columns(w.blk);
            const uint4 *const q = reinterpret_cast<const uint4 *>(p.q) + (int64_t)w.blk.row0 * (CSA2_D / 8);
            for (int i0 = 32 * pw + lane; i0 < n * 64; i0 += 8 * 32 * kWarpsProd) {
                uint4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int i = i0 + k * 32 * kWarpsProd;
                    // (zeros for a row without weight: whatever its query holds stays out)
                    const bool in = i < w.blk.rows * 64 && !no_weight(__ldg(p.lse + w.blk.row0 + (i >> 6)));
                    v[k] = in ? __ldg(q + i) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int i = i0 + k * 32 * kWarpsProd, r = i >> 6, c = i & 63;
                    if (i >= n * 64) break;
                    if (p.q_type == CSA2_BF16)
                        v[k] = make_uint4(bf16x2_to_f16x2(v[k].x), bf16x2_to_f16x2(v[k].y), bf16x2_to_f16x2(v[k].z), bf16x2_to_f16x2(v[k].w));
                    *reinterpret_cast<uint4 *>(sQ + (2 * slot_stage(c) + slot_atom(c)) * n * 128 + sw128(r, slot_piece(c))) = v[k];
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_q);
            tile += w.k1 - w.k0;
            for (int t = w.k0; t < w.k1 && ok; ++t) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int h = j >> 1, x = j & 1;
                    ok = ok && __all_sync(0xffffffffu, mbar_wait<true>(&bar_empty[stage], phase, abort_flag));
                    if (!ok) break;
                    const uint32_t to = stage * kStage;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t sc = scale_pair((gs[h][u] >> (8 * x)) & 0xFFu);
                        uint32_t a = x ? gc[h][u].z : gc[h][u].x, b = x ? gc[h][u].w : gc[h][u].y;
                        if (turn) { const uint32_t z = a; a = b; b = z; }
                        const uint32_t at = to + 512 * u, odd = (u & 1) * 64;
                        st_shared16((piece[0] ^ odd) + at, fp4x8_to_f16(a, sc));
                        st_shared16((piece[1] ^ odd) + at, fp4x8_to_f16(b, sc));
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar_full[stage]);
                    if (++stage == kStages) { stage = 0; phase ^= 1; }
                    if (j == 1) { begin(t + 1); load(0); }
                    if (j == 3) load(1);
                }
            }
        }
    } else {
        // ============================================== epilogue: a thread has an entry
        const float l2s = p.sm_scale * kLog2e;
        const uint32_t lane_q = (uint32_t)(32 * warp) << 16;
        uint32_t tile = 0;
        for (; more && ok; more = w.next(ws)) {
            if (tid < kRows) {
                float m = 0.f, r = 0.f;        // (rows past the block's, or without a sum: no weight)
                int s = 0;
                if (tid < w.blk.rows) {
                    const float lse = p.lse[w.blk.row0 + tid];
                    if (!no_weight(lse)) {
                        m = rintf(lse * kLog2e);
                        r = exp2f(-fmaf(lse, kLog2e, -m));
                    }
                    s = sees(p, w.blk.causal, w.blk.pos, w.blk.n_group, (w.blk.k0 + tid) / p.H);
                }
                sRow[tid] = make_float2(m, r);
                sSees[tid] = s;
            }
            epi_sync();
            const int all = w.blk.rows > 0 ? sSees[0] : 0;        // entries that every row sees
            const int n = columns(w.blk);
            const int64_t part = (int64_t)(w.b - b0) * p.max_n;
            float *const mass = p.mass + (int64_t)w.blk.seq * p.ld_mass;
            const float *const prev = p.prev + (int64_t)w.blk.seq * p.ld_mass;
            for (int t = w.k0; t < w.k1; ++t, ++tile) {
                const uint32_t buf = tile % kBufs;
                ok = __all_sync(0xffffffffu, mbar_wait<true>(&bar_s[buf], (tile / kBufs) & 1, abort_flag));
                tc_fence_after();
                if (!ok) break;
                const int e = t * kEnt + tid;
                const bool whole = (t + 1) * kEnt <= all;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                for (int c0 = 0; c0 < n; c0 += 16) {
                    float x[16];
                    tmem_ld16(tmem + 128 * buf + c0 + lane_q, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; c += 2) {
                        const float4 row = *reinterpret_cast<const float4 *>(sRow + c0 + c);       // m, r, m, r
                        const float2 y = fma_f32x2(make_float2(x[c], x[c + 1]), make_float2(l2s, l2s), make_float2(-row.x, -row.z));
                        // (a NaN of a row that does not see the entry stays out)
                        const float a = fmaf(fast_exp2(y.x), row.y, sum[c & 2]), b = fmaf(fast_exp2(y.y), row.w, sum[(c & 2) + 1]);
                        if (whole || e < sSees[c0 + c]) sum[c & 2] = a;
                        if (whole || e < sSees[c0 + c + 1]) sum[(c & 2) + 1] = b;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_free[buf]);
                if (e >= w.blk.n) continue;
                const float s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
                if (w.blk.alone) mass[e] = p.prev ? fmaf(p.decay, prev[e], s) : s;
                else ws.parts[part + e] = s;
            }
            // (all leave together if a wait gave up; else the block's rows are read)
            ok = !epi_any(!ok);
        }
    }
    if (!ok && lane == 0) *abort_flag = 1;
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) count_event(p.counters, CSA2_CNT_TIMEOUT);
    if (warp == kWarpsEpi + kWarpsProd) {
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
        if (l - f < 2 || lo >= hi) continue;
        const int64_t e = (item - g * chunks) * kFinishThreads + threadIdx.x;
        const Block &any = ws.blocks[f];
        if (e >= any.n_group) continue;
        float *const at = p.mass + any.seq * p.ld_mass + e;
        float s = 0.f;
        for (int b = lo; b < hi; ++b)
            if (e < ws.blocks[b].n) s += ws.parts[(int64_t)(b - b0) * p.max_n + e];
        if (lo > f) *at += s;
        else *at = p.prev ? fmaf(p.decay, p.prev[any.seq * p.ld_mass + e], s) : s;
    }
}

}  // namespace

// Parts are kept for so many blocks at a time that they take up to 256 MB; more blocks
// go in turns.
MassPlan mass_plan(int batch, int ng, int nq, int H, int64_t max_n)
{
    MassPlan pl{};
    const int64_t blocks = ((int64_t)nq * H + kRows - 1) / kRows + ng;
    pl.parts = std::max<int64_t>(64, (256ll << 20) / 4 / std::max<int64_t>(1, max_n));
    pl.blocks = blocks;
    const int64_t units = blocks * ((max_n + kEnt - 1) / kEnt);
    pl.ctas = (int)std::max<int64_t>(1, std::min<int64_t>(device_sm_count(), units));
    pl.off_groups = align_up((size_t)(blocks + 1) * sizeof(Block), 256);
    pl.off_parts = pl.off_groups + align_up(((size_t)ng + 1 + batch) * 4, 256);
    // (a single block's group has no parts, and there is none without 129 rows)
    const bool any = (int64_t)nq * H > kRows;
    pl.total = pl.off_parts + (any ? (size_t)std::min(pl.parts, blocks) * max_n * 4 : 0);
    return pl;
}

cudaError_t launch_mass(const MassParams &p, cudaStream_t st)
{
    constexpr size_t smem = 1024 + kStages * kStage + kQBytes + kRows * 12 + (2 * kStages + 2 * kBufs + 2) * 8 + 16;
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
    e = launch_k(mass_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, 0, p);
    const int64_t items = p.ng * ((p.max_n + kFinishThreads - 1) / kFinishThreads);
    for (int64_t b0 = 0; b0 < p.plan.blocks && e == cudaSuccess; b0 += p.plan.parts) {
        const int b1 = (int)std::min(b0 + p.plan.parts, p.plan.blocks);
        e = launch_k(mass_kernel, dim3(p.plan.ctas), dim3(kThreads), smem, st, 0, p, (int)b0, b1);
        if (e == cudaSuccess && (int64_t)p.nq * p.H > kRows && items > 0)
            e = launch_k(mass_finish_kernel, dim3((unsigned)std::min<int64_t>(items, device_sm_count() * 8)), dim3(kFinishThreads), 0, st, 0,
                         p, (int)b0, b1);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa2
