// csa2_dense.cu -- attention of groups of queries over whole sequences of the
// FP4 latent cache: a prompt that many sequences share (read once for all of
// them), or an encoder's entries attended by a decoder sequence's queries.
//
// Every row (query, head) of group g sees the entries j < n_g of one sequence:
//     x_j = sm_scale q . v_j,   M = max(max_j x_j, lse_prev),
//     out = (sum_j e^(x_j - M) v_j + e^(lse_prev - M) out_prev) / L,
//     lse = M + log L,  L = the same sum without v_j and out_prev.
//
// One CTA = 64 rows of a group x a range of 128-entry tiles of its sequence,
// laid out with the ENTRIES as the MMA's M = 128:
//     S^T [128 entries x 64 rows] = V [128 x 512] . Q^T
//     O^T [512 ch x 64 rows]     += V^T [512 x 128] . P^T
// V is dequantised once per tile into 128-byte-swizzled f16 shared memory
// (E2M1 x E4M3 is exact in f16); both products read the same bytes.  S^T, O^T
// and the running row sums live in tensor memory, all sums in fp32; P is
// rounded to f16 (relative 2^-11; at most 256 with the lazy rescaling below).
// Warps 0..15 dequantise and run the softmax, warp 16 issues the MMAs.  The
// reference maximum of a row moves only when a logit exceeds it by 8 (log2
// units).  A row tile's entries are divided over `splits` CTAs, whose partial
// results a second kernel joins in a fixed order (no atomics).
#include <cuda_fp16.h>

#include "csa2_attn_device.cuh"
#include "csa2_internal.h"

namespace csa2 {

namespace {

constexpr int kDThreads = 544;                 // warps 0..15 workers, warp 16 MMA issuer
constexpr int kDWorkers = 512;
constexpr int kDWarps = 16;
constexpr int kTileN = 128;                    // entries per tile (MMA M)
constexpr int kTileR = kDenseRows;             // rows per CTA (MMA N)
constexpr uint32_t kDV = kTileN * CSA2_D * 2;  // 128 KB
constexpr uint32_t kDQ = kTileR * CSA2_D * 2;  // 64 KB
constexpr uint32_t kDP = kTileN * kTileR * 2;  // 16 KB
constexpr uint32_t kDVAtom = kTileN * 128;
constexpr uint32_t kDQAtom = kTileR * 128;
constexpr float kLazy = 8.0f;                  // log2 units
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

static_assert(kTileR == 64, "lane and column maps below");

// What a group asks for.  bad: its arguments are out of contract and its rows
// are left as they are.
struct Group {
    int64_t base;
    int64_t row0;        // first row (query * H)
    int64_t rows;
    int n;
    bool bad;
};

__device__ __forceinline__ Group group_of(const DenseParams &p, int g)
{
    Group r{};
    const int b = p.g_seq[g], a = p.g_off[g], e = p.g_off[g + 1];
    r.bad = b < 0 || b >= p.batch || a < 0 || e < a || e > p.nq;
    if (r.bad) return r;
    const int64_t len = p.seq_len[b];
    const int64_t n = p.g_len ? (int64_t)p.g_len[g] : len;
    r.base = p.seq_base[b];
    r.bad = n < 0 || n > len || n > p.max_n || r.base < 0 || r.base + n > p.cap;
    if (r.bad) return r;
    r.n = (int)n;
    r.row0 = (int64_t)a * p.H;
    r.rows = (int64_t)(e - a) * p.H;
    return r;
}

// The group that row tile `tile` (counted over all groups) belongs to, and the
// tile's number within it; found by one warp.  false: past the last tile.
// count_bad: count the groups that are out of contract.
__device__ __forceinline__ bool find_tile(const DenseParams &p, int64_t tile, int lane, bool count_bad, int *g_out,
                                          int *t_out)
{
    int64_t before = 0;
    bool found = false;
    for (int g0 = 0; g0 < p.ng; g0 += 32) {
        const int g = g0 + lane;
        int64_t mine = 0;
        if (g < p.ng) {
            const Group gr = group_of(p, g);
            if (gr.bad) {
                if (count_bad) count_event(p.counters, CSA2_CNT_BAD_INPUT);
            } else {
                mine = (gr.rows + kTileR - 1) / kTileR;
            }
        }
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, before + upto > tile);
        if (hit != 0u && !found) {
            const int l = __ffs(hit) - 1;
            const int64_t first = before + __shfl_sync(0xffffffffu, upto - mine, l);
            *g_out = g0 + l;
            *t_out = (int)(tile - first);
            found = true;
            if (!count_bad) return true;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return found;
}

__device__ __forceinline__ void dworkers_sync()
{
    asm volatile("bar.sync 1, %0;" ::"n"(kDWorkers) : "memory");
}

__device__ __forceinline__ bool dworkers_and(bool v)
{
    uint32_t r;
    asm volatile(
        "{\n"
        ".reg .pred pin, pout;\n"
        "setp.ne.u32 pin, %1, 0;\n"
        "bar.red.and.pred pout, 1, %2, pin;\n"
        "selp.u32 %0, 1, 0, pout;\n"
        "}\n"
        : "=r"(r)
        : "r"((uint32_t)v), "n"(kDWorkers)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void store_out(void *out, int type, int64_t at, float v)
{
    if (type == CSA2_F32) static_cast<float *>(out)[at] = v;
    else if (type == CSA2_BF16) static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v);
    else static_cast<__half *>(out)[at] = __float2half_rn(v);
}

// A row's partial softmax (m in log2 units, l) joined with the caller's
// partial result: the weights of the two, and the joint lse.
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

__global__ void __launch_bounds__(kDThreads, 1) dense_attn_kernel(DenseParams p)
{
    const int split = (int)(blockIdx.x % (unsigned)p.splits);
    const int64_t tile_id = blockIdx.x / (unsigned)p.splits;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *sV = smem;                        // [8 atoms][128 entries][128 B]
    uint8_t *sQ = sV + kDV;                    // [8 atoms][64 rows][128 B]
    uint8_t *sP = sQ + kDQ;                    // [128 entries][64 rows] f16
    float *sRed = reinterpret_cast<float *>(sP + kDP);   // [4 quarters][64 rows]
    float *sM = sRed + 4 * 64;                 // reference max per row (log2 units)
    float *sAlpha = sM + 64;
    float *sL = sAlpha + 64;
    float *sOwn = sL + 64;                     // weight of the row's own sums in the output
    float *sPrev = sOwn + 64;                  // weight of the caller's partial result
    uint64_t *bars = reinterpret_cast<uint64_t *>(sPrev + 64);
    uint64_t *bar_v = bars;                    // [2]: V channel half h stored
    uint64_t *bar_o = bars + 2;                // [2]: PV channel blocks 2h, 2h + 1 done
    uint64_t *bar_s = bars + 4, *bar_p = bars + 5, *bar_done = bars + 6, *bar_q = bars + 7;
    int *sFlag = reinterpret_cast<int *>(bars + 8);      // [0] abort [1] rescale [2] need max
    int *sTile = sFlag + 4;                    // [0] found [1] group [2] tile of the group
    uint32_t *sTmem = reinterpret_cast<uint32_t *>(sTile + 4);
    volatile int *abort_flag = sFlag;

    if (tid == 0) {
        for (int c = 0; c < 2; ++c) {
            mbar_init(&bar_v[c], kDWarps);
            mbar_init(&bar_o[c], 1);
        }
        mbar_init(bar_s, 1);
        mbar_init(bar_p, kDWarps);
        mbar_init(bar_done, 1);
        mbar_init(bar_q, 1);
        for (int i = 0; i < 4; ++i) sFlag[i] = 0;
        fence_barrier_init();
    }
    if (tid < 64) { sM[tid] = -INFINITY; sAlpha[tid] = 1.f; sL[tid] = 0.f; }
    if (warp == 0) { tmem_alloc(sTmem, 512); tmem_relinquish(); }
    pdl_wait();
    pdl_trigger();
    if (warp == 1) {
        int g = 0, t = 0;
        const bool ok = find_tile(p, tile_id, lane, split == 0 && tile_id == 0, &g, &t);
        if (lane == 0) { sTile[0] = ok; sTile[1] = g; sTile[2] = t; }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *sTmem;
    const bool found = sTile[0] != 0;
    Group gr{};
    if (found) gr = group_of(p, sTile[1]);
    const int64_t row0 = gr.row0 + (int64_t)sTile[2] * kTileR;
    const int n_rows = found ? (int)min((int64_t)kTileR, gr.rows - (int64_t)sTile[2] * kTileR) : 0;
    const int all_tiles = (gr.n + kTileN - 1) / kTileN;
    const int tps = (all_tiles + p.splits - 1) / p.splits;
    const int t_begin = min(all_tiles, split * tps);
    const int n_tiles = found ? min(all_tiles, t_begin + tps) - t_begin : 0;
    const int e_begin = t_begin * kTileN;                       // first entry of this CTA
    const int e_end = min(gr.n, (t_begin + n_tiles) * kTileN);  // one past its last

    const uint32_t quarter = (uint32_t)(warp & 3);
    const int ent = (int)(quarter * 32 + lane);       // softmax: entry of the tile = TMEM lane
    const int r0 = 16 * (warp >> 2);                  // softmax: rows r0 .. r0 + 15
    const uint32_t lane_q = (quarter * 32u) << 16;
    const uint32_t tS = tmem, tO = tmem + 64, tL = tmem + 320 + (uint32_t)(r0 & 63) + lane_q;

    // ---- loads: warp w fills entries 8 w .. 8 w + 7 of a tile, 8 lanes per
    // entry; register slot 2 h + x holds entry 4 x + (lane >> 3), channels
    // 256 h + 32 sub .. + 31
    const int sub = lane & 7, rho = sub >> 1;
    uint4 gc[4];
    uint32_t gsc[4];
    auto load_half = [&](int tile, int h) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int e = e_begin + tile * kTileN + 8 * warp + 4 * x + (lane >> 3);
            gc[2 * h + x] = make_uint4(0, 0, 0, 0);
            gsc[2 * h + x] = 0;
            if (e < e_end) {
                const int64_t r = gr.base + e;
                gc[2 * h + x] = __ldg(reinterpret_cast<const uint4 *>(p.codes + r * CSA2_CODE_BYTES) + 8 * h + sub);
                gsc[2 * h + x] = __ldg(reinterpret_cast<const uint16_t *>(p.scales + r * CSA2_SCALE_BYTES) + 8 * h + sub);
            }
        }
    };
    // channel half h of this warp's entries into sV (entries past the end are
    // zero); the pieces are rotated so that 8 lanes hit 8 bank groups
    auto store_half = [&](int h) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int t = 2 * h + x, r = 8 * warp + 4 * x + (lane >> 3);
            const uint32_t p0 = scale_pair(gsc[t] & 0xFFu), p1 = scale_pair((gsc[t] >> 8) & 0xFFu);
            uint32_t w[4] = {gc[t].x, gc[t].y, gc[t].z, gc[t].w};
            uint32_t sp[4] = {p0, p0, p1, p1};
            if (rho & 1) {
                const uint32_t w0 = w[0], s0 = sp[0];
                w[0] = w[1]; w[1] = w[2]; w[2] = w[3]; w[3] = w0;
                sp[0] = sp[1]; sp[1] = sp[2]; sp[2] = sp[3]; sp[3] = s0;
            }
            if (rho & 2) {
                uint32_t a = w[0], b = w[1];
                w[0] = w[2]; w[1] = w[3]; w[2] = a; w[3] = b;
                a = sp[0]; b = sp[1];
                sp[0] = sp[2]; sp[1] = sp[3]; sp[2] = a; sp[3] = b;
            }
            uint8_t *dst = sV + (4 * h + (sub >> 1)) * kDVAtom;
#pragma unroll
            for (int m = 0; m < 4; ++m)
                *reinterpret_cast<uint4 *>(dst + sw128((uint32_t)r, (uint32_t)(4 * (sub & 1) + ((m + rho) & 3)))) =
                    fp4x8_to_f16(w[m], sp[m]);
        }
    };

    if (n_tiles > 0) {
        // ---- Q: raw 16-bit rows land in the V tile, then go as f16 into the
        // swizzled sQ (rows past the tile's are zero)
        if (warp < kDWarps) { load_half(0, 0); load_half(0, 1); }
        const uint32_t qbytes = (uint32_t)n_rows * CSA2_D * 2;
        if (tid == 0) {
            mbar_arrive_expect_tx(bar_q, qbytes);
            bulk_load(sV, p.q + row0 * CSA2_D, qbytes, bar_q);
        }
        volatile int no_abort = 0;
        if (!mbar_wait(bar_q, 0, &no_abort)) sFlag[0] = 1;
        for (int i = tid; i < kTileR * (CSA2_D / 8); i += kDThreads) {
            const int r = i / (CSA2_D / 8), c8 = i % (CSA2_D / 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < n_rows) {
                v = *reinterpret_cast<const uint4 *>(sV + r * 1024 + c8 * 16);
                if (p.q_type == CSA2_BF16)
                    v = make_uint4(bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y), bf16x2_to_f16x2(v.z),
                                   bf16x2_to_f16x2(v.w));
            }
            *reinterpret_cast<uint4 *>(sQ + (c8 >> 3) * kDQAtom + sw128(r, c8 & 7)) = v;
        }
        fence_async_smem();
    }
    __syncthreads();

    if (n_tiles > 0 && warp == kDWarps) {
        // ============================================== MMA issuer
        if (lane == 0) {
            const uint32_t id_qk = instr_desc(128, kTileR, 0, 0, 0, 0);
            const uint32_t id_pv = instr_desc(128, kTileR, 0, 0, 1, 1);
            const uint32_t v0 = smem_u32(sV), q0 = smem_u32(sQ), p0 = smem_u32(sP);
            for (int i = 0; i < n_tiles; ++i) {
                bool run = true;
                for (int h = 0; h < 2 && run; ++h) {
                    if (!mbar_wait<true>(&bar_v[h], i & 1, abort_flag)) { run = false; break; }
                    tc_fence_after();
#pragma unroll
                    for (int k16 = 0; k16 < 16; ++k16) {
                        const int ks = 16 * h + k16;
                        mma_f16(tS, smem_desc(v0 + (ks >> 2) * kDVAtom + (ks & 3) * 32, 16, 1024, kLayoutSW128),
                                smem_desc(q0 + (ks >> 2) * kDQAtom + (ks & 3) * 32, 16, 1024, kLayoutSW128), id_qk,
                                ks > 0);
                    }
                }
                if (!run) { *abort_flag = 1; break; }
                mma_commit(bar_s);
                if (!mbar_wait<true>(bar_p, i & 1, abort_flag)) { *abort_flag = 1; break; }
                tc_fence_after();
#pragma unroll
                for (int mb = 0; mb < 4; ++mb) {
#pragma unroll
                    for (int ks = 0; ks < kTileN / 16; ++ks)
                        mma_f16(tO + 64 * mb, smem_desc(v0 + 2 * mb * kDVAtom + ks * 2048, kDVAtom, 1024, kLayoutSW128),
                                smem_desc(p0 + ks * 2048, kDVAtom, 1024, kLayoutSW128), id_pv,
                                (i > 0 || ks > 0) ? 1u : 0u);
                    if (mb & 1) mma_commit(&bar_o[mb >> 1]);
                }
            }
            mma_commit(bar_done);       // once every MMA issued above has completed
        }
    } else if (n_tiles > 0) {
        // ============================================== 16 worker warps
        const float l2s = p.sm_scale * kLog2e;
        {
            float z[16];
#pragma unroll
            for (int h = 0; h < 16; ++h) z[h] = 0.f;
            tmem_st16(tL, z);
            tmem_wait_st();
        }
        bool ok = !sFlag[0];
        for (int i = 0; i < n_tiles && ok; ++i) {
            const bool valid = e_begin + i * kTileN + ent < e_end;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                bool got = true;
                if (i > 0) {
                    got = __all_sync(0xffffffffu, mbar_wait<true>(&bar_o[h], (i - 1) & 1, abort_flag));
                    tc_fence_after();
                }
                if (got) store_half(h);
                else ok = false;
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_v[h]);
            }
            const bool more = i + 1 < n_tiles;
            if (more) load_half(i + 1, 0);

            // ---- softmax of this entry, rows r0 .. r0 + 15
            const bool got_s = ok && mbar_wait<true>(bar_s, i & 1, abort_flag);
            tc_fence_after();
            float x[16];
            if (got_s) {
                tmem_ld16(tS + lane_q + (uint32_t)r0, x);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int h = 0; h < 16; ++h) x[h] = 0.f;
            }
            bool over = false;
#pragma unroll
            for (int h4 = 0; h4 < 4; ++h4) {
                const float4 m4 = reinterpret_cast<const float4 *>(sM + r0)[h4];
                const float mm[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int h = 4 * h4 + j;
                    x[h] = valid ? x[h] * l2s : -INFINITY;
                    over |= x[h] > mm[j] + kLazy;
                }
            }
            if (over) sFlag[2] = i + 1;
            ok = dworkers_and(got_s);
            if (!ok) {
                if (tid == 0) *abort_flag = 1;
                break;
            }
            if (sFlag[2] == i + 1) {
                float r[16];
#pragma unroll
                for (int h = 0; h < 16; ++h) r[h] = x[h];
                warp_reduce16<true>(r, lane);
                if (lane < 16) sRed[quarter * 64 + r0 + lane] = r[0];
                dworkers_sync();
                if (tid < 64) {
                    const float tmax = fmaxf(fmaxf(sRed[tid], sRed[64 + tid]), fmaxf(sRed[128 + tid], sRed[192 + tid]));
                    const float m_old = sM[tid];
                    float alpha = 1.f;
                    if (tmax > m_old + kLazy) {
                        alpha = (m_old == -INFINITY) ? 0.f : fast_exp2(m_old - tmax);
                        sM[tid] = tmax;
                        if (i > 0) sFlag[1] = 1;
                    }
                    sAlpha[tid] = alpha;
                }
                dworkers_sync();
                if (sFlag[1] != 0) {
                    // O^T and the running sums *= alpha per row; the previous tile's PV
                    // has completed (both of its barriers were waited above)
                    float al[16];
#pragma unroll
                    for (int h = 0; h < 16; ++h) al[h] = sAlpha[r0 + h];
                    float o[16];
                    tmem_ld16(tL, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int h = 0; h < 16; ++h) o[h] *= al[h];
                    tmem_st16(tL, o);
#pragma unroll 1
                    for (int mb = 0; mb < 4; ++mb) {
                        const uint32_t ta = tO + 64 * mb + (uint32_t)r0 + lane_q;
                        tmem_ld16(ta, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int h = 0; h < 16; ++h) o[h] *= al[h];
                        tmem_st16(ta, o);
                    }
                    tmem_wait_st();
                }
                dworkers_sync();
                if (tid == 0) sFlag[1] = 0;
            }
#pragma unroll
            for (int h = 0; h < 16; ++h) {
                // (no finite logit yet: e^-inf = 0 for all, and a NaN stays one)
                const float mm = sM[r0 + h];
                x[h] = fast_exp2(x[h] - (mm == -INFINITY ? 0.f : mm));
            }
#pragma unroll
            for (int c = 0; c < 2; ++c)
                *reinterpret_cast<uint4 *>(sP + sw128((uint32_t)ent, (uint32_t)(r0 / 8 + c))) =
                    make_uint4(f32x2_to_f16x2(x[8 * c], x[8 * c + 1]), f32x2_to_f16x2(x[8 * c + 2], x[8 * c + 3]),
                               f32x2_to_f16x2(x[8 * c + 4], x[8 * c + 5]), f32x2_to_f16x2(x[8 * c + 6], x[8 * c + 7]));
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_p);
            if (more) load_half(i + 1, 1);
            float o[16];
            tmem_ld16(tL, o);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 16; ++h) o[h] += x[h];
            tmem_st16(tL, o);
            tmem_wait_st();
        }
        if (!ok) *abort_flag = 1;
    }
    if (n_tiles > 0) {
        volatile int no_abort = 0;
        if (!mbar_wait<true>(bar_done, 0, &no_abort)) *abort_flag = 1;
        tc_fence_after();
        if (warp < kDWarps) {
            float l[16];
            tmem_ld16(tL, l);
            tmem_wait_ld();
            warp_reduce16<false>(l, lane);
            if (lane < 16) sRed[quarter * 64 + r0 + lane] = l[0];
        }
    }
    __syncthreads();
    const bool failed = *abort_flag != 0;
    if (tid == 0 && failed) count_event(p.counters, CSA2_CNT_TIMEOUT);
    const bool any = n_tiles > 0 && !failed;
    if (tid < 64) {
        const float l = any ? (sRed[tid] + sRed[64 + tid]) + (sRed[128 + tid] + sRed[192 + tid]) : 0.f;
        const float m = !any ? -INFINITY : l != l ? 0.f : sM[tid];     // (a NaN row is not an empty one)
        if (p.splits > 1) {
            if (found) {
                float *ml = p.part_ml + (tile_id * p.splits + split) * 128;
                ml[tid] = m;
                ml[64 + tid] = l;
            }
            sOwn[tid] = 1.f;
        } else if (tid < n_rows) {
            const Joined j = join_prev(m, l, p.prev_out != nullptr, p.prev_out ? p.prev_lse[row0 + tid] : 0.f);
            sOwn[tid] = j.own;
            sPrev[tid] = j.prev;
            if (p.lse) p.lse[row0 + tid] = j.lse;
        }
    }
    __syncthreads();
    if (found && warp < kDWarps && (p.splits == 1 || any)) {
        // lane = channel 128 mb + 32 quarter + lane, 16 rows each
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {
            float o[16];
            if (any) {
                tmem_ld16(tO + 64 * mb + (uint32_t)r0 + lane_q, o);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int h = 0; h < 16; ++h) o[h] = 0.f;
            }
            const int c = 128 * mb + ent;
            if (p.splits > 1) {
                float *dst = p.part_o + ((tile_id * p.splits + split) * 64 + r0) * CSA2_D + c;
#pragma unroll
                for (int h = 0; h < 16; ++h) dst[h * CSA2_D] = o[h];
            } else {
#pragma unroll
                for (int h = 0; h < 16; ++h) {
                    if (r0 + h >= n_rows) break;
                    const int64_t at = (row0 + r0 + h) * CSA2_D + c;
                    float v = any ? o[h] * sOwn[r0 + h] : 0.f;
                    const float pw = sPrev[r0 + h];
                    if (pw != 0.f) v = fmaf(p.prev_out[at], pw, v);
                    store_out(p.out, p.out_type, at, v);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the splits of each row tile and the caller's partial result, in split
// order.  A CTA takes 4 rows, 128 threads (4 channels each) per row.
__global__ void __launch_bounds__(512) dense_join_kernel(DenseParams p)
{
    __shared__ int sTile[3];
    const int64_t tile_id = blockIdx.x / (kTileR / 4);
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (tid < 32) {
        int g = 0, t = 0;
        const bool ok = find_tile(p, tile_id, tid, false, &g, &t);
        if (tid == 0) { sTile[0] = ok; sTile[1] = g; sTile[2] = t; }
    }
    __syncthreads();
    if (!sTile[0]) return;
    const Group gr = group_of(p, sTile[1]);
    const int r = 4 * (int)(blockIdx.x % (kTileR / 4)) + (tid >> 7), c = 4 * (tid & 127);
    const int64_t in_group = (int64_t)sTile[2] * kTileR + r;
    if (in_group >= gr.rows) return;
    const int64_t row = gr.row0 + in_group;
    const float *ml = p.part_ml + tile_id * p.splits * 128 + r;
    float m = -INFINITY;
    for (int s = 0; s < p.splits; ++s) m = fmaxf(m, ml[s * 128]);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const float *src = p.part_o + (tile_id * p.splits * 64 + r) * CSA2_D + c;
    for (int s = 0; s < p.splits; ++s) {
        const float ms = ml[s * 128];
        if (ms == -INFINITY) continue;
        const float w = fast_exp2(ms - m);
        l = fmaf(ml[s * 128 + 64], w, l);
        const float4 v = *reinterpret_cast<const float4 *>(src + (int64_t)s * 64 * CSA2_D);
        o.x = fmaf(v.x, w, o.x); o.y = fmaf(v.y, w, o.y); o.z = fmaf(v.z, w, o.z); o.w = fmaf(v.w, w, o.w);
    }
    const Joined j = join_prev(m, l, p.prev_out != nullptr, p.prev_out ? p.prev_lse[row] : 0.f);
    float4 pv = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j.prev != 0.f) pv = *reinterpret_cast<const float4 *>(p.prev_out + row * CSA2_D + c);
    const float v[4] = {fmaf(pv.x, j.prev, o.x * j.own), fmaf(pv.y, j.prev, o.y * j.own),
                        fmaf(pv.z, j.prev, o.z * j.own), fmaf(pv.w, j.prev, o.w * j.own)};
#pragma unroll
    for (int i = 0; i < 4; ++i) store_out(p.out, p.out_type, row * CSA2_D + c + i, v[i]);
    if (p.lse && c == 0) p.lse[row] = j.lse;
}

}  // namespace

cudaError_t launch_dense(const DenseParams &p, cudaStream_t st)
{
    const size_t smem = 1024 + kDV + kDQ + kDP + (4 + 5) * 64 * 4 + 8 * 8 + 8 * 4 + 16;
    cudaError_t e = cudaFuncSetAttribute(dense_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_k(dense_attn_kernel, dim3((unsigned)p.splits * p.tiles), dim3(kDThreads), smem, st, 0, p);
    if (e == cudaSuccess && p.splits > 1)
        e = launch_k(dense_join_kernel, dim3((unsigned)(kTileR / 4) * p.tiles), dim3(512), 0, st, 0, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa2
