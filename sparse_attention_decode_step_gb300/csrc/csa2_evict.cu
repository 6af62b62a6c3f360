// csa2_evict.cu -- eviction: the entries of a sequence with the largest accumulated
// attention weight (its first and last ones in any case) are copied, in order, to
// other rows.
//
// Three steps on the stream: the selection's keys (the weights, and above infinity
// what stays in any case, so that ties and order are the top-k's: the lower entry
// first), the library's top-k over them, and the copy.  Nothing is moved within a
// sequence, which would have to wait for its own reads: every kept row is read once
// and written once.
#include <algorithm>

#include "csa2_device.cuh"
#include "csa2_internal.h"

namespace csa2 {

namespace {

constexpr int kThreads = 256;
constexpr int kKeysPerThread = 8;

// Whether b's entries 0 .. n-1 have rows in c.
__device__ __forceinline__ bool has_rows(const csa2_cache &c, const PageMap &m, int b, int64_t n)
{
    if (m.table != nullptr) return n <= m.ld << m.log;
    const int64_t base = c.seq_base[b];
    return base >= 0 && base + n <= c.cap;
}

// Keys, and for each sequence to cut its entries (0 for one that is skipped) and
// whether it is skipped.  blockIdx.y: position in `seq`.
__global__ void __launch_bounds__(kThreads) evict_keys_kernel(EvictParams p, float *keys, int64_t ld, int32_t *n_valid, int32_t *skip)
{
    pdl_wait();
    pdl_trigger();
    const int s = blockIdx.y;
    const int b = p.seq ? p.seq[s] : s;
    bool bad = b < 0 || b >= p.src.batch;
    int64_t n = 0;
    if (!bad) {
        n = p.src.seq_len[b];
        bad = n < 0 || n > p.max_n || !has_rows(p.src, p.src_pages, b, n);
    }
    const int64_t left = min(n, (int64_t)p.keep);
    bool full = false;
    if (!bad) {
        full = !has_rows(p.dst, p.dst_pages, b, left);
        if (!full && p.dst_pages.table == nullptr) full = p.dst.seq_base[b] + left > p.dst.seq_base[b + 1];
    }
    if (bad || full) n = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        n_valid[s] = (int32_t)n;
        skip[s] = bad || full;
        if (bad) count_event(p.counters, CSA2_CNT_BAD_INPUT);
        else if (full) count_event(p.counters, CSA2_CNT_CAPACITY);
    }
    const float *const mass = p.mass + (int64_t)b * p.ld_mass;
    float *const out = keys + (int64_t)s * ld;
    const int64_t j0 = (int64_t)blockIdx.x * (kThreads * kKeysPerThread) + threadIdx.x;
    const int64_t last = n - p.n_last;
#pragma unroll
    for (int i = 0; i < kKeysPerThread; ++i) {
        const int64_t j = j0 + i * kThreads;
        if (j >= n) continue;
        const float v = mass[j];
        // (the top-k orders keys by their bits: a positive NaN lies above infinity)
        out[j] = j < p.n_first || j >= last ? __uint_as_float(0x7FC00000u) : v != v ? -INFINITY : v;
    }
}

// A warp copies eight kept rows: lane l < 8 looks row l up and copies its weight and key
// scale; then each row is one 16-byte load and store of 18 lanes (256 bytes of codes, 32 of
// scales) and d_idx / 16 more for the key, all eight on their way at once.  What bounds it is
// the chain of loads in front of a row (its number, its pages), so many short warps serve
// it best: 245,760 rows with keys of 128 in 49 us, by 32 rows to a warp in 61.
constexpr int kFlight = 8;

__global__ void __launch_bounds__(kThreads, 4) evict_copy_kernel(EvictParams p, const int32_t *__restrict__ cnt,
                                                              const int32_t *__restrict__ skip, uint32_t per_seq, uint64_t items)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int key_lanes = p.src.kidx ? p.src.d_idx / 16 : 0;
    // the lane's array, its 16 bytes of a row, the row's bytes
    const uint8_t *from = lane < 16 ? p.src.codes + 16 * lane : lane < 18 ? p.src.scales + 16 * (lane - 16) : p.src.kidx + 16 * (lane - 18);
    uint8_t *to = lane < 16 ? p.dst.codes + 16 * lane : lane < 18 ? p.dst.scales + 16 * (lane - 16) : p.dst.kidx + 16 * (lane - 18);
    const int64_t pitch = lane < 16 ? CSA2_CODE_BYTES : lane < 18 ? CSA2_SCALE_BYTES : p.src.d_idx;
    const bool copies = lane < 18 + key_lanes;
    const uint64_t step = (uint64_t)gridDim.x * (kThreads / 32);
    for (uint64_t item = (uint64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); item < items; item += step) {
        const int s = (int)(item / per_seq);
        const int64_t d0 = (int64_t)(item - (uint64_t)s * per_seq) * kFlight;
        if (skip[s]) continue;
        const int b = p.seq ? p.seq[s] : s;
        const int c = cnt[s];
        if (d0 == 0 && lane == 0) p.dst.seq_len[b] = c;
        if (d0 >= c) continue;
        const int64_t d = d0 + lane;
        int src = -1, dst = -1;                            // (a cache has under 2^31 rows)
        if (lane < kFlight && d < c) {
            const int j = p.kept[s * p.ld_kept + d];
            if (p.mass_out) p.mass_out[b * p.ld_out + d] = p.mass[b * p.ld_mass + j];
            auto row_of = [&](const csa2_cache &cache, const PageMap &m, int64_t e) {
                if (m.table == nullptr) return (int)(cache.seq_base[b] + e);
                const int32_t page = m.table[(int64_t)b * m.ld + (e >> m.log)];
                if ((uint32_t)page >= m.pages) return -1;
                return (int)(((int64_t)page << m.log) + (e & ((1ll << m.log) - 1)));
            };
            src = row_of(p.src, p.src_pages, j);
            dst = row_of(p.dst, p.dst_pages, d);
            if (src < 0 || dst < 0) {
                count_event(p.counters, CSA2_CNT_BAD_INPUT);
                dst = -1;
            } else if (key_lanes) {
                p.dst.kscale[dst] = p.src.kscale[src];
            }
        }
        uint4 v[kFlight];
        int at[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const int f = __shfl_sync(0xffffffffu, src, i);
            at[i] = __shfl_sync(0xffffffffu, dst, i);
            if (!copies) at[i] = -1;
            if (at[i] >= 0) v[i] = *reinterpret_cast<const uint4 *>(from + f * pitch);
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i)
            if (at[i] >= 0) *reinterpret_cast<uint4 *>(to + at[i] * pitch) = v[i];
    }
}

}  // namespace

EvictPlan evict_plan(int ns, int64_t max_n)
{
    EvictPlan pl{};
    if (max_n < 1) max_n = 1;
    pl.ld = (int64_t)align_up((size_t)max_n, 4);
    pl.off_n = align_up((size_t)ns * pl.ld * 4, 256);
    pl.off_count = pl.off_n + align_up((size_t)ns * 8, 256);       // (entries, skipped)
    pl.off_topk = pl.off_count + align_up((size_t)ns * 4, 256);
    pl.total = pl.off_topk + topk_workspace_bytes(ns, max_n);
    return pl;
}

cudaError_t launch_evict(const EvictParams &p, const EvictPlan &pl, uint8_t *ws, cudaStream_t st)
{
    float *keys = reinterpret_cast<float *>(ws);
    int32_t *n = reinterpret_cast<int32_t *>(ws + pl.off_n), *skip = n + p.ns;
    int32_t *cnt = reinterpret_cast<int32_t *>(ws + pl.off_count);
    const int64_t max_n = std::max<int64_t>(1, p.max_n);
    const int64_t per_block = kThreads * kKeysPerThread;
    cudaError_t e = launch_k(evict_keys_kernel, dim3((unsigned)((max_n + per_block - 1) / per_block), (unsigned)p.ns),
                             dim3(kThreads), 0, st, 0, p, keys, pl.ld, n, skip);
    if (e == cudaSuccess)
        e = launch_topk(keys, pl.ld, n, 0, nullptr, 0, p.ns, max_n, p.keep, p.kept, p.ld_kept, cnt, ws + pl.off_topk, st);
    if (e != cudaSuccess) return e;
    const uint32_t per_seq = (uint32_t)((std::min<int64_t>(p.keep, max_n) + kFlight - 1) / kFlight);
    const uint64_t items = (uint64_t)p.ns * per_seq, blocks = (items + kThreads / 32 - 1) / (kThreads / 32);
    e = launch_k(evict_copy_kernel, dim3((unsigned)std::min<uint64_t>(blocks, (uint64_t)device_sm_count() * 128)), dim3(kThreads), 0, st, 0,
                 p, (const int32_t *)cnt, (const int32_t *)skip, per_seq, items);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa2
