// prefill_scaled.cu -- selected-sparse prefill over a block-scaled 8-bit cache.
//
// The operation of the per-tensor prefill (each row attends to its selected
// four-token blocks and its causal tail), with the scores and weights of
// scaled_core.cuh.  Bound: the tiles' instructions, fed by a gather of every
// row's own blocks out of L2 at 10.4 TB/s.
// One CTA per (query row, KV head), or a cluster of up to 8 when there are few rows;
// it resolves a chunk of block entries into a shared-memory table (first token,
// page), so that the ring fills need no dependent global load, and its warps take
// 16-token tiles in turn.  4096 rows of 512 blocks 419 us (E4M3), 497 us (INT8).  One
// row of 512 blocks 7.8 us (39 us by one CTA, with the tiles of the time), 64 rows
// 15.1 us (40 us), 128 rows 24 us (40 us).
#include <atomic>

#include "scaled_core.cuh"

namespace pgqa {

namespace {

constexpr int kScaledEntries = 768;          // block entries of a chunk: 4 k, three CTAs fit in an SM
// Without clusters: four warps, three CTAs per SM.  With them: four warps, two CTAs,
// or eight warps, one CTA.
template <int kNW>
using PrefillSmem = scaled::Smem<kNW>;
template <int kNW, bool kClusters>
constexpr size_t kScaledPrefillSmem = PrefillSmem<kNW>::kTailOff + (size_t)kScaledEntries * sizeof(int2) +
                                      (kClusters ? sizeof(scaled::Inbox) : 0);

}  // namespace

// grid (R * size, Hkv): CTA rank of row r's cluster takes a share of its tiles.
template <bool kInt8, int kNW, bool kClusters>
__global__ void __launch_bounds__(32 * kNW, kNW > 4 ? 1 : kClusters ? 2 : 3)
    scaled_prefill_kernel(ScaledPrefillArgs a, int size)
{
    extern __shared__ __align__(128) unsigned char smem_raw[];
    if constexpr (kClusters)
        scaled::ClusterJoin::begin();
    const int r = kClusters ? blockIdx.x / size : blockIdx.x, j = blockIdx.y;
    const int rank = kClusters ? blockIdx.x - r * size : 0;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const PrefillSmem<kNW> sm = PrefillSmem<kNW>::carve(smem_raw, w);
    int2* tab = reinterpret_cast<int2*>(sm.tail);
    scaled::ClusterJoin join(*reinterpret_cast<scaled::Inbox*>(tab + kScaledEntries), kClusters ? size : 1, rank);
    int flags = 0;
    __half* out_rows = a.out + ((size_t)r * a.Hq + (size_t)j * a.G) * kD;
    enter();
    int p = a.q_pos[r];
    const bool empty = p < 0 || a.kv_len <= 0;
    if (empty) {
        flags |= PAGED_GQA_FLAG_EMPTY_ROW;
    } else if (p >= a.kv_len) {
        p = a.kv_len - 1;
        flags |= PAGED_GQA_FLAG_QPOS_CLAMPED;
    }
    const int own = p >> 2;
    const int32_t* sel_row = a.sel + (size_t)r * a.n_sel;
    scaled::stage_q(sm.qs, a.q + ((size_t)r * a.Hq + (size_t)j * a.G) * kD, a.G, lane, w, kNW);
    scaled::Core<kInt8> wc;
    wc.reset();
    // the row's entries (the tail block last), by tiles of four; none of an empty row
    const int n_entries = empty ? 0 : a.n_sel + 1, tiles = (n_entries + 3) / 4;
    const int ea = kClusters ? 4 * (int)((int64_t)tiles * rank / size) : 0;
    const int ee = kClusters ? min(4 * (int)((int64_t)tiles * (rank + 1) / size), n_entries) : n_entries;
    for (int e0 = ea; e0 < ee; e0 += kScaledEntries) {
        const int e1 = min(ee, e0 + kScaledEntries);
        __syncthreads();                             // Q staged, the previous chunk done with tab
        for (int e = e0 + (int)threadIdx.x; e < e1; e += 32 * kNW) {
            int first, page;
            prefill_entry<false>(a.c.kv, a.bt, sel_row, a.n_sel, own, e, first, page, flags);
            tab[e - e0] = make_int2(first, page);
        }
        __syncthreads();
        // tile k: block entries 4k .. 4k + 3; lane l takes token l mod 16
        auto at = [&](int k) -> scaled::Place {
            const int e = 4 * k + ((lane >> 2) & 3), u = lane & 3;
            if (e < e1) {
                const int2 en = tab[e - e0];
                if (prefill_lane_live(en.y, e, a.n_sel, en.x, u, p)) {
                    int pi, slot;
                    page_and_slot(a.c.kv, en.x + u, pi, slot);
                    return scaled::place_of(a.c, en.y, slot, j);
                }
            }
            return {scaled::kNowhere, 0};
        };
        scaled::run_tiles<kInt8>(wc, sm.ring, sm.qs, a.c, e0 / 4 + w, (e1 + 3) / 4, kNW, a.scale_log2,
                                 lane, at, [] {});
    }
    scaled::cta_merge<kInt8>(*sm.merge, wc, a.G, [&](int h, int c, const scaled::Quad& v) {
        if constexpr (kClusters)
            join.put(h, c, v, out_rows);
        else
            scaled::store_rows(out_rows, h, c, v);
    });
    raise_flag(a.err, flags);
    if constexpr (kClusters)
        join.finish(a.G, out_rows);
}

namespace {

template <bool kInt8, int kNW, bool kClusters>
cudaError_t prefill_run(const ScaledPrefillArgs& a, cudaStream_t s)
{
    static std::atomic<int> done[kMaxDevices];
    constexpr auto kernel = scaled_prefill_kernel<kInt8, kNW, kClusters>;
    constexpr size_t smem = kScaledPrefillSmem<kNW, kClusters>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= kMaxDevices || !done[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess)
            return e;
        if (dev < kMaxDevices)
            done[dev].store(1, std::memory_order_release);
    }
    return launch_step(kernel, dim3(a.R * (kClusters ? a.cluster : 1), a.Hkv), 32 * kNW, smem, s,
                       kClusters ? a.cluster : 0, a, a.cluster);
}

template <bool kInt8>
cudaError_t prefill_kind(const ScaledPrefillArgs& a, cudaStream_t s)
{
    if (a.cluster_warps == 8)
        return prefill_run<kInt8, 8, true>(a, s);
    return a.cluster > 1 ? prefill_run<kInt8, 4, true>(a, s) : prefill_run<kInt8, 4, false>(a, s);
}

}  // namespace

cudaError_t launch_prefill_scaled(const ScaledPrefillArgs& a, bool int8, cudaStream_t s)
{
    return int8 ? prefill_kind<true>(a, s) : prefill_kind<false>(a, s);
}

}  // namespace pgqa
