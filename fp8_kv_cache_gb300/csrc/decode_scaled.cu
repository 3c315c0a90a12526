// decode_scaled.cu -- batched paged decode over a block-scaled 8-bit cache.
//
// Bound: HBM, every K and V code once (512 bytes per token and KV head) and the
// scales beside them; for short contexts the latency of one kernel.  Two ways:
//  * clusters: up to 8 CTAs take a (sequence, KV head), each a share of its
//    16-token tiles, and join their results through distributed shared memory.
//    One kernel; the longest sequence decides the time.
//  * split and merge, for long contexts: the segments (sequence, KV head) are
//    laid end to end as a line of tiles, each preceded by kSplitPieceTiles
//    virtual ones for the fixed cost of a piece, and the line is cut on the
//    device into equal ranges, one per CTA.  The KV heads are dealt to `groups` of
//    CTAs with a line each, neighbouring CTAs to the same range of different
//    groups: rows that lie side by side in the pool are read at about the same
//    time.  A CTA that has all tiles of a segment writes its rows; the others leave
//    partial results (n, d, O) in slots that the merge kernel, a programmatic
//    dependent of the split kernel, joins in a fixed order.
// 16 sequences of 12K to 16K tokens, 4 KV heads: E4M3 78.0 us (0.90 of the measured
// copy bandwidth), INT8 81.6 us; 8 of 1024 tokens 6.9 us, one of 64 3.6 us.
#include <algorithm>
#include <atomic>

#include "scaled_core.cuh"

namespace pgqa {

namespace {

using scaled::ClusterJoin;
using scaled::Core;
using scaled::Inbox;
using scaled::Place;
using scaled::Smem;

__device__ __forceinline__ int length_of(const ScaledDecodeArgs& a, int b)
{
    return min(max(a.seq_lens[b], 0), a.max_seq_len);
}

// Tiles of n tokens (n + kTile - 1 would pass 31 bits for the longest).
__device__ __forceinline__ int tiles_of(int n)
{
    return n / kTile + (n % kTile != 0);
}

// Tiles of sequence b on the line, the piece cost included (0: empty).
__device__ __forceinline__ int64_t line_tiles(const ScaledDecodeArgs& a, int b)
{
    const int n = tiles_of(length_of(a, b));
    return n > 0 ? n + kSplitPieceTiles : 0;
}

// CTAs of a group that share its line of T > 0 tiles: each gets at least min_tiles
// of them, or twice that while half the launched CTAs still have work (longer
// ranges are fewer pieces to merge), and at least one.
__device__ __forceinline__ int64_t ctas_of(const ScaledDecodeArgs& a, int64_t T)
{
    int64_t C = a.C / a.groups;
    if (a.min_tiles > 0) {
        const int64_t longer = T / (2 * a.min_tiles);
        C = min(C, longer >= C / 2 ? longer : (T + a.min_tiles - 1) / a.min_tiles);
    }
    return max((int64_t)1, min(C, T));
}

// Tiles [ta, te) of segment (b, j) by the CTA's warps in turn; use(h, c, quad)
// gets the joined result.
template <bool kInt8, int kNW, class Use>
__device__ __forceinline__ void run_piece(const ScaledDecodeArgs& a, const Smem<kNW>& sm, int b, int j, int L,
                                          int ta, int te, int& flags, Use use)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    Core<kInt8> wc;
    wc.reset();
    const int32_t* bt_row = a.bt + (int64_t)b * a.bt_stride;
    auto at = [&](int k) -> Place {
        const int t = k * kTile + (lane & 15);
        if (t < L) {
            int pi, slot;
            page_and_slot(a.c.kv, t, pi, slot);
            const int page = table_page<false>(a.c.kv, bt_row, pi, flags);
            if (page >= 0)
                return scaled::place_of(a.c, page, slot, j);
        }
        return {scaled::kNowhere, 0};
    };
    __syncthreads();                                  // the rings and the merge buffer are free
    scaled::run_tiles<kInt8>(wc, sm.ring, sm.qs, a.c, ta + w, te, kNW, a.scale_log2, lane, at, [&] {
        scaled::stage_q(sm.qs, a.q + ((size_t)b * a.Hq + (size_t)j * a.G) * kD, a.G, lane, w, kNW);
        __syncthreads();
    });
    scaled::cta_merge<kInt8>(*sm.merge, wc, a.G, use);
}

// A group's slots; the one for CTA c of the group and its segment (b, j) is at
// c + b * heads + j.
__device__ __forceinline__ float* group_slots(const ScaledDecodeArgs& a, int group)
{
    return a.slots + (size_t)group * (a.C / a.groups + (size_t)a.B * a.heads) * kSlotFloats;
}

// The flags of sequence b's length.
__device__ __forceinline__ int length_flags(const ScaledDecodeArgs& a, int b)
{
    const int raw = a.seq_lens[b];
    return (raw > a.max_seq_len ? PAGED_GQA_FLAG_SEQ_CLAMPED : 0) | (raw <= 0 ? PAGED_GQA_FLAG_EMPTY_ROW : 0);
}

constexpr int kSplitCtas = 2;             // split CTAs resident per SM
constexpr int kSplitThreads = 32 * kSplitWarps;
using SplitSmem = Smem<kSplitWarps>;
template <int kNW>
using ClusterSmem = Smem<kNW>;
template <int kNW>
constexpr size_t kClusterSmem = ClusterSmem<kNW>::kTailOff + sizeof(Inbox);

}  // namespace

// One cluster of `size` CTAs per segment, each with a share of its tiles.
template <bool kInt8, int kNW>
__global__ void __launch_bounds__(32 * kNW, kNW > 4 ? 1 : 2)
    scaled_cluster_kernel(ScaledDecodeArgs a, int size)
{
    extern __shared__ __align__(128) unsigned char smem_raw[];
    ClusterJoin::begin();
    const int tid = threadIdx.x, segment = blockIdx.x / size, rank = blockIdx.x - segment * size;
    const int b = segment / a.Hkv, j = segment - b * a.Hkv;
    const ClusterSmem<kNW> sm = ClusterSmem<kNW>::carve(smem_raw, tid >> 5);
    ClusterJoin join(*reinterpret_cast<Inbox*>(sm.tail), size, rank);
    enter();
    int flags = rank == 0 && tid == 0 ? length_flags(a, b) : 0;
    const int L = length_of(a, b), n = tiles_of(L);
    __half* out_rows = a.out + ((size_t)b * a.Hq + (size_t)j * a.G) * kD;
    const int ta = (int)((int64_t)n * rank / size), te = (int)((int64_t)n * (rank + 1) / size);
    run_piece<kInt8>(a, sm, b, j, L, ta, te, flags,
                     [&](int h, int c, const scaled::Quad& v) { join.put(h, c, v, out_rows); });
    raise_flag(a.err, flags);
    join.finish(a.G, out_rows);
}

template <bool kInt8>
__global__ void __launch_bounds__(kSplitThreads, kSplitCtas) scaled_split_kernel(ScaledDecodeArgs a)
{
    extern __shared__ __align__(128) unsigned char smem_raw[];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const SplitSmem sm = SplitSmem::carve(smem_raw, w);
    int flags = 0;
    enter();

    // ---- exclusive prefix P of the sequences' tiles
    int64_t* P = reinterpret_cast<int64_t*>(sm.tail);
    int64_t* wtot = P + (a.B + 1);
    const int per = (a.B + kSplitThreads - 1) / kSplitThreads;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
        if (blockIdx.x == 0)
            flags |= length_flags(a, b);
        mine += line_tiles(a, b);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += t;
    }
    if (lane == 31)
        wtot[w] = incl;
    __syncthreads();
    int64_t run = incl - mine, total = 0;
    for (int i = 0; i < kSplitWarps; ++i) {
        run += i < w ? wtot[i] : 0;
        total += wtot[i];
    }
    for (int b = b0; b < b1; ++b) {
        P[b] = run;
        run += line_tiles(a, b);
    }
    if (tid == 0)
        P[a.B] = total;
    __syncthreads();

    const int64_t T = (int64_t)a.heads * total;
    const int64_t C = T > 0 ? ctas_of(a, T) : 0;
    if (blockIdx.x == 0 && a.B > kMergeScanMax) {
        for (int i = tid; i <= a.B; i += kSplitThreads)
            a.hdr[2 + i] = P[i];
    }
    const int group = blockIdx.x % a.groups;
    const int64_t c = blockIdx.x / a.groups;
    if (c < C) {
        float* slots = group_slots(a, group);
        const int64_t x0 = c * T / C, x1 = (c + 1) * T / C;
        int lo = 0, hi = a.B - 1;                     // the last b with heads P[b] <= x0
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int64_t)a.heads * P[mid] <= x0)
                lo = mid;
            else
                hi = mid - 1;
        }
        int b = lo;
        int64_t nb = P[b + 1] - P[b];
        int j = (int)((x0 - (int64_t)a.heads * P[b]) / nb);
        for (;;) {
            const int64_t s0 = (int64_t)a.heads * P[b] + (int64_t)j * nb;
            if (s0 >= x1)
                break;
            const int64_t r0 = s0 + kSplitPieceTiles, r1 = s0 + nb;   // the segment's real tiles
            if (max(x0, r0) < min(x1, r1)) {
                const bool whole = x0 <= r0 && x1 >= r1;
                const int head = group * a.heads + j;
                __half* out_rows = a.out + ((size_t)b * a.Hq + (size_t)head * a.G) * kD;
                float* slot = slots + (size_t)(c + (int64_t)b * a.heads + j) * kSlotFloats;
                run_piece<kInt8>(a, sm, b, head, length_of(a, b), (int)(max(x0, r0) - r0),
                                 (int)(min(x1, r1) - r0), flags,
                                 [&](int h, int c4, const scaled::Quad& v) {
                                     if (whole) {
                                         scaled::store_rows(out_rows, h, c4, v);
                                     } else {
                                         reinterpret_cast<float4*>(slot + 2 * kGMax + h * kD)[c4] = v.o;
                                         if (c4 == 0) {
                                             slot[h] = v.n;
                                             slot[kGMax + h] = v.d;
                                         }
                                     }
                                 });
            }
            if (++j == a.heads) {                     // the next segment that is not empty
                j = 0;
                do
                    ++b;
                while (b < a.B && P[b + 1] == P[b]);
                if (b >= a.B)
                    break;
                nb = P[b + 1] - P[b];
            }
        }
    }
    raise_flag(a.err, flags);
}

// grid (Hq, B): joins the pieces of one query head, four groups of 64 threads
// (four head-dim values each) taking chunks of pieces in turn:
//   M = max n_i,  out = sum 2^(n_i - M) O_i / sum 2^(n_i - M) d_i.
// Rows of empty sequences are zeroed; rows one CTA wrote are left.  What
// depends on seq_lens alone is done before the wait for the split kernel.
__global__ void __launch_bounds__(kMergeThreads * kMergeGroups) scaled_merge_kernel(ScaledDecodeArgs a)
{
    constexpr int kAll = kMergeThreads * kMergeGroups, kChunk = 8;
    __shared__ int64_t red[kAll / 32][2];
    __shared__ float g_n[kMergeGroups], g_d[kMergeGroups];
    __shared__ float4 g_o[kMergeGroups][kMergeThreads];
    const int h = blockIdx.x, b = blockIdx.y, head = h / a.G, hh = h - head * a.G;
    const int group = head / a.heads, j = head - group * a.heads;
    const int tid = threadIdx.x, grp = tid / kMergeThreads, d = 4 * (tid % kMergeThreads);
    __half2* out = reinterpret_cast<__half2*>(a.out + ((size_t)b * a.Hq + h) * kD + d);
    int64_t before = 0, total = 0;
    if (a.B <= kMergeScanMax) {
        for (int i = tid; i < a.B; i += kAll) {
            const int64_t n = line_tiles(a, i);
            total += n;
            before += i < b ? n : 0;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            before += __shfl_xor_sync(0xffffffffu, before, o);
            total += __shfl_xor_sync(0xffffffffu, total, o);
        }
        if ((tid & 31) == 0) {
            red[tid >> 5][0] = before;
            red[tid >> 5][1] = total;
        }
        __syncthreads();
        before = total = 0;
        for (int i = 0; i < kAll / 32; ++i) {
            before += red[i][0];
            total += red[i][1];
        }
    }
    const int64_t nb = line_tiles(a, b);
    enter();
    if (nb == 0) {
        if (grp == 0)
            out[0] = out[1] = __floats2half2_rn(0.f, 0.f);
        return;
    }
    if (a.B > kMergeScanMax) {
        before = a.hdr[2 + b];
        total = a.hdr[2 + a.B];
    }
    const int64_t T = (int64_t)a.heads * total, C = ctas_of(a, T);
    // the CTAs whose ranges meet the segment's real tiles
    const int64_t s0 = (int64_t)a.heads * before + (int64_t)j * nb;
    const int64_t r0 = s0 + kSplitPieceTiles, r1 = s0 + nb;
    const int64_t first = ((r0 + 1) * C + T - 1) / T - 1, last = (r1 * C + T - 1) / T - 1;
    if (first == last)
        return;                                       // one CTA wrote the rows
    const float* slots = group_slots(a, group) + (size_t)(first + (int64_t)b * a.heads + j) * kSlotFloats;
    const int64_t n_pieces = last - first + 1;
    const bool grouped = n_pieces > kChunk;           // CTA-uniform
    if (!grouped && grp != 0)
        return;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f, M = -INFINITY;
    auto add = [&](float n, float dd, const float4& o) {   // (dd, o) times 2^(n - M); n = -inf: nothing attended
        const float e = n == -INFINITY ? 0.f : ex2(n - M);
        den += e * dd;
        num.x += e * o.x;
        num.y += e * o.y;
        num.z += e * o.z;
        num.w += e * o.w;
    };
    for (int64_t c0 = (int64_t)grp * kChunk; c0 < n_pieces; c0 += (grouped ? kMergeGroups : 1) * kChunk) {
        float n[kChunk], dd[kChunk];
        float4 o[kChunk];
        float top = M;
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            n[i] = -INFINITY;
            dd[i] = 0.f;
            o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c0 + i < n_pieces) {
                const float* sl = slots + (size_t)(c0 + i) * kSlotFloats;
                n[i] = sl[hh];
                dd[i] = sl[kGMax + hh];
                o[i] = *reinterpret_cast<const float4*>(sl + 2 * kGMax + hh * kD + d);
            }
            top = fmaxf(top, n[i]);
        }
        const float4 num0 = num;
        const float den0 = den, M0 = M;
        num = make_float4(0.f, 0.f, 0.f, 0.f);
        den = 0.f;
        M = top;
        add(M0, den0, num0);
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
            add(n[i], dd[i], o[i]);
    }
    if (grouped) {
        if (d == 0) {
            g_n[grp] = M;
            g_d[grp] = den;
        }
        g_o[grp][d / 4] = num;
        __syncthreads();
        if (grp != 0)
            return;
        num = make_float4(0.f, 0.f, 0.f, 0.f);
        den = 0.f;
        M = -INFINITY;
        for (int i = 0; i < kMergeGroups; ++i)
            M = fmaxf(M, g_n[i]);
        for (int i = 0; i < kMergeGroups; ++i)
            add(g_n[i], g_d[i], g_o[i][d / 4]);
    }
    const float s = den == 0.f ? 0.f : 1.f / den;
    out[0] = __floats2half2_rn(num.x * s, num.y * s);
    out[1] = __floats2half2_rn(num.z * s, num.w * s);
}

namespace {

size_t split_smem(int B)
{
    return SplitSmem::kTailOff + (size_t)(B + 1 + kSplitWarps) * sizeof(int64_t);
}

// The kernels of one code type.
template <bool kInt8>
struct Kernels {
    static constexpr auto split = scaled_split_kernel<kInt8>;

    // The dynamic shared-memory opt-ins, once per device.
    static cudaError_t prepare()
    {
        static std::atomic<int> done[kMaxDevices];
        constexpr auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess || (dev < kMaxDevices && done[dev].load(std::memory_order_acquire)))
            return e;
        e = cudaFuncSetAttribute(split, attr, (int)split_smem(kMaxSplitBatch));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(scaled_cluster_kernel<kInt8, 4>, attr, (int)kClusterSmem<4>);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(scaled_cluster_kernel<kInt8, 8>, attr, (int)kClusterSmem<8>);
        if (e == cudaSuccess && dev < kMaxDevices)
            done[dev].store(1, std::memory_order_release);
        return e;
    }

    static int ctas_per_sm()
    {
        int n = 0;
        if (prepare() != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, split, kSplitThreads, split_smem(64)) !=
                cudaSuccess)
            return 1;
        return std::max(n, 1);
    }

    template <int kNW>
    static cudaError_t run_clusters(const ScaledDecodeArgs& a, cudaStream_t s)
    {
        const unsigned grid = (unsigned)(a.B * a.Hkv * a.cluster);
        constexpr auto kernel = scaled_cluster_kernel<kInt8, kNW>;
        return launch_step(kernel, dim3(grid), 32 * kNW, kClusterSmem<kNW>, s,
                           a.cluster == 1 ? 0 : a.cluster, a, a.cluster);
    }

    // The kernel that reads the cache.
    static cudaError_t run(const ScaledDecodeArgs& a, cudaStream_t s)
    {
        const cudaError_t e = prepare();
        if (e != cudaSuccess)
            return e;
        if (a.C == 0)
            return a.cluster_warps == 8 ? run_clusters<8>(a, s) : run_clusters<4>(a, s);
        return launch_step(split, dim3(a.C), kSplitThreads, split_smem(a.B), s, 0, a);
    }
};

}  // namespace

size_t scaled_workspace_bytes(int B, int Hkv, int C)
{
    const size_t head = (kHeaderBytes + (size_t)(B + 1) * sizeof(int64_t) + 255) & ~(size_t)255;
    return head + ((size_t)C + (size_t)B * Hkv) * kSlotFloats * sizeof(float);
}

int scaled_ctas_per_sm(bool int8)
{
    return int8 ? Kernels<true>::ctas_per_sm() : Kernels<false>::ctas_per_sm();
}

cudaError_t launch_decode_scaled(const ScaledDecodeArgs& a, bool int8, cudaStream_t s, void* ev0,
                                 void* ev1)
{
    cudaError_t e = cudaSuccess;
    const bool events = ev0 && ev1;
    if (events && (e = cudaEventRecord((cudaEvent_t)ev0, s)) != cudaSuccess)
        return e;
    e = int8 ? Kernels<true>::run(a, s) : Kernels<false>::run(a, s);
    if (e != cudaSuccess)
        return e;
    if (events && (e = cudaEventRecord((cudaEvent_t)ev1, s)) != cudaSuccess)
        return e;
    if (a.C == 0)
        return cudaSuccess;
    return launch_step(scaled_merge_kernel, dim3(a.Hq, a.B), kMergeThreads * kMergeGroups, 0, s, 0, a);
}

}  // namespace pgqa
