// step_internal.h -- argument blocks and launch wrappers of the step operators
// (include/paged_gqa_step.h), shared between api_step.cu and their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

#include "../../include/paged_gqa_step.h"
#include "pgqa_internal.h"

namespace pgqa {

// SMs of the GPU that this library is built and measured for.  The launch rules count
// with it; elsewhere they would pick other shapes than the fastest, with the same results
// but for the order of sums.  (What has to fit the device, the CTAs of the split decode,
// is asked of the device.)
constexpr int kSms = 152;

// The step's kernels are launched as programmatic dependents of whatever kernel
// precedes them on the stream: their CTAs are placed while it drains, and wait in
// enter() -- before they touch global memory -- until it has completed.  From there
// on their own successors may be placed.  What they read may have been written by a
// kernel that was still running when they started, so they read it by ordinary loads and
// copies, never by the read-only path (__ldg, __restrict__), whose data must not change
// while a kernel lives, and whose loads need not stay behind the wait.  One token rotated call after call takes
// 3.05 us a call instead of 4.10, at the same time on the host.
__device__ __forceinline__ void enter()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
}

// Launches a kernel that calls enter(); cluster: CTAs of a cluster along x (0: none).
template <class... P, class... A>
cudaError_t launch_step(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s,
                        unsigned cluster, A&&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

struct RopeArgs {
    paged_gqa_rope_rows t[2];     // q, k
    const int32_t* pos;
    const double* freq;
    int T, D, rot;
    float scale;
    bool inverse, half;
};

// Scale tensors of a block-scaled cache: strides in floats.
struct ScaleGeom {
    int64_t page, block_stride, head;
    int block;                    // tokens of a scale block
    int shift;                    // log2(block) when it is a power of two, else -1
};

// A block-scaled cache as the attention kernels read it.  Row offsets are counted in
// `unit` bytes, a power of two that divides the strides, so that they fit 32 bits.
struct CacheArgs {
    KVGeom kv;
    uint32_t unit, page_u, token_u, head_u;
    ScaleGeom sc;
    const float *ks, *vs;
};

// The block-scaled decode's split kernel: five warps a CTA, two CTAs per SM.  With weights
// of 11 bits these took 77.9 us for 16 x 12K-16K tokens of 4 KV heads (E4M3; INT8 79.3),
// 133.5 us for 64 x 4K-8K and 20.1 us for seven ragged INT8 sequences (78.0, 81.6 and 20.5
// us now); six warps 79.8 (80.4), 135.8 and 19.9 us, four 77.2 (81.4), 141.7 and 26.7 us;
// four warps and three CTAs 103 us, ten and one 81 us.  Virtual tiles charged for a
// piece's start when the line of tiles is cut: 12 took 0.8 % longer, 20 the same.  At
// least eight tiles a CTA.
constexpr int kSplitWarps = 5;
constexpr int kSplitPieceTiles = 16;
constexpr int kSplitMinTiles = 8;

struct ScaledDecodeArgs {
    const __half* q;
    CacheArgs c;
    const int32_t* bt;
    int64_t bt_stride;
    const int32_t* seq_lens;
    int B, Hq, Hkv, G, max_seq_len;
    float scale_log2;             // softmax_scale * log2(e)
    __half* out;
    // split route only
    int64_t* hdr;                 // prefix[B + 1] from [2] on, for batches above kMergeScanMax
    float* slots;                 // C + B * Hkv partial slots
    int C;                        // CTAs launched on the split route; 0: a cluster per segment
    int groups, heads;            // of CTAs, with a line of tiles each; KV heads of a group
    int cluster;                  // its CTAs (1, 2, 4 or 8)
    int cluster_warps;            // their warps (4 or 8)
    int min_tiles;                // minimum tiles per CTA when choosing C_eff
    int* err;
};

struct ScaledPrefillArgs {
    const __half* q;
    CacheArgs c;
    const int32_t* bt;
    int kv_len;
    const int32_t* sel;
    int n_sel;
    const int32_t* q_pos;
    int R, Hq, Hkv, G;
    int cluster, cluster_warps;   // CTAs of a row's cluster, their warps
    float scale_log2;
    __half* out;
    int* err;
};

struct AppendArgs {
    const void* src[2];           // K, V rows
    int64_t ts[2], hs[2];         // their token and head strides, elements
    unsigned char* cache[2];
    float* scales[2];
    KVGeom kv;
    ScaleGeom sc;
    const int32_t* bt;
    int64_t bt_stride;
    const int32_t* starts;
    const int32_t* offs;          // NULL: row b is sequence b's
    int B, T, Hkv, max_len;
    int chunk;                    // rows a CTA looks through
    int* err;
};

struct LogitsArgs {
    const void* x;
    int64_t x_stride;
    float* out;
    int64_t out_stride;
    int B, V;
    int cols;                     // columns of a CTA
    paged_gqa_logit_rules r;      // parts without effect are NULL
    int* err;
};

cudaError_t launch_logits(const LogitsArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_append(const AppendArgs& a, int src_dtype, bool int8, cudaStream_t s);
size_t scaled_workspace_bytes(int B, int Hkv, int C);
int scaled_ctas_per_sm(bool int8);
cudaError_t launch_decode_scaled(const ScaledDecodeArgs& a, bool int8, cudaStream_t s, void* ev0,
                                 void* ev1);
cudaError_t launch_prefill_scaled(const ScaledPrefillArgs& a, bool int8, cudaStream_t s);

}  // namespace pgqa
