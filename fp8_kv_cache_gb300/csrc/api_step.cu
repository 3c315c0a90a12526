// api_step.cu -- the extern "C" entry points declared in
// include/paged_gqa_step.h: host-side validation and the launches.  Nothing
// here allocates memory or synchronises the host.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "step_internal.h"

using namespace pgqa;

namespace {

constexpr double kLog2e = 1.4426950408889634;

int status_of(cudaError_t e)
{
    return e == cudaSuccess ? PAGED_GQA_OK : PAGED_GQA_ERR_CUDA;
}

bool aligned(const void* p, uintptr_t n)
{
    return (reinterpret_cast<uintptr_t>(p) % n) == 0;
}

// Bytes of an element of a paged_gqa_float_dtype, or 0.
int float_bytes(int dtype)
{
    return dtype == PAGED_GQA_F32 ? 4 : dtype == PAGED_GQA_F16 || dtype == PAGED_GQA_BF16 ? 2 : 0;
}

// One dimension of a set of rows: how many, and how far apart.
struct Dim {
    int64_t count, stride;
};

// Whether rows of n elements at sums of index * stride lie apart from one
// another: along each dimension, from the smallest stride to the largest, the
// stride passes over all that the smaller ones span.
template <size_t N>
bool rows_apart(Dim (&d)[N], int64_t n)
{
    std::sort(d, d + N, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
    for (const Dim& x : d) {
        if (x.count <= 1)
            continue;
        if (x.stride < n)
            return false;
        n += (x.count - 1) * x.stride;
    }
    return true;
}

int check_rope_rows(const paged_gqa_rope_rows& m, int T, int D, int size)
{
    if (m.heads < 1 || m.heads > 65535 || m.token_stride < 0 || m.head_stride < 0)
        return PAGED_GQA_ERR_SHAPE;
    Dim out[] = {{T, m.out_token_stride}, {m.heads, m.out_head_stride}};
    if (!rows_apart(out, D))
        return PAGED_GQA_ERR_SHAPE;
    if (m.x == nullptr || m.out == nullptr)
        return PAGED_GQA_ERR_NULL_POINTER;
    if (!aligned(m.x, size) || !aligned(m.out, size))
        return PAGED_GQA_ERR_ALIGNMENT;
    if (m.x == m.out && ((T > 1 && m.token_stride != m.out_token_stride) ||
                         (m.heads > 1 && m.head_stride != m.out_head_stride)))
        return PAGED_GQA_ERR_SHAPE;
    return PAGED_GQA_OK;
}

// Checks of a block-scaled cache: pools, strides, scales.
int check_scaled_cache(const void* k, const void* v, const paged_gqa_kv_layout& L, int kv_dtype,
                       const float* ks, const float* vs, const paged_gqa_scale_layout& S,
                       int scale_block, int page_size, int num_pages)
{
    if (kv_dtype != PAGED_GQA_KV_E4M3 && kv_dtype != PAGED_GQA_KV_INT8)
        return PAGED_GQA_ERR_UNSUPPORTED;
    if (page_size < 1 || num_pages < 1 || scale_block < 1 || page_size % scale_block != 0)
        return PAGED_GQA_ERR_SHAPE;
    if (L.page_stride < 0 || L.token_stride < 0 || L.head_stride < 0 || S.page_stride < 0 ||
        S.block_stride < 0 || S.head_stride < 0)
        return PAGED_GQA_ERR_SHAPE;
    if (k == nullptr || v == nullptr || ks == nullptr || vs == nullptr)
        return PAGED_GQA_ERR_NULL_POINTER;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(ks, 4) || !aligned(vs, 4) ||
        L.page_stride % 16 || L.token_stride % 16 || L.head_stride % 16)
        return PAGED_GQA_ERR_ALIGNMENT;
    return PAGED_GQA_OK;
}

int log2_if_pow2(int x)
{
    int s = 0;
    while (s < 30 && (1 << s) < x)
        ++s;
    return (1 << s) == x ? s : -1;
}

ScaleGeom scale_geom(const paged_gqa_scale_layout& S, int block)
{
    return {S.page_stride, S.block_stride, S.head_stride, block, log2_if_pow2(block)};
}

KVGeom scaled_geom(const void* k, const void* v, const paged_gqa_kv_layout& L, int page_size,
                   int num_pages)
{
    KVGeom g;
    g.k = static_cast<const unsigned char*>(k);
    g.v = static_cast<const unsigned char*>(v);
    g.page_b = L.page_stride;
    g.token_b = L.token_stride;
    g.head_b = L.head_stride;
    g.page_size = page_size;
    g.page_shift = log2_if_pow2(page_size);
    g.num_pages = num_pages;
    return g;
}

// The cache as the attention kernels read it; false when its rows' offsets do not fit.
bool cache_args(CacheArgs& c, const KVGeom& kv, const ScaleGeom& sc, const float* ks, const float* vs, int Hkv)
{
    const int64_t all = kv.page_b | kv.token_b | kv.head_b | (int64_t)1 << 30;
    const int64_t unit = all & -all;
    const double span = ((double)kv.num_pages * kv.page_b + (double)kv.page_size * kv.token_b +
                         (double)Hkv * kv.head_b) / unit;
    c = {kv, (uint32_t)unit, (uint32_t)(kv.page_b / unit), (uint32_t)(kv.token_b / unit),
         (uint32_t)(kv.head_b / unit), sc, ks, vs};
    return span < 4294967295.0;
}

int check_heads(int B, int Hq, int Hkv, int D)
{
    if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || (int64_t)B * Hq > INT32_MAX)
        return PAGED_GQA_ERR_SHAPE;
    return D != kD || Hq / Hkv > kGMax ? PAGED_GQA_ERR_UNSUPPORTED : PAGED_GQA_OK;
}

// CTAs of the split decode kernels that are resident on the current device at
// once ([0] E4M3, [1] INT8), looked up once per device.
int split_ctas(int (&n)[2])
{
    static std::atomic<int> known[kMaxDevices][2];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return PAGED_GQA_ERR_CUDA;
    for (int i = 0; i < 2; ++i) {
        n[i] = dev < kMaxDevices ? known[dev][i].load(std::memory_order_relaxed) : 0;
        if (n[i] > 0)
            continue;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return PAGED_GQA_ERR_CUDA;
        n[i] = sms * scaled_ctas_per_sm(i == 1);
        if (dev < kMaxDevices)
            known[dev][i].store(n[i], std::memory_order_relaxed);
    }
    return PAGED_GQA_OK;
}

// The cluster of a (sequence or row, KV head) of `tiles` tiles, one of `segments`:
// as many CTAs as leave each of four warps a tile while all clusters are resident,
// and eight warps to a CTA while those are, too (one such CTA per SM; of eight-CTA
// clusters of them only about 14 are placed at once).  Measured at the time, E4M3,
// one KV head: one sequence of 1024 tokens 5.7 us with 8 x 8 warps, 6.7 us with 8 x
// 4; 16 sequences of 512 tokens 6.0 us with 4 x 8 warps, 6.4 us with 8 x 4, 9.5 us
// with 8 x 8 (now 5.1 and 5.3 us with the chosen ones).
void choose_cluster(int64_t segments, int64_t tiles, int& cluster, int& warps)
{
    cluster = 8;
    while (cluster > 1 && (segments * cluster > 2 * kSms || tiles <= 2 * cluster))
        cluster /= 2;
    if (cluster == 8 && segments * 8 > 112 && segments * 4 <= kSms)
        cluster = 4;
    warps = segments * cluster <= (cluster == 8 ? 112 : kSms) && tiles > 4 ? 8 : 4;
}

// Whether C split CTAs and a merge kernel beat the clusters: they share all
// sequences' tiles evenly, for about 5 us more.  So clusters whose warps have up to
// six more tiles than the split ones (a quarter more when there are many) are
// faster.  Only the longest length that may come is known here.  Measured with equal
// lengths, split / cluster: 1 x 8192 tokens x 1 KV head 10.2 / 14.4 us, 16 x 8192
// 21.8 / 29.3 us, x 4 KV heads 51 / 46 us, 64 x 8192 x 4 171 / 160 us; with lengths
// of 0 to 8192: 8 x 4 21.0 / 24.9 us, 16 x 4 32.0 / 39.2 us, 64 x 4 92 / 135 us.  Of
// those batches the rule splits 1 x 1, 16 x 1 and 64 x 4: the slower way for 64 x 4 of
// equal and for 8 x 4 and 16 x 4 of ragged lengths.
bool split_pays(const ScaledDecodeArgs& a, int C)
{
    const double tiles = (a.max_seq_len + kTile - 1.0) / kTile;
    const double each = tiles / (a.cluster * a.cluster_warps);
    return each > 6.0 + 1.25 * tiles * a.B * a.Hkv / ((double)C * kSplitWarps);
}

// Groups of split CTAs that the KV heads are dealt to: as many as divide them and
// leave no more than one CTA in 24 without work (4 KV heads, 16 x 12K-16K tokens, at
// the time: four groups 77.9 us, one 79.2 us).
int split_groups(int Hkv, int C)
{
    for (int m = std::min(Hkv, C);; --m)
        if (Hkv % m == 0 && C % m <= C / 24)
            return m;
}

}  // namespace

extern "C" {

int paged_gqa_rope(const paged_gqa_rope_rows* q, const paged_gqa_rope_rows* k, int T, int D,
                   int dtype, const int32_t* positions, const double* inv_freq, int rot_dim,
                   int layout, float scale, int inverse, void* stream)
{
    if (T < 0 || D < 1 || D > 4096 || rot_dim < 0 || rot_dim > D || rot_dim % 2 != 0)
        return PAGED_GQA_ERR_SHAPE;
    const int size = float_bytes(dtype);
    if (size == 0 || (layout != PAGED_GQA_ROPE_HALF && layout != PAGED_GQA_ROPE_INTERLEAVED))
        return PAGED_GQA_ERR_UNSUPPORTED;
    if (q == nullptr || positions == nullptr || (rot_dim > 0 && inv_freq == nullptr))
        return PAGED_GQA_ERR_NULL_POINTER;
    int st = check_rope_rows(*q, T, D, size);
    if (st == PAGED_GQA_OK && k != nullptr)
        st = check_rope_rows(*k, T, D, size);
    if (st != PAGED_GQA_OK)
        return st;
    if (!aligned(positions, 4) || !aligned(inv_freq, 8))
        return PAGED_GQA_ERR_ALIGNMENT;
    if (T == 0)
        return PAGED_GQA_OK;
    RopeArgs a{};
    a.t[0] = *q;
    if (k != nullptr)
        a.t[1] = *k;
    a.pos = positions;
    a.freq = inv_freq;
    a.T = T;
    a.D = D;
    a.rot = rot_dim;
    a.scale = scale;
    a.inverse = inverse != 0;
    a.half = layout == PAGED_GQA_ROPE_HALF;
    return status_of(launch_rope(a, dtype, static_cast<cudaStream_t>(stream)));
}

int paged_gqa_rope_frequencies(double* inv_freq, int rot_dim, double base, int scaling,
                               double factor, double original_len, double low, double high)
{
    constexpr double kTwoPi = 6.283185307179586;
    if (rot_dim < 2 || rot_dim % 2 != 0 || !(base > 0.0) || std::isinf(base) || !(factor > 0.0) ||
        std::isinf(factor))
        return PAGED_GQA_ERR_SHAPE;
    if (scaling < PAGED_GQA_ROPE_SCALE_NONE || scaling > PAGED_GQA_ROPE_SCALE_RAMP)
        return PAGED_GQA_ERR_UNSUPPORTED;
    if (scaling == PAGED_GQA_ROPE_SCALE_RAMP &&
        !(original_len > 0.0 && std::isfinite(original_len) && high > low && std::isfinite(high) &&
          std::isfinite(low)))
        return PAGED_GQA_ERR_SHAPE;
    if (inv_freq == nullptr)
        return PAGED_GQA_ERR_NULL_POINTER;
    if (scaling == PAGED_GQA_ROPE_SCALE_BASE && rot_dim > 2)
        base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == PAGED_GQA_ROPE_SCALE_LINEAR)
            f /= factor;
        if (scaling == PAGED_GQA_ROPE_SCALE_RAMP) {
            double g = (original_len * f / kTwoPi - low) / (high - low);
            g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
            f *= g + (1.0 - g) / factor;
        }
        inv_freq[i] = f;
    }
    return PAGED_GQA_OK;
}

int paged_gqa_append_scaled(const void* k, int64_t k_token_stride, int64_t k_head_stride,
                            const void* v, int64_t v_token_stride, int64_t v_head_stride,
                            int src_dtype, int T, void* k_cache, void* v_cache,
                            paged_gqa_kv_layout kv_layout, int kv_dtype, float* k_scales,
                            float* v_scales, paged_gqa_scale_layout scale_layout, int scale_block,
                            const int32_t* block_table, int64_t bt_row_stride,
                            const int32_t* seq_starts, const int32_t* new_offsets, int B, int Hkv,
                            int D, int page_size, int num_pages, int max_seq_len, int* err_flag,
                            void* stream)
{
    if (B < 0 || T < 0 || Hkv < 1 || Hkv > 32767 || max_seq_len < 0 || bt_row_stride < 0)
        return PAGED_GQA_ERR_SHAPE;
    if (new_offsets == nullptr && T != B)
        return PAGED_GQA_ERR_SHAPE;
    if (k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0)
        return PAGED_GQA_ERR_SHAPE;
    const int size = float_bytes(src_dtype);
    if (D != kD || size == 0)
        return PAGED_GQA_ERR_UNSUPPORTED;
    int st = check_scaled_cache(k_cache, v_cache, kv_layout, kv_dtype, k_scales, v_scales,
                                scale_layout, scale_block, page_size, num_pages);
    if (st != PAGED_GQA_OK)
        return st;
    if (B > 1 && bt_row_stride < ((int64_t)max_seq_len + page_size - 1) / page_size)
        return PAGED_GQA_ERR_SHAPE;
    Dim rows[] = {{num_pages, kv_layout.page_stride}, {page_size, kv_layout.token_stride},
                  {Hkv, kv_layout.head_stride}};
    Dim scales[] = {{num_pages, scale_layout.page_stride},
                    {page_size / scale_block, scale_layout.block_stride},
                    {Hkv, scale_layout.head_stride}};
    if (!rows_apart(rows, kD) || !rows_apart(scales, 1))
        return PAGED_GQA_ERR_SHAPE;
    if (T == 0 || B == 0)
        return PAGED_GQA_OK;
    if (k == nullptr || v == nullptr || block_table == nullptr || seq_starts == nullptr)
        return PAGED_GQA_ERR_NULL_POINTER;
    if (!aligned(k, 16) || !aligned(v, 16) || k_token_stride * size % 16 ||
        k_head_stride * size % 16 || v_token_stride * size % 16 || v_head_stride * size % 16 ||
        !aligned(block_table, 4) || !aligned(seq_starts, 4) || !aligned(new_offsets, 4))
        return PAGED_GQA_ERR_ALIGNMENT;
    AppendArgs a{};
    a.src[0] = k;
    a.src[1] = v;
    a.ts[0] = k_token_stride;
    a.ts[1] = v_token_stride;
    a.hs[0] = k_head_stride;
    a.hs[1] = v_head_stride;
    a.cache[0] = static_cast<unsigned char*>(k_cache);
    a.cache[1] = static_cast<unsigned char*>(v_cache);
    a.scales[0] = k_scales;
    a.scales[1] = v_scales;
    a.kv = scaled_geom(k_cache, v_cache, kv_layout, page_size, num_pages);
    a.sc = scale_geom(scale_layout, scale_block);
    a.bt = block_table;
    a.bt_stride = bt_row_stride;
    a.starts = seq_starts;
    a.offs = new_offsets;
    a.B = B;
    a.T = T;
    a.Hkv = Hkv;
    a.max_len = max_seq_len;
    a.err = err_flag;
    return status_of(launch_append(a, src_dtype, kv_dtype == PAGED_GQA_KV_INT8,
                                   static_cast<cudaStream_t>(stream)));
}

size_t paged_gqa_decode_scaled_workspace_size(int B, int Hq, int Hkv, int D, int splits)
{
    if (check_heads(B, Hq, Hkv, D) != PAGED_GQA_OK || splits < 0 || B > kMaxSplitBatch)
        return 0;
    if (splits > 0)
        return scaled_workspace_bytes(B, Hkv, splits);
    int n[2];
    return split_ctas(n) == PAGED_GQA_OK ? scaled_workspace_bytes(B, Hkv, std::max(n[0], n[1])) : 0;
}

int paged_gqa_decode_scaled(const void* q, const void* k_cache, const void* v_cache,
                            paged_gqa_kv_layout kv_layout, int kv_dtype, const float* k_scales,
                            const float* v_scales, paged_gqa_scale_layout scale_layout,
                            int scale_block, const int32_t* block_table, int64_t bt_row_stride,
                            const int32_t* seq_lens, int B, int Hq, int Hkv, int D, int page_size,
                            int num_pages, int max_seq_len, float softmax_scale, void* out,
                            const paged_gqa_workspace* ws, void* stream)
{
    int st = check_heads(B, Hq, Hkv, D);
    if (st != PAGED_GQA_OK)
        return st;
    if (max_seq_len < 0 || bt_row_stride < 0)
        return PAGED_GQA_ERR_SHAPE;
    st = check_scaled_cache(k_cache, v_cache, kv_layout, kv_dtype, k_scales, v_scales, scale_layout,
                            scale_block, page_size, num_pages);
    if (st != PAGED_GQA_OK)
        return st;
    if (B > 1 && bt_row_stride < ((int64_t)max_seq_len + page_size - 1) / page_size)
        return PAGED_GQA_ERR_SHAPE;
    if (B == 0)
        return PAGED_GQA_OK;
    if (q == nullptr || block_table == nullptr || seq_lens == nullptr || out == nullptr)
        return PAGED_GQA_ERR_NULL_POINTER;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
        return PAGED_GQA_ERR_ALIGNMENT;
    const bool int8 = kv_dtype == PAGED_GQA_KV_INT8;
    ScaledDecodeArgs a{};
    a.q = static_cast<const __half*>(q);
    if (!cache_args(a.c, scaled_geom(k_cache, v_cache, kv_layout, page_size, num_pages),
                    scale_geom(scale_layout, scale_block), k_scales, v_scales, Hkv))
        return PAGED_GQA_ERR_UNSUPPORTED;
    a.bt = block_table;
    a.bt_stride = bt_row_stride;
    a.seq_lens = seq_lens;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.max_seq_len = max_seq_len;
    a.scale_log2 = (float)((double)softmax_scale * kLog2e);
    a.out = static_cast<__half*>(out);
    a.err = ws ? ws->err_flag : nullptr;
    choose_cluster((int64_t)B * Hkv, ((int64_t)max_seq_len + kTile - 1) / kTile, a.cluster, a.cluster_warps);
    if (ws != nullptr && ws->ptr != nullptr && B <= kMaxSplitBatch) {
        if (!aligned(ws->ptr, 256))
            return PAGED_GQA_ERR_WORKSPACE;
        int n[2];
        if (split_ctas(n) != PAGED_GQA_OK)
            return PAGED_GQA_ERR_CUDA;
        const int C = ws->force_splits > 0 ? ws->force_splits : n[int8];
        if (scaled_workspace_bytes(B, Hkv, C) > ws->bytes)
            return PAGED_GQA_ERR_WORKSPACE;
        if (ws->force_splits > 0 || split_pays(a, C)) {
            const size_t head = (kHeaderBytes + (size_t)(B + 1) * sizeof(int64_t) + 255) & ~(size_t)255;
            a.C = C;
            a.groups = split_groups(Hkv, C);
            a.heads = Hkv / a.groups;
            a.hdr = static_cast<int64_t*>(ws->ptr);
            a.slots = reinterpret_cast<float*>(static_cast<unsigned char*>(ws->ptr) + head);
            a.min_tiles = ws->force_splits > 0 ? 0 : kSplitMinTiles;
        }
    }
    return status_of(launch_decode_scaled(a, int8, static_cast<cudaStream_t>(stream),
                                          ws ? ws->split_events[0] : nullptr,
                                          ws ? ws->split_events[1] : nullptr));
}

int paged_gqa_sparse_prefill_scaled(const void* q, const void* k_cache, const void* v_cache,
                                    paged_gqa_kv_layout kv_layout, int kv_dtype,
                                    const float* k_scales, const float* v_scales,
                                    paged_gqa_scale_layout scale_layout, int scale_block,
                                    const int32_t* block_table, int num_pages, int kv_len,
                                    const int32_t* sel_idx, int n_sel, const int32_t* q_pos, int R,
                                    int Hq, int Hkv, int D, int page_size, float softmax_scale,
                                    void* out, int* err_flag, void* stream)
{
    int st = check_heads(R, Hq, Hkv, D);
    if (st != PAGED_GQA_OK)
        return st;
    if (n_sel < 0 || n_sel > (1 << 28) || kv_len < 0 || Hkv > 65535)
        return PAGED_GQA_ERR_SHAPE;
    st = check_scaled_cache(k_cache, v_cache, kv_layout, kv_dtype, k_scales, v_scales, scale_layout,
                            scale_block, page_size, num_pages);
    if (st != PAGED_GQA_OK)
        return st;
    if (page_size % 4 != 0)
        return PAGED_GQA_ERR_SHAPE;
    if (R == 0)
        return PAGED_GQA_OK;
    if (q == nullptr || block_table == nullptr || q_pos == nullptr || out == nullptr ||
        (n_sel > 0 && sel_idx == nullptr))
        return PAGED_GQA_ERR_NULL_POINTER;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_table, 4) || !aligned(sel_idx, 4) ||
        !aligned(q_pos, 4))
        return PAGED_GQA_ERR_ALIGNMENT;
    ScaledPrefillArgs a{};
    a.q = static_cast<const __half*>(q);
    if (!cache_args(a.c, scaled_geom(k_cache, v_cache, kv_layout, page_size, num_pages),
                    scale_geom(scale_layout, scale_block), k_scales, v_scales, Hkv))
        return PAGED_GQA_ERR_UNSUPPORTED;
    a.bt = block_table;
    a.kv_len = kv_len;
    a.sel = sel_idx;
    a.n_sel = n_sel;
    a.q_pos = q_pos;
    a.R = R;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.scale_log2 = (float)((double)softmax_scale * kLog2e);
    a.out = static_cast<__half*>(out);
    a.err = err_flag;
    choose_cluster((int64_t)R * Hkv, ((int64_t)n_sel + 4) / 4, a.cluster, a.cluster_warps);
    return status_of(launch_prefill_scaled(a, kv_dtype == PAGED_GQA_KV_INT8,
                                           static_cast<cudaStream_t>(stream)));
}

int paged_gqa_logits_process(const void* logits, int64_t logits_stride, int dtype, float* out,
                             int64_t out_stride, int B, int V, const paged_gqa_logit_rules* rules,
                             int* err_flag, void* stream)
{
    if (B < 0 || B > 65535 || V < 1 || V > INT32_MAX - 8192 || logits_stride < 0 || out_stride < 0)
        return PAGED_GQA_ERR_SHAPE;
    if (B > 1 && out_stride < V)
        return PAGED_GQA_ERR_SHAPE;
    const int size = float_bytes(dtype);
    if (size == 0)
        return PAGED_GQA_ERR_UNSUPPORTED;
    LogitsArgs a{};
    if (rules != nullptr)
        a.r = *rules;
    paged_gqa_logit_rules& r = a.r;
    if (r.history_stride < 0 || r.max_history < 0 || r.max_history > (1 << 28) || r.bias_stride < 0 ||
        r.n_bias < 0 || r.n_bias > (1 << 28) || r.mask_stride < 0 || r.mask_rows < 0)
        return PAGED_GQA_ERR_SHAPE;
    if (r.mask != nullptr && r.mask_index == nullptr && r.mask_rows < B)
        return PAGED_GQA_ERR_SHAPE;
    if (r.mask != nullptr && r.mask_rows > 1 && r.mask_stride < ((int64_t)V + 31) / 32)
        return PAGED_GQA_ERR_SHAPE;
    if (B == 0)
        return PAGED_GQA_OK;
    const bool penalties = r.repetition || r.frequency || r.presence;
    if (logits == nullptr || out == nullptr || (penalties && r.max_history > 0 && !r.history) ||
        (r.n_bias > 0 && (!r.bias_tokens || !r.bias_values)))
        return PAGED_GQA_ERR_NULL_POINTER;
    if (!aligned(logits, size))
        return PAGED_GQA_ERR_ALIGNMENT;
    const void* words[] = {out, r.history, r.history_lens, r.prompt_lens, r.repetition, r.frequency,
                           r.presence, r.bias_tokens, r.bias_values, r.mask, r.mask_index};
    for (const void* p : words)
        if (!aligned(p, 4))
            return PAGED_GQA_ERR_ALIGNMENT;
    if (logits == out && (dtype != PAGED_GQA_F32 || (B > 1 && logits_stride != out_stride)))
        return PAGED_GQA_ERR_SHAPE;
    if (!penalties || r.max_history == 0)
        r.history = nullptr;
    if (r.n_bias == 0)
        r.bias_tokens = nullptr;
    a.x = logits;
    a.x_stride = logits_stride;
    a.out = out;
    a.out_stride = out_stride;
    a.B = B;
    a.V = V;
    a.err = err_flag;
    return status_of(launch_logits(a, dtype, static_cast<cudaStream_t>(stream)));
}

int paged_gqa_rope_call(const paged_gqa_rope_args* c)
{
    if (c == nullptr)
        return PAGED_GQA_ERR_NULL_POINTER;
    return paged_gqa_rope(&c->q, c->k.heads == 0 ? nullptr : &c->k, c->T, c->D, c->dtype, c->positions,
                          c->inv_freq, c->rot_dim, c->layout, c->scale, c->inverse, c->stream);
}

int paged_gqa_append_scaled_call(const paged_gqa_append_scaled_args* c)
{
    if (c == nullptr)
        return PAGED_GQA_ERR_NULL_POINTER;
    return paged_gqa_append_scaled(c->k, c->k_token_stride, c->k_head_stride, c->v, c->v_token_stride,
                                   c->v_head_stride, c->src_dtype, c->T, c->k_cache, c->v_cache,
                                   c->kv_layout, c->kv_dtype, c->k_scales, c->v_scales, c->scale_layout,
                                   c->scale_block, c->block_table, c->bt_row_stride, c->seq_starts,
                                   c->new_offsets, c->B, c->Hkv, c->D, c->page_size, c->num_pages,
                                   c->max_seq_len, c->err_flag, c->stream);
}

int paged_gqa_decode_scaled_call(const paged_gqa_decode_scaled_args* c)
{
    if (c == nullptr)
        return PAGED_GQA_ERR_NULL_POINTER;
    const paged_gqa_workspace ws = {c->workspace, c->workspace_bytes, c->force_splits, c->err_flag,
                                    {c->split_events[0], c->split_events[1]}};
    return paged_gqa_decode_scaled(c->q, c->k_cache, c->v_cache, c->kv_layout, c->kv_dtype, c->k_scales,
                                   c->v_scales, c->scale_layout, c->scale_block, c->block_table,
                                   c->bt_row_stride, c->seq_lens, c->B, c->Hq, c->Hkv, c->D, c->page_size,
                                   c->num_pages, c->max_seq_len, c->softmax_scale, c->out, &ws, c->stream);
}

int paged_gqa_sparse_prefill_scaled_call(const paged_gqa_sparse_prefill_scaled_args* c)
{
    if (c == nullptr)
        return PAGED_GQA_ERR_NULL_POINTER;
    return paged_gqa_sparse_prefill_scaled(c->q, c->k_cache, c->v_cache, c->kv_layout, c->kv_dtype,
                                           c->k_scales, c->v_scales, c->scale_layout, c->scale_block,
                                           c->block_table, c->num_pages, c->kv_len, c->sel_idx, c->n_sel,
                                           c->q_pos, c->R, c->Hq, c->Hkv, c->D, c->page_size,
                                           c->softmax_scale, c->out, c->err_flag, c->stream);
}

int paged_gqa_logits_process_call(const paged_gqa_logits_process_args* c)
{
    if (c == nullptr)
        return PAGED_GQA_ERR_NULL_POINTER;
    return paged_gqa_logits_process(c->logits, c->logits_stride, c->dtype, c->out, c->out_stride, c->B,
                                    c->V, &c->rules, c->err_flag, c->stream);
}

}  // extern "C"
