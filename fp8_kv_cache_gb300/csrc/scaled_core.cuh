// scaled_core.cuh -- the warp core of attention over 8-bit caches with one
// scale for each block of tokens and KV head (E4M3 or INT8 codes).
//
// Mathematics, per query head, in the log2 domain.  Token t has key codes kc_t
// with scale ks_t and value codes vc_t with scale vs_t:
//     x_t = scale log2(e) ks_t <q, kc_t>,  out = sum 2^x_t vs_t vc_t / sum 2^x_t.
// The key scale multiplies the score.  The value scale joins the exponent,
//     y_t = x_t + log2 vs_t,
// and the running maximum n is of y, so that the weights p_t = 2^(y_t - n) fed
// to the second product stay in [0, 1] whatever the scales' range, and
//     out = sum p_t vc_t / sum p_t / vs_t.
// (n is a reference that the maximum may pass by 2^kSlack before the sums are
// rescaled: weights of up to 2^kSlack instead of 1.)  The second product takes
// binary16, so a weight is fed as the sum of two such numbers, its rounding and the
// rounding of what that leaves: 22 bits, below the float32 errors of the scores.
// (One number, 11 bits, moved outputs by as much as their own rounding to binary16
// does: 64 tokens, errors of 2.5e-4 instead of 2.1e-4; prefill took 378 us for
// 414, decode 6.6 for 6.9.)  They are fed as 2^kShift p_t: binary16's steps
// end at 2^-24, which then stands for 2^-(24 + kShift).  The denominator is summed
// from the float32 weights.  Scales below 2^-80 count as 2^-80 in log2 vs: their
// values are zeros in binary16 either way, and the denominator stays finite.
//
// Data path of a warp: a private ring of two 16-token tiles filled by 16-byte
// cp.async (rows of tokens that are not attended are filled with zeros), the 16
// tokens times 8 padded heads by m16n8k16 MMAs, V transposed on its way out of
// shared memory by byte-wise ldmatrix.  A lane looks up one token's place, and the
// places go round by shuffles; the tokens' scales come by 4-byte cp.async beside
// their rows.
//
// Bound where the codes come from L2 (prefill): instructions.  4096 rows x 2050
// E4M3 tokens x 6 heads take 419 us.  At one binary16 number a weight they took 378
// us; 408 us with 64-bit row offsets and four chains of score sums; 531 us also with
// fills of half tiles, a joint maximum over the lanes for every tile (now only when
// one passes the reference by 2^kSlack) and V's bytes paired by permutes; 80 us more
// with a select for every fragment of a row and a rescale whenever a maximum grew.  A
// variant of the fill for tiles whose tokens are all attended gained nothing (385 us:
// more code).
#pragma once

#include <cfloat>

#include "step_internal.h"

namespace pgqa {
namespace scaled {

constexpr float kShift = 6.f;
constexpr float kSlack = 8.f;                // 2^(kShift + kSlack) fits binary16
constexpr float kMinScale = 8.271806125530277e-25f;   // 2^-80

// A 16-token tile in shared memory: K rows of 256 bytes, then V rows.  Their 16-byte
// chunks are swizzled so that the reads below (K: eight rows' fragments by 16-byte
// loads, V: 16 x 16 bytes transposed) meet every bank once.
constexpr int kRowBytes = kD, kTileBytes = 2 * kTile * kRowBytes;

__device__ __forceinline__ uint32_t k_off(int t, int c) { return t * kRowBytes + ((16 * c) ^ (64 * (t & 1))); }
__device__ __forceinline__ uint32_t v_off(int t, int c) { return (kTile + t) * kRowBytes + 16 * (c ^ (t & 7)); }

// Two blocks of 16 rows and 16 bytes, transposed: lane (g, q) gets rows 4q .. 4q + 3
// of column g (r[0], r[2]) and of column g + 8 (r[1], r[3]); lane l passes the address
// of row l mod 16 of block l / 16.
__device__ __forceinline__ void load_transposed(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Four codes (bytes 0..3 of w) -> two f16x2 in order.  Exact: INT8 by placing
// the biased byte in the low bits of 1024 and taking 1152 off.
template <bool kInt8>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    if constexpr (kInt8) {
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t bias = 0x64806480u;   // 1152, 1152
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(bias));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(bias));
    } else {
        e4m3x4_to_f16x2x2(w, lo, hi);
    }
}

// Copies 16 bytes, or writes zeros where `live` is false (src is not read).
__device__ __forceinline__ void cp_async16_or_0(uint32_t dst, const unsigned char* src, bool live)
{
    const int n = live ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// Where a token lies: its row in units of the pools (kNowhere: not attended) and
// element offset into the scale tensors.
constexpr uint32_t kNowhere = 0xFFFFFFFFu;

struct Place {
    uint32_t row;
    int64_t scale;
};

// Scale offset of (page, slot, KV head j).
__device__ __forceinline__ int64_t scale_offset(const ScaleGeom& s, int page, int slot, int j)
{
    const int i = s.shift >= 0 ? slot >> s.shift : slot / s.block;
    return page * s.page + i * s.block_stride + j * s.head;
}

__device__ __forceinline__ Place place_of(const CacheArgs& c, int page, int slot, int j)
{
    return {page * c.page_u + slot * c.token_u + j * c.head_u, scale_offset(c.sc, page, slot, j)};
}

// A warp's ring: the rows of kTiles tiles and their scales (16 of K, 16 of V).
constexpr int kTiles = 2;

struct Ring {
    uint32_t rows;
    float* scales;

    __device__ uint32_t addr(int s) const { return rows + s * kTileBytes; }
    __device__ const float* scale(int s) const { return scales + 32 * s; }

    // Starts filling the place of tile s (one commit group); lane l passes the place
    // of token l mod 16.  Returns the mask of attended tokens.
    __device__ __forceinline__ uint32_t fill(int s, const Place& p, const CacheArgs& c, int lane) const
    {
        const bool live = p.row != kNowhere;
        const uint32_t mask = __ballot_sync(0xffffffffu, live) & 0xFFFFu;
        if (live)
            cp_async4(smem_u32(scales + 32 * s + lane), (lane < 16 ? c.ks : c.vs) + p.scale);
        const int ch = lane & 15, t0 = lane >> 4;
        const uint32_t k_to = addr(s) + k_off(t0, ch), m = mask >> t0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {                    // row 2 k + t0
            const uint64_t o = (uint64_t)__shfl_sync(0xffffffffu, p.row, 2 * k + t0) * c.unit;
            const uint32_t v_to = addr(s) + v_off(2 * (k & 3) + t0, ch) + (k >> 2) * 8 * kRowBytes;
            const bool copied = (m >> (2 * k)) & 1u;
            cp_async16_or_0(k_to + 2 * k * kRowBytes, c.kv.k + 16 * ch + o, copied);
            cp_async16_or_0(v_to, c.kv.v + 16 * ch + o, copied);
        }
        cp_async_commit();
        return mask;
    }
    __device__ void wait() const
    {
        cp_async_wait<kTiles - 1>();
        __syncwarp();
    }
    __device__ void drain() const
    {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    }
};

// Converts G query heads' rows (fp16, [G][256] at qg) into the B fragments of the 16
// k-steps, two to a uint4; the pairs are dealt to nw warps in turn.
__device__ __forceinline__ void stage_q(uint4* qs, const __half* qg, int G, int lane, int w, int nw)
{
    const int g = lane >> 2, q = lane & 3;
    const uint32_t* row = reinterpret_cast<const uint32_t*>(qg + (size_t)g * kD);
    auto two = [&](int i) { return row[WarpCore<true>::k_dim(q, i) >> 1]; };
    for (int s = w; s < 8; s += nw)
        qs[s * 32 + lane] = g < G ? make_uint4(two(8 * s), two(8 * s + 2), two(8 * s + 4), two(8 * s + 6))
                                  : make_uint4(0u, 0u, 0u, 0u);
}

// Attention state of one warp for one (sequence or row, KV head): O^T accumulators
// (acc[i]: dims 16 i + g, of two heads, and 16 i + g + 8), references n and denominators of heads 2q, 2q + 1
// (q = lane & 3; the denominators over the lane's own tokens only).
template <bool kInt8>
struct Core {
    float acc[16][4];
    float n0, n1, d0, d1;

    __device__ void reset()
    {
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                acc[i][c] = 0.f;
        n0 = n1 = -FLT_MAX;          // finite: 2^(-inf - n) is 0, and nothing is -inf - -inf
        d0 = d1 = 0.f;
    }

    // The tile at st, with scales ks of K, then V; bit t of mask says whether token t
    // is attended.  Rows g and g + 8 of the products over tokens are tokens t0 and
    // t0 + 2: a lane's four neighbouring tokens of load_transposed then are the two
    // pairs of its fragments.
    __device__ void tile(uint32_t st, const float* ks, uint32_t mask, const uint4* qs, float scale_log2, int lane)
    {
        const int g = lane >> 2, q = lane & 3, t0 = 4 * (g >> 1) + (g & 1);
        // ---- S^T = K Q^T over the 16 k-steps, two accumulation chains
        float sc[2][4];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sc[c][e] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 k0 = lds128(st + k_off(t0, q + 4 * i));
            const uint4 k1 = lds128(st + k_off(t0, q + 4 * i) + 2 * kRowBytes);
            uint4 b;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (w % 2 == 0)
                    b = qs[(2 * i + w / 2) * 32 + lane];
                uint32_t a0, a1, a2, a3;
                codes_to_f16<kInt8>(word(k0, w), a0, a2);
                codes_to_f16<kInt8>(word(k1, w), a1, a3);
                mma16816(sc[w & 1], a0, a1, a2, a3, w % 2 == 0 ? b.x : b.z, w % 2 == 0 ? b.y : b.w);
            }
        }
        // ---- y = x + log2 vs: lane holds tokens t0, t0 + 2 of heads 2q, 2q + 1
        const bool kv0 = (mask >> t0) & 1u, kv1 = (mask >> (t0 + 2)) & 1u;
        const float kf0 = scale_log2 * ks[t0], kf1 = scale_log2 * ks[t0 + 2];
        const float lv0 = lg2(fmaxf(ks[16 + t0], kMinScale));
        const float lv1 = lg2(fmaxf(ks[18 + t0], kMinScale));
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float dot = sc[0][e] + sc[1][e];
            y[e] = (e < 2 ? kv0 : kv1) ? fmaf(dot, e < 2 ? kf0 : kf1, e < 2 ? lv0 : lv1) : -INFINITY;
        }
        float m0 = fmaxf(y[0], y[2]), m1 = fmaxf(y[1], y[3]);
        if (__any_sync(0xffffffffu, m0 > n0 + kSlack || m1 > n1 + kSlack)) {
            m0 = fmaxf(m0, n0);
            m1 = fmaxf(m1, n1);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
                m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
            }
            const float al0 = ex2(n0 - m0), al1 = ex2(n1 - m1);
            n0 = m0;
            n1 = m1;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                acc[i][0] *= al0;
                acc[i][2] *= al0;
                acc[i][1] *= al1;
                acc[i][3] *= al1;
            }
            d0 *= al0;
            d1 *= al1;
        }
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            p[e] = ex2(y[e] - (((e & 1) ? n1 : n0) - kShift));
        // 1 / vs of a token that is not attended is not taken: its scale may be anything
        const float iv0 = kv0 ? ex2(-lv0) : 0.f, iv1 = kv1 ? ex2(-lv1) : 0.f;
        d0 += p[0] * iv0 + p[2] * iv1;
        d1 += p[1] * iv0 + p[3] * iv1;
        // ---- P fragments: transpose the two 8x8 blocks [token][head] -> [head][token]
        uint32_t pb[2], rest[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t h = pack_half2(p[2 * i], p[2 * i + 1]);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            const uint32_t l = pack_half2(p[2 * i] - f.x, p[2 * i + 1] - f.y);
            asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(pb[i]) : "r"(h));
            asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(rest[i]) : "r"(l));
        }
        // ---- O^T += V^T P^T, 32 dims at a time
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t r[4];
            load_transposed(r, st + v_off(lane & 15, 2 * (i & 3) + (lane >> 4)) + 128 * (i >> 2));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t a0, a1, a2, a3;
                codes_to_f16<kInt8>(r[2 * j], a0, a2);
                codes_to_f16<kInt8>(r[2 * j + 1], a1, a3);
                mma16816(acc[2 * i + j], a0, a1, a2, a3, pb[0], pb[1]);
                mma16816(acc[2 * i + j], a0, a1, a2, a3, rest[0], rest[1]);
            }
        }
    }

    // Sums the denominators over the lanes of a head.
    __device__ void finish()
    {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            d0 += __shfl_xor_sync(0xffffffffu, d0, o);
            d1 += __shfl_xor_sync(0xffffffffu, d1, o);
        }
    }
};

// Runs a warp over 16-token tiles k = first, first + stride, ... < end; at(k)
// gives lane l the place of token l mod 16 of tile k.  begin() is called once
// by every warp when its first tiles are on their way: what they need besides (the
// staged queries) is made ready there.
template <bool kInt8, class At, class Begin>
__device__ __forceinline__ void run_tiles(Core<kInt8>& wc, const Ring& rg, const uint4* qs, const CacheArgs& c,
                                          int first, int end, int stride, float scale_log2, int lane, At at,
                                          Begin begin)
{
    static_assert(kTiles == 2, "two masks to a word");
    uint32_t masks = 0u;                             // of the tile to come, and the one behind it
    int s = 0, k = first;
#pragma unroll 1
    for (int j = 0; j < kTiles; ++j, k += stride) {
        masks >>= 16;
        if (k < end)
            masks |= rg.fill(j, at(k), c, lane) << 16;
        else
            cp_async_commit();
    }
    begin();
    for (; k - kTiles * stride < end; k += stride) {
        rg.wait();
        wc.tile(rg.addr(s), rg.scale(s), masks, qs, scale_log2, lane);
        __syncwarp();
        masks >>= 16;
        if (k < end)
            masks |= rg.fill(s, at(k), c, lane) << 16;
        else
            cp_async_commit();
        s ^= 1;
    }
    rg.drain();
}

// Shared memory of a CTA of kNW warps: Q fragments, rings (the merge buffer
// aliases them), scales, then a kernel's own tail.
template <int kNW>
struct Merge {
    float n[kNW][kGMax], d[kNW][kGMax];
    float o[kNW][kGMax][kD];
};

template <int kNW>
struct Smem {
    static constexpr size_t kQBytes = (size_t)8 * 32 * sizeof(uint4);
    static constexpr size_t kRing = (size_t)kTiles * kTileBytes;         // of a warp
    static constexpr size_t kScaleOff = kQBytes + kNW * kRing;
    static constexpr size_t kTailOff = kScaleOff + (size_t)kNW * kTiles * 32 * sizeof(float);
    static_assert(kNW * kRing >= sizeof(Merge<kNW>), "the merge buffer must fit in the rings");

    uint4* qs;
    Merge<kNW>* merge;              // used only after every ring is drained
    Ring ring;                      // this warp's
    unsigned char* tail;

    __device__ static Smem carve(unsigned char* base, int w)
    {
        Smem s;
        s.qs = reinterpret_cast<uint4*>(base);
        s.merge = reinterpret_cast<Merge<kNW>*>(base + kQBytes);
        s.ring.rows = smem_u32(base + kQBytes + w * kRing);
        s.ring.scales = reinterpret_cast<float*>(base + kScaleOff) + w * kTiles * 32;
        s.tail = base + kTailOff;
        return s;
    }
};

// Four output values of head h, dims 4 c .. 4 c + 3, of partial results with
// maximum n, denominator d and numerators o.
struct Quad {
    float n, d;
    float4 o;
};

__device__ __forceinline__ void store_rows(__half* out_rows, int h, int c, const Quad& v)
{
    const float s = v.d == 0.f ? 0.f : 1.f / v.d;
    __half2* out = reinterpret_cast<__half2*>(out_rows + (size_t)h * kD + 4 * c);
    out[0] = __floats2half2_rn(v.o.x * s, v.o.y * s);
    out[1] = __floats2half2_rn(v.o.z * s, v.o.w * s);
}

// Joins the warps' states and hands every thread its quads of the CTA's result:
// use(h, c, quad) for the G heads and 64 dim quads.  In shared memory quad c of
// head h lies at c ^ 2 (h / 2), so that the lanes of a store, which hold eight
// neighbouring dims of four heads, spread over all banks.
template <bool kInt8, int kNW, class Use>
__device__ __forceinline__ void cta_merge(Merge<kNW>& sm, Core<kInt8>& wc, int G, Use use)
{
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int g = lane >> 2, q = lane & 3;
    wc.finish();
    __syncthreads();           // every ring drained, the previous use of sm finished
    if (g == 0) {
        sm.n[w][2 * q] = wc.n0;
        sm.n[w][2 * q + 1] = wc.n1;
        sm.d[w][2 * q] = wc.d0;
        sm.d[w][2 * q + 1] = wc.d1;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sm.o[w][2 * q + (e & 1)][((16 * i + 8 * (e >> 1)) ^ (8 * q)) + g] = wc.acc[i][e];
    }
    __syncthreads();
    for (int it = tid; it < G * (kD / 4); it += 32 * kNW) {
        const int h = it >> 6, c = it & 63;
        Quad v{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < kNW; ++i)
            v.n = fmaxf(v.n, sm.n[i][h]);
#pragma unroll
        for (int i = 0; i < kNW; ++i) {
            const float e = ex2(sm.n[i][h] - v.n);
            const float4 o = reinterpret_cast<const float4*>(sm.o[i][h])[c ^ (2 * (h >> 1))];
            v.d += e * sm.d[i][h];
            v.o.x += e * o.x;
            v.o.y += e * o.y;
            v.o.z += e * o.z;
            v.o.w += e * o.w;
        }
        use(h, c, v);
    }
}

// ------------------------------------------------------------------ clusters

constexpr int kClusterMax = 8;           // CTAs that share a (sequence or row, KV head), at most

// What the CTAs of a cluster push to the one that finishes their dims: per
// sender and head (n, d), and the numerators of the 256 / cluster dims.
struct Inbox {
    float2 nd[kClusterMax][kGMax];
    float4 o[kGMax * kD / 4];            // sender, head, quad
};

__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}

// Joins the results of a cluster of `size` CTAs (1, 2, 4 or 8; 1 writes its rows
// straight away): quad (h, c) goes to the CTA that finishes its dims, by stores
// into that CTA's shared memory, and after one cluster barrier each CTA writes its
// 256 / size dims of every head.  Every thread calls begin() once, put() for its
// quads, and finish() once.
struct ClusterJoin {
    Inbox& in;
    int size, rank, per;                 // per: quads of a CTA's dims
    bool waited;

    __device__ ClusterJoin(Inbox& inbox, int size_, int rank_)
        : in(inbox), size(size_), rank(rank_), per(kD / 4 / size_), waited(false)
    {
    }
    __device__ static void begin()
    {
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    }
    // Until every CTA of the cluster runs: before the first remote store.
    __device__ void wait_start()
    {
        if (!waited)
            asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        waited = true;
    }
    __device__ void put(int h, int c, const Quad& v, __half* out_rows)
    {
        if (size == 1) {
            store_rows(out_rows, h, c, v);
            return;
        }
        wait_start();
        const int to = c / per;
        const uint32_t o = remote(&in.o[(rank * kGMax + h) * per + c - to * per], to);
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(o), "f"(v.o.x), "f"(v.o.y),
                     "f"(v.o.z), "f"(v.o.w) : "memory");
        if (c < size) {
            const uint32_t nd = remote(&in.nd[rank][h], c);
            asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(nd), "f"(v.n), "f"(v.d) : "memory");
        }
    }
    __device__ void finish(int G, __half* out_rows)
    {
        wait_start();
        if (size == 1)
            return;
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        for (int it = threadIdx.x; it < G * per; it += blockDim.x) {
            const int h = it / per, c = it - h * per;
            Quad v{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
            for (int i = 0; i < size; ++i)
                v.n = fmaxf(v.n, in.nd[i][h].x);
            for (int i = 0; i < size; ++i) {
                const float2 nd = in.nd[i][h];
                const float e = ex2(nd.x - v.n);
                const float4 o = in.o[(i * kGMax + h) * per + c];
                v.d += e * nd.y;
                v.o.x += e * o.x;
                v.o.y += e * o.y;
                v.o.z += e * o.z;
                v.o.w += e * o.w;
            }
            store_rows(out_rows, h, rank * per + c, v);
        }
    }
};

}  // namespace scaled
}  // namespace pgqa
