// append.cu -- new K and V rows quantised into the paged, block-scaled cache.
//
// Mathematics: a (scale block, KV head) shares one scale s that covers the
// largest magnitude m of its rows: E4M3 the smallest power of two with
// m <= 448 s, INT8 m / 127.  code = RNE(x / s), rounded once: for E4M3 the
// quotient by a power of two is exact; for INT8 the nearest integer of x inv,
// inv ~ 1 / s, is corrected by the exact remainder x - q s (encode8).  A block
// that holds rows already keeps the larger of the two scales and codes those rows
// again when it grew.  A stored scale may be smaller than any made here, or for E4M3 no
// power of two: units for which that arithmetic is not exact take a longer way.
//
// Bound: HBM, each source row read once and its codes written once (6825 rows of 16
// bits, what ragged cuts leave of 8190 on average, x 4 heads x K and V: 6.4 us; they
// take 15.3 us for E4M3 in blocks of 64, 18.3 us for INT8, and 5.5 and 6.4 us more where
// the scales of the sequences' first blocks grow and their stored rows are coded again).
// What is left is latency: finding the unit, its rows, the joint maximum and the stores
// follow one another within a CTA, and about 16 warps per SM overlap.  A unit is one
// (block with new rows, KV head, K or V); the block's first new row leads it.  Where a
// unit has one new row (a decode step, blocks of one token) warps take units on their
// own (append_rows_kernel: 16 rows 2.1 us, 2.8 us by CTAs, and where scales grow 2.8 us
// more for E4M3 and 7.3 us for INT8; 8190 rows in blocks of one token 19.7 us, 64 us by
// CTAs).  Else a CTA takes units of one leader, kWarpsPer warps to a unit, enough that a
// warp's rows of the block stay in its registers between the maximum and the codes (up
// to 64 rows a unit; longer blocks are read twice, from L2 the second time), and looks
// through `chunk` consecutive rows for leaders.  A loop over a leader's units, the next
// one's rows prefetched, was slower (14 and 20 us at the time against 12 and 16:
// registers for two units, fewer CTAs); so was reading rows twice to fit more CTAs (four
// rows held: 20 us).
#include <cfloat>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "step_internal.h"

namespace pgqa {

namespace {

// Warps of a CTA, and rows a warp holds in registers: 64 rows a CTA, of 16-bit
// types with four warps, since every warp pays for finding its unit (8190 rows
// in INT8 blocks of 64: 13.9 us, with eight warps of eight rows 16.1 us).
template <class T>
constexpr int kAppendWarps = sizeof(T) == 4 ? 8 : 4;
template <class T>
constexpr int kHeld = 64 / kAppendWarps<T>;
// CTAs per SM that registers for h held rows are meant to leave room for.
template <class T>
constexpr int append_ctas(int h)
{
    return sizeof(T) == 4 ? (h > 4 ? 2 : 3) : h > 8 ? 4 : h > 4 ? 6 : 8;
}
constexpr int64_t kAppendCtas = 3 * kSms;    // CTAs that keep the GPU busy
constexpr int kRowThreads = 128;
constexpr int64_t kRowWarps = 64 * kSms;     // most of one unit

// A lane's 8 elements of a row, as loaded.
template <class T>
struct Row {
    static constexpr int kParts = sizeof(T) / 2;
    uint4 w[kParts];

    __device__ void load(const T* row, int lane)
    {
#pragma unroll
        for (int i = 0; i < kParts; ++i)
            w[i] = reinterpret_cast<const uint4*>(row)[kParts * lane + i];
    }
    __device__ void clear()
    {
#pragma unroll
        for (int i = 0; i < kParts; ++i)
            w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ float get(int e) const
    {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(word(w[e >> 2], e & 3));
        } else {
            const uint32_t v = word(w[0], e >> 1);
            if constexpr (std::is_same_v<T, __half>) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
                return (e & 1) ? f.y : f.x;
            } else {
                return __uint_as_float((e & 1) ? v & 0xFFFF0000u : v << 16);
            }
        }
    }
    // Largest magnitudes so far, of this row too: one number's bits (float32),
    // or two's (16-bit types: of the even and of the odd elements).  Magnitudes
    // order as their bits do, infinities and NaN above every finite one; the
    // 16-bit maxima propagate NaN.
    __device__ void top(uint32_t& m) const
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m = max(m, word(w[i >> 2], i & 3) & 0x7FFFFFFFu);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (std::is_same_v<T, __half>)
                    asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m) : "r"(word(w[0], i) & 0x7FFF7FFFu));
                else
                    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(word(w[0], i) & 0x7FFF7FFFu));
            }
        }
    }
    __device__ static uint32_t top_of(uint32_t m)
    {
        return sizeof(T) == 4 ? m : max(m & 0x7FFFu, m >> 16 & 0x7FFFu);
    }
    // The value of such bits, and whether they are a finite number's.
    __device__ static float value(uint32_t m)
    {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(m);
        else if constexpr (std::is_same_v<T, __half>)
            return __half2float(__ushort_as_half((unsigned short)m));
        else
            return __uint_as_float(m << 16);
    }
    __device__ static bool finite(uint32_t m)
    {
        return m < (sizeof(T) == 4 ? 0x7F800000u : std::is_same_v<T, __half> ? 0x7C00u : 0x7F80u);
    }
};

// Two floats in one register pair, and their fused multiply-add.
struct Pair {
    uint64_t v;

    __device__ static Pair of(float x, float y)
    {
        return {(uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x)};
    }
    __device__ float x() const { return __uint_as_float((uint32_t)v); }
    __device__ float y() const { return __uint_as_float((uint32_t)(v >> 32)); }
};

__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)
{
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}

// The scale of a block whose largest finite magnitude is m.
template <bool kInt8>
__device__ __forceinline__ float block_scale(float m)
{
    if (m == 0.f)
        return 0.f;
    if (kInt8)
        return __fdiv_rn(m, 127.f);
    // m = 1.f * 2^(E - 127) and 448 = 1.75 * 2^8; the scale stays a normal number
    const uint32_t b = __float_as_uint(m);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u);
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// The multiplier encode8 takes for scale s.
__device__ __forceinline__ float inverse_scale(float s)
{
    return s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// RNE(x / s) as a signed byte, for any x and s; inv ~ 1 / s.
__device__ __forceinline__ uint32_t int8_code(float x, float s, float inv)
{
    if (x != x || s == 0.f)
        return 0u;
    if (s < 1e-30f)                                      // s / 2 or 1 / s may leave the range
        return (uint32_t)(int)fmin(fmax(rint((double)x / (double)s), -127.0), 127.0) & 0xFFu;
    float q = rintf(x * inv);                            // within one of the nearest
    const float r = fmaf(-q, s, x), h = 0.5f * s;        // x - q s has no more than 24 bits: exact
    if (fabsf(r) > h || (fabsf(r) == h && ((int)q & 1)))
        q += copysignf(1.f, r);
    return (uint32_t)(int)fminf(fmaxf(q, -127.f), 127.f) & 0xFFu;
}

// x / s (|x| <= 448 s or infinite or NaN) rounded to odd, so that the rounding to E4M3
// is the exact quotient's; 0 where s = 0, but for NaN.  s = m 2^e and x 2^-e, of which
// no bit that could matter is lost, take the division's remainder away from the
// subnormals.
__device__ __forceinline__ float quotient_odd(float x, float s)
{
    if (s == 0.f && x == x)
        return copysignf(0.f, x);
    if (!(fabsf(x) <= FLT_MAX))
        return x;
    int e;
    const float m = frexpf(s, &e), y = scalbnf(x, -e);
    const float q = __fdiv_rn(y, m), r = fmaf(-q, m, y);
    uint32_t b = __float_as_uint(q);
    if (r != 0.f && (b & 1u) == 0u)
        b += ((r > 0.f) == (q > 0.f)) ? 1u : 0xFFFFFFFFu;
    return __uint_as_float(b);
}

// A lane's 8 codes of x / s for any elements and s; out of line, for rows that
// are not plain.
template <class T>
__device__ __noinline__ uint2 int8_codes(Row<T> x, float s, float inv)
{
    uint32_t c[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        c[e >> 2] |= int8_code(x.get(e), s, inv) << (8 * (e & 3));
    return make_uint2(c[0], c[1]);
}

template <class T>
__device__ __forceinline__ uint2 int8_row(const T* row, float s, float inv)
{
    Row<T> x;
    x.load(row, threadIdx.x & 31);
    return int8_codes(x, s, inv);
}

// The same of E4M3, for rows whose scale is not plain: one element (at x) after
// another to its code (at to), without a call, which would make the kernels spill.
template <class T>
__device__ __forceinline__ void e4m3_codes(unsigned char* to, const T* x, float s)
{
#pragma unroll 1
    for (int e = 0; e < 8; ++e)
        to[e] = (unsigned char)e4m3x2(quotient_odd((float)x[e], s), 0.f);
}

// Whether encode8 codes a unit right whose new elements are finite or not and whose
// scale is s: INT8 where s, s / 2 and 1 / s are far from the subnormals, E4M3 where s is
// a normal power of two, so that x inv is the quotient, or 0 with elements of 0.
template <bool kInt8>
__device__ __forceinline__ bool is_plain(bool finite, float s)
{
    return kInt8 ? finite && s >= 1e-30f : (__float_as_uint(s) & 0x7FFFFFu) == 0u && (finite || s > 0.f);
}

// A lane's 8 codes of a plain unit's elements.  INT8: adding 1.5 2^23
// to x inv rounds to the nearest integer, in the low byte, and is within one of
// the quotient's; the exact remainders say whether one of the eight is off
// (their largest is half a step or more: rare, and a matter of ties).
template <bool kInt8, class T>
__device__ __forceinline__ uint2 encode8(const Row<T>& x, float s, float inv)
{
    uint32_t c[2];
    if constexpr (kInt8) {
        constexpr float kMagic = 12582912.f;
        const float h = 0.5f * s;
        const Pair inv2 = Pair::of(inv, inv), s2 = Pair::of(s, s), magic = Pair::of(kMagic, kMagic);
        const Pair minus = Pair::of(-1.f, -1.f);
        float f[8], far = 0.f;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const Pair v = Pair::of(x.get(e), x.get(e + 1)), t = fma2(v, inv2, magic);
            const Pair r = fma2(fma2(t, minus, magic), s2, v);
            far = fmaxf(far, fmaxf(fabsf(r.x()), fabsf(r.y())));
            f[e] = t.x();
            f[e + 1] = t.y();
        }
        if (far >= h) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float r = fmaf(kMagic - f[e], s, x.get(e));
                if (fabsf(r) > h || (fabsf(r) == h && (__float_as_uint(f[e]) & 1u)))
                    f[e] += copysignf(1.f, r);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = __byte_perm(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), 0x0040);
            const uint32_t hi = __byte_perm(__float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]), 0x0040);
            c[i] = __byte_perm(lo, hi, 0x5410);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            c[i] = e4m3x2(x.get(4 * i) * inv, x.get(4 * i + 1) * inv) |
                   e4m3x2(x.get(4 * i + 2) * inv, x.get(4 * i + 3) * inv) << 16;
    }
    return make_uint2(c[0], c[1]);
}

// c * s rounded to odd, so that a later rounding to fewer bits is the exact
// product's.
__device__ __forceinline__ float mul_odd(float c, float s)
{
    const float p = c * s, err = fmaf(c, s, -p);
    uint32_t b = __float_as_uint(p);
    if (err != 0.f && (b & 1u) == 0u)
        b += ((err > 0.f) == (p > 0.f)) ? 1u : 0xFFFFFFFFu;
    return __uint_as_float(b);
}

// RNE(c old / s) of a stored INT8 code as a byte, s > old.  The product is
// p + lo exactly, the remainder p - q s too, and the sign of its distance from
// half a step decides.
__device__ __forceinline__ uint32_t int8_recode(int c, float old, float s, float inv)
{
    const float p = (float)c * old, lo = fmaf((float)c, old, -p), h = 0.5f * s;
    float q = rintf(p * inv);
    const float r = fmaf(-q, s, p);
    const float up = (r - h) + lo, down = (r + h) + lo;
    const bool odd = (int)q & 1;
    q += (up > 0.f || (up == 0.f && odd)) ? 1.f : (down < 0.f || (down == 0.f && odd)) ? -1.f : 0.f;
    return (uint32_t)(int)q & 0xFFu;
}

// The same of eight codes in 64 bits, for scales so small that lo, s / 2 or
// 1 / s may leave the range.
__device__ __noinline__ uint2 int8_recode_small(uint2 w, float old, float s)
{
    uint32_t r[2] = {0u, 0u};
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
        const int c = (int8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3)));
        r[e >> 2] |= ((uint32_t)(int)rint((double)c * (double)old / (double)s) & 0xFFu) << (8 * (e & 3));
    }
    return make_uint2(r[0], r[1]);
}

// Eight stored codes of scale `old`, coded again for scale s (inv = 1 / s).
template <bool kInt8>
__device__ __forceinline__ uint2 recode8(uint2 w, float old, float s, float inv)
{
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t v = i == 0 ? w.x : w.y;
        if constexpr (kInt8) {
            r[i] = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                r[i] |= int8_recode((int8_t)(v >> (8 * e)), old, s, inv) << (8 * e);
        } else {
            uint32_t lo, hi;
            e4m3x4_to_f16x2x2(v, lo, hi);
            const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
            const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
            r[i] = e4m3x2(mul_odd(a.x, old) * inv, mul_odd(a.y, old) * inv) |
                   e4m3x2(mul_odd(b.x, old) * inv, mul_odd(b.y, old) * inv) << 16;
        }
    }
    return make_uint2(r[0], r[1]);
}

// A lane's codes of n rows `step` bytes apart, coded again; the next row is loaded
// ahead.  old: negative where the stored scale was none.
template <bool kInt8>
__device__ __forceinline__ void recode_rows(unsigned char* row, int64_t step, int n, float old, float s, float inv)
{
    const bool small = kInt8 && (s < 1e-30f || old < 1e-30f);
    const bool zeros = kInt8 ? !(old > 0.f) : old < 0.f;     // E4M3 keeps its NaN under a scale of 0
    if (!kInt8 && old < 0x1p-60f) {                      // code * old and its error stay normal numbers
        old *= 0x1p64f;
        inv *= 0x1p-64f;
    }
    uint2 next = n > 0 ? *reinterpret_cast<uint2*>(row) : make_uint2(0u, 0u);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const uint2 now = next;
        uint2* at = reinterpret_cast<uint2*>(row);
        row += step;
        if (i + 1 < n)
            next = *reinterpret_cast<uint2*>(row);
        *at = zeros ? make_uint2(0u, 0u) : small ? int8_recode_small(now, old, s) : recode8<kInt8>(now, old, s, inv);
    }
}

// The last i < B with offs[i] <= row < offs[i + 1], or -1.  Every thread of the
// CTA calls it, with one round of loads; those of starts bring its line into L1.
__device__ __forceinline__ int sequence_of(const AppendArgs& a, int row, int* found)
{
    __syncthreads();                                     // found may still be read
    if (threadIdx.x == 0)
        *found = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < a.B; i += blockDim.x) {
        const int o = a.offs[i], o1 = a.offs[i + 1];
        asm volatile("prefetch.global.L1 [%0];" ::"l"(a.starts + i));
        if (o <= row && row < o1)
            atomicMax(found, i);
    }
    __syncthreads();
    return *found;
}

}  // namespace

// The largest of the values the kWarpsPer warps of a unit pass, for each unit
// of the CTA.  Every thread calls it.
template <int kWarpsPer>
__device__ __forceinline__ uint32_t unit_max(uint32_t m, uint32_t* red)
{
    m = __reduce_max_sync(0xffffffffu, m);
    if constexpr (kWarpsPer > 1) {
        const int w = threadIdx.x >> 5;
        __syncthreads();                                 // red may still be read
        if ((threadIdx.x & 31) == 0)
            red[w] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarpsPer; ++i)
            m = max(m, red[w / kWarpsPer * kWarpsPer + i]);
    }
    return m;
}

// grid (ceil(T / chunk), ceil(2 Hkv / kUnits)): chunk of rows; kUnits of a
// leader's units (all heads' K, then all heads' V).
template <class T, bool kInt8, int kWarpsPer, int H>
__global__ void __launch_bounds__(32 * kAppendWarps<T>, append_ctas<T>(H)) append_kernel(AppendArgs a)
{
    constexpr int kUnits = kAppendWarps<T> / kWarpsPer;
    __shared__ int found;
    __shared__ uint32_t red[kAppendWarps<T>];
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) % kWarpsPer;
    const int unit = blockIdx.y * kUnits + (threadIdx.x >> 5) / kWarpsPer;
    const bool active = unit < 2 * a.Hkv;                // idle warps keep to the barriers
    const int side = active && unit >= a.Hkv, j = active ? unit - side * a.Hkv : 0;
    const T* src = static_cast<const T*>(a.src[side]) + j * a.hs[side];
    const int64_t ts = a.ts[side], token_b = a.kv.token_b;
    const int block = a.sc.block;
    int flags = 0;
    enter();

    int64_t row = (int64_t)blockIdx.x * a.chunk;
    const int64_t row1 = min((int64_t)a.T, row + a.chunk);
    while (row < row1) {
        // the row's sequence b, its first row and the row behind its last
        int b = (int)row;
        int64_t off = row, end = row + 1;
        if (a.offs != nullptr) {
            b = sequence_of(a, (int)row, &found);
            if (b < 0) {
                // in front of the first sequence, or behind the last one
                const int o = a.offs[0];
                if (o <= row)
                    break;
                row = o;
                continue;
            }
            off = max(a.offs[b], 0);
            end = min(a.offs[b + 1], a.T);
        }
        const int start = a.starts[b];
        if (start < 0) {
            flags |= PAGED_GQA_FLAG_EMPTY_ROW;
            row = end;
            continue;
        }
        const int64_t stop = off + a.max_len - start;    // rows from here on lie past max_len
        if (stop < end)
            flags |= PAGED_GQA_FLAG_SEQ_CLAMPED;
        const int64_t last = min(end, stop);
        while (row < row1 && row < last) {
            const int pos = start + (int)(row - off);
            int pi, slot;
            page_and_slot(a.kv, pos, pi, slot);
            const int sb = slot / block, held = slot - sb * block;
            const int n = (int)min(last - row, (int64_t)(block - held));
            const bool leads = held == 0 || row == off;
            const T* x0 = src + (row + w) * ts;
            row += n;
            if (!leads)
                continue;                                // the rest of another CTA's block
            // ---- largest magnitude of the new rows: rows w, w + kWarpsPer, ... are the warp's
            const int mine = active ? (n - w + kWarpsPer - 1) / kWarpsPer : 0;
            const int64_t step = ts * kWarpsPer;
            Row<T> x[H];
            uint32_t m = 0u;
            for (int i0 = 0; i0 < mine; i0 += H) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    if (i0 + i < mine)
                        x[i].load(x0 + (i0 + i) * step, lane);
                    else
                        x[i].clear();
                }
#pragma unroll
                for (int i = 0; i < H; ++i)
                    x[i].top(m);
            }
            const int page = table_page<false>(a.kv, a.bt + b * a.bt_stride, pi, flags);
            if (page < 0)
                continue;                                // every warp has the same page
            float* scale = a.scales[side] + page * a.sc.page + sb * a.sc.block_stride + j * a.sc.head;
            float old = held > 0 && active ? *scale : 0.f;
            uint32_t mm = unit_max<kWarpsPer>(Row<T>::top_of(m), red);
            const bool finite = Row<T>::finite(mm);
            if (__syncthreads_or(!finite)) {
                // again, finite elements only
                m = 0u;
                for (int i = 0; i < mine; ++i) {
                    Row<T> r;
                    r.load(x0 + i * step, lane);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float f = fabsf(r.get(e));
                        if (f <= FLT_MAX)
                            m = max(m, __float_as_uint(f));
                        else
                            flags |= PAGED_GQA_FLAG_BAD_VALUE;
                    }
                }
                mm = unit_max<kWarpsPer>(m, red);
            } else {
                mm = __float_as_uint(Row<T>::value(mm));
            }
            if (!(old >= 0.f && old <= FLT_MAX)) {
                flags |= PAGED_GQA_FLAG_BAD_VALUE;
                old = -1.f;                              // its rows become zeros
            }
            const float s = fmaxf(fmaxf(old, 0.f), block_scale<kInt8>(__uint_as_float(mm)));
            const float inv = inverse_scale(s);
            unsigned char* rows = a.cache[side] + j * a.kv.head_b + page * a.kv.page_b +
                                  (int64_t)(slot - held) * token_b + 8 * lane;
            // ---- stored rows, where the scale grew
            if (active && held > 0 && s != old) {
                recode_rows<kInt8>(rows + w * token_b, kWarpsPer * token_b, (held - w + kWarpsPer - 1) / kWarpsPer,
                                   old, s, inv);
            }
            // ---- new rows
            rows += (int64_t)(held + w) * token_b;
            const int64_t row_step = token_b * kWarpsPer;
            for (int i0 = 0; i0 < mine; i0 += H) {
                if (mine > H) {
#pragma unroll
                    for (int i = 0; i < H; ++i)
                        if (i0 + i < mine)
                            x[i].load(x0 + (i0 + i) * step, lane);
                }
#pragma unroll
                for (int i = 0; i < H; ++i)
                    if (i0 + i < mine)
                        *reinterpret_cast<uint2*>(rows + (i0 + i) * row_step) = encode8<kInt8>(x[i], s, inv);
            }
            if (!is_plain<kInt8>(finite, s)) {
                for (int i = 0; i < mine; ++i) {
                    if constexpr (kInt8)
                        *reinterpret_cast<uint2*>(rows + i * row_step) = int8_row(x0 + i * step, s, inv);
                    else
                        e4m3_codes(rows + i * row_step, x0 + i * step + 8 * lane, s);
                }
            }
            // the unit's warps have all read the old scale before the barrier above
            if (active && w == 0 && lane == 0)
                *scale = s;
        }
        if (row >= last)
            row = max(row, end);
    }
    raise_flag(a.err, flags);
}

// Rows that are their blocks' only new ones (one row to a sequence, or blocks of one
// token): a warp takes U units of a row and meets no other warp.
// grid (ceil(T ceil(2 Hkv / U) / warps)).
template <class T, bool kInt8, int U>
__global__ void __launch_bounds__(kRowThreads, U > 1 ? 5 : 8) append_rows_kernel(AppendArgs a)
{
    const int lane = threadIdx.x & 31, units = 2 * a.Hkv, parts = (units + U - 1) / U;
    const int64_t wi = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int64_t row = wi / parts;
    const int u0 = (int)(wi - row * parts) * U;
    enter();
    if (row >= a.T)
        return;
    int flags = 0;
    Row<T> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int side = u0 + u >= a.Hkv;
        if (u0 + u < units)
            x[u].load(static_cast<const T*>(a.src[side]) + row * a.ts[side] + (u0 + u - side * a.Hkv) * a.hs[side],
                      lane);
        else
            x[u].clear();
    }
    // ---- the row's sequence and place
    int b = (int)row;
    int64_t off = row;
    if (a.offs != nullptr) {
        b = -1;
        for (int i = lane; i < a.B; i += 32) {
            const int o = a.offs[i], o1 = a.offs[i + 1];
            asm volatile("prefetch.global.L1 [%0];" ::"l"(a.starts + i));
            b = o <= row && row < o1 ? i : b;
        }
        b = __reduce_max_sync(0xffffffffu, b);
        if (b < 0)
            return;                                      // no sequence's
        off = max(a.offs[b], 0);
    }
    const int start = a.starts[b];
    const bool past = row >= off + a.max_len - start;
    int page = -1, slot = 0;
    if (start < 0) {
        flags |= PAGED_GQA_FLAG_EMPTY_ROW;
    } else if (past) {
        flags |= PAGED_GQA_FLAG_SEQ_CLAMPED;
    } else {
        int pi;
        page_and_slot(a.kv, start + (int)(row - off), pi, slot);
        page = table_page<false>(a.kv, a.bt + b * a.bt_stride, pi, flags);
    }
    if (page < 0) {
        raise_flag(a.err, flags);
        return;
    }
    const int block = a.sc.block, sb = slot / block, held = slot - sb * block;
    float* scale[U];
    float old[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int side = u0 + u >= a.Hkv, j = u0 + u - side * a.Hkv;
        scale[u] = a.scales[side] + page * a.sc.page + sb * a.sc.block_stride + j * a.sc.head;
        old[u] = held > 0 && u0 + u < units ? *scale[u] : 0.f;
    }
    // ---- the units one after another
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (u0 + u >= units)
            break;
        const int side = u0 + u >= a.Hkv, j = u0 + u - side * a.Hkv;
        uint32_t m = 0u;
        x[u].top(m);
        m = __reduce_max_sync(0xffffffffu, Row<T>::top_of(m));
        const bool finite = Row<T>::finite(m);
        if (finite) {
            m = __float_as_uint(Row<T>::value(m));
        } else {
            m = 0u;                                      // again, finite elements only
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = fabsf(x[u].get(e));
                if (f <= FLT_MAX)
                    m = max(m, __float_as_uint(f));
                else
                    flags |= PAGED_GQA_FLAG_BAD_VALUE;
            }
            m = __reduce_max_sync(0xffffffffu, m);
        }
        if (!(old[u] >= 0.f && old[u] <= FLT_MAX)) {
            flags |= PAGED_GQA_FLAG_BAD_VALUE;
            old[u] = -1.f;                               // its rows become zeros
        }
        const float s = fmaxf(fmaxf(old[u], 0.f), block_scale<kInt8>(__uint_as_float(m)));
        const float inv = inverse_scale(s);
        unsigned char* to = a.cache[side] + j * a.kv.head_b + page * a.kv.page_b + slot * a.kv.token_b + 8 * lane;
        if (is_plain<kInt8>(finite, s))
            *reinterpret_cast<uint2*>(to) = encode8<kInt8>(x[u], s, inv);
        else if constexpr (kInt8)
            *reinterpret_cast<uint2*>(to) = int8_codes(x[u], s, inv);
        else
            e4m3_codes(to, static_cast<const T*>(a.src[side]) + row * a.ts[side] + j * a.hs[side] + 8 * lane, s);
        if (held > 0 && s != old[u])
            recode_rows<kInt8>(to - held * a.kv.token_b, a.kv.token_b, held, old[u], s, inv);
        __syncwarp();                                    // every lane has read the old scale
        if (lane == 0)
            *scale[u] = s;
    }
    raise_flag(a.err, flags);
}

namespace {

template <class T, bool kInt8, int kWarpsPer, int H = kHeld<T>>
cudaError_t append_run(AppendArgs a, cudaStream_t s)
{
    constexpr int kUnits = kAppendWarps<T> / kWarpsPer;
    const int64_t y = (2 * a.Hkv + kUnits - 1) / kUnits;
    // Few rows a CTA while that does not fill the GPU, at most a block of them.
    a.chunk = (int)std::clamp<int64_t>(a.T * y / kAppendCtas, 1, a.sc.block);
    const int64_t chunks = ((int64_t)a.T + a.chunk - 1) / a.chunk;
    return launch_step(append_kernel<T, kInt8, kWarpsPer, H>, dim3((unsigned)chunks, (unsigned)y),
                       32 * kAppendWarps<T>, 0, s, 0, a);
}

template <class T, bool kInt8, int U>
cudaError_t append_rows(const AppendArgs& a, cudaStream_t s)
{
    const int64_t warps = (int64_t)a.T * ((2 * a.Hkv + U - 1) / U), per = kRowThreads / 32;
    return launch_step(append_rows_kernel<T, kInt8, U>, dim3((unsigned)((warps + per - 1) / per)), kRowThreads, 0, s,
                       0, a);
}

template <class T, bool kInt8>
cudaError_t append_typed(const AppendArgs& a, cudaStream_t s)
{
    // One unit to a warp while they are few, then as many as fit its registers
    // (8190 rows x 8 units, blocks of one token, E4M3, at the time: eight units 18.4 us,
    // four 19.8, two 31 and one 43 us; 1024 rows: eight 4.6 us, one 3.9 us).
    if (a.offs == nullptr || a.sc.block == 1)
        return (int64_t)a.T * 2 * a.Hkv <= kRowWarps ? append_rows<T, kInt8, 1>(a, s)
                                                     : append_rows<T, kInt8, 16 / sizeof(T)>(a, s);
    constexpr int kMost = kAppendWarps<T>;
    // short blocks: fewer rows held, more CTAs (8190 rows, E4M3, blocks of four 14.8
    // us, 22 us with sixteen held; of eight 14.0 and 16.7 us)
    if (a.sc.block <= 4)
        return append_run<T, kInt8, 1, 4>(a, s);
    if (a.sc.block <= 8)
        return append_run<T, kInt8, 1, 8>(a, s);
    if (a.sc.block <= kHeld<T>)
        return append_run<T, kInt8, 1>(a, s);
    if (kMost > 4 && a.sc.block <= kHeld<T> * kMost / 4)
        return append_run<T, kInt8, kMost / 4>(a, s);
    if (a.sc.block <= kHeld<T> * kMost / 2)
        return append_run<T, kInt8, kMost / 2>(a, s);
    return append_run<T, kInt8, kMost>(a, s);
}

template <class T>
cudaError_t append_kind(const AppendArgs& a, bool int8, cudaStream_t s)
{
    return int8 ? append_typed<T, true>(a, s) : append_typed<T, false>(a, s);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int src_dtype, bool int8, cudaStream_t s)
{
    switch (src_dtype) {
    case PAGED_GQA_F16: return append_kind<__half>(a, int8, s);
    case PAGED_GQA_BF16: return append_kind<__nv_bfloat16>(a, int8, s);
    default: return append_kind<float>(a, int8, s);
    }
}

}  // namespace pgqa
