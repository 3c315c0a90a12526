// rope.cu -- rotary positions of q and k rows.
//
// Mathematics: pair i of token t turns by a = pos_t * f_i.  cos and sin depend
// on a modulo one turn only, so the angle is kept as a fraction of a turn in
// 64-bit fixed point: u_i = frac(f_i / 2 pi) * 2^64, and pos_t * u_i modulo
// 2^64 (an integer product that wraps) is the reduced angle, off by |pos| 2^-64
// turns and the 2^-63 relative error of u -- no float32 product of a far
// position, and no 64-bit floating-point work (that pipe is slow on this GPU).
// Its upper 32 bits give the quadrant and a remainder of at most an eighth of a
// turn for sincospif.
//
// Bound: HBM, every row read once and written once.  A warp takes one token and
// a share of its heads.  It computes the token's (cos, sin) pairs once, 32 at a
// time, and each lane keeps those of its own two vectors of a row in registers
// for all its rows; two rows are in flight per lane.  (A block per token with
// the pairs in shared memory and one or two rows in flight took 46 us for 8191
// tokens x 28 heads of 256 16-bit elements, with four in flight, at fewer
// warps, 73 us.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "step_internal.h"

namespace pgqa {

namespace {

constexpr int kRopeThreads = 128;

template <class T> __device__ __forceinline__ float to_float(T x);
template <> __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_float(float x) { return x; }
template <class T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ float from_float(float x) { return x; }

// N elements as they lie in memory, and element pairs (2i, 2i + 1) as floats.
template <class T, int N>
struct alignas(sizeof(T) * N) Vec {
    using Word = std::conditional_t<sizeof(T) == 4, float2, uint32_t>;
    Word w[N / 2];

    __device__ float2 get(int i) const
    {
        if constexpr (sizeof(T) == 4)
            return w[i];
        else if constexpr (std::is_same_v<T, __half>)
            return __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        else
            return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    __device__ void set(int i, float x, float y)
    {
        if constexpr (sizeof(T) == 4) {
            w[i] = make_float2(x, y);
        } else if constexpr (std::is_same_v<T, __half>) {
            const __half2 h = __floats2half2_rn(x, y);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
};

// frac(f / 2 pi) in units of 2^-64 turns (negative f: the negative, modulo
// 2^64), in integers: f = M 2^(e - 63), 64-bit M, and 2 / pi = C 2^-64.
__device__ __forceinline__ uint64_t turns_of(double f)
{
    const uint64_t bits = (uint64_t)__double_as_longlong(f);
    const uint64_t M = (bits << 11) | (1ull << 63);
    const int sh = (int)((bits >> 52) & 0x7FFu) - 1024;      // e - 1
    const uint64_t P = __umul64hi(M, 0xA2F9836E4E44152Aull);
    uint64_t u = 0;
    if (sh >= 0)
        u = sh < 64 ? P << sh : 0ull;
    else if (sh > -64)
        u = (P + (1ull << (-sh - 1))) >> -sh;                // P < 2^63.4: the sum does not wrap
    return (bits >> 63) ? 0ull - u : u;
}

// (cos, sin) of pos * u / 2^64 turns.
__device__ __forceinline__ float2 cos_sin(int pos, uint64_t u)
{
    const uint64_t phase = (uint64_t)(int64_t)pos * u + 0x80000000ull;
    const uint32_t p = (uint32_t)(phase >> 32);
    const uint32_t quad = (p + 0x20000000u) >> 30;           // nearest quarter turn, modulo 4
    const float x = (float)(int32_t)(p - (quad << 30)) * (1.0f / 2147483648.0f);
    float s, c;
    sincospif(x, &s, &c);
    const float cc = (quad & 1u) ? s : c, ss = (quad & 1u) ? c : s;
    return make_float2((quad == 1u || quad == 2u) ? -cc : cc, (quad & 2u) ? -ss : ss);
}

// How a row of D elements falls into items of two vectors of N: first the
// items that turn (kHalf: vectors i and i + pairs / N, element against element;
// else vectors i and i + half of the turning ones, of whole pairs), then the
// ones that pass through.  Neighbouring lanes have neighbouring vectors.
template <int N, bool kHalf>
struct Items {
    int turning, all, rot, D;

    __host__ __device__ Items(int rot_, int D_) : rot(rot_), D(D_)
    {
        turning = kHalf ? rot / 2 / N : (rot / N + 1) / 2;
        all = turning + ((D - rot) / N + 1) / 2;
    }
    // Offsets of item i's vectors; the second is -1 where there is none.
    __device__ void place(int i, int& a, int& b) const
    {
        if (i < turning) {
            a = i * N;
            b = a + turning * N;
            if (b >= rot)
                b = -1;
        } else {
            a = rot + (i - turning) * N;
            b = a + (all - turning) * N;
            if (b >= D)
                b = -1;
        }
    }
};

}  // namespace

// Warps take (token, share of heads): a token's rows in steps of 32 / lanes are
// dealt to its `shares` warps.  lanes: a power of two, at most 32.
template <class T, int N, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a, int lanes, int shares)
{
    extern __shared__ __align__(16) float2 cs[];              // pairs of each warp's token
    using V = Vec<T, N>;
    const Items<N, kHalf> items(a.rot, a.D);
    const int pairs = a.rot >> 1, lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    enter();
    if (warp >= (int64_t)a.T * shares)
        return;
    const int t = (int)(warp / shares), share = (int)(warp - (int64_t)t * shares);
    float2* c = cs + (threadIdx.x >> 5) * pairs;
    const int Hq = a.t[0].heads, H = Hq + a.t[1].heads;
    const int rows = 32 / lanes, row = lane / lanes;
    const T* xq = static_cast<const T*>(a.t[0].x) + t * a.t[0].token_stride;
    const T* xk = static_cast<const T*>(a.t[1].x) + t * a.t[1].token_stride;
    T* oq = static_cast<T*>(a.t[0].out) + t * a.t[0].out_token_stride;
    T* ok = static_cast<T*>(a.t[1].out) + t * a.t[1].out_token_stride;
    const int step = rows * shares;

    bool ready = false;
    for (int i0 = 0; i0 < items.all; i0 += lanes) {
        const int i = i0 + (lane & (lanes - 1));
        const bool some = i < items.all, turns = i < items.turning;
        int da = 0, db = -1;
        if (some)
            items.place(i, da, db);
        auto load = [&](int h, V& u, V& v) {
            if (some && h < H) {
                const T* x = h < Hq ? xq + h * a.t[0].head_stride : xk + (h - Hq) * a.t[1].head_stride;
                u = *reinterpret_cast<const V*>(x + da);
                if (db >= 0)
                    v = *reinterpret_cast<const V*>(x + db);
            }
        };
        int h = share * rows + row;
        V u0, v0, u1, v1;
        load(h, u0, v0);
        load(h + step, u1, v1);
        if (!ready) {
            // the first rows are on their way while the angles are computed
            const int pos = a.pos[t];
#pragma unroll 4
            for (int p = lane; p < pairs; p += 32) {
                const float2 r = cos_sin(pos, turns_of(a.freq[p]));
                c[p] = make_float2(a.scale * r.x, a.inverse ? -a.scale * r.y : a.scale * r.y);
            }
            __syncwarp();
            ready = true;
        }
        // kHalf: pairs da .. da + N - 1; else those of the first vector, then of the second
        float2 w[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int p = kHalf ? da + e : e < N / 2 ? da / 2 + e : db / 2 + e - N / 2;
            w[e] = turns && (kHalf || e < N / 2 || db >= 0) ? c[p] : make_float2(1.f, 0.f);
        }
        auto store = [&](int h, V& u, V& v) {
            if (!some || h >= H)
                return;
            if (turns) {
                if constexpr (kHalf) {
#pragma unroll
                    for (int e = 0; e < N / 2; ++e) {
                        const float2 x = u.get(e), y = v.get(e), r = w[2 * e], s = w[2 * e + 1];
                        u.set(e, x.x * r.x - y.x * r.y, x.y * s.x - y.y * s.y);
                        v.set(e, y.x * r.x + x.x * r.y, y.y * s.x + x.y * s.y);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < N / 2; ++e) {
                        const float2 x = u.get(e), y = v.get(e), r = w[e], s = w[N / 2 + e];
                        u.set(e, x.x * r.x - x.y * r.y, x.y * r.x + x.x * r.y);
                        v.set(e, y.x * s.x - y.y * s.y, y.y * s.x + y.x * s.y);
                    }
                }
            }
            T* out = h < Hq ? oq + h * a.t[0].out_head_stride : ok + (h - Hq) * a.t[1].out_head_stride;
            *reinterpret_cast<V*>(out + da) = u;
            if (db >= 0)
                *reinterpret_cast<V*>(out + db) = v;
        };
        for (; h < H + row; h += 2 * step) {                  // the same trips for every lane
            store(h, u0, v0);
            load(h + 2 * step, u0, v0);
            store(h + step, u1, v1);
            load(h + 3 * step, u1, v1);
        }
    }
}

// Rows on which no vector fits: a pair of elements at a time.
template <class T>
__global__ void __launch_bounds__(kRopeThreads) rope_pairs_kernel(RopeArgs a)
{
    const int t = blockIdx.x, pairs = a.rot >> 1, items = pairs + a.D - a.rot;
    const int Hq = a.t[0].heads, H = Hq + a.t[1].heads;
    enter();
    const int pos = a.pos[t];
    for (int i = threadIdx.x; i < items; i += kRopeThreads) {
        float2 r = make_float2(0.f, 0.f);
        if (i < pairs) {
            r = cos_sin(pos, turns_of(a.freq[i]));
            r = make_float2(a.scale * r.x, a.inverse ? -a.scale * r.y : a.scale * r.y);
        }
        const int d0 = a.half ? i : 2 * i, d1 = a.half ? i + pairs : 2 * i + 1;
        for (int h = 0; h < H; ++h) {
            const paged_gqa_rope_rows& m = a.t[h < Hq ? 0 : 1];
            const int hh = h < Hq ? h : h - Hq;
            const T* x = static_cast<const T*>(m.x) + t * m.token_stride + hh * m.head_stride;
            T* out = static_cast<T*>(m.out) + t * m.out_token_stride + hh * m.out_head_stride;
            if (i < pairs) {
                const float p = to_float(x[d0]), q = to_float(x[d1]);
                out[d0] = from_float<T>(p * r.x - q * r.y);
                out[d1] = from_float<T>(q * r.x + p * r.y);
            } else {
                out[i + pairs] = x[i + pairs];
            }
        }
    }
}

namespace {

// Whether vectors of n elements of `size` bytes fit every row's address and
// every boundary of the row.
bool rope_fits(const RopeArgs& a, int size, int n)
{
    if (a.D % n || a.rot % n || (a.half && (a.rot / 2) % n))
        return false;
    for (const paged_gqa_rope_rows& m : a.t) {
        if (m.heads == 0)
            continue;
        const uintptr_t p = reinterpret_cast<uintptr_t>(m.x) | reinterpret_cast<uintptr_t>(m.out);
        const int64_t st = m.token_stride | m.head_stride | m.out_token_stride | m.out_head_stride;
        if (p % (size * n) || st % n)
            return false;
    }
    return true;
}

template <class T, int N, bool kHalf>
cudaError_t rope_run(const RopeArgs& a, cudaStream_t s)
{
    const int pairs = a.rot / 2, H = a.t[0].heads + a.t[1].heads;
    const int items = Items<N, kHalf>(a.rot, a.D).all;
    int lanes = 1;
    while (lanes < items && lanes < 32)
        lanes <<= 1;
    // Warps of a token: as many as have rows while the SMs have room (32 warps
    // each), then fewer with more rows for the same angles (1024 tokens: 5
    // warps each 6.6 us, 10 warps 7.9 us).
    const int64_t steps = (H + 32 / lanes - 1) / (32 / lanes);
    const int64_t shares = std::clamp<int64_t>((32 * kSms + a.T - 1) / a.T, 1, steps);
    int threads = kRopeThreads;                               // fewer where the pairs are many: 48 KB
    while (threads > 32 && (size_t)(threads / 32) * pairs * sizeof(float2) > 48 * 1024)
        threads /= 2;
    const int64_t warps = a.T * shares, per = threads / 32;
    const int64_t grid = (warps + per - 1) / per;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    return launch_step(rope_kernel<T, N, kHalf>, dim3((unsigned)grid), threads,
                       (size_t)per * pairs * sizeof(float2), s, 0, a, lanes, (int)shares);
}

// The widest vectors that fit, 16 bytes at most.
template <class T, int N = 16 / (int)sizeof(T)>
cudaError_t rope_typed(const RopeArgs& a, cudaStream_t s)
{
    if constexpr (N > 1) {
        if (!rope_fits(a, sizeof(T), N))
            return rope_typed<T, N / 2>(a, s);
        return a.half ? rope_run<T, N, true>(a, s) : rope_run<T, N, false>(a, s);
    } else {
        return launch_step(rope_pairs_kernel<T>, dim3(a.T), kRopeThreads, 0, s, 0, a);
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t s)
{
    switch (dtype) {
    case PAGED_GQA_F16: return rope_typed<__half>(a, s);
    case PAGED_GQA_BF16: return rope_typed<__nv_bfloat16>(a, s);
    default: return rope_typed<float>(a, s);
    }
}

}  // namespace pgqa
