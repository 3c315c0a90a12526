// logits.cu -- penalties for repeated tokens, biases and grammar masks on a
// step's logits.
//
// Bound: HBM, each logit read once and written once as float32, the mask bits
// beside them.  A CTA takes a.cols columns of a row.  It counts the row's
// history into shared memory, one word per column: bits 0..28 how often the
// token was generated, bit 31 that it is in the prompt, bits 29 and 30 that it
// has a bias and more than one.  Integer atomics only, so the order of the
// counts does not matter.  The first logits, the first history entries and the
// biases are all loaded before anything waits for one of them.  A column with
// a bias is finished by the thread of its bias entry, and one with several by the
// thread of the column, which sums the token's entries in their order; the stream
// leaves them out.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "step_internal.h"

namespace pgqa {

namespace {

constexpr int kAhead = 8;                    // history entries per thread loaded at the start
constexpr uint32_t kCount = (1u << 29) - 1, kBias = 1u << 29, kBiases = 1u << 30, kSeen = 1u << 31;

// Four neighbouring logits as floats; p is aligned to them.
template <class T>
__device__ __forceinline__ float4 load4(const T* p)
{
    if constexpr (std::is_same_v<T, float>) {
        return *reinterpret_cast<const float4*>(p);
    } else {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        float2 a, b;
        if constexpr (std::is_same_v<T, __half>) {
            a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
            b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
        } else {
            a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.x));
            b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.y));
        }
        return make_float4(a.x, a.y, b.x, b.y);
    }
}

// A row's parameters.
struct Penalty {
    float repetition, frequency, presence;
};

__device__ __forceinline__ float penalised(float x, uint32_t c, const Penalty& p)
{
    if (c & (kSeen | kCount))
        x = x > 0.f ? __fdiv_rn(x, p.repetition) : x * p.repetition;
    const uint32_t n = c & kCount;
    if (n != 0u)
        x = fmaf(-p.frequency, (float)n, x) - p.presence;
    return x;
}

}  // namespace

// grid (ceil(V / cols), B); a thread takes N vectors of four columns at a time.
template <class T, int N, int kLogitThreads>
__global__ void __launch_bounds__(kLogitThreads) logits_kernel(LogitsArgs a)
{
    constexpr int kWindow = 4 * kLogitThreads * N;
    extern __shared__ __align__(16) uint32_t cnt[];
    const int tid = threadIdx.x, b = blockIdx.y, lo = blockIdx.x * a.cols;
    const int n = min(a.cols, a.V - lo);
    const paged_gqa_logit_rules& r = a.r;
    const T* x = static_cast<const T*>(a.x) + b * a.x_stride + lo;
    float* out = a.out + b * a.out_stride + lo;
    const bool vec = reinterpret_cast<uintptr_t>(x) % (4 * sizeof(T)) == 0 &&
                     reinterpret_cast<uintptr_t>(out) % 16 == 0;
    int flags = 0;
    enter();

    // ---- loads: vector u of a thread is columns c0 + 4 (tid + u kLogitThreads)
    float4 v[N];
    auto load = [&](int c0) {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int c = c0 + 4 * (tid + u * kLogitThreads);
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (vec && c + 4 <= n) {
                v[u] = load4(x + c);
            } else {
                float* e = &v[u].x;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < n)
                        e[i] = (float)x[c + i];
            }
        }
    };
    load(0);
    const int32_t* hist = r.history != nullptr ? r.history + b * r.history_stride : nullptr;
    int32_t h[kAhead];
    Penalty p{1.f, 0.f, 0.f};
    int len = 0, prompt = 0;
    if (hist != nullptr) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            h[i] = tid + i * kLogitThreads < r.max_history ? hist[tid + i * kLogitThreads] : -1;
        len = r.history_lens != nullptr ? min(max(r.history_lens[b], 0), r.max_history)
                                        : r.max_history;
        prompt = r.prompt_lens != nullptr ? r.prompt_lens[b] : 0;
        p.repetition = r.repetition != nullptr ? r.repetition[b] : 1.f;
        p.frequency = r.frequency != nullptr ? r.frequency[b] : 0.f;
        p.presence = r.presence != nullptr ? r.presence[b] : 0.f;
    }
    const int32_t* bt = r.bias_tokens != nullptr ? r.bias_tokens + b * r.bias_stride : nullptr;
    const float* bv = bt != nullptr ? r.bias_values + b * r.bias_stride : nullptr;
    const int n_bias = bt != nullptr ? r.n_bias : 0;
    int bias_t = tid < n_bias ? bt[tid] : -1;        // the thread's first bias entry
    float bias_x = 0.f, bias_v = 0.f;
    if (bias_t >= lo && bias_t < lo + n) {
        bias_v = bv[tid];
        bias_x = (float)x[bias_t - lo];
    }
    const uint32_t* mask = nullptr;
    if (r.mask != nullptr) {
        const int m = r.mask_index != nullptr ? r.mask_index[b] : b;
        if (m >= r.mask_rows)
            flags |= PAGED_GQA_FLAG_BAD_INDEX;
        else if (m >= 0)
            mask = r.mask + m * r.mask_stride;
    }

    // ---- counts of the history and marks of the biases
    const bool table = hist != nullptr || bt != nullptr;
    if (table) {
        for (int i = 4 * tid; i < n; i += 4 * kLogitThreads)
            *reinterpret_cast<uint4*>(cnt + i) = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
    }
    auto count = [&](int i, int t) {
        if (t >= a.V)
            flags |= PAGED_GQA_FLAG_BAD_INDEX;
        else if (t >= lo && t < lo + n) {
            if (i >= prompt)
                atomicAdd(&cnt[t - lo], 1u);
            else
                atomicOr(&cnt[t - lo], kSeen);
        }
    };
    if (hist != nullptr) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (tid + i * kLogitThreads < len)
                count(tid + i * kLogitThreads, h[i]);
        for (int i0 = tid + kAhead * kLogitThreads; i0 < len; i0 += kAhead * kLogitThreads) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                h[i] = i0 + i * kLogitThreads < len ? hist[i0 + i * kLogitThreads] : -1;
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                count(i0 + i * kLogitThreads, h[i]);
        }
    }
    int several = 0;                                     // a token with more than one bias
    for (int i = tid; i < n_bias; i += kLogitThreads) {
        const int t = i == tid ? bias_t : bt[i];
        if (t >= a.V)
            flags |= PAGED_GQA_FLAG_BAD_INDEX;
        else if (t >= lo && t < lo + n && (atomicOr(&cnt[t - lo], kBias) & kBias)) {
            atomicOr(&cnt[t - lo], kBiases);
            several = 1;
        }
    }
    if (table)
        several = __syncthreads_or(several);

    // ---- columns with a bias
    auto finish = [&](int c, float e, uint32_t w, float sum) {
        const int t = lo + c;
        const bool ok = mask == nullptr || ((mask[t >> 5] >> (t & 31)) & 1u);
        out[c] = ok ? penalised(e, w, p) + sum : -INFINITY;
    };
    for (int i = tid; i < n_bias; i += kLogitThreads) {
        const int t = i == tid ? bias_t : bt[i];
        if (t < lo || t >= lo + n)
            continue;
        const uint32_t w = cnt[t - lo];
        if (!(w & kBiases))
            finish(t - lo, i == tid ? bias_x : (float)x[t - lo], w, i == tid ? bias_v : bv[i]);
    }
    // those with several: one sweep over the entries for each (a thread to every entry,
    // looking for the token's first one, takes the square of n_bias)
    for (int c = several ? tid : n; c < n; c += kLogitThreads) {
        if (!(cnt[c] & kBiases))
            continue;
        float sum = -0.f;                                // adds nothing
        for (int i = 0; i < n_bias; ++i)
            if (bt[i] == lo + c)
                sum += bv[i];
        finish(c, (float)x[c], cnt[c], sum);
    }

    // ---- the others: penalties and mask
    for (int c0 = 0; c0 < n; c0 += kWindow) {
        if (c0 > 0)
            load(c0);
        uint32_t bits[N];                                // ahead of the stores
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int c = c0 + 4 * (tid + u * kLogitThreads);
            bits[u] = mask != nullptr && c < n ? mask[(lo + c) >> 5] >> (c & 31) : 0u;
        }
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int c = c0 + 4 * (tid + u * kLogitThreads);
            if (c >= n)
                break;
            float* e = &v[u].x;
            uint32_t skip = 0u;
            if (table) {
                const uint4 w = *reinterpret_cast<const uint4*>(cnt + c);
                const uint32_t any = w.x | w.y | w.z | w.w;
                if (any != 0u) {
                    e[0] = penalised(e[0], w.x, p);
                    e[1] = penalised(e[1], w.y, p);
                    e[2] = penalised(e[2], w.z, p);
                    e[3] = penalised(e[3], w.w, p);
                    if (any & kBias)
                        skip = (w.x & kBias ? 1u : 0u) | (w.y & kBias ? 2u : 0u) |
                               (w.z & kBias ? 4u : 0u) | (w.w & kBias ? 8u : 0u);
                }
            }
            if (mask != nullptr) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!((bits[u] >> i) & 1u))
                        e[i] = -INFINITY;
            }
            if (vec && c + 4 <= n && skip == 0u) {
                *reinterpret_cast<float4*>(out + c) = v[u];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < n && !((skip >> i) & 1u))
                        out[c + i] = e[i];
            }
        }
    }
    raise_flag(a.err, flags);
}

namespace {

constexpr int64_t kLogitCols = 48 * 1024;    // most columns of a CTA: 192 KB of counts

template <class T, int N, int kThreads_>
cudaError_t logits_run(const LogitsArgs& a, cudaStream_t s)
{
    static std::atomic<int> done[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= kMaxDevices || !done[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(logits_kernel<T, N, kThreads_>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(kLogitCols * sizeof(uint32_t)));
        if (e != cudaSuccess)
            return e;
        if (dev < kMaxDevices)
            done[dev].store(1, std::memory_order_release);
    }
    const bool table = a.r.history != nullptr || a.r.bias_tokens != nullptr;
    const dim3 grid((unsigned)(((int64_t)a.V + a.cols - 1) / a.cols), a.B);
    return launch_step(logits_kernel<T, N, kThreads_>, grid, kThreads_,
                       table ? a.cols * sizeof(uint32_t) : 0, s, 0, a);
}

template <class T>
cudaError_t logits_typed(LogitsArgs a, cudaStream_t s)
{
    // Each row is cut into equal shares of columns, a CTA each, as many as fill the
    // SMs once, or w times in turn where shares would pass `most` (16 x 248,320,
    // 4096 tokens of history: 304 CTAs of 13,088 columns 9.8 us, 496 of 8192, which
    // is 1.6 waves, 11.4 us; 400 rows of 248,320 140 us and 173 us).
    auto share = [&](int64_t slots, int64_t most) {
        const int64_t w = ((a.V + most - 1) / most * a.B + slots - 1) / slots, k = slots * w / a.B;
        return (int)std::max<int64_t>(((a.V + k - 1) / k + 31) / 32 * 32, 2048);
    };
    a.cols = share(2 * kSms, kLogitCols / 2);
    // Every CTA reads its row's whole history: where that is half as long as the
    // share or more, one CTA of 1024 threads per SM in place of two of 512 (32,768
    // tokens 14.8 us and 18.2 us), unless they would have too few columns and a
    // history that half the threads load at once (one row, 4096 tokens: 3.8 and 3.3).
    const int64_t history = a.r.history != nullptr ? a.r.max_history : 0;
    const int wide = share(kSms, kLogitCols);
    if (2 * history > a.cols && (wide >= 4096 || history > 8192)) {
        a.cols = wide;
        return logits_run<T, 4, 1024>(a, s);
    }
    if (a.cols <= 4096)
        return a.cols <= 2048 ? logits_run<T, 1, 512>(a, s) : logits_run<T, 2, 512>(a, s);
    // seven or four vectors to a thread, whichever leaves fewer idle in the last pass
    auto padded = [&](int n) { return (a.cols + 2048 * n - 1) / (2048 * n) * n; };
    return padded(7) <= padded(4) ? logits_run<T, 7, 512>(a, s) : logits_run<T, 4, 512>(a, s);
}

}  // namespace

cudaError_t launch_logits(const LogitsArgs& a, int dtype, cudaStream_t s)
{
    switch (dtype) {
    case PAGED_GQA_F16: return logits_typed<__half>(a, s);
    case PAGED_GQA_BF16: return logits_typed<__nv_bfloat16>(a, s);
    default: return logits_typed<float>(a, s);
    }
}

}  // namespace pgqa
