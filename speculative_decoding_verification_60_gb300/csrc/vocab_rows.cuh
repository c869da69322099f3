// What the calls over vocabulary rows outside verification share (log
// probabilities, distillation): their limits, their host checks, and the
// order of logits.
#pragma once

#include <math.h>

#include "../../include/specverify.h"
#include "cluster.cuh"
#include "common.cuh"
#include "launch.cuh"

namespace sv {

constexpr long long kRowsMaxVocab = 524280;  // as the verification calls
constexpr int kMaxTop = 128;                 // alternatives or teacher entries of a row
// Below it log2(e) / T leaves the range of 32 bits, and 0 times it is no number.
constexpr float kMinTemperature = 1.17549435e-38f;  // 2^-126
constexpr double kLog2e = 1.4426950408889634;
// Limits of the waits for bulk copies, for what the CTAs of a cluster send each
// other, and for copies in flight before a CTA may end.
constexpr uint64_t kCopyWaitNs = 2000000000ull, kClusterWaitNs = 2000000000ull, kDrainNs = 2000000000ull;
// Conditions on a thread under which its wait counts as run out; a test sets
// them for a library of its own.
#ifndef SV_LATE_COPY
#define SV_LATE_COPY false
#endif
#ifndef SV_LATE_CLUSTER
#define SV_LATE_CLUSTER false
#endif
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLn2Hi = 0.693145751953125f, kLn2Lo = 1.4286068203e-6f;  // ln 2: its first 16 bits, and the rest
// The reference of a running maximum before any finite entry: -inf minus it
// is -inf (weight zero), where -inf minus -inf would be NaN.
constexpr float kNoMax = -3.4028234663852886e38f;

// A whole warp's wait, with one answer: lanes that met the limit at different
// times would go different ways.
__device__ __forceinline__ bool warp_mbar_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit_ns) && !(SV_LATE_COPY));
}
__device__ __forceinline__ bool warp_cluster_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
    return __all_sync(0xffffffffu, cluster_mbar_wait(bar, parity, limit_ns) && !(SV_LATE_CLUSTER));
}

// Maximum over a warp: NaN is passed over, or (nan) makes it NaN.
__device__ __forceinline__ float warp_max_redux(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float warp_max_redux_nan(float v) {
    float r;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// The next value of T below x; NaN below -inf.
template <typename T> __device__ __forceinline__ float next_below(float x);
template <> __device__ __forceinline__ float next_below<float>(float x) {
    const uint32_t b = __float_as_uint(x == 0.0f ? -0.0f : x);
    return __uint_as_float((b & 0x80000000u) ? b + 1u : b - 1u);
}
template <> __device__ __forceinline__ float next_below<__nv_bfloat16>(float x) {
    const uint32_t b = __float_as_uint(x == 0.0f ? -0.0f : x);
    return __uint_as_float((b & 0x80000000u) ? b + 0x10000u : b - 0x10000u);
}

// A 16-byte vector of T as pairs of floats, its maximum (NaN if there is one),
// the number of its elements that are not <= a bound, and the vector that
// stands for no elements.
template <typename T> struct RowVec;
template <> struct RowVec<__nv_bfloat16> {
    static constexpr int kPairs = 4;
    __device__ static __forceinline__ __nv_bfloat162 word(const uint4& q, int i) {
        uint32_t w = i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
        return *reinterpret_cast<__nv_bfloat162*>(&w);
    }
    // pair i with values below `least` raised to it (NaN stays)
    __device__ static __forceinline__ float2 pair_above(const uint4& q, int i, __nv_bfloat162 least) {
        const __nv_bfloat162 h = __hmax2_nan(word(q, i), least);
        const uint32_t w = *reinterpret_cast<const uint32_t*>(&h);
        return make_float2(bf16_lo(w), bf16_hi(w));
    }
    using Least = __nv_bfloat162;
    __device__ static __forceinline__ Least least(float x) { return __float2bfloat162_rn(x); }
    // Elements above the bound, counted in bf16 halves: exact up to 256 each.
    using Count = __nv_bfloat162;
    __device__ static __forceinline__ Count count_zero() { return __float2bfloat162_rn(0.0f); }
    __device__ static __forceinline__ void count(Count& n, const uint4& q, Least bound) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) n = __hadd2(n, __hgtu2(word(q, i), bound));
    }
    __device__ static __forceinline__ int count_sum(Count n) { return (int)(__low2float(n) + __high2float(n)); }
    __device__ static __forceinline__ float2 pair(const uint4& q, int i) {
        const uint32_t w = i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
        return make_float2(bf16_lo(w), bf16_hi(w));
    }
    __device__ static __forceinline__ float max(const uint4& q) {
        auto h = [](uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); };
        const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h(q.x), h(q.y)), __hmax2_nan(h(q.z), h(q.w)));
        return max_nan(__low2float(m), __high2float(m));
    }
    __device__ static __forceinline__ float2 sum(const float2* w) {
        return __fadd2_rn(__fadd2_rn(w[0], w[1]), __fadd2_rn(w[2], w[3]));
    }
    // Elements equal to x become -inf; how many there were.
    __device__ static __forceinline__ int take_out(uint4& q, float x) {
        const __nv_bfloat162 xx = __float2bfloat162_rn(x);
        int n = 0;
        auto one = [&](uint32_t& w) {
            const uint32_t same = __heq2_mask(*reinterpret_cast<__nv_bfloat162*>(&w), xx);
            n += __popc(same) >> 4;
            w = (w & ~same) | (0xff80ff80u & same);
        };
        one(q.x);
        one(q.y);
        one(q.z);
        one(q.w);
        return n;
    }
    __device__ static __forceinline__ uint4 none() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
};
template <> struct RowVec<float> {
    static constexpr int kPairs = 2;
    using Least = float;
    __device__ static __forceinline__ Least least(float x) { return x; }
    __device__ static __forceinline__ float2 pair_above(const uint4& q, int i, float least) {
        const float2 x = pair(q, i);
        return make_float2(max_nan(x.x, least), max_nan(x.y, least));
    }
    using Count = int;
    __device__ static __forceinline__ Count count_zero() { return 0; }
    __device__ static __forceinline__ void count(Count& n, const uint4& q, float bound) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const float2 x = pair(q, i);
            n += !(x.x <= bound);
            n += !(x.y <= bound);
        }
    }
    __device__ static __forceinline__ int count_sum(Count n) { return n; }
    __device__ static __forceinline__ float2 pair(const uint4& q, int i) {
        return i == 0 ? make_float2(__uint_as_float(q.x), __uint_as_float(q.y))
                      : make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
    }
    __device__ static __forceinline__ float max(const uint4& q) {
        return max_nan(max_nan(__uint_as_float(q.x), __uint_as_float(q.y)),
                       max_nan(__uint_as_float(q.z), __uint_as_float(q.w)));
    }
    __device__ static __forceinline__ float2 sum(const float2* w) { return __fadd2_rn(w[0], w[1]); }
    __device__ static __forceinline__ int take_out(uint4& q, float x) {
        int n = 0;
        auto one = [&](uint32_t& w) {
            const bool same = __uint_as_float(w) == x;
            n += same;
            if (same) w = 0xff800000u;
        };
        one(q.x);
        one(q.y);
        one(q.z);
        one(q.w);
        return n;
    }
    __device__ static __forceinline__ uint4 none() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
};

// Maximum over a warp's tile of N vectors a lane (NaN if there is one).
template <typename T, int N>
__device__ __forceinline__ float tile_max(const uint4* q) {
    float m = RowVec<T>::max(q[0]);
#pragma unroll
    for (int j = 1; j < N; ++j) m = max_nan(m, RowVec<T>::max(q[j]));
    return warp_max_redux_nan(m);
}

// (logit descending, index ascending) as one integer: larger = earlier.
// Zero is below every entry's key.
__device__ __forceinline__ uint64_t order_key(float x, int idx) {
    return ((uint64_t)okey32(x) << 32) | (uint32_t)(0x7fffffff - idx);
}
__device__ __forceinline__ int key_index(uint64_t k) { return 0x7fffffff - (int)(uint32_t)k; }
__device__ __forceinline__ float key_value(uint64_t k) { return okey32_to_float((uint32_t)(k >> 32)); }

// ln z for z > 0 in two parts, x + y: the exponent's part is exact (ln 2 to
// 16 bits, and the rest of it), only the mantissa's logarithm is rounded to
// 32 bits.
__device__ __forceinline__ float2 ln_parts(float z) {
    int e;
    const float f = frexpf(z, &e);
    const float hi = (float)e * kLn2Hi, lo = fmaf((float)e, kLn2Lo, logf(f));
    const float x = hi + lo;
    const float b = x - hi;  // hi and lo of any size: a two-sum
    return make_float2(x, (hi - (x - b)) + (lo - b));
}
// a + v, in two parts as a is.
__device__ __forceinline__ float2 add_parts(float2 a, float v) {
    const float s = a.x + v, b = s - a.x;
    return make_float2(s, ((a.x - (s - b)) + (v - b)) + a.y);
}
__device__ __forceinline__ double ln_of(float z) {
    const float2 p = ln_parts(z);
    return (double)p.x + (double)p.y;
}

// The launches of a call are dependent launches: scheduled while the kernel
// before is ending, they wait for it (rows_begin) before they read anything.
// The error word is cleared by a kernel of its own in that chain; a memset
// there would make the next launch an ordinary one (5 rows of 128256 bf16 by
// token_logprobs: 8.7 us, with a memset 2.8 more).
__device__ __forceinline__ void rows_begin() {
    grid_dep_trigger();
    grid_dep_wait();
}
static __global__ void __launch_bounds__(32) k_clear_error(int32_t* dev_error) {
    rows_begin();
    if (threadIdx.x == 0) *dev_error = 0;
}
// A call's launch, its error word (may be NULL) cleared before it: n clusters
// of S CTAs.  A grid of one CTA to one wave of CTAs per SM is placed on an idle
// GPU (its first launch is an ordinary one): on one that is still ending a
// kernel, the SMs that are free first get more than their share of CTAs, and
// nothing follows to even it out (320 rows, 192 of them live: 27 us, started
// early 4 more; fewer or more CTAs are 0.5 us faster started early).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_rows(void (*kernel)(KArgs...), long long n, int S, int block, size_t dyn_smem, int sms,
                               int per_sm, int32_t* dev_error, cudaStream_t st, Args... args) {
    const bool early = n * S <= sms || n * S > (long long)per_sm * sms;
    if (dev_error) {
        const cudaError_t e = launch_clusters(k_clear_error, 1, 1, 32, 0, early, st, dev_error);
        if (e != cudaSuccess) return e;
    }
    return launch_clusters(kernel, n, S, block, dyn_smem, early || dev_error, st, args...);
}
// The error word of a call without rows.
inline spec_status clear_error(int32_t* dev_error, cudaStream_t st) {
    if (!dev_error) return SPEC_OK;
    return launch_clusters(k_clear_error, 1, 1, 32, 0, true, st, dev_error) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
__device__ __forceinline__ void set_error(int32_t* dev_error, int bits) {
    if (dev_error) atomicOr(dev_error, bits);
}

// Arguments that every call over rows checks the same way.
inline spec_status check_rows(spec_dtype dtype, int R, int V, int64_t row_stride, float temperature) {
    if (dtype != SPEC_BF16 && dtype != SPEC_F32) return SPEC_ERR_INVALID_ARG;
    if (R < 0 || V < 1 || row_stride < V) return SPEC_ERR_INVALID_ARG;
    if (!(temperature > 0.0f) || !(temperature < INFINITY)) return SPEC_ERR_INVALID_ARG;
    if ((int64_t)V > kRowsMaxVocab || temperature < kMinTemperature) return SPEC_ERR_UNSUPPORTED;
    return SPEC_OK;
}

}  // namespace sv
