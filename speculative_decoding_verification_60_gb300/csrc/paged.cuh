// What the calls over a paged cache share (append.cu, attend.cu, keep.cu,
// adjust.cu): the layout's checks, the types' conversions, a draft's tree.
#pragma once

#include <cuda_fp16.h>

#include "vocab_rows.cuh"

namespace sv {

constexpr int kDevErrCapacity = 32;  // SPEC_DEVERR_CAPACITY
constexpr int kMaxDraftNodes = 1024;
constexpr int kMaxRequests = 65535;

inline bool layout_ok(const spec_cache_layout* l) {
    return l && l->blocks >= 1 && l->page_size >= 1 && l->heads >= 1 && l->dim >= 1 && l->block_stride >= 0 &&
           l->entry_stride >= 0 && l->head_stride >= 0;
}

// Two 16-bit values of T from a 32-bit word, and back.
template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    __device__ static __forceinline__ float2 get(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }
    __device__ static __forceinline__ uint32_t put(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <> struct Pair<__half> {
    __device__ static __forceinline__ float2 get(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
    __device__ static __forceinline__ uint32_t put(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

// Whether parent[0 .. n) is a tree rooted at 0 with parent[i] < i; the threads
// of a CTA ask together (t of nt), each sees its part.
__device__ __forceinline__ bool tree_part_ok(const int32_t* parent, int n, int t, int nt) {
    bool ok = true;
    for (int i = t; i < n; i += nt) {
        const int p = parent[i];
        ok = ok && (i == 0 ? p == -1 : p >= 0 && p < i);
    }
    return ok;
}

}  // namespace sv
