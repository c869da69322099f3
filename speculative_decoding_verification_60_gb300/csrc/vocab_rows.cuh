// What the calls over vocabulary rows outside verification share (log
// probabilities, distillation): their limits, their host checks, and the
// order of logits.
#pragma once

#include <math.h>

#include "../../include/specverify.h"
#include "common.cuh"
#include "launch.cuh"

namespace sv {

constexpr long long kRowsMaxVocab = 524280;  // as the verification calls
constexpr int kMaxTop = 128;                 // alternatives or teacher entries of a row
constexpr double kLog2e = 1.4426950408889634;
constexpr float kLn2 = 0.69314718055994531f;
// The reference of a running maximum before any finite entry: -inf minus it
// is -inf (weight zero), where -inf minus -inf would be NaN.
constexpr float kNoMax = -3.4028234663852886e38f;

// (logit descending, index ascending) as one integer: larger = earlier.
// Zero is below every entry's key.
__device__ __forceinline__ uint64_t order_key(float x, int idx) {
    return ((uint64_t)okey32(x) << 32) | (uint32_t)(0x7fffffff - idx);
}
__device__ __forceinline__ int key_index(uint64_t k) { return 0x7fffffff - (int)(uint32_t)k; }
__device__ __forceinline__ float key_value(uint64_t k) { return okey32_to_float((uint32_t)(k >> 32)); }

// ln z for z > 0, as a double of about 25 good bits near zero and better
// above: the exponent's part is exact, only the mantissa's logarithm is
// rounded to 32 bits.
__device__ __forceinline__ double ln_of(float z) {
    int e;
    const float f = frexpf(z, &e);
    return (double)e * 0.69314718055994531 + (double)logf(f);
}

// Arguments that every call over rows checks the same way.
inline spec_status check_rows(spec_dtype dtype, int R, int V, int64_t row_stride, float temperature) {
    if (dtype != SPEC_BF16 && dtype != SPEC_F32) return SPEC_ERR_INVALID_ARG;
    if (R < 0 || V < 1 || row_stride < V) return SPEC_ERR_INVALID_ARG;
    if (!(temperature > 0.0f) || !(temperature < INFINITY)) return SPEC_ERR_INVALID_ARG;
    if ((int64_t)V > kRowsMaxVocab) return SPEC_ERR_UNSUPPORTED;
    return SPEC_OK;
}

}  // namespace sv
