// Distillation of a draft model from a teacher's top-K log probabilities:
// the loss of every row with its gradient (spec_distill_topk), and the
// gradient for upstream gradients known later (spec_distill_topk_backward).
//
// With S the listed tokens, the student's softmax is split in two: over the
// tokens outside S (the tail: maximum m_T, Z_T = sum 2^((s - m_T) c)) and
// the K listed ones.  The tail's mass q_T is then a sum of its own terms,
// where 1 - sum q_j would cancel, and the gradient of every tail token is
// one coefficient times 2^((s - m_T) c).
#include "vocab_rows.cuh"

namespace sv {

struct DistillArgs {
    const void* student;
    int R, V, K;
    int64_t stride;
    const int32_t* ids;
    const float* teacher;
    const float* weights;  // forward: row weights; backward: upstream gradients
    float c;
    double inv_t;
    bool bucket;
    float* loss;
    float* stats;
    void* grad;
    int64_t grad_stride;
    int32_t* dev_error;
};

// A row's statistics, as kept for the backward call (8 floats).
struct DistillStat {
    float m_tail;  // reference of the tail's exponentials
    float coef;    // gradient of a tail token / (weight 2^((s - m_tail) c))
    float m;       // maximum of the row
    float inv_z;   // 1 / sum of 2^((s - m) c) over the row
    float mass;    // S = sum t_j + t_T
    float ln_t;    // subtracted from the teacher's values: t_j = exp(l_j - ln_t)
    float live;    // 0: the row has loss 0 and gradient 0
    float pad;
};
static_assert(sizeof(DistillStat) == 32, "row_stats is [R, 8] float");

constexpr int kDsThreads = 256;
// Where the student gives the tail nothing, this much teacher mass outside
// the listed tokens is the rounding of their log probabilities: the loss
// would be +inf for it.
constexpr float kTailRounding = 1.0f / 65536.0f;

struct DsSmem {
    float m[kDsThreads], z[kDsThreads];
    float s[kMaxTop], l[kMaxTop];  // student logits and teacher values of the listed tokens
    int id[kMaxTop];
    DistillStat st;
    float loss;
    int bad;
};

__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One warp: the row's statistics and loss from the tail's maximum and sum
// and the K listed tokens.  The differences log t - log q cancel where the
// student is near the teacher, and 1 - sum t where the listed tokens hold
// nearly all of the teacher, so both are taken in double (K per row).
__device__ __forceinline__ void distill_finish(const DistillArgs& a, float m_tail, float z_tail, const float* s,
                                               const float* l, const int* id, DistillStat* out, float* loss, int* bad) {
    const int lane = threadIdx.x & 31;
    float lmax = kNoMax, smax = kNoMax;
    int err = 0;
    for (int j = lane; j < a.K; j += 32)
        if (id[j] >= 0) {
            lmax = fmaxf(lmax, l[j]);
            smax = fmaxf(smax, s[j]);
            if (isnan(l[j]) || l[j] == INFINITY || isnan(s[j]) || s[j] == INFINITY) err = kDevErrNonfinite;
        }
    lmax = warp_max(lmax);
    const float m = fmaxf(m_tail, warp_max(smax));
    float z = 0.0f;
    double tsum = 0.0;
    const float lref = a.bucket ? 0.0f : lmax;
    for (int j = lane; j < a.K; j += 32)
        if (id[j] >= 0) {
            z += ex2((s[j] - m) * a.c);
            tsum += exp((double)l[j] - (double)lref);
        }
    tsum = warp_sum_d(tsum);
    const float zt = z_tail * ex2(fmaxf((m_tail - m) * a.c, -1000.0f));
    z = warp_sum_f(z) + zt;
    if (!(z > 0.0f && z < INFINITY) || !(tsum < (double)INFINITY)) err = kDevErrNonfinite;
    err = __reduce_or_sync(0xffffffffu, err);
    DistillStat st{};
    double sum = 0.0;
    if (!err && (a.bucket || tsum > 0.0)) {
        const double ln_z = ln_of(z);
        const double ln_t = a.bucket ? 0.0 : (double)lref + ln_of((float)tsum);
        float t_tail = a.bucket ? (float)fmax(1.0 - tsum, 0.0) : 0.0f;
        if (z_tail == 0.0f && t_tail <= kTailRounding) t_tail = 0.0f;
        const float q_tail = zt / z;
        for (int j = lane; j < a.K; j += 32)
            if (id[j] >= 0 && l[j] > -INFINITY) {
                const double lt = (double)l[j] - ln_t;
                const float t = expf((float)lt);
                const double lq = (double)(s[j] - m) * a.inv_t - ln_z;
                if (t > 0.0f) sum += (double)t * (lt - lq);
            }
        sum = warp_sum_d(sum);
        if (t_tail > 0.0f)
            sum = z_tail > 0.0f
                      ? sum + (double)t_tail * (ln_of(t_tail) - ((double)(m_tail - m) * a.inv_t + ln_of(z_tail) - ln_z))
                      : (double)INFINITY;
        st.m_tail = m_tail;
        st.m = m;
        st.inv_z = 1.0f / z;
        st.mass = a.bucket ? (float)(tsum + (double)t_tail) : 1.0f;
        st.ln_t = (float)ln_t;
        st.coef = z_tail > 0.0f ? (st.mass * q_tail - t_tail) * (float)a.inv_t / z_tail : 0.0f;
        st.live = 1.0f;
    }
    if (lane == 0) {
        *out = st;
        *loss = (float)sum;
        *bad = err;
    }
}

// Gradient of listed token j.
__device__ __forceinline__ float distill_listed_grad(const DistillStat& st, float s, float l, float c, float inv_t,
                                                     float w) {
    const float q = ex2((s - st.m) * c) * st.inv_z;
    return w * (st.mass * q - expf(l - st.ln_t)) * inv_t;
}

__device__ __forceinline__ void store_elem(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_elem(float* p, float v) { *p = v; }

template <typename T>
__device__ __forceinline__ void distill_zero_grad(const DistillArgs& a, int r) {
    if (!a.grad) return;
    T* g = static_cast<T*>(a.grad) + (size_t)r * a.grad_stride;
    for (int i = threadIdx.x; i < a.V; i += kDsThreads) store_elem(g + i, 0.0f);
}

// The gradient of a row from its statistics; the listed tokens' values are
// in sm (loaded before any write: grad may be the student's buffer).
template <typename T>
__device__ __forceinline__ void distill_write_grad(const DistillArgs& a, int r, const DistillStat& st, float w,
                                                   const DsSmem& sm) {
    const T* row = static_cast<const T*>(a.student) + (size_t)r * a.stride;
    T* g = static_cast<T*>(a.grad) + (size_t)r * a.grad_stride;
    for (int i = threadIdx.x; i < a.V; i += kDsThreads)
        store_elem(g + i, w * st.coef * ex2((ElemT<T>::load(row + i) - st.m_tail) * a.c));
    __syncthreads();  // the listed tokens overwrite what the sweep wrote there
    for (int j = threadIdx.x; j < a.K; j += kDsThreads)
        if (sm.id[j] >= 0) store_elem(g + sm.id[j], distill_listed_grad(st, sm.s[j], sm.l[j], a.c, (float)a.inv_t, w));
}

template <typename T>
__global__ void __launch_bounds__(kDsThreads) k_distill(DistillArgs a) {
    extern __shared__ uint32_t listed[];  // one bit per token
    __shared__ DsSmem sm;
    const int r = blockIdx.x, tid = threadIdx.x;
    const float w = a.weights ? a.weights[r] : 1.0f;
    if (w == 0.0f) {
        if (tid == 0) {
            a.loss[r] = 0.0f;
            if (a.stats) reinterpret_cast<DistillStat*>(a.stats)[r] = DistillStat{};
        }
        distill_zero_grad<T>(a, r);
        return;
    }
    const T* row = static_cast<const T*>(a.student) + (size_t)r * a.stride;
    for (int i = tid; i < (a.V + 31) / 32; i += kDsThreads) listed[i] = 0u;
    if (tid == 0) sm.bad = 0;
    __syncthreads();
    for (int j = tid; j < a.K; j += kDsThreads) {
        const int v = a.ids[(size_t)r * a.K + j];
        sm.l[j] = a.teacher[(size_t)r * a.K + j];
        sm.id[j] = v;
        if (v == -1) continue;
        if (v < 0 || v >= a.V || ((atomicOr(&listed[v >> 5], 1u << (v & 31)) >> (v & 31)) & 1u)) {
            sm.bad = kDevErrToken;
            sm.id[j] = -1;
        } else {
            sm.s[j] = ElemT<T>::load(row + v);
        }
    }
    __syncthreads();
    const int bad_id = sm.bad;
    float m = kNoMax, z = 0.0f;
    for (int i = tid; i < a.V; i += kDsThreads) {
        if ((listed[i >> 5] >> (i & 31)) & 1u) continue;
        const float x = ElemT<T>::load(row + i);
        if (x > m) {
            z *= ex2(fmaxf((m - x) * a.c, -1000.0f));
            m = x;
        }
        z += ex2((x - m) * a.c);
    }
    sm.m[tid] = m;
    sm.z[tid] = z;
    for (int o = kDsThreads / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (tid < o) {
            const float m2 = fmaxf(sm.m[tid], sm.m[tid + o]);
            sm.z[tid] = sm.z[tid] * ex2(fmaxf((sm.m[tid] - m2) * a.c, -1000.0f)) +
                        sm.z[tid + o] * ex2(fmaxf((sm.m[tid + o] - m2) * a.c, -1000.0f));
            sm.m[tid] = m2;
        }
    }
    __syncthreads();
    if (tid < 32) distill_finish(a, sm.m[0], sm.z[0], sm.s, sm.l, sm.id, &sm.st, &sm.loss, &sm.bad);
    __syncthreads();
    const int bad = sm.bad | bad_id;
    const DistillStat st = bad ? DistillStat{} : sm.st;
    if (tid == 0) {
        a.loss[r] = bad ? 0.0f : sm.loss;
        if (a.stats) reinterpret_cast<DistillStat*>(a.stats)[r] = st;
        if (bad && a.dev_error) atomicOr(a.dev_error, bad);
    }
    if (!a.grad) return;
    if (st.live == 0.0f)
        distill_zero_grad<T>(a, r);
    else
        distill_write_grad<T>(a, r, st, w, sm);
}

template <typename T>
__global__ void __launch_bounds__(kDsThreads) k_distill_backward(DistillArgs a) {
    __shared__ DsSmem sm;
    const int r = blockIdx.x, tid = threadIdx.x;
    const float w = a.weights ? a.weights[r] : 1.0f;
    const DistillStat st = reinterpret_cast<const DistillStat*>(a.stats)[r];
    if (w == 0.0f || st.live == 0.0f) {
        distill_zero_grad<T>(a, r);
        return;
    }
    const T* row = static_cast<const T*>(a.student) + (size_t)r * a.stride;
    for (int j = tid; j < a.K; j += kDsThreads) {
        const int v = a.ids[(size_t)r * a.K + j];
        sm.id[j] = v < a.V ? v : -1;
        sm.l[j] = a.teacher[(size_t)r * a.K + j];
        if (v >= 0 && v < a.V) sm.s[j] = ElemT<T>::load(row + v);
    }
    __syncthreads();
    distill_write_grad<T>(a, r, st, w, sm);
}

static spec_status check_distill(const void* student, spec_dtype dtype, int R, int V, int64_t row_stride,
                                 const int32_t* ids, const float* teacher, int K, float temperature, const void* grad,
                                 int64_t grad_stride) {
    const spec_status bad = check_rows(dtype, R, V, row_stride, temperature);
    if (bad != SPEC_OK) return bad;
    if (K < 1 || (grad && grad_stride < V)) return SPEC_ERR_INVALID_ARG;
    if (K > kMaxTop) return SPEC_ERR_UNSUPPORTED;
    if (R > 0 && (!student || !ids || !teacher)) return SPEC_ERR_INVALID_ARG;
    // in place means the same rows: a partly overlapping grad is not defined
    if (grad && grad == student && grad_stride != row_stride) return SPEC_ERR_INVALID_ARG;
    return SPEC_OK;
}

}  // namespace sv

using namespace sv;

extern "C" spec_status spec_distill_topk(const void* student, spec_dtype dtype, int R, int V, int64_t row_stride,
                                         const int32_t* teacher_ids, const float* teacher_logprobs, int K,
                                         const float* weights, float temperature, spec_tail_mode tail, float* loss,
                                         float* row_stats, void* grad, int64_t grad_stride, int32_t* dev_error,
                                         spec_stream_t stream) {
    DeviceGuard device_guard;  // the caller's current device is put back on return
    const spec_status bad = check_distill(student, dtype, R, V, row_stride, teacher_ids, teacher_logprobs, K,
                                          temperature, grad, grad_stride);
    if (bad != SPEC_OK) return bad;
    if ((tail != SPEC_TAIL_RENORM && tail != SPEC_TAIL_BUCKET) || (R > 0 && !loss)) return SPEC_ERR_INVALID_ARG;
    const void* on_device = R > 0 ? student : dev_error;
    if (!on_device) return SPEC_OK;  // no rows and no error word: nothing to do
    if (!select_device_of(on_device)) return SPEC_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dev_error && cudaMemsetAsync(dev_error, 0, sizeof(int32_t), st) != cudaSuccess) return SPEC_ERR_CUDA;
    if (R == 0) return SPEC_OK;
    DistillArgs a{student, R, V, K, row_stride, teacher_ids, teacher_logprobs, weights,
                  (float)(kLog2e / (double)temperature), 1.0 / (double)temperature, tail == SPEC_TAIL_BUCKET,
                  loss, row_stats, grad, grad_stride, dev_error};
    const size_t dyn = (size_t)((V + 31) / 32) * 4;
    auto* kern = dtype == SPEC_BF16 ? k_distill<__nv_bfloat16> : k_distill<float>;
    if (!set_dyn_smem(kern, (size_t)((kRowsMaxVocab + 31) / 32) * 4, kDsThreads)) return SPEC_ERR_CUDA;
    kern<<<R, kDsThreads, dyn, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

extern "C" spec_status spec_distill_topk_backward(const void* student, spec_dtype dtype, int R, int V,
                                                  int64_t row_stride, const int32_t* teacher_ids,
                                                  const float* teacher_logprobs, int K, const float* row_stats,
                                                  const float* grad_loss, float temperature, void* grad,
                                                  int64_t grad_stride, spec_stream_t stream) {
    DeviceGuard device_guard;  // the caller's current device is put back on return
    const spec_status bad = check_distill(student, dtype, R, V, row_stride, teacher_ids, teacher_logprobs, K,
                                          temperature, grad, grad_stride);
    if (bad != SPEC_OK) return bad;
    if (R == 0) return SPEC_OK;
    if (!row_stats || !grad) return SPEC_ERR_INVALID_ARG;
    if (!select_device_of(student)) return SPEC_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    DistillArgs a{student, R, V, K, row_stride, teacher_ids, teacher_logprobs, grad_loss,
                  (float)(kLog2e / (double)temperature), 1.0 / (double)temperature, false, nullptr,
                  const_cast<float*>(row_stats), grad, grad_stride, nullptr};
    if (dtype == SPEC_BF16)
        k_distill_backward<__nv_bfloat16><<<R, kDsThreads, 0, st>>>(a);
    else
        k_distill_backward<float><<<R, kDsThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
