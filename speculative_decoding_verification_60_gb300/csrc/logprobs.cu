// Log probabilities of given tokens with the entropy and the top
// alternatives of their rows (spec_token_logprobs): what is reported beside
// the tokens a verification emits, and what a target hands to the training
// of its draft.
#include "vocab_rows.cuh"

namespace sv {

struct LogprobArgs {
    const void* logits;
    int R, V, top_k;
    int64_t stride;
    const int32_t* tokens;
    float c, inv_t;
    float* logprob;
    int32_t* rank;
    float* entropy;
    int32_t* top_ids;
    float* top_logprobs;
    int32_t* dev_error;
};

constexpr int kLpThreads = 256;

struct LpSmem {
    float m[kLpThreads], z[kLpThreads], e[kLpThreads];
    int n[kLpThreads];
    uint64_t key[kLpThreads];
};

// A row that gets no result: skipped, or refused (logprob -inf).
__device__ __forceinline__ void lp_no_result(const LogprobArgs& a, int r, float logprob) {
    if (threadIdx.x == 0) {
        if (a.logprob) a.logprob[r] = logprob;
        if (a.rank) a.rank[r] = -1;
        if (a.entropy) a.entropy[r] = 0.0f;
    }
    for (int j = threadIdx.x; j < a.top_k; j += blockDim.x) {
        a.top_ids[(size_t)r * a.top_k + j] = -1;
        a.top_logprobs[(size_t)r * a.top_k + j] = -INFINITY;
    }
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads) k_token_logprobs(LogprobArgs a) {
    __shared__ LpSmem s;
    const int r = blockIdx.x, tid = threadIdx.x;
    const int tok = a.tokens ? a.tokens[r] : 0;
    if (tok < 0 || tok >= a.V) {
        if (tok != -1 && tid == 0 && a.dev_error) atomicOr(a.dev_error, kDevErrToken);
        lp_no_result(a, r, tok == -1 ? 0.0f : -INFINITY);
        return;
    }
    const T* row = static_cast<const T*>(a.logits) + (size_t)r * a.stride;
    const float xt = ElemT<T>::load(row + tok);
    // z = sum 2^t and e = sum t 2^t of t = (x - m) c, m the maximum so far
    float m = kNoMax, z = 0.0f, e = 0.0f;
    int before = 0;
    for (int i = tid; i < a.V; i += kLpThreads) {
        const float x = ElemT<T>::load(row + i);
        if (x > m) {
            const float d = fmaxf((m - x) * a.c, -1000.0f), f = ex2(d);
            e = (e + z * d) * f;
            z *= f;
            m = x;
        }
        const float t = (x - m) * a.c, w = ex2(t);
        z += w;
        e = fmaf(w, fmaxf(t, -1000.0f), e);
        before += x > xt || (x == xt && i < tok);
    }
    s.m[tid] = m; s.z[tid] = z; s.e[tid] = e; s.n[tid] = before;
    for (int o = kLpThreads / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (tid < o) {
            const float m2 = fmaxf(s.m[tid], s.m[tid + o]);
            float z2 = 0.0f, e2 = 0.0f;
            for (int k = tid; k <= tid + o; k += o) {
                const float d = fmaxf((s.m[k] - m2) * a.c, -1000.0f), f = ex2(d);
                e2 += (s.e[k] + s.z[k] * d) * f;
                z2 += s.z[k] * f;
            }
            s.m[tid] = m2; s.z[tid] = z2; s.e[tid] = e2;
            s.n[tid] += s.n[tid + o];
        }
    }
    __syncthreads();
    m = s.m[0]; z = s.z[0]; e = s.e[0]; before = s.n[0];
    if (!(z > 0.0f && z < INFINITY)) {  // NaN or +inf somewhere, or nothing finite
        if (tid == 0 && a.dev_error) atomicOr(a.dev_error, kDevErrNonfinite);
        lp_no_result(a, r, a.tokens ? -INFINITY : 0.0f);
        return;
    }
    const double ln_z = ln_of(z);
    if (tid == 0) {
        if (a.logprob) a.logprob[r] = a.tokens ? (float)((double)((xt - m) * a.inv_t) - ln_z) : 0.0f;
        if (a.rank) a.rank[r] = a.tokens ? before + 1 : -1;
        if (a.entropy) a.entropy[r] = (float)(ln_z - (double)(e / z * kLn2));
    }
    // the alternatives one after another: the largest key below the last one
    uint64_t last = ~0ull;
    for (int j = 0; j < a.top_k; ++j) {
        uint64_t best = 0;
        for (int i = tid; i < a.V; i += kLpThreads) {
            const uint64_t k = order_key(ElemT<T>::load(row + i), i);
            if (k < last && k > best) best = k;
        }
        s.key[tid] = best;
        for (int o = kLpThreads / 2; o > 0; o >>= 1) {
            __syncthreads();
            if (tid < o && s.key[tid + o] > s.key[tid]) s.key[tid] = s.key[tid + o];
        }
        __syncthreads();
        last = s.key[0];
        __syncthreads();
        if (tid == 0) {
            a.top_ids[(size_t)r * a.top_k + j] = key_index(last);
            a.top_logprobs[(size_t)r * a.top_k + j] = (float)((double)((key_value(last) - m) * a.inv_t) - ln_z);
        }
    }
}

}  // namespace sv

using namespace sv;

extern "C" spec_status spec_token_logprobs(const void* logits, spec_dtype dtype, int R, int V, int64_t row_stride,
                                           const int32_t* tokens, float temperature, int top_k, float* logprob,
                                           int32_t* rank, float* entropy, int32_t* top_ids, float* top_logprobs,
                                           int32_t* dev_error, spec_stream_t stream) {
    DeviceGuard device_guard;  // the caller's current device is put back on return
    const spec_status bad = check_rows(dtype, R, V, row_stride, temperature);
    if (bad != SPEC_OK) return bad;
    if (top_k < 0 || top_k > V) return SPEC_ERR_INVALID_ARG;
    if (top_k > kMaxTop) return SPEC_ERR_UNSUPPORTED;
    if (R > 0 && (!logits || (tokens && !logprob) || (top_k > 0 && (!top_ids || !top_logprobs))))
        return SPEC_ERR_INVALID_ARG;
    const void* on_device = R > 0 ? logits : dev_error;
    if (!on_device) return SPEC_OK;  // no rows and no error word: nothing to do
    if (!select_device_of(on_device)) return SPEC_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dev_error && cudaMemsetAsync(dev_error, 0, sizeof(int32_t), st) != cudaSuccess) return SPEC_ERR_CUDA;
    if (R == 0) return SPEC_OK;
    LogprobArgs a{logits, R, V, top_k, row_stride, tokens, (float)(kLog2e / (double)temperature),
                  (float)(1.0 / (double)temperature), logprob, rank, entropy, top_ids, top_logprobs, dev_error};
    if (dtype == SPEC_BF16)
        k_token_logprobs<__nv_bfloat16><<<R, kLpThreads, 0, st>>>(a);
    else
        k_token_logprobs<float><<<R, kLpThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
