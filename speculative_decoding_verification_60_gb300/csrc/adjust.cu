// Logits before they are verified or sampled from (spec_adjust_logits):
// penalties for tokens said before, biases, a grammar's mask.
#include "../../include/specverify.h"
#include "paged.cuh"

namespace sv {

constexpr int kAdNT = 256;
constexpr int kAdSlice = 8192;  // tokens of a CTA's slice at most
constexpr int kAdMaxBias = 1024;
constexpr uint32_t kAdSeen = 0x80000000u;  // a count's top bit: in the prompt

struct AdjustArgs {
    const void* in;
    void* out;
    int R, V, slice, rows;  // slice: tokens of a CTA, a multiple of 32; rows: rows of a CTA
    int64_t in_stride, out_stride;
    spec_adjustments p;
    int32_t* dev_error;
};

// What a slice keeps in shared memory, behind each other: counts [slice],
// biases [slice] (if there are any), three bitmaps of the slice (one word more
// each, for reads across a word's end), the draft's tokens and parents [R].
struct AdjustSlice {
    uint32_t* count;
    float* bias;
    uint32_t *touched, *drafted, *biased;
    int *token, *parent;
};
__host__ __device__ inline size_t adjust_smem(const AdjustArgs& a) {
    const size_t words = a.slice / 32 + 1;
    return ((size_t)a.slice * (a.p.bias_ids ? 2 : 1) + 3 * words + (a.p.drafted ? 2 * a.R : 0)) * 4;
}

// Bits at .. at + 31 of a bitmap.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* map, int at) {
    return __funnelshift_r(map[at >> 5], map[(at >> 5) + 1], at & 31);
}

// One logit of row i (a token of the slice at place `at`).
__device__ __noinline__ float adjust_one(float x, int at, int v, int i, bool drafted, bool biased, float repetition,
                                         float frequency, float presence, const AdjustSlice& s) {
    const uint32_t n = s.count[at];
    bool seen = n != 0;
    uint32_t c = n & ~kAdSeen;
    if (drafted)
        for (; i > 0; i = s.parent[i])
            if (s.token[i] == v) {
                seen = true;
                ++c;
            }
    float y = x;
    if (seen) y = x > 0.0f ? x / repetition : x * repetition;
    if (seen) y -= frequency * (float)c + (c ? presence : 0.0f);
    if (biased) y += s.bias[at];
    return y;
}

template <typename T> struct Logit;
template <> struct Logit<__nv_bfloat16> {
    static constexpr int kVec = 8;
    __device__ static __forceinline__ float get(const uint4& q, int k) {
        const uint32_t w = k < 2 ? q.x : k < 4 ? q.y : k < 6 ? q.z : q.w;
        return (k & 1) ? bf16_hi(w) : bf16_lo(w);
    }
    __device__ static __forceinline__ void put(uint4& q, int k, float y) {
        uint32_t& w = k < 2 ? q.x : k < 4 ? q.y : k < 6 ? q.z : q.w;
        const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rn(y));
        w = (k & 1) ? (w & 0xffffu) | (h << 16) : (w & 0xffff0000u) | h;
    }
    __device__ static __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    __device__ static __forceinline__ void store(__nv_bfloat16* p, float y) { *p = __float2bfloat16_rn(y); }
};
template <> struct Logit<float> {
    static constexpr int kVec = 4;
    __device__ static __forceinline__ float get(const uint4& q, int k) {
        return __uint_as_float(k == 0 ? q.x : k == 1 ? q.y : k == 2 ? q.z : q.w);
    }
    __device__ static __forceinline__ void put(uint4& q, int k, float y) {
        (k == 0 ? q.x : k == 1 ? q.y : k == 2 ? q.z : q.w) = __float_as_uint(y);
    }
    __device__ static __forceinline__ float load(const float* p) { return *p; }
    __device__ static __forceinline__ void store(float* p, float y) { *p = y; }
};

// A CTA takes a slice of the vocabulary for some rows of a request.  It counts
// the request's history there once, marks which tokens of the slice anything
// happens to (seen, drafted, biased), and then streams the rows: a vector
// without a mark is copied, one that the mask rules out is written without
// being read.  Marks are rare, so the stream is bound by memory; what a row's
// path adds to a count is found by walking up the tree for the few tokens that
// were drafted.
template <typename T>
__global__ void __launch_bounds__(kAdNT) k_adjust_logits(const __grid_constant__ AdjustArgs a) {
    extern __shared__ uint32_t sh_adjust[];
    rows_begin();
    const int tid = threadIdx.x, b = blockIdx.y;
    const int v0 = blockIdx.x * a.slice, v1 = min(v0 + a.slice, a.V), width = v1 - v0;
    const spec_adjustments& p = a.p;
    const int words = a.slice / 32 + 1;
    AdjustSlice s;
    s.count = sh_adjust;
    s.bias = reinterpret_cast<float*>(s.count + a.slice);
    s.touched = s.count + (size_t)a.slice * (p.bias_ids ? 2 : 1);
    s.drafted = s.touched + words;
    s.biased = s.drafted + words;
    s.token = reinterpret_cast<int*>(s.biased + words);
    s.parent = s.token + a.R;
    int err = 0;
    int rows = a.R;
    if (p.n_nodes) {
        rows = p.n_nodes[b];
        if (rows < 0 || rows > a.R) {
            err |= kDevErrLength;
            rows = a.R;
        }
    }
    const float repetition = p.repetition ? p.repetition[b] : 1.0f, frequency = p.frequency ? p.frequency[b] : 0.0f,
                presence = p.presence ? p.presence[b] : 0.0f;
    const bool penalties = repetition != 1.0f || frequency != 0.0f || presence != 0.0f;
    for (int i = tid; i < a.slice; i += kAdNT) s.count[i] = 0;
    for (int i = tid; i < 3 * words; i += kAdNT) s.touched[i] = 0;
    bool tree = true;
    if (p.drafted && penalties) {
        if (p.parent) tree = tree_part_ok(p.parent + b * p.parent_stride, rows, tid, kAdNT);
        for (int i = tid; i < rows; i += kAdNT) {
            s.token[i] = i > 0 ? p.drafted[b * p.drafted_stride + i - 1] : -1;
            s.parent[i] = p.parent ? p.parent[b * p.parent_stride + i] : i - 1;
        }
    }
    tree = __syncthreads_and(tree);
    if (!tree) err |= kDevErrParent;
    if (p.history && penalties) {
        int n = p.history_lens[b];
        if (n < 0 || n > p.history_capacity) {
            err |= kDevErrLength;
            n = 0;
        }
        int said = p.prompt_lens ? p.prompt_lens[b] : 0;
        if (said < 0 || said > n) {
            err |= kDevErrLength;
            said = said < 0 ? 0 : n;
        }
        const int32_t* ids = p.history + b * p.history_stride;
        for (int i = tid; i < n; i += kAdNT) {
            const int v = ids[i];
            if (v < 0 || v >= a.V) err |= kDevErrToken;
            if (v < v0 || v >= v1) continue;
            if (i >= said) atomicAdd(s.count + (v - v0), 1u);
            else atomicOr(s.count + (v - v0), kAdSeen);
        }
    }
    if (p.drafted && penalties && tree)
        for (int i = 1 + tid; i < rows; i += kAdNT) {
            const int v = s.token[i];
            if (v < 0 || v >= a.V) err |= kDevErrToken;
            if (v >= v0 && v < v1) atomicOr(s.drafted + ((v - v0) >> 5), 1u << ((v - v0) & 31));
        }
    if (p.bias_ids) {
        const int32_t* ids = p.bias_ids + (int64_t)b * p.bias_count;
        const float* values = p.bias_values + (int64_t)b * p.bias_count;
        for (int j = tid; j < p.bias_count; j += kAdNT) {
            const int v = ids[j];
            if (v < -1 || v >= a.V) err |= kDevErrToken;
            if (v < v0 || v >= v1) continue;
            // the first entry of an id sums them all, in order
            bool first = true;
            for (int k = 0; k < j; ++k) first = first && ids[k] != v;
            if (!first) continue;
            float sum = values[j];
            for (int k = j + 1; k < p.bias_count; ++k)
                if (ids[k] == v) sum += values[k];
            s.bias[v - v0] = sum;
            atomicOr(s.biased + ((v - v0) >> 5), 1u << ((v - v0) & 31));
        }
    }
    if (err) set_error(a.dev_error, err);
    __syncthreads();
    for (int i = tid; i < (width + 31) / 32 * 32; i += kAdNT) {  // whole warps
        const uint32_t hit = __ballot_sync(0xffffffffu, s.count[i] != 0);
        if ((i & 31) == 0) s.touched[i >> 5] = hit | s.drafted[i >> 5] | s.biased[i >> 5];
    }
    __syncthreads();

    constexpr int VE = Logit<T>::kVec;
    const int r0 = blockIdx.z * a.rows, r1 = min(r0 + a.rows, rows);
    const int last_word = (a.V - 1) >> 5;
    for (int r = r0; r < r1; ++r) {
        const int64_t row = (int64_t)b * a.R + r;
        const T* in = static_cast<const T*>(a.in) + row * a.in_stride + v0;
        T* out = static_cast<T*>(a.out) + row * a.out_stride + v0;
        const uint32_t* allowed =
            p.allowed ? reinterpret_cast<const uint32_t*>(p.allowed) + row * p.allowed_stride : nullptr;
        auto one = [&](float x, int at) {
            if (!((s.touched[at >> 5] >> (at & 31)) & 1u)) return x;
            return adjust_one(x, at, v0 + at, r, (s.drafted[at >> 5] >> (at & 31)) & 1u,
                              (s.biased[at >> 5] >> (at & 31)) & 1u, repetition, frequency, presence, s);
        };
        auto single = [&](int at) {
            const int v = v0 + at;
            if (allowed && !((allowed[v >> 5] >> (v & 31)) & 1u)) Logit<T>::store(out + at, -INFINITY);
            else Logit<T>::store(out + at, one(Logit<T>::load(in + at), at));
        };
        const uint32_t skew = (uint32_t)(reinterpret_cast<uintptr_t>(in) & 15u);
        if (skew != (uint32_t)(reinterpret_cast<uintptr_t>(out) & 15u)) {
            // in and out differ in alignment: element by element
            for (int at = tid; at < width; at += kAdNT) single(at);
            continue;
        }
        const int head = min(width, (int)((16u - skew) & 15u) / (int)sizeof(T));
        const int vecs = (width - head) / VE, tail = head + vecs * VE;
        if (tid < head) single(tid);
        if (tid >= 32 && tid - 32 < width - tail) single(tail + tid - 32);
        constexpr int U = 4;
        constexpr uint32_t kAll = (1u << VE) - 1;
        for (int i0 = tid; i0 < vecs; i0 += kAdNT * U) {
            uint4 x[U];
            uint32_t ok[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * kAdNT;
                ok[u] = i < vecs ? kAll : 0u;
                if (allowed && i < vecs) {
                    const int v = v0 + head + i * VE, w = v >> 5;
                    ok[u] = __funnelshift_r(allowed[w], allowed[min(w + 1, last_word)], v & 31) & kAll;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (ok[u]) x[u] = *reinterpret_cast<const uint4*>(in + head + (i0 + u * kAdNT) * VE);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * kAdNT;
                if (i >= vecs) continue;
                const int at = head + i * VE;
                if (!ok[u]) {
                    x[u] = RowVec<T>::none();
                } else {
                    const uint32_t mark = bits_at(s.touched, at) & ok[u];
                    if (mark | (ok[u] ^ kAll)) {
#pragma unroll
                        for (int k = 0; k < VE; ++k) {
                            if ((mark >> k) & 1u) Logit<T>::put(x[u], k, one(Logit<T>::get(x[u], k), at + k));
                            if (!((ok[u] >> k) & 1u)) Logit<T>::put(x[u], k, -INFINITY);
                        }
                    }
                }
                *reinterpret_cast<uint4*>(out + at) = x[u];
            }
        }
    }
}

template <typename T>
static cudaError_t launch_adjust(AdjustArgs a, int B, cudaStream_t st) {
    LaunchShape shape;
    const void* kernel = reinterpret_cast<const void*>(k_adjust_logits<T>);
    a.slice = kAdSlice;
    const size_t smem = adjust_smem(a);
    // the shape is asked for with the memory of the largest call, which is also what the kernel is allowed
    AdjustArgs most = a;
    most.R = kMaxDraftNodes;
    most.p.drafted = most.p.bias_ids = reinterpret_cast<const int32_t*>(&a);  // not NULL; only the size counts
    if (!launch_shape(kernel, adjust_smem(most), kAdNT, &shape)) return cudaErrorUnknown;
    const int slices = (a.V + a.slice - 1) / a.slice;
    // rows of a request are shared out only where its slices do not fill the GPU
    const long long want = 2LL * shape.sms * shape.per_sm, have = (long long)slices * B;
    int parts = (int)(have >= want ? 1 : (want + have - 1) / have);
    parts = parts < a.R ? parts : a.R;
    a.rows = (a.R + parts - 1) / parts;
    parts = (a.R + a.rows - 1) / a.rows;
    return launch_dependent(k_adjust_logits<T>, dim3(slices, B, parts), dim3(kAdNT), smem, st, a);
}

}  // namespace sv

using namespace sv;

extern "C" spec_status spec_adjust_logits(const void* logits, spec_dtype dtype, int B, int R, int V, int64_t row_stride,
                                          const spec_adjustments* adjustments, void* out, int64_t out_stride,
                                          int32_t* dev_error, spec_stream_t stream) {
    DeviceGuard device_guard;  // the caller's current device is put back on return
    if (dtype != SPEC_BF16 && dtype != SPEC_F32) return SPEC_ERR_INVALID_ARG;
    if ((B > 0 && (!logits || !out)) || !adjustments || B < 0 || R < 1 || V < 1 || row_stride < V || out_stride < V)
        return SPEC_ERR_INVALID_ARG;
    const spec_adjustments& p = *adjustments;
    if (p.history && (!p.history_lens || p.history_capacity < 0 || p.history_stride < p.history_capacity))
        return SPEC_ERR_INVALID_ARG;
    if (p.drafted && p.drafted_stride < R - 1) return SPEC_ERR_INVALID_ARG;
    if (p.parent && p.parent_stride != 0 && p.parent_stride < R) return SPEC_ERR_INVALID_ARG;
    if (p.bias_ids && (!p.bias_values || p.bias_count < 0)) return SPEC_ERR_INVALID_ARG;
    if (p.allowed && p.allowed_stride < (V + 31) / 32) return SPEC_ERR_INVALID_ARG;
    if (B > 0 && out == logits && out_stride != row_stride) return SPEC_ERR_INVALID_ARG;
    if ((int64_t)V > kRowsMaxVocab || R > kMaxDraftNodes || B > kMaxRequests ||
        (p.bias_ids && p.bias_count > kAdMaxBias))
        return SPEC_ERR_UNSUPPORTED;
    if (B == 0 && !dev_error) return SPEC_OK;
    if (!select_device_of(B > 0 ? logits : dev_error)) return SPEC_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const spec_status cleared = clear_error(dev_error, st);
    if (cleared != SPEC_OK || B == 0) return cleared;
    AdjustArgs a{logits, out, R, V, 0, 0, row_stride, out_stride, p, dev_error};
    return (dtype == SPEC_BF16 ? launch_adjust<__nv_bfloat16>(a, B, st) : launch_adjust<float>(a, B, st)) == cudaSuccess
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}
