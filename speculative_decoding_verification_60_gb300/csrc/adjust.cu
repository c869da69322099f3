// Logits before they are verified or sampled from (spec_adjust_logits):
// penalties for tokens said before, biases, a grammar's mask.
#include "../../include/specverify.h"
#include "paged.cuh"

namespace sv {

constexpr int kAdNT = 256;
constexpr int kAdSlice = 4096;  // tokens of a CTA's slice
constexpr int kAdMaxBias = 1024;
constexpr int kAdAhead = 8;  // tokens of the history of a thread on their way at once
constexpr int kAdFixes = 4;  // adjusted logits of a thread on their way at once
constexpr uint32_t kAdSeen = 0x80000000u;  // a count's top bit: in the prompt

struct AdjustArgs {
    const void* in;
    void* out;
    int R, V, rows;  // rows: of a CTA
    int64_t in_stride, out_stride;
    spec_adjustments p;
    int32_t* dev_error;
};

// What a slice keeps in shared memory: counts, biases (if there are any), which
// tokens were drafted and which are biased, the tokens that anything happens to,
// the draft's tokens and parents [R], and the slice's biases (id, value).
struct AdjustSlice {
    uint32_t* count;
    float* bias;
    uint32_t *drafted, *biased;
    uint16_t* list;
    int *token, *parent;
    int2* entry;
};
__host__ __device__ inline size_t adjust_smem(const AdjustArgs& a) {
    return kAdSlice * (a.p.bias_ids ? 8 : 4) + kAdSlice / 4 + kAdSlice * 2 + (a.p.bias_ids ? (size_t)a.p.bias_count * 8 : 0) +
           (a.p.drafted ? (size_t)a.R * 8 : 0);
}

struct Penalties {
    float repetition, frequency, presence;
};
__device__ __forceinline__ float adjust_value(float x, uint32_t count, bool seen, float bias, const Penalties& q) {
    float y = x;
    if (seen) {
        y = x > 0.0f ? x / q.repetition : x * q.repetition;
        y -= q.frequency * (float)count + (count ? q.presence : 0.0f);
    }
    return y + bias;
}
template <typename T> struct Logit;
template <> struct Logit<__nv_bfloat16> {
    static constexpr int kVec = 8;
    // -inf where a bit of ok is not set
    __device__ static __forceinline__ void rule_out(uint4& q, uint32_t ok) {
        uint32_t* w = &q.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // bits 2 i and 2 i + 1 as halves of ones
            const uint32_t keep = (ok >> (2 * i) & 1u) * 0x0000ffffu | (ok >> (2 * i + 1) & 1u) * 0xffff0000u;
            w[i] = (w[i] & keep) | (0xff80ff80u & ~keep);
        }
    }
    __device__ static __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    __device__ static __forceinline__ void store(__nv_bfloat16* p, float y) { *p = __float2bfloat16_rn(y); }
};
template <> struct Logit<float> {
    static constexpr int kVec = 4;
    __device__ static __forceinline__ void rule_out(uint4& q, uint32_t ok) {
        uint32_t* w = &q.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = ok >> i & 1u ? w[i] : 0xff800000u;
    }
    __device__ static __forceinline__ float load(const float* p) { return *p; }
    __device__ static __forceinline__ void store(float* p, float y) { *p = y; }
};

// A CTA takes a slice of the vocabulary for some rows of a request.  It counts
// the request's history there once and lists the slice's tokens that anything
// happens to (seen, drafted, biased).  Then it streams the rows with the mask
// alone (a vector that the mask rules out is written without being read), and
// then goes over the listed tokens of every row, which are still in L2: they
// are one in a hundred, but some lane of a warp nearly always has one, so
// adjusting them within the stream took three times as long, with branches or
// without.  What a row's path adds to a count is found by walking up the tree.
template <typename T>
__global__ void __launch_bounds__(kAdNT) k_adjust_logits(const __grid_constant__ AdjustArgs a) {
    extern __shared__ __align__(16) uint32_t sh_adjust[];
    __shared__ int sh_listed, sh_entries;
    rows_begin();
    const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.y;
    const int v0 = blockIdx.x * kAdSlice, v1 = min(v0 + kAdSlice, a.V), width = v1 - v0;
    const spec_adjustments& p = a.p;
    AdjustSlice s;
    s.count = sh_adjust;
    s.bias = reinterpret_cast<float*>(s.count + kAdSlice);
    s.drafted = s.count + kAdSlice * (p.bias_ids ? 2 : 1);
    s.biased = s.drafted + kAdSlice / 32;
    s.list = reinterpret_cast<uint16_t*>(s.biased + kAdSlice / 32);
    s.entry = reinterpret_cast<int2*>(s.list + kAdSlice);
    s.token = reinterpret_cast<int*>(s.entry + (p.bias_ids ? p.bias_count : 0));
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
    const Penalties q{p.repetition ? p.repetition[b] : 1.0f, p.frequency ? p.frequency[b] : 0.0f,
                      p.presence ? p.presence[b] : 0.0f};
    const bool penalties = q.repetition != 1.0f || q.frequency != 0.0f || q.presence != 0.0f;
    if (penalties)
        for (int i = tid; i < kAdSlice / 4; i += kAdNT) reinterpret_cast<uint4*>(s.count)[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < kAdSlice / 32 * 2; i += kAdNT) s.drafted[i] = 0;
    if (tid == 0) sh_listed = sh_entries = 0;
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
        for (int i0 = tid; i0 < n; i0 += kAdNT * kAdAhead) {
            int v[kAdAhead];
#pragma unroll
            for (int k = 0; k < kAdAhead; ++k) v[k] = ids[min(i0 + k * kAdNT, n - 1)];
#pragma unroll
            for (int k = 0; k < kAdAhead; ++k) {
                const uint32_t at = (uint32_t)(v[k] - v0);
                if ((uint32_t)v[k] >= (uint32_t)a.V) err |= kDevErrToken;
                const int i = i0 + k * kAdNT;
                if (at >= (uint32_t)width || i >= n) continue;
                if (i >= said) atomicAdd(s.count + at, 1u);
                else atomicOr(s.count + at, kAdSeen);
            }
        }
    }
    if (p.drafted && penalties && tree)
        for (int i = 1 + tid; i < rows; i += kAdNT) {
            const int v = s.token[i];
            if (v < 0 || v >= a.V) err |= kDevErrToken;
            if (v >= v0 && v < v1) atomicOr(s.drafted + ((v - v0) >> 5), 1u << ((v - v0) & 31));
        }
    if (p.bias_ids) {
        // the first warp picks the slice's biases, in order
        if (tid < 32) {
            const int32_t* ids = p.bias_ids + (int64_t)b * p.bias_count;
            const float* values = p.bias_values + (int64_t)b * p.bias_count;
            int n = 0;
            for (int j0 = 0; j0 < p.bias_count; j0 += 32) {
                const int j = j0 + lane, v = j < p.bias_count ? ids[j] : -1;
                if (v < -1 || v >= a.V) err |= kDevErrToken;
                const bool in = v >= v0 && v < v1;
                const uint32_t all = __ballot_sync(0xffffffffu, in);
                if (in) s.entry[n + __popc(all & ((1u << lane) - 1u))] = make_int2(v - v0, __float_as_int(values[j]));
                n += __popc(all);
            }
            if (lane == 0) sh_entries = n;
        }
        __syncthreads();
        // the first entry of an id sums them all, in order
        const int n = sh_entries;
        for (int j = tid; j < n; j += kAdNT) {
            const int at = s.entry[j].x;
            float sum = 0.0f;
            bool first = true;
            for (int k = 0; k < n; ++k)
                if (s.entry[k].x == at) {
                    first = first && k >= j;
                    sum = k == j ? __int_as_float(s.entry[k].y) : sum + __int_as_float(s.entry[k].y);
                }
            if (!first) continue;
            s.bias[at] = sum;
            atomicOr(s.biased + (at >> 5), 1u << (at & 31));
        }
    }
    if (err) set_error(a.dev_error, err);
    __syncthreads();
    if (penalties || p.bias_ids) {
        for (int i = tid; i < kAdSlice; i += kAdNT) {  // 32 tokens of a warp
            const bool hit = ((s.drafted[i >> 5] | s.biased[i >> 5]) >> lane & 1u) || (penalties && s.count[i] != 0);
            const uint32_t all = __ballot_sync(0xffffffffu, hit);
            if (!all) continue;
            int at = 0;
            if (lane == 0) at = atomicAdd(&sh_listed, __popc(all));
            at = __shfl_sync(0xffffffffu, at, 0) + __popc(all & ((1u << lane) - 1u));
            if (hit) s.list[at] = (uint16_t)i;
        }
    }

    constexpr int VE = Logit<T>::kVec;
    const int r0 = blockIdx.z * a.rows, r1 = min(r0 + a.rows, rows);
    const int last_word = (a.V - 1) >> 5;
    auto row_of = [&](int r) { return (int64_t)b * a.R + r; };
    auto in_of = [&](int r) { return static_cast<const T*>(a.in) + row_of(r) * a.in_stride + v0; };
    auto out_of = [&](int r) { return static_cast<T*>(a.out) + row_of(r) * a.out_stride + v0; };
    auto allowed_of = [&](int r) { return reinterpret_cast<const uint32_t*>(p.allowed) + row_of(r) * p.allowed_stride; };
    // a thread has kAcross vectors of a row, and kRows rows on their way at once
    constexpr int kAcross = kAdSlice / VE / kAdNT, kRows = 4 / kAcross;
    constexpr uint32_t kAll = (1u << VE) - 1;
    for (int rb = r0; rb < r1; rb += kRows) {
        const uint4* from[kRows];
        uint4* to[kRows];
        const uint32_t* allowed[kRows];
        int head[kRows], vecs[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int r = min(rb + k, r1 - 1);
            const T* in = in_of(r);
            T* out = out_of(r);
            allowed[k] = p.allowed ? allowed_of(r) : nullptr;
            const uint32_t skew = (uint32_t)(reinterpret_cast<uintptr_t>(in) & 15u);
            // vectors lie on 16 bytes in both; where in and out differ in alignment there are none
            const bool same = skew == (uint32_t)(reinterpret_cast<uintptr_t>(out) & 15u);
            head[k] = same ? min(width, (int)((16u - skew) & 15u) / (int)sizeof(T)) : width;
            vecs[k] = rb + k < r1 ? (width - head[k]) / VE : 0;
            from[k] = reinterpret_cast<const uint4*>(in + head[k]);
            to[k] = reinterpret_cast<uint4*>(out + head[k]);
            if (rb + k >= r1) continue;
            auto single = [&](int at) {
                const int v = v0 + at;
                if (allowed[k] && !((allowed[k][v >> 5] >> (v & 31)) & 1u)) Logit<T>::store(out + at, -INFINITY);
                else out[at] = in[at];
            };
            for (int at = tid; at < head[k]; at += kAdNT) single(at);
            const int tail = head[k] + vecs[k] * VE;
            if (tid < width - tail) single(tail + tid);
        }
        uint4 x[kRows][kAcross];
        uint32_t ok[kRows][kAcross];
#pragma unroll
        for (int k = 0; k < kRows; ++k)
#pragma unroll
            for (int u = 0; u < kAcross; ++u) {
                const int i = tid + u * kAdNT;
                ok[k][u] = i < vecs[k] ? kAll : 0u;
                if (p.allowed && i < vecs[k]) {
                    const int v = v0 + head[k] + i * VE, w = v >> 5;
                    ok[k][u] = __funnelshift_r(allowed[k][w], allowed[k][min(w + 1, last_word)], v & 31) & kAll;
                }
            }
#pragma unroll
        for (int k = 0; k < kRows; ++k)
#pragma unroll
            for (int u = 0; u < kAcross; ++u)
                if (ok[k][u]) x[k][u] = from[k][tid + u * kAdNT];
#pragma unroll
        for (int k = 0; k < kRows; ++k)
#pragma unroll
            for (int u = 0; u < kAcross; ++u) {
                if (tid + u * kAdNT >= vecs[k]) continue;
                if (ok[k][u] != kAll) Logit<T>::rule_out(x[k][u], ok[k][u]);
                to[k][tid + u * kAdNT] = x[k][u];
            }
    }
    __syncthreads();  // the rows are written, and the list

    // a thread has every `places`-th listed token, in every `phases`-th row
    const int listed = sh_listed;
    int places = kAdNT;
    while (places / 2 >= listed && places > 8) places /= 2;
    const int phases = kAdNT / places, phase = tid / places;
    for (int i = tid - phase * places; i < listed; i += places) {
        const int at = s.list[i], v = v0 + at;
        auto marked = [&](const uint32_t* map) { return map[at >> 5] >> (at & 31) & 1u; };
        const uint32_t n = penalties ? s.count[at] : 0u;
        const bool drafted = marked(s.drafted);
        const float bias = marked(s.biased) ? s.bias[at] : 0.0f;
        const T* in = in_of(r0 + phase) + at;
        T* out = out_of(r0 + phase) + at;
        const uint32_t* allowed = p.allowed ? allowed_of(r0 + phase) + (v >> 5) : nullptr;
        const int64_t in_step = phases * a.in_stride, out_step = phases * a.out_stride, allowed_step = phases * p.allowed_stride;
        for (int r = r0 + phase; r < r1; r += phases * kAdFixes) {
            float x[kAdFixes];
            bool live[kAdFixes];
#pragma unroll
            for (int k = 0; k < kAdFixes; ++k) {
                live[k] = r + k * phases < r1;
                if (!live[k]) continue;
                x[k] = Logit<T>::load(in + k * in_step);  // the stream left it as it was, if it is allowed
                if (allowed) live[k] = allowed[k * allowed_step] >> (v & 31) & 1u;
            }
#pragma unroll
            for (int k = 0; k < kAdFixes; ++k) {
                if (!live[k]) continue;
                uint32_t count = n & ~kAdSeen;
                bool seen = n != 0;
                if (drafted)
                    for (int i = r + k * phases; i > 0; i = s.parent[i])
                        if (s.token[i] == v) {
                            seen = true;
                            ++count;
                        }
                Logit<T>::store(out + k * out_step, adjust_value(x[k], count, seen, bias, q));
            }
            in += kAdFixes * in_step;
            out += kAdFixes * out_step;
            if (allowed) allowed += kAdFixes * allowed_step;
        }
    }
}

template <typename T>
static cudaError_t launch_adjust(AdjustArgs a, int B, cudaStream_t st) {
    LaunchShape shape;
    const void* kernel = reinterpret_cast<const void*>(k_adjust_logits<T>);
    const size_t smem = adjust_smem(a);
    // the shape is asked for with the memory of the largest call, which is also what the kernel is allowed
    AdjustArgs most = a;
    most.R = kMaxDraftNodes;
    most.p.drafted = most.p.bias_ids = reinterpret_cast<const int32_t*>(&a);  // not NULL; only the size counts
    most.p.bias_count = kAdMaxBias;
    if (!launch_shape(kernel, adjust_smem(most), kAdNT, &shape)) return cudaErrorUnknown;
    const int slices = (a.V + kAdSlice - 1) / kAdSlice;
    // rows of a request are shared out only where its slices do not fill the GPU
    const long long want = (long long)shape.sms * shape.per_sm, have = (long long)slices * B;
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
    AdjustArgs a{logits, out, R, V, 0, row_stride, out_stride, p, dev_error};
    return (dtype == SPEC_BF16 ? launch_adjust<__nv_bfloat16>(a, B, st) : launch_adjust<float>(a, B, st)) == cudaSuccess
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}
