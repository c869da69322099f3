// Logits before they are verified or sampled from (spec_adjust_logits):
// penalties for tokens said before, biases, a grammar's mask.
#include "../../include/specverify.h"
#include "paged.cuh"

namespace sv {

constexpr int kAdNT = 256;
constexpr int kAdSlice = 4096;  // tokens of a CTA's slice
constexpr int kAdWaves = 2;     // of CTAs that rows are shared out for
constexpr int kAdMaxBias = 1024;
constexpr int kAdMaxHistory = 536000000;  // with a path, below 2^29
// Tokens of the history of a lane on their way at once: 12 requests of 60 rows 97.5 us, 100 with 8, 99 with 32.
constexpr int kAdAhead = 16;
constexpr int kAdHistory = 32 * kAdAhead * 2;  // tokens of the history that a warp takes at a time
constexpr int kAdFixes = 4;  // adjusted logits of a thread on their way at once
// A token's cell: how often it was said (the prompt apart), and whether it is in
// the prompt, was drafted, is biased.  Nothing happens to a token of cell 0.
constexpr uint32_t kAdPrompt = 1u << 31, kAdDrafted = 1u << 30, kAdBiased = 1u << 29, kAdCount = kAdBiased - 1;

struct AdjustArgs {
    const void* in;
    void* out;
    int R, V, rows;  // rows: of a CTA
    int64_t in_stride, out_stride;
    spec_adjustments p;
    int32_t* dev_error;
};

// What a slice keeps in shared memory: its tokens' cells and biases (if there
// are any), a list of tokens, the draft's tokens and parents [R], and the
// slice's biases (place, value).  Cells and biases are laid out for lanes that
// have a vector of VE tokens each: the token at place `at` is in row at % VE,
// column at / VE.
struct AdjustSlice {
    uint32_t* cell;
    float* bias;
    uint16_t* list;
    int *token, *parent;
    int2* entry;
    uint32_t* kept;  // a dense request's listed tokens' cells
};
constexpr int kAdCells = kAdSlice + 8;
template <int VE> __device__ __forceinline__ int adjust_cell(int at) { return (at % VE) * (kAdSlice / VE + 1) + at / VE; }
template <int VE> __device__ __forceinline__ int adjust_place(int cell) {
    const int row = cell / (kAdSlice / VE + 1);
    return (cell - row * (kAdSlice / VE + 1)) * VE + row;
}
__host__ __device__ inline size_t adjust_smem(const AdjustArgs& a) {
    return kAdCells * (a.p.bias_ids ? 8 : 4) + kAdSlice * 2 + (a.p.bias_ids ? (size_t)a.p.bias_count * 12 : 0) +
           (a.p.drafted ? (size_t)a.R * 12 : 0);
}

// Bytes (a multiple of 16, on 16) on their way into L2.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// A request's penalties.  A product with 1 / repetition stands for the division
// where neither leaves the range of 32 bits: two roundings, 2^-23 of the value at
// most, and a third of the time that the division takes over a row of seen tokens.
struct Penalties {
    float repetition, inverse, frequency, presence;
    bool divides;
};
__device__ __forceinline__ float adjust_value(float x, uint32_t cell, const Penalties& q) {
    const uint32_t count = cell & kAdCount;
    const float y = cell & (kAdCount | kAdPrompt) ? x * (x > 0.0f ? q.inverse : q.repetition) : x;
    return count ? y - fmaf(q.frequency, (float)count, q.presence) : y;
}
// The same from what a dense request's cells become: what is taken off the logit,
// as a float; the bits of zero stand for a token that was not seen, -0 for a
// seen one that nothing is taken off.
__device__ __forceinline__ uint32_t adjust_pack(uint32_t cell, const Penalties& q) {
    const uint32_t count = cell & kAdCount;
    const uint32_t less = count ? __float_as_uint(fmaf(q.frequency, (float)count, q.presence)) : 0u;
    return cell == 0 ? 0u : less == 0 ? 0x80000000u : less;
}
__device__ __forceinline__ float adjust_packed(float x, uint32_t pack, const Penalties& q) {
    return (pack ? x * (x > 0.0f ? q.inverse : q.repetition) : x) - __uint_as_float(pack);
}
// The same with all that is rare: a draft's tokens (those on the path to node i
// count), biases, repetitions that have to be divided by.
__device__ __noinline__ float adjust_rare(float x, int v, uint32_t cell, float bias, int i, const int* token,
                                          const int* parent, const Penalties& q) {
    uint32_t count = cell & kAdCount;
    bool seen = (cell & (kAdCount | kAdPrompt)) != 0;
    if (cell & kAdDrafted)
        for (; i > 0; i = parent[i])
            if (token[i] == v) {
                seen = true;
                ++count;
            }
    float y = x;
    if (seen) y = x > 0.0f ? x / q.repetition : x * q.repetition;
    if (count) y -= fmaf(q.frequency, (float)count, q.presence);
    return cell & kAdBiased ? y + bias : y;
}

template <typename T> struct Logit;
template <> struct Logit<__nv_bfloat16> {
    static constexpr int kVec = 8;
    __device__ static __forceinline__ void get(const uint4& q, float* x) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    __device__ static __forceinline__ uint4 put(const float* x) {
        return make_uint4(Pair<__nv_bfloat16>::put(x[0], x[1]), Pair<__nv_bfloat16>::put(x[2], x[3]),
                          Pair<__nv_bfloat16>::put(x[4], x[5]), Pair<__nv_bfloat16>::put(x[6], x[7]));
    }
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
    __device__ static __forceinline__ void get(const uint4& q, float* x) {
        x[0] = __uint_as_float(q.x);
        x[1] = __uint_as_float(q.y);
        x[2] = __uint_as_float(q.z);
        x[3] = __uint_as_float(q.w);
    }
    __device__ static __forceinline__ uint4 put(const float* x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    __device__ static __forceinline__ void rule_out(uint4& q, uint32_t ok) {
        uint32_t* w = &q.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = ok >> i & 1u ? w[i] : 0xff800000u;
    }
    __device__ static __forceinline__ float load(const float* p) { return *p; }
    __device__ static __forceinline__ void store(float* p, float y) { *p = y; }
};

// A CTA takes a slice of the vocabulary for some rows of a request.  Its warps
// draw their work from a counter: parts of the request's history, whose tokens
// are counted where they fall into the slice, and parts of the rows, streamed
// with the mask alone (a vector that the mask rules out is written without being
// read).  After that, the slice's tokens that anything happens to (seen,
// drafted, biased) are listed and adjusted in every row, which is still in L2:
// they are one in a hundred, but some lane of a warp nearly always has one, so
// adjusting them within the stream took 482 us, with branches or without, where
// this took 290 (256 requests of 9 rows).  Only where the history has more than
// a 16th as many tokens as the vocabulary is it counted first and the counts
// applied within the stream (12 requests of 60 rows, 7,500 to 30,000 tokens of
// 50,021: 97.5 us, 160 without); then drafted and biased tokens alone are listed.
// What a row's path adds to a count is found by walking up the tree.
// Bound by latency: 256 requests of 9 rows at V = 128,256 take 232 us, 0.68 of the
// copy rate for what has to be moved.  A copy without history, masks and biases
// runs at 0.86; what is missing is the time in which a CTA's warps wait for each
// other around its list.  Slices of 8,192 tokens 255 us, four CTAs an SM 242, five
// of four vectors a lane 257.
template <typename T>
__global__ void __launch_bounds__(kAdNT, 3) k_adjust_logits(const __grid_constant__ AdjustArgs a) {
    constexpr int VE = Logit<T>::kVec;
    extern __shared__ __align__(16) uint32_t sh_adjust[];
    __shared__ int sh_listed, sh_task, sh_part, sh_entries;
    rows_begin();
    const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.y;
    const int v0 = blockIdx.x * kAdSlice, v1 = min(v0 + kAdSlice, a.V), width = v1 - v0;
    const spec_adjustments& p = a.p;
    AdjustSlice s;
    s.cell = sh_adjust;
    s.bias = reinterpret_cast<float*>(s.cell + kAdCells);
    s.list = reinterpret_cast<uint16_t*>(s.cell + kAdCells * (p.bias_ids ? 2 : 1));
    s.entry = reinterpret_cast<int2*>(s.list + kAdSlice);
    s.token = reinterpret_cast<int*>(s.entry + (p.bias_ids ? p.bias_count : 0));
    s.parent = s.token + a.R;
    s.kept = reinterpret_cast<uint32_t*>(s.token + (p.drafted ? 2 * a.R : 0));
    int err = 0;
    int rows = p.n_nodes ? p.n_nodes[b] : a.R;
    int told = p.history ? p.history_lens[b] : 0, said = p.history && p.prompt_lens ? p.prompt_lens[b] : 0;
    Penalties q;
    q.repetition = p.repetition ? p.repetition[b] : 1.0f;
    q.frequency = p.frequency ? p.frequency[b] : 0.0f;
    q.presence = p.presence ? p.presence[b] : 0.0f;
    q.inverse = 1.0f / q.repetition;
    q.divides = !(fabsf(q.repetition) > 0x1p-100f && fabsf(q.repetition) < 0x1p100f);
    const bool penalties = q.repetition != 1.0f || q.frequency != 0.0f || q.presence != 0.0f;
    if (rows < 0 || rows > a.R) {
        err |= kDevErrLength;
        rows = a.R;
    }
    if (!penalties) told = said = 0;
    if (told < 0 || told > p.history_capacity) {
        err |= kDevErrLength;
        told = 0;
    }
    if (said < 0 || said > told) {
        err |= kDevErrLength;
        said = said < 0 ? 0 : told;
    }
    const bool dense = (int64_t)told * 16 > a.V && !q.divides;
    if (penalties || p.bias_ids)
        for (int i = tid; i < kAdCells / 4; i += kAdNT) reinterpret_cast<uint4*>(s.cell)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) sh_listed = sh_task = sh_part = sh_entries = 0;
    int bias_id[kAdMaxBias / kAdNT];
    if (p.bias_ids)
#pragma unroll
        for (int k = 0; k < kAdMaxBias / kAdNT; ++k) {
            const int j = tid + k * kAdNT;
            bias_id[k] = j < p.bias_count ? p.bias_ids[(int64_t)b * p.bias_count + j] : -1;
        }
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
    if (p.drafted && penalties && tree)
        for (int i = 1 + tid; i < rows; i += kAdNT) {
            const int v = s.token[i];
            if (v < 0 || v >= a.V) err |= kDevErrToken;
            if (v >= v0 && v < v1) atomicOr(s.cell + adjust_cell<VE>(v - v0), kAdDrafted);
        }
    if (p.bias_ids) {
#pragma unroll
        for (int k = 0; k < kAdMaxBias / kAdNT; ++k) {
            const int v = bias_id[k];
            if (v < -1 || v >= a.V) err |= kDevErrToken;
            if (v < v0 || v >= v1) continue;
            s.entry[atomicAdd(&sh_entries, 1)] = make_int2(v - v0, tid + k * kAdNT);
            atomicOr(s.cell + adjust_cell<VE>(v - v0), kAdBiased);
        }
    }

    // A row's slice is asked for before the warps get to it (256 requests of 9 rows: 232 us, 281 without), but not
    // where the mask rules most of it out, nor where the history comes first.
    if (!dense)
        for (int r = blockIdx.z * a.rows + (tid >> 5); r < min((int)(blockIdx.z + 1) * a.rows, rows); r += kAdNT / 32) {
            const int64_t row = (int64_t)b * a.R + r;
            const uintptr_t from = reinterpret_cast<uintptr_t>(static_cast<const T*>(a.in) + row * a.in_stride + v0);
            const uintptr_t begin = (from + 15) & ~(uintptr_t)15, end = (from + (uintptr_t)width * sizeof(T)) & ~(uintptr_t)15;
            int open = width;
            if (p.allowed) {
                const uint32_t* allowed = reinterpret_cast<const uint32_t*>(p.allowed) + row * p.allowed_stride + (v0 >> 5);
                open = 0;
#pragma unroll
                for (int w = 0; w < kAdSlice / 32 / 32; ++w)
                    if (w * 32 + lane < (width + 31) / 32) open += __popc(allowed[w * 32 + lane]);
                open = __reduce_add_sync(0xffffffffu, open);
            }
            if (lane == 0 && open * 8 > width && end > begin) prefetch_l2(reinterpret_cast<const void*>(begin), (uint32_t)(end - begin));
        }

    // parts of the history
    const int32_t* ids = p.history + b * p.history_stride;
    auto history = [&](int part) {
        const int first = part * kAdHistory + lane, end = min((part + 1) * kAdHistory, told);
        for (int i0 = first; i0 < end; i0 += 32 * kAdAhead) {
            int v[kAdAhead];
#pragma unroll
            for (int k = 0; k < kAdAhead; ++k) v[k] = ids[min(i0 + k * 32, end - 1)];
#pragma unroll
            for (int k = 0; k < kAdAhead; ++k) {
                const uint32_t at = (uint32_t)(v[k] - v0);
                if ((uint32_t)v[k] >= (uint32_t)a.V) err |= kDevErrToken;
                const int i = i0 + k * 32;
                if (at >= (uint32_t)width || i >= end) continue;
                uint32_t* cell = s.cell + adjust_cell<VE>((int)at);
                if (i >= said) atomicAdd(cell, 1u);
                else atomicOr(cell, kAdPrompt);
            }
        }
    };
    // parts of the rows: 32 lanes of kAcross vectors
    constexpr int kAcross = 8, kPart = 32 * kAcross, kParts = kAdSlice / VE / kPart;
    constexpr uint32_t kAll = (1u << VE) - 1;
    const int r0 = blockIdx.z * a.rows, r1 = min(r0 + a.rows, rows);
    const int last_word = (a.V - 1) >> 5;
    auto row_of = [&](int r) { return (int64_t)b * a.R + r; };
    auto in_of = [&](int r) { return static_cast<const T*>(a.in) + row_of(r) * a.in_stride + v0; };
    auto out_of = [&](int r) { return static_cast<T*>(a.out) + row_of(r) * a.out_stride + v0; };
    auto allowed_of = [&](int r) { return reinterpret_cast<const uint32_t*>(p.allowed) + row_of(r) * p.allowed_stride; };
    // a logit of row r, by what the history, the path and the biases say
    const uint32_t rare = q.divides ? 0xffffffffu : kAdDrafted | kAdBiased;
    auto adjusted = [&](float x, int at, uint32_t cell, int r) {
        if (!(cell & rare)) return adjust_value(x, cell, q);
        return adjust_rare(x, v0 + at, cell, cell & kAdBiased ? s.bias[adjust_cell<VE>(at)] : 0.0f, r, s.token, s.parent, q);
    };
    auto row_part = [&](int r, int part) {
        const T* in = in_of(r);
        T* out = out_of(r);
        const uint32_t* allowed = p.allowed ? allowed_of(r) + (v0 >> 5) : nullptr;  // of the slice
        const uint32_t skew = (uint32_t)reinterpret_cast<uintptr_t>(in) & 15u;
        // vectors lie on 16 bytes in both; where in and out differ in alignment there are none
        const bool same = skew == ((uint32_t)reinterpret_cast<uintptr_t>(out) & 15u);
        const int head = same ? min(width, (int)((16u - skew) & 15u) / (int)sizeof(T)) : width;
        const int vecs = (width - head) / VE, tail = head + vecs * VE;
        if (head | (width - tail)) {
            auto single = [&](int at) {
                if (allowed && !((allowed[at >> 5] >> (at & 31)) & 1u)) Logit<T>::store(out + at, -INFINITY);
                else if (dense) Logit<T>::store(out + at, adjust_packed(Logit<T>::load(in + at), s.cell[adjust_cell<VE>(at)], q));
                else out[at] = in[at];
            };
            for (int at = part * 32 + lane; at < head; at += 32 * kParts) single(at);
            if (part == kParts - 1 && lane < width - tail) single(tail + lane);
        }
        const int i0 = part * kPart + lane;
        const uint4* from = reinterpret_cast<const uint4*>(in + head) + i0;
        uint4* to = reinterpret_cast<uint4*>(out + head) + i0;
        uint4 x[kAcross];
        uint32_t ok[kAcross];
        if (allowed) {
            const int last = last_word - (v0 >> 5);
            uint32_t word[kAcross], next[kAcross];
#pragma unroll
            for (int u = 0; u < kAcross; ++u) {
                const int w = min((head + (i0 + u * 32) * VE) >> 5, last);
                word[u] = allowed[w];
                next[u] = head % VE ? allowed[min(w + 1, last)] : 0u;  // a vector may end in the next word
            }
#pragma unroll
            for (int u = 0; u < kAcross; ++u)
                ok[u] = i0 + u * 32 < vecs ? __funnelshift_r(word[u], next[u], (head + (i0 + u * 32) * VE) & 31) & kAll : 0u;
        } else {
#pragma unroll
            for (int u = 0; u < kAcross; ++u) ok[u] = i0 + u * 32 < vecs ? kAll : 0u;
        }
#pragma unroll
        for (int u = 0; u < kAcross; ++u)
            if (ok[u]) x[u] = from[u * 32];
        if (dense) {
#pragma unroll
            for (int u = 0; u < kAcross; ++u) {
                if (!ok[u]) continue;
                float y[VE];
                Logit<T>::get(x[u], y);
                const int at = head + (i0 + u * 32) * VE;
#pragma unroll
                for (int k = 0; k < VE; ++k) y[k] = adjust_packed(y[k], s.cell[adjust_cell<VE>(at + k)], q);
                x[u] = Logit<T>::put(y);
            }
        }
#pragma unroll
        for (int u = 0; u < kAcross; ++u) {
            if (i0 + u * 32 >= vecs) continue;
            if (ok[u] != kAll) Logit<T>::rule_out(x[u], ok[u]);
            to[u * 32] = x[u];
        }
    };
    const int histories = (told + kAdHistory - 1) / kAdHistory, parts = max(r1 - r0, 0) * kParts;
    auto draw = [&](int* counter) {
        int t = 0;
        if (lane == 0) t = atomicAdd(counter, 1);
        return __shfl_sync(0xffffffffu, t, 0);
    };
    for (int t; (t = draw(&sh_task)) < histories + (dense ? 0 : parts);) {
        if (t < histories) history(t);
        else row_part(r0 + (t - histories) / kParts, (t - histories) % kParts);
        __syncwarp();
    }
    if (err) set_error(a.dev_error, err);
    __syncthreads();  // the counts are whole; the rows are written, but for a dense request's
    if (!penalties && !p.bias_ids) return;
    if (p.bias_ids) {
        // of the slice's biases of one id the first adds them all up, in order
        const float* values = p.bias_values + (int64_t)b * p.bias_count;
        const int n = sh_entries;
        for (int i = tid; i < n; i += kAdNT) {
            const int2 e = s.entry[i];
            bool first = true, more = false;
            for (int k = 0; k < n; ++k)
                if (s.entry[k].x == e.x) {
                    first = first && s.entry[k].y >= e.y;
                    more = more || s.entry[k].y > e.y;
                }
            if (!first) continue;
            float sum = values[e.y];
            for (int last = e.y; more;) {
                int next = kAdMaxBias;
                for (int k = 0; k < n; ++k)
                    if (s.entry[k].x == e.x && s.entry[k].y > last) next = min(next, s.entry[k].y);
                more = next < kAdMaxBias;
                if (more) sum += values[next];
                last = next;
            }
            s.bias[adjust_cell<VE>(e.x)] = sum;
        }
    }
    // the list (a dense request's: the rare, which the stream leaves): a thread looks at four cells at a time
    const uint32_t listable = dense ? kAdDrafted | kAdBiased : 0xffffffffu;
    constexpr int kLooks = (kAdCells / 4 + kAdNT - 1) / kAdNT;
    uint32_t hits = 0;
#pragma unroll
    for (int k = 0; k < kLooks; ++k) {
        const int i = tid + k * kAdNT;
        if (i >= kAdCells / 4) continue;
        const uint4 c = reinterpret_cast<const uint4*>(s.cell)[i];
        hits |= (((c.x & listable) != 0) | ((c.y & listable) != 0) << 1 | ((c.z & listable) != 0) << 2 |
                 ((c.w & listable) != 0) << 3) << (4 * k);
    }
    const int mine = __popc(hits), upto = warp_inclusive_scan_i(mine);
    int to = 0;
    if (lane == 31) to = atomicAdd(&sh_listed, upto);
    to = __shfl_sync(0xffffffffu, to, 31) + upto - mine;
    for (; hits; hits &= hits - 1) {
        const int k = __ffs(hits) - 1, i = (tid + (k >> 2) * kAdNT) * 4 + (k & 3);
        if (dense) s.kept[to] = s.cell[i];
        s.list[to++] = (uint16_t)adjust_place<VE>(i);
    }
    if (dense) {
        // this thread's cells become what the stream takes off
#pragma unroll
        for (int k = 0; k < kLooks; ++k) {
            const int i = tid + k * kAdNT;
            if (i >= kAdCells / 4) continue;
            const uint4 c = reinterpret_cast<const uint4*>(s.cell)[i];
            auto pack = [&](uint32_t cell) { return cell & listable ? 0u : adjust_pack(cell, q); };
            reinterpret_cast<uint4*>(s.cell)[i] = make_uint4(pack(c.x), pack(c.y), pack(c.z), pack(c.w));
        }
        __syncthreads();
        for (int t; (t = draw(&sh_part)) < parts;) {
            row_part(r0 + t / kParts, t % kParts);
            __syncwarp();
        }
    }
    __syncthreads();
    // a thread has every `places`-th listed token, in every `phases`-th row
    const int listed = sh_listed;
    int places = kAdNT;
    while (places / 2 >= listed && places > 8) places /= 2;
    const int phases = kAdNT / places, phase = tid / places;
    for (int i = tid - phase * places; i < listed; i += places) {
        const int at = s.list[i], v = v0 + at;
        const uint32_t cell = dense ? s.kept[i] : s.cell[adjust_cell<VE>(at)];
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
            for (int k = 0; k < kAdFixes; ++k)
                if (live[k]) Logit<T>::store(out + k * out_step, adjusted(x[k], at, cell, r + k * phases));
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
    // Rows of a request are shared out only where its slices do not fill the GPU.  Each CTA counts the history again:
    // 12 requests of 60 rows took 152 us in one wave, 99 in two, 104 in three, 109 in four.
    const long long want = (long long)shape.sms * shape.per_sm, have = (long long)slices * B;
    int parts = (int)(have >= want ? 1 : kAdWaves * want / have);
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
        (p.bias_ids && p.bias_count > kAdMaxBias) || (p.history && p.history_capacity > kAdMaxHistory))
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
