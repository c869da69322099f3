// Log probabilities of given tokens with the entropy and the top
// alternatives of their rows (spec_token_logprobs): what is reported beside
// the tokens a verification emits, and what a target hands to the training
// of its draft.
//
// One read of a row.  A row's 16-byte vectors are taken a warp's width at a
// time: 32 vectors side by side are a group (256 bf16 or 128 fp32 elements),
// and the unaligned head and tail of a row are the first and the last group.
// Per group a warp takes the maximum (one reduction instruction) and, against
// its own running maximum m, z = sum 2^t and e = sum t 2^t of t = (x - m) c,
// c = log2(e) / T.  From the merged sums
//     log p(v) = (x_v - m) / T - ln z,    entropy = ln z - ln 2 * e / z.
// The group maxima are what makes the alternatives cheap: groups are
// contiguous, so in the order (logit descending, index ascending) every
// element of a group comes after that group's first maximum, and the K best
// elements lie in the K best groups.  Only those are read again (from L2).
#include "cluster.cuh"
#include "vocab_rows.cuh"

namespace sv {

struct LogprobArgs {
    const void* logits;
    int R, V, top_k;
    int64_t stride;
    const int32_t* tokens;
    float c;
    float2 inv_t;  // 1 / T in two parts
    float* logprob;
    int32_t* rank;
    float* entropy;
    int32_t* top_ids;
    float* top_logprobs;
    int32_t* dev_error;
};

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpTile = 6;   // groups of a tile: 3 KiB
constexpr int kLpDepth = 2;  // tiles a warp has on their way
constexpr int kLpTileBytes = kLpTile * 512;
constexpr int kLpRing = kLpWarps * kLpDepth * kLpTileBytes;
constexpr int kLpMaxCluster = 8;
constexpr uint64_t kLpLimitNs = 2000000000ull;
constexpr float kLpPlain = 1024.0f;  // |m c| below this: see LpSums
constexpr float kLpLeastC = 1e-30f;  // so that m - kLpFar / c stays in range
constexpr float kLpFar = 200.0f;     // 2^-200 is zero
// The K-th best group need not be found exactly: any bound that leaves K to
// K + kLpSlack groups will do.
constexpr int kLpSlack = 36;
constexpr int kLpCands = 8 * (kMaxTop + kLpSlack);  // the elements of that many vectors
constexpr int kLpBins = 256;        // of the groups' keys, from the largest down
constexpr int kLpBinShift = 17;     // two bf16 values a bin: four binades in all
static_assert(kLpCands * 8 <= kLpRing, "the candidates take the ring's place");

// What a warp makes of its groups.
struct __align__(16) LpPart {
    float m, z, e;
    int before;
};
static_assert(sizeof(LpPart) == 16 && alignof(LpPart) == 16, "sent to the leader as one 16-byte store");

// The groups of a row: 0 is its head, 1 .. nb the vectors, nb + 1 its tail.
template <typename T>
struct LpRow : RowView<T> {
    int nb;
    __device__ __forceinline__ LpRow(const T* r, int v) : RowView<T>(r, v), nb((this->nvec + 31) / 32) {}
    // This lane's element of the head and of the tail (-inf: none).
    __device__ __forceinline__ float2 ends() const {
        const int lane = threadIdx.x & 31;
        float2 e = make_float2(-INFINITY, -INFINITY);
        if (lane < this->head) e.x = ElemT<T>::load(this->row + lane);
        if (lane < this->tail) e.y = ElemT<T>::load(this->row + this->head + this->nvec * ElemT<T>::VEC + lane);
        return e;
    }
    // This lane's elements of group g: a vector (an end's single element
    // first, the rest -inf), how many there are, the index of the first.
    __device__ __forceinline__ uint4 vector(int g) const {
        const int lane = threadIdx.x & 31;
        uint4 q = RowVec<T>::none();
        if (g >= 1 && g <= nb) {
            const int v = (g - 1) * 32 + lane;
            if (v < this->nvec) q = __ldg(this->vec() + v);
        } else if (lane < (g == 0 ? this->head : this->tail)) {
            q.x = RowVec<T>::single(ElemT<T>::load(this->row + index(g)));
        }
        return q;
    }
    __device__ __forceinline__ int count(int g) const {
        const int lane = threadIdx.x & 31;
        if (g >= 1 && g <= nb) return (g - 1) * 32 + lane < this->nvec ? ElemT<T>::VEC : 0;
        return lane < (g == 0 ? this->head : this->tail) ? 1 : 0;
    }
    __device__ __forceinline__ int index(int g) const {
        const int lane = threadIdx.x & 31;
        if (g >= 1 && g <= nb) return this->head + ((g - 1) * 32 + lane) * ElemT<T>::VEC;
        return (g == 0 ? 0 : this->head + this->nvec * ElemT<T>::VEC) + lane;
    }
};

// A row that gets no result: skipped, or refused (logprob -inf).  Thread
// tid of n.
__device__ __forceinline__ void lp_no_result(const LogprobArgs& a, int r, float logprob, int tid, int n) {
    if (tid == 0) {
        if (a.logprob) a.logprob[r] = logprob;
        if (a.rank) a.rank[r] = -1;
        if (a.entropy) a.entropy[r] = 0.0f;
    }
    for (int j = tid; j < a.top_k; j += n) {
        a.top_ids[(size_t)r * a.top_k + j] = -1;
        a.top_logprobs[(size_t)r * a.top_k + j] = -INFINITY;
    }
}

// Running sums of a lane against the warp's reference m.  Where m c is of
// ordinary size (a masked row's lowest values, a huge or tiny temperature
// are not) t = x c - mc is one fused operation, mc = m c rounded: every term
// has the same reference, and what mc is off by is taken out at the end.
struct LpSums {
    float m = kNoMax, mc = 0.0f;
    bool plain = false;  // t = x c - mc; otherwise t = (x - m) c
    float2 z = make_float2(0.0f, 0.0f), e = make_float2(0.0f, 0.0f);
    __device__ __forceinline__ void shift(float d) {  // every t moves by d
        d = fmaxf(d, -1000.0f);  // any distance whose weight is zero
        const float f = ex2(d);
        e = make_float2((e.x + z.x * d) * f, (e.y + z.y * d) * f);
        z = make_float2(z.x * f, z.y * f);
    }
    __device__ __forceinline__ void raise(float m2, float c) {  // to a higher reference
        exact(c);
        shift((m - m2) * c);
        m = m2;
        settle(c);
    }
    __device__ __forceinline__ void settle(float c) {
        mc = m * c;
        plain = fabsf(mc) < kLpPlain && c > kLpLeastC;
        if (plain) shift(fmaf(m, c, -mc));
    }
    __device__ __forceinline__ void exact(float c) {  // back to the reference m itself
        if (plain) shift(fmaf(-m, c, mc));
        plain = false;
    }
    __device__ __forceinline__ void add(float2 t, float2 t_e) {
        const float2 w = make_float2(ex2(t.x), ex2(t.y));
        z = __fadd2_rn(z, w);
        e = __ffma2_rn(w, t_e, e);
    }
    // values at least kLpFar / c below m add nothing, and -inf has no product with 0
    __device__ __forceinline__ void add_plain(float2 x, float2 cc, float2 nmc) {
        const float2 t = __ffma2_rn(x, cc, nmc);
        add(t, t);
    }
    __device__ __forceinline__ void add_any(float2 x, float2 cc) {
        const float2 t = __fmul2_rn(__fadd2_rn(x, make_float2(-m, -m)), cc);
        add(t, make_float2(fmaxf(t.x, -1000.0f), fmaxf(t.y, -1000.0f)));  // a NaN still shows in z
    }
};

// A bound above which K .. K + slack keys lie, or, where many keys are
// equal, the K-th largest key itself (then fewer than K lie above it).
// count(b) is the number of keys >= b; K or more are >= lo (or there are
// fewer than K), fewer than K are above hi.  Steps of growing width down from hi (the
// first is half a binade), then halves.
__device__ __forceinline__ int lp_slack(int K) { return min(kLpSlack, 4 + K / 4); }
template <typename F>
__device__ __forceinline__ uint32_t lp_bound(uint32_t lo, uint32_t hi, int K, F&& count) {
    const int slack = lp_slack(K);
    uint32_t step = 1u << 22;
    while (lo < hi) {
        const uint32_t mid = hi - lo > 2 * step ? hi - step : lo + (hi - lo) / 2 + 1;
        const int n = count(mid);
        if (n < K) {
            hi = mid - 1;
            step = step < (1u << 29) ? 4 * step : step;
        } else if (n <= K + slack) {
            return mid - 1;
        } else {
            lo = mid;
        }
    }
    return lo;
}

// What decides an element's place before the token: above xt, or equal to it
// and of a lower index.  In the groups before the token's own that is one
// comparison with the next value below xt.
template <typename T>
struct LpToken {
    float x;
    int tok, group;  // the token's group
    typename RowVec<T>::Least above, reach;
    __device__ __forceinline__ LpToken(const LpRow<T>& row, int t, float xt) : x(xt), tok(t) {
        constexpr int VEC = ElemT<T>::VEC;
        group = t < row.head ? 0 : t < row.head + row.nvec * VEC ? 1 + (t - row.head) / (32 * VEC) : row.nb + 1;
        above = RowVec<T>::least(xt);
        reach = RowVec<T>::least(next_below<T>(xt));
    }
    __device__ __forceinline__ int before(float v, int idx) const { return v > x || (v == x && idx < tok); }
};

// A tile of groups g0 .. g0 + kLpTile - 1: this lane's vector of each.
template <typename T>
struct LpTile {
    using Vec = RowVec<T>;
    uint4 q[kLpTile];
    float mine;  // lane j: the maximum of group j
    float most;
    __device__ __forceinline__ void maxima() {
        mine = most = -INFINITY;
#pragma unroll
        for (int j = 0; j < kLpTile; ++j) {
            const float gm = warp_max_redux(Vec::max(q[j]));
            most = fmaxf(most, gm);
            if ((threadIdx.x & 31) == j) mine = gm;
        }
    }
    // Elements before the token.
    __device__ __forceinline__ int before(const LpToken<T>& tk, const LpRow<T>& row, int g0) const {
        if (most < tk.x) return 0;
        const int at = tk.group - g0;  // the token's group among the tile's
        if (at < 0 || at >= kLpTile) {
            const typename Vec::Least bound = at < 0 ? tk.above : tk.reach;
            typename Vec::Count n = Vec::count_zero();
#pragma unroll
            for (int j = 0; j < kLpTile; ++j) Vec::count(n, q[j], bound);
            return Vec::count_sum(n);
        }
        int n = 0;
#pragma unroll
        for (int j = 0; j < kLpTile; ++j) {
            if (j != at) {
                typename Vec::Count k = Vec::count_zero();
                Vec::count(k, q[j], j < at ? tk.reach : tk.above);
                n += Vec::count_sum(k);
            } else {
                const int idx = row.head + ((g0 - 1 + j) * 32 + (threadIdx.x & 31)) * ElemT<T>::VEC;
#pragma unroll
                for (int i = 0; i < Vec::kPairs; ++i) {
                    const float2 x = Vec::pair(q[j], i);
                    n += tk.before(x.x, idx + 2 * i) + tk.before(x.y, idx + 2 * i + 1);
                }
            }
        }
        return n;
    }
    __device__ __forceinline__ void add(LpSums& sum, float c, float far) const {
        const float2 cc = make_float2(c, c), nmc = make_float2(-sum.mc, -sum.mc);
        const typename Vec::Least least = Vec::least(sum.m - far);
        if (sum.plain) {
#pragma unroll
            for (int j = 0; j < kLpTile; ++j) {
#pragma unroll
                for (int i = 0; i < Vec::kPairs; ++i) sum.add_plain(Vec::pair_above(q[j], i, least), cc, nmc);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kLpTile; ++j) {
#pragma unroll
                for (int i = 0; i < Vec::kPairs; ++i) sum.add_any(Vec::pair(q[j], i), cc);
            }
        }
    }
};

// A warp's part of a row.
__device__ __forceinline__ LpPart lp_part(LpSums& sum, int before, float c) {
    sum.exact(c);
    LpPart p;
    p.m = sum.m;
    p.z = sum.z.x + sum.z.y;
    p.e = sum.e.x + sum.e.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        p.z += __shfl_xor_sync(0xffffffffu, p.z, o);
        p.e += __shfl_xor_sync(0xffffffffu, p.e, o);
    }
    p.before = __reduce_add_sync(0xffffffffu, before);
    return p;
}

// Shared memory of the CTA that finishes a row.
struct LpFinish {
    static constexpr int kGroups = 256;               // at most this many groups are read again
    static constexpr int kHeld = kGroups / kLpWarps;  // vectors a lane compares of them
    int group[kGroups];  // the groups that hold the alternatives
    int ties[kGroups];   // elements equal to tau in each, then how many come before it
    int bin[kLpBins];
    int count[2][kLpWarps];
    int n_group, n_cand;
    uint32_t tau;  // order key: elements above it are candidates
    float m;
    float2 ln_z;  // in two parts
    int valid;
};

// d / T - ln z: with both constants in two parts, one rounding.
__device__ __forceinline__ float lp_log(const LogprobArgs& a, float d, float2 ln_z) {
    const float lp = fmaf(d, a.inv_t.x, -ln_z.x);
    return lp > -INFINITY ? lp + fmaf(d, a.inv_t.y, -ln_z.y) : lp;
}

// One warp: the row's sums from its parts and its ends, and the results that
// need no alternatives.
template <typename T>
__device__ __forceinline__ void lp_merge(const LogprobArgs& a, int r, const LpRow<T>& row, int tok, float xt,
                                         float2 ends, LpFinish& s, const LpPart* parts, int n_parts) {
    constexpr int VEC = ElemT<T>::VEC;
    const int lane = threadIdx.x & 31;
    LpPart p[2];
    float m = fmaxf(ends.x, ends.y);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        p[k] = lane + 32 * k < n_parts ? parts[lane + 32 * k] : LpPart{kNoMax, 0.0f, 0.0f, 0};
        m = fmaxf(m, p[k].m);
    }
    m = warp_max_redux(m);
    float z = 0.0f, e = 0.0f;
    int before = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float d = fmaxf((p[k].m - m) * a.c, -1000.0f), f = ex2(d);
        z += p[k].z * f;
        e += (p[k].e + p[k].z * d) * f;
        before += p[k].before;
    }
    auto end = [&](float x, int idx) {
        const float t = (x - m) * a.c, w = ex2(t);
        z += w;
        e = fmaf(w, fmaxf(t, -1000.0f), e);
        before += x > xt || (x == xt && idx < tok);
    };
    if (lane < row.head) end(ends.x, lane);
    if (lane < row.tail) end(ends.y, row.head + row.nvec * VEC + lane);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, o);
        e += __shfl_xor_sync(0xffffffffu, e, o);
    }
    before = __reduce_add_sync(0xffffffffu, before);
    // nothing is below -inf: every place of the groups before the token's
    // was counted, the empty ones of the last group too
    if (xt == -INFINITY && tok >= row.head + row.nvec * VEC) before -= (row.nb * 32 - row.nvec) * VEC;
    const bool valid = z > 0.0f && z < INFINITY;  // no NaN, no +inf, something finite
    if (lane == 0) {
        const float2 ln_z = ln_parts(z);
        s.m = m;
        s.ln_z = ln_z;
        s.valid = valid;
        if (valid) {
            if (a.logprob) a.logprob[r] = a.tokens ? lp_log(a, xt - m, ln_z) : 0.0f;
            if (a.rank) a.rank[r] = a.tokens ? before + 1 : -1;
            if (a.entropy) a.entropy[r] = fmaf(-kLn2, e / z, ln_z.x) + ln_z.y;
        } else if (a.dev_error) {
            atomicOr(a.dev_error, kDevErrNonfinite);
        }
    }
}

// The row's results, from n_parts <= 64 parts and the order keys of the
// maxima of its groups (group_key[g], 1 <= g <= nb; room for 0 and nb + 1).
// ends: this lane's element of the head and of the tail.
template <typename T>
__device__ __forceinline__ void lp_finish(const LogprobArgs& a, int r, const LpRow<T>& row, int tok, float xt,
                                          float2 ends, LpFinish& s, uint64_t* cand, uint32_t* group_key,
                                          const LpPart* parts, int n_parts) {
    using Vec = RowVec<T>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_groups = row.nb + 2;
    const bool all = n_groups <= LpFinish::kGroups;
    uint32_t top;  // the largest key
    {
        const float head_max = warp_max_redux(ends.x), tail_max = warp_max_redux(ends.y);
        float m = fmaxf(head_max, tail_max);
        for (int k = lane; k < n_parts; k += 32) m = fmaxf(m, parts[k].m);
        top = okey32(warp_max_redux(m));
        if (warp == 0 && lane == 0) {  // an empty head or tail has no key (-inf has one)
            group_key[0] = row.head ? okey32(head_max) : 0u;
            group_key[row.nb + 1] = row.tail ? okey32(tail_max) : 0u;
        }
        if (a.top_k > 0) {
            for (int i = tid; i < kLpBins; i += kLpThreads) s.bin[i] = 0;
            __syncthreads();
        }
    }
    if (a.top_k > 0) {
        // Where the K-th best group lies: the groups' keys counted in bins
        // from the largest down.  Few groups: all of them, and the bound is
        // found among their vectors.
        if (!all) {
            for (int g = tid; g < n_groups; g += kLpThreads) {
                const uint32_t k = group_key[g], bin = (top - k) >> kLpBinShift;
                if (k != 0u && bin < kLpBins) atomicAdd(&s.bin[bin], 1);
            }
            __syncthreads();
        }
        if (all) {
            for (int g = tid; g < n_groups; g += kLpThreads) s.group[g] = g;
            if (tid == 0) {
                s.tau = 0u;
                s.n_group = n_groups;
                s.n_cand = 0;
            }
        } else if (warp == 0) {
            uint32_t tau;
            int n_above = 0;
            {
                auto count = [&](uint32_t b) {
                    int n = 0;
                    for (int g = lane; g < n_groups; g += 32) n += group_key[g] >= b;
                    return __reduce_add_sync(0xffffffffu, n);
                };
                constexpr int kEach = kLpBins / 32;
                int n[kEach], sum = 0;
#pragma unroll
                for (int i = 0; i < kEach; ++i) sum += n[i] = s.bin[lane * kEach + i];
                const int incl = warp_inclusive_scan_i(sum);
                int at = incl - sum, bin = kLpBins;  // the first bin by whose end K groups are counted
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    if (at < a.top_k && at + n[i] >= a.top_k) {
                        bin = lane * kEach + i;
                        n_above = at + n[i];
                    }
                    at += n[i];
                }
                bin = warp_min_i(bin);
                n_above = __reduce_max_sync(0xffffffffu, n_above);
                const uint32_t hi = top - ((uint32_t)min(bin, kLpBins - 1) << kLpBinShift);
                if (bin == kLpBins)  // below the bins
                    tau = lp_bound(0u, hi, a.top_k, count);
                else if (n_above > a.top_k + lp_slack(a.top_k))  // many in that bin
                    tau = lp_bound(hi - ((1u << kLpBinShift) - 1u), hi, a.top_k, count);
                else
                    tau = hi - (1u << kLpBinShift);
                if (bin == kLpBins || n_above > a.top_k + lp_slack(a.top_k)) n_above = count(tau + 1);
                // fewer than K above tau: also the first that reach it
                if (n_above < a.top_k) {
                    int n_list = 0, equal = a.top_k - n_above;
                    const uint32_t lower = (1u << lane) - 1u;
                    for (int g0 = 0; g0 < n_groups; g0 += 32) {
                        const uint32_t k = g0 + lane < n_groups ? group_key[g0 + lane] : 0u;
                        const uint32_t same = __ballot_sync(0xffffffffu, k == tau);
                        const uint32_t taken =
                            __ballot_sync(0xffffffffu, k > tau || (k == tau && __popc(same & lower) < equal));
                        equal -= __popc(same);
                        const int place = n_list + __popc(taken & lower);
                        if (((taken >> lane) & 1u) && place < LpFinish::kGroups) s.group[place] = g0 + lane;
                        n_list += __popc(taken);
                    }
                    n_above = -n_list;  // the list is made
                }
            }
            if (lane == 0) {
                s.tau = tau;
                s.n_group = n_above < 0 ? -n_above : 0;
                s.n_cand = 0;
            }
        }
    }
    if (warp == 1) lp_merge<T>(a, r, row, tok, xt, ends, s, parts, n_parts);
    if (a.top_k > 0 && !all) {
        __syncthreads();
        if (s.n_group == 0) {  // every group above tau
            const uint32_t tau = s.tau;
            __syncthreads();  // all have seen the empty list
            for (int g = tid; g < n_groups; g += kLpThreads)
                if (group_key[g] > tau) {
                    const int at = atomicAdd(&s.n_group, 1);
                    if (at < LpFinish::kGroups) s.group[at] = g;  // more only in a row of NaN, refused below
                }
        }
    }
    __syncthreads();
    if (!s.valid) {
        lp_no_result(a, r, a.tokens ? -INFINITY : 0.0f, tid, kLpThreads);
        return;
    }
    if (a.top_k == 0) return;

    // --------------------------- the alternatives, from the chosen groups
    const int n_group = s.n_group;
    // f(i) for the vectors of the chosen groups whose maximum is such that
    // hit(maximum): read many at a time (under load a read takes 1 to 2 us),
    // and the few hits once more, in code that is not repeated per vector
    // (what a row runs once has to be fetched, too).
    constexpr int kAhead = 8;
    auto for_hits = [&](auto&& hit, auto&& f) {
        for (int i0 = warp; i0 < n_group; i0 += kAhead * kLpWarps) {
            uint4 q[kAhead];
            uint32_t hits = 0;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + k * kLpWarps;
                q[k] = i < n_group ? row.vector(s.group[i]) : Vec::none();
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i0 + k * kLpWarps < n_group && hit(Vec::max(q[k]))) hits |= 1u << k;
            while (hits) {
                const int i = i0 + (__ffs(hits) - 1) * kLpWarps;
                hits &= hits - 1;
                f(i);
            }
        }
    };
    // The bound of the groups leaves little more than K elements, unless the
    // row has few groups or its best elements share some (a sorted row).
    // Then the bound is raised to one that leaves about K vectors.
    bool raise = all;
    float bound;
    for (;;) {
        if (raise) {
            uint32_t held[LpFinish::kHeld];  // this lane's vectors: their maxima
#pragma unroll
            for (int k0 = 0; k0 < LpFinish::kHeld; k0 += 4) {
                uint4 q[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = warp + (k0 + k) * kLpWarps;
                    q[k] = i < n_group ? row.vector(s.group[i]) : Vec::none();
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = warp + (k0 + k) * kLpWarps;
                    held[k0 + k] = i < n_group && row.count(s.group[i]) ? okey32(Vec::max(q[k])) : 0u;
                }
            }
            int turn = 0;
            const uint32_t tau = lp_bound(s.tau, top, a.top_k, [&](uint32_t b) {
                int n = 0;
#pragma unroll
                for (int k = 0; k < LpFinish::kHeld; ++k) n += held[k] >= b;
                n = __reduce_add_sync(0xffffffffu, n);
                turn ^= 1;  // the other half: its readers have passed a barrier since
                if (lane == 0) s.count[turn][warp] = n;
                __syncthreads();
                n = 0;
#pragma unroll
                for (int w = 0; w < kLpWarps; ++w) n += s.count[turn][w];
                return n;
            });
            __syncthreads();
            if (tid == 0) {
                s.tau = tau;
                s.n_cand = 0;
            }
            __syncthreads();
        }
        // As a float: the key below zero's is -0, which compares equal to
        // zero; key 0 is a NaN, which nothing is <= to.
        bound = s.tau == 0x7fffffffu ? __uint_as_float(0x80000001u) : okey32_to_float(s.tau);
        for_hits([&](float m) { return !(m <= bound); },
                 [&](int i) {
                     const int g = s.group[i], n = row.count(g), idx = row.index(g);
#pragma unroll 1
                     for (int j = 0; j < n; ++j) {
                         const float x = ElemT<T>::load(row.row + idx + j);
                         if (x <= bound) continue;
                         const int at = atomicAdd(&s.n_cand, 1);
                         if (at < kLpCands) cand[at] = order_key(x, idx + j);
                     }
                 });
        __syncthreads();
        if (s.n_cand <= kLpCands || raise) break;
        raise = true;
    }
    int n_cand = s.n_cand;
    if (n_cand < a.top_k) {  // and the first elements equal to tau, in the order of their groups
        const int need = a.top_k - n_cand;
        auto ties_of = [&](int g) {
            const int n = row.count(g), idx = row.index(g);
            int ties = 0;
#pragma unroll 1
            for (int j = 0; j < n; ++j) ties += ElemT<T>::load(row.row + idx + j) == bound;
            return ties;
        };
#pragma unroll 1
        for (int i = warp; i < n_group; i += kLpWarps) {
            const int ties = __reduce_add_sync(0xffffffffu, ties_of(s.group[i]));
            if (lane == 0) s.ties[i] = ties;
        }
        __syncthreads();
        int earlier = 0, mine = 0;
        if (tid < n_group) {
            mine = s.ties[tid];
            for (int j = 0; j < n_group; ++j) earlier += s.group[j] < s.group[tid] ? s.ties[j] : 0;
        }
        __syncthreads();
        if (tid < n_group) s.ties[tid] = mine > 0 ? earlier : need;
        __syncthreads();
        for (int i = warp; i < n_group; i += kLpWarps) {
            if (s.ties[i] >= need) continue;  // none here, or none still wanted
            const int g = s.group[i], n = row.count(g), idx = row.index(g), ties = ties_of(g);
            int at = s.ties[i] + warp_inclusive_scan_i(ties) - ties;
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                const float x = ElemT<T>::load(row.row + idx + j);
                if (x != bound) continue;
                if (at < need) cand[n_cand + at] = order_key(x, idx + j);
                ++at;
            }
        }
        __syncthreads();
        n_cand = a.top_k;
    }
    // a candidate's place is the number of candidates before it
    for (int i = tid; i < n_cand; i += kLpThreads) {
        const uint64_t k = cand[i];
        int place = 0;
#pragma unroll 4
        for (int j = 0; j < n_cand; ++j) place += cand[j] > k;
        if (place < a.top_k) {
            a.top_ids[(size_t)r * a.top_k + place] = key_index(k);
            a.top_logprobs[(size_t)r * a.top_k + place] = lp_log(a, key_value(k) - s.m, s.ln_z);
        }
    }
}

template <typename T, bool CLUSTER>
__global__ void __launch_bounds__(kLpThreads, 4) k_token_logprobs(LogprobArgs a) {
    __shared__ LpFinish s;
    __shared__ LpPart parts[kLpMaxCluster * kLpWarps];
    __shared__ uint64_t full[kLpWarps][kLpDepth];
    extern __shared__ __align__(128) uint8_t lp_raw[];
    uint32_t* group_key = reinterpret_cast<uint32_t*>(lp_raw + kLpRing);  // [nb + 2]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = CLUSTER ? (int)cluster_size() : 1, part = CLUSTER ? (int)cluster_rank() : 0;
    const int r = blockIdx.x / S;
    const int tok = a.tokens ? a.tokens[r] : 0;
    if (tok < 0 || tok >= a.V) {
        if (part == 0) {
            if (tok != -1 && tid == 0 && a.dev_error) atomicOr(a.dev_error, kDevErrToken);
            lp_no_result(a, r, tok == -1 ? 0.0f : -INFINITY, tid, kLpThreads);
        }
        return;
    }
    if (CLUSTER) cluster_arrive();  // awaited before the first store into the leader
    const LpRow<T> row(static_cast<const T*>(a.logits) + (size_t)r * a.stride, a.V);

    // This warp's tiles, kLpDepth of them on their way through its part of
    // the ring: what is in flight does not take registers, and is enough
    // when another CTA of the SM is at its row's end.
    uint4* ring = reinterpret_cast<uint4*>(lp_raw) + warp * (kLpRing / 16 / kLpWarps);
    uint64_t* bars = full[warp];
    const uint4* vecs = row.vec();
    const int step = S * kLpWarps * kLpTile;
    int g0 = (part * kLpWarps + warp) * kLpTile;
    auto copy = [&](int g, int slot) {  // lane 0
        const uint32_t bytes = (uint32_t)min(kLpTile * 32, row.nvec - g * 32) * 16;
        mbar_arrive_expect_tx(&bars[slot], bytes);
        bulk_load(ring + slot * (kLpTileBytes / 16), vecs + (size_t)g * 32, bytes, &bars[slot]);
    };
    if (lane == 0) {
        for (int i = 0; i < kLpDepth; ++i) mbar_init(&bars[i], 1);
        mbar_fence_init();
        for (int i = 0; i < kLpDepth; ++i)
            if (g0 + i * step < row.nb) copy(g0 + i * step, i);
    }
    __syncwarp();
    const float xt = ElemT<T>::load(row.row + tok);
    const float2 ends = row.ends();
    const LpToken<T> tk(row, tok, xt);
    const float far = kLpFar / a.c;
    LpSums sum;
    LpTile<T> tile;
    int before = 0, slot = 0;
    uint32_t parity = 0;
    bool awaited = false, ok = true;
    for (; g0 < row.nb; g0 += step) {
        ok = mbar_wait(&bars[slot], parity, kLpLimitNs);
        if (!ok) break;
        const uint4* at = ring + slot * (kLpTileBytes / 16) + lane;
        if ((g0 + kLpTile) * 32 <= row.nvec) {
#pragma unroll
            for (int j = 0; j < kLpTile; ++j) tile.q[j] = at[j * 32];
        } else {
#pragma unroll
            for (int j = 0; j < kLpTile; ++j)
                tile.q[j] = (g0 + j) * 32 + lane < row.nvec ? at[j * 32] : RowVec<T>::none();
        }
        __syncwarp();  // every lane has its vectors: the slot takes the next tile
        if (lane == 0 && g0 + kLpDepth * step < row.nb) copy(g0 + kLpDepth * step, slot);
        if (++slot == kLpDepth) {
            slot = 0;
            parity ^= 1;
        }
        tile.maxima();
        if (tile.most > sum.m) sum.raise(tile.most, a.c);
        if (CLUSTER && !awaited) {
            cluster_wait();
            awaited = true;
        }
        if (lane < kLpTile && g0 + lane < row.nb) {
            const uint32_t k = okey32(tile.mine);
            if (CLUSTER)
                cluster_store(cluster_map(group_key + g0 + lane + 1, 0), __uint_as_float(k));
            else
                group_key[g0 + lane + 1] = k;
        }
        before += tile.before(tk, row, g0 + 1);
        tile.add(sum, a.c, far);
    }
    LpPart p = lp_part(sum, before, a.c);
    if (!ok) {  // the row is refused; the copies still on their way land before the CTA ends
        p.z = NAN;
        if (lane == 0) {
            if (a.dev_error) atomicOr(a.dev_error, kDevErrTimeout);
            for (int i = 0; i < kLpDepth && g0 + i * step < row.nb; ++i) {
                mbar_wait(&bars[slot], parity, kLpLimitNs);
                if (++slot == kLpDepth) {
                    slot = 0;
                    parity ^= 1;
                }
            }
        }
        __syncwarp();
    }
    if (CLUSTER) {
        if (!awaited) cluster_wait();
        if (lane == 0)
            cluster_store(cluster_map(&parts[part * kLpWarps + warp], 0),
                          make_float4(p.m, p.z, p.e, __int_as_float(p.before)));
        cluster_arrive();
        cluster_wait();
        if (part != 0) return;
    } else {
        if (lane == 0) parts[warp] = p;
        __syncthreads();
    }
    lp_finish<T>(a, r, row, tok, xt, ends, s, reinterpret_cast<uint64_t*>(lp_raw), group_key, parts, S * kLpWarps);
}

// CTAs that share a row: as many as keep every SM busy when rows are few,
// each with a tile for every warp.
template <typename T>
static cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t st) {
    const int groups = (a.V / ElemT<T>::VEC + 31) / 32;
    const size_t dyn = kLpRing + (size_t)(groups + 2) * sizeof(uint32_t);
    constexpr int kMostGroups = (int)((kRowsMaxVocab / 4 + 31) / 32);
    constexpr size_t kMost = kLpRing + (kMostGroups + 2) * sizeof(uint32_t);
    LaunchShape shape;
    if (!launch_shape(reinterpret_cast<const void*>(k_token_logprobs<T, false>), kMost, kLpThreads, &shape) ||
        !launch_shape(reinterpret_cast<const void*>(k_token_logprobs<T, true>), kMost, kLpThreads, &shape))
        return cudaErrorUnknown;
    int S = 1;
    while (S < kLpMaxCluster && (long long)a.R * S < 2 * shape.sms && groups >= 2 * S * kLpWarps * kLpTile) S *= 2;
    if (S == 1) {
        k_token_logprobs<T, false><<<a.R, kLpThreads, dyn, st>>>(a);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.R * S);
    cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = dyn;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = S;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_token_logprobs<T, true>, a);
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
    const double inv_t = 1.0 / (double)temperature;
    const float inv_hi = (float)inv_t;
    LogprobArgs a{logits, R, V, top_k, row_stride, tokens, (float)(kLog2e / (double)temperature),
                  make_float2(inv_hi, (float)(inv_t - (double)inv_hi)), logprob, rank, entropy, top_ids, top_logprobs,
                  dev_error};
    return (dtype == SPEC_BF16 ? launch_logprobs<__nv_bfloat16>(a, st) : launch_logprobs<float>(a, st)) == cudaSuccess
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}
