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
    double inv_t;
    float* logprob;
    int32_t* rank;
    float* entropy;
    int32_t* top_ids;
    float* top_logprobs;
    int32_t* dev_error;
};

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpMaxCluster = 8;
constexpr float kLpPlain = 1024.0f;  // |m c| below this: see LpSums
constexpr float kLpLeastC = 1e-30f;  // so that m - kLpFar / c stays in range
constexpr float kLpFar = 200.0f;     // 2^-200 is zero
constexpr int kLpTile = 8;  // groups a warp has in flight: 4 KiB
// The K-th best group need not be found exactly: any bound that leaves K to
// K + kLpSlack groups will do.
constexpr int kLpSlack = 36;
constexpr int kLpGroups = 256;  // at most this many groups are read again
constexpr int kLpHeld = kLpGroups / kLpWarps;
constexpr int kLpCands = 8 * (kMaxTop + kLpSlack);  // the elements of that many vectors

// What a warp makes of its groups.
struct LpPart {
    float m, z, e;
    int before;
};
static_assert(sizeof(LpPart) == 16, "sent to the leader as one 16-byte store");

struct LpSmem {
    LpPart part[kLpMaxCluster * kLpWarps];
    uint64_t cand[kLpCands];
    int group[kLpGroups];  // the groups that hold the alternatives, in index order
    int ties[kLpGroups];   // elements equal to tau in each, then how many come before it
    int count[2][kLpWarps];
    int n_group, n_cand;
    uint32_t tau;          // order key: elements above it are candidates
    uint32_t top;          // the largest key
    float m, ln_z_hi, ln_z_lo;
    int valid;
};

// The groups of a row: 0 is its head, 1 .. nb the vectors, nb + 1 its tail.
template <typename T>
struct LpRow : RowView<T> {
    int nb;
    __device__ __forceinline__ LpRow(const T* r, int v) : RowView<T>(r, v), nb((this->nvec + 31) / 32) {}
    // This lane's elements of group g: values, index of the first, how many.
    __device__ __forceinline__ int load(int g, float* x, int& idx) const {
        constexpr int VEC = ElemT<T>::VEC;
        const int lane = threadIdx.x & 31;
        if (g >= 1 && g <= nb) {
            const int v = (g - 1) * 32 + lane;
            idx = this->head + v * VEC;
            if (v >= this->nvec) return 0;
            ElemT<T>::unpack(__ldg(this->vec() + v), x);
            return VEC;
        }
        const int n = g == 0 ? this->head : this->tail;
        idx = (g == 0 ? 0 : this->head + this->nvec * VEC) + lane;
        if (lane >= n) return 0;
        x[0] = ElemT<T>::load(this->row + idx);
        return 1;
    }
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

// A bound above which K .. K + slack keys lie, found by halving the range of
// the keys, or, where many keys are equal, the K-th largest key itself (then
// fewer than K lie above it).  count(b) is the number of keys >= b; K or
// more are >= lo (or there are fewer than K), none is above hi.
template <typename F>
__device__ __forceinline__ uint32_t lp_bound(uint32_t lo, uint32_t hi, int K, F&& count) {
    const int slack = min(kLpSlack, 4 + K / 4);
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2 + 1;
        const int n = count(mid);
        if (n < K) {
            hi = mid - 1;
        } else if (n <= K + slack) {
            return mid - 1;
        } else {
            lo = mid;
        }
    }
    return lo;
}

template <typename T, bool CLUSTER>
__global__ void __launch_bounds__(kLpThreads, 4) k_token_logprobs(LogprobArgs a) {
    constexpr int VEC = ElemT<T>::VEC;
    __shared__ LpSmem s;
    extern __shared__ float group_max[];  // [nb + 2], in the leading CTA
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = CLUSTER ? (int)cluster_size() : 1, part = CLUSTER ? (int)cluster_rank() : 0;
    const int r = CLUSTER ? blockIdx.x / S : blockIdx.x;
    const int tok = a.tokens ? a.tokens[r] : 0;
    if (tok < 0 || tok >= a.V) {
        if (part == 0) {
            if (tok != -1 && tid == 0 && a.dev_error) atomicOr(a.dev_error, kDevErrToken);
            lp_no_result(a, r, tok == -1 ? 0.0f : -INFINITY);
        }
        return;
    }
    if (CLUSTER) cluster_arrive();  // awaited before the first store into the leader
    const LpRow<T> row(static_cast<const T*>(a.logits) + (size_t)r * a.stride, a.V);
    const float xt = ElemT<T>::load(row.row + tok);

    // ------------------------------------------------------- the one read
    using Vec = RowVec<T>;
    const uint4* vecs = row.vec();
    const float2 cc = make_float2(a.c, a.c);
    const float far = kLpFar / a.c;
    LpSums sum;
    // Elements before the token: above xt, and equal to it in the groups
    // before the token's own, where the bound is the next value below.
    int before = 0;
    const int tok_group = tok < row.head                    ? 0
                          : tok < row.head + row.nvec * VEC ? 1 + (tok - row.head) / (32 * VEC)
                                                            : row.nb + 1;
    const typename Vec::Least above = Vec::least(xt), reach = Vec::least(next_below<T>(xt));
    bool awaited = false;
    auto put_max = [&](int g, float v) {
        if (CLUSTER)
            cluster_store(cluster_map(group_max + g, 0), v);
        else
            group_max[g] = v;
    };
    auto count_before = [&](float x, int idx) { before += x > xt || (x == xt && idx < tok); };
    if (part == 0 && warp == 0) {  // head and tail: one element a lane
#pragma unroll
        for (int end = 0; end < 2; ++end) {
            float x = -INFINITY;
            int idx;
            const int n = row.load(end ? row.nb + 1 : 0, &x, idx);
            const float m = warp_max_redux(x);
            if (m > sum.m) sum.raise(m, a.c);
            sum.exact(a.c);
            if (n) {
                count_before(x, idx);
                sum.add_any(make_float2(x, -INFINITY), cc);
            }
            if (CLUSTER && !awaited) {
                cluster_wait();
                awaited = true;
            }
            if (lane == 0) put_max(end ? row.nb + 1 : 0, m);
        }
        sum.settle(a.c);
    }
    // A warp's tiles; a vector's register takes its successor of the next
    // tile as soon as it has been used, so 4 KiB stay on their way.
    const int step = S * kLpWarps * kLpTile;
    auto load = [&](int g) {
        const int v = g * 32 + lane;
        return v < row.nvec ? __ldg(vecs + v) : Vec::none();
    };
    int g0 = (part * kLpWarps + warp) * kLpTile;
    uint4 q[kLpTile];
#pragma unroll
    for (int j = 0; j < kLpTile; ++j) q[j] = load(g0 + j);
    for (; g0 < row.nb; g0 += step) {
        float mine = 0.0f, most = -INFINITY;
        uint32_t some = 0;  // bit j: group j holds an element that reaches xt
#pragma unroll
        for (int j = 0; j < kLpTile; ++j) {
            const float gm = warp_max_redux(Vec::max(q[j]));
            most = fmaxf(most, gm);
            if (lane == j) mine = gm;
            some |= gm >= xt ? 1u << j : 0u;
        }
        if (most > sum.m) sum.raise(most, a.c);
        if (CLUSTER && !awaited) {
            cluster_wait();
            awaited = true;
        }
        if (lane < kLpTile && g0 + lane < row.nb) put_max(g0 + lane + 1, mine);
        const float2 nmc = make_float2(-sum.mc, -sum.mc);
        const typename Vec::Least least = Vec::least(sum.m - far);
        typename Vec::Count n = Vec::count_zero();
        const int at = tok_group - 1 - g0;  // the token's place among the tile's groups
        auto count = [&](int j) {
            if (!((some >> j) & 1u)) return;
            if (j != at) {
                Vec::count(n, q[j], j < at ? reach : above);
            } else {
                const int v = (g0 + j) * 32 + lane, idx = row.head + v * VEC;
#pragma unroll
                for (int i = 0; i < Vec::kPairs; ++i) {
                    const float2 x = Vec::pair(q[j], i);
                    count_before(x.x, idx + 2 * i);
                    count_before(x.y, idx + 2 * i + 1);
                }
            }
        };
        if (sum.plain) {
#pragma unroll
            for (int j = 0; j < kLpTile; ++j) {
#pragma unroll
                for (int i = 0; i < Vec::kPairs; ++i) sum.add_plain(Vec::pair_above(q[j], i, least), cc, nmc);
                count(j);
                q[j] = load(g0 + step + j);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kLpTile; ++j) {
#pragma unroll
                for (int i = 0; i < Vec::kPairs; ++i) sum.add_any(Vec::pair(q[j], i), cc);
                count(j);
                q[j] = load(g0 + step + j);
            }
        }
        before += Vec::count_sum(n);
    }
    sum.exact(a.c);
    {
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
        if (CLUSTER) {
            if (!awaited) cluster_wait();
            if (lane == 0)
                cluster_store(cluster_map(&s.part[part * kLpWarps + warp], 0),
                              make_float4(p.m, p.z, p.e, __int_as_float(p.before)));
            cluster_arrive();
            cluster_wait();
            if (part != 0) return;
        } else {
            if (lane == 0) s.part[warp] = p;
            __syncthreads();
        }
    }

    // ------------------------------------------- the leader: merged results
    const int n_groups = row.nb + 2;
    if (warp == 1) {
        LpPart p[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            p[k] = lane + 32 * k < S * kLpWarps ? s.part[lane + 32 * k] : LpPart{kNoMax, 0.0f, 0.0f, 0};
        const float m = warp_max_redux(fmaxf(p[0].m, p[1].m));
        float z = 0.0f, e = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float d = fmaxf((p[k].m - m) * a.c, -1000.0f), f = ex2(d);
            z += p[k].z * f;
            e += (p[k].e + p[k].z * d) * f;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            z += __shfl_xor_sync(0xffffffffu, z, o);
            e += __shfl_xor_sync(0xffffffffu, e, o);
        }
        before = __reduce_add_sync(0xffffffffu, p[0].before + p[1].before);
        // nothing is below -inf: every place of the groups before the token's
        // was counted, the empty ones of the last group too
        if (xt == -INFINITY && tok_group == row.nb + 1) before -= (row.nb * 32 - row.nvec) * VEC;
        const bool valid = z > 0.0f && z < INFINITY;  // no NaN, no +inf, something finite
        const double ln_z = ln_of(z);
        if (lane == 0) {
            s.m = m;
            s.ln_z_hi = (float)ln_z;
            s.ln_z_lo = (float)(ln_z - (double)(float)ln_z);
            s.valid = valid;
            if (valid) {
                if (a.logprob) a.logprob[r] = a.tokens ? (float)((double)(xt - m) * a.inv_t - ln_z) : 0.0f;
                if (a.rank) a.rank[r] = a.tokens ? before + 1 : -1;
                if (a.entropy) a.entropy[r] = (float)(ln_z - (double)(e / z * kLn2));
            } else if (a.dev_error) {
                atomicOr(a.dev_error, kDevErrNonfinite);
            }
        }
    } else if (warp == 0 && a.top_k > 0 && n_groups <= kLpGroups) {
        float m = -INFINITY;
        for (int g = lane; g < n_groups; g += 32) {
            s.group[g] = g;
            m = fmaxf(m, group_max[g]);
        }
        m = warp_max_redux(m);
        if (lane == 0) {
            s.top = okey32(m);
            s.tau = 0u;
            s.n_group = n_groups;
            s.n_cand = 0;
        }
    } else if (warp == 0 && a.top_k > 0) {
        constexpr int kKeys = 16;  // keys a lane holds; longer rows are read from shared memory
        // an empty head or tail has no key (-inf has one)
        auto key = [&](int g) {
            const bool some = g < n_groups && !(g == 0 && row.head == 0) && !(g == row.nb + 1 && row.tail == 0);
            return some ? okey32(group_max[g]) : 0u;
        };
        uint32_t held[kKeys], top = 0;
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            held[i] = key(i * 32 + lane);
            top = max(top, held[i]);
        }
        for (int g = kKeys * 32 + lane; g < n_groups; g += 32) top = max(top, key(g));
        top = __reduce_max_sync(0xffffffffu, top);
        auto count = [&](uint32_t b) {
            int n = 0;
#pragma unroll
            for (int i = 0; i < kKeys; ++i) n += held[i] >= b;
            for (int g = kKeys * 32 + lane; g < n_groups; g += 32) n += key(g) >= b;
            return __reduce_add_sync(0xffffffffu, n);
        };
        const uint32_t tau = lp_bound(0u, top, a.top_k, count);
        // every group above tau and, if they are fewer than K, the first that reach it
        int n = 0, equal = a.top_k - count(tau + 1);
        for (int g0 = 0; g0 < n_groups; g0 += 32) {
            const uint32_t k = key(g0 + lane);
            const uint32_t same = __ballot_sync(0xffffffffu, k == tau), lower = (1u << lane) - 1u;
            const bool take = k > tau || (k == tau && __popc(same & lower) < equal);
            const uint32_t taken = __ballot_sync(0xffffffffu, take);
            if (take) s.group[n + __popc(taken & lower)] = g0 + lane;
            n += __popc(taken);
            equal -= __popc(same);
        }
        if (lane == 0) {
            s.top = top;
            s.tau = tau;
            s.n_group = n;
            s.n_cand = 0;
        }
    }
    __syncthreads();
    if (!s.valid) {
        lp_no_result(a, r, a.tokens ? -INFINITY : 0.0f);
        return;
    }
    if (a.top_k == 0) return;

    // --------------------------- the alternatives, from the chosen groups
    const int n_group = s.n_group;
    float x[VEC];
    int idx;
    // The bound of the groups leaves little more than K elements, unless the
    // row has few groups or its best elements share some (a sorted row).
    // Then the bound is raised to one that leaves about K vectors.
    bool raise = n_groups <= kLpGroups;
    for (;;) {
        if (raise) {
            uint32_t held[kLpHeld];  // this lane's vectors: their maxima
#pragma unroll
            for (int k = 0; k < kLpHeld; ++k) {
                held[k] = 0u;
                const int i = warp + k * kLpWarps;
                if (i < n_group) {
                    const int n = row.load(s.group[i], x, idx);
                    float m = x[0];
#pragma unroll
                    for (int j = 1; j < VEC; ++j)
                        if (j < n) m = fmaxf(m, x[j]);
                    held[k] = n ? okey32(m) : 0u;
                }
            }
            int turn = 0;
            const uint32_t tau = lp_bound(s.tau, s.top, a.top_k, [&](uint32_t b) {
                int n = 0;
#pragma unroll
                for (int k = 0; k < kLpHeld; ++k) n += held[k] >= b;
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
        const uint32_t tau = s.tau;
        for (int i = warp; i < n_group; i += kLpWarps) {
            const int n = row.load(s.group[i], x, idx);
            int ties = 0;
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if (j < n) {
                    const uint32_t k = okey32(x[j]);
                    ties += k == tau;
                    if (k > tau) {
                        const int at = atomicAdd(&s.n_cand, 1);
                        if (at < kLpCands) s.cand[at] = order_key(x[j], idx + j);
                    }
                }
            ties = __reduce_add_sync(0xffffffffu, ties);
            if (lane == 0) s.ties[i] = ties;
        }
        __syncthreads();
        if (s.n_cand <= kLpCands || raise) break;
        raise = true;
    }
    int n_cand = s.n_cand;
    if (n_cand < a.top_k) {  // and the first elements equal to tau
        const int need = a.top_k - n_cand;
        if (warp == 0) {
            int sum_before = 0;
            for (int i0 = 0; i0 < n_group; i0 += 32) {
                const int t = i0 + lane < n_group ? s.ties[i0 + lane] : 0;
                const int incl = warp_inclusive_scan_i(t);
                if (i0 + lane < n_group) s.ties[i0 + lane] = t > 0 ? sum_before + incl - t : need;
                sum_before += __shfl_sync(0xffffffffu, incl, 31);
            }
        }
        __syncthreads();
        const uint32_t tau = s.tau;
        for (int i = warp; i < n_group; i += kLpWarps) {
            if (s.ties[i] >= need) continue;  // none here, or none still wanted
            const int n = row.load(s.group[i], x, idx);
            int ties = 0;
#pragma unroll
            for (int j = 0; j < VEC; ++j) ties += j < n && okey32(x[j]) == tau;
            int at = s.ties[i] + warp_inclusive_scan_i(ties) - ties;
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if (j < n && okey32(x[j]) == tau) {
                    if (at < need) s.cand[n_cand + at] = order_key(x[j], idx + j);
                    ++at;
                }
        }
        __syncthreads();
        n_cand = a.top_k;
    }
    // a candidate's place is the number of candidates before it
    const double ln_z = (double)s.ln_z_hi + (double)s.ln_z_lo;
    for (int i = tid; i < n_cand; i += kLpThreads) {
        const uint64_t k = s.cand[i];
        int place = 0;
        for (int j = 0; j < n_cand; ++j) place += s.cand[j] > k;
        if (place < a.top_k) {
            a.top_ids[(size_t)r * a.top_k + place] = key_index(k);
            a.top_logprobs[(size_t)r * a.top_k + place] = (float)((double)(key_value(k) - s.m) * a.inv_t - ln_z);
        }
    }
}

// CTAs that share a row: as many as keep every SM busy when rows are few,
// each with a tile for every warp.
template <typename T>
static cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t st) {
    const int groups = (a.V / ElemT<T>::VEC + 31) / 32;
    int sms = 0, dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return cudaErrorUnknown;
    int S = 1;
    while (S < kLpMaxCluster && (long long)a.R * S < 2 * sms && groups >= 2 * S * kLpWarps * kLpTile) S *= 2;
    const size_t dyn = (size_t)(groups + 2) * sizeof(float);
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
    LogprobArgs a{logits, R, V, top_k, row_stride, tokens, (float)(kLog2e / (double)temperature),
                  1.0 / (double)temperature, logprob, rank, entropy, top_ids, top_logprobs, dev_error};
    return (dtype == SPEC_BF16 ? launch_logprobs<__nv_bfloat16>(a, st) : launch_logprobs<float>(a, st)) == cudaSuccess
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}
