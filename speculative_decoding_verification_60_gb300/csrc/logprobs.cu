// Log probabilities of given tokens with the entropy and the top
// alternatives of their rows (spec_token_logprobs): what is reported beside
// the tokens a verification emits, and what a target hands to the training
// of its draft.
//
// One read of a row.  A row's 16-byte vectors are taken a warp's width at a
// time: 32 vectors side by side are a group (256 bf16 or 128 fp32 elements),
// and the unaligned head and tail of a row are the first and the last group.
// Per group a warp takes the maximum (one reduction instruction) and, against
// a reference r near its own running maximum m, z = sum 2^t and e = sum t 2^t
// of t = x c - r, c = log2(e) / T.  From the merged sums, now against m,
//     log p(v) = (x_v - m) / T - ln z,    entropy = ln z - ln 2 * e / z.
// Exactness: r is a whole number, so a new one scales the sums by a power of
// two; a maximum that may hold most of the row is counted, not summed, so that
// ln z = ln(1 + rest) keeps every digit of the rest; and what c is off by,
// rounded to 32 bits, is put right in ln z: d ln z / d ln c is ln 2 * e / z.
// (Largest errors, 96 kinds of rows of 1000 to 524280: log p 1.5e-6, and 1.2e-6
// of its value near 0, where plain sums lose all digits.  Sums that rescale by
// exponentials and include the maximum were up to 3e-5 off and 1.5 % faster
// over many long rows, 0.6 us over few, 5 to 8 % over thousands of short ones.)
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
    float c;       // log2(e) / T
    float c_off;   // (log2(e) / T / c - 1) ln 2
    float beside;  // T ln 8: how far below another of an eighth of its weight is
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
constexpr int kLpPerSm = 4;
constexpr int kLpTile = 6;   // groups of a tile: 3 KiB
constexpr int kLpTileBytes = kLpTile * 512;
// Tiles a warp has on their way, beside the one in its registers: a second
// only where few rows are shared and a warp has two tiles in all (four CTAs of
// an SM keep enough on the way with one, and 777 fp32 rows take 3 us less).
constexpr int lp_depth(bool cluster) { return cluster ? 2 : 1; }
constexpr size_t lp_ring(bool cluster) { return (size_t)kLpWarps * lp_depth(cluster) * kLpTileBytes; }
constexpr int kLpMaxCluster = 8;
constexpr float kLpPlain = 4096.0f;  // |m c| below this: see LpSums
constexpr float kLpLeastC = 1e-30f;  // so that m - kLpFar / c stays in range
constexpr float kLpFar = 200.0f;     // 2^-200 is zero
// The K-th best group need not be found exactly: any bound that leaves K to
// K + kLpSlack groups will do.
constexpr int kLpSlack = 36;
constexpr int kLpCands = 8 * (kMaxTop + kLpSlack) + 16;  // the elements of that many vectors, and the ends
constexpr int kLpBins = 256;
constexpr uint32_t kLpNoneKey = 0x007fffffu;  // the order key of -inf
constexpr int kLpBinShift = 17;  // keys a bin at first: two bf16 values, so four binades in all
constexpr size_t kLpCandBytes = kLpCands * sizeof(uint64_t);
static_assert(kLpCandBytes % 16 == 0, "the group keys come after the candidates");

// What a warp makes of its groups (see LpSums).
struct __align__(16) LpPart {
    float m, ref, z, e;
    int n, before, pad[2];
};
static_assert(sizeof(LpPart) == 32 && alignof(LpPart) == 16, "sent to the leader as two 16-byte stores");

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
    // This lane's vector of group g (1 .. nb), and whether it has one.
    __device__ __forceinline__ bool has(int g) const { return (g - 1) * 32 + (int)(threadIdx.x & 31) < this->nvec; }
    __device__ __forceinline__ uint4 vector(int g) const {
        return has(g) ? __ldg(this->vec() + (g - 1) * 32 + (threadIdx.x & 31)) : RowVec<T>::none();
    }
    // Index of this lane's first element of group g, the ends' too.
    __device__ __forceinline__ int index(int g) const {
        const int lane = threadIdx.x & 31;
        return g == 0   ? lane
               : g > nb ? this->head + this->nvec * ElemT<T>::VEC + lane
                        : this->head + ((g - 1) * 32 + lane) * ElemT<T>::VEC;
    }
    // How many elements this lane has of group g, the ends' too.
    __device__ __forceinline__ int count(int g) const {
        if (g >= 1 && g <= nb) return has(g) ? ElemT<T>::VEC : 0;
        return (int)(threadIdx.x & 31) < (g == 0 ? this->head : this->tail) ? 1 : 0;
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
#pragma unroll 1
    for (int j = tid; j < a.top_k; j += n) {
        a.top_ids[(size_t)r * a.top_k + j] = -1;
        a.top_logprobs[(size_t)r * a.top_k + j] = -INFINITY;
    }
}

// 2^d for a whole number d <= 0.
__device__ __forceinline__ float lp_pow2(float d) { return __int_as_float(((int)fmaxf(d, -127.0f) + 127) << 23); }

// Running sums of a lane; m is the warp's largest value so far.  Where m c is
// of ordinary size (a masked row's lowest values, a huge or tiny temperature
// are not) t = x c - ref is one operation, ref = m c rounded up to a whole
// number; otherwise t = (x - m) c.
struct LpSums {
    static constexpr float kNone = INFINITY;  // ref where t = (x - m) c
    float m = -INFINITY, ref = kNone;
    bool counted = false;  // n of this lane's elements, equal to m, are not in the sums
    int n = 0;
    float2 z = make_float2(0.0f, 0.0f), e = make_float2(0.0f, 0.0f);
    __device__ __forceinline__ bool plain() const { return ref != kNone; }
    __device__ static __forceinline__ float ref_of(float m, float c) {
        const float mc = m * c;
        return fabsf(mc) < kLpPlain && c > kLpLeastC ? ceilf(mc) : kNone;
    }
    // How far the reference lies above m's own place.
    __device__ static __forceinline__ float above(float m, float ref, float c) {
        return ref != kNone ? fmaf(-m, c, ref) : 0.0f;
    }
    // By how much places fall when (m, ref) gives way to (m2, ref2); *f: 2^ that.
    __device__ static __forceinline__ float change(float m, float ref, float m2, float ref2, float c, float* f) {
        if (ref != kNone && ref2 != kNone) {
            *f = lp_pow2(ref - ref2);
            return ref - ref2;
        }
        const float d = fmaxf((m - m2) * c + above(m, ref, c) - above(m2, ref2, c), -1000.0f);
        *f = ex2(d);  // 0 for any distance whose weight is
        return d;
    }
    __device__ __forceinline__ void raise(float m2, float c) {  // to a larger value
        const float ref2 = ref_of(m2, c);
        if (m > -INFINITY) {
            if (counted) {  // joins the sums
                const float t = -above(m, ref, c), w = (float)n * ex2(t);
                z.x += w;
                e.x = fmaf(w, t, e.x);
            }
            if (ref2 != ref || ref2 == kNone) {
                float f;
                const float d = change(m, ref, m2, ref2, c, &f);
                e = make_float2((e.x + z.x * d) * f, (e.y + z.y * d) * f);
                z = make_float2(z.x * f, z.y * f);
            }
        }
        counted = false;
        n = 0;
        m = m2;
        ref = ref2;
    }
};

__device__ __forceinline__ int lp_slack(int K) { return min(kLpSlack, 4 + K / 4); }

// What decides an element's place before the token: above xt, or equal to it
// and of a lower index.  In the groups before the token's own that is one
// comparison with the next value below xt; in its own, the elements equal to
// it are counted apart.
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
            const float gm = warp_max_redux_nan(Vec::max(q[j]));
            most = max_nan(most, gm);
            if ((threadIdx.x & 31) == j) mine = gm;
        }
    }
    // Elements before the token (those equal to it in its own group apart).
    __device__ __forceinline__ int before(const LpToken<T>& tk, int g0) const {
        if (most < tk.x) return 0;
        typename Vec::Count n = Vec::count_zero();
        const int at = tk.group - g0;  // the token's group among the tile's
        if (at > 0 && at < kLpTile) {
#pragma unroll
            for (int j = 0; j < kLpTile; ++j) Vec::count(n, q[j], j < at ? tk.reach : tk.above);
        } else {
            const typename Vec::Least bound = at > 0 ? tk.reach : tk.above;
#pragma unroll
            for (int j = 0; j < kLpTile; ++j) Vec::count(n, q[j], bound);
        }
        return Vec::count_sum(n);
    }
    // The tile's maximum is the warp's new one.  Where neither the old one nor
    // another group of the tile has an eighth of its weight, it may hold
    // most of the row, and is taken out (where one has, ln z is at least 0.1,
    // and the maximum may as well be summed).  Rare in rows without such a
    // token: 4096 rows take 0.6 us more where only half its weight rules that
    // out, and up to 4 us more where every new maximum is taken out.
    __device__ __forceinline__ void raise(LpSums& sum, float c, float beside, uint4* spare) {
        const float near = most - beside;
        const bool far = sum.m < near;
        sum.raise(most, c);
        if (!far) return;
        const uint32_t groups = __ballot_sync(0xffffffffu, mine >= near && mine > -INFINITY);
        if (groups & (groups - 1)) return;
        sum.counted = true;
        // by way of shared memory: the code for one group, not for each
#pragma unroll
        for (int j = 0; j < kLpTile; ++j)
            if (groups == 1u << j) *spare = q[j];
        sum.n = Vec::take_out(*spare, most);
#pragma unroll
        for (int j = 0; j < kLpTile; ++j)
            if (groups == 1u << j) q[j] = *spare;
    }
    // z is summed by vectors, tiles and then the row: 250 adds one after
    // another (1000 in the longest rows) are off by a quarter as many roundings
    // where all weights are alike.
    __device__ __forceinline__ void add(LpSums& sum, float c, float far) const {
        const float2 cc = make_float2(c, c);
        float2 z;
        if (sum.plain()) {
            // values at least kLpFar / c below m add nothing, and -inf has no product with 0
            const float2 nr = make_float2(-sum.ref, -sum.ref);
            const typename Vec::Least least = Vec::least(sum.m - far);
#pragma unroll
            for (int j = 0; j < kLpTile; ++j) {
                float2 w[Vec::kPairs];
#pragma unroll
                for (int i = 0; i < Vec::kPairs; ++i) {
                    const float2 t = __ffma2_rn(Vec::pair_above(q[j], i, least), cc, nr);
                    w[i] = make_float2(ex2(t.x), ex2(t.y));
                    sum.e = __ffma2_rn(w[i], t, sum.e);
                }
                z = j == 0 ? Vec::sum(w) : __fadd2_rn(z, Vec::sum(w));
            }
        } else {
            const float2 nm = make_float2(-sum.m, -sum.m);
#pragma unroll
            for (int j = 0; j < kLpTile; ++j) {
                float2 w[Vec::kPairs];
#pragma unroll
                for (int i = 0; i < Vec::kPairs; ++i) {
                    const float2 t = __fmul2_rn(__fadd2_rn(Vec::pair(q[j], i), nm), cc);
                    w[i] = make_float2(ex2(t.x), ex2(t.y));  // a NaN still shows in z
                    sum.e = __ffma2_rn(w[i], make_float2(fmaxf(t.x, -1000.0f), fmaxf(t.y, -1000.0f)), sum.e);
                }
                z = j == 0 ? Vec::sum(w) : __fadd2_rn(z, Vec::sum(w));
            }
        }
        sum.z = __fadd2_rn(sum.z, z);
    }
};

// A warp's part of a row.
__device__ __forceinline__ LpPart lp_part(const LpSums& sum, int before) {
    LpPart p;
    p.m = sum.m;
    p.ref = sum.ref;
    p.z = sum.z.x + sum.z.y;
    p.e = sum.e.x + sum.e.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        p.z += __shfl_xor_sync(0xffffffffu, p.z, o);
        p.e += __shfl_xor_sync(0xffffffffu, p.e, o);
    }
    p.n = __reduce_add_sync(0xffffffffu, sum.n);
    p.before = __reduce_add_sync(0xffffffffu, before);
    return p;
}

// Shared memory of the CTA that finishes a row.
struct LpFinish {
    static constexpr int kGroups = 256;  // at most this many groups are read again
    int group[kGroups];      // the groups that hold the alternatives
    int ties[kGroups + 2];   // elements equal to tau in each and in the ends, then how many come before
    int bin[kLpBins];
    int found, at, in;       // of a round of lp_select: the K-th key's bin, keys before it, keys in it
    int n_group, n_cand;
    float m;
    float2 ln_z;  // in two parts
    int valid;
};

__device__ __forceinline__ void lp_clear(LpFinish& s) {
    for (int i = threadIdx.x; i < kLpBins; i += kLpThreads) s.bin[i] = 0;
    if (threadIdx.x == 0) s.found = kLpBins;
}
// A bound tau such that K .. K + slack keys lie above it, or, where many keys
// are equal, the K-th largest key itself (then fewer than K lie above); -inf's
// key if fewer than K keys lie above that.  Keys are counted in bins down from `top`,
// then the K-th one's bin in finer ones.  each(f) calls f(key) for the keys,
// shared among the CTA's threads.  *above: keys above tau.  cleared: the bins
// are (lp_clear and a barrier).
template <typename F>
__device__ __forceinline__ uint32_t lp_select(LpFinish& s, uint32_t top, int K, int* above, bool cleared, F&& each) {
    const int tid = threadIdx.x, lane = tid & 31;
    uint32_t hi = top;
    int shift = kLpBinShift, n = 0;  // n keys lie above hi
    for (;;) {
        if (!cleared) {
            __syncthreads();
            lp_clear(s);
            __syncthreads();
        }
        cleared = false;
        int finite = 0;  // keys above -inf's that this thread has seen
        each([&](uint32_t k) {
            const uint32_t bin = (hi - k) >> shift;
            if (k <= hi && bin < kLpBins) atomicAdd(&s.bin[bin], 1);
            finite += k > kLpNoneKey && k <= top;
        });
        if (tid == 0) s.in = 0;
        __syncthreads();
        if (tid < 32) {
            constexpr int kEach = kLpBins / 32;
            int sum = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) sum += s.bin[lane * kEach + i];
            int at = n + warp_inclusive_scan_i(sum) - sum;
            if (at < K && at + sum >= K)  // in one of this lane's bins
                for (int i = lane * kEach;; ++i) {
                    if (at + s.bin[i] >= K) {
                        s.found = i;
                        s.at = at;
                        s.in = s.bin[i];
                        break;
                    }
                    at += s.bin[i];
                }
        }
        __syncthreads();
        const uint32_t bin = (uint32_t)s.found;
        if (bin == kLpBins) {  // further down: among -inf (or past the last key), or in the whole range
            finite = __reduce_add_sync(0xffffffffu, finite);
            if (lane == 0 && finite) atomicAdd(&s.in, finite);
            __syncthreads();
            if (s.in < K || shift == 24) {
                *above = s.in;
                return kLpNoneKey;
            }
            shift = 24;  // 256 such bins are all keys: this round finds it
            continue;
        }
        n = s.at;
        hi -= bin << shift;
        const uint64_t below = 1ull << shift;
        if (n + s.in <= K + lp_slack(K)) {
            *above = n + s.in;
            return hi >= below ? hi - (uint32_t)below : 0u;
        }
        *above = n;
        if (shift == 0) return hi;
        shift = max(shift - 8, 0);
    }
}

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
        p[k] = lane + 32 * k < n_parts ? parts[lane + 32 * k] : LpPart{-INFINITY, LpSums::kNone, 0.0f, 0.0f, 0, 0};
        m = fmaxf(m, p[k].m);
    }
    m = warp_max_redux(m);
    const float ref = LpSums::ref_of(m, a.c), g = LpSums::above(m, ref, a.c);
    float z = 0.0f, e = 0.0f;
    int n = 0, before = 0;  // n: elements equal to m that are not in the sums
    auto add = [&](float x, int count) {
        const float t = ref != LpSums::kNone ? fmaf(x, a.c, -ref) : (x - m) * a.c;
        const float w = x == m ? 0.0f : (float)count * ex2(t);
        n += x == m ? count : 0;
        z += w;
        e = fmaf(w, fmaxf(t, -1000.0f), e);
    };
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float f;
        const float d = LpSums::change(p[k].m, p[k].ref, m, ref, a.c, &f);
        z += p[k].z * f;
        e += (p[k].e + p[k].z * d) * f;
        before += p[k].before;
        add(p[k].m, p[k].n);
    }
    auto end = [&](float x, int idx) {
        add(x, 1);
        before += x > xt || (x == xt && idx < tok);
    };
    if (lane < row.head) end(ends.x, lane);
    if (lane < row.tail) end(ends.y, row.head + row.nvec * VEC + lane);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, o);
        e += __shfl_xor_sync(0xffffffffu, e, o);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    before = __reduce_add_sync(0xffffffffu, before);
    // nothing is below -inf: every place of the groups before the token's
    // was counted, the empty ones of the last group too
    if (xt == -INFINITY && tok >= row.head + row.nvec * VEC) before -= (row.nb * 32 - row.nvec) * VEC;
    // no NaN, no +inf, something finite
    const bool valid = m > -INFINITY && m < INFINITY && z >= 0.0f && z < INFINITY;
    if (lane == 0) {
        // The maximum holds most of the row: z is 1 + rest against m itself.
        // Otherwise z is taken against its reference, g above m.
        const float up = ex2(g), w = (float)n * ex2(-g);
        const bool most = n == 1 && z * up < 1.0f;
        const float rest = most ? z * up : w + z, all = most ? 1.0f + rest : rest;
        const float at = (most ? fmaf(g, z, e) * up : fmaf(w, -g, e)) / all;
        const float mean = most ? at : at + g;  // of (x - m) c
        // f in [0, 1): ln z = ln(1 + f) + whole ln 2 (the sum is 1/2 or more: its exponent is in its bits)
        const int bits = __float_as_int(rest);
        const float f = most ? rest : __int_as_float((bits & 0x007fffff) | 0x3f800000) - 1.0f;
        const float whole = most ? 0.0f : (float)((bits >> 23) - 127);
        float2 ln_z = make_float2(whole * kLn2Hi, fmaf(whole, kLn2Lo, log1pf(f)));
        ln_z = add_parts(make_float2(ln_z.x, 0.0f), ln_z.y);
        const float entropy = fmaf(-kLn2, at, ln_z.x) + ln_z.y;
        if (!most) ln_z = add_parts(ln_z, g * kLn2);
        ln_z = add_parts(ln_z, a.c_off * mean);
        s.m = m;
        s.ln_z = ln_z;
        s.valid = valid;
        if (valid) {
            if (a.logprob) a.logprob[r] = a.tokens ? lp_log(a, xt - m, ln_z) : 0.0f;
            if (a.rank) a.rank[r] = a.tokens ? before + 1 : -1;
            if (a.entropy) a.entropy[r] = entropy;
        } else {
            set_error(a.dev_error, kDevErrNonfinite);
        }
    }
}

// The first `need` elements equal to `bound`, in index order, among the
// chosen groups and the ends: candidates n_cand, n_cand + 1, ...  A function of
// its own: few rows need it, and the code that all rows run stays together.
template <typename T>
__device__ __noinline__ void lp_ties(const T* logits, int V, LpFinish* fin, uint64_t* cand, int n_group, int n_cand,
                                     int need, float bound) {
    using Vec = RowVec<T>;
    LpFinish& s = *fin;
    const LpRow<T> row(logits, V);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nb = row.nb;
    auto group_of = [&](int i) { return i < n_group ? s.group[i] : i == n_group ? 0 : nb + 1; };
    auto ties_of = [&](int g) {
        const int n = row.count(g), idx = row.index(g);
        int ties = 0;
#pragma unroll 1
        for (int j = 0; j < n; ++j) ties += ElemT<T>::load(row.row + idx + j) == bound;
        return ties;
    };
    constexpr int kAhead = 4;
#pragma unroll 1
    for (int i0 = warp; i0 < n_group; i0 += kAhead * kLpWarps) {
        uint4 q[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            q[k] = i0 + k * kLpWarps < n_group ? row.vector(s.group[i0 + k * kLpWarps]) : Vec::none();
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k * kLpWarps;
            if (i >= n_group) break;
            int ties = 0;
            if (row.has(s.group[i])) {
#pragma unroll
                for (int p = 0; p < Vec::kPairs; ++p) {
                    const float2 x = Vec::pair(q[k], p);
                    ties += (x.x == bound) + (x.y == bound);
                }
            }
            ties = __reduce_add_sync(0xffffffffu, ties);
            if (lane == 0) s.ties[i] = ties;
        }
    }
    if (warp < 2) {
        const int ties = __reduce_add_sync(0xffffffffu, ties_of(group_of(n_group + warp)));
        if (lane == 0) s.ties[n_group + warp] = ties;
    }
    __syncthreads();
    int before[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        before[h] = need;
        const int i = tid + h * kLpThreads;
        if (i >= n_group + 2 || s.ties[i] == 0) continue;
        const int g = group_of(i);
        int n = 0;
#pragma unroll 1
        for (int j = 0; j < n_group + 2; ++j) n += group_of(j) < g ? s.ties[j] : 0;
        before[h] = n;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (tid + h * kLpThreads < n_group + 2) s.ties[tid + h * kLpThreads] = before[h];
    __syncthreads();
#pragma unroll 1
    for (int i = warp; i < n_group + 2; i += kLpWarps) {
        if (s.ties[i] >= need) continue;  // none here, or none still wanted
        const int g = group_of(i), n = row.count(g), idx = row.index(g), ties = ties_of(g);
        int at = s.ties[i] + warp_inclusive_scan_i(ties) - ties;
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            if (ElemT<T>::load(row.row + idx + j) != bound) continue;
            if (at < need) cand[n_cand + at] = order_key(bound, idx + j);
            ++at;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ void lp_take(LpFinish& s, int g) {
    const int at = atomicAdd(&s.n_group, 1);
    if (at < LpFinish::kGroups) s.group[at] = g;  // more only in a row of NaN, refused before they are read
}
// Takes the first n groups whose key is tau; each warp looks at a stretch of
// the row's groups (777 fp32 rows, half of them masked, 64 alternatives: 3.5 us
// of 52 less than with every thread counting the groups before its own).  A function of
// its own as lp_ties is: in line it cost rows that never get here 1 to 2 %.
__device__ __noinline__ void lp_equal(LpFinish* fin, const uint32_t* group_key, int nb, uint32_t tau, int n) {
    LpFinish& s = *fin;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int each = (nb + kLpThreads - 1) / kLpThreads * 32;
    const int from = 1 + warp * each + lane, to = min(nb, warp * each + each);
    int before = 0;
#pragma unroll 1
    for (int g = from; g - lane <= to; g += 32)
        before += __popc(__ballot_sync(0xffffffffu, g <= to && group_key[g] == tau));
    if (lane == 0) s.ties[warp] = before;
    __syncthreads();
    before = 0;
#pragma unroll 1
    for (int w = 0; w < warp; ++w) before += s.ties[w];
#pragma unroll 1
    for (int g = from; g - lane <= to && before < n; g += 32) {
        const uint32_t same = __ballot_sync(0xffffffffu, g <= to && group_key[g] == tau);
        if (((same >> lane) & 1u) && before + __popc(same & ((1u << lane) - 1u)) < n) lp_take(s, g);
        before += __popc(same);
    }
}

// The row's results, from n_parts <= 64 parts and the order keys of the
// maxima of its groups (group_key[g], 1 <= g <= nb).  ends: this lane's
// element of the head and of the tail.  stage: the warp's part of the ring,
// now free.  Loops that run once a row are not
// unrolled: their instructions have to be fetched, too.
template <typename T>
__device__ __forceinline__ void lp_finish(const LogprobArgs& a, int r, const LpRow<T>& row, int tok, float xt,
                                          float2 ends, LpFinish& s, uint64_t* cand, uint4* stage,
                                          const uint32_t* group_key, const LpPart* parts, int n_parts) {
    using Vec = RowVec<T>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nb = row.nb, K = a.top_k;
    if (warp == 1) lp_merge<T>(a, r, row, tok, xt, ends, s, parts, n_parts);
    if (K == 0) {
        __syncthreads();
        if (!s.valid) lp_no_result(a, r, a.tokens ? -INFINITY : 0.0f, tid, kLpThreads);
        return;
    }
    float m = -INFINITY;
    bool refused = false;  // what the ends add to that, the merge finds
    for (int k = lane; k < n_parts; k += 32) {
        m = fmaxf(m, parts[k].m);
        refused = refused || isnan(parts[k].z);
    }
    if (__any_sync(0xffffffffu, refused)) {  // the same in every warp
        __syncthreads();
        lp_no_result(a, r, a.tokens ? -INFINITY : 0.0f, tid, kLpThreads);
        return;
    }
    const uint32_t top = okey32(fmaxf(warp_max_redux(m), kNoMax));

    constexpr int kAhead = 6;  // groups a warp reads at a time: under load a read takes 1 to 2 us
    static_assert(kAhead <= kLpTile, "staged in the warp's part of the ring");
    int n_group = nb;
    auto for_vectors = [&](auto&& f) {  // f(i, vectors) per lane: vector k of group i + k * kLpWarps
#pragma unroll 1
        for (int i0 = warp; i0 < n_group; i0 += kAhead * kLpWarps) {
            uint4 q[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                q[k] = i0 + k * kLpWarps < n_group ? row.vector(s.group[i0 + k * kLpWarps]) : Vec::none();
            f(i0, q);
        }
    };
    // A bound from the keys of the groups, the groups that reach it, and the
    // elements above it from those.  Where the row has few groups, or the
    // bound leaves many more than K elements (the best of a sorted row share
    // some groups), the bound comes from the keys of the chosen groups'
    // vectors.  "Few" is what s.group holds, not what is faster: with the
    // groups' keys wherever there are more groups than K and the slack, 4096
    // rows of 32000 bf16 take 76 us for 5 alternatives and 104 for 64, with all
    // vectors' keys 121 and 139; of 50257, 95 and 122 against 172 and 191; of
    // 4096, 41 for 5 against 47, and the same where the groups are fewer.
    bool vectors = nb <= LpFinish::kGroups;
    if (vectors) {
        for (int g = tid; g < nb; g += kLpThreads) s.group[g] = g + 1;
        __syncthreads();
    }
    float bound;
#pragma unroll 1
    for (bool first = true;; first = false) {
        int above;
        const uint32_t tau = lp_select(s, top, K, &above, first, [&](auto&& f) {
            if (vectors) {
                for_vectors([&](int i0, const uint4* q) {
#pragma unroll
                    for (int k = 0; k < kAhead; ++k)
                        if (i0 + k * kLpWarps < n_group && row.has(s.group[i0 + k * kLpWarps]))
                            f(okey32(Vec::max(q[k])));
                });
            } else {
#pragma unroll 1
                for (int g = 1 + tid; g <= nb; g += kLpThreads) f(group_key[g]);
            }
        });
        if (!vectors) {
#pragma unroll 1
            for (int g = 1 + tid; g <= nb; g += kLpThreads)
                if (group_key[g] > tau) lp_take(s, g);
            if (above < K) lp_equal(&s, group_key, nb, tau, K - above);
        }
        __syncthreads();
        if (!s.valid) {
            lp_no_result(a, r, a.tokens ? -INFINITY : 0.0f, tid, kLpThreads);
            return;
        }
        if (!vectors) n_group = s.n_group;
        // As a float: the key below zero's is -0, which compares equal to zero.
        bound = tau == 0x7fffffffu ? __uint_as_float(0x80000001u) : okey32_to_float(tau);
        auto push = [&](float x, int idx) {
            if (x <= bound) return;
            const int at = atomicAdd(&s.n_cand, 1);
            if (at < kLpCands) cand[at] = order_key(x, idx);
        };
        for_vectors([&](int i0, const uint4* q) {
            uint32_t hits = 0;
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i0 + k * kLpWarps < n_group && !(Vec::max(q[k]) <= bound)) {
                    hits |= 1u << k;
                    stage[k * 32 + lane] = q[k];
                }
#pragma unroll 1
            for (; hits; hits &= hits - 1) {  // few: in code that is not repeated per vector
                const int k = __ffs(hits) - 1, g = s.group[i0 + k * kLpWarps], idx = row.index(g);
                if (!row.has(g)) continue;
                const uint4 v = stage[k * 32 + lane];
#pragma unroll
                for (int p = 0; p < Vec::kPairs; ++p) {
                    const float2 x = Vec::pair(v, p);
                    push(x.x, idx + 2 * p);
                    push(x.y, idx + 2 * p + 1);
                }
            }
        });
        if (warp == 0) {
            if (lane < row.head) push(ends.x, row.index(0));
            if (lane < row.tail) push(ends.y, row.index(nb + 1));
        }
        __syncthreads();
        if (s.n_cand <= kLpCands || vectors) break;
        vectors = true;
        __syncthreads();  // all have seen the count
        if (tid == 0) s.n_cand = 0;
    }
    int n_cand = s.n_cand;
    if (n_cand < K) {
        lp_ties<T>(row.row, a.V, &s, cand, n_group, n_cand, K - n_cand, bound);
        n_cand = K;
    }
    // a candidate's place is the number of candidates before it
    for (int i = tid; i < n_cand; i += kLpThreads) {
        const uint64_t k = cand[i];
        int place = 0;
#pragma unroll 4
        for (int j = 0; j < n_cand; ++j) place += cand[j] > k;
        if (place < K) {
            a.top_ids[(size_t)r * K + place] = key_index(k);
            a.top_logprobs[(size_t)r * K + place] = lp_log(a, key_value(k) - s.m, s.ln_z);
        }
    }
}

// A row by a CTA, or by a cluster whose first CTA finishes it.  Bound by
// memory, one read of the row, while rows are many: 2048 rows of 128256 bf16
// without alternatives take 86.8 us, 0.89 of the measured copy bandwidth; 3072
// live rows of 129280 with 8 alternatives 141 us, 0.83.  The rest is the rows'
// ends, where a CTA has nothing on its way: four CTAs an SM (60 registers, 24 KB
// of tiles each) cover each other's.  Fewer, larger CTAs with a ring of copies
// and teams of finishing warps took 137 and 230 us, rows split over CTAs that
// meet in global memory 195 to 252.  Few rows are bound by one row's latency:
// 5 rows 8.7 us, launch included; so are short ones, a CTA each: 4096 rows of
// 1000 take 21 us, 40 with 5 alternatives, 17 and 33 times their bytes' time.
template <typename T, bool CLUSTER>
__global__ void __launch_bounds__(kLpThreads, kLpPerSm) k_token_logprobs(LogprobArgs a) {
    __shared__ LpFinish s;
    __shared__ LpPart parts[kLpMaxCluster * kLpWarps];
    constexpr int kDepth = lp_depth(CLUSTER);
    __shared__ uint64_t full[kLpWarps][kDepth];
    extern __shared__ __align__(128) uint8_t lp_raw[];
    uint64_t* cand = reinterpret_cast<uint64_t*>(lp_raw + lp_ring(CLUSTER));  // [kLpCands]
    uint32_t* group_key = reinterpret_cast<uint32_t*>(cand + kLpCands);       // [nb + 1]; group 0 has none
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = CLUSTER ? (int)cluster_size() : 1, part = CLUSTER ? (int)cluster_rank() : 0;
    const int r = blockIdx.x / S;
    rows_begin();
    const int tok = a.tokens ? a.tokens[r] : 0;
    if (tok < 0 || tok >= a.V) {
        if (part == 0) {
            if (tok != -1 && tid == 0) set_error(a.dev_error, kDevErrToken);
            lp_no_result(a, r, tok == -1 ? 0.0f : -INFINITY, tid, kLpThreads);
        }
        return;
    }
    if (CLUSTER) cluster_arrive();  // awaited before the first store into the leader
    const LpRow<T> row(static_cast<const T*>(a.logits) + (size_t)r * a.stride, a.V);

    // This warp's tiles, kDepth of them on their way through its part of
    // the ring: what is in flight does not take registers, and is enough
    // when another CTA of the SM is at its row's end.
    uint4* ring = reinterpret_cast<uint4*>(lp_raw) + warp * (kDepth * kLpTileBytes / 16);
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
        for (int i = 0; i < kDepth; ++i) mbar_init(&bars[i], 1);
        mbar_fence_init();
        for (int i = 0; i < kDepth; ++i)
            if (g0 + i * step < row.nb) copy(g0 + i * step, i);
    }
    __syncwarp();
    lp_clear(s);  // for the row's end
    if (tid == 0) s.n_group = s.n_cand = 0;
    const float xt = ElemT<T>::load(row.row + tok);
    const float2 ends = row.ends();
    const LpToken<T> tk(row, tok, xt);
    const float far = kLpFar / a.c;
    int before = 0, slot = 0;
    if (part == 0 && warp == 0 && tk.group >= 1 && tk.group <= row.nb) {  // equal to the token, in its own group
        const uint4 q = row.vector(tk.group);
        const int idx = row.index(tk.group);
#pragma unroll
        for (int i = 0; i < RowVec<T>::kPairs; ++i) {
            const float2 x = RowVec<T>::pair(q, i);
            before += (x.x == xt && idx + 2 * i < tok) + (x.y == xt && idx + 2 * i + 1 < tok);
        }
    }
    LpSums sum;
    LpTile<T> tile;
    uint4* spare = reinterpret_cast<uint4*>(cand) + tid;  // this lane's; the candidates come after the last tile
    static_assert(kLpThreads * sizeof(uint4) <= kLpCandBytes, "a vector each");
    uint32_t parity = 0;
    bool awaited = false, ok = true, refused = false;
    for (; g0 < row.nb; g0 += step) {
        ok = warp_mbar_wait(&bars[slot], parity, kCopyWaitNs);
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
        if (lane == 0 && g0 + kDepth * step < row.nb) copy(g0 + kDepth * step, slot);
        if (++slot == kDepth) {
            slot = 0;
            parity ^= 1;
        }
        tile.maxima();
        refused = refused || !(tile.most < INFINITY);  // a NaN or +inf
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
        before += tile.before(tk, g0 + 1);
        if (tile.most > sum.m) tile.raise(sum, a.c, a.beside, spare);
        if (tile.most > -INFINITY) tile.add(sum, a.c, far);  // not all of it ruled out
    }
    LpPart p = lp_part(sum, before);
    if (refused) p.z = NAN;
    if (!ok) {  // the row is refused; the copies still on their way land before the CTA ends
        p.z = NAN;
        if (lane == 0) {
            set_error(a.dev_error, kDevErrTimeout);
            for (int i = 0; i < kDepth && g0 + i * step < row.nb; ++i) {
                mbar_wait(&bars[slot], parity, kDrainNs);
                if (++slot == kDepth) {
                    slot = 0;
                    parity ^= 1;
                }
            }
        }
        __syncwarp();
    }
    if (CLUSTER) {
        if (!awaited) cluster_wait();
        if (lane == 0) {
            LpPart* to = &parts[part * kLpWarps + warp];
            cluster_store(cluster_map(to, 0), make_float4(p.m, p.ref, p.z, p.e));
            cluster_store(cluster_map(&to->n, 0),
                          make_float4(__int_as_float(p.n), __int_as_float(p.before), 0.0f, 0.0f));
        }
        cluster_arrive();
        cluster_wait();
        if (part != 0) return;
    } else {
        if (lane == 0) parts[warp] = p;
        __syncthreads();
    }
    lp_finish<T>(a, r, row, tok, xt, ends, s, cand, ring, group_key, parts, S * kLpWarps);
}

// CTAs that share a row, each with a tile for every warp: measured at
// V = 128256 bf16 with 20 alternatives, one CTA a row against 2, 4 and 8 takes
// 14.9 / 12.9 / 10.4 / 9.4 us for 5 rows, 15.0 / 13.3 / 11.3 / 11.0 for 30,
// 15.2 / 16.1 / 12.3 / 15.0 for 60, 15.1 / 13.5 / 14.4 / 16.5 for 76, 15.5 / 16.5 /
// 14.9 / 20.2 for 100, 18.7 / 18.5 / 23.4 / 27.1 for 150 and 21.8 / 34.5 / 36.0 /
// 45.6 for 304.  At V = 262144, at 50021 fp32 with 64 alternatives and without
// alternatives the same sizes are best up to 76 rows and from 304; between
// them sharing would save up to 2.5 us (100 rows by 4) and 4 (150 by 2) of the
// 262144, and 1 without alternatives.
template <typename T>
static cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t st) {
    const int groups = (a.V / ElemT<T>::VEC + 31) / 32;
    constexpr int kMostGroups = (int)((kRowsMaxVocab / 4 + 31) / 32);
    constexpr size_t kMost = lp_ring(true) + kLpCandBytes + (kMostGroups + 1) * sizeof(uint32_t);
    LaunchShape shape;
    if (!launch_shape(reinterpret_cast<const void*>(k_token_logprobs<T, false>), kMost, kLpThreads, &shape) ||
        !launch_shape(reinterpret_cast<const void*>(k_token_logprobs<T, true>), kMost, kLpThreads, &shape))
        return cudaErrorUnknown;
    const long long R = a.R, sms = shape.sms;
    const int S_most = 5 * R <= sms ? 8 : 5 * R <= 2 * sms ? 4 : 2 * R <= sms ? 2 : 1;
    int S = 1;
    while (S < S_most && groups >= 2 * S * kLpWarps * kLpTile) S *= 2;
    const size_t dyn = lp_ring(S > 1) + kLpCandBytes + (size_t)(groups + 1) * sizeof(uint32_t);
    return launch_rows(S > 1 ? k_token_logprobs<T, true> : k_token_logprobs<T, false>, a.R, S, kLpThreads, dyn,
                       shape.sms, kLpPerSm, a.dev_error, st, a);
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
    if (R == 0) return clear_error(dev_error, st);
    const double inv_t = 1.0 / (double)temperature;
    const float inv_hi = (float)inv_t, c = (float)(kLog2e / (double)temperature);
    LogprobArgs a{logits, R, V, top_k, row_stride, tokens, c,
                  (float)((kLog2e / (double)temperature / (double)c - 1.0) * 0.69314718055994531),
                  (float)((double)temperature * 2.0794415416798359),
                  make_float2(inv_hi, (float)(inv_t - (double)inv_hi)), logprob, rank, entropy, top_ids, top_logprobs,
                  dev_error};
    return (dtype == SPEC_BF16 ? launch_logprobs<__nv_bfloat16>(a, st) : launch_logprobs<float>(a, st)) == cudaSuccess
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}
