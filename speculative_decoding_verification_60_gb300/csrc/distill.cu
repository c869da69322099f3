// Distillation of a draft model from a teacher's top-K log probabilities:
// the loss of every row with its gradient (spec_distill_topk), and the
// gradient for upstream gradients known later (spec_distill_topk_backward).
//
// With S the listed tokens, the student's softmax is split in two: over the
// tokens outside S (the tail: maximum m_T, Z_T = sum 2^((s - m_T) c)) and
// the K listed ones.  The tail's mass q_T is then a sum of its own terms,
// where 1 - sum q_j would cancel, and the gradient of every tail token is
// one coefficient times 2^((s - m_T) c):
//     t_T - S q_T  =  S q_L - sum t_j,  q_L the listed tokens' mass,
// taken from the side that does not cancel.  Sums are in 32 bits over at most
// a few thousand terms of a lane and then pairwise; the teacher's mass and
// the loss, where differences of nearly equal values are left, in 64.  The
// gradient of a bf16 student is rounded to bf16 once, when it is stored.
#include "cluster.cuh"
#include "vocab_rows.cuh"

namespace sv {

struct DistillArgs {
    const void* student;
    int R, V, K;
    int64_t stride;
    const int32_t* ids;
    const float* teacher;
    const float* weights;  // forward: row weights; backward: upstream gradients
    float c;       // log2(e) / T
    double inv_t;  // c ln 2: 1 / T for the same rounded c
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
    float ln_t;    // subtracted from the teacher's values in two parts (a constant of any
    float ln_t2;   // size may be in them): t_j = exp(l_j - ln_t - ln_t2)
    float live;    // 0: the row has loss 0 and gradient 0
    __device__ __forceinline__ float t(float l) const { return expf(l - ln_t - ln_t2); }
};
static_assert(sizeof(DistillStat) == 32, "row_stats is [R, 8] float");

constexpr int kDsWarps = 8;                          // that take tiles
constexpr int kDsThreads = (kDsWarps + 1) * 32;      // and one for the teacher and the loss
constexpr int kDsLossPerSm = 4, kDsGradPerSm = 3;     // CTAs an SM holds
constexpr int kDsTile = 8;                           // vectors a lane takes of a tile: 4 KiB a warp
constexpr int kDsTileBytes = kDsTile * 512;
constexpr int kDsMaxCluster = 16;
constexpr int kDsMaxTiles = 6;                       // of a warp, when the row stays on the chip
constexpr int kDsIds = kMaxTop / 32;                 // listed tokens a lane looks after
constexpr float kDsPlain = 1024.0f;                  // |m c| below this: t = x c - m c in one operation
// Where the student gives the tail nothing, this much teacher mass outside
// the listed tokens is the rounding of their log probabilities: the loss
// would be +inf for it.
constexpr float kTailRounding = 1.0f / 65536.0f;

// What the first CTA's extra warp finds about the teacher: as it is to the
// warp that has the loss, and rounded to 32 bits to every warp (double
// operations of 27 warps at once took 2 us a row).
struct alignas(16) DsTeacher {
    double mass;  // sum of t_j
    double ln_t;  // subtracted from the teacher's values; +inf: no teacher mass at all
    __device__ __forceinline__ float4 message(bool bucket) const {  // mass, t_T, ln_t in two parts
        if (bucket) return make_float4((float)mass, (float)fmax(1.0 - mass, 0.0), 0.0f, 0.0f);
        const float hi = (float)ln_t;
        return make_float4(1.0f, 0.0f, hi, hi < INFINITY ? (float)(ln_t - (double)hi) : 0.0f);
    }
};
// What the CTAs of a row exchange about it, and its listed tokens.
struct DsRow {
    float2 part[kDsMaxCluster * kDsWarps];  // every warp's maximum and sum of the tail
    float s[kMaxTop], l[kMaxTop];  // listed tokens: student logit, teacher's value
    float m_listed, z_listed;      // their maximum, and sum of 2^((s - m_listed) c)
    alignas(16) int id[kMaxTop];
    float4 teacher;             // from the first CTA: DsTeacher's message
    DsTeacher exact;            // in the last CTA
    float bad[kDsMaxCluster];   // from every CTA: error bits of its share of the checks
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

// A lane's sum of 2^t, t = (x - m) c, against its warp's reference m; mc is
// m c rounded, and what it is off by is taken out at the end (exact()).
struct DsSum {
    float m = kNoMax, mc = 0.0f;
    bool plain = false;
    float2 z = make_float2(0.0f, 0.0f);
    __device__ __forceinline__ void shift(float d) {
        const float f = ex2(fmaxf(d, -1000.0f));
        z = make_float2(z.x * f, z.y * f);
    }
    __device__ __forceinline__ void exact(float c) {
        if (plain) shift(fmaf(-m, c, mc));
        plain = false;
    }
    __device__ __forceinline__ void raise(float m2, float c) {
        exact(c);
        shift((m - m2) * c);
        m = m2;
        mc = m * c;
        plain = fabsf(mc) < kDsPlain;
        if (plain) shift(fmaf(m, c, -mc));
    }
    template <typename T, int N>
    __device__ __forceinline__ void add(const uint4* q, float c) {
        const float2 cc = make_float2(c, c);
        if (plain) {
            const float2 nmc = make_float2(-mc, -mc);
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int i = 0; i < RowVec<T>::kPairs; ++i) {
                    const float2 t = __ffma2_rn(RowVec<T>::pair(q[j], i), cc, nmc);
                    z = __fadd2_rn(z, make_float2(ex2(t.x), ex2(t.y)));
                }
        } else {
            const float2 nm = make_float2(-m, -m);  // x - m first: m c may not be finite
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int i = 0; i < RowVec<T>::kPairs; ++i) {
                    const float2 t = __fmul2_rn(__fadd2_rn(RowVec<T>::pair(q[j], i), nm), cc);
                    z = __fadd2_rn(z, make_float2(ex2(t.x), ex2(t.y)));
                }
        }
    }
};

// A row's listed tokens as a lane loads them (entries lane + 32 k).
struct DsListed {
    int id[kDsIds];
    float l[kDsIds], s[kDsIds];  // teacher's value, student logit
    __device__ __forceinline__ void load(const DistillArgs& a, int r) {
#pragma unroll
        for (int k = 0; k < kDsIds; ++k) {
            const int j = (threadIdx.x & 31) + 32 * k;
            id[k] = j < a.K ? a.ids[(size_t)r * a.K + j] : -1;
            l[k] = j < a.K ? a.teacher[(size_t)r * a.K + j] : 0.0f;
        }
    }
    template <typename T>
    __device__ __forceinline__ void gather(const DistillArgs& a, const T* row) {
#pragma unroll
        for (int k = 0; k < kDsIds; ++k) s[k] = (unsigned)id[k] < (unsigned)a.V ? ElemT<T>::load(row + id[k]) : 0.0f;
    }
};

// The teacher's side of a row, by one warp of each of the S CTAs while the
// row is on its way: the listed tokens' checks (each CTA a share of the
// search for doubles) and sums, and in the first CTA the sum of t_j (in
// double: 1 - sum t cancels where the listed tokens hold nearly all of it).
__device__ __forceinline__ void distill_teacher(const DistillArgs& a, const DsListed& in, DsRow& sm, int part, int S,
                                                DsTeacher* out, int* err_out) {
    const int lane = threadIdx.x & 31;
    float lmax = kNoMax, smax = kNoMax;
    int err = 0;
#pragma unroll
    for (int k = 0; k < kDsIds; ++k) {
        const int j = lane + 32 * k;
        int v = in.id[k];
        if (v != -1 && (v < 0 || v >= a.V)) {
            err |= kDevErrToken;
            v = -1;
        }
        sm.id[j] = v;
        sm.l[j] = in.l[k];
        sm.s[j] = in.s[k];
        if (v >= 0) {
            smax = fmaxf(smax, in.s[k]);
            lmax = fmaxf(lmax, in.l[k]);
            if (isnan(in.l[k]) || in.l[k] == INFINITY) err |= kDevErrNonfinite;
        }
    }
    lmax = warp_max_redux(lmax);
    smax = warp_max_redux(smax);
    __syncwarp();
    float z = 0.0f;
#pragma unroll 1
    for (int j = lane; j < a.K; j += 32)
        if (sm.id[j] >= 0) z += ex2((sm.s[j] - smax) * a.c);
    z = warp_sum_f(z);
    if (lane == 0) {
        sm.m_listed = smax;
        sm.z_listed = z;
    }
#pragma unroll 1
    for (int j0 = 32 * part; j0 < a.K; j0 += 32 * S) {  // each id of 32 against all before it
        const int v = sm.id[j0 + lane];
        bool twice = false;
#pragma unroll 4
        for (int i = 0; i < j0 + 32; i += 4) {
            const int4 u = *reinterpret_cast<const int4*>(sm.id + i);
            const int at = j0 + lane - i;  // own place in u, if 0 .. 3
            twice |= (u.x == v && at != 0) | (u.y == v && at != 1) | (u.z == v && at != 2) | (u.w == v && at != 3);
        }
        if (twice && v >= 0) err |= kDevErrToken;
    }
    if (part == 0) {
        const double ref = a.bucket ? 0.0 : (double)lmax;
        double mass = 0.0;
#pragma unroll 1
        for (int j = lane; j < a.K; j += 32)
            if (sm.id[j] >= 0) mass += exp((double)sm.l[j] - ref);
        mass = warp_sum_d(mass);
        if (!(mass <= (double)-kNoMax)) err |= kDevErrNonfinite;  // as 32 bits hold it
        out->mass = a.bucket ? mass : 1.0;
        out->ln_t = a.bucket ? 0.0 : mass > 0.0 ? ref + ln_of((float)mass) : (double)INFINITY;
    }
    *err_out = __reduce_or_sync(0xffffffffu, err);
}

// The row's statistics from every warp's part and the listed tokens, by each
// warp for itself.
struct DsSums {
    float z, z_tail;          // relative to m and to m_tail
    float listed_q, tail_q;   // the two parts of z, over z
    bool tail;                // the teacher's tail takes part
    int err;                  // error bits
};
__device__ __forceinline__ DistillStat distill_stat(const DistillArgs& a, const DsRow& sm, int S, DsSums* sums) {
    const int lane = threadIdx.x & 31, n_parts = S * kDsWarps;
    const float4 te = sm.teacher;
    DistillStat st{};
    float mt = kNoMax;
#pragma unroll 1
    for (int k = lane; k < n_parts; k += 32) mt = fmaxf(mt, sm.part[k].x);
    mt = warp_max_redux(mt);
    float zt = 0.0f;
#pragma unroll 1
    for (int k = lane; k < n_parts; k += 32) zt += sm.part[k].y * ex2(fmaxf((sm.part[k].x - mt) * a.c, -1000.0f));
    zt = warp_sum_f(zt);
    const float ms = sm.m_listed, m = fmaxf(mt, ms);
    const float in_tail = zt * ex2(fmaxf((mt - m) * a.c, -1000.0f));
    const float listed = sm.z_listed * ex2(fmaxf((ms - m) * a.c, -1000.0f)), z = listed + in_tail;
    const bool no_tail = zt == 0.0f && te.y <= kTailRounding;
    const float t_tail = no_tail ? 0.0f : te.y;
    const uint32_t bad = __reduce_or_sync(0xffffffffu, lane < S ? __float_as_uint(sm.bad[lane]) : 0u);
    *sums = DsSums{z, zt, listed / z, in_tail / z, t_tail > 0.0f, (int)bad};
    if (!(z > 0.0f && z < INFINITY)) sums->err |= kDevErrNonfinite;  // NaN, +inf, or nothing finite
    if (sums->err || te.z == INFINITY) return st;
    st.m_tail = mt;
    st.m = m;
    st.inv_z = 1.0f / z;
    st.mass = t_tail > 0.0f ? 1.0f : te.x;
    st.ln_t = te.z;
    st.ln_t2 = te.w;
    // S q_T - t_T from the smaller part: the same as sum t_j - S (1 - q_T)
    const float d = sums->tail_q < 0.5f ? st.mass * sums->tail_q - t_tail : te.x - st.mass * sums->listed_q;
    st.coef = zt > 0.0f ? d * (float)a.inv_t / zt : 0.0f;
    st.live = 1.0f;
    return st;
}

// The loss, by one warp.  log t - log q cancels where the student is near
// the teacher: in double, and with the same c that the sums were made with.
// The logarithm of a tail's mass near 1 is taken from what it lacks.
__device__ __forceinline__ float distill_loss(const DistillArgs& a, const DsRow& sm, const DistillStat& st,
                                              const DsSums& sums, const DsTeacher& te) {
    const int lane = threadIdx.x & 31;
    const double ln_z = ln_of(sums.z);
    double sum = 0.0;
#pragma unroll 1
    for (int j = lane; j < a.K; j += 32) {
        if (sm.id[j] < 0) continue;
        const double lt = (double)sm.l[j] - te.ln_t;
        const float t = expf((float)lt);
        if (t > 0.0f) sum += (double)t * (lt - ((double)(sm.s[j] - st.m) * a.inv_t - ln_z));
    }
    sum = warp_sum_d(sum);
    if (sums.tail && sums.z_tail > 0.0f) {
        const double t_tail = 1.0 - te.mass;
        const double ln_tail = te.mass < 0.5 ? (double)log1pf(-(float)te.mass) : ln_of((float)t_tail);
        const double ln_q = sums.tail_q > 0.5f ? (double)log1pf(-sums.listed_q)
                                               : (double)(st.m_tail - st.m) * a.inv_t + ln_of(sums.z_tail) - ln_z;
        sum += t_tail * (ln_tail - ln_q);
    } else if (sums.tail) {
        sum = (double)INFINITY;
    }
    return (float)sum;
}

// Gradient of a listed token.
__device__ __forceinline__ float distill_listed_grad(const DistillStat& st, float s, float t, float c, float inv_t,
                                                     float w) {
    const float q = ex2((s - st.m) * c) * st.inv_z;
    return w * (st.mass * q - t) * inv_t;
}

__device__ __forceinline__ void store_elem(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 pack(const float2* x, __nv_bfloat16) {
    return make_uint4(bf16x2_bits(x[0].x, x[0].y), bf16x2_bits(x[1].x, x[1].y), bf16x2_bits(x[2].x, x[2].y),
                      bf16x2_bits(x[3].x, x[3].y));
}
__device__ __forceinline__ uint4 pack(const float2* x, float) {
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                      __float_as_uint(x[1].y));
}

// The gradient of tail tokens: coef 2^((x - m_tail) c), for a row.  As in
// DsSum, t = x c - m_tail c in one operation where that is of ordinary size;
// what the product's rounding is off by goes into the coefficient.
struct DsTail {
    float2 cc, nm, kk;  // c; -m_tail or -m_tail c; the coefficient
    bool plain;
    __device__ __forceinline__ DsTail(float coef, float m_tail, float c) {
        const float mc = m_tail * c;
        plain = fabsf(mc) < kDsPlain;
        const float k = plain ? coef * ex2(fmaf(-m_tail, c, mc)) : coef, n = plain ? -mc : -m_tail;
        cc = make_float2(c, c);
        nm = make_float2(n, n);
        kk = make_float2(k, k);
    }
    __device__ __forceinline__ float2 operator()(float2 x) const {
        const float2 t = plain ? __ffma2_rn(x, cc, nm) : __fmul2_rn(__fadd2_rn(x, nm), cc);
        return __fmul2_rn(make_float2(ex2(t.x), ex2(t.y)), kk);
    }
    // a vector's, stored at g: 16 bytes at once, or element by element
    template <bool ALIGNED, typename T>
    __device__ __forceinline__ void store(T* g, const uint4& q) const {
        float2 y[RowVec<T>::kPairs];
#pragma unroll
        for (int i = 0; i < RowVec<T>::kPairs; ++i) y[i] = (*this)(RowVec<T>::pair(q, i));
        if (ALIGNED) {
            *reinterpret_cast<uint4*>(g) = pack(y, T{});
        } else {
#pragma unroll
            for (int i = 0; i < RowVec<T>::kPairs; ++i) {
                store_elem(g + 2 * i, y[i].x);
                store_elem(g + 2 * i + 1, y[i].y);
            }
        }
    }
};

template <typename T>
__device__ __forceinline__ bool same_alignment(const RowView<T>& row, const T* g) {
    return ((reinterpret_cast<uintptr_t>(row.row) ^ reinterpret_cast<uintptr_t>(g)) & 15u) == 0;
}

// Zero gradient of tiles first, first + step, ... of a row and, in the thread
// group that has tile 0, of its ends.  One warp.
template <typename T>
__device__ __forceinline__ void distill_zero(const RowView<T>& row, T* g, int first, int step) {
    const int lane = threadIdx.x & 31;
    const bool aligned = same_alignment(row, g);
#pragma unroll 1
    for (int v0 = first * kDsTile * 32; v0 < row.nvec; v0 += step * kDsTile * 32)
#pragma unroll 1
        for (int j = 0; j < kDsTile; ++j) {
            const int v = v0 + j * 32 + lane;
            T* at = g + row.head + (size_t)v * ElemT<T>::VEC;
            if (v >= row.nvec) continue;
            if (aligned) {
                *reinterpret_cast<uint4*>(at) = make_uint4(0u, 0u, 0u, 0u);
            } else {
#pragma unroll 1
                for (int i = 0; i < ElemT<T>::VEC; ++i) store_elem(at + i, 0.0f);
            }
        }
    if (first == 0) {
        if (lane < row.head) store_elem(g + lane, 0.0f);
        if (lane < row.tail) store_elem(g + row.head + row.nvec * ElemT<T>::VEC + lane, 0.0f);
    }
}

// The listed tokens among elements [e0, e0 + n) of a row: f(k, offset) for
// each that this lane looks after (entry lane + 32 k).
template <typename F>
__device__ __forceinline__ bool listed_in(const int* ids, int e0, int n, F&& f) {
    bool any = false;
#pragma unroll
    for (int k = 0; k < kDsIds; ++k)
        if ((unsigned)(ids[k] - e0) < (unsigned)n) {
            f(k, ids[k] - e0);
            any = true;
        }
    return any;
}
__device__ __forceinline__ void load_ids(const DistillArgs& a, int r, int* ids) {
#pragma unroll
    for (int k = 0; k < kDsIds; ++k) {
        const int j = (threadIdx.x & 31) + 32 * k;
        ids[k] = j < a.K ? a.ids[(size_t)r * a.K + j] : -1;
    }
}

// This lane's element of the head and of the tail (-inf: none, or listed),
// and their part of the sums.
template <typename T>
__device__ __forceinline__ float2 distill_ends(const RowView<T>& row, const int* ids, DsSum& sum, float c) {
    const int lane = threadIdx.x & 31, tail0 = row.head + row.nvec * ElemT<T>::VEC;
    float2 ends = make_float2(-INFINITY, -INFINITY);
    if (lane < row.head) ends.x = ElemT<T>::load(row.row + lane);
    if (lane < row.tail) ends.y = ElemT<T>::load(row.row + tail0 + lane);
    uint32_t in_head = 0, in_tail = 0;
    listed_in(ids, 0, row.head, [&](int, int o) { in_head |= 1u << o; });
    listed_in(ids, tail0, row.tail, [&](int, int o) { in_tail |= 1u << o; });
    if ((__reduce_or_sync(0xffffffffu, in_head) >> lane) & 1u) ends.x = -INFINITY;
    if ((__reduce_or_sync(0xffffffffu, in_tail) >> lane) & 1u) ends.y = -INFINITY;
    const float m = warp_max_redux(fmaxf(ends.x, ends.y));
    if (m > sum.m) sum.raise(m, c);
    sum.exact(c);
    sum.z.x += ex2((ends.x - sum.m) * c);
    sum.z.y += ex2((ends.y - sum.m) * c);
    if (sum.m > kNoMax) sum.raise(sum.m, c);  // back to one operation per pair
    return ends;
}

// A tile in shared memory, its listed tokens set to -inf there, added to the
// sum; free() is called once every lane has its vectors.
template <typename T, typename F>
__device__ __forceinline__ void distill_tile(const RowView<T>& row, int t, uint4* at, const int* ids, DsSum& sum,
                                             float c, F&& free) {
    const int lane = threadIdx.x & 31, v0 = t * kDsTile * 32, nv = min(kDsTile * 32, row.nvec - v0);
    const bool any = listed_in(ids, row.head + v0 * ElemT<T>::VEC, nv * ElemT<T>::VEC,
                               [&](int, int o) { reinterpret_cast<T*>(at)[o] = T(-INFINITY); });
    // before a later copy into the same place
    if (__any_sync(0xffffffffu, any)) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    uint4 q[kDsTile];
    if (nv == kDsTile * 32) {
#pragma unroll
        for (int j = 0; j < kDsTile; ++j) q[j] = at[j * 32 + lane];
    } else {
#pragma unroll
        for (int j = 0; j < kDsTile; ++j) q[j] = j * 32 + lane < nv ? at[j * 32 + lane] : RowVec<T>::none();
    }
    free();
    const float m = tile_max<T, kDsTile>(q);
    if (m > sum.m) sum.raise(m, c);
    if (m != -INFINITY) sum.add<T, kDsTile>(q, c);  // not all of it ruled out
}

// A warp's tiles of a row through its part of shared memory: buffer b, an
// mbarrier each.
template <typename T>
struct DsBuffers {
    uint4* ring;
    uint64_t* bars;
    __device__ __forceinline__ uint4* at(int b) const { return ring + b * (kDsTileBytes / 16); }
    __device__ __forceinline__ void copy(const RowView<T>& row, int t, int b) const {  // one lane
        const int v0 = t * kDsTile * 32;
        const uint32_t bytes = (uint32_t)min(kDsTile * 32, row.nvec - v0) * 16;
        mbar_arrive_expect_tx(&bars[b], bytes);
        bulk_load(at(b), row.vec() + v0, bytes, &bars[b]);
    }
};
template <typename T>
__device__ __forceinline__ int tiles_of(const RowView<T>& row) {
    return (row.nvec + kDsTile * 32 - 1) / (kDsTile * 32);
}
__device__ __forceinline__ void distill_no_row(const DistillArgs& a, int r) {  // one thread
    a.loss[r] = 0.0f;
    if (a.stats) reinterpret_cast<DistillStat*>(a.stats)[r] = DistillStat{};
}

// What the CTAs of a row send each other, in bytes to the one of rank `part`:
// every warp's part, every CTA's error bits, the teacher.
__device__ __forceinline__ uint32_t distill_bytes(int part, int S) {
    return (uint32_t)(S * (kDsWarps * sizeof(float2) + sizeof(float)) + sizeof(float4) +
                      (part == S - 1 ? sizeof(DsTeacher) : 0));
}
// What the extra warp does for a row.  Before its sums are exchanged: the
// teacher, sent to every CTA of the row (ready() is called before that).
// bar: the mbarrier that counts what is sent.
template <bool CLUSTER, typename R>
__device__ __forceinline__ void distill_before(const DistillArgs& a, const DsListed& in, DsRow& sm, uint64_t* bar,
                                               int part, int S, R&& ready) {
    const int lane = threadIdx.x & 31;
    DsTeacher te{};
    int bad;
    distill_teacher(a, in, sm, part, S, &te, &bad);
    const float4 message = te.message(a.bucket);
    __syncwarp();
    ready();
    if (CLUSTER) {
        if (lane == 0) mbar_arrive_expect_tx(bar, distill_bytes(part, S));  // sm's own entries are written, too
        if (lane < S) {
            const uint32_t to = cluster_map(bar, lane);
            cluster_send(cluster_map(&sm.bad[part], lane), __int_as_float(bad), to);
            if (part == 0) cluster_send(cluster_map(&sm.teacher, lane), message, to);
        }
        if (part == 0 && lane == S)
            cluster_send(cluster_map(&sm.exact, S - 1), *reinterpret_cast<const float4*>(&te), cluster_map(bar, S - 1));
    } else if (lane == 0) {
        sm.bad[0] = __int_as_float(bad);
        sm.teacher = message;
        sm.exact = te;
    }
    __syncwarp();
}
// After it, in the row's last CTA (the first one has the teacher's sums to
// do): the loss and the row's statistics.
__device__ __forceinline__ void distill_after(const DistillArgs& a, int r, const DsRow& sm, int part, int S) {
    if (part != S - 1) return;
    DsSums sums;
    const DistillStat st = distill_stat(a, sm, S, &sums);
    const float loss = st.live != 0.0f ? distill_loss(a, sm, st, sums, sm.exact) : 0.0f;
    if ((threadIdx.x & 31) == 0) {
        a.loss[r] = loss;
        if (a.stats) reinterpret_cast<DistillStat*>(a.stats)[r] = st;
        if (sums.err) set_error(a.dev_error, sums.err);
    }
}

// The loss of a row, by a CTA or a cluster of S: each warp has every (8 S)-th
// tile, one on its way while it works on the one in its registers.  Bound by
// memory, one read of the row: 2432 rows of 128256 bf16 (four full waves of
// CTAs) in 98 us, 0.94 of the measured copy bandwidth; 1024 rows in 45 us,
// 0.85 (two waves, the second two thirds full), and 49 us with 128 listed
// tokens.  Held to 56 registers, which spills 4 to 8 bytes a thread.
template <typename T, bool CLUSTER>
__global__ void __launch_bounds__(kDsThreads, kDsLossPerSm) k_distill_loss(DistillArgs a) {
    extern __shared__ __align__(128) uint8_t ds_raw[];  // [kDsWarps] tiles
    __shared__ DsRow sm;
    __shared__ uint64_t full[kDsWarps], sent;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = CLUSTER ? (int)cluster_size() : 1, part = CLUSTER ? (int)cluster_rank() : 0;
    const int r = blockIdx.x / S;
    rows_begin();
    if (a.weights && a.weights[r] == 0.0f) {
        if (part == 0 && tid == 0) distill_no_row(a, r);
        return;
    }
    if (CLUSTER) {
        if (tid == 0) {
            mbar_init(&sent, 1);
            mbar_fence_init();
        }
        __syncwarp();
        cluster_arrive();  // awaited before the first store into another CTA
    }
    auto ready = [] {
        __syncwarp();
        if (CLUSTER) cluster_wait();
    };
    const RowView<T> row(static_cast<const T*>(a.student) + (size_t)r * a.stride, a.V);
    if (warp == kDsWarps) {
        DsListed in;
        in.load(a, r);
        in.gather(a, row.row);
        distill_before<CLUSTER>(a, in, sm, &sent, part, S, ready);
        if (!CLUSTER) __syncthreads();
        if (!CLUSTER || warp_cluster_wait(&sent, 0, kClusterWaitNs)) {
            distill_after(a, r, sm, part, S);
        } else if (part == S - 1 && lane == 0) {
            set_error(a.dev_error, kDevErrTimeout | kDevErrNonfinite);
            distill_no_row(a, r);
        }
        if (CLUSTER) {
            cluster_arrive();
            cluster_wait();
        }
        return;
    }
    const int unit = part * kDsWarps + warp, units = S * kDsWarps, tiles = tiles_of(row);
    const DsBuffers<T> buf{reinterpret_cast<uint4*>(ds_raw) + warp * (kDsTileBytes / 16), &full[warp]};
    if (lane == 0) {
        mbar_init(&full[warp], 1);
        mbar_fence_init();
        if (unit < tiles) buf.copy(row, unit, 0);
    }
    __syncwarp();
    int ids[kDsIds];
    load_ids(a, r, ids);
    DsSum sum;
    if (unit == 0) distill_ends(row, ids, sum, a.c);
    bool ok = true;
    uint32_t parity = 0;
    for (int t = unit; t < tiles && ok; t += units, parity ^= 1) {
        ok = warp_mbar_wait(&full[warp], parity, kCopyWaitNs);
        if (!ok) break;
        distill_tile(row, t, buf.at(0), ids, sum, a.c, [&] {
            __syncwarp();
            if (lane == 0 && t + units < tiles) buf.copy(row, t + units, 0);
        });
    }
    if (!ok && lane == 0) {  // the row is refused; the copy still on its way lands before the CTA ends
        set_error(a.dev_error, kDevErrTimeout);
        mbar_wait(&full[warp], parity, kDrainNs);
    }
    __syncwarp();
    sum.exact(a.c);
    const float2 p = make_float2(sum.m, ok ? warp_sum_f(sum.z.x + sum.z.y) : NAN);
    ready();
    if (CLUSTER) {
        if (lane < S) cluster_send(cluster_map(&sm.part[unit], lane), p, cluster_map(&sent, lane));
        cluster_arrive();  // no CTA ends while another may write into it
        cluster_wait();
    } else {
        if (lane == 0) sm.part[unit] = p;
        __syncthreads();
    }
}

// Loss and gradient, by persistent CTAs or clusters of S that take rows in
// turn.  All tiles of a row stay in shared memory (n_buf a warp) while the
// sums are exchanged, every CTA of the cluster getting every warp's; the
// gradient is written from there, and each tile's place takes the next row's
// as soon as it has been written.  So a row is read once and written once:
// 2 + 2 bytes an element (bf16), the bound.  What the CTAs of a row exchange
// is there twice, for this row and the next.
//
// 2304 rows of 128256 bf16, clusters of 4 and two tiles a warp: 190 us with one
// listed token, 0.91 of the measured copy bandwidth; 199 with 64 (0.87), 230
// with 128 (0.76: the listed tokens are looked for in every tile, and their
// gradients stored one by one).  1216 rows of 50020 fp32: 86 us, 0.83.
//
// Its size matters: three CTAs' warps are in different phases of it, and with
// the loops that run once or twice a row unrolled (101 KB of code, 74 KB
// without) the same row took a tenth longer.  It is held to 72 registers, which
// spills up to 28 bytes a thread.
template <typename T, bool CLUSTER>
__global__ void __launch_bounds__(kDsThreads, kDsGradPerSm) k_distill_grad(DistillArgs a, int n_buf) {
    constexpr int VEC = ElemT<T>::VEC;
    extern __shared__ __align__(128) uint8_t ds_raw[];  // [kDsWarps][n_buf] tiles
    __shared__ DsRow rows[2];
    __shared__ uint64_t full[kDsWarps][kDsMaxTiles], sent[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = CLUSTER ? (int)cluster_size() : 1, part = CLUSTER ? (int)cluster_rank() : 0;
    const int step = gridDim.x / S, unit = part * kDsWarps + warp, units = S * kDsWarps;
    // What this row's CTAs sent each other has arrived (once for each of the
    // two places in turn); false if not in time.
    uint32_t turn = 0;
    auto arrived = [&] {
        if (!CLUSTER) {
            __syncthreads();
            return true;
        }
        const uint32_t n = turn++;
        return warp_cluster_wait(&sent[n & 1], (n >> 1) & 1, kClusterWaitNs);
    };
    bool waited = !CLUSTER;
    auto ready = [&] {  // every CTA of the cluster has started
        __syncwarp();
        if (!waited) cluster_wait();
        waited = true;
    };
    rows_begin();
    if (CLUSTER) {
        if (tid == 0) {
            mbar_init(&sent[0], 1);
            mbar_init(&sent[1], 1);
            mbar_fence_init();
        }
        __syncwarp();
        cluster_arrive();
    }
    auto leave = [&] {  // no CTA ends while another may write into it
        ready();
        if (CLUSTER) {
            cluster_arrive();
            cluster_wait();
        }
    };
    auto row_of = [&](int r) { return RowView<T>(static_cast<const T*>(a.student) + (size_t)r * a.stride, a.V); };
    auto grad_of = [&](int r) { return static_cast<T*>(a.grad) + (size_t)r * a.grad_stride; };
    // The rows of this cluster in turn, those of weight zero done on the way.
    int ahead = blockIdx.x / S;
    float w = 0.0f;  // of the row that next_row gave
    auto next_row = [&] {
        for (;;) {
            const int r = ahead;
            ahead += step;
            w = a.weights && r < a.R ? a.weights[r] : 1.0f;
            if (r >= a.R || w != 0.0f) return r;
            if (warp < kDsWarps)
                distill_zero(row_of(r), grad_of(r), unit, units);
            else if (part == 0 && lane == 0)
                distill_no_row(a, r);
        }
    };
    int p = 0;
    if (warp == kDsWarps) {
#pragma unroll 1
        for (int r = next_row(); r < a.R; p ^= 1) {
            DsListed in;
            in.load(a, r);
            in.gather(a, row_of(r).row);
            const int after = next_row();
            distill_before<CLUSTER>(a, in, rows[p], &sent[p], part, S, ready);
            if (!arrived()) {  // this row and those left are refused
                if (lane == 0) set_error(a.dev_error, kDevErrTimeout | kDevErrNonfinite);
                for (; r < a.R; r += step)
                    if (part == S - 1 && lane == 0) distill_no_row(a, r);  // by who has the loss
                break;
            }
            distill_after(a, r, rows[p], part, S);
            r = after;
        }
        leave();
        return;
    }
    const DsBuffers<T> buf{reinterpret_cast<uint4*>(ds_raw) + (size_t)warp * n_buf * (kDsTileBytes / 16), full[warp]};
    int next = next_row();
    uint32_t phase = 0, pending = 0;  // of each buffer; pending: a copy was started and not awaited
    if (lane == 0) {
#pragma unroll 1
        for (int b = 0; b < n_buf; ++b) mbar_init(&full[warp][b], 1);
        mbar_fence_init();
    }
    __syncwarp();
    auto fill = [&](int r, int b) {  // buffer b with row r's tile
        if (r >= a.R) return;
        const RowView<T> row = row_of(r);
        const int t = unit + b * units;
        if (t >= tiles_of(row)) return;
        if (lane == 0) buf.copy(row, t, b);
        pending |= 1u << b;
    };
#pragma unroll 1
    for (int b = 0; b < n_buf; ++b) fill(next, b);
    int ids_next[kDsIds];
    if (next < a.R) load_ids(a, next, ids_next);
    bool ok = true;
#pragma unroll 1
    while (next < a.R) {
        const int r = next;
        const float w_row = w;
        int ids[kDsIds];
#pragma unroll
        for (int k = 0; k < kDsIds; ++k) ids[k] = ids_next[k];
        next = next_row();
        if (next < a.R) load_ids(a, next, ids_next);  // needed a row later
        const RowView<T> row = row_of(r);
        T* g = grad_of(r);
        DsRow& sm = rows[p];
        const int at_row = p;
        p ^= 1;
        const int tiles = tiles_of(row), tail0 = row.head + row.nvec * VEC;
        DsSum sum;
        float2 ends = make_float2(-INFINITY, -INFINITY);
        if (unit == 0) ends = distill_ends(row, ids, sum, a.c);
#pragma unroll 1
        for (int b = 0; b < n_buf && ok; ++b) {
            if (!((pending >> b) & 1u)) continue;
            ok = warp_mbar_wait(&full[warp][b], (phase >> b) & 1u, kCopyWaitNs);
            if (!ok) {
                if (lane == 0) set_error(a.dev_error, kDevErrTimeout);
                break;
            }
            pending &= ~(1u << b);
            phase ^= 1u << b;
            distill_tile(row, unit + b * units, buf.at(b), ids, sum, a.c, [] {});
        }
        sum.exact(a.c);
        const float2 mine = make_float2(sum.m, ok ? warp_sum_f(sum.z.x + sum.z.y) : NAN);  // a wait ran out: refused
        ready();
        if (CLUSTER) {
            if (lane < S) cluster_send(cluster_map(&sm.part[unit], lane), mine, cluster_map(&sent[at_row], lane));
        } else if (lane == 0) {
            sm.part[unit] = mine;
        }
        if (!arrived()) {  // this warp's part of this row and those left is refused
            if (lane == 0) set_error(a.dev_error, kDevErrTimeout | kDevErrNonfinite);
            ok = false;
#pragma unroll 1
            for (int k = r; k < a.R; k += step) distill_zero(row_of(k), grad_of(k), unit, units);
            break;
        }
        DsSums sums;
        const DistillStat st = distill_stat(a, sm, S, &sums);
        if (st.live == 0.0f) distill_zero(row, g, unit, units);
        const bool aligned = same_alignment(row, g);
        const DsTail tail(w_row * st.coef, st.m_tail, a.c);
        auto listed = [&](T* g0, int e0, int n) {  // overwrites what was stored for them as tail tokens
            __syncwarp();
            listed_in(ids, e0, n, [&](int k, int o) {
                const int j = lane + 32 * k;
                store_elem(g0 + o, distill_listed_grad(st, sm.s[j], st.t(sm.l[j]), a.c, (float)a.inv_t, w_row));
            });
        };
        if (st.live != 0.0f && unit == 0) {
            const float2 y = tail(ends);
            if (lane < row.head) store_elem(g + lane, y.x);
            if (lane < row.tail) store_elem(g + tail0 + lane, y.y);
            listed(g, 0, row.head);
            listed(g + tail0, tail0, row.tail);
        }
#pragma unroll 1
        for (int b = 0; b < n_buf; ++b) {
            const int t = unit + b * units;
            if (st.live != 0.0f && t < tiles) {
                const uint4* at = buf.at(b);
                const int v0 = t * kDsTile * 32;
                T* g0 = g + row.head + (size_t)v0 * VEC;
                if (aligned && v0 + kDsTile * 32 <= row.nvec) {
                    if (tail.plain) {
                        DsTail t1 = tail;
                        t1.plain = true;
#pragma unroll 4
                        for (int j = 0; j < kDsTile; ++j) t1.store<true>(g0 + (j * 32 + lane) * VEC, at[j * 32 + lane]);
                    } else {
#pragma unroll 1
                        for (int j = 0; j < kDsTile; ++j) tail.store<true>(g0 + (j * 32 + lane) * VEC, at[j * 32 + lane]);
                    }
                } else {
#pragma unroll 1
                    for (int v = lane; v < row.nvec - v0 && v < kDsTile * 32; v += 32) {
                        if (aligned)
                            tail.store<true>(g0 + v * VEC, at[v]);
                        else
                            tail.store<false>(g0 + v * VEC, at[v]);
                    }
                }
                listed(g0, row.head + v0 * VEC, min(kDsTile * 32, row.nvec - v0) * VEC);
            }
            __syncwarp();  // every lane has read it
            if (ok) fill(next, b);
        }
    }
    if (!ok && lane == 0)  // the copies still on their way land before the CTA ends
#pragma unroll 1
        for (int b = 0; b < n_buf; ++b)
            if ((pending >> b) & 1u) mbar_wait(&full[warp][b], (phase >> b) & 1u, kDrainNs);
    __syncwarp();
    leave();
}

// The gradient alone, from a row's statistics: four tiles a warp, a CTA per
// stretch of a row, no exchange.  Reads and writes an element once: 1024 rows
// of 128256 bf16 in 81 us, 0.96 of the measured copy bandwidth.
constexpr int kDbThreads = 256;
constexpr int kDbTiles = 4;  // tiles a warp takes

template <typename T>
__global__ void __launch_bounds__(kDbThreads) k_distill_backward(DistillArgs a, int stretches) {
    constexpr int VEC = ElemT<T>::VEC;
    rows_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = blockIdx.x / stretches, stretch = blockIdx.x - r * stretches;
    const int unit = stretch * (kDbThreads / 32) + warp, units = stretches * (kDbThreads / 32);
    const RowView<T> row(static_cast<const T*>(a.student) + (size_t)r * a.stride, a.V);
    T* g = static_cast<T*>(a.grad) + (size_t)r * a.grad_stride;
    const float w = a.weights ? a.weights[r] : 1.0f;
    const DistillStat st = reinterpret_cast<const DistillStat*>(a.stats)[r];
    if (w == 0.0f || st.live == 0.0f) {
        distill_zero(row, g, unit, units);
        return;
    }
    int ids[kDsIds];
    load_ids(a, r, ids);
    const bool aligned = same_alignment(row, g);
    const DsTail tail(w * st.coef, st.m_tail, a.c);
    // The listed tokens of a piece of the row: their gradients are taken
    // from the logits before put() stores over the piece (grad may be the
    // student's buffer), and stored after it.
    auto with_listed = [&](int e0, int n, auto&& put) {
        float y[kDsIds];
#pragma unroll
        for (int k = 0; k < kDsIds; ++k)
            if ((unsigned)(ids[k] - e0) < (unsigned)n) {
                const size_t j = (size_t)r * a.K + lane + 32 * k;
                const float t = st.t(a.teacher[j]);
                y[k] = distill_listed_grad(st, ElemT<T>::load(row.row + ids[k]), t, a.c, (float)a.inv_t, w);
            }
        __syncwarp();
        put();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kDsIds; ++k)
            if ((unsigned)(ids[k] - e0) < (unsigned)n) store_elem(g + ids[k], y[k]);
    };
    if (unit == 0) {
        const int tail0 = row.head + row.nvec * VEC;
        with_listed(0, row.head, [&] {
            if (lane < row.head) store_elem(g + lane, tail(make_float2(ElemT<T>::load(row.row + lane), 0.0f)).x);
        });
        with_listed(tail0, row.tail, [&] {
            if (lane < row.tail)
                store_elem(g + tail0 + lane, tail(make_float2(ElemT<T>::load(row.row + tail0 + lane), 0.0f)).x);
        });
    }
    for (int t = unit; t * kDsTile * 32 < row.nvec; t += units) {
        const int v0 = t * kDsTile * 32, nv = min(kDsTile * 32, row.nvec - v0);
        uint4 q[kDsTile];
#pragma unroll
        for (int j = 0; j < kDsTile; ++j)
            q[j] = j * 32 + lane < nv ? *(row.vec() + v0 + j * 32 + lane) : RowVec<T>::none();
        with_listed(row.head + v0 * VEC, nv * VEC, [&] {
#pragma unroll
            for (int j = 0; j < kDsTile; ++j)
                if (j * 32 + lane < nv) {
                    T* at = g + row.head + (size_t)(v0 + j * 32 + lane) * VEC;
                    if (aligned)
                        tail.store<true>(at, q[j]);
                    else
                        tail.store<false>(at, q[j]);
                }
        });
    }
}

template <typename T>
static cudaError_t launch_distill_loss(const DistillArgs& a, cudaStream_t st) {
    const int tiles = (a.V / ElemT<T>::VEC + kDsTile * 32 - 1) / (kDsTile * 32);
    const size_t dyn = (size_t)kDsWarps * kDsTileBytes;
    LaunchShape shape;
    if (!launch_shape(reinterpret_cast<const void*>(k_distill_loss<T, false>), dyn, kDsThreads, &shape) ||
        !launch_shape(reinterpret_cast<const void*>(k_distill_loss<T, true>), dyn, kDsThreads, &shape))
        return cudaErrorUnknown;
    // CTAs that share a row: more than one where rows are too few for every SM
    int S = 1;
    while (S < 8 && (long long)a.R * S < 2 * shape.sms && tiles >= 2 * S * kDsWarps) S *= 2;
    return launch_rows(S > 1 ? k_distill_loss<T, true> : k_distill_loss<T, false>, a.R, S, kDsThreads, dyn,
                       shape.sms, kDsLossPerSm, a.dev_error, st, a);
}

template <typename T>
static cudaError_t launch_distill_grad(const DistillArgs& a, cudaStream_t st) {
    const int tiles = (a.V / ElemT<T>::VEC + kDsTile * 32 - 1) / (kDsTile * 32);
    LaunchShape shape;
    const size_t most = (size_t)kDsWarps * kDsTileBytes * kDsMaxTiles;
    if (!launch_shape(reinterpret_cast<const void*>(k_distill_grad<T, false>), most, kDsThreads, &shape) ||
        !launch_shape(reinterpret_cast<const void*>(k_distill_grad<T, true>), most, kDsThreads, &shape))
        return cudaErrorUnknown;
    // CTAs that share a row: enough that three rows' parts fit on an SM (two
    // tiles a warp), so that one CTA's exchange hides behind the others'
    // copies; 16 only where 8 do not hold the row; more where rows are few.
    int S = 1;
    while (S < kDsMaxCluster && tiles > 2 * S * kDsWarps) S *= 2;
    if (S > 8 && tiles <= kDsMaxTiles * 8 * kDsWarps) S = 8;
    while (S < 8 && (long long)a.R * S < 2 * shape.sms && tiles >= 2 * S * kDsWarps) S *= 2;
    const int each = (tiles + S * kDsWarps - 1) / (S * kDsWarps);  // tiles of a warp
    const int n_buf = each > 0 ? each : 1;
    const size_t dyn = (size_t)kDsWarps * kDsTileBytes * n_buf;
    int clusters = 0;  // as many as run at once: they take rows in turn, so where each starts matters little
    if (S > 1) {
        auto* kern = k_distill_grad<T, true>;
        const cudaError_t e =
            S > 8 ? cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) : cudaSuccess;
        if (e != cudaSuccess) return e;
        if (!clusters_at_once(reinterpret_cast<const void*>(kern), S, kDsThreads, dyn, &clusters))
            return cudaErrorUnknown;
        return launch_rows(kern, clusters < a.R ? clusters : a.R, S, kDsThreads, dyn, shape.sms, 0, a.dev_error, st, a,
                           n_buf);
    }
    const int per_sm = n_buf <= 2 ? 3 : n_buf <= 3 ? 2 : 1;  // by registers, and by shared memory
    clusters = shape.sms * per_sm < a.R ? shape.sms * per_sm : a.R;
    return launch_rows(k_distill_grad<T, false>, clusters, 1, kDsThreads, dyn, shape.sms, 0, a.dev_error, st, a, n_buf);
}

template <typename T>
static cudaError_t launch_distill_backward(const DistillArgs& a, cudaStream_t st) {
    const int tiles = (a.V / ElemT<T>::VEC + kDsTile * 32 - 1) / (kDsTile * 32);
    const int per = (kDbThreads / 32) * kDbTiles, stretches = tiles > per ? (tiles + per - 1) / per : 1;
    return launch_clusters(k_distill_backward<T>, (long long)a.R * stretches, 1, kDbThreads, 0, true, st, a, stretches);
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
    if (R == 0) return clear_error(dev_error, st);
    const float c = (float)(kLog2e / (double)temperature);
    DistillArgs a{student, R, V, K, row_stride, teacher_ids, teacher_logprobs, weights,
                  c, (double)c * 0.69314718055994531, tail == SPEC_TAIL_BUCKET,
                  loss, row_stats, grad, grad_stride, dev_error};
    const bool bf16 = dtype == SPEC_BF16;
    const cudaError_t e = grad ? (bf16 ? launch_distill_grad<__nv_bfloat16>(a, st) : launch_distill_grad<float>(a, st))
                               : (bf16 ? launch_distill_loss<__nv_bfloat16>(a, st) : launch_distill_loss<float>(a, st));
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
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
    const float c = (float)(kLog2e / (double)temperature);
    DistillArgs a{student, R, V, K, row_stride, teacher_ids, teacher_logprobs, grad_loss,
                  c, (double)c * 0.69314718055994531, false, nullptr,
                  const_cast<float*>(row_stats), grad, grad_stride, nullptr};
    return (dtype == SPEC_BF16 ? launch_distill_backward<__nv_bfloat16>(a, st)
                               : launch_distill_backward<float>(a, st)) == cudaSuccess
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}
