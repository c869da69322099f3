// Attention of drafted nodes over a paged cache (spec_tree_attention).
#include <type_traits>

#include "../../include/specverify.h"
#include "paged.cuh"
#include "tcgen05.cuh"

namespace sv {

constexpr int kAtTile = 128;  // cache entries of a tile; query rows of a block
constexpr int kAtPrepNT = 256;
constexpr int kAtNT = 384;     // 2 warpgroups for the softmax, warps for keys, products, values with queries, mending
constexpr int kAtMaxCtas = 160;
constexpr int kAtMaskedTiles = kMaxDraftNodes / kAtTile + 1;  // tiles that reach behind a sequence, at most
constexpr int kAtPieces = 8;   // CTAs that join a block
constexpr int kAtFew = 4;      // parts that a thread joins by itself
constexpr int kAtShare = 4;    // CTAs that share a tile's read through L2, at most
constexpr long long kAtWaitClocks = 4000000000ll;  // two seconds
#ifndef SV_LATE_ATTEND
#define SV_LATE_ATTEND false
#endif
// Nanoseconds that a thread loses before each of its waits; a test sets it for a
// library of its own, so that roles come late to what others wait for.
#ifndef SV_SLOW_ATTEND
#define SV_SLOW_ATTEND 0
#endif

// The query rows of a request and a key head: a block has as many whole nodes as
// fit in 128 rows, row i * group + j being head h * group + j of its node i.  A
// CTA takes one or two blocks (`blocks`) of one head and a run of tiles.  The
// CTAs of a group go over the same tiles at the same time, `heads` heads beside
// each other and `share` parts of the blocks: entries of several heads lie
// together in memory, and parts read the same ones.  Work is counted in units:
// (request, set of heads, chunk of blocks, tile) in this order, shared out
// evenly among `groups` groups.
struct AttendPlan {
    int nodes;  // of a block
    int blocks, chunks, share, heads, groups;
    __host__ __device__ int ctas() const { return share * heads; }  // of a group
};

struct AttendArgs {
    int B, N, q_heads, kv_heads, group, dim;
    int cache_blocks, page, box;  // box: entries of a copy
    const int32_t* table;
    int64_t table_stride, capacity;  // capacity: positions that a table row holds
    const int32_t* lens;
    const int32_t* parent;
    int64_t parent_stride;
    const int32_t* n_nodes;
    float c;  // scale * log2(e)
    uint16_t* out;
    int32_t* dev_error;
    AttendPlan plan;
    // workspace
    int32_t* err;        // [B] error bits of a request: its lengths, later its blocks
    int32_t* tree_err;   // [B], or [1] for a shared tree: error bits of the parent array
    int32_t* first;      // [B + 1] units before a request
    int32_t* late;       // [1] SPEC_DEVERR_TIMEOUT
    uint32_t* masks;     // [B or 1][N][mask_words]: bit m of node n's words: n sees node m
    float* part;         // partial results: [CTA][2][part_floats]
    int mask_words;
};

// Nodes of a request, and whether they and its length can be served.
struct AttendRequest {
    int len, n, err;
};
__device__ __forceinline__ AttendRequest attend_request(const AttendArgs& a, int b) {
    AttendRequest r;
    r.len = a.lens[b];
    r.n = a.n_nodes ? a.n_nodes[b] : a.N;
    r.err = r.len < 0 || r.n < 0 || r.n > a.N || (int64_t)r.len + r.n > a.capacity ? kDevErrLength : 0;
    return r;
}

__device__ __forceinline__ int attend_tiles(const AttendRequest& r) {
    return r.err || r.n == 0 ? 0 : (int)(((int64_t)r.len + r.n + kAtTile - 1) / kAtTile);
}

// Before the attention: the requests' error words and units, and which nodes
// each node of a tree sees.  CTA 0 has the requests, the others a tree each.
__global__ void __launch_bounds__(kAtPrepNT) k_attend_prepare(AttendArgs a) {
    __shared__ int32_t sh_parent[kMaxDraftNodes];
    __shared__ int sh_part[kAtPrepNT / 32];
    rows_begin();
    const int tid = threadIdx.x;
    if (blockIdx.x == 0) {
        const int each = (a.B + kAtPrepNT - 1) / kAtPrepNT, b0 = min(tid * each, a.B), b1 = min(b0 + each, a.B);
        const int times = a.kv_heads / a.plan.heads * a.plan.chunks;
        int sum = 0;
        for (int b = b0; b < b1; ++b) {
            const AttendRequest r = attend_request(a, b);
            a.err[b] = r.err;
            sum += attend_tiles(r) * times;
        }
        const int upto = warp_inclusive_scan_i(sum);
        if ((tid & 31) == 31) sh_part[tid >> 5] = upto;
        __syncthreads();
        int at = upto - sum;
        for (int w = 0; w < (tid >> 5); ++w) at += sh_part[w];
        for (int b = b0; b < b1; ++b) {
            a.first[b] = at;
            at += attend_tiles(attend_request(a, b)) * times;
        }
        if (tid == kAtPrepNT - 1) {
            a.first[a.B] = at;
            *a.late = 0;
        }
        return;
    }
    const int t = blockIdx.x - 1;
    // a shared tree is checked whole; one of a request as far as its nodes go
    int n = a.N;
    if (a.parent_stride && a.n_nodes) n = min(max(a.n_nodes[t], 0), a.N);
    const int32_t* parent = a.parent + t * a.parent_stride;
    for (int i = tid; i < n; i += kAtPrepNT) sh_parent[i] = parent[i];
    const bool ok = __syncthreads_and(tree_part_ok(parent, n, tid, kAtPrepNT));
    if (tid == 0) a.tree_err[t] = ok ? 0 : kDevErrParent;
    if (!ok) return;
    for (int i = tid; i < n; i += kAtPrepNT) {
        uint32_t* words = a.masks + ((int64_t)t * a.N + i) * a.mask_words;
        int m = i;  // ancestors come in descending order: each word is written once
        for (int w = a.mask_words - 1; w >= 0; --w) {
            uint32_t bits = 0;
            for (; m >= w * 32; m = sh_parent[m]) bits |= 1u << (m & 31);
            words[w] = bits;
        }
    }
}

// A run of tiles of one (request, key head, row blocks of this CTA).
struct AttendItem {
    int b, len, n, head;
    int node0, nodes;  // this CTA's first node, and how many of its nodes there are
    int t0, t1, tiles;
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
    __device__ __forceinline__ bool masked(int t) const { return (t + 1) * (int64_t)kAtTile > len; }
    // Whether values are mended in it.  All items but a run's last one: that may end before the sequence does.
    __device__ __forceinline__ bool mends() const { return masked(t1 - 1); }
};
// Groups that have units: as many as there are units, if those are fewer.
__device__ __forceinline__ int attend_groups(const AttendArgs& a, int64_t units) {
    return units < a.plan.groups ? max((int)units, 1) : a.plan.groups;
}
// The group that has a unit.
__device__ __forceinline__ int attend_group(int64_t unit, int64_t units, int groups) {
    return (int)(((unit + 1) * groups - 1) / units);
}
// A CTA's partial results: the reference and sum of the rows of its two blocks
// (or, with one block, of its two halves of columns, alike), then four columns
// at a time of its rows.  Part 1 is the beginning of an item at the end of the
// CTA's run, part 0 what goes on from the group before.
constexpr int kAtPartSums = 2 * kAtTile;
template <int DT, int NB> constexpr int kAtPartFloats = 2 * kAtPartSums + NB * kAtTile * DT;
template <int DT, int NB>
__device__ __forceinline__ float* attend_part(const AttendArgs& a, int group, int cta, bool begins) {
    return a.part + ((int64_t)(group * a.plan.ctas() + cta) * 2 + begins) * kAtPartFloats<DT, NB>;
}
// The first requests of a CTA's run, in shared memory: what the next item is must
// not take two reads of global memory at the end of every request.
constexpr int kAtNear = 20;
struct AttendNear {
    int b0, first[kAtNear + 1], len[kAtNear], n[kAtNear];
};
// The items of a CTA, one after the other; every role walks them for itself.
struct AttendWalk {
    const AttendNear* near;
    int u, u1, b, start, next, share, head;
    int len, n, tiles;
    __device__ __forceinline__ int first(const AttendArgs& a, int b) const {
        const int i = b - near->b0;
        return i <= kAtNear ? near->first[i] : a.first[b];
    }
    __device__ __forceinline__ void request(const AttendArgs& a) {
        const int i = b - near->b0;
        len = i < kAtNear ? near->len[i] : a.lens[b];
        n = i < kAtNear ? near->n[i] : a.n_nodes ? a.n_nodes[b] : a.N;
        tiles = attend_tiles({len, n, 0});  // requests that are refused have no units
    }
    // near->b0: the request of unit u0 (any one when there are no units)
    __device__ __forceinline__ AttendWalk(const AttendArgs& a, int u0, int end, const AttendNear* requests)
        : near(requests), u(u0), u1(end), b(requests->b0) {
        const int i = blockIdx.x % a.plan.ctas();
        head = i / a.plan.share;
        share = i - head * a.plan.share;
        if (u >= u1) return;
        start = first(a, b);
        next = first(a, b + 1);
        request(a);
    }
    __device__ __forceinline__ bool item(const AttendArgs& a, AttendItem* x) {
        while (u < u1) {
            if (u >= next) {
                do {
                    ++b;
                    start = next;
                    next = first(a, b + 1);
                } while (u >= next);
                request(a);
            }
            const int at = u - start, i = at / tiles;
            x->t0 = at - i * tiles;
            x->t1 = min(tiles, x->t0 + (u1 - u));
            u += x->t1 - x->t0;
            const int set = i / a.plan.chunks, most = a.plan.blocks * a.plan.nodes;
            x->head = set * a.plan.heads + head;
            x->node0 = ((i - set * a.plan.chunks) * a.plan.share + share) * most;
            x->nodes = min(n - x->node0, most);
            if (x->nodes <= 0) continue;  // a request of fewer nodes than N
            x->b = b;
            x->len = len;
            x->n = n;
            x->tiles = tiles;
            return true;
        }
        return false;
    }
};

template <int DT> struct AttendShape {
    static constexpr int kTileBytes = kAtTile * DT * 2;      // 128 entries (or rows) of DT 16-bit values
    static constexpr int kBlockBytes = kAtTile * 128;        // 64 of their columns
    static constexpr int kStages = 5 * 128 / DT;             // 160 KiB of keys and values
    static constexpr int kQueryBytes = 2 * kTileBytes;       // two blocks, or two turns of one
    static constexpr int kTiles = kQueryBytes + kStages * kTileBytes;
    // Weights of a tile that are handed over first.  A short first part starts the product sooner; two streams of many
    // rows keep the matrix unit busy anyway.
    __host__ __device__ static constexpr int first(int blocks) { return blocks == 1 ? 32 : 64; }
    // The ring's turns of the J-th tile.  Values are needed later than keys by
    // more than a tile's time, so they come a tile later.  Turn 1 is nobody's.
    __device__ static __forceinline__ int key_turn(int J) { return 2 * J; }
    __device__ static __forceinline__ int value_turn(int J) { return 2 * J + 3; }
};
struct AttendCtrl {
    uint64_t full[10], empty[10], mend[10], mended[10];
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2], ml_full, read, judged[2], drain;
    uint32_t poison[2][kAtMaskedTiles][4];  // of every other item: entries that are not finite
    uint32_t poisoned[2];                   // whether there are any
    float2 ml[2][kAtTile];
    uint32_t tmem;
    volatile int dead;
    AttendNear near;
};
template <int DT> constexpr size_t kAttendSmem = AttendShape<DT>::kTiles + sizeof(AttendCtrl);
static_assert(kAttendSmem<128> <= 232448 && kAttendSmem<64> <= 232448, "a CTA's shared memory");

// A wait of one thread; false once it, or another of the CTA's, has run out.
__device__ __noinline__ bool attend_wait_long(AttendCtrl* c, uint64_t* bar, uint32_t parity) {
    const long long t0 = clock64();  // a read of the global timer takes longer than most waits here
    while (!mbar_test(bar, parity)) {
        if (c->dead) return false;
        if (clock64() - t0 > kAtWaitClocks) {
            c->dead = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool attend_wait(AttendCtrl* c, uint64_t* bar, uint32_t parity) {
    if (SV_LATE_ATTEND) {
        c->dead = 1;
        return false;
    }
    if (SV_SLOW_ATTEND) __nanosleep(SV_SLOW_ATTEND);
    return mbar_test(bar, parity) || attend_wait_long(c, bar, parity);
}
__device__ __forceinline__ bool attend_wait_warp(AttendCtrl* c, uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, attend_wait(c, bar, parity));
}
__device__ __forceinline__ void attend_arrive_warp(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bit i: whether a node sees position base + i of those behind the sequence
// (base < 0: the sequence's own, which every node sees).
__device__ __forceinline__ uint32_t attend_sees(const AttendArgs& a, const uint32_t* mask, int node, int base) {
    if (base <= -32) return 0xffffffffu;
    if (!a.parent) {
        const int upto = node - base + 1;
        return upto >= 32 ? 0xffffffffu : upto <= 0 ? 0u : (1u << upto) - 1u;
    }
    auto word = [&](int i) { return i < a.mask_words ? mask[i] : 0u; };
    if (base < 0) return ((1u << -base) - 1u) | (word(0) << -base);
    return __funnelshift_r(word(base >> 5), word((base >> 5) + 1), base & 31);
}

// The warps that copy keys (KV = 0) and values (1) of each tile into the ring,
// the tile's pages one by one.  Blocks behind the last position are not looked
// up: the copy reads outside the cache there, which gives zeros.  (One warp for
// both took 3900 clocks a tile of eight pages, 75 a copy, and the products
// waited.)
//
// The warp of the values copies the queries, too, between an item's last values
// and the next one's first: one box of a block's nodes and heads for every 64
// columns; nodes behind the last read as zeros or as rows that nothing is
// written for.
template <int DT, int NB, int KV>
__device__ __forceinline__ void attend_copy(const AttendArgs& a, const CUtensorMap* map, const CUtensorMap* qm,
                                            AttendWalk walk, AttendCtrl* c, uint32_t queries, uint32_t ring) {
    using S = AttendShape<DT>;
    constexpr int kCopies = kAtTile / 32 * (DT / 64);  // of a lane, at most
    // a lane takes every 32nd of the tile's copies, (box, 64 columns) each
    constexpr int kWide = DT / 64;
    const uint32_t lane = threadIdx.x & 31, boxes = kAtTile / a.box, copies = boxes * kWide, per = a.page / a.box;
    AttendItem x{};
    int J = 0;
    bool ok = true;
    int block[kCopies], entry[kCopies];
    auto look_up = [&](int t) {
        const uint32_t end = (uint32_t)x.len + x.n;  // below 2^31 + 1024
#pragma unroll
        for (uint32_t k = 0; k < kCopies; ++k) {
            if (k * 32 >= copies) break;
            const uint32_t i = (uint32_t)t * boxes + (lane + 32 * k) / kWide;  // box of the sequence
            block[k] = a.cache_blocks;
            entry[k] = 0;
            if (lane + 32 * k < copies && i * a.box < end) {
                const uint32_t j = i / per;
                block[k] = a.table[x.b * a.table_stride + j];
                entry[k] = (int)((i - j * per) * a.box);
                if ((uint32_t)block[k] >= (uint32_t)a.cache_blocks) block[k] = -1;
            }
        }
    };
    // with two turns of queries the next item's are on their way during this one, with one they wait for its end
    constexpr int kTurns = NB == 1 ? 2 : 1;
    int qi = 0;
    auto copy_queries = [&](const AttendItem& x) {
        const int turn = qi % kTurns, use = qi / kTurns;
        ++qi;
        if (use > 0 && !attend_wait_warp(c, &c->q_empty[turn], (use - 1) & 1)) return false;
        if (lane == 0) {
            mbar_arrive_expect_tx(&c->q_full[turn], NB * kWide * a.plan.nodes * a.group * 128);
            for (int w = 0; w < NB; ++w)
                for (int d = 0; d < kWide; ++d)
                    tma_load_4d(queries + (turn + w) * S::kTileBytes + d * S::kBlockBytes, qm, d * 64, x.head * a.group,
                                x.node0 + w * a.plan.nodes, x.b, &c->q_full[turn]);
        }
        return true;
    };
    AttendItem ahead;
    AttendWalk walk_ahead = walk;
    if (KV == 1 && NB == 1 && walk_ahead.item(a, &ahead)) ok = copy_queries(ahead);
    while (ok && walk.item(a, &x)) {
        look_up(x.t0);
        if (KV == 1) {
            if (NB == 2) ok = copy_queries(x);
            else if (walk_ahead.item(a, &ahead)) ok = copy_queries(ahead);
        }
        for (int t = x.t0; ok && t < x.t1; ++t) {
            int to_block[kCopies], to_entry[kCopies];
#pragma unroll
            for (uint32_t k = 0; k < kCopies; ++k) {
                if (k * 32 >= copies) break;
                if (lane + 32 * k < copies && block[k] < 0) {
                    if (KV == 0) atomicOr(a.err + x.b, kDevErrCapacity);
                    block[k] = a.cache_blocks;
                }
                to_block[k] = block[k];
                to_entry[k] = entry[k];
            }
            if (t + 1 < x.t1) look_up(t + 1);  // on its way while the ring is waited for
            const int turn = KV ? S::value_turn(J) : S::key_turn(J), slot = turn % S::kStages, use = turn / S::kStages;
            if (use > 0 && !attend_wait_warp(c, &c->empty[slot], (use - 1) & 1)) {
                ok = false;
                break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&c->full[slot], S::kTileBytes);
            __syncwarp();
#pragma unroll
            for (uint32_t k = 0; k < kCopies; ++k) {
                if (k * 32 >= copies) break;
                const uint32_t i = lane + 32 * k, d = i % kWide;
                if (i < copies)
                    tma_load_4d(ring + slot * S::kTileBytes + d * S::kBlockBytes + i / kWide * a.box * 128, map, d * 64, x.head,
                                to_entry[k], to_block[k], &c->full[slot]);
            }
            if (KV == 1 && lane == 0 && x.masked(t)) mbar_arrive(&c->mend[slot]);
            ++J;
        }
    }
    // Nothing is on its way into shared memory when the CTA ends: this warp's
    // copies into slots that no later turn has had (turn + kStages).
    constexpr int kLast = S::kStages % 2 == 0 ? S::kStages / 2 : KV ? (S::kStages + 3) / 2 : (S::kStages - 3) / 2;
    for (int j = max(0, J - kLast); j < J; ++j) {
        const int turn = KV ? S::value_turn(j) : S::key_turn(j);
        if (!mbar_wait(&c->full[turn % S::kStages], (turn / S::kStages) & 1, kDrainNs)) break;
    }
    for (int i = max(0, qi - kTurns); i < qi; ++i)
        if (!mbar_wait(&c->q_full[i % kTurns], (i / kTurns) & 1, kDrainNs)) break;
    __syncwarp();
}

// The matrix warp.  Stream w: the products with S, P and O of warpgroup w.
// NB = 2: both streams take every tile, each for its own block of rows; S of a
// stream's next tile follows its product with the values of the tile before, so
// a warpgroup's softmax runs beside the other stream's products.
// NB = 1: the streams take turns, and what comes first is done first: scores as
// soon as the keys are there, a product as soon as its weights are.  An item's
// first scores do not wait for the last one's products.
template <typename T, int DT, int NB>
__device__ __forceinline__ void attend_products(const AttendArgs& a, AttendWalk walk, AttendCtrl* c, uint32_t queries,
                                                uint32_t ring, uint32_t tmem) {
    using S = AttendShape<DT>;
    constexpr bool kBf16 = !std::is_same<T, __half>::value;
    constexpr int kFirst = S::first(NB);
    constexpr uint32_t kScores = mma_shape<kBf16>(kAtTile, false), kValues = mma_shape<kBf16>(DT, true);
    const bool leader = elect_lane();
    uint32_t mended = 0;           // parity of each slot's next mending
    uint32_t weights[2] = {0, 0};  // parity of p_full
    bool ok = true;
    // O_w (+)= P_w V of tile J
    auto product = [&](int w, bool masked, int J, bool add, bool wait_values) {
        const int slot = S::value_turn(J) % S::kStages;
        const uint32_t v = uniform(mma_operand(ring + slot * S::kTileBytes, S::kBlockBytes));
        if (wait_values) {
            if (!attend_wait_warp(c, &c->full[slot], S::value_turn(J) / S::kStages & 1)) return false;
            if (masked) {
                if (!attend_wait_warp(c, &c->mended[slot], (mended >> slot) & 1u)) return false;
                mended ^= 1u << slot;
            }
        }
#pragma unroll
        for (int k = 0; k < kAtTile / 16; ++k) {
            if (k == 0 || k == kFirst / 16) {  // the weights come in two parts
                if (!attend_wait_warp(c, &c->p_full[w][k != 0], weights[w])) return false;
                tmem_fence_after();
            }
            mma_tensor(tmem + 256 + w * DT, tmem + w * 128 + k * 8, v + k * (2048 / 16), kValues, add || k > 0, leader);
        }
        weights[w] ^= 1u;
        return true;
    };
    auto values_done = [&](int J) { mma_commit(&c->empty[S::value_turn(J) % S::kStages], leader); };
    auto keys = [&](int J) { return &c->full[S::key_turn(J) % S::kStages]; };
    auto keys_parity = [&](int J) { return (uint32_t)(S::key_turn(J) / S::kStages & 1); };
    auto keys_at = [&](int J) { return uniform(mma_operand(ring + S::key_turn(J) % S::kStages * S::kTileBytes, 16)); };
    auto scores = [&](int w, uint32_t q, uint32_t k0) {
#pragma unroll
        for (int k = 0; k < DT / 16; ++k) {
            const uint32_t at = ((k / 4) * S::kBlockBytes + (k % 4) * 32) / 16;
            mma_shared(tmem + w * 128, q + at, k0 + at, kScores, k > 0, leader);
        }
        mma_commit(&c->s_full[w], leader);
    };
    if (NB == 1) {
        // s: the tile whose scores come next, p: whose product; p <= s <= p + 2, and s may be an item ahead
        AttendItem xs, xp;
        AttendWalk walk_p = walk;
        bool more_s = walk.item(a, &xs), more_p = walk_p.item(a, &xp);
        int s = 0, p = 0, ts = xs.t0, tp = xp.t0, qi = 0, ready = -1;
        long long since = clock64();
        while (ok && more_p) {
            const int w = p & 1;
            if (p < s && __all_sync(0xffffffffu, mbar_test(&c->p_full[w][0], weights[w]))) {
                // after a wait that ran out nothing is given back: a second arrival in a slot's turn is a fault
                ok = product(w, xp.masked(tp), p, tp - xp.t0 >= 2, true);
                if (!ok) break;
                values_done(p);
                if (tp >= xp.t1 - 2) mma_commit(&c->o_full[w], leader);
                ++p;
                if (++tp == xp.t1) {
                    more_p = walk_p.item(a, &xp);
                    tp = xp.t0;
                }
            } else if (more_s && s < p + 2 &&
                       (ready == qi || __all_sync(0xffffffffu, mbar_test(&c->q_full[qi & 1], (qi >> 1) & 1))) &&
                       __all_sync(0xffffffffu, mbar_test(keys(s), keys_parity(s)))) {
                ready = qi;  // this item's queries are there
                tmem_fence_after();
                scores(s & 1, uniform(mma_operand(queries + (qi & 1) * S::kTileBytes, 16)), keys_at(s));
                mma_commit(&c->empty[S::key_turn(s) % S::kStages], leader);
                ++s;
                if (++ts == xs.t1) {
                    mma_commit(&c->q_empty[qi & 1], leader);
                    ++qi;
                    more_s = walk.item(a, &xs);
                    ts = xs.t0;
                }
            } else {
                if (__any_sync(0xffffffffu, c->dead != 0 || clock64() - since > kAtWaitClocks)) {
                    c->dead = 1;
                    ok = false;
                }
                continue;
            }
            since = clock64();
        }
    } else {
        AttendItem x;
        for (int J = 0, qi = 0; ok && walk.item(a, &x); ++qi) {
            if (!attend_wait_warp(c, &c->q_full[0], qi & 1)) break;
            tmem_fence_after();
            const int n = x.t1 - x.t0, streams = x.nodes > a.plan.nodes ? 2 : 1;
            for (int j = 0; ok && j <= n; ++j)
                for (int w = 0; ok && w < streams; ++w) {
                    // the values' product goes first: it gives back the slot that a coming tile waits for
                    if (j >= 1) {
                        ok = product(w, x.masked(x.t0 + j - 1), J + j - 1, j >= 2, w == 0);
                        if (!ok) break;
                        if (w == streams - 1) values_done(J + j - 1);
                    }
                    if (j == n) {
                        mma_commit(&c->o_full[w], leader);
                        continue;
                    }
                    if (w == 0 && !(ok = attend_wait_warp(c, keys(J + j), keys_parity(J + j)))) break;
                    scores(w, uniform(mma_operand(queries + w * S::kTileBytes, 16)), keys_at(J + j));
                    if (w == streams - 1) {
                        mma_commit(&c->empty[S::key_turn(J + j) % S::kStages], leader);
                        if (j == n - 1) mma_commit(&c->q_empty[0], leader);
                    }
                }
            J += n;
        }
    }
    // no product is on its way when tensor memory is freed
    mma_commit(&c->drain, leader);
    mbar_wait(&c->drain, 0, kDrainNs);
    __syncwarp();
}

// The mending warp: in tiles that reach behind the sequence, values that no
// product may meet.  A weight of zero does not hide an infinity or a NaN, so
// entries behind the last node, and nodes' entries that are not finite, become
// zeros; the latter's places are kept for the item's end, where the rows that
// see them become NaN.
template <typename T, int DT>
__device__ __forceinline__ void attend_mend(const AttendArgs& a, AttendWalk walk, AttendCtrl* c, uint8_t* ring) {
    using S = AttendShape<DT>;
    const int lane = threadIdx.x & 31;
    AttendItem x;
    bool ok = true;
    uint32_t parity = 0;  // of each slot's next tile to mend
    for (int J = 0, item = 0; ok && walk.item(a, &x); ++item) {
        // An item without mending is the run's last.  Nobody would hold its end back for a warp that still waits for
        // the item two before, whose phase of `judged` would then be taken for the one not yet over: it has none.
        if (!x.mends()) break;
        const int turn = item & 1, use = item >> 1;
        // every item's end in order, so that none is taken for another
        if (use > 0 && !attend_wait_warp(c, &c->judged[turn], (use - 1) & 1)) break;
        if (lane == 0) c->poisoned[turn] = 0;
        for (int t = x.t0; ok && t < x.t1; ++t, ++J) {
            if (!x.masked(t)) continue;
            // This warp does not follow the ring.  Once the copy warp has named
            // the slot, its turn cannot end before it is mended.
            const int index = S::value_turn(J), slot = index % S::kStages;
            ok = attend_wait_warp(c, &c->mend[slot], (parity >> slot) & 1u) &&
                 attend_wait_warp(c, &c->full[slot], (index / S::kStages) & 1);
            if (!ok) break;
            parity ^= 1u << slot;
#pragma unroll 1
            for (int k = 0; k < kAtTile / 32; ++k) {
                const int row = k * 32 + lane;
                const int64_t node = (int64_t)t * kAtTile + row - x.len;
                bool bad = false;
                uint8_t* at = ring + slot * S::kTileBytes + row * 128;
                if (node >= 0 && node < x.n) {
                    float sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < DT / 8; ++i) {
                        const uint4 v = *reinterpret_cast<const uint4*>(at + (i / 8) * S::kBlockBytes +
                                                                        (((i % 8) ^ (row % 8)) * 16));
                        // 0 times an infinity or a NaN is NaN
                        const float2 p = Pair<T>::get(v.x), q = Pair<T>::get(v.y), r = Pair<T>::get(v.z),
                                     s = Pair<T>::get(v.w);
                        sum += (p.x * 0.0f + p.y * 0.0f) + (q.x * 0.0f + q.y * 0.0f) + (r.x * 0.0f + r.y * 0.0f) +
                               (s.x * 0.0f + s.y * 0.0f);
                    }
                    bad = sum != 0.0f;
                }
                if (bad || node >= x.n) {
#pragma unroll
                    for (int i = 0; i < DT / 8; ++i)
                        *reinterpret_cast<uint4*>(at + (i / 8) * S::kBlockBytes + (((i % 8) ^ (row % 8)) * 16)) =
                            make_uint4(0, 0, 0, 0);
                }
                const uint32_t all = __ballot_sync(0xffffffffu, bad);
                if (lane == 0) {
                    c->poison[turn][t - x.len / kAtTile][k] = all;
                    if (all) c->poisoned[turn] = 1;
                }
            }
            fence_async_shared();
            attend_arrive_warp(&c->mended[slot]);
        }
    }
}

// A warpgroup of the softmax: a thread has a query row.  The scores of a tile
// come from tensor memory, the weights go back over them in 16 bits.  The
// reference of the exponentials follows the running maximum only when that has
// grown by more than 8 (in powers of two), so that O is rarely scaled; sums and
// outputs stay in 32 bits.  Weights are rounded to the type because the matrix
// unit takes nothing wider beside values of 16 bits: half a step each, so that a
// result is off by 1.4 times its own rounding.  The row's sum is of the weights
// before that.  In fp16 weights below 2^-14 of the reference are subnormal, off
// by 2^-25; the reference is never above the row's maximum.
template <typename T, int DT, int NB>
__device__ __forceinline__ void attend_softmax(const AttendArgs& a, AttendWalk walk, AttendCtrl* c, uint32_t tmem) {
    const int w = threadIdx.x >> 7, lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    const int row = quarter * 32 + lane;  // of the block
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_at = tmem + lanes + w * 128;
    uint32_t scored = 0, done[2] = {0, 0}, met = 0;  // parities
    int J = 0;
    AttendItem x;
    for (int item = 0; walk.item(a, &x); ++item) {
        const int n = x.t1 - x.t0, J0 = J, first = NB == 2 ? w * a.plan.nodes : 0;  // the block's first node in the item
        const int live_rows = min(x.nodes - first, a.plan.nodes) * a.group;
        if (NB == 2 && live_rows <= 0) {  // the second block is empty
            J += n;
            // Nothing else holds this warpgroup back: it must not arrive for an item before the one two before it is over,
            // or it alone would count for both.
            if (x.mends()) {
                if (item >= 2 && !attend_wait_warp(c, &c->judged[item & 1], ((item >> 1) - 1) & 1)) return;
                attend_arrive_warp(&c->judged[item & 1]);
            }
            continue;
        }
        const bool live = quarter * 32 < live_rows;  // this warp has a row
        const int at_node = min(row, live_rows - 1) / a.group, node = x.node0 + first + at_node;
        const uint32_t* mask =
            a.parent ? a.masks + ((int64_t)(a.parent_stride ? x.b : 0) * a.N + node) * a.mask_words : nullptr;
        float m = kNoMax;
        float2 l = make_float2(0.0f, 0.0f);  // two sums of a row's weights
        bool begun = false;
        for (int t = x.t0; t < x.t1; ++t, ++J) {
            if (NB == 1 && (J & 1) != w) continue;
            const bool masked = x.masked(t);
            uint32_t sees[4];  // on their way while the scores are waited for
            if (masked && live) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t base = (int64_t)t * kAtTile + i * 32 - x.len;
                    sees[i] = attend_sees(a, mask, node, base < -32 ? -32 : (int)base);
                }
            }
            if (!attend_wait_warp(c, &c->s_full[w], scored)) return;
            scored ^= 1u;
            tmem_fence_after();
            if (live) {
                float s[kAtTile];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_load32(s_at + i * 32, reinterpret_cast<uint32_t*>(s) + i * 32);
                tmem_wait_load();
                if (masked) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) s[i * 32 + k] = (sees[i] >> k) & 1u ? s[i * 32 + k] : -INFINITY;
                    }
                }
                float top[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) top[i] = s[i];
#pragma unroll
                for (int i = 4; i < kAtTile; i += 8) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) top[k] = fmaxf(top[k], i + k + 4 < kAtTile ? fmaxf(s[i + k], s[i + k + 4]) : s[i + k]);
                }
                const float most = fmaxf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), m);
                const bool grows = (most - m) * a.c > 8.0f;
                if (__any_sync(0xffffffffu, grows)) {
                    const float f = grows ? exp2_fast((m - most) * a.c) : 1.0f;
                    if (grows) m = most;
                    l.x *= f;
                    l.y *= f;
                    if (begun) {
                        const uint32_t o_at = tmem + lanes + 256 + w * DT;
#pragma unroll 1
                        for (int i = 0; i < DT / 8; ++i) {
                            uint32_t o[8];
                            tmem_load8(o_at + i * 8, o);
                            tmem_wait_load();
#pragma unroll
                            for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_store8(o_at + i * 8, o);
                        }
                    }
                }
                // nothing seen yet: every score is -inf, and so is its exponent
                const float off = m == kNoMax ? 0.0f : -m * a.c;
                const float2 cc = make_float2(a.c, a.c), oo = make_float2(off, off);
                float2 part[4] = {l, {0.0f, 0.0f}, {0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t p[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float2 e = __ffma2_rn(make_float2(s[i * 32 + 2 * k], s[i * 32 + 2 * k + 1]), cc, oo);
                        e = make_float2(exp2_fast(e.x), exp2_fast(e.y));
                        part[k & 3] = __fadd2_rn(part[k & 3], e);
                        p[k] = Pair<T>::put(e.x, e.y);
                    }
                    tmem_store16(s_at + i * 16, p);
                    if (i == AttendShape<DT>::first(NB) / 32 - 1) {  // the product with the tile's first values may begin
                        tmem_wait_store();
                        tmem_fence_before();
                        attend_arrive_warp(&c->p_full[w][0]);
                    }
                }
                l = __fadd2_rn(__fadd2_rn(part[0], part[1]), __fadd2_rn(part[2], part[3]));
                tmem_wait_store();
            } else {
                attend_arrive_warp(&c->p_full[w][0]);
            }
            begun = true;
            tmem_fence_before();
            attend_arrive_warp(&c->p_full[w][1]);
        }
        // the item's end
        float total = l.x + l.y;
        float f[2] = {1.0f, 0.0f};  // factors of the streams' outputs
        const bool used[2] = {n >= 2 || (J0 & 1) == 0, n >= 2 || (J0 & 1) == 1};
        if (NB == 1) {
            c->ml[w][row] = make_float2(m, total);
            attend_arrive_warp(&c->ml_full);
            if (!attend_wait_warp(c, &c->ml_full, met)) return;
            const float2 p = c->ml[0][row], q = c->ml[1][row];
            m = fmaxf(p.x, q.x);
            f[0] = used[0] ? exp2_fast((p.x - m) * a.c) : 0.0f;
            f[1] = used[1] ? exp2_fast((q.x - m) * a.c) : 0.0f;
            total = (used[0] ? p.y * f[0] : 0.0f) + (used[1] ? q.y * f[1] : 0.0f);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (used[i]) {
                    if (!attend_wait_warp(c, &c->o_full[i], done[i])) return;
                    done[i] ^= 1u;
                }
        } else {
            if (!attend_wait_warp(c, &c->o_full[w], done[0])) return;
            done[0] ^= 1u;
        }
        tmem_fence_after();
        // every tile's values are mended by now
        if (x.mends() && c->poisoned[item & 1])
            for (int t = max(x.t0, x.len / kAtTile); t < x.t1; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t base = (int64_t)t * kAtTile + i * 32 - x.len;
                    if (attend_sees(a, mask, node, base < -32 ? -32 : (int)base) & c->poison[item & 1][t - x.len / kAtTile][i])
                        total = NAN;
                }
        if (x.mends()) attend_arrive_warp(&c->judged[item & 1]);
        if (live) {
            const bool there = row < live_rows;
            constexpr int kCols = NB == 1 ? DT / 2 : DT;  // of this thread
            const int col0 = NB == 1 ? w * kCols : 0, rows = NB * kAtTile, at_row = (NB == 2 ? w * kAtTile : 0) + row;
            const uint32_t o_at = tmem + lanes + 256 + (NB == 2 ? w * DT : 0);
            float* part = a.part + ((int64_t)blockIdx.x * 2 + (x.t0 == 0)) * kAtPartFloats<DT, NB>;
            if (!x.whole() && there) reinterpret_cast<float2*>(part)[w * kAtTile + row] = make_float2(m, total);
            float4* part_o = reinterpret_cast<float4*>(part + 2 * kAtPartSums) + at_row;
            const float inv = 1.0f / total;
            uint16_t* out = a.out + (((int64_t)x.b * a.N + node) * a.q_heads + x.head * a.group + (row - at_node * a.group)) * a.dim;
#pragma unroll 1
            for (int i = 0; i < kCols / 16; ++i) {
                const int col = col0 + i * 16;
                float o[16];
                tmem_load16(o_at + col, reinterpret_cast<uint32_t*>(o));
                if (NB == 1) {
                    float o1[16];
                    tmem_load16(o_at + DT + col, reinterpret_cast<uint32_t*>(o1));
                    tmem_wait_load();
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = (used[0] ? o[k] * f[0] : 0.0f) + (used[1] ? o1[k] * f[1] : 0.0f);
                } else {
                    tmem_wait_load();
                }
                if (there && x.whole()) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint4 v;
                        v.x = Pair<T>::put(o[k * 8] * inv, o[k * 8 + 1] * inv);
                        v.y = Pair<T>::put(o[k * 8 + 2] * inv, o[k * 8 + 3] * inv);
                        v.z = Pair<T>::put(o[k * 8 + 4] * inv, o[k * 8 + 5] * inv);
                        v.w = Pair<T>::put(o[k * 8 + 6] * inv, o[k * 8 + 7] * inv);
                        if (col + k * 8 < a.dim) *reinterpret_cast<uint4*>(out + col + k * 8) = v;
                    }
                } else if (there) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        part_o[(col / 4 + k) * rows] = make_float4(o[k * 4], o[k * 4 + 1], o[k * 4 + 2], o[k * 4 + 3]);
                }
                __syncwarp();  // the next columns are loaded by the whole warp
            }
        }
        if (NB == 1) {
            // the other warpgroup's next weights let its O be written again
            tmem_fence_before();
            attend_arrive_warp(&c->read);
            if (!attend_wait_warp(c, &c->read, met)) return;
            met ^= 1u;
        }
    }
}

// softmax(scale q K^T) V for blocks of 128 query rows against tiles of 128
// entries, on the tensor cores: S = Q K^T with both operands in shared memory
// and S in tensor memory; weights 2^((s - m) c) in 16 bits over S; O += P V with
// P read from tensor memory and O kept there.  One persistent CTA an SM, its
// roles on warps of their own, joined by mbarriers: copies, products and softmax
// overlap, within an item and from one to the next.
// Bound, with few rows a head, by memory: 64 requests of 5 nodes at lengths of
// 2048 to 8192, 8 heads of 128, pages of 16: 256 us, 5.3 TB/s or 0.78 of the copy
// rate; two sequences of 32768 and 131072: 128 us, 0.77 (the runs' ends and the
// other two launches are 15 us of it).  With many rows by the chain of S, softmax
// and P V: 32 requests of 60 nodes (480 rows a head): 285 us, 1.13 PFLOP/s or 0.59
// of the measured bf16 rate; a tile takes 2800 clocks where its products take 2048.
// Found on the way (us for these three cases): a CTA per query row on CUDA cores
// 17341, 38333, 93667; this scheme 400, 158, 453; values' products before the next
// keys are waited for, 32-bit page look-ups a tile ahead and waits timed by the
// SM's clock (the global timer's read takes longer than the wait) 330, 131, 402; a
// copy warp each for keys and values 283, 133, 372; products by a whole warp 308,
// 141, 354; an item's scores beside the last one's products, joins by runs' ends
// 273, 136, 337; a group's CTAs on neighbouring heads 272, 132, 329; queries by
// tiled copies from the values' warp, masks read ahead 269, 132, 314; operands
// known to be uniform 268, 133, 289; a short first part of the weights 256, 128.
template <typename T, int DT, int NB>
__global__ void __launch_bounds__(kAtNT, 1)
    k_attend(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap qm,
             const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm) {
    using S = AttendShape<DT>;
    extern __shared__ __align__(1024) uint8_t sh_attend[];
    AttendCtrl* c = reinterpret_cast<AttendCtrl*>(sh_attend + S::kTiles);
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&c->full[i], 1);
            mbar_init(&c->empty[i], 1);
            mbar_init(&c->mend[i], 1);
            mbar_init(&c->mended[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c->q_full[i], 1);
            mbar_init(&c->q_empty[i], 1);
            mbar_init(&c->s_full[i], 1);
            mbar_init(&c->p_full[i][0], 4);  // warps of a warpgroup
            mbar_init(&c->p_full[i][1], 4);
            mbar_init(&c->o_full[i], 1);
        }
        mbar_init(&c->ml_full, 8);
        mbar_init(&c->read, 8);
        mbar_init(&c->judged[0], 8);
        mbar_init(&c->judged[1], 8);
        mbar_init(&c->drain, 1);
        c->dead = 0;
        c->near.b0 = 0;
        mbar_fence_init();
        mbar_arrive(&c->full[1]);  // turn 1 is over
        mbar_arrive(&c->empty[1]);
        tma_prefetch_map(&qm);
        tma_prefetch_map(&km);
        tma_prefetch_map(&vm);
    }
    if (warp == 8) tmem_alloc_all(&c->tmem);
    rows_begin();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = c->tmem, queries = smem_addr(sh_attend), ring = queries + S::kQueryBytes;
    const int64_t units = a.first[a.B];
    const int g = blockIdx.x / a.plan.ctas();
    const int groups = attend_groups(a, units);
    const int u0 = (int)(units * min(g, groups) / groups), u1 = (int)(units * min(g + 1, groups) / groups);
    if (u0 < u1)
        for (int b = tid; b < a.B; b += kAtNT)
            if (a.first[b] <= u0 && u0 < a.first[b + 1]) c->near.b0 = b;
    __syncthreads();
    if (tid <= kAtNear) {
        const int b = c->near.b0 + tid;
        if (b <= a.B) c->near.first[tid] = a.first[b];
        if (tid < kAtNear && b < a.B) {
            c->near.len[tid] = a.lens[b];
            c->near.n[tid] = a.n_nodes ? a.n_nodes[b] : a.N;
        }
    }
    __syncthreads();
    const AttendWalk walk(a, u0, u1, &c->near);
    if (warp < 8) {
        attend_softmax<T, DT, NB>(a, walk, c, tmem);
    } else if (warp == 8) {
        attend_copy<DT, NB, 0>(a, &km, &qm, walk, c, queries, ring);
    } else if (warp == 9) {
        attend_products<T, DT, NB>(a, walk, c, queries, ring, tmem);
    } else if (warp == 10) {
        attend_copy<DT, NB, 1>(a, &vm, &qm, walk, c, queries, ring);
    } else {
        attend_mend<T, DT>(a, walk, c, sh_attend + S::kQueryBytes);
    }
    tmem_fence_before();
    __syncthreads();
    if (tid == 0 && c->dead) *a.late = kDevErrTimeout;
    if (warp == 8) {
        tmem_fence_after();
        tmem_free_all(tmem);
    }
}

// Joins the results of an item that several groups share: a CTA takes an eighth
// of a block's (row, four columns) pairs.  (The warps that wrote a row's parts,
// the last one at a time, took as long again as this launch: a lane has a row
// to itself there.)  The threads that share a row find its
// reference and sum together, in the same order everywhere.
template <typename T, int DT, int NB>
__device__ __forceinline__ void attend_join(const AttendArgs& a, int g0, int cta, int w, int piece, int* sh) {
    const int tid = threadIdx.x;
    const int64_t units = a.first[a.B];
    const int groups = attend_groups(a, units);
    if (g0 + 1 >= groups) return;
    // the item at the end of group g0's run, if it goes on and began in it
    const int64_t run = units * g0 / groups, next = units * (g0 + 1) / groups;
    for (int b = tid; b < a.B; b += kAtPrepNT)
        if (a.first[b] < next && next <= a.first[b + 1]) *sh = b;  // the request of unit next - 1
    __syncthreads();
    const int b = *sh;
    if (a.err[b] | (a.parent ? a.tree_err[a.parent_stride ? b : 0] : 0)) return;  // it gets zeros
    const AttendRequest r = attend_request(a, b);
    const int tiles = attend_tiles(r), i = (int)(next - 1 - a.first[b]) / tiles;
    const int64_t begin = a.first[b] + (int64_t)i * tiles, end = begin + tiles;
    if (end <= next || begin < run) return;
    const int set = i / a.plan.chunks, beside = cta / a.plan.share, share = cta - beside * a.plan.share;
    const int head = set * a.plan.heads + beside, block = ((i - set * a.plan.chunks) * a.plan.share + share) * NB + w;
    const int node0 = block * a.plan.nodes, rows = min(r.n - node0, a.plan.nodes) * a.group;
    if (rows <= 0) return;
    const int g1 = attend_group(end - 1, units, groups), count = g1 - g0 + 1;
    constexpr int R = NB * kAtTile;
    auto part = [&](int g) { return attend_part<DT, NB>(a, g, cta, g == g0); };
    const int pairs = rows * (a.dim / 4), each = (pairs + kAtPieces - 1) / kAtPieces, last = min(pairs, (piece + 1) * each);
    auto write = [&](int row, int d, float4 o, float l) {
        const float inv = 1.0f / l;
        const int node = row / a.group;
        uint2 v;
        v.x = Pair<T>::put(o.x * inv, o.y * inv);
        v.y = Pair<T>::put(o.z * inv, o.w * inv);
        *reinterpret_cast<uint2*>(a.out + (((int64_t)b * a.N + node0 + node) * a.q_heads + head * a.group + (row - node * a.group)) * a.dim +
                                  d * 4) = v;
    };
    if (count <= kAtFew) {
        // mostly two parts: all that a pair needs is on its way at once
        for (int k = piece * each + tid; k < last; k += kAtPrepNT) {
            const int d = k / rows, row = k - d * rows, at = w * kAtTile + row;
            float2 ml[kAtFew];
            float4 v[kAtFew];
#pragma unroll
            for (int i = 0; i < kAtFew; ++i) {
                ml[i] = make_float2(kNoMax, 0.0f);
                v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (i >= count) continue;
                const float* p = part(g0 + i);
                ml[i] = reinterpret_cast<const float2*>(p)[at];
                v[i] = reinterpret_cast<const float4*>(p + 2 * kAtPartSums)[d * R + at];
            }
            float m = kNoMax, l = 0.0f;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < kAtFew; ++i) m = fmaxf(m, ml[i].x);
#pragma unroll
            for (int i = 0; i < kAtFew; ++i) {
                if (i >= count) continue;
                const float f = exp2f((ml[i].x - m) * a.c);
                l += f * ml[i].y;
                o = make_float4(o.x + f * v[i].x, o.y + f * v[i].y, o.z + f * v[i].z, o.w + f * v[i].w);
            }
            write(row, d, o, l);
        }
        return;
    }
    // as many threads for a pair as are to spare, each with every so many-th part
    int beside_pair = 1;
    while (beside_pair < 32 && beside_pair < count && each * beside_pair * 2 <= kAtPrepNT) beside_pair *= 2;
    const int lane = tid & (beside_pair - 1), per = kAtPrepNT / beside_pair;
    for (int k0 = piece * each; k0 < last; k0 += per) {  // the same turns for every thread
        const int k = min(k0 + tid / beside_pair, last - 1);
        const int d = k / rows, row = k - d * rows;
        // with one block a part's sums are there twice, alike
        const int at = w * kAtTile + row;
        float m = kNoMax, l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int g = g0 + lane; g <= g1; g += beside_pair) m = fmaxf(m, reinterpret_cast<const float2*>(part(g))[at].x);
        for (int s = 1; s < beside_pair; s *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
#pragma unroll 4
        for (int g = g0 + lane; g <= g1; g += beside_pair) {
            const float* p = part(g);
            const float2 ml = reinterpret_cast<const float2*>(p)[at];
            const float4 v = reinterpret_cast<const float4*>(p + 2 * kAtPartSums)[d * R + at];
            const float f = exp2f((ml.x - m) * a.c);
            l += f * ml.y;
            o.x += f * v.x;
            o.y += f * v.y;
            o.z += f * v.z;
            o.w += f * v.w;
        }
        for (int s = 1; s < beside_pair; s *= 2) {
            l += __shfl_xor_sync(0xffffffffu, l, s);
            o.x += __shfl_xor_sync(0xffffffffu, o.x, s);
            o.y += __shfl_xor_sync(0xffffffffu, o.y, s);
            o.z += __shfl_xor_sync(0xffffffffu, o.z, s);
            o.w += __shfl_xor_sync(0xffffffffu, o.w, s);
        }
        if (lane == 0) write(row, d, o, l);
    }
}

// After the attention: joins, then refused requests' zeros and what was found.
// CTAs 0 .. zeros - 1 have every zeros-th request, the first the error word; the
// others a group's last item each, in pieces.  (A CTA for every block of every request
// took 41 us of 320 where 75 were to be joined, in turns of a microsecond.)
template <typename T, int DT, int NB>
__global__ void __launch_bounds__(kAtPrepNT) k_attend_finish(const __grid_constant__ AttendArgs a, int zeros) {
    __shared__ int sh;
    rows_begin();
    const int tid = threadIdx.x;
    auto err_of = [&](int b) { return a.err[b] | (a.parent ? a.tree_err[a.parent_stride ? b : 0] : 0); };
    if ((int)blockIdx.x >= zeros) {
        const int i = blockIdx.x - zeros, piece = i % kAtPieces, w = i / kAtPieces % NB,
                  cta = i / (kAtPieces * NB) % a.plan.ctas();
        attend_join<T, DT, NB>(a, i / (kAtPieces * NB) / a.plan.ctas(), cta, w, piece, &sh);
        return;
    }
    if (blockIdx.x == 0 && a.dev_error) {
        if (tid == 0) sh = *a.late;
        __syncthreads();
        int err = 0;
        for (int b = tid; b < a.B; b += kAtPrepNT) err |= err_of(b);
        if (err) atomicOr(&sh, err);
        __syncthreads();
        if (tid == 0) *a.dev_error = sh;
    }
    const int64_t each = (int64_t)a.q_heads * a.dim / 8;
    for (int b = blockIdx.x; b < a.B; b += zeros) {
        if (!err_of(b)) continue;
        const AttendRequest r = attend_request(a, b);
        const int n = r.n < 0 || r.n > a.N ? a.N : r.n;
        uint4* out = reinterpret_cast<uint4*>(a.out) + (int64_t)b * a.N * each;
        for (int64_t i = tid; i < n * each; i += kAtPrepNT) out[i] = make_uint4(0, 0, 0, 0);
    }
}

static AttendPlan attend_plan(int N, int heads, int group, int ctas) {
    AttendPlan p;
    p.nodes = kAtTile / group;
    p.blocks = N > p.nodes ? 2 : 1;
    const int parts = (N + p.blocks * p.nodes - 1) / (p.blocks * p.nodes);
    p.chunks = (parts + kAtShare - 1) / kAtShare;
    p.share = (parts + p.chunks - 1) / p.chunks;
    // the most heads, of up to 8, whose groups leave no more than a twentieth of the CTAs out
    p.heads = 1;
    for (int n = 2; n <= 8; ++n)
        if (heads % n == 0 && ctas / (p.share * n) * (p.share * n) * 20 >= ctas * 19) p.heads = n;
    p.groups = ctas / p.ctas();
    return p;
}
struct AttendSpace {
    size_t err, tree_err, first, late, masks, part, total;
};
static AttendSpace attend_space(int B, int N, int heads, int group, int dim) {
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    AttendSpace s;
    s.err = 0;
    s.tree_err = up((size_t)B * 4);
    s.first = s.tree_err + up((size_t)B * 4);
    s.late = s.first + up(((size_t)B + 1) * 4);
    s.masks = s.late + 256;
    s.part = s.masks + up((size_t)B * N * ((N + 31) / 32) * 4);
    const bool two = attend_plan(N, heads, group, kAtMaxCtas).blocks == 2;
    const int floats = dim > 64 ? (two ? kAtPartFloats<128, 2> : kAtPartFloats<128, 1>)
                                : (two ? kAtPartFloats<64, 2> : kAtPartFloats<64, 1>);
    s.total = s.part + (size_t)kAtMaxCtas * 2 * floats * 4;
    return s;
}

// A map of three dimensions of heads (sizes, strides in elements, boxes), 64
// columns of a head at a time.  false: the driver refuses it.
struct AttendDim {
    int64_t size, stride;
    int box;
};
static bool attend_map(CUtensorMap* map, const void* base, bool bf16, int dim, const AttendDim (&d)[3]) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return false;
    cuuint64_t sizes[4] = {(cuuint64_t)dim}, strides[3];
    cuuint32_t boxes[4] = {64}, steps[4] = {1, 1, 1, 1};
    for (int i = 0; i < 3; ++i) {
        sizes[i + 1] = (cuuint64_t)d[i].size;
        strides[i] = (cuuint64_t)(d[i].size == 1 ? dim : d[i].stride) * 2;  // one of size 1 is not used, but has to be there
        boxes[i + 1] = (cuuint32_t)d[i].box;
    }
    return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(base),
                  sizes, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct AttendMaps {
    CUtensorMap q, k, v;
};
template <typename T, int DT, int NB>
static cudaError_t launch_attend(AttendArgs a, const AttendMaps& maps, cudaStream_t st) {
    LaunchShape shape;
    if (!launch_shape(reinterpret_cast<const void*>(k_attend<T, DT, NB>), kAttendSmem<DT>, kAtNT, &shape))
        return cudaErrorUnknown;
    a.plan = attend_plan(a.N, a.kv_heads, a.group, shape.sms < kAtMaxCtas ? shape.sms : kAtMaxCtas);
    const int trees = !a.parent ? 0 : a.parent_stride ? a.B : 1;
    cudaError_t e = launch_dependent(k_attend_prepare, dim3(1 + trees), dim3(kAtPrepNT), 0, st, a);
    if (e != cudaSuccess) return e;
    e = launch_dependent(k_attend<T, DT, NB>, dim3(a.plan.groups * a.plan.ctas()), dim3(kAtNT), kAttendSmem<DT>, st, a, maps.q,
                         maps.k, maps.v);
    if (e != cudaSuccess) return e;
    const int zeros = a.B < 64 ? a.B : 64, joins = a.plan.groups * a.plan.ctas() * NB * kAtPieces;
    return launch_dependent(k_attend_finish<T, DT, NB>, dim3(zeros + joins), dim3(kAtPrepNT), 0, st, a, zeros);
}
template <typename T>
static cudaError_t launch_attend(const AttendArgs& a, const AttendMaps& maps, cudaStream_t st) {
    const bool two = a.plan.blocks == 2;
    if (a.dim > 64) return two ? launch_attend<T, 128, 2>(a, maps, st) : launch_attend<T, 128, 1>(a, maps, st);
    return two ? launch_attend<T, 64, 2>(a, maps, st) : launch_attend<T, 64, 1>(a, maps, st);
}

}  // namespace sv

using namespace sv;

extern "C" size_t spec_tree_attention_workspace(int B, int N, int q_heads, int kv_heads, int dim) {
    if (B < 1 || N < 1 || q_heads < 1 || kv_heads < 1 || dim < 1 || q_heads % kv_heads) return 0;
    return attend_space(B, N, kv_heads, q_heads / kv_heads, dim).total;
}

extern "C" spec_status spec_tree_attention(const void* q, spec_dtype dtype, int B, int N, int q_heads,
                                           int64_t q_request_stride, int64_t q_node_stride, int64_t q_head_stride,
                                           const void* k_cache, const void* v_cache, const spec_cache_layout* layout,
                                           const int32_t* block_table, int max_blocks, int64_t table_stride,
                                           const int32_t* seq_lens, const int32_t* parent, int64_t parent_stride,
                                           const int32_t* n_nodes, float scale, void* out, int32_t* dev_error,
                                           void* workspace, size_t workspace_bytes, spec_stream_t stream) {
    DeviceGuard device_guard;  // the caller's current device is put back on return
    if (dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out || !layout_ok(layout)) return SPEC_ERR_INVALID_ARG;
    if (B < 1 || N < 1 || q_heads < 1 || q_heads % layout->heads || max_blocks < 1 || table_stride < max_blocks ||
        q_request_stride < 0 || q_node_stride < 0 || q_head_stride < 0 ||
        (parent && parent_stride != 0 && parent_stride < N) || !(scale > 0.0f) || !(scale * (float)kLog2e < INFINITY))
        return SPEC_ERR_INVALID_ARG;
    const int group = q_heads / layout->heads;
    const int64_t capacity = (int64_t)max_blocks * layout->page_size;
    if (B > kMaxRequests || N > kMaxDraftNodes || layout->dim % 8 || layout->dim > 128 ||
        group > kAtTile)
        return SPEC_ERR_UNSUPPORTED;
    const AttendPlan plan = attend_plan(N, layout->heads, group, kAtMaxCtas);
    // units in 31 bits
    const int64_t parts = (int64_t)B * layout->heads * plan.chunks, tiles = (capacity + kAtTile - 1) / kAtTile;
    if (tiles > 0x7fffffffLL || parts > 0x7fffffffLL / tiles)
        return SPEC_ERR_UNSUPPORTED;
    if ((q_request_stride | q_node_stride | q_head_stride | layout->block_stride | layout->entry_stride |
         layout->head_stride) % 8 ||
        ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
          reinterpret_cast<uintptr_t>(out)) & 15u))
        return SPEC_ERR_UNSUPPORTED;
    const AttendSpace s = attend_space(B, N, layout->heads, group, layout->dim);
    if (!workspace || workspace_bytes < s.total || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return SPEC_ERR_WORKSPACE;
    if (!select_device_of(q)) return SPEC_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // a copy takes as many entries as lie together in every page and tile
    int box = 1;
    while (box < kAtTile && layout->page_size % (2 * box) == 0) box *= 2;
    const bool bf16 = dtype == SPEC_BF16;
    const int dim = layout->dim;
    const AttendDim queries[3] = {{q_heads, q_head_stride, group}, {N, q_node_stride, plan.nodes}, {B, q_request_stride, 1}};
    const AttendDim cache[3] = {{layout->heads, layout->head_stride, 1},
                                {layout->page_size, layout->entry_stride, box},
                                {layout->blocks, layout->block_stride, 1}};
    AttendMaps maps;
    if (!attend_map(&maps.q, q, bf16, dim, queries) || !attend_map(&maps.k, k_cache, bf16, dim, cache) ||
        !attend_map(&maps.v, v_cache, bf16, dim, cache))
        return SPEC_ERR_UNSUPPORTED;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    auto at = [&](size_t offset) { return reinterpret_cast<int32_t*>(w + offset); };
    AttendArgs a{B, N, q_heads, layout->heads, group, dim, layout->blocks, layout->page_size, box, block_table, table_stride,
                 capacity, seq_lens, parent, parent_stride, n_nodes, (float)((double)scale * kLog2e),
                 static_cast<uint16_t*>(out), dev_error, plan, at(s.err), at(s.tree_err), at(s.first), at(s.late),
                 reinterpret_cast<uint32_t*>(w + s.masks), reinterpret_cast<float*>(w + s.part), (N + 31) / 32};
    return (bf16 ? launch_attend<__nv_bfloat16>(a, maps, st) : launch_attend<__half>(a, maps, st)) == cudaSuccess
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}
