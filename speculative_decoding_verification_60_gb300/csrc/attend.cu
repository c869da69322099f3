// Attention of drafted nodes over a paged cache (spec_tree_attention).
#include "../../include/specverify.h"
#include "paged.cuh"

namespace sv {

constexpr int kAtPrepNT = 256;

struct AttendArgs {
    const uint16_t* q;
    int B, N, q_heads, kv_heads, group, dim;
    int64_t q_request, q_node, q_head;
    const uint16_t *k, *v;
    int blocks, page;
    int64_t block_stride, entry_stride, head_stride;
    const int32_t* table;
    int64_t table_stride, capacity;  // capacity: positions that a table row holds
    const int32_t* lens;
    const int32_t* parent;
    int64_t parent_stride;
    const int32_t* n_nodes;
    float scale;
    uint16_t* out;
    int32_t* dev_error;
    // workspace
    int32_t* err;        // [B] error bits of a request: its lengths, later its blocks
    int32_t* tree_err;   // [B], or [1] for a shared tree: error bits of the parent array
    uint32_t* masks;     // [B or 1][N][mask_words]: bit m of node n's words: n sees node m
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

// Before the attention: the requests' error words, and which nodes each node
// of a tree sees.  CTA 0 has the requests, the others a tree each.
__global__ void __launch_bounds__(kAtPrepNT) k_attend_prepare(AttendArgs a) {
    __shared__ int32_t sh_parent[kMaxDraftNodes];
    rows_begin();
    const int tid = threadIdx.x;
    if (blockIdx.x == 0) {
        for (int b = tid; b < a.B; b += kAtPrepNT) a.err[b] = attend_request(a, b).err;
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

// One CTA per query row; a warp takes every fourth entry.
template <typename T>
__global__ void __launch_bounds__(128) k_attend_rows(AttendArgs a) {
    __shared__ float sh_m[4], sh_l[4], sh_o[4][128];
    rows_begin();
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int h = blockIdx.x % a.q_heads, n = blockIdx.x / a.q_heads % a.N, b = blockIdx.x / a.q_heads / a.N;
    const AttendRequest r = attend_request(a, b);
    const int tree = a.parent_stride ? b : 0;
    if (r.err || n >= r.n || (a.parent && a.tree_err[tree])) return;
    const uint16_t* q = a.q + b * a.q_request + n * a.q_node + h * a.q_head;
    const uint32_t* mask = a.masks + ((int64_t)tree * a.N + n) * a.mask_words;
    float x[4], o[4] = {}, m = -INFINITY, l = 0.0f;
    auto get = [](uint16_t v) { return Pair<T>::get(v).x; };
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = lane + 32 * i < a.dim ? get(q[lane + 32 * i]) : 0.0f;
    for (int t = w; t < r.len + r.n; t += 4) {
        if (t >= r.len) {
            const int node = t - r.len;
            if (a.parent ? !((mask[node >> 5] >> (node & 31)) & 1u) : node > n) continue;
        }
        const int block = a.table[b * a.table_stride + t / a.page];
        if (block < 0 || block >= a.blocks) {
            if (lane == 0) atomicOr(a.err + b, kDevErrCapacity);
            continue;
        }
        const int64_t at = block * a.block_stride + (t % a.page) * a.entry_stride + (h / a.group) * a.head_stride;
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 32 * i < a.dim) dot += x[i] * get(a.k[at + lane + 32 * i]);
#pragma unroll
        for (int s = 16; s; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
        dot *= a.scale;
        const float top = fmaxf(m, dot);
        const float down = top > m ? expf(m - top) : 1.0f, e = expf(dot - top);
        m = top;
        l = l * down + e;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 32 * i < a.dim) {
                const float v = get(a.v[at + lane + 32 * i]);
                o[i] = o[i] * down + e * v;
                bad = bad || !(fabsf(v) < INFINITY);
            }
        if (t >= r.len && __any_sync(0xffffffffu, bad)) l = NAN;  // a node's entry that is not finite
    }
    if (lane == 0) {
        sh_m[w] = m;
        sh_l[w] = l;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sh_o[w][lane + 32 * i] = o[i];
    __syncthreads();
    const float top = fmaxf(fmaxf(sh_m[0], sh_m[1]), fmaxf(sh_m[2], sh_m[3]));
    float sum = 0.0f, value = 0.0f;
    for (int i = 0; i < 4; ++i) {
        const float e = sh_m[i] == -INFINITY ? 0.0f : expf(sh_m[i] - top);
        if (e == 0.0f) continue;
        sum += e * sh_l[i];
        value += e * sh_o[i][tid];
    }
    if (tid < a.dim)
        a.out[(((int64_t)b * a.N + n) * a.q_heads + h) * a.dim + tid] = (uint16_t)Pair<T>::put(value / sum, 0.0f);
}

// After the attention: refused requests get their zeros, and the error word
// what was found.
__global__ void __launch_bounds__(kAtPrepNT) k_attend_finish(AttendArgs a) {
    rows_begin();
    const int tid = threadIdx.x;
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        int err = a.err[b];
        if (a.parent) err |= a.tree_err[a.parent_stride ? b : 0];
        if (!err) continue;
        const AttendRequest r = attend_request(a, b);
        const int n = r.n < 0 || r.n > a.N ? a.N : r.n;
        const int64_t each = (int64_t)a.q_heads * a.dim;
        for (int64_t i = tid; i < n * each; i += kAtPrepNT) a.out[(int64_t)b * a.N * each + i] = 0;
    }
    if (blockIdx.x == 0 && a.dev_error) {
        int err = 0;
        for (int b = tid; b < a.B; b += kAtPrepNT) err |= a.err[b];
        if (a.parent)
            for (int t = tid; t < (a.parent_stride ? a.B : 1); t += kAtPrepNT) err |= a.tree_err[t];
        __shared__ int all;
        if (tid == 0) all = 0;
        __syncthreads();
        if (err) atomicOr(&all, err);
        __syncthreads();
        if (tid == 0) *a.dev_error = all;
    }
}

struct AttendSpace {
    size_t err, tree_err, masks, total;
};
static AttendSpace attend_space(int B, int N) {
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    AttendSpace s;
    s.err = 0;
    s.tree_err = up((size_t)B * 4);
    s.masks = s.tree_err + up((size_t)B * 4);
    s.total = s.masks + up((size_t)B * N * ((N + 31) / 32) * 4);
    return s;
}

template <typename T>
static cudaError_t launch_attend(const AttendArgs& a, cudaStream_t st) {
    const int trees = !a.parent ? 0 : a.parent_stride ? a.B : 1;
    cudaError_t e = launch_dependent(k_attend_prepare, dim3(1 + trees), dim3(kAtPrepNT), 0, st, a);
    if (e != cudaSuccess) return e;
    e = launch_dependent(k_attend_rows<T>, dim3((unsigned)((int64_t)a.B * a.N * a.q_heads)), dim3(128), 0, st, a);
    if (e != cudaSuccess) return e;
    return launch_dependent(k_attend_finish, dim3(a.B < 128 ? a.B : 128), dim3(kAtPrepNT), 0, st, a);
}

}  // namespace sv

using namespace sv;

extern "C" size_t spec_tree_attention_workspace(int B, int N, int q_heads, int kv_heads, int dim) {
    if (B < 1 || N < 1 || q_heads < 1 || kv_heads < 1 || dim < 1) return 0;
    return attend_space(B, N).total;
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
        (parent && parent_stride != 0 && parent_stride < N) || !(scale > 0.0f) || !(scale < INFINITY))
        return SPEC_ERR_INVALID_ARG;
    if (B > kMaxRequests || N > kMaxDraftNodes || layout->dim % 8 || layout->dim < 64 || layout->dim > 128 ||
        (int64_t)B * N * q_heads > 0x7fffffffLL)
        return SPEC_ERR_UNSUPPORTED;
    if ((q_request_stride | q_node_stride | q_head_stride | layout->block_stride | layout->entry_stride |
         layout->head_stride) % 8 ||
        ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
          reinterpret_cast<uintptr_t>(out)) & 15u))
        return SPEC_ERR_UNSUPPORTED;
    const AttendSpace s = attend_space(B, N);
    if (!workspace || workspace_bytes < s.total || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return SPEC_ERR_WORKSPACE;
    if (!select_device_of(q)) return SPEC_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* w = static_cast<uint8_t*>(workspace);
    AttendArgs a{static_cast<const uint16_t*>(q), B, N, q_heads, layout->heads, q_heads / layout->heads, layout->dim,
                 q_request_stride, q_node_stride, q_head_stride, static_cast<const uint16_t*>(k_cache),
                 static_cast<const uint16_t*>(v_cache), layout->blocks, layout->page_size, layout->block_stride,
                 layout->entry_stride, layout->head_stride, block_table, table_stride,
                 (int64_t)max_blocks * layout->page_size, seq_lens, parent, parent_stride, n_nodes, scale,
                 static_cast<uint16_t*>(out), dev_error, reinterpret_cast<int32_t*>(w + s.err),
                 reinterpret_cast<int32_t*>(w + s.tree_err), reinterpret_cast<uint32_t*>(w + s.masks), (N + 31) / 32};
    return (dtype == SPEC_BF16 ? launch_attend<__nv_bfloat16>(a, st) : launch_attend<__half>(a, st)) == cudaSuccess
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}
