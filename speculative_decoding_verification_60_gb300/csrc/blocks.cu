// Cache slots of the next step (spec_advance_blocks): the accepted tokens of
// a verification join every request's sequence, requests take the cache
// blocks they lack from a free list, and every new token gets its slot.
#include "../../include/specverify.h"
#include "common.cuh"
#include "launch.cuh"

namespace sv {

constexpr int kDevErrCapacity = 32;
constexpr int kBlTokens = 4;  // consecutive tokens of a thread
constexpr int kBlMaxRequests = 16384;

struct BlocksArgs {
    const int32_t* seq_lens;
    const int32_t* accepted;
    const int32_t* new_tokens;
    int B, page;
    int32_t* table;
    int max_blocks;
    int64_t table_stride;
    const int32_t* held;
    const int32_t* free_blocks;
    int free_capacity;
    const int32_t* free_count;
    int32_t* out_lens;
    int32_t* out_held;
    int32_t* out_free;
    int32_t* cu_tokens;
    int64_t* slots;
    int32_t* positions;
    int max_tokens;
    int32_t* dev_error;
    bool aligned;  // slots and positions on 16 bytes
};

// One request's step before the free list is looked at.
struct BlocksRequest {
    int len;    // length after the acceptance (seq_lens[b] when refused)
    int n;      // new tokens (0 when negative)
    int held;   // blocks it has
    int lacks;  // blocks it takes from the free list if it is served
    int err;    // SPEC_DEVERR_LENGTH or SPEC_DEVERR_CAPACITY
};
__device__ __forceinline__ BlocksRequest blocks_request(const BlocksArgs& a, int b) {
    BlocksRequest q;
    const int len0 = a.seq_lens[b], acc = a.accepted ? a.accepted[b] : -1, n = a.new_tokens[b];
    q.held = a.held[b];
    q.n = max(n, 0);
    q.len = len0;
    q.lacks = 0;
    q.err = 0;
    const long long len = (long long)len0 + acc + 1;
    if (len0 < 0 || acc < -1 || n < 0 || q.held < 0 || q.held > a.max_blocks || len > (long long)q.held * a.page ||
        len + n > 0x7fffffffLL) {
        q.err = kDevErrLength;
        return q;
    }
    q.len = (int)len;
    const long long need = (len + q.n + a.page - 1) / a.page;
    if (need > a.max_blocks)
        q.err = kDevErrCapacity;
    else
        q.lacks = max((int)need - q.held, 0);
    return q;
}

// Exclusive prefix sums of x and y over the CTA's threads in thread order;
// *total receives the sums.
template <int NT>
__device__ __forceinline__ int2 block_scan2(int x, int y, int2* part, int2* total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int ix = warp_inclusive_scan_i(x), iy = warp_inclusive_scan_i(y);
    if (lane == 31) part[w] = make_int2(ix, iy);
    __syncthreads();
    if (w == 0) {
        int2 p = lane < NT / 32 ? part[lane] : make_int2(0, 0);
        p.x = warp_inclusive_scan_i(p.x);
        p.y = warp_inclusive_scan_i(p.y);
        part[lane] = p;
    }
    __syncthreads();
    *total = part[NT / 32 - 1];
    const int2 before = w > 0 ? part[w - 1] : make_int2(0, 0);
    return make_int2(before.x + ix - x, before.y + iy - y);
}

// Every CTA sums the requests for itself (they are few and in L2; a second
// launch, or a wait for another CTA's sums, would cost more), keeps where
// each one's tokens and new blocks begin in shared memory, and then takes its
// share of the tokens and of the table entries.  The block of a new entry
// comes from the free list, not from the table, so no CTA reads what another
// writes.  CTA 0 writes the per-request outputs.  Bound by latency (the reads
// of a request's state, two scans, the search, the table): 64 requests of 5
// tokens take 8.3 us on the device back to back, launch included; 1024 requests,
// 128 of them with prompts of up to 4096 tokens (3.3 MB), 8.9 us.
template <int NT>
__global__ void __launch_bounds__(NT) k_advance_blocks(BlocksArgs a) {
    __shared__ int2 part[32];
    __shared__ int sh_err, sh_taken;
    extern __shared__ int sh_mem[];
    int* cu = sh_mem;              // [B + 1]
    int* first = sh_mem + a.B + 1;  // [B] place in the free list of a request's first new block; -1: not served
    grid_dep_trigger();
    grid_dep_wait();
    const int tid = threadIdx.x, count = *a.free_count;
    const int free_count = count >= 0 && count <= a.free_capacity ? count : 0;
    if (tid == 0) {
        sh_err = count == free_count ? 0 : kDevErrLength;
        sh_taken = 0;
    }
    const int each = (a.B + NT - 1) / NT, b0 = tid * each, b1 = min(b0 + each, a.B);
    int x = 0, y = 0;
    for (int b = b0; b < b1; ++b) {
        const BlocksRequest q = blocks_request(a, b);
        x += q.n;
        y += q.lacks;
    }
    int2 total;
    int2 at = block_scan2<NT>(x, y, part, &total);
    const int tokens = total.x;
    int err = 0, taken = 0;
    for (int b = b0; b < b1; ++b) {
        const BlocksRequest q = blocks_request(a, b);
        const bool served = !q.err && (q.lacks == 0 || at.y + q.lacks <= free_count);
        cu[b] = at.x;
        first[b] = served ? at.y : -1;
        at.x += q.n;
        at.y += q.lacks;
        if (!served) err |= q.err ? q.err : kDevErrCapacity;
        if (served && q.lacks) taken = at.y;
        if (blockIdx.x == 0) {
            a.cu_tokens[b] = cu[b];
            a.out_lens[b] = q.len;
            a.out_held[b] = q.held + (served ? q.lacks : 0);
        }
    }
    if (blockIdx.x == 0) {
        err = __reduce_or_sync(0xffffffffu, err);
        taken = __reduce_max_sync(0xffffffffu, taken);
        if ((tid & 31) == 0 && err) atomicOr(&sh_err, err);
        if ((tid & 31) == 0 && taken) atomicMax(&sh_taken, taken);
    }
    if (tid == 0) cu[a.B] = tokens;
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) {
        a.cu_tokens[a.B] = tokens;
        *a.out_free = free_count - sh_taken;
        if (a.dev_error) *a.dev_error = sh_err | (tokens > a.max_tokens ? kDevErrLength : 0);
    }
    // new table entries: a warp per request
    for (int b = blockIdx.x * (NT / 32) + (tid >> 5); b < a.B; b += gridDim.x * (NT / 32)) {
        if (first[b] < 0) continue;
        const BlocksRequest q = blocks_request(a, b);
        for (int j = tid & 31; j < q.lacks; j += 32)
            a.table[b * a.table_stride + q.held + j] = a.free_blocks[free_count - 1 - (first[b] + j)];
    }
    // slots: consecutive tokens of a thread, mostly of one request.  Their
    // index passes 2^31 - 1 in the last turn of the largest max_tokens, by at
    // most a step (SMs * NT * kBlTokens): unsigned 32 bits hold it.
    const uint32_t most = (uint32_t)a.max_tokens, live = (uint32_t)max(tokens, 0);
    for (uint32_t i0 = (blockIdx.x * NT + tid) * kBlTokens; i0 < most; i0 += gridDim.x * NT * kBlTokens) {
        int b = 0;
        if (i0 < live) {  // the last request that starts at or before i0
            int hi = a.B - 1;
            while (b < hi) {
                const int mid = (b + hi + 1) >> 1;
                if ((uint32_t)cu[mid] <= i0) b = mid;
                else hi = mid - 1;
            }
        }
        BlocksRequest q = blocks_request(a, b);
        int64_t slot[kBlTokens];
        int position[kBlTokens];
#pragma unroll
        for (int k = 0; k < kBlTokens; ++k) {
            slot[k] = -1;
            position[k] = 0;
            if (i0 + k >= live) continue;
            const int i = (int)(i0 + k);
            if (i >= cu[b + 1]) {
                while (i >= cu[b + 1] && b < a.B - 1) ++b;
                q = blocks_request(a, b);
            }
            const int in = i - cu[b];
            if (q.err == kDevErrLength || in < 0 || in >= q.n) continue;
            position[k] = q.len + in;
            if (first[b] < 0) continue;
            const int j = position[k] / a.page;
            const int block = j < q.held ? a.table[b * a.table_stride + j]
                                         : a.free_blocks[free_count - 1 - (first[b] + j - q.held)];
            slot[k] = (int64_t)block * a.page + (position[k] - j * a.page);
        }
        if (a.aligned && i0 + kBlTokens <= most) {
            longlong2* s = reinterpret_cast<longlong2*>(a.slots + i0);
            s[0] = make_longlong2(slot[0], slot[1]);
            s[1] = make_longlong2(slot[2], slot[3]);
            if (a.positions)
                *reinterpret_cast<int4*>(a.positions + i0) = make_int4(position[0], position[1], position[2], position[3]);
        } else {
#pragma unroll
            for (int k = 0; k < kBlTokens; ++k)
                if (i0 + k < most) {
                    a.slots[i0 + k] = slot[k];
                    if (a.positions) a.positions[i0 + k] = position[k];
                }
        }
    }
}

template <int NT>
static cudaError_t launch_blocks(const BlocksArgs& a, cudaStream_t st) {
    LaunchShape shape;
    if (!launch_shape(reinterpret_cast<const void*>(k_advance_blocks<NT>), (size_t)(2 * kBlMaxRequests + 1) * 4, NT, &shape))
        return cudaErrorUnknown;
    // a CTA per NT * kBlTokens tokens, at most one an SM
    const long long want = ((long long)a.max_tokens + NT * kBlTokens - 1) / (NT * kBlTokens);
    const int grid = (int)(want < 1 ? 1 : want < shape.sms ? want : shape.sms);
    return launch_dependent(k_advance_blocks<NT>, dim3(grid), dim3(NT), (size_t)(2 * a.B + 1) * 4, st, a);
}

}  // namespace sv

using namespace sv;

extern "C" spec_status spec_advance_blocks(const int32_t* seq_lens, const int32_t* accepted_len,
                                           const int32_t* new_tokens, int B, int page_size, int32_t* block_table,
                                           int max_blocks, int64_t table_stride, const int32_t* held,
                                           const int32_t* free_blocks, int free_capacity, const int32_t* free_count,
                                           int32_t* out_seq_lens, int32_t* out_held, int32_t* out_free_count,
                                           int32_t* cu_tokens, int64_t* slots, int32_t* positions, int max_tokens,
                                           int32_t* dev_error, spec_stream_t stream) {
    DeviceGuard device_guard;  // the caller's current device is put back on return
    if (!seq_lens || !new_tokens || !block_table || !held || !free_count || !out_seq_lens || !out_held ||
        !out_free_count || !cu_tokens || (max_tokens > 0 && !slots))
        return SPEC_ERR_INVALID_ARG;
    if (B < 1 || page_size < 1 || max_blocks < 1 || table_stride < max_blocks || max_tokens < 0 ||
        free_capacity < 0 || (free_capacity > 0 && !free_blocks))
        return SPEC_ERR_INVALID_ARG;
    if (out_seq_lens == seq_lens || out_held == held || out_free_count == free_count) return SPEC_ERR_INVALID_ARG;
    if (B > kBlMaxRequests || (int64_t)B * max_blocks > 0x7fffffffLL) return SPEC_ERR_UNSUPPORTED;
    if (!select_device_of(seq_lens)) return SPEC_ERR_INVALID_ARG;
    BlocksArgs a{seq_lens, accepted_len, new_tokens, B, page_size, block_table, max_blocks, table_stride, held,
                 free_blocks, free_capacity, free_count, out_seq_lens, out_held, out_free_count, cu_tokens, slots, positions,
                 max_tokens, dev_error,
                 ((reinterpret_cast<uintptr_t>(slots) | reinterpret_cast<uintptr_t>(positions)) & 15u) == 0};
    // Few requests and tokens: smaller CTAs start and meet faster.
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool few = B <= 1024 && max_tokens <= 65536;
    return (few ? launch_blocks<256>(a, st) : launch_blocks<1024>(a, st)) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
