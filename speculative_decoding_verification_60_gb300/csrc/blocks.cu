// Cache slots of the next step (spec_advance_blocks): the accepted tokens of
// a verification join every request's sequence, requests take the cache
// blocks they lack from a free list, and every new token gets its slot.
#include "../../include/specverify.h"
#include "common.cuh"
#include "launch.cuh"

namespace sv {

constexpr int kDevErrCapacity = 32;
constexpr int kBlThreads = 1024;
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

// Inclusive prefix sums of x and y over the CTA's threads in thread order.
__device__ __forceinline__ void block_scan2(int& x, int& y, int2* part) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    x = warp_inclusive_scan_i(x);
    y = warp_inclusive_scan_i(y);
    __syncthreads();
    if (lane == 31) part[w] = make_int2(x, y);
    __syncthreads();
    if (w == 0) {
        int2 p = part[lane];
        p.x = warp_inclusive_scan_i(p.x);
        p.y = warp_inclusive_scan_i(p.y);
        part[lane] = p;
    }
    __syncthreads();
    if (w > 0) {
        x += part[w - 1].x;
        y += part[w - 1].y;
    }
}

__global__ void __launch_bounds__(kBlThreads) k_advance_blocks(BlocksArgs a) {
    __shared__ int2 part[32];
    __shared__ int sh_err, sh_taken;
    extern __shared__ int sh_mem[];
    int* cu = sh_mem;              // [B + 1]
    int* first = sh_mem + a.B + 1;  // [B] place in the free list of a request's first new block; -1: not served
    const int tid = threadIdx.x, count = *a.free_count;
    const int free_count = count >= 0 && count <= a.free_capacity ? count : 0;
    if (tid == 0) {
        sh_err = count == free_count ? 0 : kDevErrLength;
        sh_taken = cu[0] = 0;
    }
    __syncthreads();
    int tokens = 0, lacking = 0;  // of the requests before this round's
    for (int b0 = 0; b0 < a.B; b0 += kBlThreads) {
        const int b = b0 + tid;
        BlocksRequest q{};
        if (b < a.B) q = blocks_request(a, b);
        int x = q.n, y = q.lacks;
        block_scan2(x, y, part);
        if (b < a.B) {
            const int end = lacking + y;
            const bool served = !q.err && (q.lacks == 0 || end <= free_count);
            cu[b + 1] = tokens + x;
            first[b] = served ? end - q.lacks : -1;
            if (!served) atomicOr(&sh_err, q.err ? q.err : kDevErrCapacity);
            if (served && q.lacks) atomicMax(&sh_taken, end);
            a.out_lens[b] = q.len;
            a.out_held[b] = q.held + (served ? q.lacks : 0);
            if (served)
                for (int j = 0; j < q.lacks; ++j)
                    a.table[b * a.table_stride + q.held + j] = a.free_blocks[free_count - 1 - (end - q.lacks + j)];
        }
        tokens += part[31].x;
        lacking += part[31].y;
        __syncthreads();
    }
    for (int b = tid; b <= a.B; b += kBlThreads) a.cu_tokens[b] = cu[b];
    if (tid == 0) {
        *a.out_free = free_count - sh_taken;
        if (a.dev_error) *a.dev_error = sh_err | (tokens > a.max_tokens ? kDevErrLength : 0);
    }
    for (int i = tid; i < a.max_tokens; i += kBlThreads) {
        int64_t slot = -1;
        int position = 0;
        if (i < tokens) {
            int lo = 0, hi = a.B - 1;  // the last request that starts at or before i
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cu[mid] <= i) lo = mid;
                else hi = mid - 1;
            }
            const BlocksRequest q = blocks_request(a, lo);
            const int at = i - cu[lo];
            if (q.err != kDevErrLength && at >= 0 && at < q.n) {
                position = q.len + at;
                if (first[lo] >= 0) {
                    const int j = position / a.page;
                    const int block = j < q.held ? a.table[lo * a.table_stride + j]
                                                 : a.free_blocks[free_count - 1 - (first[lo] + j - q.held)];
                    slot = (int64_t)block * a.page + (position - j * a.page);
                }
            }
        }
        a.slots[i] = slot;
        if (a.positions) a.positions[i] = position;
    }
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
                 max_tokens, dev_error};
    const size_t dyn = (size_t)(2 * B + 1) * 4;
    if (!set_dyn_smem(k_advance_blocks, (size_t)(2 * kBlMaxRequests + 1) * 4, kBlThreads)) return SPEC_ERR_CUDA;
    k_advance_blocks<<<1, kBlThreads, dyn, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
