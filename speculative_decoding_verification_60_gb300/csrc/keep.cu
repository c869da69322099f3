// The accepted path's cache entries moved together (spec_keep_path).
#include "../../include/specverify.h"
#include "paged.cuh"

namespace sv {

constexpr int kKpNT = 256;
constexpr int kKpPlanes = 256;  // planes of a launch: their pointers are 2 KiB of its parameters
constexpr int kKpMaxPath = 1024;
constexpr int kKpAhead = 8;  // entries of a thread on their way at once

struct KeepArgs {
    uint8_t* planes[kKpPlanes];
    int n_planes;
    int W, page, blocks, heads;
    int vecs, head_vecs;  // vectors of an entry, of a head
    int64_t block_bytes, entry_bytes, head_bytes;
    const int32_t* path;
    const int32_t* accepted;
    const int32_t* lens;
    const int32_t* table;
    int64_t table_stride, capacity;  // capacity: positions that a table row holds
    int32_t* dev_error;
};

// A CTA takes a share of a request's (plane, vector of an entry) pairs, a
// thread one pair: it reads that vector of up to 8 accepted entries, then
// writes them to their new places.  path[i] >= i and increasing, so a place
// that is written is never one that is still to be read, and no other thread
// touches this vector.  Every CTA of a request finds the same answer about it
// before it writes.  Bound by the latency of table, read and write: 32 requests
// of up to 5 moved entries in 80 planes (22 MB) take 7.4 us on the device, one
// request's 4 in 32 planes 3.3.
template <typename V>
__global__ void __launch_bounds__(kKpNT) k_keep_path(const __grid_constant__ KeepArgs a) {
    __shared__ int64_t from[kKpMaxPath], to[kKpMaxPath];
    rows_begin();
    const int b = blockIdx.y, tid = threadIdx.x;
    const int n = a.accepted[b] + 1, len = a.lens[b];
    const int32_t* path = a.path + (int64_t)b * a.W;
    const int32_t* table = a.table + b * a.table_stride;
    int err = n < 1 || n > a.W || len < 0 ? SPEC_DEVERR_LENGTH : 0;
    if (!err)
        for (int i = tid; i < n; i += kKpNT) {
            const int p = path[i];
            if (p < i || (i > 0 && path[i - 1] >= p) || (int64_t)len + p >= a.capacity) {
                err |= SPEC_DEVERR_LENGTH;
                continue;
            }
            auto place = [&](int64_t at) {
                const int64_t j = at / a.page;
                const int block = table[j];
                if (block < 0 || block >= a.blocks) err |= kDevErrCapacity;
                return block * a.block_bytes + (at - j * a.page) * a.entry_bytes;
            };
            to[i] = place((int64_t)len + i);
            from[i] = place((int64_t)len + p);
        }
    if (__syncthreads_or(err)) {
        if (err) set_error(a.dev_error, err);
        return;
    }
    const int pairs = a.n_planes * a.vecs;
    for (int x = blockIdx.x * kKpNT + tid; x < pairs; x += gridDim.x * kKpNT) {
        const int plane = x / a.vecs, vec = x - plane * a.vecs, head = vec / a.head_vecs;
        uint8_t* base = a.planes[plane] + head * a.head_bytes + (int64_t)(vec - head * a.head_vecs) * sizeof(V);
        for (int i0 = 0; i0 < n; i0 += kKpAhead) {
            V v[kKpAhead];
#pragma unroll
            for (int k = 0; k < kKpAhead; ++k)
                if (i0 + k < n && from[i0 + k] != to[i0 + k]) v[k] = *reinterpret_cast<const V*>(base + from[i0 + k]);
#pragma unroll
            for (int k = 0; k < kKpAhead; ++k)
                if (i0 + k < n && from[i0 + k] != to[i0 + k]) *reinterpret_cast<V*>(base + to[i0 + k]) = v[k];
        }
    }
}

template <typename V>
static cudaError_t launch_keep(KeepArgs& a, int B, cudaStream_t st) {
    a.head_vecs = (int)(a.head_vecs / (int64_t)sizeof(V));
    a.vecs = a.heads * a.head_vecs;
    const int64_t each = ((int64_t)a.n_planes * a.vecs + kKpNT - 1) / kKpNT;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(each < 65535 ? each : 65535), (unsigned)B);
    cfg.blockDim = dim3(kKpNT);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_keep_path<V>, a);
}

}  // namespace sv

using namespace sv;

extern "C" spec_status spec_keep_path(void* const* planes, int n_planes, int element_size,
                                      const spec_cache_layout* layout, int B, int W, const int32_t* path_nodes,
                                      const int32_t* accepted_len, const int32_t* seq_lens, const int32_t* block_table,
                                      int max_blocks, int64_t table_stride, int32_t* dev_error, spec_stream_t stream) {
    DeviceGuard device_guard;  // the caller's current device is put back on return
    if (n_planes < 0 || B < 0 || W < 1 || max_blocks < 1 || table_stride < max_blocks || !layout_ok(layout) ||
        (n_planes > 0 && !planes) || (element_size != 1 && element_size != 2 && element_size != 4))
        return SPEC_ERR_INVALID_ARG;
    if (B > 0 && (!path_nodes || !accepted_len || !seq_lens || !block_table)) return SPEC_ERR_INVALID_ARG;
    for (int i = 0; i < n_planes; ++i)
        if (!planes[i]) return SPEC_ERR_INVALID_ARG;
    const int64_t head = (int64_t)layout->dim * element_size;
    if (B > kMaxRequests || W > kKpMaxPath || head * layout->heads > 1 << 22) return SPEC_ERR_UNSUPPORTED;
    if ((n_planes == 0 || B == 0) && !dev_error) return SPEC_OK;
    if (!select_device_of(B > 0 ? path_nodes : dev_error)) return SPEC_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const spec_status cleared = clear_error(dev_error, st);
    if (cleared != SPEC_OK || B == 0) return cleared;
    for (int p0 = 0; p0 < n_planes; p0 += kKpPlanes) {
        KeepArgs a{};
        a.n_planes = n_planes - p0 < kKpPlanes ? n_planes - p0 : kKpPlanes;
        int64_t at = head | layout->block_stride * element_size | layout->entry_stride * element_size |
                     layout->head_stride * element_size;
        for (int i = 0; i < a.n_planes; ++i) {
            a.planes[i] = static_cast<uint8_t*>(planes[p0 + i]);
            at |= (int64_t)(reinterpret_cast<uintptr_t>(planes[p0 + i]) & 15u);
        }
        a.W = W;
        a.page = layout->page_size;
        a.blocks = layout->blocks;
        a.heads = layout->heads;
        a.head_vecs = (int)head;  // bytes, until the vector is chosen
        a.block_bytes = layout->block_stride * element_size;
        a.entry_bytes = layout->entry_stride * element_size;
        a.head_bytes = layout->head_stride * element_size;
        a.path = path_nodes;
        a.accepted = accepted_len;
        a.lens = seq_lens;
        a.table = block_table;
        a.table_stride = table_stride;
        a.capacity = (int64_t)max_blocks * layout->page_size;
        a.dev_error = dev_error;
        // the widest vector on which everything lies
        const cudaError_t e = at % 16 == 0  ? launch_keep<uint4>(a, B, st)
                              : at % 4 == 0 ? launch_keep<uint32_t>(a, B, st)
                              : at % 2 == 0 ? launch_keep<uint16_t>(a, B, st)
                                            : launch_keep<uint8_t>(a, B, st);
        if (e != cudaSuccess) return SPEC_ERR_CUDA;
    }
    return SPEC_OK;
}
