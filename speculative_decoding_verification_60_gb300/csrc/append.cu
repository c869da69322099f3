// New tokens into a paged cache (spec_append_kv): queries and keys normalised
// and turned by their position, keys and values stored in their slots.
#include "../../include/specverify.h"
#include "paged.cuh"

namespace sv {

constexpr int kApNT = 256;
constexpr int kApMaxDim = 256;
constexpr int kApUnroll = 3;  // heads of a thread on their way at once

struct AppendArgs {
    const uint16_t *q, *k, *v;
    int T, q_heads, kv_heads, dim, half;
    int64_t q_token, q_head, k_token, k_head, v_token, v_head;
    const uint16_t *q_norm, *k_norm;
    float eps;
    const int32_t* positions;
    const float* inv_freq;
    const int64_t* slots;
    uint16_t *out_q, *k_cache, *v_cache;
    int page;
    int64_t entries;  // blocks * page
    int64_t block_stride, entry_stride, head_stride;
    int32_t* dev_error;
};

template <int VE> struct Vec;
template <> struct Vec<8> { using type = uint4; };
template <> struct Vec<4> { using type = uint2; };

// inv / 2 pi as a fraction of a turn, in units of 2^-64 turns.  A position
// times it, modulo 2^64, is the angle modulo a turn: positions are whole
// numbers, so nothing is lost however far they are.  The product is taken in
// two parts (1 / 2 pi to 106 bits), so the unit is right to a few 2^-64.
__device__ __forceinline__ uint64_t turn_unit(float inv) {
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
    const double x = (double)inv, hi = x * kHi, lo = fma(x, kHi, -hi) + x * kLo;
    const double whole = floor(hi);
    return __double2ull_rz((hi - whole) * 0x1p64) + (uint64_t)__double2ll_rn(lo * 0x1p64);
}

// One CTA per token.  L lanes share a head, each with two vectors of VE
// elements: a pair of vectors that turn together (i and i + half), or two
// neighbours.  Cosines and sines are computed once per token, while the first
// heads are on their way.  Bound by memory: every value is read and written
// once.
template <typename T, int VE, bool INTERLEAVED>
__global__ void __launch_bounds__(kApNT) k_append(AppendArgs a, int lanes) {
    using V = typename Vec<VE>::type;
    constexpr int W = VE / 2;  // words of a vector
    __shared__ float2 turn[kApMaxDim / 2];
    __shared__ int64_t sh_entry;
    rows_begin();
    const int t = blockIdx.x, tid = threadIdx.x;
    const int per = kApNT / lanes, sub = tid % lanes, first = tid / lanes;
    const int heads = (a.q ? a.q_heads : 0), all = heads + 2 * a.kv_heads;
    // this lane's two vectors; a vector past the head's end is not there
    const int pairs = sub * VE;
    int e0, e1;
    if (INTERLEAVED) {
        e0 = 2 * pairs;
        e1 = e0 + VE;
    } else if (pairs < a.half) {
        e0 = pairs;
        e1 = a.half + pairs;
    } else {
        e0 = 2 * pairs;  // 2 half + 2 (pairs - half)
        e1 = e0 + VE;
    }
    const bool has0 = e0 < a.dim, has1 = e1 < a.dim;
    auto source = [&](int h) -> const uint16_t* {
        if (h < heads) return a.q + (int64_t)t * a.q_token + (int64_t)h * a.q_head;
        h -= heads;
        if (h < a.kv_heads) return a.k + (int64_t)t * a.k_token + (int64_t)h * a.k_head;
        return a.v + (int64_t)t * a.v_token + (int64_t)(h - a.kv_heads) * a.v_head;
    };
    union Two {
        V v[2];
        uint32_t w[2][W];
    };
    Two x[kApUnroll];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < kApUnroll; ++u) {
            const int h = h0 + u * per;
            if (h < all) {
                const uint16_t* s = source(h);
                if (has0) x[u].v[0] = *reinterpret_cast<const V*>(s + e0);
                if (has1) x[u].v[1] = *reinterpret_cast<const V*>(s + e1);
            }
        }
    };
    load(first);
    for (int i = tid; i < a.half; i += kApNT) {
        const uint64_t angle = (uint64_t)(int64_t)a.positions[t] * turn_unit(a.inv_freq[i]);
        float s, c;
        sincospif((float)(int32_t)(angle >> 32) * 0x1p-31f, &s, &c);
        turn[i] = make_float2(c, s);
    }
    if (tid == 0) {
        const int64_t slot = a.slots[t];
        int64_t entry = -1;
        if (slot >= a.entries) {
            set_error(a.dev_error, kDevErrCapacity);
        } else if (slot >= 0) {
            const int64_t block = slot / a.page;
            entry = block * a.block_stride + (slot - block * a.page) * a.entry_stride;
        }
        sh_entry = entry;
    }
    __syncthreads();
    const int64_t entry = sh_entry;
    float2 cs[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) cs[i] = pairs + i < a.half ? turn[pairs + i] : make_float2(1.0f, 0.0f);
    const int rot = 2 * a.half;
    for (int base = 0; base < all; base += per * kApUnroll) {  // the same turns for every lane of a warp
        const int h0 = base + first;
        if (base > 0) load(h0);
#pragma unroll
        for (int u = 0; u < kApUnroll; ++u) {
            const int h = h0 + u * per;
            const bool live = h < all, turns = live && h < heads + a.kv_heads;
            if (__any_sync(0xffffffffu, turns)) {
                float2 f[2][W];
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    f[0][i] = turns && has0 ? Pair<T>::get(x[u].w[0][i]) : make_float2(0.0f, 0.0f);
                    f[1][i] = turns && has1 ? Pair<T>::get(x[u].w[1][i]) : make_float2(0.0f, 0.0f);
                }
                if (a.k_norm) {
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int i = 0; i < W; ++i) sum += f[j][i].x * f[j][i].x + f[j][i].y * f[j][i].y;
                    for (int o = lanes >> 1; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    const float r = 1.0f / sqrtf(sum / (float)a.dim + a.eps);
                    const uint16_t* norm = h < heads ? a.q_norm : a.k_norm;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (j == 0 ? !has0 : !has1) continue;
                        Two n;
                        n.v[0] = *reinterpret_cast<const V*>(norm + (j == 0 ? e0 : e1));
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            const float2 w = Pair<T>::get(n.w[0][i]);
                            f[j][i].x *= r * w.x;
                            f[j][i].y *= r * w.y;
                        }
                    }
                }
                if (INTERLEAVED) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if ((j == 0 ? e0 : e1) < rot) {
#pragma unroll
                            for (int i = 0; i < W; ++i) {
                                const float2 c = cs[j * W + i], p = f[j][i];
                                f[j][i] = make_float2(p.x * c.x - p.y * c.y, p.y * c.x + p.x * c.y);
                            }
                        }
                } else if (pairs < a.half) {
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const float2 c = cs[2 * i], d = cs[2 * i + 1], p = f[0][i], q = f[1][i];
                        f[0][i] = make_float2(p.x * c.x - q.x * c.y, p.y * d.x - q.y * d.y);
                        f[1][i] = make_float2(q.x * c.x + p.x * c.y, q.y * d.x + p.y * d.y);
                    }
                }
                // values that neither the norm nor the turn touches keep their bits
                if (turns && (a.k_norm || e0 < rot)) {
#pragma unroll
                    for (int i = 0; i < W; ++i) x[u].w[0][i] = Pair<T>::put(f[0][i].x, f[0][i].y);
                }
                if (turns && (a.k_norm || e1 < rot)) {
#pragma unroll
                    for (int i = 0; i < W; ++i) x[u].w[1][i] = Pair<T>::put(f[1][i].x, f[1][i].y);
                }
            }
            if (!live) continue;
            uint16_t* to;
            if (h < heads) {
                to = a.out_q + ((int64_t)t * heads + h) * a.dim;
            } else {
                if (entry < 0) continue;
                const int g = h - heads;
                to = g < a.kv_heads ? a.k_cache + entry + g * a.head_stride
                                    : a.v_cache + entry + (g - a.kv_heads) * a.head_stride;
            }
            if (has0) *reinterpret_cast<V*>(to + e0) = x[u].v[0];
            if (has1) *reinterpret_cast<V*>(to + e1) = x[u].v[1];
        }
    }
}

template <typename T, int VE>
static cudaError_t launch_append(const AppendArgs& a, bool interleaved, cudaStream_t st) {
    // lanes of a head: the power of two that covers its slots of two vectors
    const int turned = interleaved ? 0 : a.half / VE;
    const int slots = turned + (a.dim - 2 * turned * VE + 2 * VE - 1) / (2 * VE);
    int lanes = 1;
    while (lanes < slots) lanes *= 2;
    return interleaved ? launch_clusters(k_append<T, VE, true>, a.T, 1, kApNT, 0, true, st, a, lanes)
                       : launch_clusters(k_append<T, VE, false>, a.T, 1, kApNT, 0, true, st, a, lanes);
}

}  // namespace sv

using namespace sv;

extern "C" spec_status spec_append_kv(const void* q, const void* k, const void* v, spec_dtype dtype, int T, int q_heads,
                                      int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride,
                                      int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                                      const void* q_norm, const void* k_norm, float eps, const int32_t* positions,
                                      const float* inv_freq, int rot_dim, int interleaved, const int64_t* slots,
                                      void* out_q, void* k_cache, void* v_cache, const spec_cache_layout* layout,
                                      int32_t* dev_error, spec_stream_t stream) {
    DeviceGuard device_guard;  // the caller's current device is put back on return
    if (dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (!layout_ok(layout) || T < 0 || rot_dim < 0 || rot_dim > layout->dim || (rot_dim & 1)) return SPEC_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || (T > 0 && (!k || !v || !slots)) || (q && (!out_q || q_heads < 1)))
        return SPEC_ERR_INVALID_ARG;
    if (T > 0 && rot_dim > 0 && (!positions || !inv_freq)) return SPEC_ERR_INVALID_ARG;
    if ((q && !q_norm != !k_norm) || (!q && T > 0 && q_norm) || !(eps >= 0.0f)) return SPEC_ERR_INVALID_ARG;
    if (layout->dim % 8 || layout->dim > kApMaxDim || rot_dim % 8) return SPEC_ERR_UNSUPPORTED;
    // vectors of 8 elements where everything lies on 16 bytes and pairs of them turn together, else of 4
    int64_t at = 0;
    for (int64_t s : {k_token_stride, k_head_stride, v_token_stride, v_head_stride, layout->block_stride,
                      layout->entry_stride, layout->head_stride, q ? q_token_stride : 0, q ? q_head_stride : 0})
        at |= s;
    uintptr_t p = 0;
    for (const void* x : {k, v, (const void*)k_cache, (const void*)v_cache, k_norm, q_norm, q, q ? (const void*)out_q : nullptr})
        p |= reinterpret_cast<uintptr_t>(x);
    if (at % 4 || p % 8) return SPEC_ERR_UNSUPPORTED;
    const bool wide = at % 8 == 0 && p % 16 == 0 && (interleaved || rot_dim % 16 == 0);
    if (T == 0 && !dev_error) return SPEC_OK;
    if (!select_device_of(k_cache)) return SPEC_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const spec_status cleared = clear_error(dev_error, st);
    if (cleared != SPEC_OK || T == 0) return cleared;
    auto in = [](const void* x) { return static_cast<const uint16_t*>(x); };
    auto out = [](void* x) { return static_cast<uint16_t*>(x); };
    AppendArgs a{in(q), in(k), in(v), T, q_heads, layout->heads, layout->dim, rot_dim / 2,
                 q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                 in(q_norm), in(k_norm), eps, positions, inv_freq, slots, out(out_q), out(k_cache), out(v_cache),
                 layout->page_size, (int64_t)layout->blocks * layout->page_size, layout->block_stride,
                 layout->entry_stride, layout->head_stride, dev_error};
    const bool turn = interleaved != 0;
    cudaError_t e;
    if (dtype == SPEC_BF16)
        e = wide ? launch_append<__nv_bfloat16, 8>(a, turn, st) : launch_append<__nv_bfloat16, 4>(a, turn, st);
    else
        e = wide ? launch_append<__half, 8>(a, turn, st) : launch_append<__half, 4>(a, turn, st);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
