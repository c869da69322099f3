// New tokens into a paged cache (spec_append_kv): queries and keys normalised
// and turned by their position, keys and values stored in their slots.
#include "../../include/specverify.h"
#include "paged.cuh"

namespace sv {

constexpr int kApNT = 128;
constexpr int kApMaxDim = 256;
constexpr int kApUnroll = 2;  // heads of a thread on their way at once
constexpr int kApCtas = 6;    // of an SM

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
// two parts (1 / 2 pi to 106 bits), so the unit is right to 1.5 * 2^-64 and the
// angle to 2^-32.4 turns at any position.  As a float of its upper half, which is
// what sine and cosine are taken of in 32 bits, it is right to 2^-25.9.
__device__ __forceinline__ uint64_t turn_unit(float inv) {
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
    const double x = (double)inv, hi = x * kHi, lo = fma(x, kHi, -hi) + x * kLo;
    const double whole = floor(hi);
    return __double2ull_rz((hi - whole) * 0x1p64) + (uint64_t)__double2ll_rn(lo * 0x1p64);
}

// Persistent CTAs, a token at a time.  L lanes share a head, each with two
// vectors of VE elements: a pair of vectors that turn together (i and i + half),
// or two neighbours.  A pair's unit is found once per CTA; a token's cosines and
// sines are computed once, by as many threads as there are pairs, and its first
// heads are on their way while the token before is turned.  Bound by memory:
// every value is read and written once.  16384 tokens of 64 + 2 * 8 heads of
// 128: 126 us, 0.78 of the copy rate, with 6 CTAs of 128 threads an SM (134 with
// 4 of three heads a thread, 162 with 2 of 256 threads, 158 with a CTA a token).
template <typename T, int VE, bool INTERLEAVED>
__global__ void __launch_bounds__(kApNT, kApCtas) k_append(const __grid_constant__ AppendArgs a, int lanes) {
    using V = typename Vec<VE>::type;
    constexpr int W = VE / 2;  // words of a vector
    __shared__ float2 turn[2][kApMaxDim / 2];
    __shared__ int64_t sh_entry[2];
    rows_begin();
    const int tid = threadIdx.x, extra = a.dev_error ? 1 : 0, ctas = gridDim.x - extra;
    if ((int)blockIdx.x < extra) {
        // this CTA looks over all slots for the error word: a launch that clears it first would be on every call's way
        int64_t most = -1;
#pragma unroll 16
        for (int t = tid; t < a.T; t += kApNT) most = max(most, a.slots[t]);
        const bool bad = __syncthreads_or(most >= a.entries);
        if (tid == 0) *a.dev_error = bad ? kDevErrCapacity : 0;
        return;
    }
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
    union Two {
        V v[2];
        uint32_t w[2][W];
    };
    auto load = [&](Two* x, int t, int h0) {
#pragma unroll
        for (int u = 0; u < kApUnroll; ++u) {
            int h = h0 + u * per;
            if (h >= all) continue;
            const uint16_t* s;
            if (h < heads) s = a.q + (int64_t)t * a.q_token + (int64_t)h * a.q_head;
            else if ((h -= heads) < a.kv_heads) s = a.k + (int64_t)t * a.k_token + (int64_t)h * a.k_head;
            else s = a.v + (int64_t)t * a.v_token + (int64_t)(h - a.kv_heads) * a.v_head;
            if (has0) x[u].v[0] = *reinterpret_cast<const V*>(s + e0);
            if (has1) x[u].v[1] = *reinterpret_cast<const V*>(s + e1);
        }
    };
    // a thread of a pair has its unit; the last has the slots
    const bool turns_pair = tid < a.half, has_slot = tid == kApNT - 1;
    const uint64_t unit = turns_pair ? turn_unit(a.inv_freq[tid]) : 0;
    int position = 0;
    int64_t slot = -1;
    auto look = [&](int t) {
        if (turns_pair) position = a.positions[t];
        if (has_slot) slot = a.slots[t];
    };
    Two ahead[kApUnroll];
    int t = blockIdx.x - extra;
    if (t < a.T) {
        look(t);
        load(ahead, t, first);
    }
    const int rot = 2 * a.half;
    for (int buf = 0; t < a.T; t += ctas, buf ^= 1) {
        if (turns_pair) {
            const uint64_t angle = (uint64_t)(int64_t)position * unit;
            float s, c;
            sincospif((float)(int32_t)(angle >> 32) * 0x1p-31f, &s, &c);
            turn[buf][tid] = make_float2(c, s);
        }
        if (has_slot) {
            int64_t entry = -1;
            if (slot >= 0 && slot < a.entries) {
                const int64_t block = slot / a.page;
                entry = block * a.block_stride + (slot - block * a.page) * a.entry_stride;
            }
            sh_entry[buf] = entry;
        }
        __syncthreads();  // two buffers: the next token's are written by threads that have passed the next one
        const int64_t entry = sh_entry[buf];
        float2 cs[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) cs[i] = pairs + i < a.half ? turn[buf][pairs + i] : make_float2(1.0f, 0.0f);
        for (int base = 0; base < all; base += per * kApUnroll) {  // the same turns for every lane of a warp
            const int h0 = base + first;
            Two x[kApUnroll];
            if (base > 0) {
                load(x, t, h0);
            } else {
#pragma unroll
                for (int u = 0; u < kApUnroll; ++u) x[u] = ahead[u];
                const int next = t + ctas;
                if (next < a.T) {
                    look(next);
                    load(ahead, next, first);
                }
            }
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
                        float2 squares = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int i = 0; i < W; ++i) squares = __ffma2_rn(f[j][i], f[j][i], squares);
                        float sum = squares.x + squares.y;
                        for (int o = lanes >> 1; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                        const float r = 1.0f / sqrtf(sum / (float)a.dim + a.eps);
                        const uint16_t* norm = h < heads ? a.q_norm : a.k_norm;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            if (j == 0 ? !has0 : !has1) continue;
                            Two n;
                            n.v[0] = *reinterpret_cast<const V*>(norm + (j == 0 ? e0 : e1));
#pragma unroll
                            for (int i = 0; i < W; ++i)
                                f[j][i] = __fmul2_rn(f[j][i], __fmul2_rn(Pair<T>::get(n.w[0][i]), make_float2(r, r)));
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
                            const float2 c = make_float2(cs[2 * i].x, cs[2 * i + 1].x), s = make_float2(cs[2 * i].y, cs[2 * i + 1].y);
                            const float2 p = f[0][i], q = f[1][i], minus = make_float2(-s.x, -s.y);
                            f[0][i] = __ffma2_rn(q, minus, __fmul2_rn(p, c));
                            f[1][i] = __ffma2_rn(p, s, __fmul2_rn(q, c));
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
            __syncwarp();
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
    // one CTA more for the error word, all of them at once
    int grid;
    if (!(interleaved ? launch_grid(k_append<T, VE, true>, 0, (long long)a.T + 1, &grid, kApNT)
                      : launch_grid(k_append<T, VE, false>, 0, (long long)a.T + 1, &grid, kApNT)))
        return cudaErrorUnknown;
    if (!a.dev_error && grid > a.T) grid = a.T;
    return interleaved ? launch_clusters(k_append<T, VE, true>, grid, 1, kApNT, 0, true, st, a, lanes)
                       : launch_clusters(k_append<T, VE, false>, grid, 1, kApNT, 0, true, st, a, lanes);
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
