// rope.cu -- rotary positions on the query and key heads, with one position
// axis or several (time, height, width of images and video), and the inverse
// rotation, which is the gradient of the rotation (include/fa.h, fa_rope).
//
// Pair i of a head, (x, y), is rotated by the angle a = pos[axis(i)] * f_i:
//   x' = x cos a - y sin a,   y' = x sin a + y cos a.
// The angle is taken modulo a turn in exact integer arithmetic: the table
// holds F_i = 2^64 f_i / (2 pi), and the top 32 bits of pos * F_i mod 2^64 are
// the angle in 2^-32 turns, off by less than |pos| 2^-64 + 2^-32 turns however
// far the position is, without the 64-bit floating-point units (a few per SM).
// sincospif then sees an argument in [-1, 1).
//
// The call is bound by HBM: every element is read and written once. A thread
// owns one 16-byte vector of pairs of one token: it computes their sines and
// cosines once and walks the heads, whose loads are independent.
#include <algorithm>

#include <cuda_bf16.h>

#include "fa_device.cuh"
#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeUnroll = 4;  // heads whose loads are in flight together

template <typename T> struct Conv;
template <> struct Conv<float> {
    static __device__ __forceinline__ float get(float x) { return x; }
    static __device__ __forceinline__ float put(float x) { return x; }
};
template <> struct Conv<__half> {
    static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <> struct Conv<__nv_bfloat16> {
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
    T x[V];
};

// V values a thread moves at a time: 16 bytes, or 1 where a size, a stride or
// a pointer is not a multiple of that.
template <typename T, int V, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
    using W = Vec<T, V>;
    const int half = a.rotary_dim / 2;
    const int n_rot = half / V;            // items of V pairs
    const int n_items = n_rot + a.n_copy;  // and of 2 V values that stay as they are
    const long long id = blockIdx.x * static_cast<long long>(kRopeThreads) + threadIdx.x;
    const int tok = static_cast<int>(id / n_items);
    if (tok >= a.n_tokens) return;
    const int item = static_cast<int>(id - static_cast<long long>(tok) * n_items);
    const int h0 = blockIdx.y * a.heads_per_block;
    const int h1 = min(h0 + a.heads_per_block, a.n_q_heads + a.n_kv_heads);
    // element offsets of the item's two vectors inside a head
    int o0, o1;
    bool second = true;
    float c[V], s[V];
    if (item < n_rot) {
        o0 = ADJ ? 2 * V * item : V * item;
        o1 = ADJ ? o0 + V : half + o0;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const uint4 f = __ldg(static_cast<const uint4 *>(a.table) + item * V + k);
            const int axis = min(static_cast<int>(f.z), a.n_axes - 1);
            const long long pos = __ldg(a.positions + axis * a.pos_stride + tok);
            const unsigned long long F = (static_cast<unsigned long long>(f.y) << 32) | f.x;
            const unsigned long long turn = static_cast<unsigned long long>(pos) * F;
            const int top = static_cast<int>((turn + 0x80000000ull) >> 32);
            sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s[k], &c[k]);  // 2^-31
            if (a.inverse) s[k] = -s[k];
        }
    } else {
        o0 = a.rotary_dim + 2 * V * (item - n_rot);
        o1 = o0 + V;
        second = o1 < a.head_dim;
#pragma unroll
        for (int k = 0; k < V; ++k) c[k] = 1.0f, s[k] = 0.0f;
    }
    const bool copy = item >= n_rot;
    const T *qi = static_cast<const T *>(a.q) + tok * a.q_stride;
    const T *ki = static_cast<const T *>(a.k) + tok * a.k_stride;
    T *qo = static_cast<T *>(a.q_out) + tok * a.q_out_stride;
    T *ko = static_cast<T *>(a.k_out) + tok * a.k_out_stride;
    for (int h = h0; h < h1; h += kRopeUnroll) {
        W x[kRopeUnroll], y[kRopeUnroll];
        T *out[kRopeUnroll];
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            const int hh = h + u;
            if (hh >= h1) break;
            const bool isq = hh < a.n_q_heads;
            const long long off = static_cast<long long>(isq ? hh : hh - a.n_q_heads) * a.head_dim;
            const T *in = (isq ? qi : ki) + off;
            out[u] = (isq ? qo : ko) + off;
            x[u] = *reinterpret_cast<const W *>(in + o0);
            if (second) y[u] = *reinterpret_cast<const W *>(in + o1);
        }
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            if (h + u >= h1) break;
            if (!copy) {
                T *xs = x[u].x, *ys = y[u].x;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    // halves: pair k is (xs[k], ys[k]); adjacent: it is values 2 k and
                    // 2 k + 1 of the two vectors taken one after the other
                    T *p = ADJ ? (2 * k < V ? xs + 2 * k : ys + 2 * k - V) : xs + k;
                    T *q = ADJ ? (2 * k + 1 < V ? xs + 2 * k + 1 : ys + 2 * k + 1 - V) : ys + k;
                    const float u0 = Conv<T>::get(*p), u1 = Conv<T>::get(*q);
                    *p = Conv<T>::put(u0 * c[k] - u1 * s[k]);
                    *q = Conv<T>::put(u0 * s[k] + u1 * c[k]);
                }
            }
            *reinterpret_cast<W *>(out[u] + o0) = x[u];
            if (second) *reinterpret_cast<W *>(out[u] + o1) = y[u];
        }
    }
}

template <typename T, int V>
cudaError_t launch(RopeArgs a, cudaStream_t stream) {
    const bool in_place = a.q == a.q_out && (a.n_kv_heads == 0 || a.k == a.k_out);
    const int rest = a.head_dim - a.rotary_dim;
    a.n_copy = in_place ? 0 : (rest + 2 * V - 1) / (2 * V);
    const long long threads = static_cast<long long>(a.rotary_dim / 2 / V + a.n_copy) * a.n_tokens;
    const long long blocks = (threads + kRopeThreads - 1) / kRopeThreads;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    const int heads = a.n_q_heads + a.n_kv_heads;
    // Few tokens: the heads are split over blocks too, so that the GPU's SMs
    // all have some.
    const long long want = static_cast<long long>(device_sm_count()) * 8;
    int parts = static_cast<int>(std::min<long long>((want + blocks - 1) / blocks,
                                                     (heads + kRopeUnroll - 1) / kRopeUnroll));
    a.heads_per_block = (heads + parts - 1) / parts;
    parts = (heads + a.heads_per_block - 1) / a.heads_per_block;
    const dim3 grid(static_cast<unsigned>(blocks), parts);
    if (a.adjacent)
        rope_kernel<T, V, true><<<grid, kRopeThreads, 0, stream>>>(a);
    else
        rope_kernel<T, V, false><<<grid, kRopeThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const RopeArgs &a, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const uintptr_t ptrs = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) |
                           reinterpret_cast<uintptr_t>(a.q_out) |
                           reinterpret_cast<uintptr_t>(a.k_out);
    const long long sizes = a.head_dim | (a.rotary_dim / 2) | a.q_stride | a.k_stride |
                            a.q_out_stride | a.k_out_stride;
    return (ptrs & 15) == 0 && sizes % V == 0 ? launch<T, V>(a, stream) : launch<T, 1>(a, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t stream) {
    switch (a.dtype) {
        case kTypeF32: return launch_type<float>(a, stream);
        case kTypeF16: return launch_type<__half>(a, stream);
        default: return launch_type<__nv_bfloat16>(a, stream);
    }
}

}  // namespace fa
