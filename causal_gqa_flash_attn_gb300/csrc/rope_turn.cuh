// rope_turn.cuh -- rotary positions inside a block (rope.cu, rope_append.cu): the
// sines and cosines of its tokens in shared memory, and its heads through them.
#pragma once

#include <cuda_bf16.h>

#include "fa_device.cuh"
#include "fa_internal.h"
#include "paged_launch.cuh"

namespace fa {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 16;     // tokens of a block at most

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

// A pair turned by the angle of c and s, with its roundings spelt out, as several kernels have to give the same bits:
// x0 = fma(u0, c, -(u1 s)) and x1 = fma(u0, s, u1 c), the products rounded.
__device__ __forceinline__ void turn(float u0, float u1, float c, float s, float *x0, float *x1) {
    *x0 = fmaf(u0, c, -__fmul_rn(u1, s));
    *x1 = fmaf(u0, s, __fmul_rn(u1, c));
}

// Cosines cs [tokens][half] and sines sn of tokens tok0 .. tok0 + n_tok - 1.
__device__ __forceinline__ void turn_table(const RopeArgs &a, int half, int tok0, int n_tok, float *cs, float *sn) {
    for (int i = threadIdx.x; i < n_tok * half; i += kRopeThreads) {
        const int tok = i / half, pair = i - tok * half;
        const uint4 f = load(static_cast<const uint4 *>(a.table) + pair);
        const int axis = static_cast<int>(min(f.z, static_cast<unsigned>(a.n_axes) - 1u));
        long long pos = load(a.positions + axis * a.pos_stride + tok0 + tok);
        if (f.z >= static_cast<unsigned>(a.n_axes)) pos = 0;  // a pair without positions stays as it is
        const unsigned long long F = (static_cast<unsigned long long>(f.y) << 32) | f.x;
        const unsigned long long turn = static_cast<unsigned long long>(pos) * F;
        const int top = static_cast<int>((turn + 0x80000000ull) >> 32);
        float s, c;
        sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s, &c);  // 2^-31
        cs[i] = c;
        sn[i] = a.inverse ? -s : s;
    }
}

// Heads h0 .. h0 + heads - 1 (the q heads, then the k heads) of the block's tokens through the
// table, by all of its threads.
template <typename T, int V, bool ADJ>
__device__ __forceinline__ void turn_heads(const RopeArgs &a, int half, int tok0, int n_tok, int h0, int heads,
                                           const float *cs, const float *sn) {
    using W = Vec<T, V>;
    const int n_rot = half / V;            // items of V pairs
    const int n_items = n_rot + a.n_copy;  // and of 2 V values that stay as they are
    // threads of a head, heads that the block takes at once, and this thread's first one
    const int lanes = min(n_items, kRopeThreads), rows = kRopeThreads / lanes;
    const int row = threadIdx.x / lanes, lane = threadIdx.x - row * lanes;
    int tok = row < rows ? row / heads : n_tok, head = row - tok * heads;
    while (tok < n_tok) {
        const int hh = h0 + head;
        const bool isq = hh < a.n_q_heads;
        const long long at = tok0 + tok;
        const long long off = static_cast<long long>(isq ? hh : hh - a.n_q_heads) * a.head_dim;
        const T *in = static_cast<const T *>(isq ? a.q : a.k) + at * (isq ? a.q_stride : a.k_stride) + off;
        T *out = static_cast<T *>(isq ? a.q_out : a.k_out) +
                 at * (isq ? a.q_out_stride : a.k_out_stride) + off;
        const float *c = cs + tok * half, *s = sn + tok * half;
        for (int item = lane; item < n_items; item += lanes) {
            // An item's two vectors lie apart, so that neighbouring threads' are neighbours: in the
            // two halves of the rotated dims (for adjacent pairs, V / 2 pairs in each), or of the rest.
            const bool turns = item < n_rot;
            int o0, o1;
            if (turns) {
                o0 = ADJ && V == 1 ? 2 * item : V * item;
                o1 = ADJ && V == 1 ? o0 + 1 : half + o0;
            } else {
                o0 = a.rotary_dim + V * (item - n_rot);
                o1 = o0 + V * a.n_copy;
            }
            const bool second = o1 < a.head_dim;
            W x, y;
            x = *reinterpret_cast<const W *>(in + o0);
            if (second) y = *reinterpret_cast<const W *>(in + o1);
            if (turns) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    // halves: pair k is (x[k], y[k]); adjacent: it is two neighbours of one vector
                    const int pair = !ADJ || V == 1 ? item * V + k
                                     : k < V / 2    ? item * (V / 2) + k
                                                    : half / 2 + item * (V / 2) + k - V / 2;
                    T *p = ADJ && V > 1 ? (k < V / 2 ? x.x + 2 * k : y.x + 2 * k - V) : x.x + k;
                    T *q = ADJ && V > 1 ? p + 1 : y.x + k;
                    const float u0 = Conv<T>::get(*p), u1 = Conv<T>::get(*q);
                    float x0, x1;
                    turn(u0, u1, c[pair], s[pair], &x0, &x1);
                    *p = Conv<T>::put(x0);
                    *q = Conv<T>::put(x1);
                }
            }
            *reinterpret_cast<W *>(out + o0) = x;
            if (second) *reinterpret_cast<W *>(out + o1) = y;
        }
        head += rows;
        while (head >= heads) head -= heads, ++tok;
    }
}

}  // namespace fa
