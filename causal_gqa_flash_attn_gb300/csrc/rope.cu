// rope.cu -- rotary positions on the query and key heads, with one position
// axis or several (time, height, width of images and video), and the inverse
// rotation, which is the gradient of the rotation (include/fa.h, fa_rope).
//
// Pair i of a head, (x, y), is rotated by the angle a = pos[axis(i)] * f_i:
//   x' = x cos a - y sin a,   y' = x sin a + y cos a.
// The angle is taken modulo a turn in exact integer arithmetic: the table
// holds F_i = 2^64 f_i / (2 pi), and the top 32 bits of pos * F_i mod 2^64 are
// the angle in 2^-32 turns, without the 64-bit floating-point units (a few per
// SM). sincospif then sees an argument in [-1, 1). In turns the angle is off by
// |pos| (2^-64 + 2^-53 f_i / (2 pi)) at most from the table's entry, which is formed
// in double, by 2^-33 from the 32 bits and by 2^-26 from becoming an fp32 argument.
//
// The call is bound by HBM: every element is read and written once. A block
// takes a few tokens, puts their sines and cosines into shared memory (one for
// all heads) and streams the heads through, a thread two 16-byte vectors of a
// head at a time. What hides the latency is the number of threads, so these
// have few registers: with two or four heads in flight per thread (64 and 100
// registers), 20011 tokens of 40 heads took 71 and 105 us against 66. Sines in
// registers, a thread walking all heads of its pairs, took 88 us.
// 8192 tokens x 18 heads x 256 in bf16, a quarter rotated: 28.6 us (0.78 of HBM;
// the start and the sines take 3 us of it); 20011 x 40 x 128 in fp16: 67 us (0.90).
#include <algorithm>

#include <cuda_bf16.h>

#include "fa_device.cuh"
#include "fa_internal.h"
#include "paged_launch.cuh"

namespace fa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeItems = 1024;    // items (two vectors) that a block is given
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

// V values a thread moves at a time: 16 bytes, or 1 where a size, a stride or
// a pointer is not a multiple of that.
template <typename T, int V, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads, 6) rope_kernel(RopeArgs a) {
    wait_for_stream();
    using W = Vec<T, V>;
    extern __shared__ float4 rope_smem[];
    const int half = a.rotary_dim / 2;
    const int n_rot = half / V;            // items of V pairs
    const int n_items = n_rot + a.n_copy;  // and of 2 V values that stay as they are
    float *cs = reinterpret_cast<float *>(rope_smem);  // [tokens][half] cosines, then sines
    float *sn = cs + a.tokens_per_block * half;
    const int tok0 = blockIdx.x * a.tokens_per_block;
    const int n_tok = min(a.tokens_per_block, a.n_tokens - tok0);
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
    // (flagged by one block alone: in the loop above it took 7 registers, and 29.4 us instead of 28.6)
    if (blockIdx.x + blockIdx.y == 0)
        for (int i = threadIdx.x; i < half; i += kRopeThreads)
            if (load(static_cast<const uint4 *>(a.table) + i).z >= static_cast<unsigned>(a.n_axes))
                flag_error(a.err, FA_ERRBIT_DEVICE);
    __syncthreads();
    const int h0 = blockIdx.y * a.heads_per_block;
    const int heads = min(a.heads_per_block, a.n_q_heads + a.n_kv_heads - h0);
    // threads of a head, heads that the block takes at once, and this thread's first one
    const int lanes = min(n_items, kRopeThreads), rows = kRopeThreads / lanes;
    const int row = threadIdx.x / lanes, lane = threadIdx.x - row * lanes;
    if (row >= rows) return;
    int tok = row / heads, head = row - tok * heads;
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
                    *p = Conv<T>::put(u0 * c[pair] - u1 * s[pair]);
                    *q = Conv<T>::put(u0 * s[pair] + u1 * c[pair]);
                }
            }
            *reinterpret_cast<W *>(out + o0) = x;
            if (second) *reinterpret_cast<W *>(out + o1) = y;
        }
        head += rows;
        while (head >= heads) head -= heads, ++tok;
    }
}

template <typename T, int V>
cudaError_t launch(RopeArgs a, cudaStream_t stream) {
    const bool in_place = (a.n_q_heads == 0 || a.q == a.q_out) && (a.n_kv_heads == 0 || a.k == a.k_out);
    const int rest = a.head_dim - a.rotary_dim, half = a.rotary_dim / 2;
    a.n_copy = in_place ? 0 : (rest / V + 1) / 2;
    const int heads = a.n_q_heads + a.n_kv_heads;
    const long long row = static_cast<long long>(heads) * (half / V + a.n_copy);  // items of a token
    const int fit = std::min<int>(kRopeTokens, 48 * 1024 / (half * 8));
    int tokens = static_cast<int>(std::min<long long>(fit, std::max<long long>(1, kRopeItems / row)));
    // few tokens: a block takes one, and the heads are split over blocks too, so that
    // the GPU's SMs all have some
    const int sms = device_sm_count();
    if (a.n_tokens <= sms * tokens) tokens = std::max(1, a.n_tokens / sms);
    a.tokens_per_block = tokens;
    const int blocks = (a.n_tokens - 1) / tokens + 1;
    int parts = std::max(1, std::min(sms * 2 / blocks, heads / 2));
    a.heads_per_block = (heads + parts - 1) / parts;
    parts = (heads + a.heads_per_block - 1) / a.heads_per_block;
    const dim3 grid(static_cast<unsigned>(blocks), parts);
    const size_t smem = static_cast<size_t>(tokens) * half * 8;
    if (a.adjacent)
        return launch_after(rope_kernel<T, V, true>, grid, kRopeThreads, smem, stream, a);
    return launch_after(rope_kernel<T, V, false>, grid, kRopeThreads, smem, stream, a);
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
