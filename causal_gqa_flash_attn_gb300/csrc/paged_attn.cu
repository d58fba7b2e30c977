// paged_attn.cu -- attention of ragged queries over 4-bit pages (include/fa.h,
// fa_paged_attn).
//
// Query t of a request with n queries and L rows sits at position p = L - n + t
// and attends keys j <= p (with win > 0 only sinks and the recent window):
//   s_j = scale * q . k_j,  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
//   lse = m + log sum_j exp(s_j - m),  m = max_j s_j.
//
// One block per (token, q head). Its warps take the row groups in turn, a lane
// holds head_dim / 32 dims, and the warps' running maxima, sums and outputs
// are joined in shared memory at the end.
#include <cuda_bf16.h>

#include <cmath>

#include "fa_device.cuh"
#include "fa_internal.h"
#include "paged_layout.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;

template <typename T> __device__ __forceinline__ float to_f(T x) { return static_cast<float>(x); }
template <typename T> __device__ __forceinline__ T from_f(float x) { return static_cast<T>(x); }

template <typename T, int HD>
__global__ void __launch_bounds__(32 * kWarps) paged_attn_kernel(PagedAttnArgs a) {
    constexpr int V = HD / 32;  // values a lane holds: V * lane ..
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int tok = blockIdx.x, h = blockIdx.y, hk = h / (a.n_q_heads / a.pages.n_kv);
    if (tok == 0 && h == 0)
        for (int r = threadIdx.x; r < a.n_reqs; r += 32 * kWarps) {
            const int c0 = __ldg(a.cu_q + r), c1 = __ldg(a.cu_q + r + 1);
            if (c0 < 0 || c1 < c0 || c1 > a.n_tokens) flag_error(a.err, FA_ERRBIT_DEVICE);
        }
    // the request that holds the token
    int lo = 0, hi = a.n_reqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu_q + mid) <= tok) lo = mid; else hi = mid;
    }
    const int q0 = __ldg(a.cu_q + lo), q1 = __ldg(a.cu_q + lo + 1);
    const int rows = __ldg(a.seq_lens + lo);
    if (tok < q0 || tok >= q1) return;
    const long long room = static_cast<long long>(a.pages.max_pages) * a.pages.groups * kGroupRows;
    if (rows < 0 || rows > room || q1 > a.n_tokens) {
        if (threadIdx.x == 0) flag_error(a.err, FA_ERRBIT_DEVICE);
        return;
    }
    const int p = rows - q1 + tok;
    float q[V], o[V], m = -INFINITY, l = 0.0f;
    const T *qp = static_cast<const T *>(a.q) + tok * a.q_stride + h * HD + V * lane;
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] = to_f(qp[i]) * a.scale, o[i] = 0.0f;
    const int b = V * lane / 32, e0 = V * lane % 32;
    for (int gi = w; gi * kGroupRows <= p; gi += kWarps) {
        const int j0 = gi * kGroupRows;
        if (a.win > 0 && j0 >= a.sink && j0 + kGroupRows - 1 < p - a.win + 1) continue;
        const uint8_t *src = group_at<HD>(a.pages, lo, hk, gi, lane ? nullptr : a.err);
        if (!src) continue;
        const uint8_t *sv = src + part_bytes(HD);
        for (int r = 0; r < kGroupRows; ++r) {
            if (!key_visible(p, j0 + r, a.sink, a.win)) continue;
            auto factor = [&](const uint8_t *part) {
                return __uint_as_float(static_cast<uint32_t>(
                    *reinterpret_cast<const uint16_t *>(part + factor_offset(HD) + 2 * r)) << 16);
            };
            auto scale = [&](const uint8_t *x) {
                return __half2float(*reinterpret_cast<const __half *>(x));
            };
            const float sk = scale(src + k_scale_at<HD>(r, b)) * factor(src);
            const float sc = scale(sv + v_scale_at<HD>(r, b)) * factor(sv);
            float dot = 0.0f, v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = e0 + i;
                const int kb = src[k_word_at<HD>(r, b, e / 8) + e % 8 / 2] >> (e % 2 * 4) & 15;
                const int vb = sv[v_half_at<HD>(r, b, e / 4) + e % 4 / 2] >> (e % 2 * 4) & 15;
                dot += q[i] * (static_cast<float>(kb - 8) * sk);
                v[i] = static_cast<float>(vb - 8) * sc;
            }
#pragma unroll
            for (int k = 16; k; k >>= 1) dot += __shfl_xor_sync(~0u, dot, k);
            const float mn = fmaxf(m, dot), c = expf(m - mn), x = expf(dot - mn);
            m = mn;
            l = l * c + x;
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = o[i] * c + x * v[i];
        }
    }
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][HD];
    if (lane == 0) sm[w] = m, sl[w] = l;
#pragma unroll
    for (int i = 0; i < V; ++i) so[w][V * lane + i] = o[i];
    __syncthreads();
    float M = sm[0], L = 0.0f;
    for (int k = 1; k < kWarps; ++k) M = fmaxf(M, sm[k]);
    const float ref = M == -INFINITY ? 0.0f : M;
    for (int k = 0; k < kWarps; ++k) L += sl[k] * expf(sm[k] - ref);
    for (int d = threadIdx.x; d < HD; d += 32 * kWarps) {
        float x = 0.0f;
        for (int k = 0; k < kWarps; ++k) x += so[k][d] * expf(sm[k] - ref);
        static_cast<T *>(a.out)[tok * a.out_stride + h * HD + d] =
            from_f<T>(L > 0.0f ? x / L : 0.0f);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[static_cast<size_t>(h) * a.n_tokens + tok] =
            L > 0.0f ? M + logf(L) : -INFINITY;
}

template <typename T>
cudaError_t launch_type(const PagedAttnArgs &a, int hd, cudaStream_t stream) {
    const dim3 grid(a.n_tokens, a.n_q_heads);
    auto kernel = hd == 64    ? paged_attn_kernel<T, 64>
                  : hd == 128 ? paged_attn_kernel<T, 128>
                              : paged_attn_kernel<T, 256>;
    kernel<<<grid, 32 * kWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t paged_attn_ws_bytes(int hd) { return 256; }

cudaError_t launch_paged_attn(const PagedAttnArgs &a, int dtype, int hd, cudaStream_t stream) {
    switch (dtype) {
        case kTypeF32: return launch_type<float>(a, hd, stream);
        case kTypeF16: return launch_type<__half>(a, hd, stream);
        default: return launch_type<__nv_bfloat16>(a, hd, stream);
    }
}

}  // namespace fa
