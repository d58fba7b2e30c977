// paged_kv.cu -- 4-bit pages written and read back (include/fa.h,
// fa_paged_append and fa_paged_gather; byte order in paged_layout.cuh).
//
// Append: one row of K or V of one kv head takes head_dim / 8 lanes, 8
// consecutive values each (one word of codes). A 32-value block is four lanes:
// amax by two shuffles, d = amax / -8, code = round(x / d) + 8 as in the Q4_0
// planes; the row's largest d, by shuffles over its lanes, gives the row's
// power-of-two factor. One pass, bound by HBM on long prompts.
//
// Gather: one warp per 16-row group reads its fragments with 16-byte loads and
// writes the dequantised rows, rounded to binary16, into fp16 planes that
// fa_prefill_chunk reads in place. Bound by HBM (it writes 3.5 bytes for each
// byte read).
#include <algorithm>

#include <cuda_bf16.h>

#include "fa_device.cuh"
#include "fa_internal.h"
#include "paged_layout.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T *p, float *x);
template <>
__device__ __forceinline__ void load8<float>(const float *p, float *x) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__half>(const __half *p, float *x) {
    const uint4 w = __ldg(reinterpret_cast<const uint4 *>(p));
    const __half2 *h = reinterpret_cast<const __half2 *>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float *x) {
    const uint4 w = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(h[i] << 16);
        x[2 * i + 1] = __uint_as_float(h[i] & 0xffff0000u);
    }
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(PagedAppendArgs a) {
    constexpr int LANES = HD / 8;  // lanes of a row
    const long long id = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x;
    const long long row = id / LANES;  // (token, kv head, part): part fastest
    const int l = static_cast<int>(id) & (LANES - 1);
    const int part = static_cast<int>(row & 1);
    const long long th = row >> 1;
    const int tok = static_cast<int>(th / a.n_kv), h = static_cast<int>(th % a.n_kv);
    const bool in = tok < a.n_tokens;
    const int slot = in ? __ldg(a.slot_map + tok) : -1;
    const int page = slot >> a.page_shift;
    const bool live = slot >= 0 && page < a.n_pages;
    if (in && slot != -1 && !live && l == 0) flag_error(a.err, FA_ERRBIT_DEVICE);
    float x[8];
    if (live) {
        const T *src = static_cast<const T *>(part ? a.v : a.k) +
                       tok * (part ? a.v_stride : a.k_stride) + static_cast<long long>(h) * HD;
        load8<T>(src + 8 * l, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.0f;
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
    amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
    const float d = __fdiv_rn(amax, -8.0f);
    const float inv = d != 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = min(max(__float2int_rn(__fmul_rn(x[i], inv)), -8), 7) + 8;
        word |= static_cast<uint32_t>(c) << (4 * i);
    }
    // the row's factor: the power of two at or below its largest |d|, kept
    // inside the normal range so that it and its inverse are exact
    float top = fabsf(d);
#pragma unroll
    for (int m = 4; m < LANES; m <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, m));
    const uint32_t ex = min(max(__float_as_uint(top) >> 23, 1u), 254u);
    const float factor = top > 0.0f ? __uint_as_float(ex << 23) : 1.0f;
    const __half scale = __float2half_rn(__fdiv_rn(d, factor));
    if (!live) return;
    const int pos = slot & ((1 << a.page_shift) - 1);
    const int r = pos & (kGroupRows - 1), b = l >> 2, t = l & 3;
    uint8_t *dst = a.pages + ((static_cast<size_t>(page) * a.n_kv + h) *
                                  ((1 << a.page_shift) / kGroupRows) + pos / kGroupRows) *
                                 group_bytes(HD) + part * part_bytes(HD);
    if (part == 0) {
        *reinterpret_cast<uint32_t *>(dst + k_word_at<HD>(r, b, t)) = word;
    } else {
        *reinterpret_cast<uint16_t *>(dst + v_half_at<HD>(r, b, 2 * t)) =
            static_cast<uint16_t>(word);
        *reinterpret_cast<uint16_t *>(dst + v_half_at<HD>(r, b, 2 * t + 1)) =
            static_cast<uint16_t>(word >> 16);
    }
    if (t == 0)
        *reinterpret_cast<__half *>(
            dst + (part == 0 ? k_scale_at<HD>(r, b) : v_scale_at<HD>(r, b))) = scale;
    if (l == 0)
        *reinterpret_cast<uint16_t *>(dst + factor_offset(HD) + 2 * r) =
            static_cast<uint16_t>(__float_as_uint(factor) >> 16);
}

// 4 codes (the low 16 bits) -> 4 binary16 values (c - 8) * s, the product in
// fp32 as the attention's definition has it.
__device__ __forceinline__ uint2 dequant4(uint32_t c, float s) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = __fmul_rn(static_cast<float>(static_cast<int>((c >> (4 * i)) & 15u) - 8), s);
    return make_uint2(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]));
}

__device__ __forceinline__ float row_factor(const uint8_t *part, int hd, int r) {
    const uint32_t w = __ldg(reinterpret_cast<const uint16_t *>(part + factor_offset(hd)) + r);
    return __uint_as_float(w << 16);
}
__device__ __forceinline__ float block_scale(const uint8_t *p) {
    return __half2float(__ldg(reinterpret_cast<const __half *>(p)));
}

template <int HD>
__global__ void __launch_bounds__(kThreads) paged_gather_kernel(PagedGatherArgs a) {
    constexpr int NB = HD / 32;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int h = blockIdx.y, r = blockIdx.z;
    int rows = __ldg(a.seq_lens + r);
    const long long room = min(static_cast<long long>(a.max_seq),
                               static_cast<long long>(a.pages.max_pages) * a.pages.groups *
                                   kGroupRows);
    if (rows < 0 || rows > room) {
        if (threadIdx.x == 0 && blockIdx.x == 0) flag_error(a.err, FA_ERRBIT_DEVICE);
        rows = rows < 0 ? 0 : static_cast<int>(room);
    }
    const int n = (rows + kGroupRows - 1) / kGroupRows;
    for (int i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < n;
         i += gridDim.x * (kThreads / 32)) {
        const uint8_t *src = group_at<HD>(a.pages, r, h, i, lane ? nullptr : a.err);
        if (!src) continue;
        const int left = rows - i * kGroupRows;  // rows of the group that exist
        const size_t at = static_cast<size_t>(r) * a.plane_bytes +
                          (static_cast<size_t>(h) * a.max_seq + i * kGroupRows) * (HD * 2);
#pragma unroll
        for (int c = 0; c < NB / 2; ++c) {
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(src) + c * 32 + lane);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = 4 * c + k, row = g + (j / NB) * 8, b = j % NB;
                if (row >= left) continue;
                const float s = block_scale(src + k_scale_at<HD>(row, b)) *
                                row_factor(src, HD, row);
                const uint2 lo = dequant4(ws[k], s), hi = dequant4(ws[k] >> 16, s);
                *reinterpret_cast<uint4 *>(a.k_planes + at + (row * HD + 32 * b + 8 * t) * 2) =
                    make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
        }
        const uint8_t *sv = src + part_bytes(HD);
#pragma unroll
        for (int c = 0; c < NB / 2; ++c) {
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(sv) + c * 32 + lane);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int j = 8 * c + k, x = j / NB, b = j % NB;
                const int row = 2 * t + (x & 1) + 8 * (x >> 1);
                if (row >= left) continue;
                const float s = block_scale(sv + v_scale_at<HD>(row, b)) *
                                row_factor(sv, HD, row);
                *reinterpret_cast<uint2 *>(a.v_planes + at + (row * HD + 32 * b + 4 * g) * 2) =
                    dequant4(ws[k >> 1] >> (16 * (k & 1)), s);
            }
        }
    }
}

template <typename T>
cudaError_t append_type(const PagedAppendArgs &a, int hd, cudaStream_t stream) {
    const long long threads = 2ll * a.n_tokens * a.n_kv * (hd / 8);
    const long long blocks = (threads + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    auto kernel = hd == 64    ? paged_append_kernel<T, 64>
                  : hd == 128 ? paged_append_kernel<T, 128>
                              : paged_append_kernel<T, 256>;
    kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs &a, int dtype, int hd, cudaStream_t stream) {
    switch (dtype) {
        case kTypeF32: return append_type<float>(a, hd, stream);
        case kTypeF16: return append_type<__half>(a, hd, stream);
        default: return append_type<__nv_bfloat16>(a, hd, stream);
    }
}

cudaError_t launch_paged_gather(const PagedGatherArgs &a, int n_reqs, int hd,
                                cudaStream_t stream) {
    const int groups = (a.max_seq + kGroupRows - 1) / kGroupRows;
    const long long pairs = static_cast<long long>(n_reqs) * a.pages.n_kv;
    const int need = (groups + kThreads / 32 - 1) / (kThreads / 32);
    const long long cap = std::max<long long>(1, device_sm_count() * 16ll / pairs);
    const dim3 grid(static_cast<unsigned>(std::min<long long>(need, cap)), a.pages.n_kv, n_reqs);
    auto kernel = hd == 64    ? paged_gather_kernel<64>
                  : hd == 128 ? paged_gather_kernel<128>
                              : paged_gather_kernel<256>;
    kernel<<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace fa
