// paged_kv.cu -- 4-bit pages written and read back (include/fa.h,
// fa_paged_append and fa_paged_gather; byte order in paged_layout.cuh).
//
// Append: one token's rows of K and V of one kv head take head_dim / 16 lanes, 16
// consecutive values of each a lane (two words of codes). A 32-value block is two lanes:
// amax by a shuffle, d = amax / -8, code = round(x / d) + 8 as in the Q4_0
// planes; the row's largest d, by shuffles over its lanes, gives the row's
// power-of-two factor. One pass, bound by the instructions that a value costs:
// 131072 tokens of 2 kv heads x 256 in bf16 take 69 us, 5.0 TB/s (8 values a lane,
// each converted and clamped as an integer, with K and V in different lanes and a
// division for each row's place: 143 us; with K and V in one lane, 100).
//
// Gather: one warp per 16-row group reads its fragments with 16-byte loads and
// writes the dequantised rows, rounded to binary16, into fp16 planes that
// fa_prefill_chunk reads in place. Bound by HBM, and there by its writes, 3.5
// bytes for each byte read: 12 requests of 9517 rows (8 kv heads x 128), 632 MB with the
// append, take 99.5 us, 6.35 TB/s (a copy reaches 6.8, a fill alone 4.0). Dequantising
// in fp32 instead of packed binary16 took 114 us, scalar loads of the scales 16.5 instead
// of 14.5 us for 8192 rows.
#include <algorithm>

#include <cuda_bf16.h>

#include "fa_device.cuh"
#include "fa_internal.h"
#include "paged_launch.cuh"
#include "paged_layout.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;        // of the gather
constexpr int kAppendThreads = 128;

template <typename T>
__device__ __forceinline__ void load8(const T *p, float *x);
template <>
__device__ __forceinline__ void load8<float>(const float *p, float *x) {
    const float4 a = load(reinterpret_cast<const float4 *>(p));
    const float4 b = load(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__half>(const __half *p, float *x) {
    const uint4 w = load(reinterpret_cast<const uint4 *>(p));
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
    const uint4 w = load(reinterpret_cast<const uint4 *>(p));
    const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(h[i] << 16);
        x[2 * i + 1] = __uint_as_float(h[i] & 0xffff0000u);
    }
}

// max(a, |x|), NaN if either is one.
__device__ __forceinline__ float max_abs(float a, float x) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(x)));
    return d;
}

// 16 values of a row, half a block, as codes (two words), their block's scale and the row's
// factor. With finite values and a finite 1 / d the products lie in [-8, 8] but for a rounding,
// so that one minimum clamps them, and the sum with 1.5 * 2^23 + 8 rounds half to even and has
// the code in its lowest 4 bits.
template <int LANES>
__device__ __forceinline__ void quantise16(const float *x, uint32_t *word, __half *scale, uint16_t *factor) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) most = max_abs(most, x[i]);
    most = max_abs(most, __shfl_xor_sync(~0u, most, 1));
    float amax = most;
    if (most != most) {  // a NaN never raises the largest magnitude
        amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
    }
    amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
    const float d = __fmul_rn(amax, -0.125f);  // amax / -8, rounded alike
    const float inv = d != 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
    if (fabsf(inv) <= 3.4e38f && most <= 3.4e38f) {  // and not a NaN
        constexpr float kMagic = 12582920.0f;
        constexpr uint32_t kBits = 0x4b400000u * 0x11111111u;  // what the sums' other bits add up to
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t w = 0;
#pragma unroll
            for (int i = 7; i >= 0; --i)
                w = w * 16u + __float_as_uint(__fadd_rn(fminf(__fmul_rn(x[8 * j + i], inv), 7.0f), kMagic));
            word[j] = w - kBits;
        }
    } else {
        // as Q4_0's encoder for anything: a NaN product is 0, +-inf the last code of its side
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            word[j] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = min(max(__float2int_rn(__fmul_rn(x[8 * j + i], inv)), -8), 7) + 8;
                word[j] |= static_cast<uint32_t>(c) << (4 * i);
            }
        }
    }
    // the row's factor: the power of two at or below its largest |d|, kept
    // inside the normal range so that it and its inverse are exact
    float top = fabsf(d);
#pragma unroll
    for (int m = 2; m < LANES; m <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, m));
    const uint32_t ex = top > 0.0f ? min(max(__float_as_uint(top) >> 23, 1u), 254u) : 127u;
    // 2^(127 - ex), the factor's inverse: for ex = 254 it is below the normal range
    const float down = ex < 254u ? __uint_as_float((254u - ex) << 23) : __uint_as_float(1u << 22);
    *scale = __float2half_rn(__fmul_rn(d, down));
    *factor = static_cast<uint16_t>(ex << 7);
}

template <typename T, int HD>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(PagedAppendArgs a) {
    wait_for_stream();
    constexpr int LANES = HD / 16;  // lanes of a row
    const int tok = blockIdx.x * (kAppendThreads / LANES) + threadIdx.x / LANES, h = blockIdx.y;
    const int l = threadIdx.x & (LANES - 1);
    const bool in = tok < a.n_tokens;
    const int slot = in ? load(a.slot_map + tok) : -1;
    const int page = slot >> a.page_shift;
    const bool live = slot >= 0 && page < a.n_pages;
    if (in && slot != -1 && !live && l == 0) flag_error(a.err, FA_ERRBIT_DEVICE);
    float k[16] = {}, v[16] = {};
    if (live) {
        const long long at = static_cast<long long>(h) * HD + 16 * l;
        const T *src = static_cast<const T *>(a.k) + tok * a.k_stride + at;
        load8<T>(src, k);
        load8<T>(src + 8, k + 8);
        src = static_cast<const T *>(a.v) + tok * a.v_stride + at;
        load8<T>(src, v);
        load8<T>(src + 8, v + 8);
    }
    uint32_t kw[2], vw[2];
    __half ks, vs;
    uint16_t kf, vf;
    quantise16<LANES>(k, kw, &ks, &kf);
    quantise16<LANES>(v, vw, &vs, &vf);
    if (!live) return;
    const int pos = slot & ((1 << a.page_shift) - 1);
    const int r = pos & (kGroupRows - 1), b = l >> 1, t = 2 * (l & 1);
    uint8_t *dst = a.pages + ((static_cast<size_t>(page) * a.n_kv + h) *
                                  ((1 << a.page_shift) / kGroupRows) + pos / kGroupRows) *
                                 group_bytes(HD);
    uint8_t *dv = dst + part_bytes(HD);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        *reinterpret_cast<uint32_t *>(dst + k_word_at<HD>(r, b, t + j)) = kw[j];
        *reinterpret_cast<uint16_t *>(dv + v_half_at<HD>(r, b, 2 * (t + j))) = static_cast<uint16_t>(vw[j]);
        *reinterpret_cast<uint16_t *>(dv + v_half_at<HD>(r, b, 2 * (t + j) + 1)) =
            static_cast<uint16_t>(vw[j] >> 16);
    }
    if (t == 0) {
        *reinterpret_cast<__half *>(dst + k_scale_at<HD>(r, b)) = ks;
        *reinterpret_cast<__half *>(dv + v_scale_at<HD>(r, b)) = vs;
    }
    if (l == 0) {
        *reinterpret_cast<uint16_t *>(dst + factor_offset(HD) + 2 * r) = kf;
        *reinterpret_cast<uint16_t *>(dv + factor_offset(HD) + 2 * r) = vf;
    }
}

// 8 codes c of a word -> (c - 8) * s rounded to binary16, in order. The product
// is exact in fp32 (4 bits times 11); in binary16 arithmetic it is the same,
// rounded once, where s itself is a binary16 number. A code in bits 0-3 or 4-7
// of a half word under the bits of 1024 is 1024 + c or 1024 + 16 c: a well-known way
// of 4-bit products, whose constants (1032, 72 = 64 + 8) follow from binary16.
__device__ __forceinline__ uint32_t lop_or(uint32_t w, uint32_t mask, uint32_t bits) {
    return (w & mask) | bits;
}
__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<__half2 *>(&w); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }

__device__ __forceinline__ uint4 dequant8(uint32_t w, float s) {
    const __half sh = __float2half_rn(s);
    if (__half2float(sh) != s) {  // beyond binary16's range, or below its normal one
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = pack_half2(static_cast<float>(static_cast<int>(w >> (8 * i) & 15u) - 8) * s,
                              static_cast<float>(static_cast<int>(w >> (8 * i + 4) & 15u) - 8) * s);
        return make_uint4(o[0], o[1], o[2], o[3]);
    }
    const __half2 s2 = __half2half2(sh);
    const __half2 off = __float2half2_rn(-1032.0f), sixteenth = __float2half2_rn(0.0625f);
    const __half2 off16 = __float2half2_rn(-72.0f);
    const uint32_t v = w >> 8;
    // codes (0, 4), (1, 5), (2, 6), (3, 7)
    const uint32_t a = as_u32(__hmul2(__hadd2(as_half2(lop_or(w, 0x000f000fu, 0x64006400u)), off), s2));
    const uint32_t b = as_u32(
        __hmul2(__hfma2(as_half2(lop_or(w, 0x00f000f0u, 0x64006400u)), sixteenth, off16), s2));
    const uint32_t c = as_u32(__hmul2(__hadd2(as_half2(lop_or(v, 0x000f000fu, 0x64006400u)), off), s2));
    const uint32_t d = as_u32(
        __hmul2(__hfma2(as_half2(lop_or(v, 0x00f000f0u, 0x64006400u)), sixteenth, off16), s2));
    return make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(c, d, 0x5410), __byte_perm(a, b, 0x7632),
                      __byte_perm(c, d, 0x7632));
}

__device__ __forceinline__ float half_of(uint32_t w, int hi) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(hi ? w >> 16 : w & 0xffffu)));
}
__device__ __forceinline__ float factor_of(uint32_t w, int hi) {  // bfloat16
    return __uint_as_float(hi ? w & 0xffff0000u : w << 16);
}
template <int N>
__device__ __forceinline__ void load_words(uint32_t *w, const uint8_t *p) {
    if constexpr (N == 4) {
        const uint4 x = load(reinterpret_cast<const uint4 *>(p));
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else if constexpr (N == 2) {
        const uint2 x = load(reinterpret_cast<const uint2 *>(p));
        w[0] = x.x; w[1] = x.y;
    } else {
        w[0] = load(reinterpret_cast<const uint32_t *>(p));
    }
}

template <int HD>
__global__ void __launch_bounds__(kThreads) paged_gather_kernel(PagedGatherArgs a) {
    wait_for_stream();
    constexpr int NB = HD / 32;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int h = blockIdx.y, r = blockIdx.z;
    int rows = load(a.seq_lens + r);
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
        const uint8_t *sv = src + part_bytes(HD);
        const int left = rows - i * kGroupRows;  // rows of the group that exist
        const size_t at = static_cast<size_t>(r) * a.plane_bytes +
                          (static_cast<size_t>(h) * a.max_seq + i * kGroupRows) * (HD * 2);
        // everything the lane needs of the group: codes, scales and factors
        uint32_t kw[2 * NB], vw[2 * NB], ks[NB], vs[2 * NB];
#pragma unroll
        for (int c = 0; c < NB / 2; ++c) {
            load_words<4>(kw + 4 * c, src + (c * 32 + lane) * 16);
            load_words<4>(vw + 4 * c, sv + (c * 32 + lane) * 16);
            load_words<4>(vs + 4 * c, sv + scale_offset(HD) + (c * 4 + t) * 16);
        }
        load_words<NB / 2>(ks, src + scale_offset(HD) + g * (2 * NB));
        load_words<NB / 2>(ks + NB / 2, src + scale_offset(HD) + (g + 8) * (2 * NB));
        const uint16_t *kf = reinterpret_cast<const uint16_t *>(src + factor_offset(HD)) + g;
        const uint32_t *vf = reinterpret_cast<const uint32_t *>(sv + factor_offset(HD)) + t;
        const uint32_t kf01 = load(kf) | static_cast<uint32_t>(load(kf + 8)) << 16;
        const uint32_t vf01 = load(vf), vf23 = load(vf + 4);
        // K: the lane's word (row g or g + 8, block b) is dims 32 b + 8 t ..
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j) {
            const int row = g + (j / NB) * 8, b = j % NB;
            if (row >= left) continue;
            const float s = half_of(ks[(j / NB) * (NB / 2) + b / 2], b & 1) * factor_of(kf01, j / NB);
            *reinterpret_cast<uint4 *>(a.k_planes + at + (row * HD + 32 * b + 8 * t) * 2) =
                dequant8(kw[j], s);
        }
        // V: a word is two blocks of row 2 t + (x & 1) + 8 (x >> 1), dims 32 b + 4 g .. of each
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j) {
            const int x = 2 * j / NB, b = 2 * j % NB;
            const int row = 2 * t + (x & 1) + 8 * (x >> 1);
            if (row >= left) continue;
            // scales of blocks b, b + 1: four rows each in words b and b + 1
            const float f = factor_of(x < 2 ? vf01 : vf23, x & 1);
            const float s0 = half_of(vs[2 * b + (x >> 1)], x & 1) * f;
            const float s1 = half_of(vs[2 * b + 2 + (x >> 1)], x & 1) * f;
            const uint4 lo = dequant8(vw[j], s0), hi = dequant8(vw[j], s1);
            uint8_t *dst = a.v_planes + at + (row * HD + 32 * b + 4 * g) * 2;
            *reinterpret_cast<uint2 *>(dst) = make_uint2(lo.x, lo.y);
            *reinterpret_cast<uint2 *>(dst + 64) = make_uint2(hi.z, hi.w);
        }
    }
}

template <typename T>
cudaError_t append_type(const PagedAppendArgs &a, int hd, cudaStream_t stream) {
    const int rows = kAppendThreads / (hd / 16);  // tokens of a block, one kv head of each
    const dim3 grid((a.n_tokens - 1) / rows + 1, a.n_kv);
    auto kernel = hd == 64    ? paged_append_kernel<T, 64>
                  : hd == 128 ? paged_append_kernel<T, 128>
                              : paged_append_kernel<T, 256>;
    return launch_after(kernel, grid, kAppendThreads, 0, stream, a);
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
    const long long cap = std::max<long long>(1, device_sm_count() * 64ll / pairs);
    const dim3 grid(static_cast<unsigned>(std::min<long long>(need, cap)), a.pages.n_kv, n_reqs);
    auto kernel = hd == 64    ? paged_gather_kernel<64>
                  : hd == 128 ? paged_gather_kernel<128>
                              : paged_gather_kernel<256>;
    return launch_after(kernel, grid, kThreads, 0, stream, a);
}

}  // namespace fa
