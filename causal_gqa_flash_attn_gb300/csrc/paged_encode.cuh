// paged_encode.cuh -- rows encoded into 4-bit pages (paged_kv.cu, rope_append.cu;
// byte order in paged_layout.cuh).
#pragma once

#include <cuda_bf16.h>

#include "fa_device.cuh"
#include "fa_internal.h"
#include "paged_launch.cuh"
#include "paged_layout.cuh"

namespace fa {

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

// A row's 16 values of lane l, quantised, into the K (or V) part of its page.
template <int HD, bool V>
__device__ __forceinline__ void put_row(const PagedAppendArgs &a, const uint32_t *w, __half scale, uint16_t factor,
                                        int slot, int page, int h, int l) {
    const int pos = slot & ((1 << a.page_shift) - 1);
    const int r = pos & (kGroupRows - 1), b = l >> 1, t = 2 * (l & 1);
    uint8_t *dst = a.pages + ((static_cast<size_t>(page) * a.n_kv + h) * ((1 << a.page_shift) / kGroupRows) +
                              pos / kGroupRows) * group_bytes(HD) + (V ? part_bytes(HD) : 0);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (V) {
            *reinterpret_cast<uint16_t *>(dst + v_half_at<HD>(r, b, 2 * (t + j))) = static_cast<uint16_t>(w[j]);
            *reinterpret_cast<uint16_t *>(dst + v_half_at<HD>(r, b, 2 * (t + j) + 1)) = static_cast<uint16_t>(w[j] >> 16);
        } else {
            *reinterpret_cast<uint32_t *>(dst + k_word_at<HD>(r, b, t + j)) = w[j];
        }
    }
    if (t == 0) *reinterpret_cast<__half *>(dst + (V ? v_scale_at<HD>(r, b) : k_scale_at<HD>(r, b))) = scale;
    if (l == 0) *reinterpret_cast<uint16_t *>(dst + factor_offset(HD) + 2 * r) = factor;
}

// 16 values of K and of V of a token's row of kv head h, those of lane l, into the pages. All
// lanes of a row, and of the warp, call; rows that are not live are encoded and left out.
template <int HD>
__device__ __forceinline__ void encode_rows(const PagedAppendArgs &a, const float *k, const float *v, bool live,
                                            int slot, int page, int h, int l) {
    uint32_t kw[2], vw[2];
    __half ks, vs;
    uint16_t kf, vf;
    quantise16<HD / 16>(k, kw, &ks, &kf);
    quantise16<HD / 16>(v, vw, &vs, &vf);
    if (!live) return;
    put_row<HD, false>(a, kw, ks, kf, slot, page, h, l);
    put_row<HD, true>(a, vw, vs, vf, slot, page, h, l);
}

// The same for one of both: 16 values of a row of K (or V).
template <int HD, bool V>
__device__ __forceinline__ void encode_row(const PagedAppendArgs &a, const float *x, bool live, int slot, int page,
                                           int h, int l) {
    uint32_t w[2];
    __half scale;
    uint16_t factor;
    quantise16<HD / 16>(x, w, &scale, &factor);
    if (live) put_row<HD, V>(a, w, scale, factor, slot, page, h, l);
}

}  // namespace fa
