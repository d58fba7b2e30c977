// paged_layout.cuh -- byte order of the 4-bit pages (include/fa.h, "4-bit
// pages") and the block-table lookup that the paged kernels share.
//
// A group of 16 rows of one kv head is a K part followed by a V part. The
// codes of a part are stored as the A operand fragments of mma.m16n8k16 that
// the attention kernel feeds to the tensor cores, so that a warp reads them
// with conflict-free 16-byte loads and no shuffle: lane 4 g + t finds its
// codes in the 16-byte chunks [c][lane], c < head_dim / 64.
//   K: the lane's words, in order j = (r / 8) * nb + b, are block b of row
//      r = g or g + 8; word (b, t) holds dims 32 b + 8 t .. + 7.
//   V: the lane's 16-bit halves, in order j = x * nb + b, are block b of row
//      r = 2 t + (x & 1) + 8 (x >> 1); half (b, g) holds dims 32 b + 4 g .. + 3.
// nb = head_dim / 32; the code of the lowest dim is in the lowest 4 bits.
#pragma once

#include <cstddef>
#include <cstdint>

#include "fa_device.cuh"
#include "fa_internal.h"
#include "paged_launch.cuh"

namespace fa {

constexpr int kGroupRows = 16;  // rows of a stored group

__host__ __device__ constexpr int part_bytes(int hd) { return 9 * hd + 32; }
__host__ __device__ constexpr int group_bytes(int hd) { return 2 * part_bytes(hd); }
__host__ __device__ constexpr int scale_offset(int hd) { return 8 * hd; }
__host__ __device__ constexpr int factor_offset(int hd) { return 9 * hd; }

// Byte of the word that holds dims 32 b + 8 t .. + 7 of K row r.
template <int HD>
__device__ __forceinline__ int k_word_at(int r, int b, int t) {
    const int j = (r >> 3) * (HD / 32) + b;
    return ((j >> 2) * 32 + (r & 7) * 4 + t) * 16 + (j & 3) * 4;
}
// Byte of the 16-bit half that holds dims 32 b + 4 g .. + 3 of V row r.
template <int HD>
__device__ __forceinline__ int v_half_at(int r, int b, int g) {
    const int x = (r & 1) + 2 * (r >> 3), t = (r & 7) >> 1;
    const int j = x * (HD / 32) + b;
    return ((j >> 3) * 32 + g * 4 + t) * 16 + (j & 7) * 2;
}
// Bytes of block scales inside a part.
template <int HD>
__device__ __forceinline__ int k_scale_at(int r, int b) {
    return scale_offset(HD) + 2 * (r * (HD / 32) + b);
}
template <int HD>
__device__ __forceinline__ int v_scale_at(int r, int b) {
    const int x = (r & 1) + 2 * (r >> 3), t = (r & 7) >> 1;
    return scale_offset(HD) + 2 * ((((b >> 1) * 4 + t) << 3) + (b & 1) * 4 + x);
}

// The pages of one call.
struct Pages {
    const uint8_t *base;
    const int32_t *table;  // [requests][max_pages]
    int n_pages, n_kv, max_pages;
    int groups;            // row groups of a page and head (page_rows / 16)
    int group_shift;       // log2(groups)
};

struct PagedGatherArgs {
    Pages pages;
    const int32_t *seq_lens;
    uint8_t *k_planes, *v_planes;
    size_t plane_bytes;
    int max_seq;
    unsigned *err;
};

struct PagedAttnArgs {
    const void *q;
    void *out;
    float *lse;  // [n_q_heads][n_tokens] or null
    long long q_stride, out_stride;  // elements between tokens
    const int32_t *cu_q, *seq_lens;
    Pages pages;
    int n_reqs, n_tokens, n_q_heads, sink, win;
    float scale;
    uint8_t *workspace;
    unsigned *err;
    // fa_paged_attn_scored
    float cap = 0.0f;     // 0: none
    float cap_in = 0.0f;  // of a score in the exp2 domain: 2 / cap, or 1 / (cap log2 e) for fp32
    const float *slopes = nullptr;
};

// Address of group `i` of kv head h of request r, or nullptr (flagged) where
// the table names no page.
template <int HD>
__device__ __forceinline__ const uint8_t *group_at(const Pages &P, int r, int h, int i,
                                                   unsigned *err) {
    const int page = load(P.table + static_cast<size_t>(r) * P.max_pages + (i >> P.group_shift));
    if (page < 0 || page >= P.n_pages) {
        flag_error(err, FA_ERRBIT_DEVICE);
        return nullptr;
    }
    return P.base + ((static_cast<size_t>(page) * P.n_kv + h) * P.groups +
                     (i & (P.groups - 1))) * group_bytes(HD);
}

}  // namespace fa
