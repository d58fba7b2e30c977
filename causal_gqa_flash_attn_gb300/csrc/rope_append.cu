// rope_append.cu -- q and k rotated to their positions, and the new rows of K and
// V written into 4-bit pages, in one pass (include/fa.h, fa_rope_append).
//
// What fa_rope and fa_paged_append do one after the other, bit for bit: k is rotated
// in fp32, rounded to its type and encoded. The rotated k is not written and read
// back, and a step has one launch less. A block takes a few tokens: their sines and
// cosines into shared memory, the q heads through them as in rope.cu, then each row
// of K and V by head_dim / 16 lanes as in paged_kv.cu, where a lane reads its 16
// values of k and the 16 that they are paired with.
//
// Bound by HBM and, close behind, by instructions (two thirds of the issue slots): 30000 tokens, 16/4 heads x 128 in
// bf16 68 us, 0.70 of HBM (fa_rope and fa_paged_append one behind the other 70.5: the rotated k stays in L2);
// 15000 tokens, 16/2 x 256 in fp32 97 (103); 30 tokens 3.7 (4.5), and one call less on the host.
#include <algorithm>

#include "paged_encode.cuh"
#include "rope_turn.cuh"

namespace fa {
namespace {

// Blocks of an SM: what hides q's latency is the number of threads, as in rope.cu (30000 tokens, 16/4 heads x 128,
// blocks of 16 tokens, in bf16: 122 us with 2 blocks, 90 with 3, 78 with 4, 70 with 6, 78 with 8; blocks of 8 tokens
// 71 with 5, 68 with 6; in fp32 105 with 5, 114 with 4).
template <typename T>
constexpr int kRopeBlocks = sizeof(T) == 4 ? 5 : 6;
constexpr int kItems = 1024;  // items (two vectors of q, or a lane's values of K and V) of a block

template <typename T, int HD, int V, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks<T>) rope_append_kernel(RopeAppendArgs b) {
    wait_for_stream();
    const RopeArgs &a = b.rope;
    const PagedAppendArgs &p = b.append;
    extern __shared__ float4 rope_smem[];
    constexpr int LANES = HD / 16;  // lanes of a row
    const int rd = a.rotary_dim, half = rd / 2;
    float *cs = reinterpret_cast<float *>(rope_smem);  // [tokens][half] cosines, then sines
    float *sn = cs + a.tokens_per_block * half;
    const int tok0 = blockIdx.x * a.tokens_per_block;
    const int n_tok = min(a.tokens_per_block, a.n_tokens - tok0);
    turn_table(a, half, tok0, n_tok, cs, sn);
    if (blockIdx.x + blockIdx.y == 0)
        for (int i = threadIdx.x; i < half; i += kRopeThreads)
            if (load(static_cast<const uint4 *>(a.table) + i).z >= static_cast<unsigned>(a.n_axes))
                flag_error(a.err, FA_ERRBIT_DEVICE);
    __syncthreads();
    // this block's heads: of the q heads, and then of the kv heads
    const int h0 = blockIdx.y * a.heads_per_block, h1 = min(h0 + a.heads_per_block, a.n_q_heads + p.n_kv);
    const int q_end = min(h1, a.n_q_heads);
    // ---- K and V
    const int kv0 = max(h0, a.n_q_heads) - a.n_q_heads, n_kv = h1 - a.n_q_heads - kv0;
    if (n_kv > 0) {
        const int rows = n_tok * n_kv, l = threadIdx.x & (LANES - 1);
        for (int r0 = 0; r0 < rows; r0 += kRopeThreads / LANES) {
            const int row = r0 + threadIdx.x / LANES;
            // tokens first: a warp's rows are neighbours in a page, whose words they share
            const int nth = row < rows ? row / n_tok : 0, tok = row < rows ? row - nth * n_tok : 0, h = kv0 + nth;
            const int slot = row < rows ? load(p.slot_map + tok0 + tok) : -1;
            const int page = slot >> p.page_shift;
            const bool live = slot >= 0 && page < p.n_pages;
            if (slot != -1 && !live && l == 0) flag_error(p.err, FA_ERRBIT_DEVICE);
            const long long t = tok0 + tok;
            float x[16] = {};
            const T *src = static_cast<const T *>(p.v) + t * p.v_stride + static_cast<long long>(h) * HD;
            if (live) {
                load8<T>(src + 16 * l, x);
                load8<T>(src + 16 * l + 8, x + 8);
            }
            encode_row<HD, true>(p, x, live, slot, page, h, l);
            src = static_cast<const T *>(p.k) + t * p.k_stride + static_cast<long long>(h) * HD;
            if (live) {
                load8<T>(src + 16 * l, x);
                load8<T>(src + 16 * l + 8, x + 8);
                const float *c = cs + tok * half, *s = sn + tok * half;
                if (ADJ) {
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const int pair = 8 * l + i / 2;
                        if (pair < half) {
                            float x0, x1;
                            turn(x[i], x[i + 1], c[pair], s[pair], &x0, &x1);
                            x[i] = Conv<T>::get(Conv<T>::put(x0));
                            x[i + 1] = Conv<T>::get(Conv<T>::put(x1));
                        }
                    }
                } else if (V > 1) {  // half is a multiple of 8: eight values on one side
#pragma unroll
                    for (int e = 0; e < 16; e += 8) {
                        const int d = 16 * l + e;
                        if (d >= rd) continue;
                        // One side of turn(): the low one fma(own, cos, -(other * sin)), the high one
                        // fma(other, sin, own * cos).
                        const bool low = d < half;
                        const int pair = low ? d : d - half;
                        const float *f = (low ? c : s) + pair, *g = (low ? s : c) + pair;
                        float o[8];
                        load8<T>(src + (low ? d + half : d - half), o);
#pragma unroll
                        for (int i = 0; i < 8; i += 4) {
                            const float4 fv = lds_f4(f + i), gv = lds_f4(g + i);
                            const float f4[4] = {fv.x, fv.y, fv.z, fv.w}, g4[4] = {gv.x, gv.y, gv.z, gv.w};
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                const float own = x[e + i + m], other = o[i + m];
                                const float r = fmaf(low ? own : other, f4[m], __fmul_rn(low ? -other : own, g4[m]));
                                x[e + i + m] = Conv<T>::get(Conv<T>::put(r));
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int d = 16 * l + i;
                        if (d >= rd) continue;
                        const bool low = d < half;
                        const float o = Conv<T>::get(src[low ? d + half : d - half]);
                        const int pair = low ? d : d - half;
                        float x0, x1;
                        turn(low ? x[i] : o, low ? o : x[i], c[pair], s[pair], &x0, &x1);
                        x[i] = Conv<T>::get(Conv<T>::put(low ? x0 : x1));
                    }
                }
            }
            encode_row<HD, false>(p, x, live, slot, page, h, l);
        }
    }
    // ---- q
    if (h0 < q_end) turn_heads<T, V, ADJ>(a, half, tok0, n_tok, h0, q_end - h0, cs, sn);
}

template <typename T, int HD, int V>
cudaError_t launch(RopeAppendArgs b, cudaStream_t stream) {
    RopeArgs &a = b.rope;
    const int rest = a.head_dim - a.rotary_dim, half = a.rotary_dim / 2;
    a.n_copy = a.n_q_heads == 0 || a.q == a.q_out ? 0 : (rest / V + 1) / 2;
    const int heads = a.n_q_heads + b.append.n_kv;
    const long long row = static_cast<long long>(a.n_q_heads) * (half / V + a.n_copy) +
                          static_cast<long long>(b.append.n_kv) * (HD / 16);  // items of a token
    const int fit = std::min<int>(kRopeTokens, 48 * 1024 / (half * 8));
    int tokens = static_cast<int>(std::min<long long>(fit, std::max<long long>(1, kItems / row)));
    // many tokens: blocks of 8, which share a page's words and a start, and are many enough to end together (30000
    // tokens, 16/4 heads x 128 in bf16: 76.6 us with 4, 67.7 with 8, 72.0 with 16; 20000, 16/2 x 256: 81, 77, 82)
    if (a.n_tokens >= 2 * kRopeTokens * device_sm_count()) tokens = std::min(fit, 8);
    // few tokens: a block takes one, and the heads are split over blocks too, as in rope.cu
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
        return launch_after(rope_append_kernel<T, HD, V, true>, grid, kRopeThreads, smem, stream, b);
    return launch_after(rope_append_kernel<T, HD, V, false>, grid, kRopeThreads, smem, stream, b);
}

// q moves 16 bytes at a time, and k's values eight at a time, where those lie on one side of their pairs.
template <typename T, int HD>
cudaError_t launch_hd(const RopeAppendArgs &b, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    return b.rope.rotary_dim / 2 % 8 == 0 ? launch<T, HD, V>(b, stream) : launch<T, HD, 1>(b, stream);
}

template <typename T>
cudaError_t launch_type(const RopeAppendArgs &b, cudaStream_t stream) {
    switch (b.rope.head_dim) {
        case 64: return launch_hd<T, 64>(b, stream);
        case 128: return launch_hd<T, 128>(b, stream);
        default: return launch_hd<T, 256>(b, stream);
    }
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendArgs &b, cudaStream_t stream) {
    switch (b.rope.dtype) {
        case kTypeF32: return launch_type<float>(b, stream);
        case kTypeF16: return launch_type<__half>(b, stream);
        default: return launch_type<__nv_bfloat16>(b, stream);
    }
}

}  // namespace fa
