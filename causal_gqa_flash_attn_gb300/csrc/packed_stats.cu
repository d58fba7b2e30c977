// packed_stats.cu -- what the gradient of packed attention needs of each row
// (include/fa.h, fa_packed_attn_grad): the log-sum-exp in the exp2 domain and
// D = dout . out, both negative as they are added, in the order of the rows, 128-row
// blocks a document. Rows of a block past the document's end get an L that makes
// every weight 0.
//
// One pass over out and dout, a row by HD / 8 lanes with 16-byte loads; bound by HBM, or where the batch is
// small by the time of one load. Four rows a thread are on their way at once, with their log-sum-exps, and
// four blocks an SM: 16384 tokens, 8 heads x 128: 13.5 us, 10 of them the bytes (21.5 with each row's log-sum-exp
// loaded behind its sums); 10007 tokens, 16 heads x 64 in fp16 13.8 (23.3).
#include "packed_common.cuh"

namespace fa {
namespace {

constexpr int kStatsThreads = 256;
constexpr float kNoRow = -1e30f;

template <int HD, bool BF16>
__global__ void __launch_bounds__(kStatsThreads, 4) packed_stats_kernel(PackedStatsArgs a) {
    wait_for_stream();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the next kernel sets itself up meanwhile
    constexpr int LANES = HD / 8, ROWS = kStatsThreads / LANES;  // lanes of a row, rows at once
    constexpr int AHEAD = 4;
    const int row0 = threadIdx.x / LANES, l = threadIdx.x % LANES, lane = threadIdx.x & 31;
    const int lg = a.log_group;
    const bool direct = a.direct.cu != nullptr;
    __shared__ unsigned most_of[2];
    PackedTile own;  // without a plan: the block's one tile
    int n_tiles = 0;
    if (direct)
        n_tiles = direct_tile<false>(a.direct, blockIdx.x / a.n_kv, 128 >> lg, 1, 7 - lg, a.sink, a.win, a.err, &own);
    const int units = a.n_kv * (direct ? n_tiles : a.header->row_tiles);
    auto dot = [](uint4 x, uint4 y) {
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 u = unpack2<BF16>(xs[k]), v = unpack2<BF16>(ys[k]);
            s = fmaf(u.x, v.x, s);
            s = fmaf(u.y, v.y, s);
        }
        return s;
    };
    auto sum = [](float x) {
#pragma unroll
        for (int d = 1; d < LANES; d <<= 1) x += __shfl_xor_sync(~0u, x, d);
        return x;
    };
    for (int w = blockIdx.x; w < units; w += gridDim.x) {
        const PackedTile u = direct ? own : a.rows[w / a.n_kv];
        const int g = w % a.n_kv;
        const size_t base = (static_cast<size_t>(g) * a.blocks + u.rb + (static_cast<long long>(u.p0) << lg >> 7)) * 128;
        float most = 0.0f, most_v = 0.0f;
        for (int r0 = 0; r0 < 128; r0 += ROWS * AHEAD) {
            uint4 o[AHEAD], d[AHEAD];
            float lse[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {  // all of these on their way at once
                const int r = r0 + k * ROWS + row0, tok = u.p0 + (r >> lg), head = (g << lg) + (r & ((1 << lg) - 1));
                const long long t = static_cast<long long>(u.tok0) + tok, at = static_cast<long long>(head) * HD + 8 * l;
                o[k] = d[k] = make_uint4(0, 0, 0, 0);
                lse[k] = 0.0f;
                if (tok < u.len) {
                    o[k] = load(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.out) + t * a.out_stride + at));
                    d[k] = load(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.dout) + t * a.dout_stride + at));
                    lse[k] = load(a.lse + static_cast<size_t>(head) * a.n_tokens + t);
                }
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const int r = r0 + k * ROWS + row0;
                const float D = sum(dot(o[k], d[k]));
                if (!BF16) {
                    const float n = sum(dot(d[k], d[k]));
                    most = n > most || n != n ? n : most;  // a NaN stays
                }
                if (l == 0) {
                    a.D[base + r] = -D;
                    a.L[base + r] = u.p0 + (r >> lg) < u.len ? fmaf(lse[k], -kPackedLog2e, BF16 ? 0.0f : kGradShift)
                                                             : kNoRow;
                }
            }
        }
        if (!BF16) {
            const int tokens = 128 >> lg;
            for (int r0 = 0; r0 < tokens; r0 += ROWS) {
                const int tok = u.p0 + r0 + row0;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r0 + row0 < tokens && tok < u.len)
                    v = load(reinterpret_cast<const uint4 *>(
                        static_cast<const uint16_t *>(a.v) + (static_cast<long long>(u.tok0) + tok) * a.v_stride +
                        static_cast<long long>(g) * HD + 8 * l));
                const float n = sum(dot(v, v));
                most_v = n > most_v || n != n ? n : most_v;
            }
            // largest bits: those of numbers that are not negative are in their order, a NaN above them
            const unsigned md = __reduce_max_sync(~0u, __float_as_uint(most) & 0x7fffffffu);
            const unsigned mv = __reduce_max_sync(~0u, __float_as_uint(most_v) & 0x7fffffffu);
            __syncthreads();  // the unit before has been read
            if (threadIdx.x < 2) most_of[threadIdx.x] = 0;
            __syncthreads();
            if (lane == 0) {
                atomicMax(most_of, md);
                atomicMax(most_of + 1, mv);
            }
            __syncthreads();
            if (threadIdx.x < 2) {
                if (direct)
                    a.doc_most[(static_cast<size_t>(threadIdx.x) * a.n_kv) * a.blocks + base / 128] = most_of[threadIdx.x];
                else
                    atomicMax(a.doc_most + threadIdx.x * a.n_docs + u.doc, most_of[threadIdx.x]);
            }
        }
    }
}

template <int HD>
cudaError_t launch_hd(const PackedStatsArgs &a, int dtype, int blocks, cudaStream_t stream) {
    return launch_after(dtype == kTypeBF16 ? packed_stats_kernel<HD, true> : packed_stats_kernel<HD, false>,
                        dim3(blocks), kStatsThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_packed_stats(const PackedStatsArgs &a, int dtype, int hd, int blocks, cudaStream_t stream) {
    switch (hd) {
        case 64: return launch_hd<64>(a, dtype, blocks, stream);
        case 128: return launch_hd<128>(a, dtype, blocks, stream);
        default: return launch_hd<256>(a, dtype, blocks, stream);
    }
}

}  // namespace fa
