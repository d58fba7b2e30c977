// packed_api.cu -- the C ABI of packed attention (include/fa.h): argument checks,
// the workspace's parts and the tensor maps. Host code only.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/fa.h"
#include "packed_common.cuh"

namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
fa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

int log2_of(int n) {
    int s = 0;
    while (1 << s < n) ++s;
    return s;
}

fa_status check_sizes(int n_docs, int n_tokens, int n_q_heads, int n_kv_heads, int head_dim) {
    if (n_docs < 0 || n_tokens < 0 || n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads ||
        head_dim < 32 || head_dim % 32)
        return FA_ERR_INVALID;
    const int group = n_q_heads / n_kv_heads;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || group > 16 || (group & (group - 1)) ||
        n_docs > 65536 || n_tokens > 1 << 26 || static_cast<long long>(n_tokens) * n_q_heads > 1 << 30)
        return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

// Where the parts of a workspace lie; `rows` is the rows of a row tile.
struct Layout {
    size_t row_tiles, key_tiles, doc_tiles, doc_most, stats, arrived, partial, bytes;
    int most_rows, most_keys, slots;
    size_t blocks;  // 128-row blocks of a kv head
};
constexpr size_t kPartialBytes = 48 << 20;  // of partial sums at most, so that they stay in L2
constexpr int kParts = 2;  // pieces of the work of dk and dv an SM, about; more of them cost joins

Layout layout(int n_docs, int n_tokens, int n_q_heads, int n_kv_heads, int head_dim, int rows, bool grad) {
    Layout w;
    const int group = n_q_heads / n_kv_heads;
    // Tiles of keys are cut where one has more than a few row tiles and there are not enough of them for
    // all SMs: into no more pieces than there are slots for.
    const long long tiles = static_cast<long long>(n_tokens / 128 + n_docs) * n_kv_heads;
    const long long row_tiles = static_cast<long long>(n_tokens) * group / fa::packed_grad_rows(head_dim) + 1;
    const size_t slot = sizeof(float) * 128 * head_dim * (head_dim < 256 ? 2 : 1);
    w.slots = 0;
    if (grad && row_tiles > 2 * fa::kPackedLeastPiece)
        w.slots = static_cast<int>(std::min<long long>(kPartialBytes / slot, tiles * (row_tiles / fa::kPackedLeastPiece + 1)));
    w.most_rows = static_cast<int>(static_cast<long long>(n_tokens) * group / rows) + n_docs;
    w.most_keys = grad ? n_tokens / 128 + n_docs + w.slots : 0;
    w.blocks = static_cast<size_t>(n_tokens) * group / 128 + n_docs;
    size_t at = sizeof(fa::PackedHeader);
    auto take = [&](size_t n) {
        const size_t from = at;
        at += up256(n);
        return from;
    };
    w.row_tiles = take(sizeof(fa::PackedTile) * w.most_rows);
    w.key_tiles = take(sizeof(fa::PackedTile) * w.most_keys);
    w.doc_tiles = take(sizeof(int) * 3 * (grad ? 2 : 1) * (static_cast<size_t>(n_docs) + 1));
    w.doc_most = take(grad ? sizeof(unsigned) * 2 * std::max<size_t>(n_docs, n_kv_heads * w.blocks) : 0);
    w.stats = take(grad ? sizeof(float) * 2 * n_kv_heads * w.blocks * 128 : 0);
    w.arrived = take(sizeof(int) * w.slots);
    w.partial = take(slot * w.slots);
    w.bytes = at;
    return w;
}

bool good_heads(const void *p, int64_t stride, int heads, int head_dim, int n_tokens) {
    const int64_t row = static_cast<int64_t>(heads) * head_dim;
    return p && aligned(p, 16) && stride % 8 == 0 && stride >= row &&
           stride <= (int64_t(1) << 38) / (n_tokens > 0 ? n_tokens : 1);  // a tensor map's strides: below 2^40 bytes
}

// What both directions check beside their tensors.
fa_status check_rule(int dtype, const int32_t *cu, const int32_t *prefix, int sink, float scale, float cap,
                     const float *slopes, const void *workspace) {
    if (sink < 0 || !(scale >= 0.0f) || !std::isfinite(scale) || !(cap >= 0.0f) || !std::isfinite(cap))
        return FA_ERR_INVALID;
    // The factor of a score (score_rule): an infinite one would make scores of 0 a NaN, and one below the normal range,
    // which counts as 0, the -inf of masked ones.
    if ((scale > 0.0f && !std::isnormal(scale)) || !std::isfinite(4.0f * scale) ||
        (cap > 0.0f && !std::isfinite(4.0f * std::fmax(scale, 1.0f) / cap)))
        return FA_ERR_INVALID;
    if (dtype == FA_T_F32 || cap > fa::kMostCap) return FA_ERR_UNSUPPORTED;
    if (dtype != FA_T_F16 && dtype != FA_T_BF16) return FA_ERR_INVALID;
    if (!aligned(cu, 4) || !aligned(prefix, 4) || !aligned(slopes, 4) || !aligned(workspace, 16))
        return FA_ERR_INVALID;
    return FA_OK;
}

// q-like rows: tiles of `rows` rows, 64 dims wide, tokens of all heads of a group.
bool map_rows(CUtensorMap *m, int dtype, const void *p, int64_t stride, int n_tokens, int n_kv, int group,
              int hd, int rows) {
    const uint64_t dims[4] = {static_cast<uint64_t>(hd), static_cast<uint64_t>(group), static_cast<uint64_t>(n_kv),
                              static_cast<uint64_t>(n_tokens)};
    const uint64_t strides[3] = {2ull * hd, 2ull * hd * group, 2ull * stride};
    const uint32_t box[4] = {64, static_cast<uint32_t>(group), 1, static_cast<uint32_t>(rows / group)};
    return fa::encode_tiled(m, dtype == FA_T_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                            4, p, dims, strides, box);
}
// k-like rows: tiles of `rows` tokens of one kv head.
bool map_keys(CUtensorMap *m, int dtype, const void *p, int64_t stride, int n_tokens, int n_kv, int hd, int rows) {
    const uint64_t dims[3] = {static_cast<uint64_t>(hd), static_cast<uint64_t>(n_kv), static_cast<uint64_t>(n_tokens)};
    const uint64_t strides[2] = {2ull * hd, 2ull * stride};
    const uint32_t box[3] = {64, 1, static_cast<uint32_t>(rows)};
    return fa::encode_tiled(m, dtype == FA_T_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                            3, p, dims, strides, box);
}

int bounded(int n) { return std::min(std::max(n, 0), 1 << 30); }

}  // namespace

extern "C" {

size_t fa_packed_attn_workspace_bytes(int n_docs, int n_tokens, int n_q_heads, int n_kv_heads, int head_dim) {
    if (check_sizes(n_docs, n_tokens, n_q_heads, n_kv_heads, head_dim) != FA_OK) return 0;
    return layout(n_docs, n_tokens, n_q_heads, n_kv_heads, head_dim, 128 * fa::packed_fwd_tiles(head_dim), false).bytes;
}

fa_status fa_packed_attn(const void *q, const void *k, const void *v, void *out, float *lse, int dtype,
                         int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t out_stride,
                         const int32_t *cu_docs, const int32_t *prefix, int n_docs, int n_tokens, int n_q_heads,
                         int n_kv_heads, int head_dim, int sink, int win, float scale, float cap,
                         const float *slopes, void *workspace, size_t workspace_bytes, fa_stream_t stream) {
    fa_status st = check_sizes(n_docs, n_tokens, n_q_heads, n_kv_heads, head_dim);
    if (st != FA_OK) return st;
    st = check_rule(dtype, cu_docs, prefix, sink, scale, cap, slopes, workspace);
    if (st != FA_OK) return st;
    if (n_docs == 0 || n_tokens == 0) return FA_OK;
    if (!cu_docs || !workspace || !aligned(lse, 4) || !good_heads(q, q_stride, n_q_heads, head_dim, n_tokens) ||
        !good_heads(k, k_stride, n_kv_heads, head_dim, n_tokens) ||
        !good_heads(v, v_stride, n_kv_heads, head_dim, n_tokens) ||
        !good_heads(out, out_stride, n_q_heads, head_dim, n_tokens))
        return FA_ERR_INVALID;
    if (out == q || out == k || out == v) return FA_ERR_INVALID;
    const int group = n_q_heads / n_kv_heads, rows = 128 * fa::packed_fwd_tiles(head_dim);
    const Layout w = layout(n_docs, n_tokens, n_q_heads, n_kv_heads, head_dim, rows, false);
    if (workspace_bytes < w.bytes) return FA_ERR_WORKSPACE;
    unsigned *err = fa::device_error_word();
    if (!err) return FA_ERR_CUDA;
    uint8_t *ws = static_cast<uint8_t *>(workspace);

    fa::PackedPlanArgs p;
    p.cu = cu_docs;
    p.prefix = prefix;
    p.n_docs = n_docs;
    p.n_tokens = n_tokens;
    p.sink = bounded(sink);
    p.win = bounded(win);
    p.row_tokens = rows / group;
    p.block_tokens_log = 7 - log2_of(group);
    p.key_tile = 128;
    p.step_tokens = 1;
    p.n_kv = n_kv_heads;
    p.parts = 1;
    p.most_rows = w.most_rows;
    p.most_keys = 0;
    p.slots = 0;
    p.arrived = nullptr;
    p.header = reinterpret_cast<fa::PackedHeader *>(ws);
    p.rows = reinterpret_cast<fa::PackedTile *>(ws + w.row_tiles);
    p.keys = nullptr;
    p.doc_tiles = reinterpret_cast<int *>(ws + w.doc_tiles);
    p.doc_most = nullptr;
    p.err = err;

    fa::PackedFwdArgs a;
    if (!map_rows(&a.q, dtype, q, q_stride, n_tokens, n_kv_heads, group, head_dim, 128) ||
        !map_keys(&a.k, dtype, k, k_stride, n_tokens, n_kv_heads, head_dim, 128) ||
        !map_keys(&a.v, dtype, v, v_stride, n_tokens, n_kv_heads, head_dim, 128) ||
        !map_rows(&a.o, dtype, out, out_stride, n_tokens, n_kv_heads, group, head_dim, 32))
        return FA_ERR_CUDA;
    a.header = p.header;
    a.rows = p.rows;
    a.counter = &p.header->counters[0];
    a.out = out;
    a.out_stride = out_stride;
    a.lse = lse;
    a.slopes = slopes;
    a.n_tokens = n_tokens;
    a.n_kv = n_kv_heads;
    a.log_group = log2_of(group);
    a.sink = p.sink;
    a.win = p.win;
    a.score = fa::score_rule(scale > 0.0f ? scale : 1.0f / sqrtf(static_cast<float>(head_dim)), cap);
    a.err = err;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const long long units = static_cast<long long>(w.most_rows) * n_kv_heads;
    const int blocks = static_cast<int>(std::min<long long>(fa::device_sm_count(), units));
    a.direct = fa::PackedDirect{};
    if (n_docs <= fa::kDirectDocs && units <= fa::device_sm_count()) {
        a.direct = fa::PackedDirect{cu_docs, prefix, n_docs, n_tokens};
    } else {
        const cudaError_t e = fa::launch_packed_plan(p, s);
        if (e != cudaSuccess) return from_cuda(e);
    }
    return from_cuda(dtype == FA_T_BF16 ? fa::launch_packed_fwd_bf16(a, head_dim, cap > 0.0f, blocks, s)
                                        : fa::launch_packed_fwd_f16(a, head_dim, cap > 0.0f, blocks, s));
}

size_t fa_packed_attn_grad_workspace_bytes(int n_docs, int n_tokens, int n_q_heads, int n_kv_heads,
                                           int head_dim) {
    if (check_sizes(n_docs, n_tokens, n_q_heads, n_kv_heads, head_dim) != FA_OK) return 0;
    return layout(n_docs, n_tokens, n_q_heads, n_kv_heads, head_dim, 128, true).bytes;
}

fa_status fa_packed_attn_grad(const void *q, const void *k, const void *v, const void *out, const float *lse,
                              const void *dout, void *dq, void *dk, void *dv, int dtype, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, int64_t out_stride, int64_t dout_stride,
                              int64_t dq_stride, int64_t dk_stride, int64_t dv_stride, const int32_t *cu_docs,
                              const int32_t *prefix, int n_docs, int n_tokens, int n_q_heads, int n_kv_heads,
                              int head_dim, int sink, int win, float scale, float cap, const float *slopes,
                              void *workspace, size_t workspace_bytes, fa_stream_t stream) {
    fa_status st = check_sizes(n_docs, n_tokens, n_q_heads, n_kv_heads, head_dim);
    if (st != FA_OK) return st;
    st = check_rule(dtype, cu_docs, prefix, sink, scale, cap, slopes, workspace);
    if (st != FA_OK) return st;
    if (n_docs == 0 || n_tokens == 0) return FA_OK;
    if (!cu_docs || !workspace || !lse || !aligned(lse, 4) ||
        !good_heads(q, q_stride, n_q_heads, head_dim, n_tokens) ||
        !good_heads(k, k_stride, n_kv_heads, head_dim, n_tokens) ||
        !good_heads(v, v_stride, n_kv_heads, head_dim, n_tokens) ||
        !good_heads(out, out_stride, n_q_heads, head_dim, n_tokens) ||
        !good_heads(dout, dout_stride, n_q_heads, head_dim, n_tokens) ||
        !good_heads(dq, dq_stride, n_q_heads, head_dim, n_tokens) ||
        !good_heads(dk, dk_stride, n_kv_heads, head_dim, n_tokens) ||
        !good_heads(dv, dv_stride, n_kv_heads, head_dim, n_tokens))
        return FA_ERR_INVALID;
    const void *in[5] = {q, k, v, out, dout};
    const void *made[3] = {dq, dk, dv};
    for (int i = 0; i < 3; ++i) {
        for (int k2 = 0; k2 < 5; ++k2)
            if (made[i] == in[k2]) return FA_ERR_INVALID;
        if (made[i] == made[(i + 1) % 3]) return FA_ERR_INVALID;
    }
    const int group = n_q_heads / n_kv_heads, step = fa::packed_grad_rows(head_dim);
    const Layout w = layout(n_docs, n_tokens, n_q_heads, n_kv_heads, head_dim, 128, true);
    if (workspace_bytes < w.bytes) return FA_ERR_WORKSPACE;
    unsigned *err = fa::device_error_word();
    if (!err) return FA_ERR_CUDA;
    uint8_t *ws = static_cast<uint8_t *>(workspace);

    fa::PackedPlanArgs p;
    p.cu = cu_docs;
    p.prefix = prefix;
    p.n_docs = n_docs;
    p.n_tokens = n_tokens;
    p.sink = bounded(sink);
    p.win = bounded(win);
    p.row_tokens = 128 / group;
    p.block_tokens_log = 7 - log2_of(group);
    p.key_tile = step;
    p.step_tokens = step / group;
    p.n_kv = n_kv_heads;
    p.parts = kParts * fa::device_sm_count();
    p.most_rows = w.most_rows;
    p.most_keys = w.most_keys;
    p.slots = w.slots;
    p.arrived = reinterpret_cast<int *>(ws + w.arrived);
    p.header = reinterpret_cast<fa::PackedHeader *>(ws);
    p.rows = reinterpret_cast<fa::PackedTile *>(ws + w.row_tiles);
    p.keys = reinterpret_cast<fa::PackedTile *>(ws + w.key_tiles);
    p.doc_tiles = reinterpret_cast<int *>(ws + w.doc_tiles);
    p.doc_most = reinterpret_cast<unsigned *>(ws + w.doc_most);
    p.err = err;

    fa::PackedStatsArgs t;
    t.header = p.header;
    t.rows = p.rows;
    t.out = out;
    t.dout = dout;
    t.v = v;
    t.out_stride = out_stride;
    t.dout_stride = dout_stride;
    t.v_stride = v_stride;
    t.lse = lse;
    t.n_tokens = n_tokens;
    t.n_kv = n_kv_heads;
    t.log_group = log2_of(group);
    t.n_docs = n_docs;
    t.blocks = static_cast<long long>(w.blocks);
    t.L = reinterpret_cast<float *>(ws + w.stats);
    t.D = t.L + static_cast<size_t>(n_kv_heads) * w.blocks * 128;
    t.doc_most = p.doc_most;
    t.sink = p.sink;
    t.win = p.win;
    t.err = err;
    // no plan where every unit has a block of its own and no tile of keys has rows enough to be cut
    const int sms = fa::device_sm_count();
    const bool direct = n_docs <= fa::kDirectDocs && w.slots == 0 &&
                        static_cast<long long>(w.most_rows) * n_kv_heads <= sms &&
                        static_cast<long long>(w.most_keys) * n_kv_heads <= sms;
    t.direct = direct ? fa::PackedDirect{cu_docs, prefix, n_docs, n_tokens} : fa::PackedDirect{};

    fa::PackedGradPair pair;
    fa::PackedGradArgs &a = pair.q, &b = pair.k;  // of dq, and of dk and dv
    a.header = p.header;
    a.L = t.L;
    a.D = t.D;
    a.blocks = t.blocks;
    a.direct = t.direct;
    a.partial = reinterpret_cast<float *>(ws + w.partial);
    a.arrived = p.arrived;
    a.doc_most = p.doc_most;
    a.slopes = slopes;
    a.n_docs = n_docs;
    a.n_kv = n_kv_heads;
    a.log_group = t.log_group;
    a.sink = p.sink;
    a.win = p.win;
    a.scale = scale > 0.0f ? scale : 1.0f / sqrtf(static_cast<float>(head_dim));
    a.score = fa::score_rule(a.scale, cap);
    a.err = err;
    b = a;
    a.tiles = p.rows;
    a.n_tiles = &p.header->row_tiles;
    a.counter = &p.header->counters[0];
    a.g1 = dq;
    a.g1_stride = dq_stride;
    a.g2 = nullptr;
    a.g2_stride = 0;
    b.tiles = p.keys;
    b.n_tiles = &p.header->key_tiles;
    b.counter = &p.header->counters[1];
    b.g1 = dk;
    b.g1_stride = dk_stride;
    b.g2 = dv;
    b.g2_stride = dv_stride;
    if (!map_rows(&a.x1, dtype, q, q_stride, n_tokens, n_kv_heads, group, head_dim, 128) ||
        !map_rows(&a.x2, dtype, dout, dout_stride, n_tokens, n_kv_heads, group, head_dim, 128) ||
        !map_keys(&a.y1, dtype, k, k_stride, n_tokens, n_kv_heads, head_dim, step) ||
        !map_keys(&a.y2, dtype, v, v_stride, n_tokens, n_kv_heads, head_dim, step) ||
        !map_keys(&b.x1, dtype, k, k_stride, n_tokens, n_kv_heads, head_dim, 128) ||
        !map_keys(&b.x2, dtype, v, v_stride, n_tokens, n_kv_heads, head_dim, 128) ||
        !map_rows(&b.y1, dtype, q, q_stride, n_tokens, n_kv_heads, group, head_dim, step) ||
        !map_rows(&b.y2, dtype, dout, dout_stride, n_tokens, n_kv_heads, group, head_dim, step))
        return FA_ERR_CUDA;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto blocks_of = [&](int tiles, int most) {
        return static_cast<int>(std::min<long long>(most, static_cast<long long>(tiles) * n_kv_heads));
    };
    pair.q_blocks = blocks_of(w.most_rows, sms);
    pair.k_blocks = blocks_of(w.most_keys, sms);
    fa::PackedGradArgs dv_alone = b;  // head_dim 256
    dv_alone.counter = &p.header->counters[2];
    cudaError_t e = direct ? cudaSuccess : fa::launch_packed_plan(p, s);
    if (e == cudaSuccess)
        e = fa::launch_packed_stats(t, dtype, head_dim, blocks_of(w.most_rows, direct ? sms : 64 * sms), s);
    if (e == cudaSuccess)
        e = dtype == FA_T_BF16 ? fa::launch_packed_grad_bf16(pair, &dv_alone, head_dim, cap > 0.0f, s)
                               : fa::launch_packed_grad_f16(pair, &dv_alone, head_dim, cap > 0.0f, s);
    return from_cuda(e);
}

}  // extern "C"
