// paged_api.cu -- the C ABI of paged serving (include/fa.h): argument checks
// and the arguments of the kernels in paged_plan.cu, rope.cu, rope_append.cu,
// paged_kv.cu and paged_attn.cuh. Host code only.
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/fa.h"
#include "fa_internal.h"
#include "paged_layout.cuh"

namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool aligned4(const void *p) { return aligned(p, 4); }

fa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

bool known_type(int t) { return t == FA_T_F32 || t == FA_T_F16 || t == FA_T_BF16; }
int type_bytes(int t) { return t == FA_T_F32 ? 4 : 2; }

// log2(page_rows), or -1
int page_shift(int page_rows) {
    for (int s = 4; s <= 8; ++s)
        if (page_rows == 1 << s) return s;
    return -1;
}

fa_status check_geometry(int n_kv_heads, int head_dim, int page_rows) {
    if (n_kv_heads < 1 || head_dim < 32 || head_dim % 32 || page_shift(page_rows) < 0)
        return FA_ERR_INVALID;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || n_kv_heads > 65535)
        return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

// A page and its number in 31 bits of slots; the table's rows in 30.
bool good_pages(int n_pages, int max_pages, int page_rows) {
    return n_pages >= 1 && max_pages >= 1 &&
           static_cast<long long>(n_pages) * page_rows < (1ll << 31) &&
           static_cast<long long>(max_pages) * page_rows <= (1ll << 30);
}

// Rows of `heads` heads `stride` elements apart: no overlap, within 64 bits.
bool good_stride(int64_t stride, int heads, int head_dim, int n_tokens) {
    const int64_t row = static_cast<int64_t>(heads) * head_dim;
    return stride >= row && stride <= (int64_t(1) << 58) / (n_tokens > 0 ? n_tokens : 1);
}

bool row_aligned(const void *p, int64_t stride, int type) {
    return aligned(p, 16) && stride * type_bytes(type) % 16 == 0;
}

fa::Pages make_pages(const void *pages, const int32_t *table, int n_pages, int n_kv,
                     int max_pages, int page_rows) {
    fa::Pages P;
    P.base = static_cast<const uint8_t *>(pages);
    P.table = table;
    P.n_pages = n_pages;
    P.n_kv = n_kv;
    P.max_pages = max_pages;
    P.groups = page_rows / fa::kGroupRows;
    P.group_shift = page_shift(page_rows) - 4;
    return P;
}

fa_status paged_attn(const void *q, void *out, float *lse, int dtype, int64_t q_stride,
                     int64_t out_stride, const int32_t *cu_q, const int32_t *seq_lens,
                     const int32_t *block_table, int max_pages, const void *pages, int n_pages,
                     int page_rows, int n_reqs, int n_tokens, int n_q_heads, int n_kv_heads,
                     int head_dim, int sink, int win, float scale, float cap, const float *slopes,
                     void *workspace, size_t workspace_bytes, fa_stream_t stream) {
    fa_status st = check_geometry(n_kv_heads, head_dim, page_rows);
    if (st != FA_OK) return st;
    if (n_q_heads < 1 || n_q_heads % n_kv_heads || !known_type(dtype) || n_reqs < 0 ||
        n_tokens < 0 || sink < 0 || !good_pages(n_pages, max_pages, page_rows) ||
        !(scale >= 0.0f) || !std::isfinite(scale) || !(cap >= 0.0f) || !std::isfinite(cap) ||
        (cap > 0.0f && !std::isfinite(4.0f / cap)) || !aligned4(slopes))
        return FA_ERR_INVALID;
    if (cap > fa::kMostCap) return FA_ERR_UNSUPPORTED;
    const int group = n_q_heads / n_kv_heads;
    if (group > 16 || (group & (group - 1)) || n_reqs > 65536 || n_tokens > 1 << 26 ||
        static_cast<long long>(n_tokens) * n_q_heads > 1 << 30)
        return FA_ERR_UNSUPPORTED;
    if (n_reqs == 0 || n_tokens == 0) return FA_OK;
    if (!q || !out || !cu_q || !seq_lens || !block_table || !pages || !workspace ||
        !aligned4(lse) || !aligned4(cu_q) || !aligned4(seq_lens) || !aligned4(block_table) ||
        !aligned(pages, 16) || !aligned(workspace, 16) ||
        !good_stride(q_stride, n_q_heads, head_dim, n_tokens) ||
        !good_stride(out_stride, n_q_heads, head_dim, n_tokens) ||
        !row_aligned(q, q_stride, dtype) || !row_aligned(out, out_stride, dtype))
        return FA_ERR_INVALID;
    if (workspace_bytes < fa::paged_attn_ws_bytes(head_dim)) return FA_ERR_WORKSPACE;
    if (q == out) return FA_ERR_INVALID;  // a row's q may be read after its neighbours' out is written
    fa::PagedAttnArgs a;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.cu_q = cu_q;
    a.seq_lens = seq_lens;
    a.pages = make_pages(pages, block_table, n_pages, n_kv_heads, max_pages, page_rows);
    a.n_reqs = n_reqs;
    a.n_tokens = n_tokens;
    a.n_q_heads = n_q_heads;
    a.sink = sink;
    a.win = win < 1 << 30 ? win : 1 << 30;  // the most rows a request can have
    a.scale = scale > 0.0f ? scale : 1.0f / sqrtf(static_cast<float>(head_dim));
    a.workspace = static_cast<uint8_t *>(workspace);
    a.err = fa::device_error_word();
    if (!a.err) return FA_ERR_CUDA;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cap == 0.0f && !slopes) return from_cuda(fa::launch_paged_attn(a, dtype, head_dim, s));
    a.cap = cap;
    if (cap > 0.0f) a.cap_in = dtype == FA_T_F32 ? 1.0f / (cap * 1.4426950408889634f) : 2.0f / cap;
    a.slopes = slopes;
    return from_cuda(fa::launch_paged_attn_scored(a, dtype, head_dim, s));
}

}  // namespace

extern "C" {

size_t fa_page_bytes(int n_kv_heads, int head_dim, int page_rows) {
    if (check_geometry(n_kv_heads, head_dim, page_rows) != FA_OK) return 0;
    return static_cast<size_t>(n_kv_heads) * (page_rows / fa::kGroupRows) *
           fa::group_bytes(head_dim);
}

fa_status fa_page_plan(const int32_t *cached, const int32_t *fresh, int n_reqs,
                       int32_t *free_ring, int n_pages, const int32_t *ring_state,
                       int32_t *ring_state_out, int32_t *block_table, int max_pages,
                       int page_rows, int32_t *seq_lens, int32_t *cu_fresh, int32_t *slot_map,
                       int32_t *positions, int max_tokens, fa_stream_t stream) {
    if (n_reqs < 0 || max_tokens < 0 || page_shift(page_rows) < 0 ||
        !good_pages(n_pages, max_pages, page_rows))
        return FA_ERR_INVALID;
    // a thread's next token is counted in 31 bits
    if (n_reqs > fa::kPlanMaxReqs || max_tokens > 1 << 30) return FA_ERR_UNSUPPORTED;
    if (!free_ring || !ring_state || !ring_state_out || !cu_fresh) return FA_ERR_INVALID;
    if (n_reqs > 0 && (!cached || !fresh || !block_table || !seq_lens)) return FA_ERR_INVALID;
    if (max_tokens > 0 && (!slot_map || !positions)) return FA_ERR_INVALID;
    if (!aligned4(cached) || !aligned4(fresh) || !aligned4(free_ring) || !aligned4(ring_state) ||
        !aligned4(ring_state_out) || !aligned4(block_table) || !aligned4(seq_lens) ||
        !aligned4(cu_fresh) || !aligned4(slot_map) || !aligned4(positions))
        return FA_ERR_INVALID;
    if (ring_state == ring_state_out || (n_reqs > 0 && (cached == seq_lens || fresh == seq_lens)))
        return FA_ERR_INVALID;
    fa::PlanArgs a;
    a.cached = cached;
    a.fresh = fresh;
    a.n_reqs = n_reqs;
    a.ring = free_ring;
    a.state = ring_state;
    a.n_pages = n_pages;
    a.state_out = ring_state_out;
    a.block_table = block_table;
    a.max_pages = max_pages;
    a.page_shift = page_shift(page_rows);
    a.seq_lens = seq_lens;
    a.cu_fresh = cu_fresh;
    a.slot_map = slot_map;
    a.positions = positions;
    a.max_tokens = max_tokens;
    a.err = fa::device_error_word();
    if (!a.err) return FA_ERR_CUDA;
    return from_cuda(fa::launch_page_plan(a, reinterpret_cast<cudaStream_t>(stream)));
}

fa_status fa_rope_table(uint32_t *table, const double *inv_freq, int pairs, const int *sections,
                        int n_axes, int interleaved) {
    if (!table || !inv_freq || !sections || pairs < 1 || n_axes < 1 || n_axes > 8)
        return FA_ERR_INVALID;
    long long sum = 0;
    for (int a = 0; a < n_axes; ++a) {
        if (sections[a] < 0) return FA_ERR_INVALID;
        sum += sections[a];
    }
    if (sum != pairs) return FA_ERR_INVALID;
    int count[8] = {0};
    int ordered = 0, end = sections[0];  // the axis whose run holds pair i, and where it ends
    for (int i = 0; i < pairs; ++i) {
        if (!std::isfinite(inv_freq[i]) || inv_freq[i] < 0.0) return FA_ERR_INVALID;
        while (i >= end) end += sections[++ordered];
        int axis = ordered;
        if (interleaved) {
            axis = i % n_axes;
            if (i >= static_cast<long long>(n_axes) * sections[axis]) axis = 0;
        }
        ++count[axis];
        const double turns = inv_freq[i] / 6.283185307179586476925;
        const uint64_t f = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64));
        table[4 * i] = static_cast<uint32_t>(f);
        table[4 * i + 1] = static_cast<uint32_t>(f >> 32);
        table[4 * i + 2] = static_cast<uint32_t>(axis);
        table[4 * i + 3] = 0;
    }
    for (int a = 0; a < n_axes; ++a)
        if (count[a] != sections[a]) return FA_ERR_INVALID;
    return FA_OK;
}

fa_status fa_rope(const void *q, void *q_out, const void *k, void *k_out, int dtype, int n_tokens,
                  int n_q_heads, int n_kv_heads, int head_dim, int rotary_dim, int64_t q_stride,
                  int64_t q_out_stride, int64_t k_stride, int64_t k_out_stride,
                  const int32_t *positions, int64_t pos_stride, int n_axes, const void *table,
                  int adjacent, int inverse, fa_stream_t stream) {
    if (!known_type(dtype) || n_tokens < 0 || n_q_heads < 0 || n_kv_heads < 0 ||
        head_dim < 2 || head_dim > 8192 || rotary_dim < 2 || rotary_dim % 2 ||
        rotary_dim > head_dim || n_axes < 1 || n_axes > 8 || n_q_heads > 65536 ||
        n_kv_heads > 65536)
        return FA_ERR_INVALID;
    if (n_tokens == 0 || n_q_heads + n_kv_heads == 0) return FA_OK;
    const size_t el = type_bytes(dtype);
    if (n_q_heads > 0) {
        if (!q || !q_out || !aligned(q, el) || !aligned(q_out, el) ||
            !good_stride(q_stride, n_q_heads, head_dim, n_tokens) ||
            !good_stride(q_out_stride, n_q_heads, head_dim, n_tokens) ||
            (q == q_out && q_stride != q_out_stride))
            return FA_ERR_INVALID;
    }
    if (n_kv_heads > 0) {
        if (!k || !k_out || !aligned(k, el) || !aligned(k_out, el) ||
            !good_stride(k_stride, n_kv_heads, head_dim, n_tokens) ||
            !good_stride(k_out_stride, n_kv_heads, head_dim, n_tokens) ||
            (k == k_out && k_stride != k_out_stride))
            return FA_ERR_INVALID;
    }
    if (!positions || !table || !aligned4(positions) || !aligned(table, 16) ||
        pos_stride < n_tokens || pos_stride > (int64_t(1) << 58))
        return FA_ERR_INVALID;
    fa::RopeArgs a;
    a.q = n_q_heads ? q : nullptr;
    a.k = n_kv_heads ? k : nullptr;
    a.q_out = n_q_heads ? q_out : nullptr;
    a.k_out = n_kv_heads ? k_out : nullptr;
    a.q_stride = n_q_heads ? q_stride : 0;
    a.q_out_stride = n_q_heads ? q_out_stride : 0;
    a.k_stride = n_kv_heads ? k_stride : 0;
    a.k_out_stride = n_kv_heads ? k_out_stride : 0;
    a.dtype = dtype;
    a.n_tokens = n_tokens;
    a.n_q_heads = n_q_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.rotary_dim = rotary_dim;
    a.positions = positions;
    a.pos_stride = pos_stride;
    a.n_axes = n_axes;
    a.table = table;
    a.adjacent = adjacent != 0;
    a.inverse = inverse != 0;
    a.err = fa::device_error_word();
    if (!a.err) return FA_ERR_CUDA;
    return from_cuda(fa::launch_rope(a, reinterpret_cast<cudaStream_t>(stream)));
}

fa_status fa_paged_append(const void *k_new, const void *v_new, int dtype, int64_t k_stride,
                          int64_t v_stride, const int32_t *slot_map, int n_tokens, void *pages,
                          int n_pages, int n_kv_heads, int head_dim, int page_rows,
                          fa_stream_t stream) {
    fa_status st = check_geometry(n_kv_heads, head_dim, page_rows);
    if (st != FA_OK) return st;
    if (!known_type(dtype) || n_tokens < 0 || !good_pages(n_pages, 1, page_rows))
        return FA_ERR_INVALID;
    if (n_tokens > 1 << 30) return FA_ERR_UNSUPPORTED;  // a block's last token in 31 bits
    if (n_tokens == 0) return FA_OK;
    if (!k_new || !v_new || !slot_map || !pages || !aligned4(slot_map) || !aligned(pages, 16) ||
        !good_stride(k_stride, n_kv_heads, head_dim, n_tokens) ||
        !good_stride(v_stride, n_kv_heads, head_dim, n_tokens) ||
        !row_aligned(k_new, k_stride, dtype) || !row_aligned(v_new, v_stride, dtype))
        return FA_ERR_INVALID;
    fa::PagedAppendArgs a;
    a.k = k_new;
    a.v = v_new;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.slot_map = slot_map;
    a.n_tokens = n_tokens;
    a.n_kv = n_kv_heads;
    a.pages = static_cast<uint8_t *>(pages);
    a.n_pages = n_pages;
    a.page_shift = page_shift(page_rows);
    a.err = fa::device_error_word();
    if (!a.err) return FA_ERR_CUDA;
    return from_cuda(
        fa::launch_paged_append(a, dtype, head_dim, reinterpret_cast<cudaStream_t>(stream)));
}

fa_status fa_paged_gather(const void *pages, int n_pages, const int32_t *block_table,
                          int max_pages, const int32_t *seq_lens, int n_reqs, int n_kv_heads,
                          int head_dim, int page_rows, void *k_planes, void *v_planes,
                          int max_seq, fa_stream_t stream) {
    fa_status st = check_geometry(n_kv_heads, head_dim, page_rows);
    if (st != FA_OK) return st;
    if (n_reqs < 0 || max_seq < 1 || !good_pages(n_pages, max_pages, page_rows))
        return FA_ERR_INVALID;
    if (n_reqs > 65535 || max_seq > 1 << 30) return FA_ERR_UNSUPPORTED;
    if (n_reqs == 0) return FA_OK;
    if (!pages || !block_table || !seq_lens || !k_planes || !v_planes || !aligned(pages, 16) ||
        !aligned4(block_table) || !aligned4(seq_lens) || !aligned(k_planes, 16) ||
        !aligned(v_planes, 16))
        return FA_ERR_INVALID;
    fa::PlaneGeom g;
    if (!fa::plane_geom(FA_KV_F16, n_kv_heads, max_seq, head_dim, &g)) return FA_ERR_INVALID;
    fa::PagedGatherArgs a;
    a.pages = make_pages(pages, block_table, n_pages, n_kv_heads, max_pages, page_rows);
    a.seq_lens = seq_lens;
    a.k_planes = static_cast<uint8_t *>(k_planes) + g.body_off;
    a.v_planes = static_cast<uint8_t *>(v_planes) + g.body_off;
    a.plane_bytes = g.bytes;
    a.max_seq = max_seq;
    a.err = fa::device_error_word();
    if (!a.err) return FA_ERR_CUDA;
    return from_cuda(
        fa::launch_paged_gather(a, n_reqs, head_dim, reinterpret_cast<cudaStream_t>(stream)));
}

size_t fa_paged_attn_workspace_bytes(int head_dim) {
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
    return fa::paged_attn_ws_bytes(head_dim);
}

fa_status fa_paged_attn(const void *q, void *out, float *lse, int dtype, int64_t q_stride,
                        int64_t out_stride, const int32_t *cu_q, const int32_t *seq_lens,
                        const int32_t *block_table, int max_pages, const void *pages, int n_pages,
                        int page_rows, int n_reqs, int n_tokens, int n_q_heads, int n_kv_heads,
                        int head_dim, int sink, int win, float scale, void *workspace,
                        size_t workspace_bytes, fa_stream_t stream) {
    return paged_attn(q, out, lse, dtype, q_stride, out_stride, cu_q, seq_lens, block_table, max_pages, pages,
                      n_pages, page_rows, n_reqs, n_tokens, n_q_heads, n_kv_heads, head_dim, sink, win, scale,
                      0.0f, nullptr, workspace, workspace_bytes, stream);
}

fa_status fa_paged_attn_scored(const void *q, void *out, float *lse, int dtype, int64_t q_stride,
                               int64_t out_stride, const int32_t *cu_q, const int32_t *seq_lens,
                               const int32_t *block_table, int max_pages, const void *pages, int n_pages,
                               int page_rows, int n_reqs, int n_tokens, int n_q_heads, int n_kv_heads,
                               int head_dim, int sink, int win, float scale, float cap, const float *slopes,
                               void *workspace, size_t workspace_bytes, fa_stream_t stream) {
    return paged_attn(q, out, lse, dtype, q_stride, out_stride, cu_q, seq_lens, block_table, max_pages, pages,
                      n_pages, page_rows, n_reqs, n_tokens, n_q_heads, n_kv_heads, head_dim, sink, win, scale,
                      cap, slopes, workspace, workspace_bytes, stream);
}

fa_status fa_rope_append(const void *q, void *q_out, const void *k_new, const void *v_new, int dtype, int n_tokens,
                         int n_q_heads, int n_kv_heads, int head_dim, int rotary_dim, int64_t q_stride,
                         int64_t q_out_stride, int64_t k_stride, int64_t v_stride, const int32_t *positions,
                         int64_t pos_stride, int n_axes, const void *table, int adjacent, const int32_t *slot_map,
                         void *pages, int n_pages, int page_rows, fa_stream_t stream) {
    fa_status st = check_geometry(n_kv_heads, head_dim, page_rows);
    if (st != FA_OK) return st;
    if (!known_type(dtype) || n_tokens < 0 || n_q_heads < 0 || n_q_heads > 65536 || rotary_dim < 2 ||
        rotary_dim % 2 || rotary_dim > head_dim || n_axes < 1 || n_axes > 8 || !good_pages(n_pages, 1, page_rows))
        return FA_ERR_INVALID;
    if (n_tokens > 1 << 30) return FA_ERR_UNSUPPORTED;  // a block's last token in 31 bits
    if (n_tokens == 0) return FA_OK;
    if (n_q_heads > 0 && (!q || !q_out || !good_stride(q_stride, n_q_heads, head_dim, n_tokens) ||
                          !good_stride(q_out_stride, n_q_heads, head_dim, n_tokens) ||
                          !row_aligned(q, q_stride, dtype) || !row_aligned(q_out, q_out_stride, dtype) ||
                          (q == q_out && q_stride != q_out_stride)))
        return FA_ERR_INVALID;
    if (!k_new || !v_new || !slot_map || !pages || !aligned4(slot_map) || !aligned(pages, 16) ||
        !good_stride(k_stride, n_kv_heads, head_dim, n_tokens) ||
        !good_stride(v_stride, n_kv_heads, head_dim, n_tokens) || !row_aligned(k_new, k_stride, dtype) ||
        !row_aligned(v_new, v_stride, dtype) || !positions || !table || !aligned4(positions) ||
        !aligned(table, 16) || pos_stride < n_tokens || pos_stride > (int64_t(1) << 58))
        return FA_ERR_INVALID;
    fa::RopeAppendArgs b;
    b.rope.q = n_q_heads ? q : nullptr;
    b.rope.q_out = n_q_heads ? q_out : nullptr;
    b.rope.k = b.rope.k_out = nullptr;
    b.rope.q_stride = n_q_heads ? q_stride : 0;
    b.rope.q_out_stride = n_q_heads ? q_out_stride : 0;
    b.rope.k_stride = b.rope.k_out_stride = 0;
    b.rope.dtype = dtype;
    b.rope.n_tokens = n_tokens;
    b.rope.n_q_heads = n_q_heads;
    b.rope.n_kv_heads = 0;
    b.rope.head_dim = head_dim;
    b.rope.rotary_dim = rotary_dim;
    b.rope.positions = positions;
    b.rope.pos_stride = pos_stride;
    b.rope.n_axes = n_axes;
    b.rope.table = table;
    b.rope.adjacent = adjacent != 0;
    b.rope.inverse = false;
    b.append.k = k_new;
    b.append.v = v_new;
    b.append.k_stride = k_stride;
    b.append.v_stride = v_stride;
    b.append.slot_map = slot_map;
    b.append.n_tokens = n_tokens;
    b.append.n_kv = n_kv_heads;
    b.append.pages = static_cast<uint8_t *>(pages);
    b.append.n_pages = n_pages;
    b.append.page_shift = page_shift(page_rows);
    b.rope.err = b.append.err = fa::device_error_word();
    if (!b.rope.err) return FA_ERR_CUDA;
    return from_cuda(fa::launch_rope_append(b, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
