// paged_attn.cu -- attention of ragged queries over 4-bit pages (include/fa.h,
// fa_paged_attn).
//
// Query t of a request with n queries and L rows sits at position p = L - n + t
// and attends keys j <= p (with win > 0 only sinks and the recent window):
//   s_j = scale * q . k_j,  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
//   lse = m + log sum_j exp(s_j - m).
//
// What bounds it: HBM for one query row per request (18 hd + 64 bytes per 16
// rows and kv head, read once), and just below that the issue slots, since each
// 4-bit code has to become a tensor-core operand. The layout of the pages and
// the arithmetic below are chosen to spend few instructions on a code:
//   - Codes are stored as mma.m16n8k16 A fragments (paged_layout.cuh): no
//     shuffles, no transposes; K with 16 rows as M, V with 16 dims as M.
//   - A code c in bits 0-3 or 4-7 of a half word IS a binary16 subnormal, c *
//     2^-24 or c * 2^-20, exact: one AND makes two operands. The factors 2^-24
//     and 2^-20 are undone in q (by 2^-4) and at the end; the offset -8 enters as
//     the accumulator's start (K), by a constant operand (V) or, for fp32 and
//     fp16, by one packed addition.
//   - The columns (N = 8) are 8 query rows of one kv head: the group's q heads,
//     times as many tokens as fit ("row group").
//   - V's block scales multiply the softmax weights (8 columns) instead of the
//     codes; each V row's power-of-two factor 2^e is added to its score's
//     exponent, so the scaled weights stay in binary16's range whatever the
//     values' magnitude. The sum of weights takes 2^-e back out.
//   - The reference that scores are taken relative to is moved only when a score
//     passes it by 2^14 (kLift above the last maximum, up to binary16's range):
//     one vote per 16 rows instead of a reduction.
// fp32 queries are split into two binary16 terms, and for fp32 and fp16 so are
// the scaled weights; their products go through a fresh accumulator per 16 rows
// that fp32 adds collect, as the tensor core's own sums lose a step per addition.
//
// Work split. The 16-row groups that are read, over all (request, kv head, row
// group) units, are cut into equal runs, one per warp of one block per SM; a
// warp streams its run through its own ring of bulk copies and starts the next
// unit's rows while it works on this one's. A unit inside one warp's run is
// written directly. Pieces of longer units are joined: those that end the runs
// of neighbouring warps of a block in shared memory, the others (at most two per
// warp) through the workspace by a second kernel, in a fixed order.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "fa_device.cuh"
#include "fa_internal.h"
#include "paged_layout.cuh"

namespace fa {
namespace {

constexpr float kLowest = -1e30f;  // reference of a row that has seen no key
constexpr float kLift = 6.0f;      // log2 of the largest weight right after a move
constexpr float kMost = 14.0f;     // log2 weight that moves the reference
constexpr int kMinGroups = 4;      // groups per warp below which fewer warps work
constexpr int kRows = 8;           // query rows of a row group

template <typename T, int HD>
struct Cfg {
    static constexpr bool QSPLIT = sizeof(T) == 4;
    static constexpr bool PSPLIT = !std::is_same<T, __nv_bfloat16>::value;
    static constexpr int NB = HD / 32;
    static constexpr int GB = group_bytes(HD);
    static constexpr int WARPS = PSPLIT ? 8 : 12;
    static constexpr int STAGES = HD == 256 ? (PSPLIT ? 5 : 4) : HD == 128 ? 7 : 12;
    static constexpr int RING = STAGES * GB;
    static constexpr int QLO = QSPLIT ? NB * 32 * 16 : 0;  // low terms of q, per warp
    static constexpr int OFF_BAR = WARPS * RING;
    static constexpr int OFF_BIAS = OFF_BAR + WARPS * STAGES * 8;
    static constexpr int OFF_QLO = OFF_BIAS + WARPS * NB * kRows * 4;
    static constexpr int SMEM = (OFF_QLO + WARPS * QLO + 127) / 128 * 128;
    static constexpr int THREADS = WARPS * 32;
    // a partial: m and l of 8 rows, then O as the lanes hold it
    static constexpr int PARTIAL = 2 * kRows + kRows * HD;  // floats
    static_assert(OFF_BAR % 8 == 0 && OFF_QLO % 16 == 0, "alignment");
    static_assert(RING >= kRows * HD * 4, "a warp's O fits its ring");
    static_assert(SMEM <= 225 * 1024, "shared memory");
};
constexpr int kMostWarps = 12;

// How a request's rows are read, from its lengths.
struct Req {
    int q0, nq, rows;      // first token, queries, rows
    int ns, skip, ng;      // sink groups, groups left out after them, groups read
    int rgs;               // row groups of each kv head (0: nothing to do)
    bool bad;
};

__device__ __forceinline__ Req load_req(const PagedAttnArgs &a, int r, int log_group) {
    Req q;
    q.q0 = __ldg(a.cu_q + r);
    const int q1 = __ldg(a.cu_q + r + 1);
    q.rows = __ldg(a.seq_lens + r);
    const long long room = static_cast<long long>(a.pages.max_pages) * a.pages.groups * kGroupRows;
    q.bad = q.q0 < 0 || q1 < q.q0 || q1 > a.n_tokens || q.rows < 0 || q.rows > room;
    q.nq = q.bad ? 0 : q1 - q.q0;
    q.rgs = static_cast<int>(((static_cast<long long>(q.nq) << log_group) + kRows - 1) / kRows);
    const int all = (q.rows + kGroupRows - 1) / kGroupRows;
    q.ns = q.skip = 0;
    q.ng = all;
    if (a.win > 0) {
        // the first key of any query's window; the sinks' groups before it
        const int lo = max(0, q.rows - q.nq - a.win + 1) / kGroupRows;  // the host bounds all three
        q.ns = min(lo, static_cast<int>((static_cast<long long>(a.sink) + kGroupRows - 1) /
                                        kGroupRows));
        q.skip = lo - q.ns;
        q.ng = max(0, all - q.skip);
    }
    return q;
}
// Groups a request counts for: at least one per unit, so that rows without any
// key are visited and written too.
__device__ __forceinline__ long long req_work(const Req &q, int n_kv) {
    return static_cast<long long>(max(q.ng, 1)) * q.rgs * n_kv;
}

// The cut of the work: N groups over W warps, A of them in each block.
struct Cut {
    long long N;
    int W, A;
    __device__ __forceinline__ long long start(int w) const { return N * w / W; }
};
__device__ __forceinline__ Cut make_cut(long long N, int blocks, int warps) {
    Cut c;
    c.N = N;
    const long long want = (N + kMinGroups - 1) / kMinGroups;
    c.W = static_cast<int>(min(static_cast<long long>(blocks) * warps, max(want, 1ll)));
    c.A = (c.W + blocks - 1) / blocks;
    c.W = min(c.W, c.A * blocks);
    return c;
}

// A unit that other blocks share, for the join: written by the warp whose run
// holds its first group.
struct Task {
    int valid, r, unit, w;  // w: that warp
    long long first, last;  // its groups [first, last)
    long long N;            // the cut
    int W, A;
};
struct Ws {
    Task *tasks;     // one per warp
    float *partial;  // two per warp: the end of its run, the start of its run
};
__host__ __device__ inline Ws carve(uint8_t *ws, int blocks) {
    Ws w;
    w.tasks = reinterpret_cast<Task *>(ws);
    w.partial = reinterpret_cast<float *>(
        ws + (static_cast<size_t>(blocks) * kMostWarps * sizeof(Task) + 255) / 256 * 256);
    return w;
}

template <typename T>
__device__ __forceinline__ void store4(T *p, float4 v);
template <>
__device__ __forceinline__ void store4<float>(float *p, float4 v) {
    *reinterpret_cast<float4 *>(p) = v;
}
template <>
__device__ __forceinline__ void store4<__half>(__half *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_half2(v.x, v.y), pack_half2(v.z, v.w));
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16 *p, float4 v) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<uint32_t *>(&lo),
                                               *reinterpret_cast<uint32_t *>(&hi));
}

// 8 consecutive values as fp32.
__device__ __forceinline__ void load8(const float *p, float *x) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    const float4 b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __half *p, float *x) {
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const __half2 *h = reinterpret_cast<const __half2 *>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float *x) {
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(h[i] << 16);
        x[2 * i + 1] = __uint_as_float(h[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ float2 half2_f(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
__device__ __forceinline__ void mma(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
    const uint32_t a[4] = {a0, a1, a2, a3}, b[2] = {b0, b1};
    mma_16816(d, a, b);
}

// 2^-24 and 2^-20 come out of O's rows g and g + 8.
constexpr float kUnshift0 = 16777216.0f, kUnshift1 = 1048576.0f;

// Row and head of a unit's column n; token < 0 past the unit's last row.
struct Col {
    int token, head, pos;
};
__device__ __forceinline__ Col column(const Req &q, int rg, int n, int h, int log_group) {
    const int row = rg * kRows + n, i = row >> log_group;
    Col c;
    c.token = i < q.nq ? q.q0 + i : -1;
    c.head = (h << log_group) + (row & ((1 << log_group) - 1));
    c.pos = i < q.nq ? q.rows - q.nq + i : -1;
    return c;
}

// The state of one piece: O, reference and weight sum of the lane's columns
// 2 t and 2 t + 1 (O: dims 32 b + 4 g + 0, 2 in rows g of tiles 0, 1 and
// 32 b + 4 g + 1, 3 in rows g + 8).
template <int NB>
struct State {
    float o[NB][2][4];
    float m[2], l[2];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 8; ++i) o[b][i >> 2][i & 3] = 0.0f;
        m[0] = m[1] = kLowest;
        l[0] = l[1] = 0.0f;
    }
    // four consecutive dims of column 2 t + c in block b
    __device__ __forceinline__ float4 quad(int b, int c) const {
        return make_float4(o[b][0][c] * kUnshift0, o[b][0][2 + c] * kUnshift1,
                           o[b][1][c] * kUnshift0, o[b][1][2 + c] * kUnshift1);
    }
    __device__ __forceinline__ void sum_lanes() {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
            l[0] += __shfl_xor_sync(~0u, l[0], d);
            l[1] += __shfl_xor_sync(~0u, l[1], d);
        }
    }
};

__device__ __forceinline__ float scaled(float x, float inv) { return x * inv; }
__device__ __forceinline__ float4 scaled(float4 v, float s) {
    return make_float4(v.x * s, v.y * s, v.z * s, v.w * s);
}

constexpr float kLn2 = 0.693147180559945309f, kLog2e = 1.442695040888963407f;

template <typename T, int HD>
__global__ void __launch_bounds__((Cfg<T, HD>::THREADS), 1) paged_attn_kernel(PagedAttnArgs a) {
    using C = Cfg<T, HD>;
    constexpr int NB = C::NB, S = C::STAGES;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long scan_part[C::WARPS];
    __shared__ int start_r[C::WARPS];
    __shared__ long long start_x[C::WARPS];
    __shared__ long long fin_first[C::WARPS], fin_last[C::WARPS];  // its last unit's groups
    __shared__ int fin_r[C::WARPS], fin_unit[C::WARPS];            // fin_unit -1: none
    __shared__ float fin_m[C::WARPS][kRows], fin_l[C::WARPS][kRows];
    __shared__ int abort_flag;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int n_kv = a.pages.n_kv;
    const int log_group = 31 - __clz(a.n_q_heads / n_kv);
    uint8_t *ring = smem + warp * C::RING;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR) + warp * S;
    float *bias = reinterpret_cast<float *>(smem + C::OFF_BIAS) + warp * NB * kRows;
    uint8_t *qlo = smem + C::OFF_QLO + warp * C::QLO;
    const Ws ws = carve(a.workspace, gridDim.x);

    if (lane == 0) {
        for (int i = 0; i < S; ++i) mbar_init(bars + i, 1);
        mbar_fence_init();
    }
    if (tid == 0) abort_flag = 0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the cut: sums over all requests, each thread a run of them
    const int per = (a.n_reqs + C::THREADS - 1) / C::THREADS;
    const int r0 = min(a.n_reqs, tid * per), r1 = min(a.n_reqs, r0 + per);
    long long mine = 0;
    bool bad = false;
    for (int r = r0; r < r1; ++r) {
        const Req q = load_req(a, r, log_group);
        bad |= q.bad;
        mine += req_work(q, n_kv);
    }
    if (bad && blockIdx.x == 0) flag_error(a.err, FA_ERRBIT_DEVICE);
    long long inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(~0u, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) scan_part[warp] = inc;
    __syncthreads();
    long long base = 0, N = 0;
    for (int i = 0; i < C::WARPS; ++i) {
        if (i == warp) base = N;
        N += scan_part[i];
    }
    const Cut cut = make_cut(N, gridDim.x, C::WARPS);
    {
        long long x = base + inc - mine;
        const int w0 = blockIdx.x * cut.A, w1 = min(w0 + cut.A, cut.W);
        if (w0 < w1 && x < cut.start(w1) && x + mine > cut.start(w0)) {
            for (int r = r0; r < r1; ++r) {
                const long long n = req_work(load_req(a, r, log_group), n_kv);
                for (int w = w0; w < w1; ++w) {
                    const long long s = cut.start(w);
                    if (x <= s && s < x + n) {
                        start_r[w - w0] = r;
                        start_x[w - w0] = x;
                    }
                }
                x += n;
            }
        }
    }
    __syncthreads();

    const int wid = blockIdx.x * cut.A + warp;
    const bool works = warp < cut.A && wid < cut.W && N > 0;
    State<NB> st;
    st.clear();
    int last_unit = -1, last_r = 0;  // the piece that ends the run, when other warps have more of its unit
    long long last_first = 0, last_last = 0;
    const int slot = blockIdx.x * C::WARPS + warp;
    if (lane == 0) ws.tasks[slot].valid = 0;

    if (works) {
        const long long x0 = cut.start(wid), x1 = cut.start(wid + 1);
        int todo = static_cast<int>(x1 - x0);  // groups to compute
        // ---- copies: their own walk over the run, S groups ahead
        int cr = start_r[warp];
        Req cq = load_req(a, cr, log_group);
        int cn = max(cq.ng, 1);
        long long off = x0 - start_x[warp];
        int cu = static_cast<int>(off / cn), ci = static_cast<int>(off - static_cast<long long>(cu) * cn);
        int ch = cu / cq.rgs;
        int left = todo;               // groups not yet looked up
        uint32_t dead = 0, parity = 0; // stages without a copy; barrier phases
        int page = 0, group = 0;       // of the next copy, looked up one step early
        bool has = false;
        auto look = [&]() {            // table entry of the walk's next group, then a step on
            has = left > 0;
            if (!has) return;
            --left;
            const bool any = ci < cq.ng;
            group = ci < cq.ns ? ci : ci + cq.skip;
            page = any ? __ldg(a.pages.table + static_cast<size_t>(cr) * a.pages.max_pages +
                               (group >> a.pages.group_shift)) : -2;
            group = (group & (a.pages.groups - 1)) + ch * a.pages.groups;
            if (++ci == cn && left > 0) {
                ci = 0;
                if (++cu == cq.rgs * n_kv) {
                    cu = 0;
                    do cq = load_req(a, ++cr, log_group); while (cq.rgs == 0);
                    cn = max(cq.ng, 1);
                }
                ch = cu / cq.rgs;
            }
        };
        auto issue = [&](int stage) {  // the looked-up group into a stage, and the next look-up
            if (!has) return;
            const bool live = page >= 0 && page < a.pages.n_pages;
            if (live) {
                dead &= ~(1u << stage);
                if (lane == 0) {
                    mbar_arrive_expect_tx(bars + stage, C::GB);
                    bulk_copy_g2s(ring + stage * C::GB,
                                  a.pages.base + (static_cast<size_t>(page) * n_kv *
                                                      a.pages.groups + group) * C::GB,
                                  C::GB, bars + stage);
                }
            } else {
                dead |= 1u << stage;
                if (page != -2 && lane == 0) flag_error(a.err, FA_ERRBIT_DEVICE);
            }
            look();
        };
        look();
#pragma unroll 1
        for (int i = 0; i < S; ++i) issue(i);

        // ---- the run, piece by piece
        int r = start_r[warp];
        Req q = load_req(a, r, log_group);
        int n = max(q.ng, 1);
        int unit = static_cast<int>((x0 - start_x[warp]) / n);
        int gi = static_cast<int>((x0 - start_x[warp]) - static_cast<long long>(unit) * n);
        int stage = 0;
        bool ok = true;
#pragma unroll 1
        while (todo > 0) {
            const int h = unit / q.rgs, rg = unit - h * q.rgs;
            const int g_first = gi;
            const int g_end = min(n, gi + todo);
            // ---- q of row g as B fragments: dims 32 b + 8 t + (0,4 | 1,5 | 2,6 | 3,7),
            // the second and fourth times 2^-4; brought to a maximum in [2^10, 2^11)
            uint32_t qf[NB][4];
            float km[2];
            {
                const Col c = column(q, rg, g, h, log_group);
                float x[NB][8], top = 0.0f;
                if (c.token >= 0) {
                    const T *src = static_cast<const T *>(a.q) + c.token * a.q_stride +
                                   static_cast<long long>(c.head) * HD + 8 * t;
#pragma unroll
                    for (int b = 0; b < NB; ++b) load8(src + 32 * b, x[b]);
                } else {
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[b][i] = 0.0f;
                }
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[b][i]));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                int up = 0;
                if (top > 0.0f)
                    up = min(max(137 - static_cast<int>(__float_as_uint(top) >> 23), -96), 126);
                const float lift = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
                const float mul = a.scale * kLog2e *
                                  __uint_as_float(static_cast<uint32_t>(127 - up) << 23) *
                                  16777216.0f;  // 2^24
                km[0] = __shfl_sync(~0u, mul, 8 * t);
                km[1] = __shfl_sync(~0u, mul, 8 * t + 4);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[b][i] *= lift;
                        sum += x[b][i];
                    }
                    sum += __shfl_xor_sync(~0u, sum, 1);
                    sum += __shfl_xor_sync(~0u, sum, 2);
                    if (t == 0) bias[b * kRows + g] = sum * -4.76837158203125e-7f;  // -8 * 2^-24
                    uint32_t lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t hi = pack_half2(x[b][i], x[b][i + 4]);
                        const float2 f = half2_f(hi);
                        const float sc = i & 1 ? 0.0625f : 1.0f;
                        qf[b][i] = i & 1 ? pack_half2(f.x * sc, f.y * sc) : hi;
                        if (C::QSPLIT)
                            lo[i] = pack_half2((x[b][i] - f.x) * sc, (x[b][i + 4] - f.y) * sc);
                    }
                    if (C::QSPLIT)
                        *reinterpret_cast<uint4 *>(qlo + (b * 32 + lane) * 16) =
                            make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            __syncwarp();
            const int p0 = column(q, rg, 2 * t, h, log_group).pos;
            const int p1 = column(q, rg, 2 * t + 1, h, log_group).pos;
            const int p_min = q.rows - q.nq + ((rg * kRows) >> log_group);
            const int p_max = q.rows - q.nq +
                              min(q.nq - 1, (rg * kRows + kRows - 1) >> log_group);
            st.clear();

#pragma unroll 1
            for (; gi < g_end; ++gi) {
                const bool live = !(dead >> stage & 1);
                if (live && ok) {
                    ok = mbar_wait(bars + stage, parity >> stage & 1, &abort_flag, a.err);
                    parity ^= 1u << stage;
                }
                if (live && ok) {
                    const uint8_t *kp = ring + stage * C::GB, *vp = kp + part_bytes(HD);
                    // ---- scores of rows g, g + 8 (y[0..1], y[2..3]) and columns 2 t, 2 t + 1
                    uint32_t kw[2 * NB];
#pragma unroll
                    for (int c = 0; c < NB / 2; ++c) {
                        const uint4 w = lds_v4(kp + (c * 32 + lane) * 16);
                        kw[4 * c] = w.x; kw[4 * c + 1] = w.y; kw[4 * c + 2] = w.z; kw[4 * c + 3] = w.w;
                    }
                    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    const uint32_t *ks = reinterpret_cast<const uint32_t *>(kp + scale_offset(HD));
#pragma unroll
                    for (int b2 = 0; b2 < NB / 2; ++b2) {
                        const float2 sA = half2_f(ks[g * (NB / 2) + b2]);
                        const float2 sB = half2_f(ks[(g + 8) * (NB / 2) + b2]);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int b = 2 * b2 + k;
                            const float2 c0 = *reinterpret_cast<const float2 *>(bias + b * kRows + 2 * t);
                            float d[4] = {c0.x, c0.y, c0.x, c0.y};
                            const uint32_t wA = kw[b], wB = kw[NB + b];
                            const uint32_t vA = wA >> 8, vB = wB >> 8;
                            const uint32_t e0 = wA & 0x000f000fu, e1 = wB & 0x000f000fu;
                            const uint32_t e2 = wA & 0x00f000f0u, e3 = wB & 0x00f000f0u;
                            const uint32_t f0 = vA & 0x000f000fu, f1 = vB & 0x000f000fu;
                            const uint32_t f2 = vA & 0x00f000f0u, f3 = vB & 0x00f000f0u;
                            mma(d, e0, e1, e2, e3, qf[b][0], qf[b][1]);
                            mma(d, f0, f1, f2, f3, qf[b][2], qf[b][3]);
                            if (C::QSPLIT) {
                                const uint4 lo = lds_v4(qlo + (b * 32 + lane) * 16);
                                mma(d, e0, e1, e2, e3, lo.x, lo.y);
                                mma(d, f0, f1, f2, f3, lo.z, lo.w);
                            }
                            const float a0 = k ? sA.y : sA.x, a1 = k ? sB.y : sB.x;
                            y[0] = fmaf(a0, d[0], y[0]);
                            y[1] = fmaf(a0, d[1], y[1]);
                            y[2] = fmaf(a1, d[2], y[2]);
                            y[3] = fmaf(a1, d[3], y[3]);
                        }
                    }
                    const uint16_t *kf = reinterpret_cast<const uint16_t *>(kp + factor_offset(HD));
                    const uint16_t *vf = reinterpret_cast<const uint16_t *>(vp + factor_offset(HD));
                    const float fA = __uint_as_float(static_cast<uint32_t>(kf[g]) << 16);
                    const float fB = __uint_as_float(static_cast<uint32_t>(kf[g + 8]) << 16);
                    const int xA = vf[g] >> 7, xB = vf[g + 8] >> 7;  // biased exponents of V's factors
                    const float eA = static_cast<float>(xA - 127), eB = static_cast<float>(xB - 127);
                    float iA = __uint_as_float(static_cast<uint32_t>(254 - xA) << 23);
                    float iB = __uint_as_float(static_cast<uint32_t>(254 - xB) << 23);
                    y[0] = fmaf(y[0] * fA, km[0], eA);
                    y[1] = fmaf(y[1] * fA, km[1], eA);
                    y[2] = fmaf(y[2] * fB, km[0], eB);
                    y[3] = fmaf(y[3] * fB, km[1], eB);
                    // V's block scales of rows 2t, 2t+1 | 2t+8, 2t+9
                    uint32_t vs[2 * NB];
#pragma unroll
                    for (int c = 0; c < NB / 2; ++c) {
                        const uint4 w = lds_v4(vp + scale_offset(HD) + (c * 4 + t) * 16);
                        vs[4 * c] = w.x; vs[4 * c + 1] = w.y; vs[4 * c + 2] = w.z; vs[4 * c + 3] = w.w;
                    }
                    const int j0 = (gi < q.ns ? gi : gi + q.skip) * kGroupRows;
                    const bool whole = j0 + kGroupRows - 1 <= p_min &&
                                       (a.win <= 0 || j0 + kGroupRows <= a.sink ||
                                        j0 > p_max - a.win);
                    if (!whole) {
                        // rows that no query sees may hold anything: their scales and
                        // sums must not reach a product, not even with a zero
                        auto seen = [&](int j) {
                            return j <= p_max && (a.win <= 0 || j < a.sink || j > p_min - a.win);
                        };
                        const int jA = j0 + g, jB = jA + 8;
                        if (!key_visible(p0, jA, a.sink, a.win)) y[0] = -INFINITY;
                        if (!key_visible(p1, jA, a.sink, a.win)) y[1] = -INFINITY;
                        if (!key_visible(p0, jB, a.sink, a.win)) y[2] = -INFINITY;
                        if (!key_visible(p1, jB, a.sink, a.win)) y[3] = -INFINITY;
                        if (!seen(jA)) iA = 0.0f;
                        if (!seen(jB)) iB = 0.0f;
                        const int k0 = j0 + 2 * t;
                        const uint32_t m01 = (seen(k0) ? 0xffffu : 0u) | (seen(k0 + 1) ? 0xffff0000u : 0u);
                        const uint32_t m23 = (seen(k0 + 8) ? 0xffffu : 0u) | (seen(k0 + 9) ? 0xffff0000u : 0u);
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            vs[2 * b] &= m01;
                            vs[2 * b + 1] &= m23;
                        }
                    }
                    // ---- weights relative to the reference
                    float d0 = y[0] - st.m[0], d1 = y[1] - st.m[1], d2 = y[2] - st.m[0],
                          d3 = y[3] - st.m[1];
                    if (__any_sync(~0u, fmaxf(fmaxf(d0, d1), fmaxf(d2, d3)) > kMost)) {
                        float u0 = fmaxf(y[0], y[2]), u1 = fmaxf(y[1], y[3]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            u0 = fmaxf(u0, __shfl_xor_sync(~0u, u0, d));
                            u1 = fmaxf(u1, __shfl_xor_sync(~0u, u1, d));
                        }
                        const float n0 = u0 - st.m[0] > kMost ? u0 - kLift : st.m[0];
                        const float n1 = u1 - st.m[1] > kMost ? u1 - kLift : st.m[1];
                        const float c0 = ex2(st.m[0] - n0), c1 = ex2(st.m[1] - n1);
                        st.m[0] = n0;
                        st.m[1] = n1;
                        st.l[0] *= c0;
                        st.l[1] *= c1;
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                st.o[b][i][0] *= c0;
                                st.o[b][i][1] *= c1;
                                st.o[b][i][2] *= c0;
                                st.o[b][i][3] *= c1;
                            }
                        d0 = y[0] - n0;
                        d1 = y[1] - n1;
                        d2 = y[2] - n0;
                        d3 = y[3] - n1;
                    }
                    d0 = ex2(d0);
                    d1 = ex2(d1);
                    d2 = ex2(d2);
                    d3 = ex2(d3);
                    st.l[0] += fmaf(d0, iA, d2 * iB);
                    st.l[1] += fmaf(d1, iA, d3 * iB);
                    const uint32_t hA = pack_half2(d0, d1), hB = pack_half2(d2, d3);
                    const uint32_t b0 = movmatrix_trans(hA), b1 = movmatrix_trans(hB);
                    uint32_t l0 = 0, l1 = 0;
                    if (C::PSPLIT) {
                        const float2 rA = half2_f(hA), rB = half2_f(hB);
                        l0 = movmatrix_trans(pack_half2(d0 - rA.x, d1 - rA.y));
                        l1 = movmatrix_trans(pack_half2(d2 - rB.x, d3 - rB.y));
                    }
                    // ---- O += V^T P
                    uint32_t vw[2 * NB];
#pragma unroll
                    for (int c = 0; c < NB / 2; ++c) {
                        const uint4 w = lds_v4(vp + (c * 32 + lane) * 16);
                        vw[4 * c] = w.x; vw[4 * c + 1] = w.y; vw[4 * c + 2] = w.z; vw[4 * c + 3] = w.w;
                    }
                    constexpr uint32_t kM8a = 0x80088008u, kM8b = 0x80808080u;  // -8 * 2^-24, -8 * 2^-20
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const uint32_t sel = b & 1 ? 0x7632u : 0x5410u;
                        const uint32_t x01 = __byte_perm(vw[b / 2], vw[(NB + b) / 2], sel);
                        const uint32_t x23 = __byte_perm(vw[(2 * NB + b) / 2], vw[(3 * NB + b) / 2], sel);
                        const uint32_t z01 = x01 >> 8, z23 = x23 >> 8;
                        const uint32_t s01 = vs[2 * b], s23 = vs[2 * b + 1];
                        const uint32_t w0 = hmul2(b0, s01), w1 = hmul2(b1, s23);
                        const uint32_t e0 = x01 & 0x000f000fu, e1 = x01 & 0x00f000f0u;
                        const uint32_t e2 = x23 & 0x000f000fu, e3 = x23 & 0x00f000f0u;
                        const uint32_t f0 = z01 & 0x000f000fu, f1 = z01 & 0x00f000f0u;
                        const uint32_t f2 = z23 & 0x000f000fu, f3 = z23 & 0x00f000f0u;
                        if (C::PSPLIT) {
                            const uint32_t v0 = hfma2(l0, s01, hfma2(b0, s01, w0 ^ 0x80008000u));
                            const uint32_t v1 = hfma2(l1, s23, hfma2(b1, s23, w1 ^ 0x80008000u));
                            // c - 8 exactly: the tensor core's sums lose a step towards zero per
                            // addition, which an offset taken out afterwards would leave behind
                            float u[4] = {0.0f, 0.0f, 0.0f, 0.0f}, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            const uint32_t g0 = hadd2(e0, kM8a), g1 = hadd2(e1, kM8b);
                            const uint32_t g2 = hadd2(e2, kM8a), g3 = hadd2(e3, kM8b);
                            mma(u, g0, g1, g2, g3, w0, w1);
                            mma(u, g0, g1, g2, g3, v0, v1);
                            const uint32_t h0 = hadd2(f0, kM8a), h1 = hadd2(f1, kM8b);
                            const uint32_t h2 = hadd2(f2, kM8a), h3 = hadd2(f3, kM8b);
                            mma(v, h0, h1, h2, h3, w0, w1);
                            mma(v, h0, h1, h2, h3, v0, v1);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                st.o[b][0][i] += u[i];
                                st.o[b][1][i] += v[i];
                            }
                        } else {
                            mma(st.o[b][0], e0, e1, e2, e3, w0, w1);
                            mma(st.o[b][1], f0, f1, f2, f3, w0, w1);
                            mma(st.o[b][0], kM8a, kM8b, kM8a, kM8b, w0, w1);
                            mma(st.o[b][1], kM8a, kM8b, kM8a, kM8b, w0, w1);
                        }
                    }
                }
                __syncwarp();  // every lane has read the stage
                if (ok) issue(stage);
                if (++stage == S) stage = 0;
            }
            todo -= g_end - g_first;

            // ---- the piece is done
            const bool begins = g_first == 0, ends = g_end == n;
            const long long first = x1 - todo - g_end;  // the unit's first group in the cut
            if (begins && ends) {
                st.sum_lanes();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const Col col = column(q, rg, 2 * t + c, h, log_group);
                    if (col.token < 0) continue;
                    const float inv = st.l[c] > 0.0f ? 1.0f / st.l[c] : st.l[c];
                    T *dst = static_cast<T *>(a.out) + col.token * a.out_stride +
                             static_cast<long long>(col.head) * HD + 4 * g;
#pragma unroll
                    for (int b = 0; b < NB; ++b) store4<T>(dst + 32 * b, scaled(st.quad(b, c), inv));
                    if (a.lse && g == 0)
                        a.lse[static_cast<size_t>(col.head) * a.n_tokens + col.token] =
                            (st.m[c] + log2f(st.l[c])) * kLn2;
                }
            } else if (todo > 0) {  // the start of the run: to the workspace
                st.sum_lanes();
                float *dst = ws.partial + (static_cast<size_t>(wid) * 2 + 1) * C::PARTIAL;
                if (g == 0) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        dst[2 * t + c] = st.m[c];
                        dst[kRows + 2 * t + c] = st.l[c];
                    }
                }
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        *reinterpret_cast<float4 *>(dst + 2 * kRows + ((b * 2 + c) * 32 + lane) * 4) =
                            st.quad(b, c);
            } else {
                last_unit = unit;
                last_r = r;
                last_first = first;
                last_last = first + n;
            }
            if (todo > 0) {
                gi = 0;
                if (++unit == q.rgs * n_kv) {
                    unit = 0;
                    do q = load_req(a, ++r, log_group); while (q.rgs == 0);
                    n = max(q.ng, 1);
                }
            }
        }
        if (!ok) {  // a wait ran out: let this warp's copies end before its memory is given up
            const long long t0 = clock64();
            for (int i = 0; i < S; ++i)
                while (!(dead >> i & 1) && !mbar_try_wait(bars + i, parity >> i & 1) &&
                       clock64() - t0 < kSpinCycles) {}
        }
    }

    // ---- join the pieces that end the warps' runs, unit by unit
    if (last_unit >= 0) st.sum_lanes();
    if (lane == 0) {
        fin_unit[warp] = last_unit;
        fin_r[warp] = last_r;
        fin_first[warp] = last_first;
        fin_last[warp] = last_last;
    }
    if (g == 0) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            fin_m[warp][2 * t + c] = st.m[c];
            fin_l[warp][2 * t + c] = st.l[c];
        }
    }
    if (last_unit >= 0) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                *reinterpret_cast<float4 *>(ring + ((b * 2 + c) * 32 + lane) * 16) = st.quad(b, c);
    }
    __syncthreads();
    if (last_unit < 0) return;
    auto same = [&](int w) { return fin_unit[w] == last_unit && fin_r[w] == last_r; };
    int w0 = warp, w1 = warp + 1;  // warps [w0, w1) hold pieces of this unit
    while (w0 > 0 && same(w0 - 1)) --w0;
    while (w1 < C::WARPS && same(w1)) ++w1;
    const int id0 = blockIdx.x * cut.A + w0, id1 = blockIdx.x * cut.A + w1;
    const bool from_start = cut.start(id0) <= last_first, to_end = cut.start(id1) >= last_last;
    float M[2] = {kLowest, kLowest}, L[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        for (int w = w0; w < w1; ++w) M[c] = fmaxf(M[c], fin_m[w][2 * t + c]);
        for (int w = w0; w < w1; ++w) L[c] += fin_l[w][2 * t + c] * ex2(fin_m[w][2 * t + c] - M[c]);
    }
    const Req q = load_req(a, last_r, log_group);
    const int h = last_unit / q.rgs, rg = last_unit - h * q.rgs;
    float *dst = ws.partial + static_cast<size_t>(id0) * 2 * C::PARTIAL;
    if (from_start && !to_end && warp == w0 && lane == 0) {
        Task k;
        k.valid = 1;
        k.r = last_r;
        k.unit = last_unit;
        k.w = id0;
        k.first = last_first;
        k.last = last_last;
        k.N = N;
        k.W = cut.W;
        k.A = cut.A;
        ws.tasks[slot] = k;
    }
    const bool direct = from_start && to_end;
    if (!direct && warp == w0 && g == 0) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            dst[2 * t + c] = M[c];
            dst[kRows + 2 * t + c] = L[c];
        }
    }
    for (int i = warp - w0; i < 2 * NB; i += w1 - w0) {  // (block, column) pairs
        const int b = i >> 1, c = i & 1;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int w = w0; w < w1; ++w) {
            const float4 y = *reinterpret_cast<const float4 *>(smem + w * C::RING + (i * 32 + lane) * 16);
            const float f = ex2(fin_m[w][2 * t + c] - M[c]);
            x.x = fmaf(y.x, f, x.x);
            x.y = fmaf(y.y, f, x.y);
            x.z = fmaf(y.z, f, x.z);
            x.w = fmaf(y.w, f, x.w);
        }
        if (direct) {
            const Col col = column(q, rg, 2 * t + c, h, log_group);
            if (col.token < 0) continue;
            const float inv = L[c] > 0.0f ? 1.0f / L[c] : L[c];
            store4<T>(static_cast<T *>(a.out) + col.token * a.out_stride +
                          static_cast<long long>(col.head) * HD + 32 * b + 4 * g, scaled(x, inv));
            if (a.lse && g == 0 && b == 0)
                a.lse[static_cast<size_t>(col.head) * a.n_tokens + col.token] =
                    (M[c] + log2f(L[c])) * kLn2;
        } else {
            *reinterpret_cast<float4 *>(dst + 2 * kRows + (i * 32 + lane) * 4) = x;
        }
    }
}

// One block per warp of the first kernel: the pieces of the unit that begins
// in its run, in ascending order.
constexpr int kJoinThreads = 128;
template <typename T, int HD>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(PagedAttnArgs a, int blocks) {
    using C = Cfg<T, HD>;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Ws ws = carve(a.workspace, blocks);
    const Task k = ws.tasks[blockIdx.x];
    if (!k.valid) return;
    const int w0 = k.w;
    Cut cut;
    cut.N = k.N;
    cut.W = k.W;
    cut.A = k.A;
    // pieces: the joined one of each block from w0's on, and the last warp's
    // first piece if its run goes on past the unit
    int w1 = w0;  // the warp that holds the unit's last group
    {
        int lo = w0, hi = k.W;  // the last w with start(w) < last
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cut.start(mid) < k.last) lo = mid; else hi = mid;
        }
        w1 = lo;
    }
    const bool tail = cut.start(w1 + 1) > k.last;
    const int b0 = w0 / k.A, b1 = (tail ? w1 - 1 : w1) / k.A;
    const int pieces = b1 - b0 + 1 + (tail ? 1 : 0);
    auto piece = [&](int i) {
        const size_t slot = i > b1 - b0 ? static_cast<size_t>(w1) * 2 + 1
                            : i == 0    ? static_cast<size_t>(w0) * 2
                                        : static_cast<size_t>(b0 + i) * k.A * 2;
        return ws.partial + slot * C::PARTIAL;
    };
    const int log_group = 31 - __clz(a.n_q_heads / a.pages.n_kv);
    const Req q = load_req(a, k.r, log_group);
    const int h = k.unit / q.rgs, rg = k.unit - h * q.rgs;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    for (int i = threadIdx.x >> 5; i < 2 * C::NB; i += kJoinThreads / 32) {
        const int b = i >> 1, n = 2 * t + (i & 1);
        float M = kLowest, L = 0.0f;
        for (int e = 0; e < pieces; ++e) M = fmaxf(M, piece(e)[n]);
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int e = 0; e < pieces; ++e) {
            const float *p = piece(e);
            const float f = ex2(p[n] - M);
            const float4 y = *reinterpret_cast<const float4 *>(p + 2 * kRows + (i * 32 + lane) * 4);
            L = fmaf(p[kRows + n], f, L);
            x.x = fmaf(y.x, f, x.x);
            x.y = fmaf(y.y, f, x.y);
            x.z = fmaf(y.z, f, x.z);
            x.w = fmaf(y.w, f, x.w);
        }
        const Col col = column(q, rg, n, h, log_group);
        if (col.token < 0) continue;
        const float inv = L > 0.0f ? 1.0f / L : L;
        store4<T>(static_cast<T *>(a.out) + col.token * a.out_stride +
                      static_cast<long long>(col.head) * HD + 32 * b + 4 * g, scaled(x, inv));
        if (a.lse && g == 0 && b == 0)
            a.lse[static_cast<size_t>(col.head) * a.n_tokens + col.token] = (M + log2f(L)) * kLn2;
    }
}

template <typename T, int HD>
cudaError_t launch(const PagedAttnArgs &a, cudaStream_t stream) {
    using C = Cfg<T, HD>;
    cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<T, HD>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const int blocks = device_sm_count();
    paged_attn_kernel<T, HD><<<blocks, C::THREADS, C::SMEM, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // programmatic dependent launch: the join's blocks are set up while the
    // first kernel drains, and wait for it at their start
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks * C::WARPS);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_join_kernel<T, HD>, a, blocks);
}

template <typename T>
cudaError_t launch_type(const PagedAttnArgs &a, int hd, cudaStream_t stream) {
    return hd == 64    ? launch<T, 64>(a, stream)
           : hd == 128 ? launch<T, 128>(a, stream)
                       : launch<T, 256>(a, stream);
}

}  // namespace

size_t paged_attn_ws_bytes(int hd) {
    const size_t warps = static_cast<size_t>(device_sm_count()) * kMostWarps;
    return (warps * sizeof(Task) + 255) / 256 * 256 + warps * 2 * (2 * kRows + kRows * hd) * 4;
}

cudaError_t launch_paged_attn(const PagedAttnArgs &a, int dtype, int hd, cudaStream_t stream) {
    switch (dtype) {
        case kTypeF32: return launch_type<float>(a, hd, stream);
        case kTypeF16: return launch_type<__half>(a, hd, stream);
        default: return launch_type<__nv_bfloat16>(a, hd, stream);
    }
}

}  // namespace fa
