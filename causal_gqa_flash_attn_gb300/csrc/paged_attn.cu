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
constexpr int kMostWarps = 16;     // computing warps of a block that the workspace is made for

template <typename T, int HD>
struct Cfg {
    static constexpr bool QSPLIT = sizeof(T) == 4;
    static constexpr bool PSPLIT = !std::is_same<T, __nv_bfloat16>::value;
    static constexpr int NB = HD / 32;
    static constexpr int GB = group_bytes(HD);
    // Warps that compute, and one more that copies; registers for one block of
    // them per SM, ring stages for what is left of shared memory.
#ifdef PA_WARPS
    static constexpr bool PP = sizeof(T) == PA_SIZE && HD == PA_HD;
    static constexpr int WARPS = PP ? PA_WARPS : 7;
    static constexpr int STAGES = PP ? PA_STAGES : 4;
#else
    static constexpr int WARPS = HD == 256 ? (PSPLIT ? 7 : 11) : PSPLIT ? 11 : 15;
    static constexpr int STAGES = HD == 256 ? (PSPLIT ? 4 : 3) : HD == 128 ? 4 : 8;
#endif
    static constexpr int RING = STAGES * GB;
    static constexpr int QF = NB * 32 * 16;           // q as B fragments
    static constexpr int QB = QF * (QSPLIT ? 2 : 1);  // and their low terms
    static constexpr int BIAS = NB * 4 * 16;          // the accumulators' start, as lanes hold it
    static constexpr int OFF_Q = WARPS * RING;
    static constexpr int OFF_BIAS = OFF_Q + WARPS * QB;
    static constexpr int OFF_BAR = OFF_BIAS + WARPS * BIAS;
    static constexpr int OFF_DEAD = OFF_BAR + WARPS * STAGES * 16;  // full and empty barriers
    static constexpr int SMEM = OFF_DEAD + WARPS * STAGES * 4;
    static constexpr int THREADS = (WARPS + 1) * 32;
    // a partial: m and l of 8 rows, then O as the lanes hold it
    static constexpr int PARTIAL = 2 * kRows + kRows * HD;  // floats
    static_assert(GB % 16 == 0 && OFF_BAR % 16 == 0, "alignment");
    static_assert(2 * WARPS * STAGES <= THREADS && WARPS <= 32, "one thread per barrier, one lane per warp");
    static_assert(WARPS <= kMostWarps, "the workspace has room for every warp's pieces");
    static_assert(RING >= kRows * HD * 4, "a warp's O fits its ring");
    static_assert(SMEM <= 225 * 1024, "shared memory");
};

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

template <int N>
__device__ __forceinline__ void lds_words(uint32_t *w, const uint8_t *p) {
    if (N == 2)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[N - 1]) : "r"(smem_u32(p)));
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(smem_u32(p)));
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
// D (16x8 fp32) += A (16x16 fp16) * B (16x8 fp16); not volatile, so that the
// compiler may interleave the chains of different blocks.
__device__ __forceinline__ void mma(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// A warp's place in its run and what the unit it is in needs once per piece or
// in the groups that not every row sees whole. In shared memory: the loop over
// the groups has no registers to spare.
struct Piece {
    int r, unit, gi, todo;      // request, unit (kv head and row group), group, groups left in the run
    int n, end;                 // groups of the unit, and where the piece ends
    int pos[kRows];             // the columns' positions
    int p_min, p_max;           // of all of them
    int ns, skip;               // group i of the unit is i, or i + skip from ns on
    int fin_r, fin_unit;        // the piece that ends the run, if other warps have more of its unit (else -1)
    long long fin_first, fin_last;  // that unit's groups in the cut
    float m[kRows], l[kRows];   // and the piece's references and sums
};

constexpr float kLn2 = 0.693147180559945309f, kLog2e = 1.442695040888963407f;

template <typename T, int HD>
__global__ void __launch_bounds__((Cfg<T, HD>::THREADS), 1) paged_attn_kernel(PagedAttnArgs a) {
    using C = Cfg<T, HD>;
    constexpr int NB = C::NB, S = C::STAGES;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long scan_part[C::WARPS + 1];
    __shared__ int start_r[C::WARPS];
    __shared__ long long start_x[C::WARPS];
    __shared__ Piece pieces[C::WARPS];
    __shared__ int abort_flag;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int n_kv = a.pages.n_kv, page_groups = n_kv * a.pages.groups;
    const int log_group = 31 - __clz(a.n_q_heads / n_kv);
    uint8_t *ring = smem + warp * C::RING;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);  // [warp][stage]
    uint64_t *empty = full + C::WARPS * S;
    volatile int *dead = reinterpret_cast<int *>(smem + C::OFF_DEAD);  // stages without rows
    uint8_t *qs = smem + C::OFF_Q + warp * C::QB;
    uint8_t *bias = smem + C::OFF_BIAS + warp * C::BIAS;
    const Ws ws = carve(a.workspace, gridDim.x);

    if (tid < 2 * C::WARPS * S) mbar_init(full + tid, 1);
    if (tid == 0) abort_flag = 0;
    mbar_fence_init();
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
    for (int i = 0; i <= C::WARPS; ++i) {
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

    if (warp == C::WARPS) {
        // ---- the copying warp: lane w walks the run of warp w, up to S groups ahead of it
        const int wid = blockIdx.x * cut.A + lane;
        int left = 0;  // groups to copy
        int r = 0, unit = 0, units = 1, rgs = 1, ci = 0, cn = 1, ns = 0, skip = 0, head = 0;
        const int32_t *table = a.pages.table;
        auto enter = [&](const Req &q) {
            cn = max(q.ng, 1);
            ns = q.ng > 0 ? q.ns : -1;  // -1: nothing to read
            skip = q.skip;
            rgs = q.rgs;
            units = q.rgs * n_kv;
            table = a.pages.table + static_cast<size_t>(r) * a.pages.max_pages;
        };
        if (lane < cut.A && wid < cut.W && N > 0) {
            const long long x0 = cut.start(wid);
            left = static_cast<int>(cut.start(wid + 1) - x0);
            r = start_r[lane];
            enter(load_req(a, r, log_group));
            const long long off = x0 - start_x[lane];
            unit = static_cast<int>(off / cn);
            ci = static_cast<int>(off - static_cast<long long>(unit) * cn);
            head = unit / rgs * a.pages.groups;
        }
        int stage = 0, lap = 0, page = 0, group = 0;
        auto look = [&]() {  // the table entry of the next group, one step before its copy
            group = ci < ns ? ci : ci + skip;
            page = ns >= 0 ? __ldg(table + (group >> a.pages.group_shift)) : -2;
            group = (group & (a.pages.groups - 1)) + head;
        };
        if (left > 0) look();
        long long t0 = clock64();
        while (__any_sync(~0u, left > 0)) {
            bool went = false;
            uint64_t *bar = full + lane * S + stage;
            if (left > 0 && (lap == 0 || mbar_try_wait(empty + lane * S + stage, (lap - 1) & 1))) {
                went = true;
                if (static_cast<unsigned>(page) < static_cast<unsigned>(a.pages.n_pages)) {
                    dead[lane * S + stage] = 0;
                    mbar_arrive_expect_tx(bar, C::GB);
                    bulk_copy_g2s(smem + lane * C::RING + stage * C::GB,
                                  a.pages.base + (static_cast<size_t>(page) * page_groups + group) * C::GB,
                                  C::GB, bar);
                } else {
                    dead[lane * S + stage] = 1;
                    mbar_arrive(bar);
                    if (page != -2) flag_error(a.err, FA_ERRBIT_DEVICE);
                }
                if (++stage == S) stage = 0, ++lap;
                if (--left > 0) {
                    if (++ci == cn) {
                        ci = 0;
                        if (++unit == units) {
                            unit = 0;
                            Req q;
                            do q = load_req(a, ++r, log_group); while (q.rgs == 0);
                            enter(q);
                        }
                        head = unit / rgs * a.pages.groups;
                    }
                    look();
                }
            }
            if (__any_sync(~0u, went)) {
                t0 = clock64();
            } else {
                __nanosleep(40);
                const bool late = clock64() - t0 > 2 * kSpinCycles;
                if (late && lane == 0) {
                    abort_flag = 1;
                    flag_error(a.err, FA_ERRBIT_TIMEOUT);
                }
                if (__any_sync(~0u, late || *static_cast<volatile int *>(&abort_flag))) break;
            }
        }
    }

    volatile Piece *pc = pieces + min(warp, C::WARPS - 1);
    State<NB> st;
    st.clear();
    if (warp < C::WARPS) {
        const int wid = blockIdx.x * cut.A + warp;
        if (lane == 0) {
            ws.tasks[blockIdx.x * C::WARPS + warp].valid = 0;
            pc->fin_unit = -1;
            pc->todo = 0;
            if (warp < cut.A && wid < cut.W && N > 0) {
                const long long x0 = cut.start(wid), off = x0 - start_x[warp];
                const int n = max(load_req(a, start_r[warp], log_group).ng, 1);
                const int unit = static_cast<int>(off / n);
                pc->r = start_r[warp];
                pc->unit = unit;
                pc->gi = static_cast<int>(off - static_cast<long long>(unit) * n);
                pc->todo = static_cast<int>(cut.start(wid + 1) - x0);
            }
        }
        __syncwarp();
        // ---- the run, piece by piece
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
#pragma unroll 1
        while (pc->todo > 0) {
            int gi = pc->gi, g_end, f0, f1;
            float km[2];
            {
            const Req q = load_req(a, pc->r, log_group);
            const int n = max(q.ng, 1), unit = pc->unit;
            const int h = unit / q.rgs, rg = unit - h * q.rgs;
            g_end = min(n, gi + pc->todo);
            // ---- q of row g as B fragments: dims 32 b + 8 t + (0,4 | 1,5 | 2,6 | 3,7),
            // the second and fourth times 2^-4; brought to a maximum in [2^10, 2^11)
            {
                const Col c = column(q, rg, g, h, log_group);
                const T *src = static_cast<const T *>(a.q) + max(c.token, 0) * a.q_stride +
                               static_cast<long long>(c.head) * HD + 8 * t;
                float x[8], top = 0.0f;
                if (c.token >= 0) {
#pragma unroll 4
                    for (int b = 0; b < NB; ++b) {
                        load8(src + 32 * b, x);
#pragma unroll
                        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
                    }
                }
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
#pragma unroll 2
                for (int b = 0; b < NB; ++b) {
                    float sum = 0.0f;
                    if (c.token >= 0) load8(src + 32 * b, x);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] = c.token >= 0 ? x[i] * lift : 0.0f;
                        sum += x[i];
                    }
                    sum += __shfl_xor_sync(~0u, sum, 1);
                    sum += __shfl_xor_sync(~0u, sum, 2);
                    // -8 * 2^-24 of columns 2 t, 2 t + 1 in the order of an accumulator
                    sum *= -4.76837158203125e-7f;
                    const float s0 = __shfl_sync(~0u, sum, 8 * t), s1 = __shfl_sync(~0u, sum, 8 * t + 4);
                    if (g == 0)
                        *reinterpret_cast<float4 *>(bias + (b * 4 + t) * 16) = make_float4(s0, s1, s0, s1);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        hi[i] = pack_half2(x[i], x[i + 4]);
                        const float2 f = half2_f(hi[i]);
                        const float sc = i & 1 ? 0.0625f : 1.0f;
                        if (i & 1) hi[i] = pack_half2(f.x * sc, f.y * sc);
                        lo[i] = pack_half2((x[i] - f.x) * sc, (x[i + 4] - f.y) * sc);
                    }
                    *reinterpret_cast<uint4 *>(qs + (b * 32 + lane) * 16) =
                        make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    if (C::QSPLIT)
                        *reinterpret_cast<uint4 *>(qs + C::QF + (b * 32 + lane) * 16) =
                            make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            const int p_min = q.rows - q.nq + ((rg * kRows) >> log_group);
            const int p_max = q.rows - q.nq +
                              min(q.nq - 1, (rg * kRows + kRows - 1) >> log_group);
            if (lane < kRows) pc->pos[lane] = column(q, rg, lane, h, log_group).pos;
            if (lane == 0) {
                pc->n = n;
                pc->end = g_end;
                pc->p_min = p_min;
                pc->p_max = p_max;
                pc->ns = q.ns;
                pc->skip = q.skip;
            }
            // groups [f0, f1) of the unit are seen whole by every row
            f0 = 0;
            f1 = max(0, p_min + 1) / kGroupRows - q.skip;
            if (a.win > 0)
                f0 = max(q.ns, (max(-1, p_max - a.win) + kGroupRows) / kGroupRows - q.skip);
            }
            __syncwarp();
            st.clear();

#pragma unroll 1
            for (; gi < g_end; ++gi) {
                uint64_t *bar = full + warp * S + stage;
                if (ok) ok = mbar_wait(bar, phase, &abort_flag, a.err);
                if (ok && !dead[warp * S + stage]) {
                    const uint8_t *kp = ring + stage * C::GB, *vp = kp + part_bytes(HD);
                    // ---- scores of rows g, g + 8 (y[0..1], y[2..3]) and columns 2 t, 2 t + 1
                    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    // codes of rows g, g + 8 and their block scales, 4 blocks (2 of head_dim 64)
                    // at a time: with all of a group's at once the registers do not suffice
                    constexpr int KB = NB < 4 ? NB : 4;
                    uint32_t wAs[KB], wBs[KB], sA[KB / 2], sB[KB / 2];
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        if (b % KB == 0) {
                            if (NB == 2) {
                                const uint4 w = lds_v4(kp + lane * 16);
                                wAs[0] = w.x; wAs[1] = w.y; wBs[0] = w.z; wBs[1] = w.w;
                            } else {
                                const uint4 w = lds_v4(kp + ((b / 4) * 32 + lane) * 16);
                                const uint4 x = lds_v4(kp + (((NB + b) / 4) * 32 + lane) * 16);
                                wAs[0] = w.x; wAs[1] = w.y; wAs[2 % KB] = w.z; wAs[3 % KB] = w.w;
                                wBs[0] = x.x; wBs[1] = x.y; wBs[2 % KB] = x.z; wBs[3 % KB] = x.w;
                            }
                            lds_words<KB / 2>(sA, kp + scale_offset(HD) + g * (2 * NB) + 2 * b);
                            lds_words<KB / 2>(sB, kp + scale_offset(HD) + (g + 8) * (2 * NB) + 2 * b);
                        }
                        const uint4 qf = lds_v4(qs + (b * 32 + lane) * 16);
                        const float4 c0 = lds_f4(bias + (b * 4 + t) * 16);
                        float d[4] = {c0.x, c0.y, c0.z, c0.w};
                        const uint32_t wA = wAs[b % KB], wB = wBs[b % KB];
                        const uint32_t vA = wA >> 8, vB = wB >> 8;
                        const uint32_t e0 = wA & 0x000f000fu, e1 = wB & 0x000f000fu;
                        const uint32_t e2 = wA & 0x00f000f0u, e3 = wB & 0x00f000f0u;
                        const uint32_t f0 = vA & 0x000f000fu, f1 = vB & 0x000f000fu;
                        const uint32_t f2 = vA & 0x00f000f0u, f3 = vB & 0x00f000f0u;
                        mma(d, e0, e1, e2, e3, qf.x, qf.y);
                        mma(d, f0, f1, f2, f3, qf.z, qf.w);
                        if (C::QSPLIT) {
                            const uint4 lo = lds_v4(qs + C::QF + (b * 32 + lane) * 16);
                            mma(d, e0, e1, e2, e3, lo.x, lo.y);
                            mma(d, f0, f1, f2, f3, lo.z, lo.w);
                        }
                        const float2 uA = half2_f(sA[b % KB / 2]), uB = half2_f(sB[b % KB / 2]);
                        const float a0 = b & 1 ? uA.y : uA.x, a1 = b & 1 ? uB.y : uB.x;
                        y[0] = fmaf(a0, d[0], y[0]);
                        y[1] = fmaf(a0, d[1], y[1]);
                        y[2] = fmaf(a1, d[2], y[2]);
                        y[3] = fmaf(a1, d[3], y[3]);
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
                    if (gi < f0 || gi >= f1) {
                        const int j0 = (gi < pc->ns ? gi : gi + pc->skip) * kGroupRows;
                        const int p0 = pc->pos[2 * t], p1 = pc->pos[2 * t + 1];
                        const int p_min = pc->p_min, p_max = pc->p_max;
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
                        if (g < NB / 2) {  // V's scales of rows 2t, 2t+1 | 2t+8, 2t+9 and two blocks
                            uint4 *w = reinterpret_cast<uint4 *>(ring + stage * C::GB + part_bytes(HD) +
                                                                 scale_offset(HD) + (g * 4 + t) * 16);
                            *w = make_uint4(w->x & m01, w->y & m23, w->z & m01, w->w & m23);
                        }
                        fence_proxy_async_smem();  // before the next copy into the stage
                        __syncwarp();
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
                    uint4 vs;
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
                        if (b % 2 == 0) vs = lds_v4(vp + scale_offset(HD) + ((b / 2) * 4 + t) * 16);
                        const uint32_t s01 = b & 1 ? vs.z : vs.x, s23 = b & 1 ? vs.w : vs.y;
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
                if (ok && lane == 0) mbar_arrive(bar + C::WARPS * S);
                if (++stage == S) stage = 0, phase ^= 1;
            }

            // ---- the piece is done
            st.sum_lanes();
            const int r = pc->r, unit = pc->unit, n = pc->n, first = pc->gi, end = pc->end;
            const int todo = pc->todo - (end - first);
            const int wid = blockIdx.x * cut.A + warp;
            const Req q = load_req(a, r, log_group);
            if (first == 0 && end == n) {
                const int h = unit / q.rgs, rg = unit - h * q.rgs;
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
            } else {  // the end of the run: into the ring, whose copies have all been used
                if (g == 0) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        pc->m[2 * t + c] = st.m[c];
                        pc->l[2 * t + c] = st.l[c];
                    }
                }
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        *reinterpret_cast<float4 *>(ring + ((b * 2 + c) * 32 + lane) * 16) = st.quad(b, c);
            }
            __syncwarp();
            if (lane == 0) {
                if (todo == 0 && !(first == 0 && end == n)) {
                    pc->fin_r = r;
                    pc->fin_unit = unit;
                    pc->fin_first = cut.start(wid + 1) - end;
                    pc->fin_last = cut.start(wid + 1) - end + n;
                }
                int next = unit + 1, nr = r;
                if (todo > 0 && next == q.rgs * n_kv) {
                    next = 0;
                    while (load_req(a, ++nr, log_group).rgs == 0) {}
                }
                pc->r = nr;
                pc->unit = next;
                pc->gi = 0;
                pc->todo = todo;
            }
            __syncwarp();
        }
    }
    if (*static_cast<volatile int *>(&abort_flag)) {
        // a wait ran out: give copies in flight half a millisecond before their memory is given up
        const long long t0 = clock64();
        while (clock64() - t0 < 1000000) {}
    }

    // ---- join the pieces that end the warps' runs, unit by unit
    __syncthreads();
    if (warp >= C::WARPS || pc->fin_unit < 0) return;
    const int r = pc->fin_r, unit = pc->fin_unit;
    const long long first = pc->fin_first, last = pc->fin_last;
    auto same = [&](int w) { return pieces[w].fin_unit == unit && pieces[w].fin_r == r; };
    int w0 = warp, w1 = warp + 1;  // warps [w0, w1) hold pieces of this unit
    while (w0 > 0 && same(w0 - 1)) --w0;
    while (w1 < C::WARPS && same(w1)) ++w1;
    const int id0 = blockIdx.x * cut.A + w0, id1 = blockIdx.x * cut.A + w1;
    const bool from_start = cut.start(id0) <= first, direct = from_start && cut.start(id1) >= last;
    float M[2] = {kLowest, kLowest}, L[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int n = 2 * t + c;
        for (int w = w0; w < w1; ++w) M[c] = fmaxf(M[c], pieces[w].m[n]);
        for (int w = w0; w < w1; ++w) L[c] += pieces[w].l[n] * ex2(pieces[w].m[n] - M[c]);
    }
    const Req q = load_req(a, r, log_group);
    const int h = unit / q.rgs, rg = unit - h * q.rgs;
    float *dst = ws.partial + static_cast<size_t>(id0) * 2 * C::PARTIAL;
    if (from_start && !direct && warp == w0 && lane == 0)
        ws.tasks[blockIdx.x * C::WARPS + warp] = Task{1, r, unit, id0, first, last, cut.N, cut.W, cut.A};
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
            const float f = ex2(pieces[w].m[2 * t + c] - M[c]);
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
