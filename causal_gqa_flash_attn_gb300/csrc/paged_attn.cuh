// paged_attn.cuh -- attention of ragged queries over 4-bit pages (include/fa.h,
// fa_paged_attn and fa_paged_attn_scored); instantiated in paged_attn.cu and, with
// SCORED, in paged_attn_scored.cu.
//
// Query t of a request with n queries and L rows sits at position p = L - n + t
// and attends keys j <= p (with win > 0 only sinks and the recent window):
//   s_j = scale * q . k_j,  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
//   lse = m + log sum_j exp(s_j - m).
// SCORED: s_j becomes cap * tanh(s_j / cap) where a cap is given, less slope * (p - j)
// where slopes are.
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
//     the accumulator's start (K) or by a constant operand (V).
//   - The columns (N = 8) are 8 query rows of one kv head: the group's q heads,
//     times as many tokens as fit ("row group"; 16 rows where 16 heads share).
//   - V's block scales multiply the softmax weights (8 columns) instead of the
//     codes; each V row's power-of-two factor 2^e is added to its score's
//     exponent, so the scaled weights 2^(s + e - m) stay in binary16's range
//     whatever the values' magnitude.
//   - The reference m that these are taken relative to is moved only when one
//     passes it by 2^14 (kLift above the last maximum, up to binary16's range):
//     one vote per tile instead of a reduction.
//   - The sum of weights has nothing to do with V. While every e is within
//     +-kNear a scaled weight times 2^-e is what it needs, relative to the same m:
//     at most 2^44, and one that fp32 loses on the way is below 2^-72 of the
//     largest. Columns that see other rows take the weights of such a group from
//     the scores, and have a reference r of these for their sums where m is not near
//     enough to serve (sum_apart).
//   - A row of zeros (a null token) is stored with e = 0, which says nothing of its
//     V: it does not move m, below which smaller rows would be lost. Nor does a row
//     whose blocks are infinite or 0 (an infinity makes e 127): any weight times its
//     infinite scales is the NaN that these blocks stand for.
// fp32 queries are split into two binary16 terms, and for fp32 and fp16 so are
// the scaled weights. Their codes become (c - 8) * 2^-9 (one AND and one packed
// multiply-add for two): the tensor core aligns a sum's terms by their
// exponents and cuts them, so that subnormal operands, whose leading bits are
// zeros, and an offset that is taken out later lose bits (outputs off by 3e-6
// instead of 3e-7). Its sums lose a step towards zero per addition, too: a tile's
// products with V go through a fresh accumulator that is added in fp32.
//
// Work split. The 16-row groups that are read, over all (request, kv head, row
// group) units, are cut into equal runs, one per warp of one block per SM; a
// warp streams its run through its own ring of bulk copies, which one more warp
// issues. A unit inside one warp's run is written directly. Pieces of longer
// units are joined by their block: they end the runs of neighbouring warps and
// lie in their rings, but for a last one that begins a run, which waits in the
// workspace (TAILS). Units that several blocks share are joined by a second
// kernel. All in a fixed order.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <type_traits>

#include "fa_device.cuh"
#include "fa_internal.h"
#include "paged_launch.cuh"
#include "paged_layout.cuh"

namespace fa {
namespace {

constexpr float kLowest = -3e38f;  // reference of a row that has seen no key: below any score
constexpr float kLift = 6.0f;      // log2 of the largest weight right after a move
constexpr float kMost = 14.0f;     // log2 weight that moves the reference
constexpr int kNear = 30;          // |e| of V's rows whose scaled weights the sum of weights can use
constexpr int kBias = 127;         // of fp32's exponents
// The start and end of a unit (its rows of q as operands, its output) cost a
// warp about as much as kUnitCost groups: 6000 against 2200 cycles.
constexpr int kUnitCost = 3;
// Work per warp below which fewer warps work. One request of 600 rows 11.7 us
// (12.3 with 6, 13.9 with 9), 32 of 64 rows 13.5 (15.3, 17.5), long ones alike.
constexpr int kMinWork = 4;
// Requests that each warp sums by itself, one a lane, without a step of the whole
// block: 32 requests of 2048 rows 21.1 us instead of 22.0, one of 600 rows 12.7 instead
// of 13.4 (when measured). With several requests a lane nothing is left of that (64: 21.9 and 22.1, 256:
// 42.5 and 41.3, 1000: 75 and 58).
constexpr int kFewReqs = 32;
constexpr int kMostBlocks = 256;   // blocks, whose warps' tasks the join lists
constexpr int kMostWarps = 16;     // computing warps of a block that the workspace is made for
constexpr float kLn2 = 0.693147180559945309f, kLog2e = 1.442695040888963407f;

template <typename T, int HD, int NT_>
struct Cfg {
    static constexpr int NT = NT_, ROWS = 8 * NT;  // columns of a unit, in eights and all
    static constexpr bool QSPLIT = sizeof(T) == 4;
    static constexpr bool PSPLIT = !std::is_same<T, __nv_bfloat16>::value;
    static constexpr int NB = HD / 32;
    static constexpr int GB = group_bytes(HD);
    // Warps that compute (and one more that copies), groups that are taken at once (TILE) and
    // tiles of a warp's ring, as measured: as many warps as have registers for their state, with
    // the copying one a multiple of the SM's four schedulers, and tiles that give that one few
    // copies to issue. Head_dim 256, bf16 (32 x 32768 rows, 2 kv heads): 11 warps 112 us, 10 120,
    // 12 124, 13 128, 7 130, 11 with tiles of two groups 2% slower; head_dim 128 (32 x 16384 rows,
    // 8 kv heads): bf16 15 warps 114 us, 14 121, 13 127, fp32 11 warps 158 us, 12 162, 10 171,
    // 13 with single groups 183; head_dim 64, bf16 (64 x 16384 rows, 4 kv heads): tiles of four
    // groups 69 us, single groups 124.
    static constexpr int WARPS = HD == 256 || (HD == 128 ? PSPLIT || NT == 2 : PSPLIT && NT == 2) ? 11 : 15;
    static constexpr int TILE = HD == 256 ? 1 : HD == 128 || NT == 2 ? 2 : 4;
    static constexpr int STAGES = HD == 256 ? (QSPLIT ? 2 : 3) : HD == 64 && NT == 2 ? 4 : 2;
    // What a warp begins its run with is joined by its block, if that has the unit's other pieces:
    // 256 x 300 rows of 8 kv heads x 128, 41.1 -> 35.3 us, when each unit has such an end. With
    // head_dim 256 the second kernel does it better (128 windowed requests 19.5 us, 23.4 here; 32
    // requests of 32768 rows 109.3 and 114.1).
    static constexpr bool TAILS = HD < 256;
    static constexpr int STAGE = TILE * GB;
    static constexpr int RING = STAGES * STAGE;
    static constexpr int QF = NB * 32 * 16;           // q as B fragments
    static constexpr int QB = QF * NT * (QSPLIT ? 2 : 1);  // of each eight, and their low terms
    static constexpr int BIAS = QSPLIT ? 0 : NT * NB * 4 * 16;  // the accumulators' start, as lanes hold it
    static constexpr int OFF_Q = WARPS * RING;
    static constexpr int OFF_BIAS = OFF_Q + WARPS * QB;
    static constexpr int OFF_BAR = OFF_BIAS + WARPS * BIAS;
    static constexpr int OFF_DEAD = OFF_BAR + WARPS * STAGES * 8;
    static constexpr int SMEM = OFF_DEAD + WARPS * STAGES * 4;
    static constexpr int THREADS = (WARPS + 1) * 32;
    // a partial: m and l of the rows, then O as the lanes hold it
    static constexpr int PARTIAL = 2 * ROWS + ROWS * HD;  // floats
    static_assert(GB % 16 == 0 && OFF_BAR % 16 == 0, "alignment");
    static_assert(WARPS * STAGES <= THREADS && WARPS <= 32, "one thread per barrier, one lane per warp");
    static_assert(WARPS <= kMostWarps, "the workspace has room for every warp's pieces");
    static_assert(RING >= ROWS * HD * 4, "a warp's O fits its ring");
    static_assert(SMEM <= 224 * 1024, "shared memory");
};

// How a request's rows are read, from its lengths.
struct Req {
    int q0, nq, rows;      // first token, queries, rows
    int ns, skip, ng;      // sink groups, groups left out after them, groups read
    int rgs;               // row groups of each kv head (0: nothing to do)
    bool bad;
};

template <int ROWS>
__device__ __forceinline__ Req load_req(const PagedAttnArgs &a, int r, int log_group) {
    Req q;
    q.q0 = a.cu_q[r];
    const int q1 = a.cu_q[r + 1];
    q.rows = a.seq_lens[r];
    const long long room = static_cast<long long>(a.pages.max_pages) * a.pages.groups * kGroupRows;
    q.bad = q.q0 < 0 || q1 < q.q0 || q1 > a.n_tokens || q.rows < 0 || q.rows > room;
    q.nq = q.bad ? 0 : q1 - q.q0;
    q.rgs = static_cast<int>(((static_cast<long long>(q.nq) << log_group) + ROWS - 1) / ROWS);
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
// The next request with queries, whose index goes into *r: there is one, as the
// run goes on (and no reading past the last one, should lengths change meanwhile).
template <int ROWS>
__device__ __forceinline__ Req next_req(const PagedAttnArgs &a, int *r, int log_group) {
    Req q;
    do {
        *r = min(*r + 1, a.n_reqs - 1);
        q = load_req<ROWS>(a, *r, log_group);
    } while (q.rgs == 0 && *r < a.n_reqs - 1);
    return q;
}
// Groups of a unit: at least one, so that rows without any key are visited and
// written too.
__device__ __forceinline__ int unit_groups(const Req &q) { return max(q.ng, 1); }

// Quotients of 64-bit counts, which mostly have 32.
__device__ __forceinline__ long long quotient(long long n, int d) {
    return n >> 32 ? n / d : static_cast<long long>(static_cast<unsigned>(n) / static_cast<unsigned>(d));
}

// The cut of the work. Its measure is a group, and kUnitCost ahead of those of
// each unit: N in all, c for each of B blocks, cw of those for each of A warps
// (the last ones may have fewer, or none). A warp's run is the groups whose
// measure lies in its part. A part may have none: a block's last, or one that lies
// wholly ahead of a unit's first group (parts are kUnitCost long where a block has 5, 6
// or 9). Between two groups of a unit there is no such part, so that the warps of a
// block that hold a unit's pieces are neighbours, as the joins take for granted.
struct Cut {
    long long N, c;
    int cw, B, A;
    __device__ __forceinline__ long long start(int b, int i) const {
        return min(b * c + min(static_cast<long long>(i) * cw, c), N);
    }
    __device__ __forceinline__ int warp_of(long long x) const {  // c < 2^31: 2^40 groups at most
        const int b = static_cast<int>(quotient(x, static_cast<int>(c)));
        return b * A + static_cast<int>(quotient(x - b * c, cw));
    }
};
template <int WARPS>
__device__ __forceinline__ Cut make_cut(long long N, int blocks) {
    Cut t;  // with few divisions, most of them by constants
    t.N = N;
    t.B = blocks;
    if (N < static_cast<long long>(blocks) * kMinWork)
        t.B = max(static_cast<int>((static_cast<unsigned>(N) + kMinWork - 1) / kMinWork), 1);
    t.c = max(quotient(N + t.B - 1, t.B), 1ll);
    const unsigned c = static_cast<unsigned>(t.c);
    t.A = c < WARPS * kMinWork ? static_cast<int>((c + kMinWork - 1) / kMinWork) : WARPS;
    t.cw = static_cast<int>(t.A == WARPS ? (c + WARPS - 1) / WARPS : (c + t.A - 1) / static_cast<unsigned>(t.A));
    return t;
}

// A unit that other blocks share, for the join: written by the warp whose run
// holds its first group. Where its pieces lie is one word:
//   bits 0-8    the blocks that hold joined pieces (0: no task)
//   bits 9-13   the warps of a block that work
//   bits 14-26  1 + the warp (over all blocks) that begins its run with the unit's last piece
//               and goes on, where its block does not join that piece, or 0
struct Task {
    int h, rg;
    Req q;
};
__device__ __forceinline__ uint32_t pack_pieces(int blocks, int warps, int tail) {
    return static_cast<uint32_t>(blocks) | static_cast<uint32_t>(warps) << 9 |
           static_cast<uint32_t>(tail + 1) << 14;
}
// Where a part of the cut begins.
struct Place {
    int r, unit, gi;   // its first group
    int ahead;         // measure of the unit's start that lies before it (of kUnitCost)
    long long groups;  // groups before it
};
struct Ws {
    uint32_t *pieces;   // [block][kMostWarps]: pack_pieces, or 0
    Task *tasks;        // [block][kMostWarps]
    float *partial;  // two per warp: the end of its run, the start of its run
};
__host__ __device__ constexpr size_t ws_head(int blocks, size_t each) {
    return (static_cast<size_t>(blocks) * kMostWarps * each + 255) / 256 * 256;
}
__host__ __device__ inline Ws carve(uint8_t *ws, int blocks) {
    Ws w;
    w.pieces = reinterpret_cast<uint32_t *>(ws);
    w.tasks = reinterpret_cast<Task *>(ws + ws_head(blocks, 4));
    w.partial = reinterpret_cast<float *>(ws + ws_head(blocks, 4) + ws_head(blocks, sizeof(Task)));
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

// 8 consecutive values as they lie in memory.
template <typename T>
struct Raw8 {
    static constexpr int N = sizeof(T) / 2;
    uint4 w[N];
    __device__ __forceinline__ void load(const T *p, bool there) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            w[i] = there ? *(reinterpret_cast<const uint4 *>(p) + i) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float *x) const {
        if constexpr (N == 2) {
            x[0] = __uint_as_float(w[0].x); x[1] = __uint_as_float(w[0].y);
            x[2] = __uint_as_float(w[0].z); x[3] = __uint_as_float(w[0].w);
            x[4] = __uint_as_float(w[1].x); x[5] = __uint_as_float(w[1].y);
            x[6] = __uint_as_float(w[1].z); x[7] = __uint_as_float(w[1].w);
        } else {
            const uint32_t h[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (std::is_same<T, __half>::value) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
                    x[2 * i] = f.x;
                    x[2 * i + 1] = f.y;
                } else {
                    x[2 * i] = __uint_as_float(h[i] << 16);
                    x[2 * i + 1] = __uint_as_float(h[i] & 0xffff0000u);
                }
            }
        }
    }
};

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// a * b - c
__device__ __forceinline__ uint32_t hfms2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("{.reg .b32 n; neg.f16x2 n, %3; fma.rn.f16x2 %0, %1, %2, n;}" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// All bits of each half that is not zero (or a NaN).
__device__ __forceinline__ uint32_t not_zero2(uint32_t h) {
    return (h & 0x7fffu ? 0xffffu : 0u) | (h & 0x7fff0000u ? 0xffff0000u : 0u);
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

// D = A * B
__device__ __forceinline__ void mma0(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                     uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// -8 * 2^-24 and -8 * 2^-20, twice.
constexpr uint32_t kM8a = 0x80088008u, kM8b = 0x80808080u;
constexpr uint32_t kLo = 0x000f000fu, kHi = 0x00f000f0u;  // codes c * 2^-24, c * 2^-20

// Two codes (bits 0-3, or 4-7, of each half of w) as (c - 8) * 2^-9: normal
// numbers, from c * 2^-24 and c * 2^-20.
__device__ __forceinline__ uint32_t minus8_lo(uint32_t w) {
    return hfma2(w & kLo, 0x78007800u, 0xa400a400u);  // * 2^15 - 2^-6
}
__device__ __forceinline__ uint32_t minus8_hi(uint32_t w) {
    return hfma2(w & kHi, 0x68006800u, 0xa400a400u);  // * 2^11 - 2^-6
}

// A count in shared memory from warp to warp: what its writer did before is done
// for who reads it.
__device__ __forceinline__ void release_s32(volatile int *p, int v) {
    asm volatile("st.release.cta.shared.s32 [%0], %1;" ::"r"(smem_u32(const_cast<int *>(p))), "r"(v) : "memory");
}
__device__ __forceinline__ int acquire_s32(volatile int *p) {
    int v;
    asm volatile("ld.acquire.cta.shared.s32 %0, [%1];" : "=r"(v) : "r"(smem_u32(const_cast<int *>(p))) : "memory");
    return v;
}

// Row and head of a unit's column n; token < 0 past the unit's last row.
__device__ __forceinline__ int log_group_of(const PagedAttnArgs &a) {
    return 31 - __clz(a.n_q_heads / a.pages.n_kv);
}
struct Col {
    int token, head, pos;
};
template <int ROWS>
__device__ __forceinline__ Col column(const Req &q, int rg, int n, int h, int log_group) {
    const int row = rg * ROWS + n, i = row >> log_group;
    Col c;
    c.token = i < q.nq ? q.q0 + i : -1;
    c.head = (h << log_group) + (row & ((1 << log_group) - 1));
    c.pos = i < q.nq ? q.rows - q.nq + i : -1;
    return c;
}

// The state of one piece: O, references and weight sum of the lane's columns
// 8 e + 2 t and 8 e + 2 t + 1 (O: dims 32 b + 4 g + 0, 2 in rows g of tiles 0, 1
// and 32 b + 4 g + 1, 3 in rows g + 8).
template <typename C>
struct State {
    static constexpr int NB = C::NB, NT = C::NT;
    // the codes' factors come out of rows g and g + 8
    static constexpr float U0 = C::PSPLIT ? 512.0f : 16777216.0f, U1 = C::PSPLIT ? 512.0f : 1048576.0f;
    float o[NT][NB][2][4];
    float m[NT][2], l[NT][2];  // (r is m, or in the Piece)
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int e = 0; e < NT; ++e) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 8; ++i) o[e][b][i >> 2][i & 3] = 0.0f;
            m[e][0] = m[e][1] = kLowest;
            l[e][0] = l[e][1] = 0.0f;
        }
    }
    // four consecutive dims of column 8 e + 2 t + c in block b
    __device__ __forceinline__ float4 quad(int e, int b, int c) const {
        return make_float4(o[e][b][0][c] * U0, o[e][b][0][2 + c] * U1, o[e][b][1][c] * U0,
                           o[e][b][1][2 + c] * U1);
    }
    __device__ __forceinline__ void sum_lanes() {
#pragma unroll
        for (int e = 0; e < NT; ++e)
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
                l[e][0] += __shfl_xor_sync(~0u, l[e][0], d);
                l[e][1] += __shfl_xor_sync(~0u, l[e][1], d);
            }
    }
    // Columns with an r of their own get one reference for O and l, halfway between m and r: with 2^+-140
    // between them at most (V's largest and smallest numbers), both stay far from the ends of fp32.
    __device__ __forceinline__ void join_references(uint32_t own, const volatile float *base) {
        const int t = threadIdx.x & 3;
#pragma unroll
        for (int e = 0; e < NT; ++e)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (!(own >> (8 * e + 2 * t + c) & 1)) continue;
                // (if all rows were without content, m is kLowest and O 0)
                const float ahead = fmaxf(m[e][c] - base[8 * e + 2 * t + c], -160.0f), up = floorf(0.5f * ahead);
                const float f = ex2(up);
                l[e][c] *= ex2(up - ahead);
                m[e][c] = base[8 * e + 2 * t + c] + ahead - up;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        o[e][b][i][c] *= f;
                        o[e][b][i][2 + c] *= f;
                    }
            }
    }
    // where quad(e, b, c) lies in a partial or a ring, in float4s of the warp's lanes
    __device__ __forceinline__ static int quad_at(int e, int b, int c) { return (e * NB + b) * 2 + c; }
};

__device__ __forceinline__ float4 scaled(float4 v, float s) {
    return make_float4(v.x * s, v.y * s, v.z * s, v.w * s);
}

// Four dims of a finished row, and with the first ones its log-sum-exp.
template <typename T>
__device__ __forceinline__ void write_row(const PagedAttnArgs &a, const Col &col, int hd, int dim,
                                          float4 x, float m, float l) {
    if (col.token < 0) return;
    store4<T>(static_cast<T *>(a.out) + col.token * a.out_stride +
                  static_cast<long long>(col.head) * hd + dim,
              scaled(x, l > 0.0f ? 1.0f / l : l));  // nothing attended: 0 (a NaN stays one)
    if (a.lse && dim == 0)
        a.lse[static_cast<size_t>(col.head) * a.n_tokens + col.token] = (m + log2f(l)) * kLn2;
}

// Groups that are taken at once from group i of a unit on, which is read up to
// group `end`: a tile begins at a multiple of TILE, and at its page's if the
// page has TILE groups or more.
template <int TILE>
__device__ __forceinline__ int tile_size(int i, int end, int ns, int skip) {
    if (TILE == 1) return 1;
    const int most = i < ns ? min(ns, end) - i : end - i;
    return min(TILE - ((i < ns ? i : i + skip) & (TILE - 1)), most);
}

// A warp's place in its run and what the unit it is in needs once per piece or
// in the groups that not every row sees whole. In shared memory: the loop over
// the groups has no registers to spare.
struct Piece {
    int r, unit, gi, todo;      // request, unit (kv head and row group), group, groups left in the run
    int ahead;                  // measure between the run's last group and the end of its part
    int n, end;                 // groups of the unit, and where the piece ends
    int pos[16];                // the columns' positions
    int ns, skip;               // group i of the unit is i, or i + skip from ns on
    int holes;                  // the run has met a group without rows to read
    int gone;                   // tiles of the run that are done, whose stages are free (released, acquired)
    int fin_r, fin_unit;        // the piece that ends the run, if other warps have more of its unit (else -1)
    long long fin_first, fin_last;  // that unit's groups in the cut's measure
    float m[16], l[16];         // and the piece's references and sums
    uint32_t own;               // columns whose r is not m (a bit for each)
    float base[16];             // and their r
};

// The new reference where the largest value is u. Whole numbers: 2^(m - r) is then exact.
__device__ __forceinline__ float moved(float from, float u) { return u - from > kMost ? floorf(u) - kLift : from; }

__device__ __forceinline__ int exponent(float inv) {  // e of 2^-e
    return kBias - static_cast<int>(__float_as_uint(inv) >> 23);
}

__device__ __forceinline__ float highest(float a, float b) {  // of a column's values in all its lanes
    float u = fmaxf(a, b);
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) u = fmaxf(u, __shfl_xor_sync(~0u, u, d));
    return u;
}

// The sum's weights of two rows in a column, from their scaled ones (which are 0 for an unseen row,
// whose factor may be anything).
template <bool EDGE>
__device__ __forceinline__ float weight_of(float dA, float dB, float invA, float invB) {
    return fmaf(dA, EDGE && dA == 0.0f ? 0.0f : invA, EDGE && dB == 0.0f ? 0.0f : dB * invB);
}

// Whether rows g (bit 0) and g + 8 (bit 1) of a V part have a block scale that is finite and not 0:
// lane t looks at two blocks of both.
template <int HD>
__device__ __forceinline__ uint32_t with_content(const uint8_t *vp) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint4 w = lds_v4(vp + scale_offset(HD) + ((t & (HD / 64 - 1)) * 4 + (g >> 1)) * 16);
    auto fine = [&](uint32_t h) { return (h >> 16 * (g & 1) & 0x7fffu) - 1u < 0x7bffu; };
    uint32_t has = (fine(w.x) || fine(w.z) ? 1u : 0u) | (fine(w.y) || fine(w.w) ? 2u : 0u);
    has |= __shfl_xor_sync(~0u, has, 1);
    return has | __shfl_xor_sync(~0u, has, 2);
}

// A group's weights for columns that see a row of V beyond kNear, or without content, into their sums:
// from the scores, relative to a reference r that follows the scores alone. Where m comes out near that,
// the sum goes back to m. The scaled weights of rows without content become binary16's least, which
// keeps the NaN of infinite blocks apart from unseen rows, whose weights are 0. What enters a column's
// sum, and how, depends on what that column sees and not on its neighbours.
// False, and nothing done, if no column sees such a row. A call, as it is rare: inside step() the 199
// ragged requests in fp32 take 113 us instead of 111.
template <int NT>
struct Group {
    float y[NT][4], inv[2];    // s + e (rows without content: also for their weight) and 2^-e of the lane's rows
    float m[NT][2], l[NT][2];  // as in State, before the group; l: after it
};
template <int HD, int NT>
__device__ __noinline__ bool sum_apart(Group<NT> *group, const uint8_t *kp, volatile Piece *pc) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t had = pc->own, full = with_content<HD>(kp + part_bytes(HD));
    uint32_t apart = had, own = 0;  // columns summed here, and columns whose r stays their own
    for (int e = 0; e < NT; ++e)
        for (int c = 0; c < 2; ++c) {
            bool far = false;
            for (int i = 0; i < 2; ++i)
                far |= (abs(exponent(group->inv[i])) > kNear || !(full >> i & 1)) && group->y[e][2 * i + c] != -INFINITY;
            if (__ballot_sync(~0u, far) >> t & 0x11111111u) apart |= 1u << (8 * e + 2 * t + c);
        }
    if (!__any_sync(~0u, apart != 0)) return false;
    for (int e = 0; e < NT; ++e)
        for (int c = 0; c < 2; ++c) {
            const int col = 8 * e + 2 * t + c;
            const bool its = apart >> col & 1;
            const float yA = group->y[e][c], yB = group->y[e][2 + c];
            const float sA = yA - exponent(group->inv[0]), sB = yB - exponent(group->inv[1]);
            const float m = group->m[e][c], v = highest(sA, sB);
            const float n = moved(m, highest(full & 1 ? yA : -INFINITY, full & 2 ? yB : -INFINITY));
            const float from = had >> col & 1 ? pc->base[col] : m, r = its ? moved(from, v) : n;
            float l = group->l[e][c] * ex2(from - r);
            l += its ? ex2(sA - r) + ex2(sB - r)
                     : weight_of<true>(ex2(yA - n), ex2(yB - n), group->inv[0], group->inv[1]);
            for (int i = 0; i < 2; ++i) {
                float &y = group->y[e][2 * i + c];
                if (y == -INFINITY) continue;
                if (!(full >> i & 1)) y = n - 24.0f;
                if (exponent(group->inv[i]) > 126) y = fmaxf(y, n - 24.0f);  // content and an infinity
            }
            if (fabsf(n - r) <= kNear)
                l *= ex2(r - n);
            else
                own |= 1u << col;  // (a NaN too)
            group->l[e][c] = l;
            __syncwarp();  // every lane has read the old r
            if (g == 0) pc->base[col] = r;
        }
    own = __reduce_or_sync(~0u, own);
    if (lane == 0) pc->own = own;
    __syncwarp();
    return true;
}

// Scores of SCORED calls, from z = score * log2 e: capped, and less slope2 * far. In the exp2
// domain a cap b gives b tanh(z / b) = b - 2 b / (1 + 2^(2 log2 e z / b)), off by 2^-21 of b at most (2^-21.5 seen): what
// fp32 scores of the cap's size have. fp32 activations take tanhf, which small scores keep all
// their bits in.
template <bool EXACT>
__device__ __forceinline__ float scored(float z, const PagedAttnArgs &a, float slope2, int far) {
    if (a.cap > 0.0f) {
        const float b = a.cap * kLog2e;
        if (EXACT) {
            z = b * tanhf(z * a.cap_in);
        } else {
            float r;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + ex2(z * a.cap_in)));
            z = fmaf(-2.0f * b, r, b);
        }
    }
    return fmaf(-slope2, static_cast<float>(far), z);
}

// M groups of the run, at kp[0..M-1] in shared memory: scores, weights, O.
// EDGE: not every row of the unit sees the (one) group whole; j0 is its first
// key and pc says what is seen. Rows of V beyond kNear or without content are looked at in edges
// alone. True: the groups have to be taken as such, one by one, and nothing is done; or,
// of an edge, those that follow in the piece, as a column's sum has its own reference.
template <typename C, int M, bool EDGE, bool SCORED>
__device__ __forceinline__ bool step(State<C> &st, uint8_t *const (&kp)[M], const uint8_t *qs,
                                     const uint8_t *bias, const float (&km)[C::NT][2],
                                     volatile Piece *pc, int j0, int sink, int win,
                                     const PagedAttnArgs &a, const volatile float *slopes) {
    constexpr int NB = C::NB, HD = NB * 32, NT = C::NT;
    static_assert(M == 1 || !EDGE, "edges are taken one by one");
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // ---- scores of rows g, g + 8 (y[0..1], y[2..3]) and columns 2 t, 2 t + 1
    float y[M][NT][4];
#pragma unroll
    for (int k = 0; k < M * NT * 4; ++k) y[k / (NT * 4)][k / 4 % NT][k % 4] = 0.0f;
    // codes of rows g, g + 8 and their block scales, 4 blocks (2 of head_dim 64) at
    // a time: with all of a group's at once the registers do not suffice
    constexpr int KB = NB < 4 ? NB : 4;
    uint32_t wA[M][KB], wB[M][KB], sA[M][KB / 2], sB[M][KB / 2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        if (b % KB == 0) {
#pragma unroll
            for (int k = 0; k < M; ++k) {
                if (NB == 2) {
                    const uint4 w = lds_v4(kp[k] + lane * 16);
                    wA[k][0] = w.x; wA[k][1] = w.y; wB[k][0] = w.z; wB[k][1] = w.w;
                } else {
                    const uint4 w = lds_v4(kp[k] + ((b / 4) * 32 + lane) * 16);
                    const uint4 x = lds_v4(kp[k] + (((NB + b) / 4) * 32 + lane) * 16);
                    wA[k][0] = w.x; wA[k][1] = w.y; wA[k][2 % KB] = w.z; wA[k][3 % KB] = w.w;
                    wB[k][0] = x.x; wB[k][1] = x.y; wB[k][2 % KB] = x.z; wB[k][3 % KB] = x.w;
                }
                lds_words<KB / 2>(sA[k], kp[k] + scale_offset(HD) + g * (2 * NB) + 2 * b);
                lds_words<KB / 2>(sB[k], kp[k] + scale_offset(HD) + (g + 8) * (2 * NB) + 2 * b);
            }
        }
        uint4 qf[NT], lo[NT];
        float4 c0[NT];
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            qf[e] = lds_v4(qs + (e * NB + b) * 512 + lane * 16);
            if (C::QSPLIT)
                lo[e] = lds_v4(qs + NT * C::QF + (e * NB + b) * 512 + lane * 16);
            else
                c0[e] = lds_f4(bias + ((e * NB + b) * 4 + t) * 16);
        }
#pragma unroll
        for (int k = 0; k < M; ++k) {
            const uint32_t a = wA[k][b % KB], c = wB[k][b % KB], a8 = a >> 8, c8 = c >> 8;
            const float2 uA = half2_f(sA[k][b % KB / 2]), uB = half2_f(sB[k][b % KB / 2]);
            const float a0 = b & 1 ? uA.y : uA.x, a1 = b & 1 ? uB.y : uB.x;
            uint32_t x[8];
            if (C::QSPLIT) {
                x[0] = minus8_lo(a), x[1] = minus8_lo(c), x[2] = minus8_hi(a), x[3] = minus8_hi(c);
                x[4] = minus8_lo(a8), x[5] = minus8_lo(c8), x[6] = minus8_hi(a8), x[7] = minus8_hi(c8);
            } else {
                x[0] = a & kLo, x[1] = c & kLo, x[2] = a & kHi, x[3] = c & kHi;
                x[4] = a8 & kLo, x[5] = c8 & kLo, x[6] = a8 & kHi, x[7] = c8 & kHi;
            }
#pragma unroll
            for (int e = 0; e < NT; ++e) {
                float d[4];
                if (C::QSPLIT) {  // the low terms first: sums stay small
                    mma0(d, x[0], x[1], x[2], x[3], lo[e].x, lo[e].y);
                    mma(d, x[4], x[5], x[6], x[7], lo[e].z, lo[e].w);
                } else {
                    d[0] = c0[e].x, d[1] = c0[e].y, d[2] = c0[e].z, d[3] = c0[e].w;
                }
                mma(d, x[0], x[1], x[2], x[3], qf[e].x, qf[e].y);
                mma(d, x[4], x[5], x[6], x[7], qf[e].z, qf[e].w);
                y[k][e][0] = fmaf(a0, d[0], y[k][e][0]);
                y[k][e][1] = fmaf(a0, d[1], y[k][e][1]);
                y[k][e][2] = fmaf(a1, d[2], y[k][e][2]);
                y[k][e][3] = fmaf(a1, d[3], y[k][e][3]);
            }
        }
    }
    float iA[M], iB[M];  // 2^-e of V's rows
    int least = 255, most = 0;  // of their biased exponents
#pragma unroll
    for (int k = 0; k < M; ++k) {
        const uint8_t *kf = kp[k] + factor_offset(HD) + 2 * g, *vf = kf + part_bytes(HD);
        const float fA = __uint_as_float(lds_u16(kf) << 16), fB = __uint_as_float(lds_u16(kf + 16) << 16);
        const int xA = lds_u16(vf) >> 7, xB = lds_u16(vf + 16) >> 7;  // biased exponents
        const float eA = static_cast<float>(xA - 127), eB = static_cast<float>(xB - 127);
        iA[k] = __uint_as_float(static_cast<uint32_t>(254 - xA) << 23);
        iB[k] = __uint_as_float(static_cast<uint32_t>(254 - xB) << 23);
        least = min(least, min(xA, xB));
        most = max(most, max(xA, xB));
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            if (SCORED) {
                const int jA = j0 + kGroupRows * k + g;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int p = pc->pos[8 * e + 2 * t + c];
                    const float slope2 = slopes[8 * e + 2 * t + c];
                    y[k][e][c] = scored<C::QSPLIT>(y[k][e][c] * fA * km[e][c], a, slope2, p - jA) + eA;
                    y[k][e][2 + c] = scored<C::QSPLIT>(y[k][e][2 + c] * fB * km[e][c], a, slope2, p - jA - 8) + eB;
                }
                continue;
            }
            y[k][e][0] = fmaf(y[k][e][0] * fA, km[e][0], eA);
            y[k][e][1] = fmaf(y[k][e][1] * fA, km[e][1], eA);
            y[k][e][2] = fmaf(y[k][e][2] * fB, km[e][0], eB);
            y[k][e][3] = fmaf(y[k][e][3] * fB, km[e][1], eB);
        }
    }
    if (EDGE) {
        const int jA = j0 + g, jB = jA + 8;
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            const int p0 = pc->pos[8 * e + 2 * t], p1 = pc->pos[8 * e + 2 * t + 1];
            if (!key_visible(p0, jA, sink, win)) y[0][e][0] = -INFINITY;
            if (!key_visible(p1, jA, sink, win)) y[0][e][1] = -INFINITY;
            if (!key_visible(p0, jB, sink, win)) y[0][e][2] = -INFINITY;
            if (!key_visible(p1, jB, sink, win)) y[0][e][3] = -INFINITY;
        }
    }
    // ---- weights relative to the reference
    float top = kLowest;
#pragma unroll
    for (int k = 0; k < M; ++k)
#pragma unroll
        for (int e = 0; e < NT; ++e)
            top = fmaxf(top, fmaxf(fmaxf(y[k][e][0], y[k][e][2]) - st.m[e][0],
                                   fmaxf(y[k][e][1], y[k][e][3]) - st.m[e][1]));
    bool apart = false;
    // (an edge looks at every row with an infinity: its weight must not become 0)
    const bool looks = EDGE && (most > 253 || pc->own);
    if (__any_sync(~0u, least < kBias - kNear || looks || top > kMost)) {
        auto far_or_zeros = [](int e) { return e == 0 || abs(e) > kNear; };
        bool far = looks;
#pragma unroll
        for (int k = 0; k < M; ++k) far |= far_or_zeros(exponent(iA[k])) || far_or_zeros(exponent(iB[k]));
        if (__any_sync(~0u, far)) {
            if (!EDGE) return true;
            Group<NT> group{{}, {iA[0], iB[0]}};
#pragma unroll
            for (int e = 0; e < NT; ++e) {
#pragma unroll
                for (int i = 0; i < 4; ++i) group.y[e][i] = y[0][e][i];
#pragma unroll
                for (int c = 0; c < 2; ++c) group.m[e][c] = st.m[e][c], group.l[e][c] = st.l[e][c];
            }
            apart = sum_apart<HD>(&group, kp[0], pc);
            if (apart) {
#pragma unroll
                for (int e = 0; e < NT; ++e)
#pragma unroll
                    for (int c = 0; c < 2; ++c) st.l[e][c] = group.l[e][c];
#pragma unroll
                for (int e = 0; e < NT; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[0][e][i] = group.y[e][i];
                iA[0] = iB[0] = 0.0f;  // these weights are in the sums
            }
        }
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            float u0 = y[0][e][0], u1 = y[0][e][1];
#pragma unroll
            for (int k = 0; k < M; ++k) {
                u0 = fmaxf(u0, fmaxf(y[k][e][0], y[k][e][2]));
                u1 = fmaxf(u1, fmaxf(y[k][e][1], y[k][e][3]));
            }
            const float n0 = moved(st.m[e][0], highest(u0, u0)), n1 = moved(st.m[e][1], highest(u1, u1));
            const float c0 = ex2(st.m[e][0] - n0), c1 = ex2(st.m[e][1] - n1);
            st.m[e][0] = n0;
            st.m[e][1] = n1;
            if (!apart) {
                st.l[e][0] *= c0;
                st.l[e][1] *= c1;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    st.o[e][b][i][0] *= c0;
                    st.o[e][b][i][1] *= c1;
                    st.o[e][b][i][2] *= c0;
                    st.o[e][b][i][3] *= c1;
                }
        }
    }
    uint32_t b0[M][NT], b1[M][NT], l0[M][NT], l1[M][NT];
#pragma unroll
    for (int k = 0; k < M; ++k)
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            const float d0 = ex2(y[k][e][0] - st.m[e][0]), d1 = ex2(y[k][e][1] - st.m[e][1]);
            const float d2 = ex2(y[k][e][2] - st.m[e][0]), d3 = ex2(y[k][e][3] - st.m[e][1]);
            st.l[e][0] += weight_of<EDGE>(d0, d2, iA[k], iB[k]);
            st.l[e][1] += weight_of<EDGE>(d1, d3, iA[k], iB[k]);
            const uint32_t hA = pack_half2(d0, d1), hB = pack_half2(d2, d3);
            b0[k][e] = movmatrix_trans(hA);
            b1[k][e] = movmatrix_trans(hB);
            if (C::PSPLIT) {
                const float2 rA = half2_f(hA), rB = half2_f(hB);
                l0[k][e] = movmatrix_trans(pack_half2(d0 - rA.x, d1 - rA.y));
                l1[k][e] = movmatrix_trans(pack_half2(d2 - rB.x, d3 - rB.y));
            }
        }
    // ---- O += V^T P. Groups that are taken together stay together per block where the
    // products go through a fresh accumulator (its sum is added once), else one by one.
    constexpr int MI = C::PSPLIT ? M : 1;
#pragma unroll
    for (int k0 = 0; k0 < M; k0 += MI) {
        uint32_t vw[MI][2 * NB];
        uint4 vs[MI];
#pragma unroll
        for (int k = 0; k < MI; ++k)
#pragma unroll
            for (int c = 0; c < NB / 2; ++c) {
                const uint4 w = lds_v4(kp[k0 + k] + part_bytes(HD) + (c * 32 + lane) * 16);
                vw[k][4 * c] = w.x; vw[k][4 * c + 1] = w.y; vw[k][4 * c + 2] = w.z; vw[k][4 * c + 3] = w.w;
            }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float u[NT][4], v[NT][4];
#pragma unroll
            for (int k = 0; k < MI; ++k) {
                const uint32_t sel = b & 1 ? 0x7632u : 0x5410u;
                const uint32_t x01 = __byte_perm(vw[k][b / 2], vw[k][(NB + b) / 2], sel);
                const uint32_t x23 = __byte_perm(vw[k][(2 * NB + b) / 2], vw[k][(3 * NB + b) / 2], sel);
                const uint32_t z01 = x01 >> 8, z23 = x23 >> 8;
                if (b % 2 == 0)
                    vs[k] = lds_v4(kp[k0 + k] + part_bytes(HD) + scale_offset(HD) + ((b / 2) * 4 + t) * 16);
                const uint32_t s01 = b & 1 ? vs[k].z : vs[k].x, s23 = b & 1 ? vs[k].w : vs[k].y;
                uint32_t w0[NT], w1[NT], v0[NT], v1[NT];
#pragma unroll
                for (int e = 0; e < NT; ++e) {
                    const uint32_t p0 = b0[k0 + k][e], p1 = b1[k0 + k][e];
                    // rows that a query does not see may hold anything, also where another of the
                    // unit sees them: what they give is 0 even if their scales are not finite
                    const uint32_t n0 = EDGE ? not_zero2(p0) : ~0u, n1 = EDGE ? not_zero2(p1) : ~0u;
                    w0[e] = hmul2(p0, s01) & n0;
                    w1[e] = hmul2(p1, s23) & n1;
                    if (C::PSPLIT) {
                        // the product's low term, exact but for the weight's own low term
                        v0[e] = hfma2(l0[k0 + k][e], s01, hfms2(p0, s01, w0[e])) & n0;
                        v1[e] = hfma2(l1[k0 + k][e], s23, hfms2(p1, s23, w1[e])) & n1;
                    }
                }
                uint32_t x[8];
                if (C::PSPLIT) {
                    x[0] = minus8_lo(x01), x[1] = minus8_hi(x01), x[2] = minus8_lo(x23), x[3] = minus8_hi(x23);
                    x[4] = minus8_lo(z01), x[5] = minus8_hi(z01), x[6] = minus8_lo(z23), x[7] = minus8_hi(z23);
                } else {
                    x[0] = x01 & kLo, x[1] = x01 & kHi, x[2] = x23 & kLo, x[3] = x23 & kHi;
                    x[4] = z01 & kLo, x[5] = z01 & kHi, x[6] = z23 & kLo, x[7] = z23 & kHi;
                }
#pragma unroll
                for (int e = 0; e < NT; ++e) {
                    if (C::PSPLIT) {
                        if (k == 0) {
                            mma0(u[e], x[0], x[1], x[2], x[3], v0[e], v1[e]);
                            mma0(v[e], x[4], x[5], x[6], x[7], v0[e], v1[e]);
                        } else {
                            mma(u[e], x[0], x[1], x[2], x[3], v0[e], v1[e]);
                            mma(v[e], x[4], x[5], x[6], x[7], v0[e], v1[e]);
                        }
                        mma(u[e], x[0], x[1], x[2], x[3], w0[e], w1[e]);
                        mma(v[e], x[4], x[5], x[6], x[7], w0[e], w1[e]);
                    } else {
                        mma(st.o[e][b][0], x[0], x[1], x[2], x[3], w0[e], w1[e]);
                        mma(st.o[e][b][1], x[4], x[5], x[6], x[7], w0[e], w1[e]);
                        mma(st.o[e][b][0], kM8a, kM8b, kM8a, kM8b, w0[e], w1[e]);
                        mma(st.o[e][b][1], kM8a, kM8b, kM8a, kM8b, w0[e], w1[e]);
                    }
                }
            }
            if (C::PSPLIT) {
#pragma unroll
                for (int e = 0; e < NT; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        st.o[e][b][0][i] += u[e][i];
                        st.o[e][b][1][i] += v[e][i];
                    }
            }
        }
    }
    return EDGE && apart && pc->own;
}

template <typename T, int HD, int NT, bool SCORED>
__global__ void __launch_bounds__((Cfg<T, HD, NT>::THREADS), 1) paged_attn_kernel(PagedAttnArgs a) {
    using C = Cfg<T, HD, NT>;
    constexpr int ROWS = C::ROWS;
    constexpr int NB = C::NB, S = C::STAGES;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long scan_part[2][C::WARPS + 1];
    __shared__ int start_r[C::WARPS + 1], start_n[C::WARPS + 1];  // the request in which part i
                                                                  // begins, groups of its units
    __shared__ long long start_x[2][C::WARPS + 1];  // and what lies before it (measure, groups)
    __shared__ Piece pieces[C::WARPS];
    __shared__ float slope_of[SCORED ? C::WARPS : 1][ROWS];  // SCORED: of the columns, times log2 e
    __shared__ int abort_flag;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int n_kv = a.pages.n_kv, page_groups = n_kv * a.pages.groups;
    const int log_group = log_group_of(a);
    uint8_t *ring = smem + warp * C::RING;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);  // [warp][stage]
    uint64_t *bars = full + min(warp, C::WARPS - 1) * S;
    volatile uint32_t *dead = reinterpret_cast<uint32_t *>(smem + C::OFF_DEAD);  // groups without rows
    uint8_t *qs = smem + C::OFF_Q + warp * C::QB;
    uint8_t *bias = smem + C::OFF_BIAS + warp * C::BIAS;
    const Ws ws = carve(a.workspace, gridDim.x);

    if (tid < C::WARPS * S) mbar_init(full + tid, 1);
    if (tid == 0) abort_flag = 0;
    if (tid < C::WARPS) pieces[tid].holes = pieces[tid].gone = 0;
    mbar_fence_init();
    __syncthreads();
    // programmatic dependent launch: what came before is done from here on, and
    // the join may be set up while this kernel drains
    wait_for_stream();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the cut: sums over all requests, which the block's threads share, or, where a warp has
    // a lane for each, every warp for itself
    const bool few = a.n_reqs <= kFewReqs;
    const int per = few ? 1 : (a.n_reqs + C::THREADS - 1) / C::THREADS;
    const int r0 = min(a.n_reqs, (few ? lane : tid) * per), r1 = min(a.n_reqs, r0 + per);
    long long work = 0, count = 0;  // measure and groups
    int of_unit = 1;                // groups of a unit of the last request
    bool bad = false;
    for (int r = r0; r < r1; ++r) {
        const Req q = load_req<ROWS>(a, r, log_group);
        of_unit = unit_groups(q);
        const long long units = static_cast<long long>(q.rgs) * n_kv;
        bad |= q.bad;
        work += units * (of_unit + kUnitCost);
        count += units * of_unit;
    }
    if (bad && blockIdx.x == 0) flag_error(a.err, FA_ERRBIT_DEVICE);
    // lengths that contradict each other (overlapping requests) must not wrap the sums: what is
    // cut here is refused below
    work = min(work, 1ll << 41);
    count = min(count, 1ll << 41);
    long long inc = work, inc_g = count;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(~0u, inc, d), p = __shfl_up_sync(~0u, inc_g, d);
        if (lane >= d) inc += o, inc_g += p;
    }
    long long base = 0, base_g = 0, N = 0, all_groups = 0;
    if (few) {
        N = __shfl_sync(~0u, inc, 31);
        all_groups = __shfl_sync(~0u, inc_g, 31);
    } else {
        if (lane == 31) scan_part[0][warp] = inc, scan_part[1][warp] = inc_g;
        __syncthreads();
#pragma unroll
        for (int i = 0; i <= C::WARPS; ++i) {
            if (i == warp) base = N, base_g = all_groups;
            N += scan_part[0][i];
            all_groups += scan_part[1][i];
        }
    }
    if (N >> 30 >= gridDim.x) {  // runs are counted in 31 bits (2^34 rows an SM), and B < 2^11
        if (tid == 0 && blockIdx.x == 0) flag_error(a.err, FA_ERRBIT_DEVICE);
        N = 0;
    }
    const Cut cut = make_cut<C::WARPS>(N, gridDim.x);
    // Where the warp's part of the cut begins (lane 0) and the next one (lane 1); for the copying
    // warp, part i in lane i: request, its unit, group, and the measure and groups before them.
    Place place;
    {
        const long long s = cut.start(blockIdx.x, min(warp == C::WARPS ? lane : warp + (lane & 1), cut.A));
        int r = 0, n = 1;             // the request, groups of its units
        long long x, xg;              // measure and groups before it
        if (few) {
            int j = 0;  // the lane whose request holds s
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                const long long v = __shfl_sync(~0u, inc, j + d - 1);
                if (v <= s) j += d;
            }
            x = __shfl_sync(~0u, inc - work, j);
            xg = __shfl_sync(~0u, inc_g - count, j);
            n = __shfl_sync(~0u, of_unit, j);
            r = j;
        } else {
            // the requests in which the block's parts begin, and the one after them
            x = base + inc - work, xg = base_g + inc_g - count;
            const long long s0 = cut.start(blockIdx.x, 0), s1 = cut.start(blockIdx.x, cut.A);
            if (work > 0 && x <= s1 && x + work > s0) {
                for (int k = r0; k < r1; ++k) {
                    long long m = work, mg = count;
                    if (per > 1) {
                        const Req q = load_req<ROWS>(a, k, log_group);
                        of_unit = unit_groups(q);
                        mg = static_cast<long long>(q.rgs) * n_kv * of_unit;
                        m = mg + static_cast<long long>(q.rgs) * n_kv * kUnitCost;
                    }
                    for (int i = 0; i <= cut.A; ++i) {
                        const long long at = cut.start(blockIdx.x, i);
                        if (x <= at && at < x + m) {
                            start_r[i] = k;
                            start_n[i] = of_unit;
                            start_x[0][i] = x;
                            start_x[1][i] = xg;
                        }
                    }
                    x += m;
                    xg += mg;
                }
            }
            __syncthreads();
            if (s < N) {
                const int i = min(warp == C::WARPS ? lane : warp + (lane & 1), cut.A);
                r = start_r[i], n = start_n[i], x = start_x[0][i], xg = start_x[1][i];
            }
        }
        place.r = -1;
        place.unit = place.gi = place.ahead = 0;
        place.groups = all_groups;
        if (s < N) {
            const long long off = s - x;
            place.r = r;
            place.unit = off < n + kUnitCost ? 0 : static_cast<int>(quotient(off, n + kUnitCost));
            const int at = static_cast<int>(off - static_cast<long long>(place.unit) * (n + kUnitCost));
            place.gi = max(0, at - kUnitCost);
            place.ahead = min(at, kUnitCost);
            place.groups = xg + static_cast<long long>(place.unit) * n + place.gi;
        }
    }

    if (warp == C::WARPS) {
        // ---- the copying warp: lane w walks the run of warp w, up to S tiles ahead of it.
        // (A walk costs a warp registers that it needs for O.) The copy instruction takes
        // one lane at a time, about 140 cycles each: a tile has one where its page has room.
        int left = 0;  // groups to copy
        int r = 0, unit = 0, units = 1, rgs = 1, ci = 0, cn = 1, ns = 0, skip = 0, head = 0;
        bool any = false;
        const int32_t *table = a.pages.table;
        auto enter = [&](const Req &q) {
            cn = unit_groups(q);
            any = q.ng > 0;
            ns = q.ns;
            skip = q.skip;
            rgs = q.rgs;
            units = q.rgs * n_kv;
            table = a.pages.table + static_cast<size_t>(r) * a.pages.max_pages;
        };
        {
            const Place &p = place;
            const long long end = __shfl_down_sync(~0u, p.groups, 1);
            if (lane < cut.A) left = static_cast<int>(end - p.groups);
            if (left > 0) {
                r = p.r;
                enter(load_req<ROWS>(a, r, log_group));
                unit = p.unit;
                ci = p.gi;
                head = unit / rgs * a.pages.groups;
            }
        }
        int page = 0, group = 0, made = 0, stage = 0;
        auto look = [&]() {  // the table entry of the next tile, one step before its copy
            group = ci < ns ? ci : ci + skip;
            page = any ? table[group >> a.pages.group_shift] : -2;
        };
        if (left > 0) look();
        volatile Piece *its = pieces + min(lane, C::WARPS - 1);
        long long t0 = clock64();
        while (__any_sync(~0u, left > 0)) {
            const bool went = left > 0 && made - acquire_s32(&its->gone) < S;
            if (went) {
                const int n = tile_size<C::TILE>(ci, min(cn, ci + left), ns, skip);
                uint32_t holes = 0;
                uint64_t *bar = full + lane * S + stage;
                uint8_t *dst = smem + lane * C::RING + stage * C::STAGE;
                // the tile's pages: one if pages have TILE groups or more, else up to TILE
                for (int k = 0;;) {
                    const int sub = group & (a.pages.groups - 1);
                    const int run = min(n - k, a.pages.groups - sub);
                    if (static_cast<unsigned>(page) < static_cast<unsigned>(a.pages.n_pages)) {
                        mbar_expect_tx(bar, run * C::GB);
                        bulk_copy_g2s(dst + k * C::GB,
                                      a.pages.base + (static_cast<size_t>(page) * page_groups + head + sub) * C::GB,
                                      run * C::GB, bar);
                    } else {  // no rows: rows of no request, or a bad entry of the table
                        holes |= ((1u << run) - 1u) << k;
                        if (page != -2) flag_error(a.err, FA_ERRBIT_DEVICE);
                    }
                    k += run;
                    if (k == n) break;
                    group += run;
                    page = table[group >> a.pages.group_shift];
                }
                dead[lane * S + stage] = holes;
                if (holes) its->holes = 1;
                mbar_arrive(bar);
                if (++stage == S) stage = 0;
                ++made;
                if ((left -= n) > 0) {
                    if ((ci += n) == cn) {
                        ci = 0;
                        if (++unit == units) {
                            unit = 0;
                            Req q;
                            q = next_req<ROWS>(a, &r, log_group);
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
    State<C> st;
    st.clear();
    if (warp < C::WARPS) {
        if (lane == 0) {
            ws.pieces[blockIdx.x * kMostWarps + warp] = 0;
            pc->fin_unit = -1;
            pc->todo = 0;
        }
        __syncwarp();
        if (warp < cut.A) {
            const Place &p = place;
            const long long end = __shfl_down_sync(~0u, p.groups, 1);
            const int ahead = __shfl_down_sync(~0u, p.ahead, 1), gi_end = __shfl_down_sync(~0u, p.gi, 1);
            if (lane == 0) {
                pc->r = p.r;
                pc->unit = p.unit;
                pc->gi = p.gi;
                pc->ahead = gi_end > 0 ? 0 : ahead;
                pc->todo = static_cast<int>(end - p.groups);
            }
        }
        __syncwarp();
        // ---- the run, piece by piece
        int stage = 0, tiles = 0;  // tiles: done
        uint32_t phase = 0;
        bool ok = true;
#pragma unroll 1
        while (pc->todo > 0) {
            int gi = pc->gi, g_end, f0, f1;
            float km[NT][2];
            {
                const Req q = load_req<ROWS>(a, pc->r, log_group);
                const int n = unit_groups(q), unit = pc->unit;
                const int h = unit / q.rgs, rg = unit - h * q.rgs;
                g_end = min(n, gi + pc->todo);
                // ---- q of row g as B fragments: dims 32 b + 8 t + (0,4 | 1,5 | 2,6 | 3,7),
                // the second and fourth times 2^-4; brought to a maximum in [2^10, 2^11)
#pragma unroll 1
                for (int e = 0; e < NT; ++e) {
                    const Col c = column<ROWS>(q, rg, 8 * e + g, h, log_group);
                    const T *src = static_cast<const T *>(a.q) + max(c.token, 0) * a.q_stride +
                                   static_cast<long long>(c.head) * HD + 8 * t;
                    Raw8<T> raw[NB];
#pragma unroll
                    for (int b = 0; b < NB; ++b) raw[b].load(src + 32 * b, c.token >= 0);
                    float top = 0.0f;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        float x[8];
                        raw[b].get(x);
#pragma unroll
                        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
                    }
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                    int up = 0;
                    if (top > 0.0f)
                        up = min(max(137 - static_cast<int>(__float_as_uint(top) >> 23), -96), 126);
                    const float lift = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
                    const float mul = a.scale * kLog2e *
                                      __uint_as_float(static_cast<uint32_t>(127 - up) << 23) *
                                      (C::QSPLIT ? 512.0f : 16777216.0f);  // 2^9, 2^24
                    km[e][0] = __shfl_sync(~0u, mul, 8 * t);
                    km[e][1] = __shfl_sync(~0u, mul, 8 * t + 4);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        float x[8];
                        raw[b].get(x);
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float u = x[i] * lift, v = x[i + 4] * lift;
                            hi[i] = pack_half2(u, v);
                            const float2 f = half2_f(hi[i]);
                            if (!C::QSPLIT && (i & 1)) hi[i] = pack_half2(f.x * 0.0625f, f.y * 0.0625f);
                            lo[i] = pack_half2(u - f.x, v - f.y);
                        }
                        *reinterpret_cast<uint4 *>(qs + (e * NB + b) * 512 + lane * 16) =
                            make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        if (C::QSPLIT) {
                            *reinterpret_cast<uint4 *>(qs + NT * C::QF + (e * NB + b) * 512 + lane * 16) =
                                make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        } else {
                            // -8 times the block's sum, where the accumulators start: "code -8" in every row
                            float d[4];
                            mma0(d, kM8a, kM8a, kM8b, kM8b, hi[0], hi[1]);
                            mma(d, kM8a, kM8a, kM8b, kM8b, hi[2], hi[3]);
                            if (g == 0)
                                *reinterpret_cast<float4 *>(bias + ((e * NB + b) * 4 + t) * 16) =
                                    make_float4(d[0], d[1], d[2], d[3]);
                        }
                    }
                }
                const int p_min = q.rows - q.nq + ((rg * ROWS) >> log_group);
                const int p_max = q.rows - q.nq +
                                  min(q.nq - 1, (rg * ROWS + ROWS - 1) >> log_group);
                if (lane < ROWS) {
                    const Col c = column<ROWS>(q, rg, lane, h, log_group);
                    pc->pos[lane] = c.pos;
                    if (SCORED) slope_of[warp][lane] = a.slopes ? load(a.slopes + c.head) * kLog2e : 0.0f;
                }
                if (lane == 0) {
                    pc->own = 0;
                    pc->n = n;
                    pc->end = g_end;
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
            while (gi < g_end) {
                const int n = tile_size<C::TILE>(gi, g_end, pc->ns, pc->skip);
                uint8_t *kp = ring + stage * C::STAGE;
                if (ok) ok = mbar_wait(bars + stage, phase, &abort_flag, a.err);
                if (ok) {
                    const uint32_t holes = pc->holes ? dead[warp * S + stage] : 0u;
                    bool edges = n < C::TILE || holes || gi < f0 || gi + n > f1;
                    if (!edges) {
                        uint8_t *tile[C::TILE];
#pragma unroll
                        for (int k = 0; k < C::TILE; ++k) tile[k] = kp + k * C::GB;
                        const int j0 = SCORED ? (gi < pc->ns ? gi : gi + pc->skip) * kGroupRows : 0;
                        edges = step<C, C::TILE, false, SCORED>(st, tile, qs, bias, km, pc, j0, a.sink, a.win, a,
                                                                slope_of[SCORED ? warp : 0]);
                    }
                    if (edges) {
#pragma unroll 1
                        for (int k = 0; k < n; ++k) {
                            if (holes >> k & 1) continue;
                            const int i = gi + k;
                            uint8_t *const one[1] = {kp + k * C::GB};
                            if (step<C, 1, true, SCORED>(st, one, qs, bias, km, pc,
                                                         (i < pc->ns ? i : i + pc->skip) * kGroupRows, a.sink,
                                                         a.win, a, slope_of[SCORED ? warp : 0]))
                                f1 = INT_MIN;
                        }
                    }
                }
                __syncwarp();  // every lane has read the stage
                gi += n;
                ++tiles;
                if (lane == 0) release_s32(&pc->gone, tiles);
                if (++stage == S) stage = 0, phase ^= 1;
            }

            // ---- the piece is done
            st.sum_lanes();
            if (pc->own) st.join_references(pc->own, pc->base);
            const int r = pc->r, unit = pc->unit, n = pc->n, first = pc->gi, end = pc->end;
            const int todo = pc->todo - (end - first);
            if (first == 0 && end == n) {
                const Req q = load_req<ROWS>(a, r, log_group);
                const int h = unit / q.rgs, rg = unit - h * q.rgs;
#pragma unroll
                for (int e = 0; e < NT; ++e)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const Col col = column<ROWS>(q, rg, 8 * e + 2 * t + c, h, log_group);
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            write_row<T>(a, col, HD, 32 * b + 4 * g, st.quad(e, b, c), st.m[e][c], st.l[e][c]);
                    }
            } else {
                // the start of the run: to the workspace; its end: into the ring, whose copies
                // have all been used
                const bool start = todo > 0;
                float *dst = ws.partial +
                             (static_cast<size_t>(blockIdx.x * cut.A + warp) * 2 + 1) * C::PARTIAL;
                if (g == 0) {
#pragma unroll
                    for (int e = 0; e < NT; ++e)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int i = 8 * e + 2 * t + c;
                            if (start) {
                                dst[i] = st.m[e][c];
                                dst[ROWS + i] = st.l[e][c];
                            } else {
                                pc->m[i] = st.m[e][c];
                                pc->l[i] = st.l[e][c];
                            }
                        }
                }
                float4 *quads = start ? reinterpret_cast<float4 *>(dst + 2 * ROWS)
                                      : reinterpret_cast<float4 *>(ring);
#pragma unroll
                for (int e = 0; e < NT; ++e)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            quads[st.quad_at(e, b, c) * 32 + lane] = st.quad(e, b, c);
            }
            __syncwarp();
            if (lane == 0) {
                if (todo > 0) {
                    const Req q = load_req<ROWS>(a, r, log_group);
                    int next = unit + 1, nr = r;
                    if (next == q.rgs * n_kv) {
                        next = 0;
                        next_req<ROWS>(a, &nr, log_group);
                    }
                    pc->r = nr;
                    pc->unit = next;
                    pc->gi = 0;
                } else if (first > 0 || end < n) {
                    const long long x1 = cut.start(blockIdx.x, warp + 1) - pc->ahead;
                    pc->fin_r = r;
                    pc->fin_unit = unit;
                    pc->fin_first = x1 - end;
                    pc->fin_last = x1 - end + n;
                }
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
    // warps [w0, w1) hold pieces of this unit: neighbours, as runs follow each other
    const unsigned same = __ballot_sync(~0u, lane < C::WARPS && pieces[min(lane, C::WARPS - 1)].fin_unit == unit &&
                                                 pieces[min(lane, C::WARPS - 1)].fin_r == r);
    const int w0 = __ffs(same) - 1, w1 = 32 - __clz(same);
    // The unit's end may be what the next warp began its run with: in the workspace, and joined
    // here too, if that warp is the block's (whose last parts may be empty; TAILS).
    const bool from_start = cut.start(blockIdx.x, w0) <= first, more = cut.start(blockIdx.x, w1) < last;
    const bool tail_here = C::TAILS && more && w1 < cut.A && cut.start(blockIdx.x, w1 + 1) > cut.start(blockIdx.x, w1);
    const bool direct = from_start && (tail_here || !more);
    const Req q = load_req<ROWS>(a, r, log_group);
    const int h = unit / q.rgs, rg = unit - h * q.rgs;
    float *dst = ws.partial + static_cast<size_t>(blockIdx.x * cut.A + w0) * 2 * C::PARTIAL;
    const float *tail = ws.partial + (static_cast<size_t>(blockIdx.x * cut.A + w1) * 2 + 1) * C::PARTIAL;
    if (from_start && !direct && warp == w0 && lane == 0) {
        const int e = cut.warp_of(last - 1);  // the warp that holds the unit's last group
        // its run goes on, and its block does not join what it began with: a piece for the join
        const bool alone = (!C::TAILS || e % cut.A == 0) && cut.start(e / cut.A, e % cut.A + 1) > last + kUnitCost;
        ws.pieces[blockIdx.x * kMostWarps + warp] =
            pack_pieces((alone ? e - 1 : e) / cut.A - static_cast<int>(blockIdx.x) + 1, cut.A, alone ? e : -1);
        ws.tasks[blockIdx.x * kMostWarps + warp] = Task{h, rg, q};
    }
    // Factors of the pieces, one lane for each column and every (32 / ROWS)-th piece, into the
    // memory of q: factor[piece][column], the tail's after the others, and then M and L.
    float *factor = reinterpret_cast<float *>(qs);
    static_assert((C::WARPS + 3) * ROWS * 4 <= C::QB, "the factors fit the memory of q");
    const int n_pieces = w1 - w0 + (tail_here ? 1 : 0);
    {
        constexpr int STEP = 32 / ROWS;
        const int n = lane % ROWS;
        auto m_of = [&](int k) { return k < w1 - w0 ? pieces[w0 + k].m[n] : tail[n]; };
        float M = kLowest, L = 0.0f;
        for (int k = lane / ROWS; k < n_pieces; k += STEP) M = fmaxf(M, m_of(k));
#pragma unroll
        for (int d = ROWS; d < 32; d <<= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, d));
        for (int k = lane / ROWS; k < n_pieces; k += STEP) {
            const float f = ex2(m_of(k) - M);
            factor[k * ROWS + n] = f;
            L = fmaf(k < w1 - w0 ? pieces[w0 + k].l[n] : tail[ROWS + n], f, L);
        }
#pragma unroll
        for (int d = ROWS; d < 32; d <<= 1) L += __shfl_xor_sync(~0u, L, d);
        if (lane < ROWS) {
            factor[(C::WARPS + 1) * ROWS + n] = M;
            factor[(C::WARPS + 2) * ROWS + n] = L;
            if (!direct && warp == w0) {
                dst[n] = M;
                dst[ROWS + n] = L;
            }
        }
        __syncwarp();
    }
    for (int i = warp - w0; i < 2 * NB * NT; i += w1 - w0) {  // (eight, block, column) triples
        const int n = 8 * (i / (2 * NB)) + 2 * t + (i & 1), b = (i >> 1) % NB, at = i * 32 + lane;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (tail_here)
            x = scaled(*(reinterpret_cast<const float4 *>(tail + 2 * ROWS) + at), factor[(w1 - w0) * ROWS + n]);
#pragma unroll 4
        for (int w = w0; w < w1; ++w) {
            const float4 y = *(reinterpret_cast<const float4 *>(smem + w * C::RING) + at);
            const float k = factor[(w - w0) * ROWS + n];
            x.x = fmaf(y.x, k, x.x);
            x.y = fmaf(y.y, k, x.y);
            x.z = fmaf(y.z, k, x.z);
            x.w = fmaf(y.w, k, x.w);
        }
        if (direct)
            write_row<T>(a, column<ROWS>(q, rg, n, h, log_group), HD, 32 * b + 4 * g, x,
                         factor[(C::WARPS + 1) * ROWS + n], factor[(C::WARPS + 2) * ROWS + n]);
        else
            *(reinterpret_cast<float4 *>(dst + 2 * ROWS) + at) = x;
    }
}

// The units that no block of the first kernel could finish, each as items (block
// of 32 dims, column half) that are shared out over all blocks, one a warp. Where
// a block gets fewer items than it has warps, several take slices of an item's
// pieces: a long request in a small batch is in many. When a block took the units
// that begin in its own runs, one request of 70000 rows (152 pieces) took 29 us
// instead of 17, 128 windowed requests of all lengths 24 instead of 21, and 32
// equal ones, where there is nothing to even out, 20.5 instead of 21.9. The pieces
// of a slice are added in ascending order, and so are the slices.
constexpr int kJoinThreads = 512, kJoinWarps = kJoinThreads / 32;
template <typename T, int HD, int NT>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(PagedAttnArgs a) {
    using C = Cfg<T, HD, NT>;
    constexpr int ITEMS = 2 * C::NB * NT, BATCH = 8;
    __shared__ int counts[kJoinWarps];
    constexpr int MOST = kMostBlocks * kMostWarps;
    __shared__ uint32_t list[MOST], where[MOST];  // tasks: their words, and whose they are
    static_assert(kMostBlocks <= kJoinThreads && kMostBlocks < 512 && kMostBlocks * kMostWarps < 8191 &&
                      kMostWarps < 32 && kMostWarps % 4 == 0,
                  "a thread reads a block's words, whose fields hold these");
    __shared__ float4 part_o[kJoinWarps][32];
    __shared__ float part_m[kJoinWarps][4], part_l[kJoinWarps][4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    wait_for_stream();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Ws ws = carve(a.workspace, gridDim.x);
    // the tasks, in order of the warps
    unsigned has = 0;
    uint32_t words[kMostWarps];
    if (threadIdx.x < gridDim.x) {
        const uint4 *src = reinterpret_cast<const uint4 *>(ws.pieces + threadIdx.x * kMostWarps);
#pragma unroll
        for (int i = 0; i < kMostWarps / 4; ++i) {
            const uint4 f = src[i];
            words[4 * i] = f.x; words[4 * i + 1] = f.y; words[4 * i + 2] = f.z; words[4 * i + 3] = f.w;
        }
#pragma unroll
        for (int i = 0; i < C::WARPS; ++i) has |= (words[i] ? 1u : 0u) << i;
    }
    int before = __popc(has);  // inclusive, then exclusive
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(~0u, before, d);
        if (lane >= d) before += o;
    }
    if (lane == 31) counts[warp] = before;
    __syncthreads();
    const int of_warp = lane < kJoinWarps ? counts[lane] : 0;
    const int n_tasks = __reduce_add_sync(~0u, of_warp);
    before += __reduce_add_sync(~0u, lane < warp ? of_warp : 0) - __popc(has);
#pragma unroll
    for (int i = 0; i < C::WARPS; ++i)
        if (has >> i & 1) {
            where[before] = threadIdx.x * kMostWarps + i;
            list[before++] = words[i];
        }
    __syncthreads();
    if (n_tasks == 0) return;
    const int items = n_tasks * ITEMS;
    const int mine = (items + gridDim.x - 1) / gridDim.x;
    const int j0 = blockIdx.x * mine, j1 = min(items, j0 + mine);
    // slices of an item: the largest power of two with slices * mine <= kJoinWarps, or 1
    const int log_slices = mine <= 1 ? 4 : mine <= 2 ? 3 : mine <= 4 ? 2 : mine <= 8 ? 1 : 0;
    static_assert(kJoinWarps == 16, "log_slices");
    const int slices = 1 << log_slices, at_once = kJoinWarps >> log_slices, slice = warp & (slices - 1);
    for (int jb = j0; jb < j1; jb += at_once) {  // the same turns for every warp of the block
        const int j = jb + (warp >> log_slices);
        const bool in = j < j1;
        const int nth = static_cast<unsigned>(in ? j : jb) / ITEMS;
        const uint32_t id = where[nth], word = list[nth];
        const int i = (in ? j : jb) & (ITEMS - 1), b = (i >> 1) % C::NB;
        const int n = 8 * (i / (2 * C::NB)) + 2 * t + (i & 1);  // i = quad_at of the item
        const Task k = ws.tasks[id];
        const int block = id / kMostWarps, blocks = word & 511u, warps = word >> 9 & 31u;
        const int tail = static_cast<int>(word >> 14) - 1, pieces = blocks + (tail >= 0);
        // this slice's pieces
        const int e0 = pieces * slice >> log_slices, e1 = pieces * (slice + 1) >> log_slices;
        auto piece = [&](int e) {
            const int slot = e == 0       ? (block * warps + static_cast<int>(id % kMostWarps)) * 2
                             : e < blocks ? (block + e) * warps * 2
                                          : tail * 2 + 1;
            return ws.partial + static_cast<size_t>(slot) * C::PARTIAL;
        };
        float M = kLowest, L = 0.0f;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int eb = e0; in && eb < e1; eb += BATCH) {
            float m[BATCH], l[BATCH];
            float4 y[BATCH];
#pragma unroll
            for (int e = 0; e < BATCH; ++e) {
                const float *p = piece(min(eb + e, e1 - 1));
                m[e] = p[n];
                l[e] = p[C::ROWS + n];
                y[e] = *reinterpret_cast<const float4 *>(p + 2 * C::ROWS + (i * 32 + lane) * 4);
            }
            float top = M;
#pragma unroll
            for (int e = 0; e < BATCH; ++e) top = fmaxf(top, m[e]);
            const float s = ex2(M - top);
            M = top;
            L *= s;
            x = scaled(x, s);
#pragma unroll
            for (int e = 0; e < BATCH; ++e) {
                if (eb + e >= e1) continue;
                const float f = ex2(m[e] - top);
                L = fmaf(l[e], f, L);
                x.x = fmaf(y[e].x, f, x.x);
                x.y = fmaf(y[e].y, f, x.y);
                x.z = fmaf(y[e].z, f, x.z);
                x.w = fmaf(y[e].w, f, x.w);
            }
        }
        if (slices > 1) {
            __syncthreads();  // the turn before has been read
            part_o[warp][lane] = x;
            if (g == 0) {
                part_m[warp][t] = M;
                part_l[warp][t] = L;
            }
            __syncthreads();
            if (slice == 0) {
                for (int s = 1; s < slices; ++s) {
                    const float m = part_m[warp + s][t], top = fmaxf(M, m);
                    const float f0 = ex2(M - top), f1 = ex2(m - top);
                    const float4 y = part_o[warp + s][lane];
                    M = top;
                    L = fmaf(part_l[warp + s][t], f1, L * f0);
                    x = make_float4(fmaf(y.x, f1, x.x * f0), fmaf(y.y, f1, x.y * f0),
                                    fmaf(y.z, f1, x.z * f0), fmaf(y.w, f1, x.w * f0));
                }
            }
        }
        if (in && slice == 0)
            write_row<T>(a, column<C::ROWS>(k.q, k.rg, n, k.h, log_group_of(a)), HD, 32 * b + 4 * g, x, M, L);
    }
}

template <typename T, int HD, int NT, bool SCORED>
cudaError_t launch(const PagedAttnArgs &a, cudaStream_t stream) {
    using C = Cfg<T, HD, NT>;
    // once for each device, as the call takes a microsecond; two threads that are first may both
    // make it
    static std::atomic<uint64_t> made{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !(made.load(std::memory_order_acquire) >> dev & 1))) {
        e = cudaFuncSetAttribute(paged_attn_kernel<T, HD, NT, SCORED>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e == cudaSuccess && dev < 64) made.fetch_or(1ull << dev, std::memory_order_release);
    }
    const int blocks = std::min(device_sm_count(), kMostBlocks);
    if (e == cudaSuccess)
        e = launch_after(paged_attn_kernel<T, HD, NT, SCORED>, blocks, C::THREADS, C::SMEM, stream, a);
    if (e == cudaSuccess)
        e = launch_after(paged_join_kernel<T, HD, NT>, blocks, kJoinThreads, 0, stream, a);
    return e;
}

// Where 16 or more q heads share a kv head a unit is 16 rows: its codes become
// operands once for both eights (32 x 16384 rows of 2 kv heads, bf16: head_dim 128
// 64.2 us with 8 rows, 58.5 with 16; head_dim 64 42.5 and 39.0; fp16 76.5 and 72.0,
// 48.5 and 44.5). With fewer heads 16 rows may be half empty, which costs more than
// full ones save (8 heads, bf16: 113 us with 8 rows, 176 with 16). For fp32 the
// saving went to the registers (batches of all lengths: 111 us with 8 rows, 115 with
// 16), and with head_dim 256 O would take all of them.
template <typename T, int HD, bool SCORED>
cudaError_t launch_rows(const PagedAttnArgs &a, cudaStream_t stream) {
    if constexpr (HD < 256 && sizeof(T) == 2) {
        if (a.n_q_heads / a.pages.n_kv >= 16) return launch<T, HD, 2, SCORED>(a, stream);
    }
    return launch<T, HD, 1, SCORED>(a, stream);
}

template <typename T, bool SCORED>
cudaError_t launch_type(const PagedAttnArgs &a, int hd, cudaStream_t stream) {
    return hd == 64    ? launch_rows<T, 64, SCORED>(a, stream)
           : hd == 128 ? launch_rows<T, 128, SCORED>(a, stream)
                       : launch_rows<T, 256, SCORED>(a, stream);
}

template <bool SCORED>
cudaError_t launch_paged(const PagedAttnArgs &a, int dtype, int hd, cudaStream_t stream) {
    switch (dtype) {
        case kTypeF32: return launch_type<float, SCORED>(a, hd, stream);
        case kTypeF16: return launch_type<__half, SCORED>(a, hd, stream);
        default: return launch_type<__nv_bfloat16, SCORED>(a, hd, stream);
    }
}

}  // namespace
}  // namespace fa
