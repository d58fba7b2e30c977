// packed_common.cuh -- what the kernels of packed attention and of its gradient
// share: the batch, the tiles of its documents, the attended set and the scores
// (include/fa.h, fa_packed_attn).
//
// Rows. The q heads of one kv head are rows of one matrix: row i * G + h is
// token i of the document and head h of the group of G, so that a tile of 128
// rows holds 128 / G tokens of all G heads. A unit's rows then share their keys
// whatever the group is, the gradients of K and V sum over the group inside the
// products, and a short document fills its tiles G times better than head by head.
#pragma once

#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "fa_device.cuh"
#include "fa_internal.h"
#include "paged_launch.cuh"

namespace fa {

constexpr float kPackedLog2e = 1.4426950408889634f;
constexpr float kPackedLn2 = 0.69314718055994531f;

// A tile of a document, of its rows or of its keys. (Whole vectors: in words, a warp's tiles, which go to as many
// places, took the plan half of its time: 8192 tokens in 23 documents, 16/2 heads x 256 capped, 76 -> 73 us with it.)
struct alignas(16) PackedTile {
    int tok0, len;   // the document's first token in the batch, and its tokens
    int p0;          // position of the tile's first token
    int prefix;      // keys that every query of the document sees
    int rb;          // 128-row blocks of the documents before this one
    int doc;
    int head;        // kv head (set by the kernel that takes the unit)
    // Tiles of keys: the row tiles of this piece, [from, from + rows), the pieces of the tile, and
    // where their partial sums go (piece 0 of kv head 0; -1: there is one piece).
    int from, rows, piece, pieces, slot;
};
static_assert(sizeof(PackedTile) == 48, "three 16-byte loads");

// Key tiles of BK that the queries at positions p0 .. p1 see any key of, in
// ascending order: those of the prefix and the sinks, then the window's (or all).
struct KeyTiles {
    int ns, lo, count;
    __device__ __forceinline__ int at(int i) const { return i < ns ? i : lo + (i - ns); }
};
template <int BK>
__device__ __forceinline__ KeyTiles key_tiles(int p0, int p1, int prefix, int sink, int win) {
    KeyTiles t;
    const int head = max(prefix, win > 0 ? min(sink, p1 + 1) : 0);
    t.ns = (head + BK - 1) / BK;
    t.lo = max(win > 0 ? max(0, p0 - win + 1) / BK : 0, t.ns);
    t.count = t.ns + max(0, p1 / BK - t.lo + 1);
    return t;
}
// Every query in [p0, p1] sees every key in [j0, j1] (j0 > j1 or queries past the end: never mind).
__device__ __forceinline__ bool sees_all(int p0, int p1, int j0, int j1, int prefix, int sink, int win) {
    if (j1 < prefix) return true;
    return j1 <= p0 && (win <= 0 || j1 < sink || j0 > p1 - win);
}

// Queries that see any key of [j0, j1], one run of positions: [first, last].
__device__ __forceinline__ void query_range(int j0, int j1, int len, int prefix, int sink, int win,
                                            int *first, int *last) {
    *first = j0 < prefix ? 0 : j0;
    *last = win <= 0 || j0 < max(prefix, sink) ? len - 1 : min(len - 1, j1 + win - 1);
}

// A batch of a few documents whose units have a block each needs no plan: a warp finds the x-th tile from
// the documents' lengths, a document a lane. (One launch less: 3 documents of 203 tokens 12.9 -> 8.5 us.)
constexpr int kDirectDocs = 32;
struct PackedDirect {
    const int32_t *cu, *prefix;  // cu null: there is a plan
    int n_docs, n_tokens;
};
// All lanes of a warp. KEYS: tiles of 128 keys, else of tile_tokens tokens; step_tokens of the row tiles that
// move past keys; block_log: log2 of the tokens of 128 rows. The number of tiles.
template <bool KEYS>
__device__ __forceinline__ int direct_tile(const PackedDirect &b, int x, int tile_tokens, int step_tokens, int block_log,
                                           int sink, int win, unsigned *err, PackedTile *u) {
    const int lane = threadIdx.x & 31;
    const bool mine = lane < b.n_docs;
    const int from = mine ? load(b.cu + lane) : 0, to = mine ? load(b.cu + lane + 1) : 0;
    const bool bad = mine && (from < 0 || to < from || to > b.n_tokens);
    const int prefix = mine && b.prefix ? load(b.prefix + lane) : 0;
    if (__any_sync(~0u, bad)) {
        if (lane == 0) flag_error(err, FA_ERRBIT_DEVICE);
        return 0;
    }
    const int len = to - from;
    const int tiles = KEYS ? (len + 127) / 128 : (len + tile_tokens - 1) / tile_tokens;
    const int blocks = (len + (1 << block_log) - 1) >> block_log;
    int upto = tiles, rb = blocks;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(~0u, upto, d), p = __shfl_up_sync(~0u, rb, d);
        if (lane >= d) upto += o, rb += p;
    }
    const int n = __shfl_sync(~0u, upto, 31);
    if (x >= n) return n;
    const int doc = __ffs(__ballot_sync(~0u, upto > x)) - 1;
    u->tok0 = __shfl_sync(~0u, from, doc);
    u->len = __shfl_sync(~0u, len, doc);
    u->p0 = (x - __shfl_sync(~0u, upto - tiles, doc)) * (KEYS ? 128 : tile_tokens);
    u->prefix = min(max(__shfl_sync(~0u, prefix, doc), 0), u->len);
    u->rb = __shfl_sync(~0u, rb - blocks, doc);
    u->doc = doc;
    u->head = u->from = u->rows = u->piece = 0;
    u->pieces = 1;
    u->slot = -1;
    if (KEYS) {
        int first, last;
        query_range(u->p0, min(u->p0 + 128, u->len) - 1, u->len, u->prefix, sink, win, &first, &last);
        u->from = first / step_tokens;
        u->rows = last / step_tokens - u->from + 1;
    }
    return n;
}

// Two fp32 values in a pair of registers: one instruction for both. The pipes take as long as for two,
// but the issue slots that this leaves are what the warp that feeds the tensor cores lives on.
struct Two {
    uint64_t v;
};
__device__ __forceinline__ Two two(float x, float y) {
    Two t;
    asm("mov.b64 %0, {%1, %2};" : "=l"(t.v) : "f"(x), "f"(y));
    return t;
}
__device__ __forceinline__ Two two(float x) { return two(x, x); }
__device__ __forceinline__ float2 both(Two t) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(t.v));
    return f;
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
    Two t;
    asm("add.rn.ftz.f32x2 %0, %1, %2;" : "=l"(t.v) : "l"(a.v), "l"(b.v));
    return t;
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
    Two t;
    asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(t.v) : "l"(a.v), "l"(b.v));
    return t;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two t;
    asm("fma.rn.ftz.f32x2 %0, %1, %2, %3;" : "=l"(t.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return t;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The score in the exp2 domain from the product s of q and k.
//   no cap: s * a          (a = scale * log2 e)
//   cap:    b * tanh(..)   = b - 2 b r, r = 1 / (1 + 2^(s * a)),  a = 2 scale log2 e / cap, b = cap log2 e
// off by 2^-21 of b at most (2^-21.01 is the most seen: 11 caps from 0.37 to 4096, 5 scales, 2^21 scores, 11 neighbours
// in cap_r), as fp32 scores of the cap's size are.
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
struct ScoreRule {
    float a, b;
};
inline ScoreRule score_rule(float scale, float cap) {
    ScoreRule r;
    r.a = cap > 0.0f ? 2.0f * scale * kPackedLog2e / cap : scale * kPackedLog2e;
    r.b = cap > 0.0f ? cap * kPackedLog2e : 0.0f;
    return r;
}
__device__ __forceinline__ float min_nan(float x, float y) {  // NaN if either is one
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(x), "f"(y));
    return d;
}
// r of two scores. Their reciprocals from that of the product, as a reciprocal costs the special units
// what two exponentials do; 2^63 is where tanh has long been 1. A NaN in one makes both NaN, so that
// both have to be the document's own (or 0), even where one of them is masked afterwards.
__device__ __forceinline__ Two cap_r(Two s, const ScoreRule &c) {
    const float2 z = both(s * two(c.a));
    const Two p = two(ex2(min_nan(z.x, 63.0f)), ex2(min_nan(z.y, 63.0f))) + two(1.0f);
    const float2 q = both(p);
    return two(q.y, q.x) * two(rcp_approx(q.x * q.y));
}
__device__ __forceinline__ Two capped(Two r, const ScoreRule &c) { return fma2(r, two(-2.0f * c.b), two(c.b)); }
// A quarter of the derivative of cap * tanh(x / cap): (1 - tanh^2) / 4 = r (1 - r).
__device__ __forceinline__ Two cap_slope(Two r) { return r * fma2(r, two(-1.0f), two(1.0f)); }

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    return pack_half2(lo, hi);
}
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// 16 values of a row as two 16-byte stores, or one of 32 bytes where rows allow it: threads hold a row each, and
// a store that fills a 32-byte sector is worth two that fill half of one.
__device__ __forceinline__ void store16(uint16_t *p, const uint32_t *w, bool wide) {
    if (wide)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    else
#pragma unroll
        for (int k = 0; k < 8; k += 4)
            *reinterpret_cast<uint4 *>(p + 2 * k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
}
__device__ __forceinline__ bool wide_rows(const void *p, long long stride) {
    return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(stride) * 2) & 31) == 0;
}

// The shared memory that a kernel may have, set once for each device, as the call takes a microsecond (two threads that
// are first may both make it).
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, size_t bytes, std::atomic<uint64_t> *made) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !(made->load(std::memory_order_acquire) >> dev & 1))) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
        if (e == cudaSuccess && dev < 64) made->fetch_or(1ull << dev, std::memory_order_release);
    }
    return e;
}

// Instruction descriptor with both operands fp16 or both bf16.
template <bool BF16>
__host__ __device__ constexpr uint32_t idesc_16(int M, int N, int a_mn_major, int b_mn_major) {
    return idesc_f16(M, N, a_mn_major, b_mn_major) | (BF16 ? (1u << 7) | (1u << 10) : 0u);
}

// One arrival for a warp, behind what all of its lanes did. (An arrival of every thread costs the
// shared memory's atomics more than the products they announce.)
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// N columns of this thread's lane of TMEM.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t col, uint32_t *r) {
    if constexpr (N == 16) tmem_ld16(col, r);
    else
#pragma unroll
        for (int i = 0; i < N; i += 32) tmem_ld32(col + i, r + i);
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t col, const uint32_t *r) {
    if constexpr (N == 8) tmem_st8(col, r);
    else if constexpr (N == 16) tmem_st16(col, r);
    else
#pragma unroll
        for (int i = 0; i < N; i += 32) tmem_st32(col + i, r + i);
}

// Products are issued by a warp whose lanes all walk the same loop, so that descriptors live in uniform
// registers, with one lane that issues. (A single lane in a branch of its own, with the descriptors
// computed in its registers, took 100 cycles a product instead of the 64 that the tensor cores take.)
__device__ __forceinline__ bool elect_lane() {
    uint32_t yes;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(yes));
    return yes != 0;
}
// A value that all lanes share, known as such to the compiler.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(~0u, x); }
__device__ __forceinline__ bool uniform(bool x) { return __all_sync(~0u, x); }

// Registers of this warp's threads from here on: all four warps of a warpgroup, and in sum at most what
// the block was launched with.
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Wait ignoring the abort flag (still bounded): lets copies and MMAs in flight
// finish before a block that gave up releases its TMEM and exits.
__device__ __forceinline__ void wait_out(uint64_t *bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > kSpinCycles) return;
}

// A barrier of copies whose arrivals are counted, so that a block that gives up
// knows which copies it has to wait out.
struct Arms {
    int n = 0;
    __device__ __forceinline__ void drain(uint64_t *bar) const {
        if (n) wait_out(bar, (n - 1) & 1);
    }
};

// Rows [from, rows) of a tile of `chunks` 128-byte-wide pieces become zeros (the
// swizzle keeps a row's 128 bytes together). All lanes of the warp.
__device__ __forceinline__ void zero_rows(uint8_t *tile, int chunks, int chunk_bytes, int from, int rows) {
    const int lane = threadIdx.x & 31;
    for (int c = 0; c < chunks; ++c)
        for (int at = from * 128 + lane * 16; at < rows * 128; at += 512)
            *reinterpret_cast<uint4 *>(tile + c * chunk_bytes + at) = make_uint4(0, 0, 0, 0);
}

// Units of a persistent kernel: block b starts with unit b, later ones come from
// a counter; the producer warp hands them on through a ring in shared memory.
constexpr int kPackedRing = 4;
struct UnitRing {
    uint64_t full[kPackedRing], empty[kPackedRing];
    PackedTile unit[kPackedRing];  // head < 0: no more
};

// ---- packed_plan.cu
// What the plan leaves in the workspace: counts, the work counters (zeroed) and
// the tiles, heaviest first.
struct PackedHeader {
    int row_tiles, key_tiles;  // in the lists
    unsigned counters[4];
    int pad[58];
};
static_assert(sizeof(PackedHeader) == 256, "header");

struct PackedPlanArgs {
    const int32_t *cu, *prefix;
    int n_docs, n_tokens, sink, win;
    int row_tokens;       // tokens of a row tile
    int block_tokens_log; // log2 of the tokens of 128 rows
    int key_tile;         // keys of a row tile's key tiles, for the weights
    int step_tokens;      // tokens of the row tiles that move past a tile of keys
    int n_kv, parts;      // a key tile's row tiles are cut into pieces of about 1 / parts of the work
    int most_rows, most_keys;  // room in the lists (most_keys 0: no key tiles)
    int slots;            // partial sums that there is room for
    int *arrived;         // [slots], zeroed
    PackedHeader *header;
    PackedTile *rows, *keys;
    int *doc_tiles;       // [lists][3][n_docs + 1]: row tiles, key tiles and 128-row blocks before each document
    unsigned *doc_most;   // [2][n_docs], zeroed, or null
    unsigned *err;
};
cudaError_t launch_packed_plan(const PackedPlanArgs &a, cudaStream_t stream);

// ---- packed_fwd.cuh
struct PackedFwdArgs {
    CUtensorMap q, k, v, o;  // o: boxes of 32 rows
    PackedDirect direct;
    const PackedHeader *header;
    const PackedTile *rows;
    unsigned *counter;
    void *out;
    long long out_stride;
    float *lse;           // [n_q_heads][n_tokens] or null
    const float *slopes;  // [n_q_heads] or null
    int n_tokens, n_kv, log_group, sink, win;
    ScoreRule score;
    unsigned *err;
};
cudaError_t launch_packed_fwd_bf16(const PackedFwdArgs &a, int hd, bool cap, int blocks, cudaStream_t stream);
cudaError_t launch_packed_fwd_f16(const PackedFwdArgs &a, int hd, bool cap, int blocks, cudaStream_t stream);
// Row tiles of 128 that a block of the forward kernel works on at once.
constexpr int packed_fwd_tiles(int hd) { return hd == 256 ? 1 : 2; }

// ---- packed_stats.cu
// What the gradient needs of each row: L, less its log-sum-exp in the exp2 domain (plus
// kGradShift for binary16), and D = -dout . out; and of each document, for binary16,
// the largest row of dout and of V.
struct PackedStatsArgs {
    PackedDirect direct;
    int sink, win;
    unsigned *err;
    const PackedHeader *header;
    const PackedTile *rows;  // tiles of 128 rows
    const void *out, *dout, *v;
    long long out_stride, dout_stride, v_stride;
    const float *lse;
    int n_tokens, n_kv, log_group, n_docs;
    long long blocks;        // 128-row blocks of a kv head
    float *L, *D;            // [n_kv][blocks][128]
    // Bits of the largest |dout row|^2 and |v row|^2: [2][n_docs], of documents; without a plan, which zeroes
    // them, [2][n_kv][blocks], of 128-row blocks.
    unsigned *doc_most;
};
cudaError_t launch_packed_stats(const PackedStatsArgs &a, int dtype, int hd, int blocks, cudaStream_t stream);
constexpr float kGradShift = 14.0f;

// ---- packed_bwd.cuh
struct PackedGradArgs {
    // Stationary tiles x1, x2 and moving ones y1, y2: q, dout and k, v for dq; the other way round
    // for dk and dv.
    CUtensorMap x1, x2, y1, y2;
    PackedDirect direct;
    const PackedHeader *header;
    const PackedTile *tiles;
    const int *n_tiles;
    unsigned *counter;
    void *g1, *g2;           // dq; or dk and dv (one of them null where a kernel makes the other)
    long long g1_stride, g2_stride;
    const float *L, *D;
    long long blocks;
    float *partial;          // [slots][dk, dv or one of them][head_dim][128]
    int *arrived;            // [slots]: pieces of the tile that are done, at the slot of its first
    const unsigned *doc_most;
    const float *slopes;
    int n_docs, n_kv, log_group, sink, win;
    float scale;
    ScoreRule score;
    unsigned *err;
};
enum { kGradQ = 0, kGradKV = 1, kGradK = 2, kGradV = 3 };
// One launch: dq, and dk with dv (head_dim 256: dk alone).
struct PackedGradPair {
    PackedGradArgs q, k;
    int q_blocks, k_blocks;
};
// Pieces of a key tile are no smaller than this many row tiles: each writes 128 x head_dim
// fp32 sums of dk and of dv, which are read again, and begins with copies that nothing hides.
constexpr int kPackedLeastPiece = 4;
// Rows (or keys) of a moving tile.
constexpr int packed_grad_rows(int hd) { return hd == 256 ? 64 : 128; }
// v: of dv, for head_dim 256.
cudaError_t launch_packed_grad_bf16(const PackedGradPair &p, const PackedGradArgs *v, int hd, bool cap, cudaStream_t stream);
cudaError_t launch_packed_grad_f16(const PackedGradPair &p, const PackedGradArgs *v, int hd, bool cap, cudaStream_t stream);

}  // namespace fa
