// packed_bwd.cuh -- the gradient of packed attention on sm_103a tensor cores
// (include/fa.h, fa_packed_attn_grad); instantiated in packed_bwd_*.cu.
//
// With the weights P_ij = e^(x_ij - lse_i) of the forward pass and D_i = dout_i . out_i,
//   dv_j = sum_i P_ij dout_i
//   t_ij = P_ij (dout_i . v_j - D_i) f'(s_ij)        (f' = 1 - tanh^2 where scores are capped)
//   dq_i = scale sum_j t_ij k_j,   dk_j = scale sum_i t_ij q_i.
//
// Sums in a fixed order: some blocks hold 128 rows of queries and
// stream the keys past them (dq), others hold 128 keys and stream the rows of queries
// past them, the heads of the group among them (dk and dv; with head_dim 256, whose
// accumulators take half of TMEM each, dk here and dv in a kernel of its own). The price is
// that S and dout V^T are made twice: 7 products instead of 5 (8 with head_dim 256).
// All are one template: with stationary tiles X1, X2 and moving tiles Y1, Y2,
//   S = X1 Y1^T, T = X2 Y2^T,  acc1 += t Y1 (dq or dk),  acc2 += P Y2 (dv)
// where P and t take the places of S and T in TMEM, as the left operand of the products.
//
//   warp 0      copies: X1, X2 of a unit, then Y1, Y2 and (for dk, dv) L and D of the rows.
//               Rows past a document's end become zeros where a product sums over them.
//   warp 1      issues the products, so that those of one tile run under the weights of another:
//               dk, dv: acc2(i), S(i + 1), acc1(i), T(i + 1); dq, dk: S(i + 1), acc1(i), T(i + 1); where
//               TMEM has room for a second T it precedes acc1.
//   warps 4-11  weights: a thread has one lane of TMEM and half of a tile's columns.
//
// What bounds it: for dk and dv the bandwidth of shared memory, from which the products take both
// operands of S and T and one of the others (128 bytes a clock: a product of 128 x 128 x 128 with
// both of them there takes 517 clocks either way, so that the copies into it and the reads of L and
// D come on top), and for dq the chain S, T -> t -> acc1. 16384 tokens, 8/2 heads x 128 in bf16:
// 1211 us, 1135 TFLOP/s counted as 5 products, 1589 as the 7 that run, of 1921 measured (call after call for a
// second 1278 us: at 1330 W the power limit takes the clock from 2070 to 1950 MHz). 8192
// tokens in 23 documents, 16/2 heads x 256 capped: 318 us; there the ends of units (first copies, joins, output) show.
//
// binary16: P has 2^14 of its weight and t a power of two per document that brings the largest
// |dout| |v| near 2^13, so that neither leaves binary16's normal range on either side; bfloat16
// has the range. Both are rounded to the inputs' type, half a step each, as the products take operands of one type.
#pragma once

#include "packed_common.cuh"

namespace fa {
namespace {

template <int HD_, int MODE>
struct GradCfg {
    static constexpr int HD = HD_;
    static constexpr bool ROWS_STAY = MODE == kGradQ;  // the stationary tile is of query rows
    static constexpr bool HAS_T = MODE != kGradV, HAS_P = MODE == kGradKV || MODE == kGradV;
    static constexpr int BN = packed_grad_rows(HD);    // rows of a moving tile
    static constexpr int NWG = 2;                      // warpgroups that compute weights
    static constexpr int PART = BN / NWG;              // columns of a thread
    static constexpr int NCHUNK = HD / 64;
    static constexpr uint32_t XCHUNK = 128 * 128, YCHUNK = BN * 128;
    static constexpr uint32_t XTILE = NCHUNK * XCHUNK, YTILE = NCHUNK * YCHUNK;
    // Stationary tiles in shared memory. With head_dim 256 X1 is in TMEM, where the scores take it from as their
    // left operand: that leaves room for more stages, and the products less to fetch. On its way there it
    // passes through where X2 goes next, or for dv a place of its own.
    static constexpr bool X1_TMEM = HD == 256;
    static constexpr int NX = X1_TMEM ? 1 : 2;
    static constexpr uint32_t OFF_X2 = X1_TMEM ? 0 : XTILE;
    static constexpr int N1 = HAS_T ? 3 : 2;           // stages of Y1 and Y2
    static constexpr int N2 = HD == 64 || !HAS_T ? 3 : 2;
    static constexpr int NL = 2;                       // stages of L and D
    static constexpr uint32_t OFF_Y1 = NX * XTILE;
    static constexpr uint32_t OFF_Y2 = OFF_Y1 + N1 * YTILE;
    static constexpr uint32_t OFF_END = OFF_Y2 + N2 * YTILE;
    static constexpr uint32_t OFF_STATS = OFF_END;     // [NL][2][BN] L and D of a tile's rows
    static constexpr uint32_t OFF_BIAS = OFF_STATS + (ROWS_STAY ? 0 : NL * 2 * BN * 4);  // [2][16]
    static constexpr uint32_t OFF_BARS = OFF_BIAS + 128;
    static constexpr uint32_t SMEM = OFF_BARS + 640 > 120u * 1024u ? OFF_BARS + 640 : 120u * 1024u;
    // TMEM: S, T (dv alone: a second S), acc1, acc2; a second T where there is room
    static constexpr int NT = HAS_T && 256 + HD * (MODE == kGradKV ? 2 : 1) + 128 <= 512 ? 2 : 1;
    static constexpr uint32_t S_COL = 0, T_COL = BN, S2_COL = BN;
    static constexpr uint32_t X1_COL = 128;
    static constexpr uint32_t ACC1 = 256, ACC2 = MODE == kGradKV ? 256 + HD : 256;
    static constexpr uint32_t T2_COL = 384;
    __host__ __device__ static constexpr uint32_t t_col(int tt) { return NT == 2 && (tt & 1) ? T2_COL : T_COL; }
    static constexpr int COMPUTE = 128 * NWG;          // threads that compute weights
    static constexpr int THREADS = 128 + COMPUTE;
    static_assert(SMEM <= 227u * 1024u, "shared memory");
};

struct GradBars {
    uint64_t x_full, x_empty, x1_full, xs_full, xs_free;
    uint64_t y1_full[3], y1_empty[3], y2_full[3], y2_empty[3];
    uint64_t l_full[2], l_empty[2];
    uint64_t s_full[2], s_free, p_full[2], t_full[2], dt_full[2];
    uint64_t acc_last, acc_free, meet;
    uint64_t patch, drain;
    UnitRing ring;
    uint32_t tmem_base;
    int abort, last;
};
static_assert(sizeof(GradBars) <= 640, "barrier block");

// The units of one gradient (or of dk and dv), for block `block` of `blocks` that share them.
template <int HD, bool BF16, bool CAP, bool BIAS, int MODE>
__device__ __forceinline__ void grad_units(const PackedGradArgs &a, int block, int blocks) {
    using C = GradCfg<HD, MODE>;
    constexpr int BN = C::BN, PART = C::PART, N1 = C::N1, N2 = C::N2;
    constexpr uint32_t IDESC_S = idesc_16<BF16>(128, BN, 0, 0);
    constexpr uint32_t IDESC_ACC = idesc_16<BF16>(128, HD, 0, 1);
    // All of it dynamic: the tiles, which want 1024 bytes, begin where a block's shared memory does.
    extern __shared__ __align__(1024) uint8_t smem[];
    GradBars &bars = *reinterpret_cast<GradBars *>(smem + C::OFF_BARS);
    float *stats = reinterpret_cast<float *>(smem + C::OFF_STATS);
    // keys stay and scores fall with the distance: slopes of 16 columns, and their tokens (a group is 16
    // heads at most, so that all columns repeat these)
    float *bias_s = reinterpret_cast<float *>(smem + C::OFF_BIAS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort = &bars.abort;
    unsigned *err = a.err;
    if (smem_u32(smem) & 1023u) {  // (never so far: nothing static lies before it)
        flag_error(err, FA_ERRBIT_DEVICE);
        return;
    }

    if (threadIdx.x == 0) {
        mbar_init(&bars.x_full, 1);
        mbar_init(&bars.x_empty, 1);
        mbar_init(&bars.x1_full, C::COMPUTE / 32);
        mbar_init(&bars.xs_full, 1);
        mbar_init(&bars.xs_free, C::COMPUTE / 32);
        for (int s = 0; s < 3; ++s) {
            mbar_init(&bars.y1_full[s], 1);
            mbar_init(&bars.y1_empty[s], 1);
            mbar_init(&bars.y2_full[s], 1);
            mbar_init(&bars.y2_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars.l_full[s], 1);
            mbar_init(&bars.l_empty[s], 4 * C::NWG);
            mbar_init(&bars.s_full[s], 1);
            mbar_init(&bars.p_full[s], C::COMPUTE / 32);
            mbar_init(&bars.t_full[s], 1);
            mbar_init(&bars.dt_full[s], C::COMPUTE / 32);
        }
        mbar_init(&bars.s_free, C::COMPUTE / 32);
        mbar_init(&bars.acc_last, 1);
        mbar_init(&bars.meet, C::COMPUTE / 32);
        mbar_init(&bars.acc_free, C::COMPUTE / 32);
        mbar_init(&bars.patch, 1);
        mbar_init(&bars.drain, 1);
        for (int k = 0; k < kPackedRing; ++k) {
            mbar_init(&bars.ring.full[k], 1);
            mbar_init(&bars.ring.empty[k], 1 + 4 * C::NWG);
        }
        bars.abort = 0;
        mbar_fence_init();
        tma_prefetch_desc(&a.x1);
        tma_prefetch_desc(&a.x2);
        tma_prefetch_desc(&a.y1);
        tma_prefetch_desc(&a.y2);
    }
    if (warp == 1) {
        tmem_alloc(&bars.tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base;
    wait_for_stream();

    auto next_unit = [&](int j, PackedTile *u) -> bool {
        const int slot = j % kPackedRing;
        if (!mbar_wait(&bars.ring.full[slot], (j / kPackedRing) & 1, abort, err)) return false;
        *u = bars.ring.unit[slot];
        return u->head >= 0;
    };
    const int lg = a.log_group;
    const int tile_tokens = 128 >> lg;  // of a row tile
    const int step_tokens = BN >> lg;   // of a moving tile of rows
    // The moving tiles of a unit: of keys, or of rows (of queries that see a key of the tile).
    auto plan_of = [&](const PackedTile &u) {
        if (C::ROWS_STAY)
            return key_tiles<BN>(u.p0, min(u.p0 + tile_tokens, u.len) - 1, u.prefix, a.sink, a.win);
        KeyTiles t;
        t.ns = 0;
        t.lo = u.from;
        t.count = u.rows;
        return t;
    };
    // Rows from the last to the first: without a window the units of a document begin with the same
    // rows then, and find them in L2.
    auto place = [&](const KeyTiles &t, int i) { return C::ROWS_STAY ? t.at(i) : t.lo + t.count - 1 - i; };

    if (warp < 4) {
        fewer_registers<72>();  // 128 x 72 + 256 x 216 = the launch's 384 x 168
        if (warp == 0) {
            // ------------------------------------------------------------- copies
            // without a plan: the one unit of this block
            const bool direct = a.direct.cu != nullptr;
            PackedTile own;
            const int units = a.n_kv * (direct ? direct_tile<!C::ROWS_STAY>(a.direct, block / a.n_kv, tile_tokens, step_tokens,
                                                                            7 - lg, a.sink, a.win, err, &own)
                                               : *a.n_tiles);
            Arms x_arms, xs_arms, y1_arms[3], y2_arms[3], l_arms[2];
            int patches = 0;
            bool ok = true;
            auto fetch = [&](int w, PackedTile *u) {
                u->head = -1;
                if (w >= units || (direct && w != block)) return false;
                *u = direct ? own : a.tiles[w / a.n_kv];
                u->head = w % a.n_kv;
                return true;
            };
            auto publish = [&](int j, const PackedTile &u) {
                const int slot = j % kPackedRing;
                if (j >= kPackedRing &&
                    !mbar_wait(&bars.ring.empty[slot], ((j / kPackedRing) - 1) & 1, abort, err))
                    return false;
                if (lane == 0) {
                    bars.ring.unit[slot] = u;
                    mbar_arrive(&bars.ring.full[slot]);
                }
                return true;
            };
            // tokens from `tok` on: rows of the whole group, or keys
            auto copy = [&](const CUtensorMap *map, uint8_t *dst, uint32_t chunk, uint64_t *bar, bool rows, int head,
                            int tok) {
                for (int c = 0; c < C::NCHUNK; ++c) {
                    if (rows)
                        tma_load_4d(dst + c * chunk, map, bar, c * 64, 0, head, tok);
                    else
                        tma_load_3d(dst + c * chunk, map, bar, c * 64, head, tok);
                }
            };
            // X1 on its way to TMEM, or both
            auto load_x = [&](int j, const PackedTile &u) {
                if (j > 0 && !mbar_wait(C::HAS_T ? &bars.x_empty : &bars.xs_free, (j - 1) & 1, abort, err)) return false;
                uint64_t *bar = C::X1_TMEM ? &bars.xs_full : &bars.x_full;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, C::NX * C::XTILE);
                    copy(&a.x1, smem, C::XCHUNK, bar, C::ROWS_STAY, u.head, u.tok0 + u.p0);
                    if (!C::X1_TMEM)
                        copy(&a.x2, smem + C::OFF_X2, C::XCHUNK, bar, C::ROWS_STAY, u.head, u.tok0 + u.p0);
                }
                if (C::X1_TMEM) ++xs_arms.n; else ++x_arms.n;
                return true;
            };
            // X2 behind X1
            auto load_x2 = [&](int j, const PackedTile &u) {
                if (!mbar_wait(&bars.xs_free, j & 1, abort, err)) return false;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bars.x_full, C::XTILE);
                    copy(&a.x2, smem + C::OFF_X2, C::XCHUNK, &bars.x_full, C::ROWS_STAY, u.head, u.tok0 + u.p0);
                }
                ++x_arms.n;
                return true;
            };
            auto load_y = [&](int tt, int at, const PackedTile &u, bool first) {
                const int n = first ? N1 : N2, st = tt % n;
                uint64_t *full = first ? bars.y1_full : bars.y2_full, *empty = first ? bars.y1_empty : bars.y2_empty;
                if (tt >= n && !mbar_wait(empty + st, ((tt / n) - 1) & 1, abort, err)) return false;
                uint8_t *dst = smem + (first ? C::OFF_Y1 : C::OFF_Y2) + st * C::YTILE;
                const int p = at * (C::ROWS_STAY ? BN : step_tokens);  // its first token's position
                const int rows = min(BN, (u.len - p) << (C::ROWS_STAY ? 0 : lg));
                // a product sums over the rows of this tile (or they meet weights that are not masked)
                const bool patch = rows < BN && (first || !C::ROWS_STAY);
                uint64_t *bar = patch ? &bars.patch : full + st;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, C::YTILE);
                    copy(first ? &a.y1 : &a.y2, dst, C::YCHUNK, bar, !C::ROWS_STAY, u.head, u.tok0 + p);
                }
                if (patch) {
                    if (!mbar_wait(bar, patches++ & 1, abort, err)) return false;
                    zero_rows(dst, C::NCHUNK, C::YCHUNK, rows, BN);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full + st);
                }
                if (first) ++y1_arms[st].n; else ++y2_arms[st].n;
                return true;
            };
            auto load_stats = [&](int tt, int at, const PackedTile &u) {
                const int st = tt % C::NL;
                if (tt >= C::NL && !mbar_wait(&bars.l_empty[st], ((tt / C::NL) - 1) & 1, abort, err)) return false;
                if (lane == 0) {
                    const size_t from = (static_cast<size_t>(u.head) * a.blocks + u.rb) * 128 + static_cast<size_t>(at) * BN;
                    mbar_arrive_expect_tx(&bars.l_full[st], 2 * BN * 4);
                    bulk_copy_g2s(stats + st * 2 * BN, a.L + from, BN * 4, &bars.l_full[st]);
                    bulk_copy_g2s(stats + st * 2 * BN + BN, a.D + from, BN * 4, &bars.l_full[st]);
                }
                ++l_arms[st].n;
                return true;
            };
            int t = 0, w = block;
            PackedTile u, un;
            bool have = fetch(w, &u);
            ok = publish(0, u);
            if (have && ok) ok = load_x(0, u);
            for (int j = 0; have && ok; ++j) {
                const KeyTiles plan = plan_of(u);
                const int cnt = plan.count;
                bool more = false;
                for (int i = 0; i < cnt && ok; ++i) {
                    const int at = place(plan, i);
                    ok = load_y(t + i, at, u, true);
                    if (ok && !C::ROWS_STAY) ok = load_stats(t + i, at, u);
                    if (ok) ok = load_y(t + i, at, u, false);
                    if (C::X1_TMEM && C::HAS_T && ok && i == 0) ok = load_x2(j, u);
                    if (ok && i == cnt - 1) {
                        if (lane == 0) w = direct ? units : blocks + static_cast<int>(atomicAdd(a.counter, 1u));
                        w = __shfl_sync(~0u, w, 0);
                        more = fetch(w, &un);
                    }
                }
                t += cnt;
                if (!ok) break;
                ok = publish(j + 1, un);
                have = more;
                if (have && ok) ok = load_x(j + 1, un);
                u = un;
            }
            if (!ok) {  // copies already issued land before the block exits
                x_arms.drain(&bars.x_full);
                xs_arms.drain(&bars.xs_full);
                for (int s = 0; s < 3; ++s) {
                    y1_arms[s].drain(&bars.y1_full[s]);
                    y2_arms[s].drain(&bars.y2_full[s]);
                    if (s < 2) l_arms[s].drain(&bars.l_full[s]);
                }
                if (patches) wait_out(&bars.patch, (patches - 1) & 1);
            }
        } else if (warp == 1) {
            // ----------------------------------------------------------- products
            {
                const bool one = elect_lane();
                const uint32_t tmem = uniform(static_cast<int>(bars.tmem_base));
                // descriptors of the tiles' beginnings: an offset is added to their address field
                const uint64_t x1 = desc_sw128(smem_u32(smem), 16, 1024), x2 = x1 + (C::OFF_X2 >> 4);
                const uint64_t y1 = desc_sw128(smem_u32(smem + C::OFF_Y1), 16, 1024);   // rows as they lie
                const uint64_t y2 = desc_sw128(smem_u32(smem + C::OFF_Y2), 16, 1024);
                const uint64_t g1 = desc_sw128(smem_u32(smem + C::OFF_Y1), C::YCHUNK, 1024);  // dims as columns
                const uint64_t g2 = desc_sw128(smem_u32(smem + C::OFF_Y2), C::YCHUNK, 1024);
                constexpr uint32_t STAGE = C::YTILE >> 4;
                // scores: X (128 rows) times a moving tile's rows, summed over head_dim
                auto scores = [&](uint64_t x, uint64_t y, uint32_t col) {
                    if (one)
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk)
                            mma_ss(tmem + col, x + (((kk >> 2) * C::XCHUNK + (kk & 3) * 32) >> 4),
                                   y + (((kk >> 2) * C::YCHUNK + (kk & 3) * 32) >> 4), IDESC_S, kk > 0 ? 1u : 0u);
                };
                // the same with X in TMEM
                auto scores_tmem = [&](uint32_t x, uint64_t y, uint32_t col) {
                    if (one)
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk)
                            mma_ts(tmem + col, tmem + x + kk * 8, y + (((kk >> 2) * C::YCHUNK + (kk & 3) * 32) >> 4),
                                   IDESC_S, kk > 0 ? 1u : 0u);
                };
                // weights in TMEM (a part of the columns where its threads wrote them) times the tile itself
                auto gather = [&](uint32_t col, uint64_t y, uint32_t acc, bool first) {
                    constexpr int per = PART / 16;
                    if (one)
#pragma unroll
                        for (int kk = 0; kk < BN / 16; ++kk)
                            mma_ts(tmem + acc, tmem + col + (kk / per) * PART + (kk % per) * 8, y + (kk * 2048 >> 4),
                                   IDESC_ACC, (!first || kk > 0) ? 1u : 0u);
                };
                auto wait = [&](uint64_t *bar, uint32_t parity) { return uniform(mbar_wait(bar, parity, abort, err)); };
                auto commit = [&](uint64_t *bar) {
                    if (one) tc_commit(bar);
                };
                int t = 0;
                bool ok = true;
                PackedTile u;
                for (int j = 0; ok && uniform(next_unit(j, &u)); ++j) {
                    const int count = uniform(plan_of(u).count);
                    warp_arrive(&bars.ring.empty[j % kPackedRing]);
                    if (!(ok = wait(C::X1_TMEM ? &bars.x1_full : &bars.x_full, j & 1))) break;
                    tc_fence_after();
                    // Two barriers at once, each looked at by half of the lanes: a look takes a hundred cycles
                    // and more (dq, 16384 tokens, 8/2 heads x 128: 530 -> 504 us; where P is made, too, waiting
                    // for more than the next product wants costs as much as it saves).
                    auto wait2 = [&](uint64_t *b0, uint32_t p0, uint64_t *b1, uint32_t p1) {
                        return wait(lane & 1 ? b1 : b0, lane & 1 ? p1 : p0);
                    };
                    auto do_s = [&](int i) {
                        const int tt = t + i, st = tt % N1;
                        uint64_t *there = &bars.y1_full[st];
                        const uint32_t phase = (tt / N1) & 1;
                        // S is read whole: in the others its P was, or a product in between waited for it
                        if (!C::HAS_P && tt > 0 ? !wait2(there, phase, &bars.s_free, (tt - 1) & 1) : !wait(there, phase))
                            return false;
                        tc_fence_after();
                        const uint32_t col = C::S_COL + (C::HAS_T ? 0 : (tt & 1) * C::S2_COL);
                        if (C::X1_TMEM)
                            scores_tmem(C::X1_COL, y1 + st * STAGE, col);
                        else
                            scores(x1, y1 + st * STAGE, col);
                        commit(&bars.s_full[C::HAS_T ? 0 : tt & 1]);
                        if (!C::HAS_T) {
                            commit(&bars.y1_empty[st]);
                            if (i == count - 1) commit(&bars.x_empty);
                        }
                        return true;
                    };
                    auto do_t = [&](int i) {
                        const int tt = t + i, st = tt % N2;
                        if (C::X1_TMEM && i == 0 && !wait(&bars.x_full, j & 1)) return false;
                        if (!wait(&bars.y2_full[st], (tt / N2) & 1)) return false;
                        tc_fence_after();
                        scores(x2, y2 + st * STAGE, C::t_col(tt));
                        commit(&bars.t_full[tt % C::NT]);
                        if (!C::HAS_P) commit(&bars.y2_empty[st]);
                        if (i == count - 1) commit(&bars.x_empty);
                        return true;
                    };
                    auto acc_ready = [&](int i) {
                        return i > 0 || j == 0 || wait(&bars.acc_free, (j - 1) & 1);
                    };
                    auto do_acc2 = [&](int i) {
                        const int tt = t + i, st = tt % N2, b = C::HAS_T ? 0 : tt & 1;
                        if (!wait(&bars.p_full[b], (C::HAS_T ? tt : tt >> 1) & 1) || !acc_ready(i)) return false;
                        if (!C::HAS_T && !wait(&bars.y2_full[st], (tt / N2) & 1)) return false;
                        tc_fence_after();
                        gather(C::S_COL + b * C::S2_COL, g2 + st * STAGE, C::ACC2, i == 0);
                        commit(&bars.y2_empty[st]);
                        return true;
                    };
                    auto do_acc1 = [&](int i) {
                        const int tt = t + i, st = tt % N1;
                        if (!wait(&bars.dt_full[tt % C::NT], (tt / C::NT) & 1) || !acc_ready(i)) return false;
                        tc_fence_after();
                        gather(C::t_col(tt), g1 + st * STAGE, C::ACC1, i == 0);
                        commit(&bars.y1_empty[st]);
                        return true;
                    };
                    if (MODE == kGradV) {
                        for (int i = 0; i <= count && ok; ++i) {
                            if (i < count) ok = do_s(i);
                            if (ok && i > 0) ok = do_acc2(i - 1);
                        }
                    } else {
                        ok = do_s(0) && do_t(0);
                        for (int i = 0; i < count && ok; ++i) {
                            if (C::HAS_P) ok = do_acc2(i);
                            if (ok && i + 1 < count) ok = do_s(i + 1);
                            if (C::NT == 2 && ok && i + 1 < count) ok = do_t(i + 1);
                            ok = ok && do_acc1(i);
                            if (C::NT == 1 && ok && i + 1 < count) ok = do_t(i + 1);
                        }
                    }
                    if (ok) commit(&bars.acc_last);
                    t += count;
                }
                // every product issued completes before TMEM is released
                commit(&bars.drain);
                wait_out(&bars.drain, 0);
                __syncwarp();
            }
        }
    } else {
        more_registers<216>();
        // -------------------------------------------------- weights and output
        const int part = (warp - 4) >> 2;           // this thread's part of a tile's columns
        const int r = threadIdx.x & 127;            // its lane of TMEM: row of the stationary tile
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int group = 1 << lg;
        const ScoreRule rule = a.score;
        // all of these threads: what each wrote before is there for the others (a wait with a bound)
        int meets = 0;
        auto meet = [&]() {
            warp_arrive(&bars.meet);
            return static_cast<bool>(__all_sync(~0u, mbar_wait(&bars.meet, meets++ & 1, abort, err)));
        };
        auto take = [&](int j, PackedTile *u) {
            const bool got = next_unit(j, u);
            warp_arrive(&bars.ring.empty[j % kPackedRing]);
            return static_cast<bool>(__all_sync(~0u, got));
        };
        // This thread's row of X1, a half of its dims, from shared memory into TMEM. Every S of the unit
        // before is done. (Rows straight from memory, each by its thread, took 5 us.)
        auto load_x1 = [&](int j) {
            const bool got = mbar_wait(&bars.xs_full, j & 1, abort, err);
            if (!__all_sync(~0u, got)) return false;
#pragma unroll
            for (int c = 0; c < HD / 2; c += 64) {  // 64 dims: a chunk's row
                const uint8_t *row = smem + ((part * (HD / 2) + c) / 64) * C::XCHUNK + r * 128;
                uint32_t w[32];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint4 x = lds_v4(row + ((k ^ (r & 7)) << 4));
                    w[4 * k] = x.x, w[4 * k + 1] = x.y, w[4 * k + 2] = x.z, w[4 * k + 3] = x.w;
                }
                tmem_st32(tmem + lane_base + C::X1_COL + (part * (HD / 2) + c) / 2, w);
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&bars.x1_full);
            if (lane == 0) mbar_arrive(&bars.xs_free);
            return true;
        };
        int t = 0;
        bool ok = true;
        PackedTile u;
        for (int j = 0; ok && take(j, &u); ++j) {
            if (C::X1_TMEM && !(ok = load_x1(j))) break;
            const KeyTiles plan = plan_of(u);
            // rows stay: this thread's query; keys stay: its key
            const int mine = u.p0 + (C::ROWS_STAY ? r >> lg : r);
            const int head = (u.head << lg) + (r & (group - 1));  // of its query
            float L = 0.0f, D = 0.0f, slope2 = 0.0f;
            if (C::ROWS_STAY) {
                const size_t at = (static_cast<size_t>(u.head) * a.blocks + u.rb) * 128 +
                                  (static_cast<size_t>(u.p0) << lg) + r;
                L = load(a.L + at);
                D = load(a.D + at);
                if (BIAS) slope2 = load(a.slopes + head) * -kPackedLog2e;
            }
            if (BIAS && !C::ROWS_STAY) {  // (the slopes of the last unit have been used)
                if (!(ok = meet())) break;
                const int c = threadIdx.x - 128;
                if (c < 16) {
                    bias_s[c] = load(a.slopes + (u.head << lg) + (c & (group - 1))) * -kPackedLog2e;
                    bias_s[16 + c] = static_cast<float>(c >> lg);
                }
                if (!(ok = meet())) break;
            }
            float up = 1.0f;  // the document's power of two
            if (!BF16) {
                unsigned most[2];
                if (a.direct.cu) {  // of all blocks of the document
                    const int blocks = ((u.len << lg) + 127) >> 7;
                    for (int k = 0; k < 2; ++k) {
                        unsigned m = 0;
                        for (int e = lane; e < blocks * a.n_kv; e += 32)
                            m = max(m, load(a.doc_most + (static_cast<size_t>(k) * a.n_kv + e / blocks) * a.blocks + u.rb + e % blocks));
                        most[k] = __reduce_max_sync(~0u, m);
                    }
                } else {
                    most[0] = load(a.doc_most + u.doc);
                    most[1] = load(a.doc_most + a.n_docs + u.doc);
                }
                const float b = 2.0f * sqrtf(__uint_as_float(most[0])) * sqrtf(__uint_as_float(most[1]));
                if (b > 0.0f && b < 3e38f) {
                    const int e = static_cast<int>(__float_as_uint(b) >> 23) - 127;  // b < 2^(e + 1)
                    up = __uint_as_float(static_cast<uint32_t>(127 + min(max(13 - e, -100), 100)) << 23);
                }
            }
            const float t_scale = up * 6.103515625e-05f;  // 2^-14: P has 2^14 of it
            for (int i = 0; i < plan.count; ++i) {
                const int tt = t + i;
                const int sb = C::HAS_T ? 0 : tt & 1, ls = tt % C::NL;
                ok = mbar_wait(&bars.s_full[sb], (C::HAS_T ? tt : tt >> 1) & 1, abort, err);
                if (!C::ROWS_STAY) ok = ok && mbar_wait(&bars.l_full[ls], (tt / C::NL) & 1, abort, err);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t scol = tmem + lane_base + C::S_COL + sb * C::S2_COL + part * PART;
                const uint32_t tcol = tmem + lane_base + C::t_col(tt) + part * PART;
                uint32_t s[PART];
                tmem_ld<PART>(scol, s);
                tmem_wait_ld();
                reg_fence<PART>(s);
                if (!C::HAS_P) {  // S may be overwritten
                    tc_fence_before();
                    warp_arrive(&bars.s_free);
                }
                // ---- what is seen of this part: columns [lo, hi], and those below `first`
                int first = 0, lo, hi;
                bool whole;
                float far;         // query less key at column 0
                const int c0 = part * PART;
                if (C::ROWS_STAY) {
                    const int j0 = place(plan, i) * BN + c0, j1 = j0 + PART - 1;
                    whole = sees_all(u.p0, min(u.p0 + tile_tokens, u.len) - 1, j0, j1, u.prefix, a.sink, a.win) &&
                            (!BIAS || j1 <= u.p0);
                    hi = mine - j0;
                    lo = a.win > 0 ? mine - a.win + 1 - j0 : 0;
                    first = max(u.prefix - j0, a.win > 0 ? min(a.sink - j0, hi + 1) : 0);
                    far = static_cast<float>(mine - j0);
                } else {
                    const int i0 = place(plan, i) * step_tokens, i1 = min(i0 + step_tokens, u.len) - 1;
                    const int j1 = min(u.p0 + 128, u.len) - 1;
                    whole = sees_all(i0, i1, u.p0, j1, u.prefix, a.sink, a.win) && (!BIAS || j1 <= i0);
                    const bool always = mine < u.prefix;
                    lo = (min(max(always ? 0 : mine - i0, 0), BN) << lg) - c0;
                    hi = always || a.win <= 0 || mine < a.sink
                             ? BN
                             : (max(min(mine + a.win - 1 - i0, BN), -1) + 1 << lg) - 1 - c0;
                    far = static_cast<float>(i0 - mine);
                }
                const float *Ls = stats + ls * 2 * BN + c0, *Ds = Ls + BN;
                // ---- P, and with capped scores P f' / 4 (in s)
                uint32_t pk[PART / 2];
                auto weights = [&](auto masks) {
                    constexpr bool MASK = decltype(masks)::value;
                    float far_at[(PART + 15) / 16];
#pragma unroll
                    for (int c = 0; c < (PART + 15) / 16; ++c)
                        far_at[c] = far + static_cast<float>((c0 + 16 * c) >> lg);
#pragma unroll
                    for (int c = 0; c < PART; c += 4) {
                        float4 lv = make_float4(L, L, L, L), sv, tv;
                        if (!C::ROWS_STAY) {
                            lv = lds_f4(Ls + c);
                            if (BIAS) sv = lds_f4(bias_s + (c & 15)), tv = lds_f4(bias_s + 16 + (c & 15));
                        }
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            Two x = two(__uint_as_float(s[c + e]), __uint_as_float(s[c + e + 1]));
                            Two off = e ? two(lv.z, lv.w) : two(lv.x, lv.y), down;
                            if (BIAS) {  // (slopes are negative here)
                                Two d, sl = two(slope2);
                                if (C::ROWS_STAY) {
                                    d = two(far) + two(-static_cast<float>(c + e), -static_cast<float>(c + e + 1));
                                } else {
                                    d = two(far_at[c / 16]) + (e ? two(tv.z, tv.w) : two(tv.x, tv.y));
                                    sl = e ? two(sv.z, sv.w) : two(sv.x, sv.y);
                                }
                                if (MASK) {
                                    const float2 f = both(d);
                                    d = two(fabsf(f.x), fabsf(f.y));
                                }
                                off = fma2(sl, d, off);
                            }
                            if (CAP) {
                                const Two q = cap_r(x, rule);
                                down = cap_slope(q);
                                x = capped(q, rule) + off;
                            } else {
                                x = fma2(x, two(rule.a), off);
                            }
                            float2 f = both(x);
                            if (MASK) {
                                const int k = c + e;
                                if (!((k < first) | ((k >= lo) & (k <= hi)))) f.x = -INFINITY;
                                if (!((k + 1 < first) | ((k + 1 >= lo) & (k + 1 <= hi)))) f.y = -INFINITY;
                            }
                            f = make_float2(ex2(f.x), ex2(f.y));
                            if (C::HAS_P) pk[(c + e) / 2] = pack2<BF16>(f.x, f.y);
                            if (CAP) f = both(two(f.x, f.y) * down);
                            s[c + e] = __float_as_uint(f.x);
                            s[c + e + 1] = __float_as_uint(f.y);
                        }
                    }
                };
                if (whole) weights(std::false_type{}); else weights(std::true_type{});
                if (C::HAS_P) {
                    tmem_st<PART / 2>(scol, pk);
                    tmem_wait_st();
                    tc_fence_before();
                    warp_arrive(&bars.p_full[sb]);
                }
                if (C::HAS_T) {
                    ok = mbar_wait(&bars.t_full[tt % C::NT], (tt / C::NT) & 1, abort, err);
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t d[PART];
                    tmem_ld<PART>(tcol, d);
                    tmem_wait_ld();
                    reg_fence<PART>(d);
                    auto slopes_of = [&](auto masks) {
                        constexpr bool MASK = decltype(masks)::value;
#pragma unroll
                        for (int c = 0; c < PART; c += 4) {
                            float4 dv = make_float4(D, D, D, D);
                            if (!C::ROWS_STAY) dv = lds_f4(Ds + c);
#pragma unroll
                            for (int e = 0; e < 4; e += 2) {
                                const Two w = two(__uint_as_float(s[c + e]), __uint_as_float(s[c + e + 1]));
                                Two x = two(__uint_as_float(d[c + e]), __uint_as_float(d[c + e + 1])) +
                                        (e ? two(dv.z, dv.w) : two(dv.x, dv.y));
                                x = x * w;
                                if (!BF16) x = x * two(t_scale);
                                float2 f = both(x);
                                if (MASK) {
                                    if (s[c + e] == 0u) f.x = 0.0f;
                                    if (s[c + e + 1] == 0u) f.y = 0.0f;
                                }
                                d[(c + e) / 2] = pack2<BF16>(f.x, f.y);
                            }
                        }
                    };
                    // V past the document's end may hold anything
                    if (C::ROWS_STAY && !whole) slopes_of(std::true_type{}); else slopes_of(std::false_type{});
                    tmem_st<PART / 2>(tcol, d);
                    tmem_wait_st();
                    tc_fence_before();
                    warp_arrive(&bars.dt_full[tt % C::NT]);
                }
                if (!C::ROWS_STAY) {
                    warp_arrive(&bars.l_empty[ls]);
                }
            }
            if (!ok) break;
            t += plan.count;
            ok = mbar_wait(&bars.acc_last, j & 1, abort, err);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            tc_fence_after();
            const bool live = mine < u.len;
            // half of the threads store dk and half dv, or all of them the one gradient
            constexpr bool BOTH = MODE == kGradKV;
            constexpr int COLS = HD / (BOTH ? C::NWG / 2 : C::NWG);
            const bool of_v = BOTH ? part >= C::NWG / 2 : MODE == kGradV;
            const int col0 = (BOTH ? part % (C::NWG / 2) : part) * COLS;
            const float factor = of_v ? (BF16 ? 1.0f : 6.103515625e-05f) : (CAP ? 4.0f : 1.0f) * a.scale / up;
            const long long stride = of_v ? a.g2_stride : a.g1_stride;
            uint16_t *out = static_cast<uint16_t *>(of_v ? a.g2 : a.g1) +
                            (static_cast<long long>(u.tok0) + mine) * stride +
                            static_cast<long long>(C::ROWS_STAY ? head : u.head) * HD + col0;
            const bool wide = wide_rows(of_v ? a.g2 : a.g1, stride);
            auto store = [&](int c, const uint32_t *o) {
                if (!live) return;
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[e] = pack2<BF16>(__uint_as_float(o[2 * e]) * factor, __uint_as_float(o[2 * e + 1]) * factor);
                store16(out + 16 * c, w, wide);
            };
            const bool alone = C::ROWS_STAY || u.pieces == 1;
            // pieces of this tile and head lie one behind another, [column][lane] of each
            constexpr int SLOT = (BOTH ? 2 : 1) * HD * 128;
            const int slot0 = alone ? 0 : u.slot + u.head * u.pieces;
            float *sums = a.partial + static_cast<size_t>(slot0) * SLOT + ((BOTH && of_v ? HD : 0) + col0) * 128 + r;
#pragma unroll 1
            for (int c = 0; c < COLS / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(tmem + lane_base + (of_v ? C::ACC2 : C::ACC1) + col0 + 16 * c, o);
                tmem_wait_ld();
                reg_fence<16>(o);
                if (c == COLS / 16 - 1) {
                    tc_fence_before();
                    warp_arrive(&bars.acc_free);
                }
                if (alone) {
                    store(c, o);
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        __stcg(sums + static_cast<size_t>(u.piece) * SLOT + (16 * c + k) * 128, __uint_as_float(o[k]));
                }
            }
            if (!alone) {
                // the block that is done last adds the pieces, in their order
                __threadfence();
                if (!(ok = meet())) break;
                if (threadIdx.x == 128) {
                    bars.last = atomicAdd(a.arrived + slot0, 1) == u.pieces - 1;
                    if (bars.last) a.arrived[slot0] = 0;  // for the next kernel
                    __threadfence();
                }
                if (!(ok = meet())) break;
                if (*static_cast<volatile int *>(&bars.last)) {
                    __threadfence();
#pragma unroll 1
                    for (int c = 0; c < COLS / 32; ++c) {
                        float x[32] = {};
#pragma unroll 1
                        for (int k = 0; k < u.pieces; ++k)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                x[e] += __ldcg(sums + static_cast<size_t>(k) * SLOT + (32 * c + e) * 128);
                        uint32_t o[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(x[e]);
                        store(2 * c, o);
                        store(2 * c + 1, o + 16);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// One launch for both, as neither uses what the other makes: the blocks of dk (and dv) are those behind dq's, and take
// the SMs that dq's leave. (As a kernel that dq's let begin early they would have to do without the wait for what is
// before dq in the stream, which is what makes the rows' sums visible to them.)
template <int HD, bool BF16, bool CAP, bool BIAS, int SECOND>
__global__ void __launch_bounds__((GradCfg<HD, kGradQ>::THREADS), 1)
    packed_grad_kernel(const __grid_constant__ PackedGradPair p) {
    const int block = blockIdx.x;
    if (block < p.q_blocks)
        grad_units<HD, BF16, CAP, BIAS, kGradQ>(p.q, block, p.q_blocks);
    else
        grad_units<HD, BF16, CAP, BIAS, SECOND>(p.k, block - p.q_blocks, p.k_blocks);
}
// dv of head_dim 256, whose partial sums take the places of dk's: a launch after it.
template <int HD, bool BF16, bool CAP, bool BIAS>
__global__ void __launch_bounds__((GradCfg<HD, kGradV>::THREADS), 1)
    packed_grad_v_kernel(const __grid_constant__ PackedGradArgs a) {
    grad_units<HD, BF16, CAP, BIAS, kGradV>(a, blockIdx.x, gridDim.x);
}

template <int HD, bool BF16, bool CAP, bool BIAS>
cudaError_t launch_grad(const PackedGradPair &p, const PackedGradArgs *v, cudaStream_t stream) {
    constexpr int SECOND = HD < 256 ? kGradKV : kGradK;
    using Q = GradCfg<HD, kGradQ>;
    using K = GradCfg<HD, SECOND>;
    using V = GradCfg<HD, kGradV>;
    static_assert(Q::THREADS == K::THREADS, "one launch");
    constexpr size_t SMEM = Q::SMEM > K::SMEM ? Q::SMEM : K::SMEM;
    static std::atomic<uint64_t> made{0}, made_v{0};
    auto kernel = packed_grad_kernel<HD, BF16, CAP, BIAS, SECOND>;
    cudaError_t e = allow_smem(kernel, SMEM, &made);
    if (e == cudaSuccess) e = launch_after(kernel, dim3(p.q_blocks + p.k_blocks), Q::THREADS, SMEM, stream, p);
    if constexpr (HD == 256) {
        auto kernel_v = packed_grad_v_kernel<HD, BF16, CAP, BIAS>;
        if (e == cudaSuccess) e = allow_smem(kernel_v, V::SMEM, &made_v);
        if (e == cudaSuccess) e = launch_after(kernel_v, dim3(p.k_blocks), V::THREADS, V::SMEM, stream, *v);
    }
    return e;
}

template <int HD, bool BF16>
cudaError_t launch_grad_rule(const PackedGradPair &p, const PackedGradArgs *v, bool cap, cudaStream_t stream) {
    if (cap)
        return p.q.slopes ? launch_grad<HD, BF16, true, true>(p, v, stream) : launch_grad<HD, BF16, true, false>(p, v, stream);
    return p.q.slopes ? launch_grad<HD, BF16, false, true>(p, v, stream) : launch_grad<HD, BF16, false, false>(p, v, stream);
}

template <bool BF16>
cudaError_t launch_grad_type(const PackedGradPair &p, const PackedGradArgs *v, int hd, bool cap, cudaStream_t stream) {
    switch (hd) {
        case 64: return launch_grad_rule<64, BF16>(p, v, cap, stream);
        case 128: return launch_grad_rule<128, BF16>(p, v, cap, stream);
        default: return launch_grad_rule<256, BF16>(p, v, cap, stream);
    }
}

}  // namespace
}  // namespace fa
