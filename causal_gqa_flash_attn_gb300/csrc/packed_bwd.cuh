// packed_bwd.cuh -- the gradient of packed attention on sm_103a tensor cores
// (include/fa.h, fa_packed_attn_grad); instantiated in packed_bwd_*.cu.
//
// With the weights P_ij = e^(x_ij - lse_i) of the forward pass and D_i = dout_i . out_i,
//   dv_j = sum_i P_ij dout_i
//   t_ij = P_ij (dout_i . v_j - D_i) f'(s_ij)        (f' = 1 - tanh^2 where scores are capped)
//   dq_i = scale sum_j t_ij k_j,   dk_j = scale sum_i t_ij q_i.
//
// Sums in a fixed order, without atomics: one kernel holds 128 rows of queries and
// streams the keys past them (dq), one holds 128 keys and streams the rows of queries
// past them, the heads of the group among them (dk and dv; with head_dim 256, whose
// accumulators take half of TMEM each, a kernel for dk and one for dv). The price is
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
// binary16: P has 2^14 of its weight and t a power of two per document that brings the largest
// |dout| |v| near 2^13, so that neither leaves binary16's normal range on either side; bfloat16
// has the range.
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
    static constexpr int HALF = BN / 2;                // columns of a thread
    static constexpr int NCHUNK = HD / 64;
    static constexpr uint32_t XCHUNK = 128 * 128, YCHUNK = BN * 128;
    static constexpr uint32_t XTILE = NCHUNK * XCHUNK, YTILE = NCHUNK * YCHUNK;
    static constexpr int NX = HAS_T ? 2 : 1;
    // Stages of Y1 and Y2: Y2 of dq and dk alone is read once, right after it lands.
    static constexpr int N1 = HD == 64 ? 3 : 2;
    static constexpr int N2 = HD == 64 ? 3 : HD == 256 && HAS_T ? 1 : 2;
    static constexpr int NL = 2;                       // stages of L and D
    static constexpr uint32_t OFF_Y1 = NX * XTILE;
    static constexpr uint32_t OFF_Y2 = OFF_Y1 + N1 * YTILE;
    static constexpr uint32_t OFF_END = OFF_Y2 + N2 * YTILE;
    static constexpr uint32_t SMEM = (OFF_END + 1024 > 120u * 1024u) ? OFF_END + 1024 : 120u * 1024u;
    // TMEM: S, T (dv alone: a second S), acc1, acc2; a second T where there is room
    static constexpr int NT = HAS_T && 256 + HD * (MODE == kGradKV ? 2 : 1) + 128 <= 512 ? 2 : 1;
    static constexpr uint32_t S_COL = 0, T_COL = 128;
    static constexpr uint32_t ACC1 = 256, ACC2 = MODE == kGradKV ? 256 + HD : 256;
    static constexpr uint32_t T2_COL = 384;
    __host__ __device__ static constexpr uint32_t t_col(int tt) { return NT == 2 && (tt & 1) ? T2_COL : T_COL; }
    static constexpr int THREADS = 384;
    static_assert(OFF_END <= 224u * 1024u, "shared memory");
};

struct GradBars {
    uint64_t x_full, x_empty;
    uint64_t y1_full[3], y1_empty[3], y2_full[3], y2_empty[3];
    uint64_t l_full[2], l_empty[2];
    uint64_t s_full[2], s_free, p_full[2], t_full[2], dt_full[2];
    uint64_t acc_last, acc_free;
    uint64_t patch, drain;
    UnitRing ring;
    uint32_t tmem_base;
    int abort;
};

template <int HD, bool BF16, bool CAP, bool BIAS, int MODE>
__global__ void __launch_bounds__(384, 1) packed_grad_kernel(const __grid_constant__ PackedGradArgs a) {
    using C = GradCfg<HD, MODE>;
    constexpr int BN = C::BN, HALF = C::HALF, N1 = C::N1, N2 = C::N2;
    constexpr uint32_t IDESC_S = idesc_16<BF16>(128, BN, 0, 0);
    constexpr uint32_t IDESC_ACC = idesc_16<BF16>(128, HD, 0, 1);
    extern __shared__ uint8_t smem_raw[];
    __shared__ GradBars bars;
    __shared__ __align__(16) float stats[C::ROWS_STAY ? 1 : C::NL][2][C::ROWS_STAY ? 4 : BN];
    // keys stay and scores fall with the distance: slopes of a tile's columns, and their tokens
    __shared__ __align__(16) float bias_s[2][BIAS && !C::ROWS_STAY ? BN : 4];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort = &bars.abort;
    unsigned *err = a.err;

    if (threadIdx.x == 0) {
        mbar_init(&bars.x_full, 1);
        mbar_init(&bars.x_empty, 1);
        for (int s = 0; s < 3; ++s) {
            mbar_init(&bars.y1_full[s], 1);
            mbar_init(&bars.y1_empty[s], 1);
            mbar_init(&bars.y2_full[s], 1);
            mbar_init(&bars.y2_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars.l_full[s], 1);
            mbar_init(&bars.l_empty[s], 8);
            mbar_init(&bars.s_full[s], 1);
            mbar_init(&bars.p_full[s], 256);
            mbar_init(&bars.t_full[s], 1);
            mbar_init(&bars.dt_full[s], 256);
        }
        mbar_init(&bars.s_free, 256);
        mbar_init(&bars.acc_last, 1);
        mbar_init(&bars.acc_free, 256);
        mbar_init(&bars.patch, 1);
        mbar_init(&bars.drain, 1);
        for (int k = 0; k < kPackedRing; ++k) {
            mbar_init(&bars.ring.full[k], 1);
            mbar_init(&bars.ring.empty[k], 1 + 8);
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
    // The moving tiles of a unit: of keys, or of rows (from the first query that sees a key of the
    // tile to the last).
    auto plan_of = [&](const PackedTile &u) {
        if (C::ROWS_STAY)
            return key_tiles<BN>(u.p0, min(u.p0 + tile_tokens, u.len) - 1, u.prefix, a.sink, a.win);
        int first, last;
        query_range(u.p0, min(u.p0 + 128, u.len) - 1, u.len, u.prefix, a.sink, a.win, &first, &last);
        KeyTiles t;
        t.ns = 0;
        t.lo = first / step_tokens;
        t.count = last / step_tokens - t.lo + 1;
        return t;
    };
    // Rows from the last to the first: without a window the units of a document begin with the same
    // rows then, and find them in L2.
    auto place = [&](const KeyTiles &t, int i) { return C::ROWS_STAY ? t.at(i) : t.lo + t.count - 1 - i; };

    if (warp == 0) {
        // ------------------------------------------------------------- copies
        const int units = *a.n_tiles * a.n_kv;
        Arms x_arms, y1_arms[3], y2_arms[3], l_arms[2];
        int patches = 0;
        bool ok = true;
        auto fetch = [&](int w, PackedTile *u) {
            u->head = -1;
            if (w >= units) return false;
            *u = a.tiles[w / a.n_kv];
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
        auto load_x = [&](int j, const PackedTile &u) {
            if (j > 0 && !mbar_wait(&bars.x_empty, (j - 1) & 1, abort, err)) return false;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars.x_full, C::NX * C::XTILE);
                copy(&a.x1, smem, C::XCHUNK, &bars.x_full, C::ROWS_STAY, u.head, u.tok0 + u.p0);
                if (C::NX == 2)
                    copy(&a.x2, smem + C::XTILE, C::XCHUNK, &bars.x_full, C::ROWS_STAY, u.head, u.tok0 + u.p0);
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
                bulk_copy_g2s(stats[st][0], a.L + from, BN * 4, &bars.l_full[st]);
                bulk_copy_g2s(stats[st][1], a.D + from, BN * 4, &bars.l_full[st]);
            }
            ++l_arms[st].n;
            return true;
        };
        int t = 0, w = blockIdx.x;
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
                if (ok && i == cnt - 1) {
                    if (lane == 0) w = static_cast<int>(gridDim.x + atomicAdd(a.counter, 1u));
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
            for (int s = 0; s < 3; ++s) {
                y1_arms[s].drain(&bars.y1_full[s]);
                y2_arms[s].drain(&bars.y2_full[s]);
                if (s < 2) l_arms[s].drain(&bars.l_full[s]);
            }
            if (patches) wait_out(&bars.patch, (patches - 1) & 1);
        }
    } else if (warp == 1) {
        // ----------------------------------------------------------- products
        if (lane == 0) {
            const uint32_t sX = smem_u32(smem), sY1 = smem_u32(smem + C::OFF_Y1), sY2 = smem_u32(smem + C::OFF_Y2);
            // scores: X (128 rows) times a moving tile's rows, summed over head_dim
            auto scores = [&](uint32_t x, uint32_t y, uint32_t col) {
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk)
                    mma_ss(tmem + col, desc_sw128(x + (kk >> 2) * C::XCHUNK + (kk & 3) * 32, 16, 1024),
                           desc_sw128(y + (kk >> 2) * C::YCHUNK + (kk & 3) * 32, 16, 1024), IDESC_S, kk > 0 ? 1u : 0u);
            };
            // weights in TMEM (each half of the columns where its threads wrote them) times the tile itself
            auto gather = [&](uint32_t col, uint32_t y, uint32_t acc, bool first) {
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk) {
                    constexpr int per = HALF / 16;
                    mma_ts(tmem + acc, tmem + col + (kk / per) * HALF + (kk % per) * 8,
                           desc_sw128(y + kk * 2048, C::YCHUNK, 1024), IDESC_ACC, (!first || kk > 0) ? 1u : 0u);
                }
            };
            int t = 0;
            bool ok = true;
            PackedTile u;
            for (int j = 0; ok && next_unit(j, &u); ++j) {
                mbar_arrive(&bars.ring.empty[j % kPackedRing]);
                const int count = plan_of(u).count;
                if (!(ok = mbar_wait(&bars.x_full, j & 1, abort, err))) break;
                tc_fence_after();
                auto do_s = [&](int i) {
                    const int tt = t + i, st = tt % N1;
                    if (!mbar_wait(&bars.y1_full[st], (tt / N1) & 1, abort, err)) return false;
                    // S is read whole: in the others its P was, or a product in between waited for it
                    if (!C::HAS_P && tt > 0 && !mbar_wait(&bars.s_free, (tt - 1) & 1, abort, err)) return false;
                    tc_fence_after();
                    scores(sX, sY1 + st * C::YTILE, C::S_COL + (C::HAS_T ? 0 : (tt & 1) * 128));
                    tc_commit(&bars.s_full[C::HAS_T ? 0 : tt & 1]);
                    if (!C::HAS_T) {
                        tc_commit(&bars.y1_empty[st]);
                        if (i == count - 1) tc_commit(&bars.x_empty);
                    }
                    return true;
                };
                auto do_t = [&](int i) {
                    const int tt = t + i, st = tt % N2;
                    if (!mbar_wait(&bars.y2_full[st], (tt / N2) & 1, abort, err)) return false;
                    tc_fence_after();
                    scores(sX + C::XTILE, sY2 + st * C::YTILE, C::t_col(tt));
                    tc_commit(&bars.t_full[tt % C::NT]);
                    if (!C::HAS_P) tc_commit(&bars.y2_empty[st]);
                    if (i == count - 1) tc_commit(&bars.x_empty);
                    return true;
                };
                auto acc_ready = [&](int i) {
                    return i > 0 || j == 0 || mbar_wait(&bars.acc_free, (j - 1) & 1, abort, err);
                };
                auto do_acc2 = [&](int i) {
                    const int tt = t + i, st = tt % N2, b = C::HAS_T ? 0 : tt & 1;
                    if (!mbar_wait(&bars.p_full[b], (C::HAS_T ? tt : tt >> 1) & 1, abort, err) || !acc_ready(i)) return false;
                    if (!C::HAS_T && !mbar_wait(&bars.y2_full[st], (tt / N2) & 1, abort, err)) return false;
                    tc_fence_after();
                    gather(C::S_COL + b * 128, sY2 + st * C::YTILE, C::ACC2, i == 0);
                    tc_commit(&bars.y2_empty[st]);
                    return true;
                };
                auto do_acc1 = [&](int i) {
                    const int tt = t + i, st = tt % N1;
                    if (!mbar_wait(&bars.dt_full[tt % C::NT], (tt / C::NT) & 1, abort, err) || !acc_ready(i)) return false;
                    tc_fence_after();
                    gather(C::t_col(tt), sY1 + st * C::YTILE, C::ACC1, i == 0);
                    tc_commit(&bars.y1_empty[st]);
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
                if (ok) tc_commit(&bars.acc_last);
                t += count;
            }
            // every product issued completes before TMEM is released
            tc_commit(&bars.drain);
            wait_out(&bars.drain, 0);
        }
    } else if (warp >= 4) {
        // -------------------------------------------------- weights and output
        const int half = (warp - 4) >> 2;           // this thread's half of a tile's columns
        const int r = threadIdx.x & 127;            // its lane of TMEM: row of the stationary tile
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int group = 1 << lg;
        const ScoreRule rule = a.score;
        int t = 0;
        bool ok = true;
        PackedTile u;
        for (int j = 0; ok; ++j) {
            const bool have = next_unit(j, &u);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.ring.empty[j % kPackedRing]);
            if (!__all_sync(~0u, have)) break;
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
                if (BIAS) slope2 = load(a.slopes + head) * kPackedLog2e;
            }
            if (BIAS && !C::ROWS_STAY) {  // (the slopes of the last unit have been used)
                named_barrier_sync(1, 256);
                const int c = threadIdx.x - 128;
                if (c < BN) {
                    bias_s[0][c] = load(a.slopes + (u.head << lg) + (c & (group - 1))) * kPackedLog2e;
                    bias_s[1][c] = static_cast<float>(c >> lg);
                }
                named_barrier_sync(1, 256);
            }
            float up = 1.0f;  // the document's power of two
            if (!BF16) {
                const float b = 2.0f * sqrtf(__uint_as_float(load(a.doc_most + u.doc))) *
                                sqrtf(__uint_as_float(load(a.doc_most + a.n_docs + u.doc)));
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
                const uint32_t scol = tmem + lane_base + C::S_COL + sb * 128 + half * HALF;
                const uint32_t tcol = tmem + lane_base + C::t_col(tt) + half * HALF;
                uint32_t s[HALF];
#pragma unroll
                for (int c = 0; c < HALF; c += 32) tmem_ld32(scol + c, s + c);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < HALF; c += 32) reg_fence32(s + c);
                if (!C::HAS_P) {  // S may be overwritten
                    tc_fence_before();
                    mbar_arrive(&bars.s_free);
                }
                // ---- what is seen of this half: columns [lo, hi], and those below `first`
                int first = 0, lo, hi;
                bool whole;
                float far;         // query less key at column 0
                const int c0 = half * HALF;
                if (C::ROWS_STAY) {
                    const int j0 = place(plan, i) * BN + c0, j1 = j0 + HALF - 1;
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
                const float *Ls = stats[C::ROWS_STAY ? 0 : ls][0] + c0, *Ds = stats[C::ROWS_STAY ? 0 : ls][1] + c0;
                // ---- P, and with capped scores P f' (in s)
                uint32_t pk[HALF / 2];
                auto weights = [&](auto masks) {
                    constexpr bool MASK = decltype(masks)::value;
                    const float base = slope2 * far;
#pragma unroll
                    for (int c = 0; c < HALF; c += 4) {
                        float4 lv = make_float4(L, L, L, L), sv, tv;
                        if (!C::ROWS_STAY) {
                            lv = lds_f4(Ls + c);
                            if (BIAS) sv = lds_f4(bias_s[0] + c0 + c), tv = lds_f4(bias_s[1] + c0 + c);
                        }
                        const float l4[4] = {lv.x, lv.y, lv.z, lv.w};
                        float w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float x = __uint_as_float(s[c + e]), down = 1.0f, off = l4[e];
                            if (BIAS && C::ROWS_STAY) {
                                off += MASK ? slope2 * fabsf(far - static_cast<float>(c + e))
                                            : fmaf(-slope2, static_cast<float>(c + e), base);
                            } else if (BIAS) {
                                const float s4[4] = {sv.x, sv.y, sv.z, sv.w}, t4[4] = {tv.x, tv.y, tv.z, tv.w};
                                const float d = far + t4[e];
                                off = fmaf(s4[e], MASK ? fabsf(d) : d, off);
                            }
                            x = CAP ? capped(x, rule, &down) - off : fmaf(x, rule.a, -off);
                            if (MASK) {
                                const bool seen = (c + e < first) | ((c + e >= lo) & (c + e <= hi));
                                x = seen ? x : -INFINITY;
                            }
                            w[e] = ex2(x);
                            s[c + e] = __float_as_uint(CAP ? w[e] * down : w[e]);
                        }
                        if (C::HAS_P) {
                            pk[c / 2] = pack2<BF16>(w[0], w[1]);
                            pk[c / 2 + 1] = pack2<BF16>(w[2], w[3]);
                        }
                    }
                };
                if (whole) weights(std::false_type{}); else weights(std::true_type{});
                if (C::HAS_P) {
                    if (HALF == 64) tmem_st32(scol, pk); else tmem_st16(scol, pk);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(&bars.p_full[sb]);
                }
                if (C::HAS_T) {
                    ok = mbar_wait(&bars.t_full[tt % C::NT], (tt / C::NT) & 1, abort, err);
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t d[HALF];
#pragma unroll
                    for (int c = 0; c < HALF; c += 32) tmem_ld32(tcol + c, d + c);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < HALF; c += 32) reg_fence32(d + c);
                    auto slopes_of = [&](auto masks) {
                        constexpr bool MASK = decltype(masks)::value;
#pragma unroll
                        for (int c = 0; c < HALF; c += 4) {
                            float4 dv = make_float4(D, D, D, D);
                            if (!C::ROWS_STAY) dv = lds_f4(Ds + c);
                            const float d4[4] = {dv.x, dv.y, dv.z, dv.w};
                            float x[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float w = __uint_as_float(s[c + e]);
                                x[e] = w * (__uint_as_float(d[c + e]) - d4[e]);
                                if (!BF16) x[e] *= t_scale;
                                if (MASK) x[e] = w == 0.0f ? 0.0f : x[e];
                            }
                            d[c / 2] = pack2<BF16>(x[0], x[1]);
                            d[c / 2 + 1] = pack2<BF16>(x[2], x[3]);
                        }
                    };
                    // V past the document's end may hold anything
                    if (C::ROWS_STAY && !whole) slopes_of(std::true_type{}); else slopes_of(std::false_type{});
                    if (HALF == 64) tmem_st32(tcol, d); else tmem_st16(tcol, d);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(&bars.dt_full[tt % C::NT]);
                }
                if (!C::ROWS_STAY) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.l_empty[ls]);
                }
            }
            if (!ok) break;
            t += plan.count;
            ok = mbar_wait(&bars.acc_last, j & 1, abort, err);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            tc_fence_after();
            const bool live = mine < u.len;
            // the first half of the threads stores dk and the other dv, or each half its columns
            constexpr bool BOTH = MODE == kGradKV;
            constexpr int COLS = BOTH ? HD : HD / 2;
            const bool of_v = BOTH ? half == 1 : MODE == kGradV;
            const int col0 = BOTH ? 0 : half * COLS;
            const float factor = of_v ? (BF16 ? 1.0f : 6.103515625e-05f) : a.scale / up;
            const long long stride = of_v ? a.g2_stride : a.g1_stride;
            uint16_t *out = static_cast<uint16_t *>(of_v ? a.g2 : a.g1) +
                            (static_cast<long long>(u.tok0) + mine) * stride +
                            static_cast<long long>(C::ROWS_STAY ? head : u.head) * HD + col0;
#pragma unroll 1
            for (int c = 0; c < COLS / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tmem + lane_base + (of_v ? C::ACC2 : C::ACC1) + col0 + 32 * c, o);
                tmem_wait_ld();
                reg_fence32(o);
                if (c == COLS / 32 - 1) {
                    tc_fence_before();
                    mbar_arrive(&bars.acc_free);
                }
                if (live) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack2<BF16>(__uint_as_float(o[8 * k + 2 * e]) * factor,
                                               __uint_as_float(o[8 * k + 2 * e + 1]) * factor);
                        *reinterpret_cast<uint4 *>(out + 32 * c + 8 * k) = make_uint4(w[0], w[1], w[2], w[3]);
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

template <int HD, bool BF16, bool CAP, bool BIAS, int MODE>
cudaError_t launch_grad(const PackedGradArgs &a, int blocks, cudaStream_t stream) {
    using C = GradCfg<HD, MODE>;
    auto kernel = packed_grad_kernel<HD, BF16, CAP, BIAS, MODE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, dim3(blocks), C::THREADS, C::SMEM, stream, a);
}

template <int HD, bool BF16, int MODE>
cudaError_t launch_grad_rule(const PackedGradArgs &a, bool cap, int blocks, cudaStream_t stream) {
    if (cap)
        return a.slopes ? launch_grad<HD, BF16, true, true, MODE>(a, blocks, stream)
                        : launch_grad<HD, BF16, true, false, MODE>(a, blocks, stream);
    return a.slopes ? launch_grad<HD, BF16, false, true, MODE>(a, blocks, stream)
                    : launch_grad<HD, BF16, false, false, MODE>(a, blocks, stream);
}

// Head_dim 64 and 128 have dq, and dk with dv; 256 has each by itself.
template <bool BF16>
cudaError_t launch_grad_type(const PackedGradArgs &a, int mode, int hd, bool cap, int blocks, cudaStream_t stream) {
    if (hd == 64)
        return mode == kGradQ ? launch_grad_rule<64, BF16, kGradQ>(a, cap, blocks, stream)
                              : launch_grad_rule<64, BF16, kGradKV>(a, cap, blocks, stream);
    if (hd == 128)
        return mode == kGradQ ? launch_grad_rule<128, BF16, kGradQ>(a, cap, blocks, stream)
                              : launch_grad_rule<128, BF16, kGradKV>(a, cap, blocks, stream);
    switch (mode) {
        case kGradQ: return launch_grad_rule<256, BF16, kGradQ>(a, cap, blocks, stream);
        case kGradK: return launch_grad_rule<256, BF16, kGradK>(a, cap, blocks, stream);
        default: return launch_grad_rule<256, BF16, kGradV>(a, cap, blocks, stream);
    }
}

}  // namespace
}  // namespace fa
