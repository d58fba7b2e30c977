// packed_fwd.cuh -- attention of packed documents on sm_103a tensor cores
// (include/fa.h, fa_packed_attn); instantiated in packed_fwd_*.cu.
//
// For the query at position i of a document, over the keys j that it sees,
//   x_j = f(scale q . k_j) - slope |i - j|,  f(s) = s or cap tanh(s / cap),
//   out = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m),  lse = m + log sum_j e^(x_j - m).
//
// A persistent block takes units, 256 rows (two tiles of 128; one with head_dim 256)
// of one kv head, and streams the key tiles past them:
//   warp 0      copies Q, K and V tiles (TMA, 128-byte swizzle). In the last tile of a
//               document V's rows past its end become zeros, as other documents and
//               padding may hold anything and 0 * inf is not 0.
//   warp 1      issues the products: S = Q K^T into TMEM, O += P V with P from TMEM.
//   warps 4-11  softmax, one thread a row and tile (or, with one tile, two threads a row, each
//               with half of the columns): the running maximum in the exp2 domain, which moves
//               only when a score passes it by 2^8, so that O is seldom rescaled; P over S, rounded
//               to the inputs' type, as a product's operands have one type (half a step of each
//               weight: results are 1.1 to 1.4 times as far from 64 bits as with fp32 weights);
//               sums of the unrounded weights in fp32; and the output.
// With two tiles the products of one run under the softmax of the other; with one (whose O takes
// half of TMEM) S has two places, and S(i + 1) runs under the softmax of S(i). TMEM is full at
// 128 and 256: 2 x (O 128 + S 128) columns, or O 256 + 2 x S 128. At 64 a quarter of it is free (columns 128 to 255):
// a third S or the next unit's O would fit there.
//
// What bounds it: at head_dim 128 the chain S -> softmax -> P V of each tile, of which TMEM holds
// two and no third (16384 tokens, 8/2 heads: 370 us, 1485 TFLOP/s of 1921 measured for bf16); at
// 256 the tensor cores (8192 tokens, 16/2 heads: 327 us, 1680 TFLOP/s); at 64, and wherever scores
// are capped, the softmax warps, two a scheduler, with issue slots and special units half full each
// and the latter's slow ones (a clock and SM: 32 exponentials, but 16 reciprocals) behind one another
// (64: 279 us; 128 capped: 597 us). Documents of a few tiles spend as long on a unit's first copies and
// its output as on the products (8192 tokens in 23 documents, 16/2 heads x 256 capped: 74 us, 692
// TFLOP/s).
#pragma once

#include "packed_common.cuh"

namespace fa {
namespace {

constexpr float kFwdLift = 8.0f;   // log2 growth of a score that moves the reference
constexpr float kFwdShift = 6.0f;  // log2 of a weight at the reference: fp16 has its normal range below

template <int HD_>
struct FwdCfg {
    static constexpr int HD = HD_;
    static constexpr int NT = packed_fwd_tiles(HD);
    static constexpr int BK = 128;
    static constexpr int NCHUNK = HD / 64;
    static constexpr uint32_t CHUNK = 128 * 128;  // 128 rows of 128 bytes
    static constexpr uint32_t TILE = NCHUNK * CHUNK;
    static constexpr int NS = HD == 256 ? 1 : 2;  // stages of K and of V
    static constexpr uint32_t OFF_K = NT * TILE;
    static constexpr uint32_t OFF_V = OFF_K + NS * TILE;
    static constexpr uint32_t OFF_OUT = OFF_V + NS * TILE;  // a box of 32 rows of 128 bytes for each warp
    static constexpr uint32_t OFF_END = OFF_OUT + 8 * 4096;
    static constexpr uint32_t OFF_BARS = OFF_END + (NT == 2 ? 0 : 2 * 2 * 128 * 4);  // behind a row's two maxima
    // one block an SM, which owns all of TMEM
    static constexpr uint32_t SMEM = OFF_BARS + 512 > 120u * 1024u ? OFF_BARS + 512 : 120u * 1024u;
    static_assert(SMEM <= 227u * 1024u, "shared memory");
    static constexpr uint32_t S_COL = 256;  // O in columns 0 .. 255
    static constexpr int THREADS = 384;
    // Two warpgroups: one for each tile, or with one tile each half of its columns.
    static constexpr int COLS = NT == 2 ? 128 : 64;  // columns of S of a thread
    static constexpr int DIMS = NT == 2 ? HD : HD / 2;  // and of O
    static constexpr int ARRIVE = NT == 2 ? 4 : 8;   // warps that a tile's barriers wait for
};

struct FwdBars {
    uint64_t q_full, q_empty;
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t s_full[2], p_full[2], o_last[2], o_free[2];
    uint64_t o_done, patch, drain, meet;
    UnitRing ring;
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(FwdBars) <= 512, "barrier block");

template <int HD, bool BF16, bool CAP, bool BIAS>
__global__ void __launch_bounds__(FwdCfg<HD>::THREADS, 1)
    packed_fwd_kernel(const __grid_constant__ PackedFwdArgs a) {
    using C = FwdCfg<HD>;
    constexpr int NT = C::NT, NS = C::NS, BK = C::BK;
    constexpr uint32_t IDESC_QK = idesc_16<BF16>(128, BK, 0, 0);
    constexpr uint32_t IDESC_PV = idesc_16<BF16>(128, HD, 0, 1);
    // All of it dynamic: the tiles, which want 1024 bytes, begin where a block's shared memory does.
    extern __shared__ __align__(1024) uint8_t smem[];
    FwdBars &bars = *reinterpret_cast<FwdBars *>(smem + C::OFF_BARS);
    // one tile: [turn][half][row], maxima of a row's two halves
    volatile float *row_max = reinterpret_cast<float *>(smem + C::OFF_END);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort = &bars.abort;
    unsigned *err = a.err;
    if (smem_u32(smem) & 1023u) {  // (never so far: nothing static lies before it)
        flag_error(err, FA_ERRBIT_DEVICE);
        return;
    }

    if (threadIdx.x == 0) {
        mbar_init(&bars.q_full, 1);
        mbar_init(&bars.q_empty, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars.k_full[s], 1);
            mbar_init(&bars.k_empty[s], 1);
            mbar_init(&bars.v_full[s], 1);
            mbar_init(&bars.v_empty[s], 1);
            mbar_init(&bars.s_full[s], 1);
            mbar_init(&bars.p_full[s], C::ARRIVE);
            mbar_init(&bars.o_last[s], 1);
            mbar_init(&bars.o_free[s], C::ARRIVE);
        }
        mbar_init(&bars.o_done, 1);
        mbar_init(&bars.patch, 1);
        mbar_init(&bars.drain, 1);
        mbar_init(&bars.meet, 8);
        for (int k = 0; k < kPackedRing; ++k) {
            mbar_init(&bars.ring.full[k], 1);
            mbar_init(&bars.ring.empty[k], 1 + 8);  // the MMA thread and the softmax warps
        }
        bars.abort = 0;
        mbar_fence_init();
        tma_prefetch_desc(&a.q);
        tma_prefetch_desc(&a.k);
        tma_prefetch_desc(&a.v);
        tma_prefetch_desc(&a.o);
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

    // the j-th unit of this block; false at the end of the work
    auto next_unit = [&](int j, PackedTile *u) -> bool {
        const int slot = j % kPackedRing;
        if (!mbar_wait(&bars.ring.full[slot], (j / kPackedRing) & 1, abort, err)) return false;
        *u = bars.ring.unit[slot];
        return u->head >= 0;
    };
    const int row_tokens = (128 * NT) >> a.log_group;  // tokens of a unit
    auto last_of = [&](const PackedTile &u) { return min(u.p0 + row_tokens, u.len) - 1; };
    auto plan_of = [&](const PackedTile &u) {
        return key_tiles<BK>(u.p0, last_of(u), u.prefix, a.sink, a.win);
    };

    if (warp < 4) {
        fewer_registers<72>();  // 128 x 72 + 256 x 216 = the launch's 384 x 168
        if (warp == 0) {
            // ------------------------------------------------------------- copies
            // without a plan: the one unit of this block
            const bool direct = a.direct.cu != nullptr;
            PackedTile own;
            const int units = a.n_kv * (direct ? direct_tile<false>(a.direct, blockIdx.x / a.n_kv, row_tokens, 1,
                                                                    7 - a.log_group, a.sink, a.win, err, &own)
                                               : a.header->row_tiles);
            Arms q_arms, k_arms[2], v_arms[2];
            int patches = 0;
            bool ok = true;
            auto fetch = [&](int w, PackedTile *u) {
                u->head = -1;
                if (w >= units || (direct && w != static_cast<int>(blockIdx.x))) return false;
                *u = direct ? own : a.rows[w / a.n_kv];
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
            auto load_q = [&](int j, const PackedTile &u) {
                if (j > 0 && !mbar_wait(&bars.q_empty, (j - 1) & 1, abort, err)) return false;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bars.q_full, NT * C::TILE);
                    for (int t = 0; t < NT; ++t)
                        for (int c = 0; c < C::NCHUNK; ++c)
                            tma_load_4d(smem + t * C::TILE + c * C::CHUNK, &a.q, &bars.q_full, c * 64, 0, u.head,
                                        u.tok0 + u.p0 + t * (row_tokens / NT));
                }
                ++q_arms.n;
                return true;
            };
            auto load_kv = [&](int tt, int kt, const PackedTile &u, bool is_k) {
                const int st = tt % NS;
                if (tt >= NS && !mbar_wait(is_k ? &bars.k_empty[st] : &bars.v_empty[st], ((tt / NS) - 1) & 1, abort, err))
                    return false;
                uint64_t *full = is_k ? &bars.k_full[st] : &bars.v_full[st];
                uint8_t *dst = smem + (is_k ? C::OFF_K : C::OFF_V) + st * C::TILE;
                const int rows = min(BK, u.len - kt * BK);
                // scores past the end are masked, but V's rows are summed
                const bool patch = !is_k && rows < BK;
                uint64_t *bar = patch ? &bars.patch : full;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, C::TILE);
                    for (int c = 0; c < C::NCHUNK; ++c)
                        tma_load_3d(dst + c * C::CHUNK, is_k ? &a.k : &a.v, bar, c * 64, u.head, u.tok0 + kt * BK);
                }
                if (patch) {
                    if (!mbar_wait(bar, patches++ & 1, abort, err)) return false;
                    zero_rows(dst, C::NCHUNK, C::CHUNK, rows, BK);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full);
                }
                if (is_k) ++k_arms[st].n; else ++v_arms[st].n;
                return true;
            };
            int t = 0, w = blockIdx.x;
            PackedTile u, un;
            bool have = fetch(w, &u);
            ok = publish(0, u);
            if (have && ok) ok = load_q(0, u);
            for (int j = 0; have && ok; ++j) {
                const KeyTiles plan = plan_of(u);
                const int cnt = plan.count;
                bool more = false;
                for (int i = 0; i < cnt && ok; ++i) {
                    ok = load_kv(t + i, plan.at(i), u, true);
                    if (ok && i == cnt - 1) {  // the next unit, under the waits for the last tiles
                        if (lane == 0) w = direct ? units : static_cast<int>(gridDim.x + atomicAdd(a.counter, 1u));
                        w = __shfl_sync(~0u, w, 0);
                        more = fetch(w, &un);
                    }
                    if (ok && i >= 1) ok = load_kv(t + i - 1, plan.at(i - 1), u, false);
                }
                if (ok) ok = load_kv(t + cnt - 1, plan.at(cnt - 1), u, false);
                t += cnt;
                if (!ok) break;
                ok = publish(j + 1, un);
                have = more;
                if (have && ok) ok = load_q(j + 1, un);
                u = un;
            }
            if (!ok) {  // copies already issued land before the block exits
                q_arms.drain(&bars.q_full);
                for (int s = 0; s < 2; ++s) {
                    k_arms[s].drain(&bars.k_full[s]);
                    v_arms[s].drain(&bars.v_full[s]);
                }
                if (patches) wait_out(&bars.patch, (patches - 1) & 1);
            }
        } else if (warp == 1) {
            // ----------------------------------------------------------- products
            {
                const bool one = elect_lane();
                const uint32_t tmem = uniform(static_cast<int>(bars.tmem_base));
                // descriptors of the tiles' beginnings: an offset is added to their address field
                const uint64_t dq = desc_sw128(smem_u32(smem), 16, 1024);
                const uint64_t dk = desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
                const uint64_t dv = desc_sw128(smem_u32(smem + C::OFF_V), C::CHUNK, 1024);  // dims as columns
                // which: the tile of the unit, or with one tile the S
                auto issue_s = [&](int which, int tt) {
                    const uint64_t q = dq + (NT == 2 ? which * C::TILE >> 4 : 0), k = dk + (tt % NS) * (C::TILE >> 4);
                    const uint32_t col = tmem + C::S_COL + which * 128;
                    if (one)
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk) {
                            const uint32_t off = ((kk >> 2) * C::CHUNK + (kk & 3) * 32) >> 4;
                            mma_ss(col, q + off, k + off, IDESC_QK, kk > 0 ? 1u : 0u);
                        }
                };
                auto issue_pv = [&](int which, int tt, bool first) {
                    const uint64_t v = dv + (tt % NS) * (C::TILE >> 4);
                    const uint32_t o = tmem + (NT == 2 ? which * HD : 0), p = tmem + C::S_COL + which * 128;
                    if (one)
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            mma_ts(o, p + kk * 8, v + (kk * 2048 >> 4), IDESC_PV, (!first || kk > 0) ? 1u : 0u);
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
                    if (!(ok = wait(&bars.q_full, j & 1))) break;
                    tc_fence_after();
                    // P of tile tt is there, and O free for a unit's first product
                    auto wait_p = [&](int tile, int tt, bool first, uint32_t bar, uint32_t parity) {
                        if (!wait(&bars.p_full[bar], parity)) return false;
                        if (first && j > 0 && !wait(&bars.o_free[tile], (j - 1) & 1)) return false;
                        return true;
                    };
                    auto wait_kv = [&](uint64_t *full, int tt) {
                        return wait(full + tt % NS, (tt / NS) & 1);
                    };
                    if (NT == 2) {
                        // one S for each tile: its next product follows the one that reads its P
                        for (int i = 0; i <= count && ok; ++i) {
                            const int tt = t + i;
                            // K of this step and V of the last one, each looked at by half of the lanes
                            const int kt = i < count ? tt : tt - 1, vt = i > 0 ? tt - 1 : tt;
                            const bool on_k = i == 0 || (i < count && (lane & 1));
                            if (!(ok = wait(on_k ? &bars.k_full[kt % NS] : &bars.v_full[vt % NS],
                                            ((on_k ? kt : vt) / NS) & 1)))
                                break;
                            tc_fence_after();
#pragma unroll
                            for (int tile = 0; tile < 2; ++tile) {
                                if (i > 0) {
                                    if (!(ok = wait_p(tile, tt - 1, i == 1, tile, (tt - 1) & 1))) break;
                                    tc_fence_after();
                                    issue_pv(tile, tt - 1, i == 1);
                                    if (tile == 1) commit(&bars.v_empty[(tt - 1) % NS]);
                                    if (i == count) commit(&bars.o_last[tile]);
                                }
                                if (i < count) {
                                    issue_s(tile, tt);
                                    commit(&bars.s_full[tile]);
                                    if (tile == 1) {
                                        commit(&bars.k_empty[tt % NS]);
                                        if (i == count - 1) commit(&bars.q_empty);
                                    }
                                }
                            }
                        }
                    } else {
                        // two S for the tile, which take turns
                        for (int i = 0; i <= count && ok; ++i) {
                            const int tt = t + i;
                            if (i < count) {
                                if (!(ok = wait_kv(bars.k_full, tt))) break;
                                tc_fence_after();
                                issue_s(tt & 1, tt);
                                commit(&bars.k_empty[tt % NS]);
                                commit(&bars.s_full[tt & 1]);
                                if (i == count - 1) commit(&bars.q_empty);
                            }
                            if (i > 0) {
                                const int pt = tt - 1;
                                if (!(ok = wait_p(0, pt, i == 1, pt & 1, (pt >> 1) & 1) && wait_kv(bars.v_full, pt))) break;
                                tc_fence_after();
                                issue_pv(pt & 1, pt, i == 1);
                                commit(&bars.v_empty[pt % NS]);
                                commit(&bars.o_done);
                                if (i == count) commit(&bars.o_last[0]);
                            }
                        }
                    }
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
        // ------------------------------------------------- softmax and output
        constexpr int COLS = C::COLS, DIMS = C::DIMS;
        const int group = (warp - 4) >> 2;
        const int tile = NT == 2 ? group : 0;  // this warp's tile of the unit
        const int part = NT == 2 ? 0 : group;  // and its half of the columns
        const int r = threadIdx.x & 127;       // row of the tile: TMEM lane
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int lg = a.log_group, tile_tokens = 128 >> lg;
        const ScoreRule rule = a.score;
        // both halves' threads: what each wrote before is there for the other (a wait with a bound)
        int meets = 0;
        auto meet = [&]() {
            tc_fence_before();
            warp_arrive(&bars.meet);
            const bool got = mbar_wait(&bars.meet, meets++ & 1, abort, err);
            tc_fence_after();
            return static_cast<bool>(__all_sync(~0u, got));
        };
        int t = 0;
        bool ok = true;
        PackedTile u;
        for (int j = 0; ok; ++j) {
            const bool have = next_unit(j, &u);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.ring.empty[j % kPackedRing]);
            if (!__all_sync(~0u, have)) break;
            const KeyTiles plan = plan_of(u);
            const int p0 = u.p0 + tile * tile_tokens;                // of this tile
            const int p1 = min(p0 + tile_tokens, u.len) - 1;         // (below p0: no rows)
            const int p = p0 + (r >> lg);
            const int head = (u.head << lg) + (r & ((1 << lg) - 1));
            const float slope2 = BIAS ? load(a.slopes + head) * kPackedLog2e : 0.0f;
            float m_used = -INFINITY;  // reference of O and l
            float l = 0.0f;
            for (int i = 0; i < plan.count; ++i) {
                const int tt = t + i;
                const int bar = NT == 2 ? tile : tt & 1;
                const int j0 = plan.at(i) * BK + part * COLS, j1 = j0 + COLS - 1;  // its keys
                const bool whole = sees_all(p0, p1, j0, j1, u.prefix, a.sink, a.win) && (!BIAS || j1 <= p0);
                ok = mbar_wait(&bars.s_full[bar], (NT == 2 ? tt : tt >> 1) & 1, abort, err);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t scol = tmem + lane_base + C::S_COL + bar * 128;
                uint32_t s[COLS];
                tmem_ld<COLS>(scol + part * COLS, s);
                tmem_wait_ld();
                reg_fence<COLS>(s);

                if (CAP && !whole) {
                    // A reciprocal serves two columns: what lies behind an odd document, masked further down, must
                    // not reach the document's last key. (Zeros in K's tile instead, as in V's, keep the copies
                    // waiting: 8192 tokens in 23 documents, 16/2 heads x 256, 75.5 us for 73.)
                    const int past = u.len - j0;  // the first column behind it
                    if ((past & 1) && past > 0 && past < COLS) {
#pragma unroll
                        for (int c = 1; c < COLS; c += 2) s[c] = c == past ? 0u : s[c];
                    }
                }
                constexpr bool kScaled = CAP || BIAS;  // s goes to the exp2 domain first
                if (kScaled) {
                    const float far = static_cast<float>(p - j0);  // exact up to 2^24
                    auto score = [&](auto masks) {
                        constexpr bool MASK = decltype(masks)::value;
#pragma unroll
                        for (int c = 0; c < COLS; c += 2) {
                            Two x = two(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), off = two(0.0f);
                            if (BIAS) {
                                Two d = two(far) + two(-static_cast<float>(c), -static_cast<float>(c + 1));
                                if (MASK) {
                                    const float2 f = both(d);
                                    d = two(fabsf(f.x), fabsf(f.y));
                                }
                                off = two(-slope2) * d;
                            }
                            if (CAP)
                                x = BIAS ? capped(cap_r(x, rule), rule) + off : capped(cap_r(x, rule), rule);
                            else
                                x = fma2(x, two(rule.a), off);
                            const float2 f = both(x);
                            s[c] = __float_as_uint(f.x);
                            s[c + 1] = __float_as_uint(f.y);
                        }
                    };
                    if (!BIAS || whole) score(std::false_type{}); else score(std::true_type{});
                }
                if (!whole) {
                    // key j0 + c is seen iff c < head or lo <= c <= hi
                    const int hi = p - j0;
                    const int lo = a.win > 0 ? p - a.win + 1 - j0 : 0;
                    const int first = max(u.prefix - j0, a.win > 0 ? min(a.sink - j0, hi + 1) : 0);
#pragma unroll
                    for (int c = 0; c < COLS; ++c)
                        if (!((c < first) | ((c >= lo) & (c <= hi)))) s[c] = __float_as_uint(-INFINITY);
                }
                // four chains, so that none of them is waited for
                float mx4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) mx4[e] = __uint_as_float(s[e]);
#pragma unroll
                for (int c = 4; c < COLS - 4; c += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mx4[e] = max3(mx4[e], __uint_as_float(s[c + 2 * e]), __uint_as_float(s[c + 2 * e + 1]));
#pragma unroll
                for (int e = 0; e < 4; ++e) mx4[e] = fmaxf(mx4[e], __uint_as_float(s[COLS - 4 + e]));
                float mx = max3(mx4[0], mx4[1], fmaxf(mx4[2], mx4[3]));
                if (!kScaled) mx *= rule.a;
                if (NT == 1) {  // of the whole row; and every S of the tile is read, where P goes
                    row_max[((tt & 1) * 2 + part) * 128 + r] = mx;
                    if (!(ok = meet())) break;
                    mx = fmaxf(mx, row_max[((tt & 1) * 2 + (part ^ 1)) * 128 + r]);
                }
                const float m_new = fmaxf(m_used, mx);
                float corr = 1.0f;
                bool moves = false;
                if (m_new > m_used + kFwdLift) {
                    if (m_used != -INFINITY) {
                        corr = ex2(m_used - m_new);
                        moves = true;
                        l *= corr;
                    }
                    m_used = m_new;
                }
                // O is rescaled when every product into it is done. With one S a tile that
                // holds already: S(tt) was issued after them. With two, PV(tt - 1) may still run.
                if (__any_sync(~0u, moves)) {
                    if (NT == 1) {
                        ok = mbar_wait(&bars.o_done, (tt - 1) & 1, abort, err);
                        ok = __all_sync(~0u, ok);
                        if (!ok) break;
                        tc_fence_after();
                    }
#pragma unroll 1
                    for (int c = 0; c < DIMS / 32; ++c) {
                        uint32_t o[32];
                        const uint32_t oc = tmem + lane_base + tile * HD + part * DIMS + 32 * c;
                        tmem_ld32(oc, o);
                        tmem_wait_ld();
                        reg_fence32(o);
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * corr);
                        tmem_st32(oc, o);
                    }
                }
                const Two ref = two(m_used == -INFINITY ? 0.0f : kFwdShift - m_used);
                Two sums[2] = {two(0.0f), two(0.0f)};
#pragma unroll
                for (int half = 0; half < COLS; half += 64) {
                    uint32_t pk[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const Two x = two(__uint_as_float(s[half + 2 * c]), __uint_as_float(s[half + 2 * c + 1]));
                        float2 f = both(kScaled ? x + ref : fma2(x, two(rule.a), ref));
                        f = make_float2(ex2(f.x), ex2(f.y));
                        sums[c & 1] = sums[c & 1] + two(f.x, f.y);
                        pk[c] = pack2<BF16>(f.x, f.y);
                    }
                    tmem_st32(scol + part * (COLS / 2) + half / 2, pk);
                }
                const float2 sum = both(sums[0] + sums[1]);
                l += sum.x + sum.y;
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&bars.p_full[bar]);
            }
            if (!ok) break;
            t += plan.count;
            ok = mbar_wait(&bars.o_last[tile], j & 1, abort, err);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            tc_fence_after();
            if (NT == 1) {
                // (the buffer that the next tile does not begin with: who is there has read this one)
                row_max[(((t & 1) ^ 1) * 2 + part) * 128 + r] = l;
                if (!(ok = meet())) break;
                const float other = row_max[(((t & 1) ^ 1) * 2 + (part ^ 1)) * 128 + r];
                l = part ? other + l : l + other;
            }
            const bool live = p < u.len, wide = wide_rows(a.out, a.out_stride);
            const float inv = 1.0f / l;  // a row sees itself, so that l > 0 (or a NaN)
            if (a.lse && live && part == 0)
                a.lse[static_cast<size_t>(head) * a.n_tokens + u.tok0 + p] =
                    (m_used - kFwdShift + log2f(l)) * kPackedLn2;
            uint16_t *out = static_cast<uint16_t *>(a.out) + (static_cast<long long>(u.tok0) + p) * a.out_stride +
                            static_cast<long long>(head) * HD + part * DIMS;
            // 32 rows that are all there leave through this warp's box (128-byte swizzle) by a tensor copy; at
            // a document's end each thread stores its own. (Threads' stores, each to a row of its own, took
            // 3.5 us of a unit with head_dim 256.)
            const int row0 = (warp & 3) * 32;
            const bool full = p0 + ((row0 + 31) >> lg) < u.len;
            uint8_t *box = smem + C::OFF_OUT + (warp - 4) * 4096;
#pragma unroll 1
            for (int c = 0; c < DIMS / 64; ++c) {
                uint32_t o[64], w[32];
                tmem_ld<64>(tmem + lane_base + tile * HD + part * DIMS + 64 * c, o);
                tmem_wait_ld();
                reg_fence<64>(o);
                if (c == DIMS / 64 - 1) {  // read whole: the next unit may overwrite it
                    tc_fence_before();
                    warp_arrive(&bars.o_free[tile]);
                }
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    w[e] = pack2<BF16>(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                if (full) {
                    if (lane == 0) bulk_wait_group_read<0>();  // the box has been copied
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint4 *>(box + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                            make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_4d(&a.o, box, part * DIMS + 64 * c, 0, u.head, u.tok0 + p0 + (row0 >> lg));
                        bulk_commit_group();
                    }
                } else if (live) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) store16(out + 64 * c + 16 * k, w + 8 * k, wide);
                }
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int HD, bool BF16, bool CAP, bool BIAS>
cudaError_t launch_fwd(const PackedFwdArgs &a, int blocks, cudaStream_t stream) {
    using C = FwdCfg<HD>;
    auto kernel = packed_fwd_kernel<HD, BF16, CAP, BIAS>;
    static std::atomic<uint64_t> made{0};
    const cudaError_t e = allow_smem(kernel, C::SMEM, &made);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, dim3(blocks), C::THREADS, C::SMEM, stream, a);
}

template <int HD, bool BF16>
cudaError_t launch_fwd_rule(const PackedFwdArgs &a, bool cap, int blocks, cudaStream_t stream) {
    if (cap)
        return a.slopes ? launch_fwd<HD, BF16, true, true>(a, blocks, stream)
                        : launch_fwd<HD, BF16, true, false>(a, blocks, stream);
    return a.slopes ? launch_fwd<HD, BF16, false, true>(a, blocks, stream)
                    : launch_fwd<HD, BF16, false, false>(a, blocks, stream);
}

template <bool BF16>
cudaError_t launch_fwd_type(const PackedFwdArgs &a, int hd, bool cap, int blocks, cudaStream_t stream) {
    switch (hd) {
        case 64: return launch_fwd_rule<64, BF16>(a, cap, blocks, stream);
        case 128: return launch_fwd_rule<128, BF16>(a, cap, blocks, stream);
        default: return launch_fwd_rule<256, BF16>(a, cap, blocks, stream);
    }
}

}  // namespace
}  // namespace fa
