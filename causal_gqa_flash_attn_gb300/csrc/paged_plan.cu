// paged_plan.cu -- block tables, slot maps and positions of one serving step,
// built on the GPU from the requests' lengths (include/fa.h, fa_page_plan).
//
// With c rows cached and f fresh ones, request r needs ceil((c + f) / P) -
// ceil(c / P) new pages; X_r, the sum over the requests before it, is where
// its pages start behind the ring's head, and the same sum over finished
// requests' pages is where theirs go behind its tail. Everything else follows
// element by element: page k of r is ring[head + X_r + k], token t of the step
// belongs to the request whose token range holds t.
//
// The call is bound by latency: a few dependent reads of a few KB. So it is
// one launch without a grid-wide step: every block computes the three prefix
// sums over all requests for itself (in shared memory, 12 bytes a request;
// the lengths come from L2), and then takes its share of the flattened list
// of tokens, new pages and returned pages, each found by bisection. 256 decodes
// take 4.4 us, 4096 requests with prompt chunks among them (341000 tokens) 9.5
// (about 1 us more with one block an SM instead of two, and 1 more with a scan over
// the whole block instead of one a warp).
#include <algorithm>

#include "fa_device.cuh"
#include "fa_internal.h"
#include "paged_launch.cuh"

namespace fa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr unsigned kMost = 0x7fffffffu;  // where sums stop (bad lengths can pass 32 bits)

// Tokens of the packed batch (whatever becomes of them), pages to take from
// the ring and pages to return to it.
struct Len3 {
    unsigned v[3];
    bool bad;  // lengths out of range: no pages
};

__device__ __forceinline__ Len3 plan_len(const PlanArgs &a, int c, int f) {
    Len3 p{{f > 0 ? static_cast<unsigned>(f) : 0u, 0u, 0u}, false};
    const long long rows = static_cast<long long>(c) + p.v[0];
    p.bad = c < 0 || f < -1 || rows > static_cast<long long>(a.max_pages) << a.page_shift;
    if (p.bad) return p;
    const unsigned mask = (1u << a.page_shift) - 1u;  // rows and the table's rows are below 2^30
    const unsigned used = (static_cast<unsigned>(c) + mask) >> a.page_shift;
    if (f < 0)
        p.v[2] = used;
    else
        p.v[1] = ((static_cast<unsigned>(rows) + mask) >> a.page_shift) - used;
    return p;
}

// a + b, at most kMost (both are): sums that stop there can be taken in any order.
__device__ __forceinline__ unsigned add(unsigned a, unsigned b) { return min(a + b, kMost); }

__device__ __forceinline__ unsigned warp_scan(unsigned x) {  // inclusive
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned o = __shfl_up_sync(~0u, x, d);
        if ((threadIdx.x & 31) >= d) x = add(x, o);
    }
    return x;
}

// The last index r < n with start[r] <= x (start[0] = 0 <= x).
__device__ __forceinline__ int find(const int *start, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads, 2) page_plan_kernel(PlanArgs a) {
    wait_for_stream();
    extern __shared__ int sm[];
    int *tok0 = sm, *need0 = sm + a.n_reqs + 1, *back0 = need0 + a.n_reqs + 1;
    const int R = a.n_reqs, N = a.n_pages;
    int head = load(a.state), count = load(a.state + 1);
    const bool bad_ring = head < 0 || head >= N || count < 0 || count > N;
    if (bad_ring) head = count = 0;  // hand out nothing, take nothing back
    // Each warp takes a run of requests, 32 at a time, and leaves the sums before
    // each of them within its run; then the runs before it are added.
    __shared__ unsigned part[3][kPlanWarps];
    __shared__ unsigned taken_sh;
    __shared__ int bad_sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = ((R + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32;
    const int r0 = min(R, warp * per), r1 = min(R, r0 + per);
    if (threadIdx.x == 0) taken_sh = 0, bad_sh = 0;
    int *const sums[3] = {tok0, need0, back0};
    unsigned run[3] = {0, 0, 0};
    bool bad = false;
#pragma unroll 4
    for (int b = r0; b < r1; b += 32) {
        const int r = b + lane;
        Len3 p{{0, 0, 0}, false};
        if (r < r1) p = plan_len(a, load(a.cached + r), load(a.fresh + r));
        bad |= p.bad;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const unsigned inc = warp_scan(min(p.v[k], kMost));
            // exclusive: the inclusive sum of the lane before
            const unsigned ex = __shfl_up_sync(~0u, inc, 1);
            if (r < r1) sums[k][r] = static_cast<int>(add(run[k], lane ? ex : 0u));
            run[k] = add(run[k], __shfl_sync(~0u, inc, 31));
        }
    }
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < 3; ++k) part[k][warp] = run[k];
    __syncthreads();
    if (bad) bad_sh = 1;
    unsigned all[3], before[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const unsigned inc = warp_scan(part[k][lane]);
        all[k] = __shfl_sync(~0u, inc, 31);
        before[k] = warp ? __shfl_sync(~0u, inc, warp - 1) : 0u;
    }
    const unsigned room = static_cast<unsigned>(a.max_tokens);
    for (int r = r0 + lane; r < r1; r += 32) {
        tok0[r] = static_cast<int>(min(add(tok0[r], before[0]), room));
        need0[r] = static_cast<int>(add(need0[r], before[1]));
        back0[r] = static_cast<int>(add(back0[r], before[2]));
    }
    if (threadIdx.x == 0) {
        tok0[R] = static_cast<int>(min(all[0], room));
        need0[R] = static_cast<int>(all[1]);
        back0[R] = static_cast<int>(all[2]);
    }
    __syncthreads();
    // a request of `fresh` tokens that are not all below max_tokens (then none behind it that has some are)
    auto cut = [&](int r, unsigned fresh) { return fresh > room - static_cast<unsigned>(tok0[r]); };
    // one that gets its slots: its pages are left, and none of its tokens is cut off
    auto fits = [&](int r, const Len3 &p) {
        return !p.bad && (p.v[1] == 0 || need0[r + 1] <= count) && !cut(r, p.v[0]);
    };
    // the pages handed out: those of the requests that fit
    unsigned fits_to = 0;
    for (int r = threadIdx.x; r < R; r += kPlanThreads)
        if (need0[r + 1] > need0[r] && need0[r + 1] <= count &&
            !(all[0] > room && cut(r, static_cast<unsigned>(load(a.fresh + r)))))
            fits_to = max(fits_to, static_cast<unsigned>(need0[r + 1]));
    fits_to = __reduce_max_sync(~0u, fits_to);
    if (lane == 0 && fits_to) atomicMax(&taken_sh, fits_to);
    __syncthreads();
    const int taken = static_cast<int>(taken_sh);
    const int returned = bad_ring ? 0 : min(back0[R], N - count);
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0 && (bad_sh || bad_ring || back0[R] > returned || all[0] > room))
            flag_error(a.err, FA_ERRBIT_DEVICE);
        if (threadIdx.x == 0) {
            const int next = head + taken;
            a.state_out[0] = next >= N ? next - N : next;
            a.state_out[1] = count - taken + returned;
            a.state_out[2] = need0[R] - taken;
            a.cu_fresh[R] = tok0[R];
        }
    }
    const int i0 = blockIdx.x * kPlanThreads + threadIdx.x, step = gridDim.x * kPlanThreads;
    for (int r = i0; r < R; r += step) {
        const int c = load(a.cached + r), f = load(a.fresh + r);
        const Len3 p = plan_len(a, c, f);
        a.seq_lens[r] = p.bad || f < 0 ? 0 : fits(r, p) ? c + static_cast<int>(p.v[0]) : c;
        a.cu_fresh[r] = tok0[r];
    }
    const int mask = (1 << a.page_shift) - 1;
    auto ring_at = [&](int i) {  // head + i around the ring (i < N)
        const unsigned k = static_cast<unsigned>(head) + static_cast<unsigned>(i);
        return static_cast<int>(k >= static_cast<unsigned>(N) ? k - N : k);
    };
    for (int t = i0; t < a.max_tokens; t += step) {
        int slot = -1, pos = 0;
        if (t < tok0[R]) {
            const int r = find(tok0, R, t);
            const int c = load(a.cached + r);
            const Len3 p = plan_len(a, c, load(a.fresh + r));
            if (!p.bad) {
                pos = c + (t - tok0[r]);
                if (fits(r, p)) {
                    const int k = pos >> a.page_shift;
                    const int used = (c + mask) >> a.page_shift;
                    const int page =
                        k < used ? a.block_table[static_cast<size_t>(r) * a.max_pages + k]
                                 : a.ring[ring_at(need0[r] + k - used)];
                    if (page >= 0 && page < N)
                        slot = (page << a.page_shift) + (pos & mask);
                    else
                        flag_error(a.err, FA_ERRBIT_DEVICE);
                }
            }
        }
        a.slot_map[t] = slot;
        a.positions[t] = pos;
    }
    for (int i = i0; i < taken; i += step) {
        const int r = find(need0, R, i);
        const int used = (load(a.cached + r) + mask) >> a.page_shift;
        a.block_table[static_cast<size_t>(r) * a.max_pages + used + (i - need0[r])] =
            a.ring[ring_at(i)];
    }
    for (int i = i0; i < returned; i += step) {
        const int r = find(back0, R, i);
        a.ring[ring_at(count + i)] =
            a.block_table[static_cast<size_t>(r) * a.max_pages + (i - back0[r])];
    }
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs &a, cudaStream_t stream) {
    const size_t smem = 3 * (static_cast<size_t>(a.n_reqs) + 1) * sizeof(int);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(
            page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    const int items = std::max(a.max_tokens, a.n_reqs);
    const int blocks = std::min(2 * device_sm_count(), (items + kPlanThreads - 1) / kPlanThreads);
    return launch_after(page_plan_kernel, dim3(std::max(blocks, 1)), kPlanThreads, smem, stream, a);
}

}  // namespace fa
