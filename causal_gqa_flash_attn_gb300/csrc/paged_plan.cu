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
// of tokens, new pages and returned pages, each found by bisection.
#include <algorithm>

#include "fa_device.cuh"
#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;

struct PlanLen {
    long long tokens;  // fresh tokens (in the packed batch, whatever becomes of them)
    int need, back;    // pages to take from the ring, pages to return to it
    bool bad;          // lengths out of range
};

__device__ __forceinline__ PlanLen plan_len(const PlanArgs &a, int r) {
    const int c = __ldg(a.cached + r), f = __ldg(a.fresh + r);
    PlanLen p{f > 0 ? f : 0, 0, 0, false};
    const long long rows = static_cast<long long>(c) + p.tokens;
    p.bad = c < 0 || f < -1 || rows > static_cast<long long>(a.max_pages) << a.page_shift;
    if (p.bad) return p;
    const int used = static_cast<int>((c + (1ll << a.page_shift) - 1) >> a.page_shift);
    if (f < 0)
        p.back = used;
    else
        p.need = static_cast<int>((rows + (1ll << a.page_shift) - 1) >> a.page_shift) - used;
    return p;
}

// Inclusive scan of three values over the block; returns this thread's
// exclusive sums and the block totals.
struct Sum3 {
    long long v[3];
};
__device__ __forceinline__ Sum3 block_scan(Sum3 mine, Sum3 *total) {
    __shared__ long long part[3][kPlanWarps];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    Sum3 inc = mine;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(~0u, inc.v[k], d);
            if (lane >= d) inc.v[k] += o;
        }
        if (lane == 31) part[k][w] = inc.v[k];
    }
    __syncthreads();
    Sum3 ex;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        long long base = 0, all = 0;
#pragma unroll
        for (int i = 0; i < kPlanWarps; ++i) {
            if (i == w) base = all;
            all += part[k][i];
        }
        ex.v[k] = base + inc.v[k] - mine.v[k];
        total->v[k] = all;
    }
    return ex;
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

__device__ __forceinline__ int clip(long long x, int most) {
    return static_cast<int>(x < most ? x : most);
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(PlanArgs a) {
    extern __shared__ int sm[];
    int *tok0 = sm, *need0 = sm + a.n_reqs + 1, *back0 = need0 + a.n_reqs + 1;
    const int R = a.n_reqs, N = a.n_pages;
    // each thread sums a run of requests
    const int per = (R + kPlanThreads - 1) / kPlanThreads;
    const int r0 = min(R, static_cast<int>(threadIdx.x) * per), r1 = min(R, r0 + per);
    int head = __ldg(a.state), count = __ldg(a.state + 1);
    const bool bad_ring = head < 0 || head >= N || count < 0 || count > N;
    if (bad_ring) head = count = 0;  // hand out nothing, take nothing back
    Sum3 mine{{0, 0, 0}}, total;
    for (int r = r0; r < r1; ++r) {
        const PlanLen p = plan_len(a, r);
        mine.v[0] += p.tokens;
        mine.v[1] += p.need;
        mine.v[2] += p.back;
    }
    Sum3 at = block_scan(mine, &total);
    const int most = 0x7fffffff;
    bool bad = false;
    for (int r = r0; r < r1; ++r) {
        const PlanLen p = plan_len(a, r);
        bad |= p.bad;
        tok0[r] = clip(at.v[0], a.max_tokens);
        need0[r] = clip(at.v[1], most);
        back0[r] = clip(at.v[2], most);
        at.v[0] += p.tokens;
        at.v[1] += p.need;
        at.v[2] += p.back;
    }
    // the pages handed out: those of the requests whose whole need is left
    __shared__ int taken_sh;
    if (threadIdx.x == 0) {
        tok0[R] = clip(total.v[0], a.max_tokens);
        need0[R] = clip(total.v[1], most);
        back0[R] = clip(total.v[2], most);
        taken_sh = 0;
    }
    __syncthreads();
    for (int r = r0; r < r1; ++r)
        if (need0[r + 1] > need0[r] && need0[r + 1] <= count) atomicMax(&taken_sh, need0[r + 1]);
    __syncthreads();
    const int taken = taken_sh;
    const int returned = bad_ring ? 0 : min(back0[R], N - count);
    if (blockIdx.x == 0) {
        if (bad || (threadIdx.x == 0 &&
                    (bad_ring || back0[R] > returned || total.v[0] > a.max_tokens)))
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
        const int c = __ldg(a.cached + r);
        const PlanLen p = plan_len(a, r);
        const bool fits = !p.bad && (p.need == 0 || need0[r + 1] <= count);
        a.seq_lens[r] = p.bad || __ldg(a.fresh + r) < 0 ? 0
                        : fits ? c + static_cast<int>(p.tokens) : c;
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
            const PlanLen p = plan_len(a, r);
            const int c = __ldg(a.cached + r);
            if (!p.bad) {
                pos = c + (t - tok0[r]);
                if (p.need == 0 || need0[r + 1] <= count) {
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
        const int used = (__ldg(a.cached + r) + mask) >> a.page_shift;
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
    const int blocks = std::min(device_sm_count(), (items + kPlanThreads - 1) / kPlanThreads);
    page_plan_kernel<<<std::max(blocks, 1), kPlanThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace fa
