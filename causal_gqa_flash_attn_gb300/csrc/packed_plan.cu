// packed_plan.cu -- the tiles of a packed batch, heaviest first, and the work
// counters of the kernels that walk them (include/fa.h, fa_packed_attn).
//
// A block for each list. Documents are summed (tiles before each of them), then the tiles are
// counted into bins of their number of key tiles (or row tiles, for a tile of keys)
// and put into the lists from the heaviest bin on. Within a bin the order may differ
// from call to call: units do not depend on each other, so that no result does.
//
// A tile of keys whose rows are many (the first keys of a long document are seen by all of it) is
// cut into pieces, so that a few such tiles do not keep a few SMs busy alone; their sums are
// added in the order of the pieces.
//
// Bound by latency: a launch, dependent reads and shared atomics (7 us of 23 documents),
// of which the kernel behind it hides its start. Batches of up to 32 documents whose units all have
// an SM go without (direct_tile).
#include "packed_common.cuh"

namespace fa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBins = 1024;
constexpr int kDocsInSmem = 2048;

// Sums of a, b, c over the threads before this one, and over all.
__device__ __forceinline__ void scan3(int &a, int &b, int &c, int *sum, int (*part)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int v[3] = {a, b, c}, own[3] = {a, b, c};
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int o = __shfl_up_sync(~0u, v[k], d);
            if (lane >= d) v[k] += o;
        }
    if (lane == 31)
        for (int k = 0; k < 3; ++k) part[k][warp] = v[k];
    __syncthreads();
    if (warp < 3) {
        int x = part[warp][lane], s = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(~0u, s, d);
            if (lane >= d) s += o;
        }
        part[warp][lane] = s - x;
        if (lane == 31) sum[warp] = s;
    }
    __syncthreads();
    a = v[0] - own[0] + part[0][warp];
    b = v[1] - own[1] + part[1][warp];
    c = v[2] - own[2] + part[2][warp];
}

// The document that holds tile x: the last one with before[d] <= x that has tiles.
__device__ __forceinline__ int find_doc(const int *before, int n, int x) {
    int lo = 0, hi = n;  // before[lo] <= x < before[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(PackedPlanArgs a) {
    wait_for_stream();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the next kernel sets itself up meanwhile
    __shared__ int part[3][32], sum[3];
    __shared__ int bins[kBins];
    __shared__ int small[3][kDocsInSmem + 1], cu_s[kDocsInSmem + 1];
    __shared__ int bad_docs, n_slots;
    __shared__ unsigned long long all_rows;
    const int tid = threadIdx.x, D = a.n_docs, list = blockIdx.x;
    const bool fits = D <= kDocsInSmem;
    int *before[3];
    for (int k = 0; k < 3; ++k) before[k] = fits ? small[k] : a.doc_tiles + static_cast<size_t>(3 * list + k) * (D + 1);
    if (tid == 0) bad_docs = 0;
    if (fits)
        for (int d = tid; d <= D; d += kPlanThreads) cu_s[d] = load(a.cu + d);
    const int32_t *cu = fits ? cu_s : a.cu;
    if (list == 0 && tid < 4) a.header->counters[tid] = 0;
    if (list == 1)
        for (int i = tid; i < a.slots; i += kPlanThreads) a.arrived[i] = 0;
    __syncthreads();

    // ---- tiles before each document: a thread sums a run of documents
    const int per = (D + kPlanThreads - 1) / kPlanThreads;
    const int d0 = min(D, tid * per), d1 = min(D, d0 + per);
    int nr = 0, nk = 0, nb = 0;
    bool bad = false;
    auto length = [&](int d) {
        const int from = cu[d], to = cu[d + 1];
        if (from < 0 || to < from || to > a.n_tokens) {
            bad = true;
            return 0;
        }
        return to - from;
    };
    auto tiles = [&](int n, int *r, int *k, int *b) {
        *r = (n + a.row_tokens - 1) / a.row_tokens;
        *k = a.most_keys ? (n + 127) / 128 : 0;
        *b = (n + (1 << a.block_tokens_log) - 1) >> a.block_tokens_log;
    };
    for (int d = d0; d < d1; ++d) {
        int r, k, b;
        tiles(length(d), &r, &k, &b);
        nr += r, nk += k, nb += b;
        if (list == 0 && a.doc_most) a.doc_most[d] = a.doc_most[D + d] = 0u;
    }
    if (bad) bad_docs = 1;
    scan3(nr, nk, nb, sum, part);
    for (int d = d0; d < d1; ++d) {
        before[0][d] = nr, before[1][d] = nk, before[2][d] = nb;
        int r, k, b;
        tiles(length(d), &r, &k, &b);
        nr += r, nk += k, nb += b;
    }
    if (tid == 0)
        for (int k = 0; k < 3; ++k) before[k][D] = sum[k];
    __syncthreads();
    // documents that overlap (cu decreases) could have more tiles than there is room for
    const bool wrong = bad_docs || sum[0] > a.most_rows || sum[1] > a.most_keys;
    if (wrong && tid == 0) flag_error(a.err, FA_ERRBIT_DEVICE);
    const int n = wrong ? 0 : sum[list];

    PackedTile *out = list ? a.keys : a.rows;
    const int room = list ? a.most_keys : a.most_rows;
    // tile x, and how many tiles move past it
    auto tile = [&](int x, PackedTile *t) {
        const int d = find_doc(before[list], D, x);
        t->tok0 = cu[d];
        t->len = cu[d + 1] - t->tok0;
        t->p0 = (x - before[list][d]) * (list ? 128 : a.row_tokens);
        t->prefix = a.prefix ? min(max(load(a.prefix + d), 0), t->len) : 0;
        t->rb = before[2][d];
        t->doc = d;
        t->head = t->from = t->piece = 0;
        t->pieces = 1;
        t->slot = -1;
        if (list) {
            int first, last;
            query_range(t->p0, min(t->p0 + 128, t->len) - 1, t->len, t->prefix, a.sink, a.win, &first, &last);
            t->from = first / a.step_tokens;
            t->rows = last / a.step_tokens - t->from + 1;
        } else {
            const int p1 = min(t->p0 + a.row_tokens, t->len) - 1;
            t->rows = a.key_tile == 64 ? key_tiles<64>(t->p0, p1, t->prefix, a.sink, a.win).count
                                       : key_tiles<128>(t->p0, p1, t->prefix, a.sink, a.win).count;
        }
    };
    // few tiles: each thread makes its own once
    const bool once = n <= kPlanThreads;
    PackedTile t;
    if (once && tid < n) tile(tid, &t);
    // the largest piece: at first 1 / parts of all row tiles, then what there is room for
    int most = 1 << 30;
    if (list && a.slots > 0 && n > 0) {
        if (tid == 0) all_rows = 0;
        __syncthreads();
        unsigned long long mine = 0;
        for (int x = tid; x < n; x += kPlanThreads) {
            if (!once) tile(x, &t);
            mine += t.rows;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(~0u, mine, d);
        if ((tid & 31) == 0 && mine > 0) atomicAdd(&all_rows, mine);
        __syncthreads();
        const unsigned long long each = (all_rows * a.n_kv + a.parts - 1) / a.parts;
        most = max(kPackedLeastPiece, static_cast<int>(min(each, 1ull << 30)));
    }
    auto pieces_of = [&](int rows) { return rows > most ? (rows + most - 1) / most : 1; };
    int entries = n;
    while (list && a.slots > 0 && n > 0) {
        if (tid == 0) n_slots = 0;
        int need = 0, more = 0, zero = 0;
        for (int x = tid; x < n; x += kPlanThreads) {
            if (!once) tile(x, &t);
            const int p = pieces_of(t.rows);
            more += p - 1;
            if (p > 1) need += p;
        }
        scan3(need, more, zero, sum, part);
        const bool fits = static_cast<long long>(sum[0]) * a.n_kv <= a.slots && n + sum[1] <= room;
        entries = n + sum[1];
        __syncthreads();
        if (fits) break;
        most *= 2;
    }
    if (tid == 0) (list ? a.header->key_tiles : a.header->row_tiles) = entries;
    if (n == 0) return;
    int shift = 0;  // bins of a power of two of tiles
    const int step = list ? a.step_tokens : a.key_tile;
    while ((a.n_tokens / step + 1) >> shift >= kBins) ++shift;
    auto bin_of = [&](int rows) { return kBins - 1 - min(rows >> shift, kBins - 1); };  // heaviest first
    for (int i = tid; i < kBins; i += kPlanThreads) bins[i] = 0;
    __syncthreads();
    // the pieces of a tile differ by one row tile at most, and share a bin
    for (int x = tid; x < n; x += kPlanThreads) {
        if (!once) tile(x, &t);
        const int p = pieces_of(t.rows);
        atomicAdd(&bins[bin_of((t.rows + p - 1) / p)], p);
    }
    __syncthreads();
    static_assert(kBins == kPlanThreads, "a bin for each thread");
    int at = bins[tid], z0 = 0, z1 = 0;
    scan3(at, z0, z1, sum, part);
    bins[tid] = at;
    __syncthreads();
    for (int x = tid; x < n; x += kPlanThreads) {
        if (!once) tile(x, &t);
        const int p = pieces_of(t.rows), rows = t.rows, from = t.from;
        const int place = atomicAdd(&bins[bin_of((rows + p - 1) / p)], p);
        t.pieces = p;
        if (p > 1) t.slot = atomicAdd(&n_slots, p * a.n_kv);
        for (int k = 0; k < p; ++k) {
            const int r0 = static_cast<int>(static_cast<long long>(rows) * k / p);
            t.piece = k;
            t.from = from + r0;
            t.rows = static_cast<int>(static_cast<long long>(rows) * (k + 1) / p) - r0;
            out[place + k] = t;
        }
    }
}

}  // namespace

cudaError_t launch_packed_plan(const PackedPlanArgs &a, cudaStream_t stream) {
    return launch_after(packed_plan_kernel, dim3(a.most_keys ? 2 : 1), kPlanThreads, 0, stream, a);
}

}  // namespace fa
