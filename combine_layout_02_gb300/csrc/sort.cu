// sort.cu -- rows into expert order and back, with the gradients of both directions.
//
// Placement (ep_sort_layout): a stable counting sort of the N*k entries by expert. Entries
// are cut into segments, one per warp, in order. A segment's rows of expert e start at
//   sum over e' < e of all entries of e'  +  sum over earlier segments of their entries of e
// and within a segment a warp takes 32 entries at a time: an entry's rank among them is the
// number of lower lanes with the same expert (__match_any_sync), on top of the warp's running
// count in shared memory. Counts only, no global atomics: the placement is the same in every
// run. These kernels let the next one launch as soon as it has itself waited (the next waits for
// its end before it reads): the launch is then over by that end. Few entries: one block does all
// of it (sort_small_kernel). More: count, scan (one block per expert over the segments' counts)
// and place, three kernels without any inter-block wait.
//
// Rows (ep_sort_rows, ep_unsort_rows, ep_unsort_rows_backward): one warp per row in row order,
// its placed entries' sorted rows as destinations or sources, as in the expert-major dispatch
// and combine. Everything is bound by memory: each row is read once and each sorted row written
// (or read) once. 21673 rows of 7168 bf16 channels, 1.34 entries a row: placement 9 us beside
// its launches, rows 103 us (666 MB, 6.5 TB/s), back 116 us (6.2); both gradients of 16384 rows
// of 4096, top-6 of 128 experts: 261 us (1.75 GB, 6.7 TB/s) and 136 us for the rows' own.
#include "rowops.cuh"
#include "sort.cuh"

namespace ep {
namespace {

constexpr int kSortWarps = 8;                  // warps per block of the count / place kernels
// Up to here one block sorts everything, in less time than three kernels or hardly more, 1 to 8192 experts (us, one
// block and three: 8 experts, 5120 entries 5.9 and 6.3; 64, 4096 8.0 and 7.7, 5120 9.0 and 7.7, 8192 12.0 and 8.6; 256,
// 5120 10.4 and 10.6, 8192 14.0 and 11.5; 1024, 5120 11.9 and 24; 4096, 5120 27 and 43; 8192, where the table has
// room for one warp, 2048 33 and 58, 5120 71 and 65).
constexpr int kSmallEntries = 5120;
constexpr int kSmallThreads = 1024;
constexpr int kTableInts = 48 * 1024 / 4;      // per-warp counts of a block, in shared memory
constexpr int kSortSmemMax = (kTableInts + EP_MAX_EXPERTS + 8) * 4;
constexpr size_t kSmemPlain = 40 * 1024;       // dynamic shared memory without opting in: 48 KB with the static
constexpr int kSegment = 128;                  // entries per segment, at least
constexpr int kMaxSegments = 152 * 16;

struct SortArgs {
    const int64_t* topk_idx;
    int32_t* entry_rows;      // nullable
    int32_t* row_entries;     // nullable
    int32_t* expert_prefix;
    int32_t* ws;              // [E][S] segment counts ([S] of changes), then [E] totals
    int64_t num_rows;
    int n, E, S, seg_len, warps;
    int rest;                 // bucket of ids that are none of [0, E), or -1 to leave them out
    int32_t* changes;         // nullable: how many entries differ from the one before
    uint32_t bad_bit;
    uint32_t* err;
};

// Segments of a sort of n entries: seg_len entries each (a multiple of 32).
inline int segment_length(int64_t n) {
    int64_t len = (n + kMaxSegments - 1) / kMaxSegments;
    len = (len + 31) / 32 * 32;
    return (int)(len < kSegment ? kSegment : len);
}

// Warps a block's count table has room for.
inline int table_warps(int E, int most) {
    const int w = kTableInts / E;
    return w < 1 ? 1 : w < most ? w : most;
}

// An entry's expert, or -1 if masked or out of range (flagged).
__device__ __forceinline__ int entry_expert(const SortArgs& a, int64_t e, bool flag) {
    if (e >= 0 && e < (a.rest < 0 ? a.E : a.rest)) return (int)e;
    if (flag && e != -1) raise_flag(a.err, a.bad_bit);
    return a.rest;
}

// A lane's entries of the next kAhead times 32 of a segment, all loaded before the first is used (one after
// another, their latency is what a sort of a few thousand entries takes); -1 past the end.
constexpr int kAhead = 8;
__device__ __forceinline__ void load_entries(const SortArgs& a, int i0, int end, int lane, int64_t (&v)[kAhead]) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) v[u] = i0 + u * 32 + lane < end ? a.topk_idx[i0 + u * 32 + lane] : -1;
}

// One warp: counts its segment's entries per expert into its (zeroed) table. Returns, if asked for,
// this lane's share of the entries that differ from the one before.
__device__ __forceinline__ int count_segment(const SortArgs& a, int seg, int* table, int lane) {
    const int begin = seg * a.seg_len, end = min(a.n, begin + a.seg_len);
    int changes = 0, before = -2;          // lane 0's: the entry before these 32
    if (a.changes != nullptr && begin > 0 && begin < end) before = entry_expert(a, a.topk_idx[begin - 1], false);
    for (int i0 = begin; i0 < end; i0 += kAhead * 32) {
        int64_t v[kAhead];
        load_entries(a, i0, end, lane, v);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * 32 + lane, e = entry_expert(a, v[u], true);
            if (i < end && e >= 0) atomicAdd(&table[e], 1);      // shared memory; a count, so order is immaterial
            if (a.changes != nullptr) {
                const int up = __shfl_up_sync(0xFFFFFFFFu, e, 1);
                changes += i < end && i > 0 && (lane > 0 ? up : before) != e;
                before = __shfl_sync(0xFFFFFFFFu, e, 31);
            }
        }
    }
    return changes;
}

// One warp: places its segment's entries; table[e] holds the segment's first row of expert e.
__device__ __forceinline__ void place_segment(const SortArgs& a, int seg, int* table, int lane) {
    const int begin = seg * a.seg_len, end = min(a.n, begin + a.seg_len);
    for (int i0 = begin; i0 < end; i0 += kAhead * 32) {
        int64_t v[kAhead];
        load_entries(a, i0, end, lane, v);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (i0 + u * 32 >= end) break;
            const int i = i0 + u * 32 + lane, e = i < end ? entry_expert(a, v[u], false) : -1;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
            int row = -1;
            if (e >= 0) row = table[e] + __popc(same & lanemask_lt());
            __syncwarp();
            if (e >= 0 && (same & lanemask_lt()) == 0) table[e] += __popc(same);
            __syncwarp();
            if (i < end) {
                if (row >= a.num_rows) {
                    raise_flag(a.err, EP_DEVERR_RECV_OVERFLOW);
                    row = -1;
                }
                if (a.entry_rows != nullptr) a.entry_rows[i] = row;
                if (row >= 0 && a.row_entries != nullptr) a.row_entries[row] = i;
            }
        }
    }
}

// Block-wide: v[0..E) counts -> exclusive prefix in place (shared memory); returns the sum.
// Each thread scans a run of ceil(E / threads) values, then the runs' sums are scanned.
__device__ __forceinline__ int block_exclusive_scan(int* v, int E) {
    __shared__ int warp_sums[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
    const int per = (E + blockDim.x - 1) / blockDim.x;
    const int lo = min(E, (int)threadIdx.x * per), hi = min(E, lo + per);
    int sum = 0;
    for (int e = lo; e < hi; ++e) sum += v[e];
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int s = lane < nwarps ? warp_sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s += up;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    int run = inc - sum + (warp > 0 ? warp_sums[warp - 1] : 0);
    for (int e = lo; e < hi; ++e) {
        const int c = v[e];
        v[e] = run;
        run += c;
    }
    const int total = warp_sums[nwarps - 1];
    __syncthreads();
    return total;
}

// Every entry in one block: a.warps warps with one segment each.
__global__ void __launch_bounds__(kSmallThreads) sort_small_kernel(SortArgs a) {
    extern __shared__ int smem[];
    int* first = smem;                 // [E]
    int* tables = smem + a.E;          // [warps][E]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < a.warps * a.E; i += blockDim.x) tables[i] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int changes = warp < a.warps ? count_segment(a, warp, tables + warp * a.E, lane) : 0;
    __shared__ int s_changes;
    if (threadIdx.x == 0) s_changes = 0;
    __syncthreads();
    if (a.changes != nullptr && changes > 0) atomicAdd(&s_changes, changes);
    __syncthreads();
    if (a.changes != nullptr && threadIdx.x == 0) *a.changes = s_changes;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int run = 0;
        for (int w = 0; w < a.warps; ++w) {
            const int c = tables[w * a.E + e];
            tables[w * a.E + e] = run;
            run += c;
        }
        first[e] = run;
    }
    __syncthreads();
    const int total = block_exclusive_scan(first, a.E);
    for (int i = threadIdx.x; i < a.warps * a.E; i += blockDim.x) tables[i] += first[i % a.E];
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.expert_prefix[e] = e < a.E ? first[e] : total;
    __syncthreads();
    if (warp < a.warps) place_segment(a, warp, tables + warp * a.E, lane);
}

__global__ void __launch_bounds__(kSortWarps * 32) sort_count_kernel(SortArgs a) {
    extern __shared__ int tables[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < a.warps * a.E; i += blockDim.x) tables[i] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int seg0 = blockIdx.x * a.warps;
    if (warp < a.warps && seg0 + warp < a.S) {
        const int changes = warp_sum(count_segment(a, seg0 + warp, tables + warp * a.E, lane));
        if (a.changes != nullptr && lane == 0) a.ws[(int64_t)a.E * a.S + seg0 + warp] = changes;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.warps * a.E; i += blockDim.x) {
        const int e = i / a.warps, w = i - e * a.warps;
        if (seg0 + w < a.S) a.ws[(int64_t)e * a.S + seg0 + w] = tables[w * a.E + e];
    }
}

// One block per expert: its segments' counts -> exclusive prefix in place, and their total (one block
// more for the changes, which stand like an expert's after the last one's). A thread has a run of
// up to kRun counts, all loaded before the first is used.
__global__ void __launch_bounds__(kSortWarps * 32) sort_scan_kernel(SortArgs a) {
    constexpr int kRun = (kMaxSegments + kSortWarps * 32 - 1) / (kSortWarps * 32);
    __shared__ int s_sum[kSortWarps];
    const int e = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const int columns = a.E + (a.changes != nullptr);
    int32_t* v = a.ws + (int64_t)e * a.S;
    const int per = (a.S + kSortWarps * 32 - 1) / (kSortWarps * 32), first = threadIdx.x * per;
    int c[kRun], sum = 0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) c[i] = i < per && first + i < a.S ? v[first + i] : 0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) sum += c[i];
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += up;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    int run = upto - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        if (w < warp) run += s_sum[w];
        total += s_sum[w];
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        if (i < per && first + i < a.S) v[first + i] = run;
        run += c[i];
    }
    if (threadIdx.x == 0) {
        if (e < a.E) a.ws[(int64_t)columns * a.S + e] = total;
        else *a.changes = total;
    }
}

__global__ void __launch_bounds__(kSortWarps * 32) sort_place_kernel(SortArgs a) {
    extern __shared__ int smem[];
    int* first = smem;                 // [E]
    int* tables = smem + a.E;          // [warps][E]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const int seg0 = blockIdx.x * a.warps;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x)
        first[e] = a.ws[(int64_t)(a.E + (a.changes != nullptr)) * a.S + e];
    for (int i = threadIdx.x; i < a.warps * a.E; i += blockDim.x) {
        const int e = i / a.warps, w = i - e * a.warps;
        tables[w * a.E + e] = seg0 + w < a.S ? a.ws[(int64_t)e * a.S + seg0 + w] : 0;
    }
    __syncthreads();
    const int total = block_exclusive_scan(first, a.E);
    for (int i = threadIdx.x; i < a.warps * a.E; i += blockDim.x) tables[i] += first[i % a.E];
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.expert_prefix[e] = e < a.E ? first[e] : total;
    __syncthreads();
    if (warp < a.warps && seg0 + warp < a.S) place_segment(a, seg0 + warp, tables + warp * a.E, lane);
}

// ------------------------------------------------------------------ rows

constexpr int kRowWarps = 4;

struct RowArgs {
    const char* x;
    const char* x_scales;      // nullable
    const float* topk_weights; // nullable: 1
    const int32_t* entry_rows;
    const char* y;
    char* out;
    char* out_scales;
    const char* dout;
    char* dy;                  // nullable
    float* dweights;           // nullable
    int64_t num_rows;
    int N, H, k;
    uint32_t row_bytes, scale_bytes;
    uint32_t* err;
};

// Sorted rows (and coefficients, and entry indices) of row t's placed entries, ascending j.
__device__ __forceinline__ int placed_rows(const RowArgs& a, int64_t t, int lane, int64_t* s_row, float* s_coef,
                                           int* s_entry) {
    int64_t row = -1;
    float w = 1.0f;
    if (lane < a.k) {
        row = a.entry_rows[t * a.k + lane];
        if (a.topk_weights != nullptr) w = a.topk_weights[t * a.k + lane];
        if (row >= a.num_rows) {
            raise_flag(a.err, EP_DEVERR_RECV_OVERFLOW);
            row = -1;
        }
    }
    const unsigned bal = __ballot_sync(0xFFFFFFFFu, row >= 0);
    if (row >= 0) {
        const int p = __popc(bal & lanemask_lt());
        s_row[p] = row;
        if (s_coef != nullptr) s_coef[p] = w;
        if (s_entry != nullptr) s_entry[p] = lane;
    }
    return __popc(bal);
}

// The e4m3 row's scales to every destination.
__device__ __forceinline__ void copy_scales(const RowArgs& a, int64_t t, const int64_t* rows, int nd, int lane) {
    if (a.x_scales == nullptr) return;
    const char* src = a.x_scales + t * a.scale_bytes;
    if ((a.scale_bytes & 3) == 0 && (((uintptr_t)a.x_scales | (uintptr_t)a.out_scales) & 3) == 0) {
        for (uint32_t i = lane * 4; i < a.scale_bytes; i += 128) {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(src + i);
            for (int p = 0; p < nd; ++p) *reinterpret_cast<uint32_t*>(a.out_scales + rows[p] * a.scale_bytes + i) = v;
        }
    } else {
        for (uint32_t i = lane; i < a.scale_bytes; i += 32) {
            const char v = src[i];
            for (int p = 0; p < nd; ++p) a.out_scales[rows[p] * a.scale_bytes + i] = v;
        }
    }
}

// Bulk copies: one load of the row into shared memory, one store per placed entry.
__global__ void __launch_bounds__(kTmaWarps * 32) sort_rows_tma_kernel(RowArgs a) {
    extern __shared__ __align__(128) unsigned char rowbuf[];
    __shared__ int64_t s_row[kTmaWarps][EP_MAX_TOPK];
    __shared__ __align__(8) uint64_t s_bar[kTmaWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned char* buf = rowbuf + (size_t)warp * a.row_bytes;
    const int64_t nw = (int64_t)gridDim.x * kTmaWarps;
    if (lane == 0) mbar_init(&s_bar[warp], 1);
    __syncwarp();
    pdl_wait();
    uint32_t parity = 0;
    bool live = true;       // lane 0: false once a row load failed to land in time
    for (int64_t t = (int64_t)blockIdx.x * kTmaWarps + warp; t < a.N; t += nw) {
        if (lane == 0 && live) tma_row_load(buf, a.x + t * (int64_t)a.row_bytes, a.row_bytes, &s_bar[warp]);
        const int nd = placed_rows(a, t, lane, s_row[warp], nullptr, nullptr);
        __syncwarp();
        copy_scales(a, t, s_row[warp], nd, lane);
        if (lane == 0 && live)
            live = tma_row_store(buf, a.out, s_row[warp], nd, a.row_bytes, &s_bar[warp], parity, a.err);
        __syncwarp();
    }
    if (lane == 0) bulk_wait_all();
    pdl_trigger();
}

// Rows too wide for the shared-memory buffers: 16-byte vector copies.
__global__ void __launch_bounds__(kRowWarps * 32) sort_rows_wide_kernel(RowArgs a) {
    __shared__ int64_t s_row[kRowWarps][EP_MAX_TOPK];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    const int64_t t = (int64_t)blockIdx.x * kRowWarps + warp;
    if (t < a.N) {
        const int nd = placed_rows(a, t, lane, s_row[warp], nullptr, nullptr);
        __syncwarp();
        copy_scales(a, t, s_row[warp], nd, lane);
        scatter_copy_row<8>(a.x + t * (int64_t)a.row_bytes, a.out, s_row[warp], nd, a.row_bytes, lane, 32);
    }
    pdl_trigger();
}

// The batch shape (units per lane U, rows P) and the resident blocks follow the row length and
// the entries per row, as in the expert-major combine (unsort_form).
template <int U, int P, bool V32, int MIN_BLOCKS = 0>
__global__ void __launch_bounds__(kRowWarps * 32, MIN_BLOCKS) unsort_kernel(RowArgs a) {
    __shared__ int64_t s_row[kRowWarps][EP_MAX_TOPK];
    __shared__ float s_coef[kRowWarps][EP_MAX_TOPK];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    const int64_t t = (int64_t)blockIdx.x * kRowWarps + warp;
    if (t < a.N) {
        const int nd = placed_rows(a, t, lane, s_row[warp], s_coef[warp], nullptr);
        __syncwarp();
        char* out = a.out + t * (int64_t)a.H * 2;
        if (V32) gather_reduce_row32<U, P>(a.y, s_row[warp], s_coef[warp], nd, a.H, out, lane, 32);
        else gather_reduce_row<U, P>(a.y, s_row[warp], s_coef[warp], nd, a.H, out, lane, 32);
    }
    pdl_trigger();
}

// Few rows: the four warps of a block share a row.
template <int U, int P, bool V32>
__global__ void __launch_bounds__(kRowWarps * 32) unsort_wide_kernel(RowArgs a) {
    __shared__ int64_t s_row[EP_MAX_TOPK];
    __shared__ float s_coef[EP_MAX_TOPK];
    __shared__ int s_n;
    pdl_wait();
    const int64_t t = blockIdx.x;
    if (threadIdx.x < 32) {
        const int nd = placed_rows(a, t, threadIdx.x, s_row, s_coef, nullptr);
        if (threadIdx.x == 0) s_n = nd;
    }
    __syncthreads();
    char* out = a.out + t * (int64_t)a.H * 2;
    if (V32) gather_reduce_row32<U, P>(a.y, s_row, s_coef, s_n, a.H, out, threadIdx.x, kRowWarps * 32);
    else gather_reduce_row<U, P>(a.y, s_row, s_coef, s_n, a.H, out, threadIdx.x, kRowWarps * 32);
    pdl_trigger();
}

using UnsortKernel = void (*)(RowArgs);
UnsortKernel unsort_form(int H, int k, bool y32) {
    if (H <= 256) return unsort_kernel<1, 4, false, 10>;
    if (!y32) return unsort_kernel<4, 4, false>;
    if (H <= 1024) return unsort_kernel<1, 4, true, 8>;
    if (k <= 2) return unsort_kernel<2, 2, true, 5>;
    return unsort_kernel<2, 4, true>;
}

// SHARE warps per row: its gradient dout[t] is read once per batch of P placed entries (from L1 / L2
// after the first), each entry's row of y once, each entry's dy written once; the weights'
// gradients are summed in fp32, per lane over the row's units, over the lanes by a fixed tree, and
// over the warps in order. dy may be y: a lane reads its unit of y before it writes the same unit of dy.
// Wide rows are shared by a block's four warps, so that few rows still keep enough loads in flight
// (both gradients of 1528 rows of 6912 channels: 62.5 -> 38.6 us).
template <int P, int SHARE>
__global__ void __launch_bounds__(kRowWarps * 32) unsort_backward_kernel(RowArgs a) {
    constexpr int kRows = kRowWarps / SHARE;     // of a block
    __shared__ int64_t s_row[kRows][EP_MAX_TOPK];
    __shared__ float s_coef[kRows][EP_MAX_TOPK];
    __shared__ int s_entry[kRows][EP_MAX_TOPK], s_n[kRows];
    __shared__ float s_sum[kRowWarps][EP_MAX_TOPK];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slot = warp / SHARE, first = threadIdx.x % (SHARE * 32);
    pdl_wait();
    const int64_t t = (int64_t)blockIdx.x * kRows + slot;
    if (t < a.N && warp % SHARE == 0) {
        const int nd = placed_rows(a, t, lane, s_row[slot], s_coef[slot], s_entry[slot]);
        if (lane == 0) s_n[slot] = nd;
    }
    __syncthreads();
    if (t < a.N) {
        const int nd = s_n[slot];
        const int64_t row_bytes = (int64_t)a.H * 2;
        const char* g = a.dout + t * row_bytes;
        for (int p0 = 0; p0 < nd; p0 += P) {
            float acc[P];
#pragma unroll
            for (int p = 0; p < P; ++p) acc[p] = 0.0f;
#pragma unroll 2
            for (int u = first; u < a.H >> 3; u += SHARE * 32) {
                const uint4 d4 = *reinterpret_cast<const uint4*>(g + (int64_t)u * 16);
                const uint32_t d[4] = {d4.x, d4.y, d4.z, d4.w};
                uint4 v[P];
                if (a.dweights != nullptr) {
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        if (p0 + p < nd) v[p] = *reinterpret_cast<const uint4*>(a.y + s_row[slot][p0 + p] * row_bytes + (int64_t)u * 16);
                }
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    if (p0 + p >= nd) break;
                    if (a.dweights != nullptr) {
                        const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            acc[p] = fmaf(bf16_lo(d[j]), bf16_lo(w[j]), acc[p]);
                            acc[p] = fmaf(bf16_hi(d[j]), bf16_hi(w[j]), acc[p]);
                        }
                    }
                    if (a.dy != nullptr) {
                        const float c = s_coef[slot][p0 + p];
                        const uint4 o = make_uint4(pack_bf16x2(c * bf16_lo(d[0]), c * bf16_hi(d[0])),
                                                   pack_bf16x2(c * bf16_lo(d[1]), c * bf16_hi(d[1])),
                                                   pack_bf16x2(c * bf16_lo(d[2]), c * bf16_hi(d[2])),
                                                   pack_bf16x2(c * bf16_lo(d[3]), c * bf16_hi(d[3])));
                        st_v4(a.dy + s_row[slot][p0 + p] * row_bytes + (int64_t)u * 16, o);
                    }
                }
            }
            if (a.dweights != nullptr) {
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    float s = acc[p];
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
                    if (p0 + p < nd && lane == 0) s_sum[warp][p0 + p] = s;
                }
            }
        }
    }
    __syncthreads();
    if (t < a.N && a.dweights != nullptr && warp % SHARE == 0) {
        // lane j: the gradient of entry j's weight, zero unless placed
        const int nd = s_n[slot];
        float mine = 0.0f;
        for (int p = 0; p < nd; ++p) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < SHARE; ++w) s += s_sum[warp + w][p];
            if (lane == s_entry[slot][p]) mine = s;
        }
        if (lane < a.k) a.dweights[t * a.k + lane] = mine;
    }
    pdl_trigger();
}

// ------------------------------------------------------------------ host

ep_status check_sort(const ep_shape* sh, const ep_sort* sort, const ep_launch* launch) {
    ep_status st = check_shape(sh);
    if (st != EP_OK) return st;
    if (sh->num_ranks != 1 || sort == nullptr || launch == nullptr || sort->num_rows < 0) return EP_ERR_INVALID_ARG;
    if ((int64_t)sh->num_tokens * sh->num_topk > (int64_t)1 << 30) return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

RowArgs row_args(const ep_shape* sh, const ep_sort* sort, const ep_launch* launch) {
    RowArgs a{};
    a.entry_rows = sort->entry_rows;
    a.num_rows = sort->num_rows;
    a.N = sh->num_tokens;
    a.H = sh->hidden;
    a.k = sh->num_topk;
    a.row_bytes = (uint32_t)sh->hidden * 2u;
    a.err = launch->error_flags;
    return a;
}

unsigned row_blocks(int N, int warps) { return (unsigned)((N + warps - 1) / warps); }

}  // namespace

size_t sort_ids_workspace(int64_t n, int E) {
    if (n <= kSmallEntries) return 16;
    const int64_t len = segment_length(n), S = (n + len - 1) / len;
    return (size_t)(S + 1) * (size_t)E * sizeof(int32_t);
}
size_t sort_ids_workspace_changes(int64_t n, int E) {
    return sort_ids_workspace(n, E) + (size_t)(kMaxSegments + 1) * sizeof(int32_t);
}

cudaError_t launch_sort_ids(const int64_t* ids, int n, int E, int64_t num_rows, int32_t* entry_rows,
                            int32_t* row_entries, int32_t* prefix, void* ws, uint32_t bad_bit, uint32_t* err,
                            cudaStream_t stream, int rest, int32_t* changes) {
    SortArgs a{};
    a.rest = rest;
    a.changes = changes;
    a.topk_idx = ids;
    a.entry_rows = entry_rows;
    a.row_entries = row_entries;
    a.expert_prefix = prefix;
    a.ws = reinterpret_cast<int32_t*>(ws);
    a.num_rows = num_rows;
    a.n = n;
    a.E = E;
    a.bad_bit = bad_bit;
    a.err = err;
    cudaError_t e = cudaSuccess;
    if (n <= kSmallEntries) {
        a.warps = table_warps(E, kSmallThreads / 32);
        a.seg_len = ceil_div(ceil_div(n > 0 ? n : 1, a.warps), 32) * 32;
        a.S = a.warps;
        const size_t smem = (size_t)(a.warps + 1) * E * sizeof(int);
        if (smem > kSmemPlain)
            e = cudaFuncSetAttribute(sort_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmemMax);
        if (e == cudaSuccess) e = launch_pdl(sort_small_kernel, dim3(1), dim3(kSmallThreads), smem, stream, a);
    } else {
        a.warps = table_warps(E, kSortWarps);
        a.seg_len = segment_length(n);
        a.S = ceil_div(n, a.seg_len);
        const unsigned blocks = (unsigned)ceil_div(a.S, a.warps);
        const size_t tables = (size_t)a.warps * E * sizeof(int), smem = tables + (size_t)E * sizeof(int);
        if (smem > kSmemPlain)
            e = cudaFuncSetAttribute(sort_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmemMax);
        if (e == cudaSuccess && tables > kSmemPlain)
            e = cudaFuncSetAttribute(sort_count_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmemMax);
        if (e == cudaSuccess) e = launch_pdl(sort_count_kernel, dim3(blocks), dim3(kSortWarps * 32), tables, stream, a);
        if (e == cudaSuccess)
            e = launch_pdl(sort_scan_kernel, dim3((unsigned)(E + (changes != nullptr))), dim3(kSortWarps * 32), 0,
                           stream, a);
        if (e == cudaSuccess) e = launch_pdl(sort_place_kernel, dim3(blocks), dim3(kSortWarps * 32), smem, stream, a);
    }
    return e;
}

}  // namespace ep

extern "C" {

size_t ep_sort_workspace_size(const ep_shape* sh) {
    using namespace ep;
    if (check_shape(sh) != EP_OK || sh->num_ranks != 1) return 0;
    const int64_t n = (int64_t)sh->num_tokens * sh->num_topk;
    if (n > (int64_t)1 << 30) return 0;
    return sort_ids_workspace(n, sh->num_experts);
}

ep_status ep_sort_layout(const ep_shape* sh, const int64_t* topk_idx, const ep_sort* sort, void* workspace,
                         size_t workspace_bytes, const ep_launch* launch) {
    using namespace ep;
    ep_status st = check_sort(sh, sort, launch);
    if (st != EP_OK) return st;
    const int n = sh->num_tokens * sh->num_topk;
    if (sort->expert_prefix == nullptr) return EP_ERR_INVALID_ARG;
    if (n > 0 && (topk_idx == nullptr || sort->entry_rows == nullptr)) return EP_ERR_INVALID_ARG;
    if (n > kSmallEntries && (workspace == nullptr || ((uintptr_t)workspace & 15) != 0 ||
                   workspace_bytes < ep_sort_workspace_size(sh)))
        return EP_ERR_INVALID_ARG;
    if ((st = begin_call(launch)) != EP_OK) return st;
    const cudaError_t e = launch_sort_ids(topk_idx, n, sh->num_experts, sort->num_rows, sort->entry_rows,
                                          sort->row_entries, sort->expert_prefix, workspace, EP_DEVERR_BAD_EXPERT,
                                          launch->error_flags, launch->stream);
    if (e != cudaSuccess) return cuda_fail(e);
    return end_call(launch);
}

ep_status ep_sort_rows(const ep_shape* sh, const void* x, ep_dtype x_dtype, const void* x_scales,
                       int32_t scale_format, const ep_sort* sort, void* out_x, void* out_scales,
                       const ep_launch* launch) {
    using namespace ep;
    ep_status st = check_sort(sh, sort, launch);
    if (st != EP_OK) return st;
    if (x_dtype != EP_BF16 && x_dtype != EP_FP8_E4M3) return EP_ERR_INVALID_ARG;
    if (scale_format < EP_FP8_SCALE_FP32 || scale_format > EP_FP8_SCALE_TENSOR) return EP_ERR_INVALID_ARG;
    const int N = sh->num_tokens;
    const bool rows = N > 0 && sort->num_rows > 0;
    if (N > 0 && sort->entry_rows == nullptr) return EP_ERR_INVALID_ARG;
    if (rows && (x == nullptr || out_x == nullptr)) return EP_ERR_INVALID_ARG;
    if (rows && (x_scales == nullptr) != (out_scales == nullptr)) return EP_ERR_INVALID_ARG;
    if (x_dtype == EP_BF16 && (x_scales != nullptr || out_scales != nullptr)) return EP_ERR_INVALID_ARG;
    if (((uintptr_t)x & 15) != 0 || ((uintptr_t)out_x & 15) != 0) return EP_ERR_INVALID_ARG;
    if (scale_format != EP_FP8_SCALE_UE8M0 && (((uintptr_t)x_scales | (uintptr_t)out_scales) & 3) != 0)
        return EP_ERR_INVALID_ARG;
    RowArgs a = row_args(sh, sort, launch);
    a.x = reinterpret_cast<const char*>(x);
    a.x_scales = reinterpret_cast<const char*>(x_scales);
    a.out = reinterpret_cast<char*>(out_x);
    a.out_scales = reinterpret_cast<char*>(out_scales);
    if (x_dtype == EP_FP8_E4M3) a.row_bytes = (uint32_t)sh->hidden;
    a.scale_bytes = (uint32_t)(sh->hidden / EP_FP8_GROUP) * (scale_format == EP_FP8_SCALE_UE8M0 ? 1u : 4u);
    if ((st = begin_call(launch)) != EP_OK) return st;
    if (rows) {
        const size_t smem = (size_t)kTmaWarps * a.row_bytes;
        cudaError_t e = cudaSuccess;
        if (smem <= (size_t)kTmaSmemMax) {
            if (smem > kSmemPlain)
                e = cudaFuncSetAttribute(sort_rows_tma_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTmaSmemMax);
            if (e == cudaSuccess)
                e = launch_pdl(sort_rows_tma_kernel, dim3(row_blocks(N, kTmaWarps)), dim3(kTmaWarps * 32), smem,
                               launch->stream, a);
        } else {
            e = launch_pdl(sort_rows_wide_kernel, dim3(row_blocks(N, kRowWarps)), dim3(kRowWarps * 32), 0,
                           launch->stream, a);
        }
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return end_call(launch);
}

ep_status ep_unsort_rows(const ep_shape* sh, const void* y, const float* topk_weights, const ep_sort* sort,
                         void* out, const ep_launch* launch) {
    using namespace ep;
    ep_status st = check_sort(sh, sort, launch);
    if (st != EP_OK) return st;
    const int N = sh->num_tokens;
    if (N > 0 && (sort->entry_rows == nullptr || out == nullptr || (sort->num_rows > 0 && y == nullptr)))
        return EP_ERR_INVALID_ARG;
    if (((uintptr_t)y & 15) != 0 || ((uintptr_t)out & 15) != 0) return EP_ERR_INVALID_ARG;
    RowArgs a = row_args(sh, sort, launch);
    a.y = reinterpret_cast<const char*>(y);
    a.out = reinterpret_cast<char*>(out);
    a.topk_weights = topk_weights;
    if ((st = begin_call(launch)) != EP_OK) return st;
    if (N > 0) {
        // One warp per row needs about eight rows per SM to have its loads in flight.
        const bool few = sort->num_rows <= 2 * (int64_t)N;          // at most two entries a row on average
        const bool y32 = ((uintptr_t)y & 31) == 0, share = a.H >= 2048 && N < 8 * sm_count();
        cudaError_t e = launch_pdl(share ? (y32 ? unsort_wide_kernel<1, 8, true> : unsort_wide_kernel<2, 4, false>)
                                         : unsort_form(a.H, few ? 2 : a.k, y32),
                                   dim3(share ? (unsigned)N : row_blocks(N, kRowWarps)), dim3(kRowWarps * 32), 0,
                                   launch->stream, a);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return end_call(launch);
}

ep_status ep_unsort_rows_backward(const ep_shape* sh, const void* dout, const void* y, const float* topk_weights,
                                  const ep_sort* sort, void* dy, float* dweights, const ep_launch* launch) {
    using namespace ep;
    ep_status st = check_sort(sh, sort, launch);
    if (st != EP_OK) return st;
    const int N = sh->num_tokens;
    if (dy == nullptr && dweights == nullptr && N > 0 && sort->num_rows > 0) return EP_ERR_INVALID_ARG;
    if (N > 0 && (sort->entry_rows == nullptr || dout == nullptr)) return EP_ERR_INVALID_ARG;
    if (N > 0 && sort->num_rows > 0 && dweights != nullptr && y == nullptr) return EP_ERR_INVALID_ARG;
    if ((((uintptr_t)dout | (uintptr_t)y | (uintptr_t)dy) & 15) != 0) return EP_ERR_INVALID_ARG;
    RowArgs a = row_args(sh, sort, launch);
    a.dout = reinterpret_cast<const char*>(dout);
    a.y = reinterpret_cast<const char*>(y);
    a.dy = reinterpret_cast<char*>(dy);
    a.dweights = dweights;
    a.topk_weights = topk_weights;
    if ((st = begin_call(launch)) != EP_OK) return st;
    if (N > 0) {
        const bool share = a.H >= 2048;
        cudaError_t e = launch_pdl(share ? unsort_backward_kernel<4, kRowWarps> : unsort_backward_kernel<4, 1>,
                                   dim3(share ? (unsigned)N : row_blocks(N, kRowWarps)), dim3(kRowWarps * 32), 0,
                                   launch->stream, a);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return end_call(launch);
}

}  // extern "C"
