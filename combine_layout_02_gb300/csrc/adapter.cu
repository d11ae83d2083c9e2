// adapter.cu -- a projection that all rows share plus each row's own low-rank adapter:
//   y[t] = W x[t] + scales[i] * B_i (A_i x[t]),  i = adapter_idx[t]
// low[t] = scales[i] * A_i x[t] in fp32 (many rows: by adapter, after a sort of the rows),
// then the projection with B_i low[t] added to its fp32 sums before the one rounding. With few rows
// the projection starts while low is still computed; its epilogue waits for it.
#include <type_traits>

#include "gemm.cuh"
#include "rowops.cuh"
#include "sort.cuh"

namespace ep {
namespace {

struct AdapterArgs {
    const __nv_bfloat16 *x, *a;
    const float* scales;
    const int64_t* idx;
    const int32_t* order;      // rows by adapter, and [L + 1] where each adapter's begin (many rows)
    const int32_t* prefix;
    const int32_t* changes;    // wide: scattered rows' x is copied to sorted_x in that order, by
    char* sorted_x;            // the blocks from copy_from on (one warp per row)
    float* low;                // [parts][T][r], scaled if there is one part
    int T, K, L, r, parts;
    unsigned copy_from;
    int slots;                 // blocks per 32 rows, where they are taken as they are
    uint32_t* err;
};

__device__ __forceinline__ int adapter_of(const AdapterArgs& a, int64_t t, bool flag) {
    const int64_t i = a.idx[t];
    if (i >= 0 && i < a.L) return (int)i;
    if (flag && i != -1) raise_flag(a.err, EP_DEVERR_BAD_ADAPTER);
    return -1;
}

// One 16 x 8 product of 16 contracted bf16 values, fp32 sums.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kLowRows = 32, kLowWarps = 8, kLowPartsMost = 16, kLowBlocks = 304;
constexpr int kLowPlain = 128;          // rows up to which they are taken as they are

// Blocks of the low-rank kernel. As the rows are: 32 rows are looked through for their distinct
// adapters, a block for each by its position among them. By adapter: after a sort of the rows, each
// adapter's rows cut into 32 at a time. Up to 128 rows the first saves the sort's time (61 rows of as
// many adapters, 7168 x 7168: 37 -> 34 us); with more it would start too many idle blocks.
inline int low_slots(int T, int L) { return (T < L ? T : L) < kLowRows ? (T < L ? T : L) : kLowRows; }
inline int64_t low_blocks(int T, int L, bool by_adapter) {
    return by_adapter ? (int64_t)T / kLowRows + (T < L ? T : L) : (int64_t)ceil_div(T, kLowRows) * low_slots(T, L);
}
// Ranks that a block takes at a time, in eights: few while there are few blocks, others then take the rest
// (one row 4096 -> 1024, rank 128: 12 us, else 20), up to 64, which read x once for all of them.
inline int low_tiles(int64_t blocks, int r) {
    int nt = r <= 8 ? 1 : 2;
    while (nt < 8 && nt * 8 < r && blocks * ceil_div(r, nt * 8) > kLowBlocks) nt *= 2;
    return nt;
}
// Parts of the contraction, for as many blocks as two per SM: every part is at least four steps of
// 32 for each warp.
inline int low_parts(int64_t blocks, int K, int r) {
    if (blocks == 0) return 1;
    int most = ceil_div(K, 32 * kLowWarps * 4);
    if (most > kLowPartsMost) most = kLowPartsMost;
    const int64_t want = kLowBlocks / (blocks * ceil_div(r, low_tiles(blocks, r) * 8));
    return (int)(want < 1 ? 1 : want < most ? want : most);
}

// Rows in many short runs of one adapter (under sixteen on average): the projection then takes them by
// adapter, out of a copy in that order, and scatters its results. (8191 rows in any order of 16
// adapters, 7168 -> 4096, rank 64: 820 -> 390 us; a run's rows are read where they are.)
__device__ __forceinline__ bool scattered(int changes, int T) { return changes > T / 16; }

// One warp: block number -> adapter and up to 32 of its rows in the order, 32 adapters at a time; -1
// past the last.
__device__ __forceinline__ int find_rows(const AdapterArgs& a, int lane, int& from, int& to) {
    int first = 0;
    for (int i0 = 0; i0 < a.L; i0 += 32) {
        int begin = 0, end = 0;
        if (i0 + lane < a.L) {
            begin = a.prefix[i0 + lane];
            end = a.prefix[i0 + lane + 1];
        }
        const int tiles = (end - begin + kLowRows - 1) / kLowRows;
        int upto = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += up;
        }
        const int start = first + upto - tiles, b = (int)blockIdx.x;
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, b >= start && b < start + tiles);
        if (hit != 0) {
            const int src = __ffs(hit) - 1;
            from = __shfl_sync(0xFFFFFFFFu, begin + (b - start) * kLowRows, src);
            to = min(from + kLowRows, __shfl_sync(0xFFFFFFFFu, end, src));
            return i0 + src;
        }
        first += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    from = to = 0;
    return -1;
}

// The blocks from copy_from on: one warp copies a row to its place in the order. True for them.
__device__ __forceinline__ bool copy_block(const AdapterArgs& a, int warp, int lane) {
    if (blockIdx.x < a.copy_from) return false;
    const int64_t p = (int64_t)(blockIdx.x - a.copy_from) * kLowWarps + warp, row_bytes = (int64_t)a.K * 2;
    if (blockIdx.y == 0 && blockIdx.z == 0 && p < a.T && scattered(*a.changes, a.T))
        scatter_copy_row<4>(reinterpret_cast<const char*>(a.x) + a.order[p] * row_bytes, a.sorted_x, &p, 1, row_bytes, lane, 32);
    return true;
}

// low[part][t][q] = sum over the part's k of x[t][k] A_i[q][k], times scales[i] if it is the only part (a part's
// own product may overflow where that of the sum does not), for up to 32 rows of one adapter; NT * 8 ranks at a time (blockIdx.z: which, where there are blocks for all). The warps
// share the part and join in shared memory in warp order; the parts are added up by the
// projection's epilogue. Operands come straight from memory: a
// lane of quad position c loads the 8 values c*8 .. c*8+7 of a 32-deep step with one 16-byte load,
// for a row of x and for a rank of A alike; which of them a product calls its k-th is immaterial as
// long as both agree, so the lane's four words feed two products. Rows of other adapters are not
// read (zero) and not written. Bound by the loads' latency at two blocks per SM and by the warp-level
// tensor rate (8191 rows of 7168, rank 64: 57 us, the tensor pipe 26 % active).
template <int NT, bool SORTED>
__global__ void __launch_bounds__(kLowWarps * 32, 2) adapter_low_kernel(AdapterArgs a) {
    extern __shared__ float parts[];                    // [warps][32][NT * 8]
    __shared__ int s_row[kLowRows];
    __shared__ int s_adapter;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    if (SORTED) {
        // The sort before this kernel has waited for all earlier work before its own trigger, so the
        // projection may start on the call's inputs now.
        pdl_trigger();
        pdl_wait();
    } else {
        pdl_wait();
        pdl_trigger();
    }
    if (SORTED && copy_block(a, warp, lane)) return;
    if (!SORTED && blockIdx.y == 0 && blockIdx.z == 0)
        for (int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; t < a.T; t += (int64_t)gridDim.x * blockDim.x)
            adapter_of(a, t, true);
    if (warp == 0) {
        int adapter = -1, row = -1;
        if (SORTED) {
            int begin, end;
            adapter = find_rows(a, lane, begin, end);
            if (adapter >= 0 && begin + lane < end) row = a.order[begin + lane];
        } else {
            const int slots = a.slots, t0 = (int)blockIdx.x / slots * kLowRows, slot = (int)blockIdx.x % slots;
            const int id = t0 + lane < a.T ? adapter_of(a, t0 + lane, false) : -1;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
            unsigned firsts = __ballot_sync(0xFFFFFFFFu, id >= 0 && (same & lanemask_lt()) == 0);
            for (int d = 0; d < slot && firsts != 0; ++d) firsts &= firsts - 1;
            if (firsts != 0) adapter = __shfl_sync(0xFFFFFFFFu, id, __ffs(firsts) - 1);
            if (adapter >= 0 && id == adapter) row = t0 + lane;
        }
        s_row[lane] = row;
        if (lane == 0) s_adapter = adapter;
    }
    __syncthreads();
    const int i = s_adapter;
    if (i < 0) return;
    const int steps = (a.K + 31) / 32, share = gridDim.y * kLowWarps, w = blockIdx.y * kLowWarps + warp;
    const int s0 = (int)((int64_t)steps * w / share), s1 = (int)((int64_t)steps * (w + 1) / share);
    const __nv_bfloat16* xr[4];
    bool take[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const int row = s_row[h * 8 + g];
        take[h] = row >= 0;
        xr[h] = a.x + (int64_t)max(row, 0) * a.K;
    }
    const float scale = gridDim.y > 1 ? 1.0f : a.scales[i];
    for (int q0 = blockIdx.z * NT * 8; q0 < a.r; q0 += gridDim.z * NT * 8) {
        float acc[2][NT][4] = {};
        const __nv_bfloat16* ar = a.a + ((int64_t)i * a.r + q0 + g) * a.K;
        const int ranks = a.r - q0;
#pragma unroll(NT <= 2 ? 4 : NT <= 4 ? 2 : 1)
        for (int s = s0; s < s1; ++s) {
            const int k = s * 32 + c * 8;
            const bool in = k < a.K;
            uint4 xv[4], av[NT];
#pragma unroll
            for (int h = 0; h < 4; ++h)
                xv[h] = in && take[h] ? *reinterpret_cast<const uint4*>(xr[h] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                av[n] = in && n * 8 < ranks ? *reinterpret_cast<const uint4*>(ar + (int64_t)n * 8 * a.K + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mma_16816(acc[h][n], xv[2 * h].x, xv[2 * h + 1].x, xv[2 * h].y, xv[2 * h + 1].y, av[n].x, av[n].y);
                    mma_16816(acc[h][n], xv[2 * h].z, xv[2 * h + 1].z, xv[2 * h].w, xv[2 * h + 1].w, av[n].z, av[n].w);
                }
        }
        float* part = parts + warp * kLowRows * NT * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                *reinterpret_cast<float2*>(part + (h * 16 + g) * NT * 8 + n * 8 + c * 2) = make_float2(acc[h][n][0], acc[h][n][1]);
                *reinterpret_cast<float2*>(part + (h * 16 + 8 + g) * NT * 8 + n * 8 + c * 2) = make_float2(acc[h][n][2], acc[h][n][3]);
            }
        __syncthreads();
        for (int p = threadIdx.x; p < kLowRows * NT * 8; p += blockDim.x) {
            const int row = s_row[p / (NT * 8)], q = p % (NT * 8);
            if (row >= 0 && q < ranks) {
                float sum = 0.0f;
#pragma unroll
                for (int v = 0; v < kLowWarps; ++v) sum += parts[v * kLowRows * NT * 8 + p];
                a.low[((int64_t)blockIdx.y * a.T + row) * a.r + q0 + q] = scale * sum;
            }
        }
        __syncthreads();
    }
}

template <int NT, bool SORTED>
cudaError_t launch_low(const AdapterArgs& g, cudaStream_t stream) {
    const size_t smem = (size_t)kLowWarps * kLowRows * NT * 8 * sizeof(float);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(adapter_low_kernel<NT, SORTED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const unsigned copies = SORTED && g.sorted_x != nullptr ? (unsigned)ceil_div(g.T, kLowWarps) : 0u;
    // Without adapters the ids are only looked at: a thread for each.
    const unsigned blocks = SORTED ? g.copy_from + copies
                            : g.L > 0 ? (unsigned)low_blocks(g.T, g.L, false)
                                      : (unsigned)ceil_div(g.T, kLowWarps * 32);
    const unsigned ranks = NT < 8 ? (unsigned)ceil_div(g.r, NT * 8) : 1u;
    return launch_pdl(adapter_low_kernel<NT, SORTED>, dim3(blocks, (unsigned)g.parts, ranks), dim3(kLowWarps * 32), smem, stream, g);
}

template <bool SORTED>
cudaError_t launch_low_of(const AdapterArgs& g, cudaStream_t stream) {
    switch (low_tiles(low_blocks(g.T, g.L, SORTED), g.r)) {
        case 1: return launch_low<1, SORTED>(g, stream);
        case 2: return launch_low<2, SORTED>(g, stream);
        case 4: return launch_low<4, SORTED>(g, stream);
        default: return launch_low<8, SORTED>(g, stream);
    }
}

// Workspace: low; more than kLowPlain rows: the order, where each adapter's rows begin, the changes,
// the sort's scratch and room for x in that order.
struct AdapterWorkspace {
    size_t order, prefix, changes, scratch, x, bytes;
    int parts;             // of the contraction
};
AdapterWorkspace adapter_workspace(const ep_adapter_shape* sh) {
    AdapterWorkspace w{};
    const auto round = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t T = (size_t)sh->num_rows, L = (size_t)sh->num_adapters;
    const bool by_adapter = sh->num_rows > kLowPlain;
    w.parts = low_parts(low_blocks(sh->num_rows, sh->num_adapters, by_adapter), sh->in_features, sh->rank);
    w.order = round((size_t)w.parts * T * sh->rank * sizeof(float));
    w.prefix = w.changes = w.scratch = w.x = w.bytes = w.order;
    if (by_adapter && L > 0) {
        w.prefix = w.order + round(T * 4);
        w.changes = w.prefix + round((L + 2) * 4);
        w.scratch = w.changes + 256;
        w.x = w.scratch + round(sort_ids_workspace_changes(sh->num_rows, sh->num_adapters + 1));
        w.bytes = w.x + T * sh->in_features * 2;
    }
    return w;
}

// The epilogue's part: y += B_i low. A row only ever meets its own adapter's values.
struct AdapterSide {
    const __nv_bfloat16* b;
    const float* low;
    const float* scales;
    const int64_t* idx;
    int64_t part;          // floats from one part of low to the next
    int parts, F, L, r;

    // Row t's adapter, -1 without one.
    __device__ __forceinline__ int adapter(int64_t t) const {
        const int64_t i = idx[t];
        return i >= 0 && i < L ? (int)i : -1;
    }
    // Four low values of row t, ranks from q on: the sum of the parts, times the scale of its adapter (not looked
    // at if there is one part).
    __device__ __forceinline__ float4 low4(int64_t t, int q, const float* scale) const {
        const float* at = low + t * r + q;
        const float s = parts > 1 ? *scale : 1.0f;
        float4 v = *reinterpret_cast<const float4*>(at);
        for (int p0 = 1; p0 < parts; p0 += 4) {
            float4 x[4];
#pragma unroll
            for (int p = 0; p < 4; ++p)
                x[p] = p0 + p < parts ? *reinterpret_cast<const float4*>(at + (p0 + p) * part) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int p = 0; p < 4; ++p) v.x += x[p].x, v.y += x[p].y, v.z += x[p].z, v.w += x[p].w;
        }
        return make_float4(v.x * s, v.y * s, v.z * s, v.w * s);
    }
};

// gemm_split_kernel, few rows, each usually with another adapter: one output feature per lane, four
// rows at a time, fp32. Their B values are requested before their low values are staged, and towards
// L2 while the projection is computed. G lanes share G features: each takes 8 of 8G ranks of all G (so
// that a load of the warp covers whole runs of B, 16 bytes times G, not 32 far lines), and they
// exchange their sums. Bound by latency (61 rows of 64 adapters, 7168 -> 7168, rank 16: 33 us, where W alone
// takes 21): low has to be there first.
// G: 8-rank pieces of B taken at a time (their latency is what a group of rows waits for).
template <int G>
struct AdapterFew : AdapterSide {
    static constexpr bool kFollows = true;
    static constexpr int kGroup = 4, kRows = 256, kTaken = 8 / G;          // rows whose B is in registers at a time
    // shared: low of each half, then the rows' adapters
    static constexpr int kLow = kGroup * EP_ADAPTER_MAX_RANK, kIds = 2 * kLow, kFloats = kIds + kRows;
    int together;          // groups whose low is held at a time: a power of two, one with 256 ranks

    explicit AdapterFew(const AdapterSide& side) : AdapterSide(side), together(1) {
        while (together * 2 * r <= EP_ADAPTER_MAX_RANK) together *= 2;
    }
    __device__ __forceinline__ void ahead(float* shared, int64_t row0, int rows, int m, int half) const {
        int* ids = reinterpret_cast<int*>(shared + kIds);
        const int tid = threadIdx.x - 64;
        if (tid < rows) ids[tid] = adapter(row0 + tid);
        epilogue_barrier<256>();
        const int lane = threadIdx.x & 31, m0 = m - lane, bytes = min(32, F - m0) * r * 2;          // <= 0: none
        for (int j = half; j < rows; j += 2) {
            if (ids[j] < 0) continue;
            const char* at = reinterpret_cast<const char*>(b + ((int64_t)ids[j] * F + m0) * r);
            for (int o = lane * 128; o < bytes + 127; o += 32 * 128)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(at + min(o, bytes - 1)));
        }
    }
    __device__ __forceinline__ void apply(float* shared, float (&v)[kGroup], int64_t row0, int rows, int c, int m,
                                          int half) const {
        const int* ids = reinterpret_cast<const int*>(shared + kIds) + c;
        const int tid = (threadIdx.x - 64) & 127;
        shared += half * kLow;
        // low of as many of this half's groups at a time as there is room for.
        const int nth = c / (2 * kGroup) & (together - 1);
        int id[kGroup];
#pragma unroll
        for (int j = 0; j < kGroup; ++j) id[j] = c + j < rows ? ids[j] : -1;
        const int p = threadIdx.x % G, m0 = m - p;          // this lane's piece of each of G features
        uint4 u[kTaken][G];
        const auto load_b = [&](int q0, int j0) {
#pragma unroll
            for (int j = 0; j < kTaken; ++j) {
                const __nv_bfloat16* at = b + ((int64_t)max(id[j0 + j], 0) * F + m0) * r + q0 + p * 8;
                const bool has = id[j0 + j] >= 0 && q0 + p * 8 < r;
#pragma unroll
                for (int g = 0; g < G; ++g)
                    u[j][g] = has && m0 + g < F ? *reinterpret_cast<const uint4*>(at + g * r) : make_uint4(0, 0, 0, 0);
            }
        };
        const bool any = max(max(id[0], id[1]), max(id[2], id[3])) >= 0;          // for all of this half alike
        if (any) load_b(0, 0);
        if (nth == 0) {
            epilogue_barrier<128>(2 + half);          // the groups before have been read
            const int pieces = r / 4;
            for (int e = tid; e < together * kGroup * pieces; e += 128) {
                const int n = e / pieces, q = (e - n * pieces) * 4, j = (n / kGroup) * 2 * kGroup + n % kGroup;
                const bool has = c + j < rows && ids[j] >= 0;
                *reinterpret_cast<float4*>(shared + n * r + q) = has ? low4(row0 + c + j, q, scales + ids[j]) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            epilogue_barrier<128>(2 + half);
        }
        if (!any) return;
        shared += nth * kGroup * r;
#pragma unroll 1
        for (int q0 = 0; q0 < r; q0 += 8 * G) {
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
                if (j % kTaken == 0 && q0 + j > 0) load_b(q0, j);
                float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f), y = x;
                if (q0 + p * 8 < r) {
                    const float4* l = reinterpret_cast<const float4*>(shared + j * r + q0 + p * 8);
                    x = l[0], y = l[1];
                }
                float sum[G];
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const uint4 w = u[j % kTaken][g];
                    float d = x.x * bf16_lo(w.x);
                    d = fmaf(x.y, bf16_hi(w.x), d);
                    d = fmaf(x.z, bf16_lo(w.y), d);
                    d = fmaf(x.w, bf16_hi(w.y), d);
                    d = fmaf(y.x, bf16_lo(w.z), d);
                    d = fmaf(y.y, bf16_hi(w.z), d);
                    d = fmaf(y.z, bf16_lo(w.w), d);
                    sum[g] = fmaf(y.w, bf16_hi(w.w), d);
                }
                // Lane p of G keeps feature p's sum.
#pragma unroll
                for (int h = G / 2; h > 0; h /= 2)
#pragma unroll
                    for (int g = 0; g < h; ++g) {
                        const float give = p & h ? sum[g] : sum[g + h], keep = p & h ? sum[g + h] : sum[g];
                        sum[g] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, h);
                    }
                v[j] += sum[0];
            }
        }
    }
};

// gemm_kernel, many rows. A warp has 32 output features; it takes the sums of sixteen rows at a time out of
// tensor memory in the layout of warp-level products, and adds B_i (32 features x 64 ranks, held in
// registers as long as the adapter stays) times low by such products. low is fp32: it enters as
// two bf16 terms, hi + lo, which leave 2^-17 of it; the sums are fp32. (An infinite value of B meets a lo that
// is zero or of the other sign: NaN instead of an infinity. Telling such values apart, one look at each run's
// B, took 5 to 9 % of 4096 rows 512 or 2048 -> 8192 with rank 16 to 64.) The terms of the tile's rows
// are staged in shared memory while the tile's own products run, and the tile is cut into runs of
// rows of one adapter; the next run's part of B is on its way while a run is worked on. Where sixteen
// rows hold several runs, a product is taken of one run's adapter for eight rows and added to the
// run's rows alone.
// (One feature per lane with low broadcast out of shared memory was bound by that broadcast, and
// low taken from memory row by row by its latency: 500 and 365 us where this is 290. Now these products
// are what counts where the contraction is short: they share the tensor cores with the tiles at
// work. 4096 rows 2048 -> 8192: 116 us with rank 16, 142 with 64, 75 without adapters; PLAIN 107.)
// hi and lo terms of two fp32 values. hi stays finite: a value that rounds beyond bf16's largest has that
// as its hi term and what is left as lo (an infinity is left whole; a NaN is in lo).
__device__ __forceinline__ void split_pair(float a, float b, uint32_t& hi, uint32_t& lo) {
    constexpr float kMost = 0x1.FEp127f;
    hi = pack_bf16x2(fminf(fmaxf(a, -kMost), kMost), fminf(fmaxf(b, -kMost), kMost));
    lo = pack_bf16x2(a - bf16_lo(hi), b - bf16_hi(hi));
}

// Rows of a split tile of more than 64 up to which AdapterFew is the faster: its time grows with
// rows x ranks, AdapterWide's hardly does. (Rank 16: 320 rows 4096 -> 1024, 64 a CTA, 22 us, else 34;
// 2560 -> 4096, 128 a CTA, 31 and 28. Rank 64: 240 rows 4096 -> 1024, 60 a CTA, 43 and 48; 2560 -> 4096,
// 120 a CTA, 71 and 39.)
inline int few_rows(int rank) { return 7168 / (rank + 48); }
// Tiles of at most 64 rows, AdapterFew's, where there are few: more CTAs share its work, and up to 128
// rows nothing is sorted. (Rank 16: 128 rows 1024 -> 648 13 us, else 23; 7168 -> 7168 39 and 38. 200 rows
// 2048 -> 2048, 64 tiles, 16 and 29; 7168 -> 4096, 128 tiles, 37 and 30.)
inline int widest_tile(int T, int F) {
    return T <= kLowPlain || (T <= 256 && (int64_t)ceil_div(T, 64) * ceil_div(F, kBM) <= sm_count() / 2) ? 64 : 256;
}

// d += a * b, both halves.
__device__ __forceinline__ void fma_pair(float2& d, float2 a, float2 b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;"
        : "+l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
}

// RANKS: 16, 32 or 64 at a time.
// PLAIN (16): multiply-adds in fp32 in the same layout, with low as it is and all 16 values of B of a lane's
// four features in registers. They leave the tensor cores to the tiles, but take longer by themselves.
template <int RANKS, bool PLAIN>
struct AdapterWide : AdapterSide {
    static constexpr bool kFollows = false;
    // shared: which rows the tile has, the run each is in, each run's adapter (and one -1 after), the warps'
    // counts of runs, and the rows' scales
    static constexpr int kRows = 256, kHeld = RANKS, kScale = 3 * kRows + 4 + 8, kFloats = kScale + kRows;
    // A lane's pieces of B, and its ranks in one.
    using Piece = typename std::conditional<RANKS == 16 && !PLAIN, uint2, uint4>::type;
    static constexpr int kPer = sizeof(Piece) / 2, NS = PLAIN ? 2 : RANKS / (4 * kPer);
    const int32_t* order;
    const int32_t* changes;
    int T;

    __device__ __forceinline__ bool reordered() const { return order != nullptr && scattered(*changes, T); }

    // Bytes from one row's terms to the next's: the rows' pieces that are read together lie in
    // different banks.
    static constexpr int kPitch = PLAIN ? 80 : 2 * kHeld + (RANKS == 16 ? 0 : 16), kBeside = (PLAIN ? 1 : 2) * kRows * kPitch;

    // The tile's rows' low, or its hi and lo terms: kHeld ranks from q0 on, zero past the last rank.
    __device__ __forceinline__ void stage(const int* which, unsigned char* terms, int rows, int q0) const {
        const float* scale_of = reinterpret_cast<const float*>(which) + kScale;
        constexpr int kPieces = kHeld / (PLAIN ? 4 : 8);
#pragma unroll 2
        for (int e = threadIdx.x - 128; e < rows * kPieces; e += 256) {
            const int j = e / kPieces, q = e % kPieces * (PLAIN ? 4 : 8);
            const bool has = q0 + q < r;
            const float4 x = has ? low4(which[j], q0 + q, scale_of + j) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if constexpr (PLAIN) {
                *reinterpret_cast<float4*>(terms + j * kPitch + q * 4) = x;
            } else {
                const float4 y = has ? low4(which[j], q0 + q + 4, scale_of + j) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                uint4 hi, lo;
                split_pair(x.x, x.y, hi.x, lo.x);
                split_pair(x.z, x.w, hi.y, lo.y);
                split_pair(y.x, y.y, hi.z, lo.z);
                split_pair(y.z, y.w, hi.w, lo.w);
                *reinterpret_cast<uint4*>(terms + j * kPitch + q * 2) = hi;
                *reinterpret_cast<uint4*>(terms + (kRows + j) * kPitch + q * 2) = lo;
            }
        }
    }
    __device__ __forceinline__ void prepare(float* shared, unsigned char* terms, int64_t row0, int rows) const {
        int* which = reinterpret_cast<int*>(shared);
        int* run_of = which + kRows;
        int* runs = run_of + kRows;
        int* counts = runs + kRows + 4;
        const int tid = threadIdx.x - 128, lane = tid & 31, warp = tid >> 5;
        const bool by_adapter = reordered();
        const auto row_at = [&](int j) { return by_adapter ? order[row0 + j] : (int)row0 + j; };
        const int row = tid < rows ? row_at(tid) : 0;
        const int mine = tid < rows ? adapter(row) : -1;
        const int before = tid < rows && tid > 0 ? adapter(row_at(tid - 1)) : -2;
        const bool starts = tid < rows && mine != before;
        const unsigned mask = __ballot_sync(0xFFFFFFFFu, starts);
        const float scale = parts > 1 && mine >= 0 ? scales[mine] : 0.0f;
        epilogue_barrier<256>();          // the tile before has been read
        which[tid] = row;
        shared[kScale + tid] = scale;
        if (lane == 0) counts[warp] = __popc(mask);
        epilogue_barrier<256>();
        int run = __popc(mask & (lanemask_lt() | 1u << lane)) - 1, all = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (w < warp) run += counts[w];
            all += counts[w];
        }
        run_of[tid] = tid < rows ? run : all;
        if (starts) runs[run] = mine;
        if (tid == 0) runs[all] = -1;
        stage(which, terms, rows, 0);
        epilogue_barrier<256>();
    }

    // B_i's values of the warp's 32 features (from m0 on), kHeld ranks from q0 on: of features 8h + g, the
    // quarter c of each 4 * kPer ranks (PLAIN: all ranks). Zero past the edges; nothing for i = -1.
    __device__ __forceinline__ void load_b(int i, int m0, int q0, int g, int c, Piece (&w)[NS][4]) const {
        const int q = q0 + (PLAIN ? 0 : c * kPer);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int m = m0 + h * 8 + g;
            const __nv_bfloat16* at = b + ((int64_t)max(i, 0) * F + m) * r + q;
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int on = s * (PLAIN ? kPer : 4 * kPer);
                w[s][h] = i >= 0 && m < F && q + on < r ? *reinterpret_cast<const Piece*>(at + on) : Piece{};
            }
        }
    }
    // Where a lane begins to read for eight rows from n on.
    __device__ __forceinline__ const unsigned char* row_terms(const unsigned char* terms, int n, int g, int c) const {
        return PLAIN ? terms + (n + 2 * c) * kPitch : terms + (n + g) * kPitch + c * (int)sizeof(Piece);
    }
    // d[n] += B_i times low of eight rows (`at`: row_terms), for N times eight rows. Products
    // that wait for one another are far apart: each waits for those of the tile that are at work.
    template <int N>
    __device__ __forceinline__ void product(const Piece (&w)[NS][4], const unsigned char* at, float (&d)[N][2][4]) const {
        if constexpr (PLAIN) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float2 sum[2][4] = {};          // over even and over odd ranks
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    if (s * kPer >= r) break;
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        const unsigned char* low_at = at + n * 8 * kPitch + (s * 2 + part) * 16;
                        const float4 l0 = *reinterpret_cast<const float4*>(low_at), l1 = *reinterpret_cast<const float4*>(low_at + kPitch);
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const uint32_t u = part ? w[s][h].z : w[s][h].x, v = part ? w[s][h].w : w[s][h].y;
                            const float2 x = make_float2(bf16_lo(u), bf16_hi(u)), y = make_float2(bf16_lo(v), bf16_hi(v));
                            fma_pair(sum[0][h], x, make_float2(l0.x, l0.y));
                            fma_pair(sum[1][h], x, make_float2(l1.x, l1.y));
                            fma_pair(sum[0][h], y, make_float2(l0.z, l0.w));
                            fma_pair(sum[1][h], y, make_float2(l1.z, l1.w));
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < 4; ++h) d[n][h >> 1][(h & 1) * 2 + i] += sum[i][h].x + sum[i][h].y;
            }
        } else {
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                Piece hi[N], lo[N];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    hi[n] = *reinterpret_cast<const Piece*>(at + n * 8 * kPitch + s * 64);
                    lo[n] = *reinterpret_cast<const Piece*>(at + (kRows + n * 8) * kPitch + s * 64);
                }
#pragma unroll
                for (int part = 0; part < kPer / 4; ++part)
#pragma unroll
                    for (int term = 0; term < 2; ++term)
#pragma unroll
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (int n = 0; n < N; ++n) {
                                const Piece x = w[s][2 * t], y = w[s][2 * t + 1], l = term ? lo[n] : hi[n];
                                if (part == 0) mma_16816(d[n][t], x.x, y.x, x.y, y.y, l.x, l.y);
                                if constexpr (kPer == 8)
                                    if (part == 1) mma_16816(d[n][t], x.z, y.z, x.w, y.w, l.z, l.w);
                            }
            }
        }
    }
    __device__ __forceinline__ void tile(uint32_t tmem, float* shared, unsigned char* terms, __nv_bfloat16* out, int64_t,
                                         int rows, int m0, int M, int half, int lane) const {
        const int g = lane >> 2, c = lane & 3;
        const int* which = reinterpret_cast<const int*>(shared);
        const int* run_of = which + kRows;
        const int* runs = run_of + kRows;
        const bool in = m0 + c * 8 < M;
        out += m0 + c * 8;
        const int split = (rows + 31) / 32 * 16, begin = half * split, end = half ? rows : min(rows, split);
        for (int q0 = 0; q0 < r; q0 += kHeld) {
            const bool last = q0 + kHeld >= r;
            if (q0 > 0) {
                epilogue_barrier<256>();
                stage(which, terms, rows, q0);
                epilogue_barrier<256>();
            }
            if (begin >= end) continue;
            int held = run_of[begin];
            Piece w[NS][4], next[PLAIN ? 1 : NS][4];       // of the run at work and of the one after it
            load_b(runs[held], m0, q0, g, c, w);
            if constexpr (!PLAIN) load_b(runs[run_of[rows - 1] > held ? held + 1 : held], m0, q0, g, c, next);
            const auto hold = [&](int run) {
                if constexpr (PLAIN) {          // (no registers for the one after)
                    if (held < run) load_b(runs[run], m0, q0, g, c, w);
                    held = run;
                } else {
                    while (held < run) {
#pragma unroll
                        for (int s = 0; s < NS; ++s)
#pragma unroll
                            for (int h = 0; h < 4; ++h) w[s][h] = next[s][h];
                        ++held;
                        load_b(runs[run_of[rows - 1] > held ? held + 1 : held], m0, q0, g, c, next);
                    }
                }
            };
#pragma unroll 1
            for (int n = begin; n < end; n += 16) {
                float v[2][2][4];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    tmem_load_16x8(tmem + n + b * 8, v[b][0]);
                    tmem_load_16x8(tmem + n + b * 8 + (16u << 16), v[b][1]);
                }
                const int first = run_of[n];
                const unsigned char* at = row_terms(terms, n, g, c);
                hold(first);
                tmem_wait(v[0]);
                tmem_wait(v[1]);
                if (run_of[min(n + 15, rows - 1)] == first) {
                    if (runs[first] >= 0) product(w, at, v);
                } else {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        if (n + b * 8 >= rows) break;
                        const int run0 = run_of[n + b * 8 + 2 * c], run1 = run_of[n + b * 8 + 2 * c + 1];      // of this lane's columns
                        const int to = run_of[min(n + b * 8 + 7, rows - 1)];
#pragma unroll 1
                        for (int run = run_of[n + b * 8]; run <= to; ++run) {
                            hold(run);
                            if (runs[run] < 0) continue;
                            float d[1][2][4] = {};
                            product(w, at + b * 8 * kPitch, d);
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                if (run0 == run) v[b][t][0] += d[0][t][0], v[b][t][2] += d[0][t][2];
                                if (run1 == run) v[b][t][1] += d[0][t][1], v[b][t][3] += d[0][t][3];
                            }
                        }
                    }
                }
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (!last) {
                        tmem_store_16x8(tmem + n + b * 8, v[b][0]);
                        tmem_store_16x8(tmem + n + b * 8 + (16u << 16), v[b][1]);
                        continue;
                    }
                    const uint4 p = rows_of_features(v[b], c);
                    if (in && n + b * 8 + g < rows) st_v4(out + (int64_t)which[n + b * 8 + g] * M, p);
                }
            }
            if (!last) tmem_store_wait();
        }
    }
};

template <int RANKS, bool PLAIN>
cudaError_t launch_wide(const GemmMaps& maps, const GemmArgs& m, const AdapterSide& side, const int32_t* order,
                        const int32_t* changes, int T, cudaStream_t stream) {
    AdapterWide<RANKS, PLAIN> wide{side};
    wide.order = order;
    wide.changes = changes;
    wide.T = T;
    return launch_gemm<kForward>(maps, m, wide, AdapterFew<(RANKS < 32 ? 2 : 4)>{side}, stream);
}

// Few ranks by plain multiply-adds (AdapterWide's PLAIN) where a tile's own products are long enough to
// hide them, and where there are tiles after it that do. (4096 rows -> 8192, plain and not, us: rank 8, K 512
// 70 and 62, 1024 77 and 80, 2048 93 and 115; rank 16, 1536 102 and 99, 2048 107 and 116, 4096 166 and 185. 600
// rows 2048 -> 4096, rank 16, 48 tiles: 28 and 24.)
inline bool plain_low(int T, int K, int F, int rank) {
    return rank <= 16 && K >= 128 * rank && (int64_t)ceil_div(T, 256) * ceil_div(F, 2 * kBM) >= sm_count();
}

ep_status check_adapter(const ep_adapter_shape* sh) {
    if (sh == nullptr) return EP_ERR_INVALID_ARG;
    if (sh->num_rows < 0 || sh->num_adapters < 0 || !features_ok(sh->in_features) || !features_ok(sh->out_features) ||
        sh->rank < 8 || sh->rank % 8 != 0)
        return EP_ERR_INVALID_ARG;
    if (sh->num_rows > 1 << 30 || sh->in_features > EP_GEMM_MAX_FEATURES || sh->out_features > EP_GEMM_MAX_FEATURES ||
        sh->rank > EP_ADAPTER_MAX_RANK || sh->num_adapters > EP_MAX_EXPERTS)
        return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

}  // namespace
}  // namespace ep

extern "C" {

size_t ep_adapter_workspace_size(const ep_adapter_shape* sh) {
    if (ep::check_adapter(sh) != EP_OK) return 0;
    return ep::adapter_workspace(sh).bytes;
}

ep_status ep_adapter_gemm(const ep_adapter_shape* sh, const void* x, const void* w, const void* a, const void* b,
                          const float* scales, const int64_t* adapter_idx, void* y, void* workspace,
                          size_t workspace_bytes, const ep_launch* launch) {
    using namespace ep;
    ep_status st = check_adapter(sh);
    if (st != EP_OK) return st;
    if (launch == nullptr || w == nullptr) return EP_ERR_INVALID_ARG;
    const bool rows = sh->num_rows > 0;
    if (rows && (x == nullptr || y == nullptr || adapter_idx == nullptr || workspace == nullptr)) return EP_ERR_INVALID_ARG;
    if (rows && sh->num_adapters > 0 && (a == nullptr || b == nullptr || scales == nullptr)) return EP_ERR_INVALID_ARG;
    if (rows && workspace_bytes < ep_adapter_workspace_size(sh)) return EP_ERR_INVALID_ARG;
    if ((((uintptr_t)x | (uintptr_t)w | (uintptr_t)a | (uintptr_t)b | (uintptr_t)y | (uintptr_t)workspace) & 15) != 0)
        return EP_ERR_INVALID_ARG;
    if (((uintptr_t)scales & 3) != 0 || ((uintptr_t)adapter_idx & 7) != 0) return EP_ERR_INVALID_ARG;
    GemmArgs m{};
    GemmMaps maps{};
    const AdapterWorkspace ws = adapter_workspace(sh);
    bool wide = false;
    if (rows) {
        m.out = reinterpret_cast<__nv_bfloat16*>(y);
        m.num_rows = sh->num_rows;
        m.E = 1;
        m.M = sh->out_features;
        m.N = m.C = sh->in_features;
        m.err = launch->error_flags;
        const int beside = plain_low(sh->num_rows, sh->in_features, sh->out_features, sh->rank) ? AdapterWide<16, true>::kBeside
                           : sh->rank <= 16 ? AdapterWide<16, false>::kBeside
                           : sh->rank <= 32 ? AdapterWide<32, false>::kBeside
                                            : AdapterWide<64, false>::kBeside;
        gemm_tiles(&m, false, beside, few_rows(sh->rank),
                   widest_tile(sh->num_rows, sh->out_features), 4);
        const uint64_t K = (uint64_t)sh->in_features, F = (uint64_t)sh->out_features, T = (uint64_t)sh->num_rows;
        const uint64_t da[3] = {K, F, 1}, db[2] = {K, T};
        const uint32_t ba[3] = {64, (uint32_t)kBM, 1};
        uint32_t bb[2] = {64, (uint32_t)m.box};
        if ((st = encode_map(&maps.a, w, 3, da, ba)) != EP_OK) return st;
        if ((st = encode_map(&maps.b, x, 2, db, bb)) != EP_OK) return st;
        bb[1] *= 2;
        if ((st = encode_map(&maps.b2, x, 2, db, bb)) != EP_OK) return st;
        wide = !gemm_by_split(m);
        if (wide && sh->num_adapters > 0) {
            const void* sorted = reinterpret_cast<const char*>(workspace) + ws.x;
            if ((st = encode_map(&maps.other_b[1], sorted, 2, db, bb)) != EP_OK) return st;
            bb[1] /= 2;
            if ((st = encode_map(&maps.other_b[0], sorted, 2, db, bb)) != EP_OK) return st;
        }
    }
    if ((st = begin_call(launch)) != EP_OK) return st;
    if (rows) {
        const bool by_adapter = sh->num_rows > kLowPlain && sh->num_adapters > 0;
        char* base = reinterpret_cast<char*>(workspace);
        int32_t* order = reinterpret_cast<int32_t*>(base + ws.order);
        int32_t* prefix = reinterpret_cast<int32_t*>(base + ws.prefix);
        int32_t* changes = reinterpret_cast<int32_t*>(base + ws.changes);
        const AdapterArgs g{reinterpret_cast<const __nv_bfloat16*>(x), reinterpret_cast<const __nv_bfloat16*>(a), scales,
                            adapter_idx, order, prefix, changes, wide ? base + ws.x : nullptr,
                            reinterpret_cast<float*>(workspace), sh->num_rows, sh->in_features, sh->num_adapters, sh->rank,
                            ws.parts, (unsigned)low_blocks(sh->num_rows, sh->num_adapters, true),
                            low_slots(sh->num_rows, sh->num_adapters) > 0 ? low_slots(sh->num_rows, sh->num_adapters) : 1,
                            launch->error_flags};
        const AdapterSide side{reinterpret_cast<const __nv_bfloat16*>(b), g.low, scales, adapter_idx, (int64_t)g.T * g.r, g.parts,
                               sh->out_features, g.L, g.r};
        cudaError_t e = cudaSuccess;
        if (!by_adapter) {
            e = launch_low_of<false>(g, launch->stream);
        } else {
            e = launch_sort_ids(adapter_idx, g.T, g.L + 1, g.T, nullptr, order, prefix, base + ws.scratch,
                                EP_DEVERR_BAD_ADAPTER, launch->error_flags, launch->stream, g.L, changes);
            if (e == cudaSuccess) e = launch_low_of<true>(g, launch->stream);
        }
        if (e == cudaSuccess) {
            const int32_t* sorted = by_adapter ? order : nullptr;
            e = plain_low(g.T, g.K, sh->out_features, g.r) ? launch_wide<16, true>(maps, m, side, sorted, changes, g.T, launch->stream)
                : g.r <= 16         ? launch_wide<16, false>(maps, m, side, sorted, changes, g.T, launch->stream)
                : g.r <= 32         ? launch_wide<32, false>(maps, m, side, sorted, changes, g.T, launch->stream)
                                    : launch_wide<64, false>(maps, m, side, sorted, changes, g.T, launch->stream);
        }
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return end_call(launch);
}

}  // extern "C"
