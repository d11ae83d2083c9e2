// adapter.cu -- a projection that all rows share plus each row's own low-rank adapter:
//   y[t] = W x[t] + scales[i] * B_i (A_i x[t]),  i = adapter_idx[t]
// Two kernels: low[t] = scales[i] * A_i x[t] in fp32, then the projection with B_i low[t] added
// to its fp32 sums before the one rounding.
#include "ep_internal.cuh"
#include "gemm.cuh"

namespace ep {
namespace {

struct AdapterArgs {
    const __nv_bfloat16 *x, *w, *a, *b;
    const float* scales;
    const int64_t* idx;
    __nv_bfloat16* y;
    float* low;        // [T][r]
    int T, K, F, L, r;
    uint32_t* err;
};

__device__ __forceinline__ int adapter_of(const AdapterArgs& a, int t, bool flag) {
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

constexpr int kLowRows = 32, kLowWarps = 8;

// low[t][q] = scales[i] * sum_k x[t][k] A_i[q][k] for 32 rows and the d-th of their distinct adapters,
// d = blockIdx.y, + gridDim.y, ...; NT * 8 ranks at a time. The warps share the contraction and
// join in shared memory in warp order. Operands come straight from memory: a lane of quad position
// c loads the 8 values c*8 .. c*8+7 of a 32-deep step with one 16-byte load, for a row of x and for a
// rank of A alike; which of them a product calls its k-th is immaterial as long as both agree, so
// the lane's first four words feed two products. Rows of other adapters are not read (zero), and
// each row is written by its own adapter's block alone.
template <int NT>
__global__ void __launch_bounds__(kLowWarps * 32) adapter_low_kernel(AdapterArgs a) {
    extern __shared__ float parts[];                    // [warps][32][NT * 8]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    pdl_wait();
    pdl_trigger();       // the projection may start; it reads low after this kernel's end only
    const int64_t t0 = (int64_t)blockIdx.x * kLowRows;
    int id = -1;
    if (t0 + lane < a.T) id = adapter_of(a, (int)(t0 + lane), warp == 0 && blockIdx.y == 0);
    const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
    unsigned firsts = __ballot_sync(0xFFFFFFFFu, id >= 0 && (same & lanemask_lt()) == 0);
    const int steps = (a.K + 31) / 32;
    const int s0 = (int)((int64_t)steps * warp / kLowWarps), s1 = (int)((int64_t)steps * (warp + 1) / kLowWarps);
    for (int d = 0; firsts != 0; ++d, firsts &= firsts - 1) {
        if (d % gridDim.y != blockIdx.y) continue;
        const int i = __shfl_sync(0xFFFFFFFFu, id, __ffs(firsts) - 1);
        const unsigned mine = __ballot_sync(0xFFFFFFFFu, id == i);
        for (int q0 = 0; q0 < a.r; q0 += NT * 8) {
            float acc[2][NT][4] = {};
            const __nv_bfloat16* xr[4];
            bool take[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                take[h] = (mine >> (h * 8 + g)) & 1;
                xr[h] = a.x + (t0 + h * 8 + g) * a.K;
            }
            const __nv_bfloat16* ar = a.a + ((int64_t)i * a.r + q0 + g) * a.K;
            const int ranks = a.r - q0;
#pragma unroll 2
            for (int s = s0; s < s1; ++s) {
                const int k = s * 32 + c * 8;
                const bool in = k < a.K;
                uint4 xv[4], av[NT];
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    xv[h] = in && take[h] ? *reinterpret_cast<const uint4*>(xr[h] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    av[n] = in && n * 8 < ranks ? ld_stream_v4(ar + (int64_t)n * 8 * a.K + k) : make_uint4(0, 0, 0, 0);
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
            const float scale = a.scales[i];
            for (int p = threadIdx.x; p < kLowRows * NT * 8; p += blockDim.x) {
                const int row = p / (NT * 8), q = p % (NT * 8);
                if (((mine >> row) & 1) && q < ranks) {
                    float sum = 0.0f;
#pragma unroll
                    for (int w = 0; w < kLowWarps; ++w) sum += parts[w * kLowRows * NT * 8 + p];
                    a.low[(t0 + row) * a.r + q0 + q] = scale * sum;
                }
            }
            __syncthreads();
        }
    }
}

template <int NT>
cudaError_t launch_low(const AdapterArgs& g, cudaStream_t stream) {
    const int tiles = ceil_div(g.T, kLowRows);
    // Few tiles: a block for each of a tile's adapters; many: each block takes them in turn.
    int slots = 4 * sm_count() / tiles;
    slots = slots < 1 ? 1 : slots > kLowRows ? kLowRows : slots;
    const size_t smem = (size_t)kLowWarps * kLowRows * NT * 8 * sizeof(float);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(adapter_low_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(adapter_low_kernel<NT>, dim3((unsigned)tiles, (unsigned)slots), dim3(kLowWarps * 32), smem, stream, g);
}

// The epilogue's part: 32 rows (columns of the tile) of one output feature per lane. A row's adapter
// is the same for the whole warp; B_i's row of the feature is loaded when the adapter changes.
struct AdapterExtra {
    const __nv_bfloat16* b;
    const float* low;
    const int64_t* idx;
    int F, L, r;
    static constexpr bool kFollows = true;
    __device__ __forceinline__ void operator()(float (&v)[32], int64_t row0, int rows, int m) const {
        for (int q0 = 0; q0 < r; q0 += 32) {
            int cur = -1;
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                if (j >= rows) break;
                const int64_t id = idx[row0 + j];
                if (id < 0 || id >= L) continue;
                if (id != cur) {
                    cur = (int)id;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        uint4 u = make_uint4(0, 0, 0, 0);
                        if (m < F && q0 + g * 8 < r)
                            u = *reinterpret_cast<const uint4*>(b + ((int64_t)cur * F + m) * r + q0 + g * 8);
                        w[4 * g] = u.x, w[4 * g + 1] = u.y, w[4 * g + 2] = u.z, w[4 * g + 3] = u.w;
                    }
                }
                const float4* l = reinterpret_cast<const float4*>(low + (int64_t)(row0 + j) * r + q0);
                float acc = v[j];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (q0 + g * 8 >= r) break;
                    const float4 lo = l[2 * g], hi = l[2 * g + 1];
                    acc = fmaf(lo.x, bf16_lo(w[4 * g]), acc);
                    acc = fmaf(lo.y, bf16_hi(w[4 * g]), acc);
                    acc = fmaf(lo.z, bf16_lo(w[4 * g + 1]), acc);
                    acc = fmaf(lo.w, bf16_hi(w[4 * g + 1]), acc);
                    acc = fmaf(hi.x, bf16_lo(w[4 * g + 2]), acc);
                    acc = fmaf(hi.y, bf16_hi(w[4 * g + 2]), acc);
                    acc = fmaf(hi.z, bf16_lo(w[4 * g + 3]), acc);
                    acc = fmaf(hi.w, bf16_hi(w[4 * g + 3]), acc);
                }
                v[j] = acc;
            }
        }
    }
};

ep_status check_adapter(const ep_adapter_shape* sh) {
    if (sh == nullptr) return EP_ERR_INVALID_ARG;
    if (sh->num_rows < 0 || sh->num_adapters < 0 || !features_ok(sh->in_features) || !features_ok(sh->out_features) ||
        sh->rank < 8 || sh->rank % 8 != 0)
        return EP_ERR_INVALID_ARG;
    if (sh->num_rows > 1 << 30 || sh->in_features > EP_GEMM_MAX_FEATURES || sh->out_features > EP_GEMM_MAX_FEATURES ||
        sh->rank > EP_ADAPTER_MAX_RANK)
        return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

}  // namespace
}  // namespace ep

extern "C" {

size_t ep_adapter_workspace_size(const ep_adapter_shape* sh) {
    if (ep::check_adapter(sh) != EP_OK) return 0;
    return (size_t)sh->num_rows * sh->rank * sizeof(float);
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
    if (rows) {
        m.out = reinterpret_cast<__nv_bfloat16*>(y);
        m.num_rows = sh->num_rows;
        m.E = 1;
        m.M = sh->out_features;
        m.N = m.C = sh->in_features;
        m.err = launch->error_flags;
        gemm_tiles(&m, false);
        const uint64_t K = (uint64_t)sh->in_features, F = (uint64_t)sh->out_features, T = (uint64_t)sh->num_rows;
        const uint64_t da[3] = {K, F, 1}, db[2] = {K, T};
        const uint32_t ba[3] = {64, (uint32_t)kBM, 1}, bb[2] = {64, (uint32_t)m.box};
        if ((st = encode_map(&maps.a, w, 3, da, ba)) != EP_OK) return st;
        if ((st = encode_map(&maps.b, x, 2, db, bb)) != EP_OK) return st;
    }
    if ((st = begin_call(launch)) != EP_OK) return st;
    if (rows) {
        AdapterArgs g{reinterpret_cast<const __nv_bfloat16*>(x), reinterpret_cast<const __nv_bfloat16*>(w),
                      reinterpret_cast<const __nv_bfloat16*>(a), reinterpret_cast<const __nv_bfloat16*>(b), scales,
                      adapter_idx, reinterpret_cast<__nv_bfloat16*>(y), reinterpret_cast<float*>(workspace),
                      sh->num_rows, sh->in_features, sh->out_features, sh->num_adapters, sh->rank, launch->error_flags};
        cudaError_t e = g.r <= 8    ? launch_low<1>(g, launch->stream)
                        : g.r <= 16 ? launch_low<2>(g, launch->stream)
                        : g.r <= 32 ? launch_low<4>(g, launch->stream)
                                    : launch_low<8>(g, launch->stream);
        if (e == cudaSuccess)
            e = launch_gemm<kForward>(maps, m, AdapterExtra{g.b, g.low, g.idx, g.F, g.L, g.r}, launch->stream);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return end_call(launch);
}

}  // extern "C"
