// adapter.cu -- a projection that all rows share plus each row's own low-rank adapter:
//   y[t] = W x[t] + scales[i] * B_i (A_i x[t]),  i = adapter_idx[t]
// Two kernels: low[t] = scales[i] * A_i x[t] in fp32, then the projection with B_i low[t] added
// to its fp32 sums before the one rounding.
#include "ep_internal.cuh"
#include "gemm.cuh"

namespace ep {
namespace {

constexpr int kTile = 64, kDepth = 16;

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

// One warp per (row, rank).
__global__ void __launch_bounds__(256) adapter_low_simple_kernel(AdapterArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item < (int64_t)a.T * a.r) {
        const int t = (int)(item / a.r), q = (int)(item % a.r);
        const int i = adapter_of(a, t, lane == 0 && q == 0);
        float acc = 0.0f;
        if (i >= 0) {
            const __nv_bfloat16* row = a.a + ((int64_t)i * a.r + q) * a.K;
            for (int k = lane; k < a.K; k += 32)
                acc = fmaf(__bfloat162float(a.x[(int64_t)t * a.K + k]), __bfloat162float(row[k]), acc);
            for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
            acc *= a.scales[i];
        }
        if (lane == 0) a.low[item] = acc;
    }
    pdl_trigger();
}

__global__ void __launch_bounds__(256) adapter_gemm_simple_kernel(AdapterArgs a) {
    __shared__ float sa[kDepth][kTile + 1], sb[kDepth][kTile + 1];
    pdl_wait();
    const int i0 = blockIdx.y * kTile, j0 = blockIdx.x * kTile;
    float acc[4][4] = {};
    const int ti = threadIdx.x / 16 * 4, tj = threadIdx.x % 16 * 4;
    for (int k0 = 0; k0 < a.K; k0 += kDepth) {
        for (int q = threadIdx.x; q < kDepth * kTile; q += 256) {
            const int k = k0 + q / kTile, i = i0 + q % kTile, j = j0 + q % kTile;
            sa[q / kTile][q % kTile] = k < a.K && i < a.T ? __bfloat162float(a.x[(int64_t)i * a.K + k]) : 0.0f;
            sb[q / kTile][q % kTile] = k < a.K && j < a.F ? __bfloat162float(a.w[(int64_t)j * a.K + k]) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < kDepth; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ti + i], sb[k][tj + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
        const int t = i0 + ti + i;
        if (t >= a.T) break;
        const int id = adapter_of(a, t, false);
        for (int j = 0; j < 4; ++j) {
            const int f = j0 + tj + j;
            if (f >= a.F) break;
            float v = acc[i][j];
            if (id >= 0)
                for (int q = 0; q < a.r; ++q)
                    v = fmaf(a.low[(int64_t)t * a.r + q], __bfloat162float(a.b[((int64_t)id * a.F + f) * a.r + q]), v);
            a.y[(int64_t)t * a.F + f] = __float2bfloat16_rn(v);
        }
    }
    pdl_trigger();
}

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
    if ((st = begin_call(launch)) != EP_OK) return st;
    if (rows) {
        AdapterArgs g{reinterpret_cast<const __nv_bfloat16*>(x), reinterpret_cast<const __nv_bfloat16*>(w),
                      reinterpret_cast<const __nv_bfloat16*>(a), reinterpret_cast<const __nv_bfloat16*>(b), scales,
                      adapter_idx, reinterpret_cast<__nv_bfloat16*>(y), reinterpret_cast<float*>(workspace),
                      sh->num_rows, sh->in_features, sh->out_features, sh->num_adapters, sh->rank, launch->error_flags};
        const int64_t items = (int64_t)g.T * g.r;
        cudaError_t e = launch_pdl(adapter_low_simple_kernel, dim3((unsigned)((items + 7) / 8)), dim3(256), 0,
                                   launch->stream, g);
        if (e == cudaSuccess)
            e = launch_pdl(adapter_gemm_simple_kernel, dim3((unsigned)ceil_div(g.F, kTile), (unsigned)ceil_div(g.T, kTile)),
                           dim3(256), 0, launch->stream, g);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return end_call(launch);
}

}  // extern "C"
