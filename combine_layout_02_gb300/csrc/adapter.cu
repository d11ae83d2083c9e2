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

// The epilogue's part: 32 rows (columns of the tile) of one output feature per lane. A row's adapter
// is the same for the whole warp; B_i's row of the feature is loaded when the adapter changes.
struct AdapterExtra {
    const __nv_bfloat16* b;
    const float* low;
    const int64_t* idx;
    int T, F, L, r;
    __device__ __forceinline__ void operator()(float (&v)[32], const Tile& t, int c, int m, int) const {
        const int row0 = t.n0 + c;
        for (int q0 = 0; q0 < r; q0 += 32) {
            int cur = -1;
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                if (row0 + j >= T) break;
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
        const int64_t items = (int64_t)g.T * g.r;
        cudaError_t e = launch_pdl(adapter_low_simple_kernel, dim3((unsigned)((items + 7) / 8)), dim3(256), 0,
                                   launch->stream, g);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(gemm_kernel<kForward, AdapterExtra>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kGemmSmemMax);
        if (e == cudaSuccess)
            e = launch_pdl(gemm_kernel<kForward, AdapterExtra>, dim3(gemm_blocks(m, false)), dim3(kGemmThreads),
                           gemm_smem(m), launch->stream, maps, m, AdapterExtra{g.b, g.low, g.idx, g.T, g.F, g.L, g.r});
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return end_call(launch);
}

}  // extern "C"
