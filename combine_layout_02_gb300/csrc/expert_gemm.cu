// expert_gemm.cu -- products of each expert's rows with the expert's matrix, and their gradients:
//   forward  y[i]  = W_e x[i]            rows i of expert e
//   dgrad    dx[i] = W_e^T dy[i]
//   wgrad    dW_e  = sum_i dy[i] x[i]^T
#include "ep_internal.cuh"
#include "gemm.cuh"

namespace ep {
namespace {

// C[i][j] = sum_k A(i, k) B(k, j) in 64 x 64 tiles, 4 x 4 values a thread, fp32.
constexpr int kTile = 64, kDepth = 16;

enum Direction { kForward, kDgrad, kWgrad };

struct GemmArgs {
    const __nv_bfloat16* rows_a;    // x, dy, dy
    const __nv_bfloat16* other;     // w, w, x
    __nv_bfloat16* out;
    const int32_t* prefix;
    int num_rows, E, K, F;
    uint32_t* err;
};

template <Direction D>
__global__ void __launch_bounds__(256) expert_gemm_simple_kernel(GemmArgs a) {
    __shared__ float sa[kDepth][kTile + 1], sb[kDepth][kTile + 1];
    __shared__ int s_e, s_begin, s_end;
    pdl_wait();
    if (threadIdx.x == 0) {
        int tile = blockIdx.y;
        s_e = -1;
        if (D == kWgrad) {
            const int per = (a.F + kTile - 1) / kTile;
            s_e = tile / per;
            s_begin = expert_begin(a.prefix, s_e, a.num_rows);
            s_end = expert_end(a.prefix, s_e, a.num_rows);
        } else {
            for (int e = 0; e < a.E; ++e) {
                const int b = expert_begin(a.prefix, e, a.num_rows), n = expert_end(a.prefix, e, a.num_rows) - b;
                const int tiles = n > 0 ? (n + kTile - 1) / kTile : 0;
                if (tile < tiles) {
                    s_e = e;
                    s_begin = b + tile * kTile;
                    s_end = b + n;
                    break;
                }
                tile -= tiles;
            }
        }
    }
    if (blockIdx.x == 0 && blockIdx.y == 0) check_prefix(a.prefix, a.E, a.num_rows, a.err);
    __syncthreads();
    if (s_e < 0) return;
    const int e = s_e;
    const int ni = D == kWgrad ? a.F : s_end - s_begin;                  // rows of C in this group
    const int nj = D == kForward ? a.F : a.K;
    const int nk = D == kForward ? a.K : D == kDgrad ? a.F : max(0, s_end - s_begin);
    const int i0 = D == kWgrad ? (blockIdx.y % ((a.F + kTile - 1) / kTile)) * kTile : 0;
    const int j0 = blockIdx.x * kTile;
    const __nv_bfloat16* w = a.other + (int64_t)e * a.F * a.K;
    float acc[4][4] = {};
    const int ti = threadIdx.x / 16 * 4, tj = threadIdx.x % 16 * 4;
    for (int k0 = 0; k0 < nk; k0 += kDepth) {
        for (int q = threadIdx.x; q < kDepth * kTile; q += 256) {
            const int k = k0 + q / kTile, i = i0 + q % kTile, j = j0 + q % kTile;
            float va = 0.0f, vb = 0.0f;
            if (k < nk && i < ni) {
                if (D == kForward) va = __bfloat162float(a.rows_a[(int64_t)(s_begin + i) * a.K + k]);
                if (D == kDgrad) va = __bfloat162float(a.rows_a[(int64_t)(s_begin + i) * a.F + k]);
                if (D == kWgrad) va = __bfloat162float(a.rows_a[(int64_t)(s_begin + k) * a.F + i]);
            }
            if (k < nk && j < nj) {
                if (D == kForward) vb = __bfloat162float(w[(int64_t)j * a.K + k]);
                if (D == kDgrad) vb = __bfloat162float(w[(int64_t)k * a.K + j]);
                if (D == kWgrad) vb = __bfloat162float(a.other[(int64_t)(s_begin + k) * a.K + j]);
            }
            sa[q / kTile][q % kTile] = va;
            sb[q / kTile][q % kTile] = vb;
        }
        __syncthreads();
        for (int k = 0; k < kDepth; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ti + i], sb[k][tj + j], acc[i][j]);
        __syncthreads();
    }
    __nv_bfloat16* out = D == kWgrad ? a.out + (int64_t)e * a.F * a.K : a.out + (int64_t)s_begin * nj;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j)
            if (i0 + ti + i < ni && j0 + tj + j < nj)
                out[(int64_t)(i0 + ti + i) * nj + j0 + tj + j] = __float2bfloat16_rn(acc[i][j]);
    pdl_trigger();
}

ep_status check_gemm(const ep_gemm_shape* sh, const void* rows_a, const void* other, bool other_rows,
                     const int32_t* prefix, const void* out, bool out_rows, const ep_launch* launch) {
    if (sh == nullptr || launch == nullptr) return EP_ERR_INVALID_ARG;
    if (sh->num_rows < 0 || sh->num_experts < 1 || !features_ok(sh->in_features) || !features_ok(sh->out_features))
        return EP_ERR_INVALID_ARG;
    if (sh->num_experts > EP_MAX_EXPERTS || sh->in_features > EP_GEMM_MAX_FEATURES ||
        sh->out_features > EP_GEMM_MAX_FEATURES || sh->num_rows > 1 << 30)
        return EP_ERR_UNSUPPORTED;
    const bool rows = sh->num_rows > 0;
    if (prefix == nullptr || (rows && rows_a == nullptr)) return EP_ERR_INVALID_ARG;
    if ((rows || !other_rows) && other == nullptr) return EP_ERR_INVALID_ARG;
    if ((rows || !out_rows) && out == nullptr) return EP_ERR_INVALID_ARG;
    if ((((uintptr_t)rows_a | (uintptr_t)other | (uintptr_t)out) & 15) != 0) return EP_ERR_INVALID_ARG;
    if (((uintptr_t)prefix & 3) != 0) return EP_ERR_INVALID_ARG;
    return EP_OK;
}

template <Direction D>
ep_status run_gemm(const ep_gemm_shape* sh, const void* rows_a, const void* other, const int32_t* prefix, void* out,
                   const ep_launch* launch) {
    ep_status st = check_gemm(sh, rows_a, other, D == kWgrad, prefix, out, D != kWgrad, launch);
    if (st != EP_OK) return st;
    if ((st = begin_call(launch)) != EP_OK) return st;
    GemmArgs a{reinterpret_cast<const __nv_bfloat16*>(rows_a), reinterpret_cast<const __nv_bfloat16*>(other),
               reinterpret_cast<__nv_bfloat16*>(out), prefix, sh->num_rows, sh->num_experts, sh->in_features,
               sh->out_features, launch->error_flags};
    if (sh->num_rows > 0 || D == kWgrad) {
        const int nj = D == kForward ? a.F : a.K;
        const unsigned gy = D == kWgrad ? (unsigned)(a.E * ceil_div(a.F, kTile))
                                        : (unsigned)(a.num_rows / kTile + (a.E < a.num_rows ? a.E : a.num_rows));
        cudaError_t e = launch_pdl(expert_gemm_simple_kernel<D>, dim3((unsigned)ceil_div(nj, kTile), gy), dim3(256), 0,
                                   launch->stream, a);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return end_call(launch);
}

}  // namespace
}  // namespace ep

extern "C" {

ep_status ep_expert_gemm(const ep_gemm_shape* sh, const void* x, const void* w, const int32_t* expert_prefix, void* y,
                         const ep_launch* launch) {
    return ep::run_gemm<ep::kForward>(sh, x, w, expert_prefix, y, launch);
}

ep_status ep_expert_gemm_dgrad(const ep_gemm_shape* sh, const void* dy, const void* w, const int32_t* expert_prefix,
                               void* dx, const ep_launch* launch) {
    return ep::run_gemm<ep::kDgrad>(sh, dy, w, expert_prefix, dx, launch);
}

ep_status ep_expert_gemm_wgrad(const ep_gemm_shape* sh, const void* dy, const void* x, const int32_t* expert_prefix,
                               void* dw, const ep_launch* launch) {
    return ep::run_gemm<ep::kWgrad>(sh, dy, x, expert_prefix, dw, launch);
}

}  // extern "C"
