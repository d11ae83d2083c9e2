// expert_gemm.cu -- products of each expert's rows with the expert's matrix, and their gradients:
//   forward  y[i]  = W_e x[i]            rows i of expert e
//   dgrad    dx[i] = W_e^T dy[i]
//   wgrad    dW_e  = sum_i dy[i] x[i]^T
// All three are gemm_kernel (gemm.cuh) with other operands:
//            M side (K-major / MN-major)     N side                       contracted
//   forward  W_e, out_features, K-major      x, rows, K-major             in_features
//   dgrad    W_e, in_features, MN-major      dy, rows, K-major            out_features
//   wgrad    dy, out_features, MN-major      x, in_features, MN-major     the expert's rows
#include "checkpoint.cuh"
#include "gemm.cuh"

namespace ep {

namespace {
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
using CurrentFn = CUresult (*)(CUcontext*);

// A driver function, looked up once (the library does not link the driver library).
void* driver_function(const char* name) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion(name, &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        p = nullptr;
    return p;
}

// The encoder wants a current context, which a thread that has only been given a device (an
// autograd thread's first call, for one) does not have yet.
bool bind_context() {
    static const CurrentFn current = reinterpret_cast<CurrentFn>(driver_function("cuCtxGetCurrent"));
    CUcontext ctx = nullptr;
    if (current != nullptr && current(&ctx) == CUDA_SUCCESS && ctx != nullptr) return true;
    int device = 0;
    return cudaGetDevice(&device) == cudaSuccess && cudaSetDevice(device) == cudaSuccess;
}
}  // namespace

ep_status check_gemm_shape(const ep_gemm_shape* sh) {
    if (sh == nullptr) return EP_ERR_INVALID_ARG;
    if (sh->num_rows < 0 || sh->num_experts < 1 || !features_ok(sh->in_features) || !features_ok(sh->out_features))
        return EP_ERR_INVALID_ARG;
    if (sh->num_experts > EP_MAX_EXPERTS || sh->in_features > EP_GEMM_MAX_FEATURES ||
        sh->out_features > EP_GEMM_MAX_FEATURES || sh->num_rows > 1 << 30)
        return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

ep_status encode_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint32_t* box,
                     const uint64_t* given) {
    static const EncodeFn fn = reinterpret_cast<EncodeFn>(driver_function("cuTensorMapEncodeTiled"));
    if (fn == nullptr || !bind_context()) return cuda_fail(cudaErrorNotSupported);
    cuuint64_t d[5], strides[4];
    cuuint32_t b[5], ones[5] = {1, 1, 1, 1, 1};
    uint64_t stride = 2;
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        stride *= dims[i];
        if (i + 1 < rank) strides[i] = given != nullptr ? given[i] : stride;
    }
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), d, strides, b,
                          ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_ERROR_INVALID_VALUE) return EP_ERR_UNSUPPORTED;
    return r == CUDA_SUCCESS ? EP_OK : cuda_fail(cudaErrorUnknown);
}

namespace {

ep_status check_gemm(const ep_gemm_shape* sh, const void* rows_a, const void* other, bool other_rows,
                     const int32_t* prefix, const void* out, bool out_rows, const ep_launch* launch) {
    if (launch == nullptr) return EP_ERR_INVALID_ARG;
    const ep_status st = check_gemm_shape(sh);
    if (st != EP_OK) return st;
    const bool rows = sh->num_rows > 0;
    if (prefix == nullptr || (rows && rows_a == nullptr)) return EP_ERR_INVALID_ARG;
    if ((rows || !other_rows) && other == nullptr) return EP_ERR_INVALID_ARG;
    if ((rows || !out_rows) && out == nullptr) return EP_ERR_INVALID_ARG;
    if ((((uintptr_t)rows_a | (uintptr_t)other | (uintptr_t)out) & 15) != 0) return EP_ERR_INVALID_ARG;
    if (((uintptr_t)prefix & 3) != 0) return EP_ERR_INVALID_ARG;
    return EP_OK;
}

struct NothingBefore {
    cudaError_t operator()() const { return cudaSuccess; }
};

// `before` enqueues what the product reads.
template <Direction D, class Before = NothingBefore>
ep_status run_gemm(const ep_gemm_shape* sh, const void* rows_a, const void* other, const int32_t* prefix, void* out,
                   const ep_launch* launch, int loads = GemmArgs{}.loads, uint64_t wait_ns = GemmArgs{}.wait_ns,
                   const Before& before = {}) {
    ep_status st = check_gemm(sh, rows_a, other, D == kWgrad, prefix, out, D != kWgrad, launch);
    if (st != EP_OK) return st;
    const uint64_t K = (uint64_t)sh->in_features, F = (uint64_t)sh->out_features, E = (uint64_t)sh->num_experts,
                   rows = (uint64_t)sh->num_rows;
    if (D == kWgrad && rows == 0) {
        if ((st = begin_call(launch)) != EP_OK) return st;
        cudaError_t e = cudaMemsetAsync(out, 0, E * F * K * 2, launch->stream);
        if (e != cudaSuccess) return cuda_fail(e);
        return end_call(launch);
    }
    GemmArgs a{};
    a.prefix = prefix;
    a.out = reinterpret_cast<__nv_bfloat16*>(out);
    a.num_rows = sh->num_rows;
    a.E = sh->num_experts;
    a.M = D == kDgrad ? sh->in_features : sh->out_features;
    a.N = sh->in_features;
    a.C = D == kForward ? sh->in_features : sh->out_features;
    a.err = launch->error_flags;
    a.loads = loads;
    a.wait_ns = wait_ns;
    gemm_tiles(&a, D == kWgrad);
    GemmMaps maps{};
    if (rows > 0) {
        if (D == kWgrad) {
            const uint64_t da[2] = {F, rows}, db[2] = {K, rows};
            const uint32_t box[2] = {64, 64};
            if ((st = encode_map(&maps.a, rows_a, 2, da, box)) != EP_OK) return st;
            if ((st = encode_map(&maps.b, other, 2, db, box)) != EP_OK) return st;
            for (int i = 0; i < 6; ++i) {
                const uint32_t some[2] = {64, 1u << i};
                if ((st = encode_map(&maps.part_a[i], rows_a, 2, da, some)) != EP_OK) return st;
                if ((st = encode_map(&maps.part_b[i], other, 2, db, some)) != EP_OK) return st;
            }
            const uint64_t dout[3] = {K, F, E};
            const uint32_t bout[3] = {64, 32, 1};
            if ((st = encode_map(&maps.out, out, 3, dout, bout)) != EP_OK) return st;
        } else {
            const uint64_t da[3] = {K, F, E}, db[2] = {(uint64_t)a.C, rows};
            const uint32_t ba[3] = {64, D == kForward ? (uint32_t)kBM : 64u, 1};
            uint32_t bb[2] = {64, (uint32_t)a.box};
            if ((st = encode_map(&maps.a, other, 3, da, ba)) != EP_OK) return st;
            if ((st = encode_map(&maps.b, rows_a, 2, db, bb)) != EP_OK) return st;
            bb[1] *= 2;
            if ((st = encode_map(&maps.b2, rows_a, 2, db, bb)) != EP_OK) return st;
        }
    }
    if ((st = begin_call(launch)) != EP_OK) return st;
    if (rows > 0) {
        cudaError_t e = before();
        if (e == cudaSuccess) e = launch_gemm<D>(maps, a, NoExtra{}, NoExtra{}, launch->stream);
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

size_t ep_wgrad_checkpoint_workspace_size(const ep_gemm_shape* sh) {
    if (ep::check_gemm_shape(sh) != EP_OK) return 0;
    const size_t bytes = (size_t)sh->num_rows * sh->in_features * 2;
    return bytes > 16 ? bytes : 16;
}

ep_status ep_expert_gemm_wgrad_checkpoint(const ep_gemm_shape* sh, const void* dy, const ep_checkpoint* x,
                                          const int32_t* expert_prefix, void* dw, void* workspace, size_t workspace_bytes,
                                          const ep_launch* launch) {
    using namespace ep;
    ep_status st = check_gemm(sh, dy, workspace, true, expert_prefix, dw, false, launch);
    if (st != EP_OK) return st;
    if ((st = check_checkpoint(x, sh->num_rows > 0, false)) != EP_OK) return st;
    if (!kept_fits(sh->num_rows, sh->in_features)) return EP_ERR_UNSUPPORTED;
    if (workspace == nullptr || workspace_bytes < ep_wgrad_checkpoint_workspace_size(sh)) return EP_ERR_INVALID_ARG;
    return run_gemm<kWgrad>(sh, dy, workspace, expert_prefix, dw, launch, GemmArgs{}.loads, GemmArgs{}.wait_ns, [&] {
        return launch_restore(sh->num_rows, sh->in_features, x->values, x->scales, workspace, launch->stream);
    });
}

ep_status ep_selftest_gemm_timeout(const ep_gemm_shape* sh, int32_t product, const void* rows, const void* other,
                                   const int32_t* expert_prefix, void* out, int32_t loads, int32_t timeout_ms,
                                   const ep_launch* launch) {
    using namespace ep;
    if (launch == nullptr || launch->error_flags == nullptr || loads < 0 || loads % kBK != 0 || timeout_ms < 1 ||
        timeout_ms > 10000)
        return EP_ERR_INVALID_ARG;
    const uint64_t ns = (uint64_t)timeout_ms * 1000000ull;
    switch (product) {
        case 0: return run_gemm<kForward>(sh, rows, other, expert_prefix, out, launch, loads, ns);
        case 1: return run_gemm<kDgrad>(sh, rows, other, expert_prefix, out, launch, loads, ns);
        case 2: return run_gemm<kWgrad>(sh, rows, other, expert_prefix, out, launch, loads, ns);
        default: return EP_ERR_INVALID_ARG;
    }
}

}  // extern "C"
