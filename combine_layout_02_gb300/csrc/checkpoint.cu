// checkpoint.cu -- rows into 8 bits and back (see checkpoint.cuh).
#include "checkpoint.cuh"

namespace ep {
namespace {

constexpr int kThreads = kKeptThreads;

// A thread has a group: 32 bytes of bf16, 16 of e4m3, one byte for the power of two, which 32 lanes write
// side by side.
__global__ void __launch_bounds__(kThreads) keep_kernel(const uint4* __restrict__ x, int64_t groups, int per_row, int features,
                                                        uint4* __restrict__ values, uint8_t* __restrict__ scales) {
    pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i < groups) {
        uint4 a, b = make_uint4(0, 0, 0, 0);
        if ((features & 15) == 0) {
            a = ld_stream_v4(x + 2 * i);
            b = ld_stream_v4(x + 2 * i + 1);
        } else {
            const int64_t row = i / per_row;
            const int f = (int)(i - row * per_row) * kKeptGroup;
            const uint4* at = x + (row * features + f) / 8;
            a = ld_stream_v4(at);
            if (f + 8 < features) b = ld_stream_v4(at + 1);
        }
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = larger_bf16x2(m, magnitudes(w[j]));
        const uint32_t e = kept_exponent(larger_bf16x2(m, m >> 16) & 0xFFFFu);
        const float inv = kept_inverse(e);
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = keep_pair(w[2 * j], inv) | keep_pair(w[2 * j + 1], inv) << 16;
        st_v4(values + i, make_uint4(q[0], q[1], q[2], q[3]));
        scales[i] = (uint8_t)e;
    }
    pdl_trigger();
}

__global__ void __launch_bounds__(kThreads) restore_kernel(const uint4* __restrict__ values, const uint8_t* __restrict__ scales,
                                                           int64_t groups, int per_row, int features, uint4* __restrict__ x) {
    pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i < groups) {
        const uint4 q = ld_stream_v4(values + i);
        const float s = kept_scale(scales[i]);
        const uint4 a = make_uint4(kept_pair(q.x, s), kept_pair(q.x >> 16, s), kept_pair(q.y, s), kept_pair(q.y >> 16, s));
        const uint4 b = make_uint4(kept_pair(q.z, s), kept_pair(q.z >> 16, s), kept_pair(q.w, s), kept_pair(q.w >> 16, s));
        if ((features & 15) == 0) {
            st_v4(x + 2 * i, a);
            st_v4(x + 2 * i + 1, b);
        } else {
            const int64_t row = i / per_row;
            const int f = (int)(i - row * per_row) * kKeptGroup;
            uint4* at = x + (row * features + f) / 8;
            st_v4(at, a);
            if (f + 8 < features) st_v4(at + 1, b);
        }
    }
    pdl_trigger();
}

ep_status check_rows(int32_t rows, int32_t features, const void* x, const ep_checkpoint* c, const ep_launch* launch) {
    if (launch == nullptr || rows < 0 || features < 8 || features % 8 != 0) return EP_ERR_INVALID_ARG;
    if (rows > 1 << 30 || features > EP_GEMM_MAX_FEATURES) return EP_ERR_UNSUPPORTED;
    if ((rows > 0 && x == nullptr) || ((uintptr_t)x & 15) != 0) return EP_ERR_INVALID_ARG;
    if (!kept_fits(rows, features)) return EP_ERR_UNSUPPORTED;
    return check_checkpoint(c, rows > 0, false);
}

}  // namespace

cudaError_t launch_restore(int rows, int features, const void* values, const uint8_t* scales, void* x, cudaStream_t stream) {
    const int per_row = kept_features(features) / kKeptGroup;
    const int64_t groups = (int64_t)rows * per_row;
    if (groups == 0) return cudaSuccess;
    return launch_pdl(restore_kernel, dim3((unsigned)((groups + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream,
                      (const uint4*)values, scales, groups, per_row, features, (uint4*)x);
}

}  // namespace ep

extern "C" {

ep_status ep_checkpoint_rows(int32_t num_rows, int32_t features, const void* x, const ep_checkpoint* out, const ep_launch* launch) {
    using namespace ep;
    ep_status st = check_rows(num_rows, features, x, out, launch);
    if (st != EP_OK) return st;
    if ((st = begin_call(launch)) != EP_OK) return st;
    const int per_row = kept_features(features) / kKeptGroup;
    const int64_t groups = (int64_t)num_rows * per_row;
    if (groups > 0) {
        cudaError_t e = launch_pdl(keep_kernel, dim3((unsigned)((groups + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                                   launch->stream, (const uint4*)x, groups, per_row, features, (uint4*)out->values, out->scales);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return end_call(launch);
}

ep_status ep_restore_rows(int32_t num_rows, int32_t features, const ep_checkpoint* checkpoint, void* x, const ep_launch* launch) {
    using namespace ep;
    ep_status st = check_rows(num_rows, features, x, checkpoint, launch);
    if (st != EP_OK) return st;
    if ((st = begin_call(launch)) != EP_OK) return st;
    cudaError_t e = launch_restore(num_rows, features, checkpoint->values, checkpoint->scales, x, launch->stream);
    if (e != cudaSuccess) return cuda_fail(e);
    return end_call(launch);
}

}  // extern "C"
