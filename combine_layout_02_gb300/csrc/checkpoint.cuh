// checkpoint.cuh -- activations kept in 8 bits: e4m3 values with a power of two for each 16 features of a
// row. For a group with the largest magnitude amax, the least 2^k with amax <= 448 * 2^k (448: e4m3's
// largest value), so that nothing saturates and x / 2^k is exact; k + 127 is stored in a byte. With
// powers of two a value comes back exactly in bf16 (three bits after the first), and neither amax nor k
// needs a division or a logarithm: 448 = 1.75 * 2^8, so k goes by amax's exponent and by whether its
// mantissa is above 1.75.
// 16 features, not more: that is what two neighbouring lanes hold of a row in the gated product's epilogue, and a
// byte in 16 makes 1.0625 bytes a value.
#pragma once

#include <cuda_fp16.h>

#include "ep_internal.cuh"

namespace ep {

constexpr int kKeptGroup = EP_CHECKPOINT_GROUP;
__host__ __device__ __forceinline__ int kept_features(int features) { return (features + kKeptGroup - 1) & ~(kKeptGroup - 1); }

// Magnitudes of a bf16 pair, and the larger of two pairs' values, half by half; NaN gives way to a number.
__device__ __forceinline__ uint32_t magnitudes(uint32_t a) { return a & 0x7FFF7FFFu; }
__device__ __forceinline__ uint32_t larger_bf16x2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
}

// k + 127 from a group's largest magnitude (the bits of a bf16 without its sign, no NaN): its exponent less 8,
// and one more where its mantissa is above 1.75, which then carries over. 1 for zeros (2^-126), 247 or less for
// an infinity, whose e4m3 value 448 * 2^120 comes back as one.
__device__ __forceinline__ uint32_t kept_exponent(uint32_t amax) { return max((amax + 0x1Fu) >> 7, 9u) - 8; }
__device__ __forceinline__ float kept_scale(uint32_t exponent) { return __uint_as_float(exponent << 23); }
__device__ __forceinline__ float kept_inverse(uint32_t exponent) { return __uint_as_float((254u - exponent) << 23); }

// A bf16 pair to two e4m3 bytes, and two bytes to a pair. Both products are by powers of two.
__device__ __forceinline__ uint32_t keep_pair(uint32_t pair, float inverse) {
    return pack_e4m3x2(bf16_lo(pair) * inverse, bf16_hi(pair) * inverse);
}
__device__ __forceinline__ float2 kept_values(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint32_t kept_pair(uint32_t two, float scale) {
    const float2 v = kept_values(two);
    return pack_bf16x2(v.x * scale, v.y * scale);
}

// Host: a checkpoint's pointers. `rows`: whether there are any.
inline ep_status check_checkpoint(const ep_checkpoint* c, bool rows, bool any_type) {
    if (c == nullptr || (c->dtype != EP_FP8_E4M3 && (!any_type || c->dtype != EP_BF16))) return EP_ERR_INVALID_ARG;
    if (rows && (c->values == nullptr || (c->dtype == EP_FP8_E4M3 && c->scales == nullptr))) return EP_ERR_INVALID_ARG;
    if (c->dtype == EP_BF16 && c->scales != nullptr) return EP_ERR_INVALID_ARG;
    return ((uintptr_t)c->values & 15) != 0 ? EP_ERR_INVALID_ARG : EP_OK;
}

// Whether a launch of blocks of kKeptThreads, a thread a group, reaches all of them.
constexpr int kKeptThreads = 256;
inline bool kept_fits(int rows, int features) {
    return (int64_t)rows * (kept_features(features) / kKeptGroup) <= (int64_t)0x7FFFFFFF * kKeptThreads;
}

// Enqueues the values of a checkpoint's rows [rows][features] in bf16 (checkpoint.cu).
cudaError_t launch_restore(int rows, int features, const void* values, const uint8_t* scales, void* x, cudaStream_t stream);

}  // namespace ep
