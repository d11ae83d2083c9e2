// gemm.cuh -- what the experts' products and the adapters' projection share.
#pragma once

#include "ep_internal.cuh"

namespace ep {

inline bool features_ok(int f) { return f >= 8 && f % 8 == 0; }

// Rows of expert e, clipped to the row buffers; end <= begin where there are none.
__device__ __forceinline__ int expert_begin(const int32_t* prefix, int e, int num_rows) {
    return min(max(prefix[e], 0), num_rows);
}
__device__ __forceinline__ int expert_end(const int32_t* prefix, int e, int num_rows) {
    return min(max(prefix[e + 1], 0), num_rows);
}

// Flags a prefix that leaves [0, num_rows] or decreases. One block calls it.
__device__ __forceinline__ void check_prefix(const int32_t* prefix, int E, int num_rows, uint32_t* err) {
    bool bad = false;
    for (int e = threadIdx.x; e <= E; e += blockDim.x) {
        const int v = prefix[e];
        bad |= v < 0 || v > num_rows || (e < E && prefix[e + 1] < v);
    }
    if (bad) raise_flag(err, EP_DEVERR_RECV_OVERFLOW);
}

}  // namespace ep
