// sort.cuh -- the stable sort by id behind the expert sort and the adapters' order (sort.cu).
#pragma once

#include "ep_internal.cuh"

namespace ep {

// Stable sort of n ids (n <= 2^30) by value in [0, E), as ep_sort_layout places them. ids out of range
// other than -1 raise `bad_bit`. rest >= 0 (the last of the E <= EP_MAX_EXPERTS + 1 buckets): where
// ids outside [0, rest) go, instead of being left out. changes (nullable): gets how many ids
// differ from the one before. ws: sort_ids_workspace bytes (with changes: _changes).
size_t sort_ids_workspace(int64_t n, int E);
size_t sort_ids_workspace_changes(int64_t n, int E);
cudaError_t launch_sort_ids(const int64_t* ids, int n, int E, int64_t num_rows, int32_t* entry_rows,
                            int32_t* row_entries, int32_t* prefix, void* ws, uint32_t bad_bit, uint32_t* err,
                            cudaStream_t stream, int rest = -1, int32_t* changes = nullptr);

}  // namespace ep
