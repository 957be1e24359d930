// Device helpers shared by the cache operators: sequence lengths and which
// keys a query row sees.
#pragma once

#include "pbs_common.cuh"
#include "pbs_internal.h"

namespace pbs {

// kv_len[b] (or q_len[b]) within [0, most]; a length outside sets the error
// word and is clamped.
__device__ __forceinline__ int64_t cache_len(const int32_t* len, int64_t b, int64_t most, int* err) {
  if (!len) return most;
  const int64_t n = len[b];
  if (n >= 0 && n <= most) return n;
  set_error(err, kErrDeviceCheck);
  return n < 0 ? 0 : most;
}

__device__ __forceinline__ bool key_visible(int64_t j, int64_t pos, int64_t window, int64_t n_sink) {
  return j <= pos && (j > pos - window || j < n_sink);
}

}  // namespace pbs
