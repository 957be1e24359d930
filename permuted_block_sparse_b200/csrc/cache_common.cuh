// Device helpers shared by the cache operators: sequence lengths, and the
// keys that a set of query rows sees.
#pragma once

#include "pbs_common.cuh"
#include "pbs_internal.h"

namespace pbs {

constexpr int kSMs = 148;   // B200

// kv_len[b] (or q_len[b]) within [0, most]; a length outside sets the error
// word and is clamped.
__device__ __forceinline__ int cache_len(const int32_t* len, int64_t b, int64_t most, int* err) {
  if (!len) return static_cast<int>(most);
  const int n = len[b];
  if (n >= 0 && n <= most) return n;
  set_error(err, kErrDeviceCheck);
  return n < 0 ? 0 : static_cast<int>(most);
}

// The keys that the rows at positions first .. last of a sequence see, as one
// run of virtual indices 0 .. n-1 without the gap between the sinks and the
// window: index v is key v below `sink_end`, and key v + delta from there on
// (delta is 0 where the two meet).  sink_end is the number of sinks rounded up
// to ALIGN, so indices n_sink .. sink_end - 1 may be keys that no row sees.
struct KeyRun {
  int n_sink, sink_end, delta, n;
  __device__ __forceinline__ int key(int v) const { return v < sink_end ? v : v + delta; }
  // Bounds of what a row at `pos` (one of first .. last) sees: indices v <=
  // hi with v < n_sink or v >= lo.
  __device__ __forceinline__ int hi(int pos) const { return pos - delta; }
  __device__ __forceinline__ int lo(int pos, int64_t window) const {
    return static_cast<int>(max(static_cast<int64_t>(0), pos - window + 1)) - delta;
  }
};
template <int ALIGN>
__device__ __forceinline__ KeyRun key_run(int first, int last, int64_t window, int n_sink) {
  KeyRun k;
  if (last < 0) return KeyRun{0, 0, 0, 0};
  const int lo = static_cast<int>(max(static_cast<int64_t>(0), first - window + 1));
  k.n_sink = min(n_sink, last + 1);
  k.sink_end = (k.n_sink + ALIGN - 1) / ALIGN * ALIGN;
  k.delta = lo > k.sink_end ? lo - k.sink_end : 0;
  k.n = last + 1 - k.delta;
  return k;
}

// Tensor maps with 128-byte swizzle for tma_rows_4d, 64 columns a box, rows and
// sequences outside the tensor read as zeros.  Queries: coordinates (column,
// head, row, sequence), so a box's rows in shared memory are (sequence, row,
// head) with the head innermost.  Keys: coordinates (column, key, head,
// sequence); broadcast (zero-stride) heads or sequences have extent 1.
// (cache_attn_wide.cu)
bool encode_queries_map(CUtensorMap* map, const TensorDesc& t, int heads, int rows, int seqs);
bool encode_keys_map(CUtensorMap* map, const TensorDesc& t, int rows);

// Either bf16 of a pair is NaN or infinite.
__device__ __forceinline__ bool nonfinite_bf16x2(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t finite_or_zero_bf16x2(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
  return w;
}

}  // namespace pbs
