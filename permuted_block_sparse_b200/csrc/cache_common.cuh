// Device helpers shared by the cache operators: sequence lengths, and the
// keys that a set of query rows sees.
#pragma once

#include <atomic>

#include "pbs_common.cuh"
#include "pbs_internal.h"

namespace pbs {

constexpr int kSMs = 148;   // B200

// Every kernel here is launched so that it may be set up while the one before it
// in the stream still runs, and waits for that one's results before it reads
// anything.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Two kernels that need nothing of each other run side by side: the first lets the
// next one start once everything before both is done, and the second, which
// therefore need not wait before it reads, waits for the first before its last CTA
// ends (one CTA is enough, and the places of the others come free), so that the one
// after them finds both done.
enum class Order { kAlone, kFirst, kSecond };
__device__ __forceinline__ void begin_in(Order order) {
  if (order != Order::kSecond) wait_for_previous_kernel();
  if (order == Order::kFirst) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void end_in(Order order) {
  if (order == Order::kSecond && blockIdx.x + 1 == gridDim.x && blockIdx.y + 1 == gridDim.y) wait_for_previous_kernel();
}

template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, int smem, int cluster, cudaStream_t s,
                         Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

// Lets `kernel` use `bytes` of dynamic shared memory, asking the runtime once
// per device (`done`: one bit per device, a static of the caller's).
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
  return e;
}

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
