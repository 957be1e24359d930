// pbs_evict: the kept positions of every cache, and the rows they hold.
//
// The mass of a key that may be dropped is mapped to an unsigned integer of
// the same order (NaN lowest), keys that always stay to the largest one.  A
// radix select (four passes of 8 bits from the top) finds the budget-th
// largest value; everything above it stays, and of its equals the lowest
// positions that fill the budget.
#include <math.h>

#include "cache_common.cuh"

namespace pbs {
namespace {

constexpr int kThreads = 1024;

// 1 .. 2^32 - 2 in the order of the mass; 0 for NaN, 2^32 - 1 for keys that
// always stay (no float maps to either: +inf gives 0xff800000).
__device__ __forceinline__ uint32_t mass_key(float x, int64_t j, int64_t L, int recent, int n_sink) {
  if (j < n_sink || j >= L - recent) return 0xffffffffu;
  return isnan(x) ? 0u : ordered_u32(x);
}

// One CTA per (b, KV head).
__global__ void __launch_bounds__(kThreads) evict_select_kernel(EvictParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t sh_prefix, sh_need;
  __shared__ int wsum[2][kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x, b = row / p.K.H, N = p.K.N;
  const int64_t L = cache_len(p.kv_len, b, N, p.err);
  const float* mass = p.mass + row * p.mass_stride;
  int32_t* keep = p.keep + row * p.budget;
  const int n_keep = static_cast<int>(min(L, static_cast<int64_t>(p.budget)));
  if (tid == 0 && p.new_len && row % p.K.H == 0) p.new_len[b] = n_keep;
  uint32_t prefix = 0, mask = 0;
  uint32_t need = static_cast<uint32_t>(n_keep);   // still to take among the keys that match the prefix
  for (int shift = 24; shift >= 0 && n_keep > 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int64_t j = tid; j < L; j += kThreads) {
      const uint32_t u = mass_key(mass[j], j, L, p.recent, p.n_sink);
      if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t left = need;
      int d = 255;
      while (hist[d] < left) left -= hist[d--];
      sh_need = left;
      sh_prefix = prefix | (static_cast<uint32_t>(d) << shift);
    }
    __syncthreads();
    need = sh_need;
    prefix = sh_prefix;
    mask |= 255u << shift;
  }
  // ascending positions: all above the threshold, the first `need` equal to it
  int out = 0, eq = 0;
  for (int64_t j0 = 0; j0 < L && n_keep > 0; j0 += kThreads) {
    const int64_t j = j0 + tid;
    const uint32_t u = j < L ? mass_key(mass[j], j, L, p.recent, p.n_sink) : 0u;
    const bool is_eq = j < L && u == prefix;
    const uint32_t be = __ballot_sync(0xffffffffu, is_eq);
    if (lane == 0) wsum[0][warp] = __popc(be);
    __syncthreads();
    int rank = eq + __popc(be & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) rank += wsum[0][w];
    const bool take = j < L && (u > prefix || (is_eq && rank < static_cast<int>(need)));
    const uint32_t bt = __ballot_sync(0xffffffffu, take);
    if (lane == 0) wsum[1][warp] = __popc(bt);
    __syncthreads();
    int at = out + __popc(bt & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) at += wsum[1][w];
    if (take) keep[at] = static_cast<int32_t>(j);
    for (int w = 0; w < kThreads / 32; ++w) {
      eq += wsum[0][w];
      out += wsum[1][w];
    }
    __syncthreads();
  }
  for (int i = n_keep + tid; i < p.budget; i += kThreads) keep[i] = -1;
}

// 16-byte chunks of the kept K and V rows, and their mass.
__global__ void __launch_bounds__(256) evict_gather_kernel(EvictParams p) {
  const int64_t row = blockIdx.y, b = row / p.K.H, h = row % p.K.H;
  const int CH = static_cast<int>(p.K.D / 8);
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t i = id / CH;
  const int c = static_cast<int>(id % CH) * 8;
  if (i >= p.budget) return;
  const int64_t j = p.keep[row * p.budget + i];
  if (j < 0) return;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.K.ptr) + b * p.K.sB + h * p.K.sH + j * p.K.sN + c;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.V.ptr) + b * p.V.sB + h * p.V.sH + j * p.V.sN + c;
  __nv_bfloat16* ko = static_cast<__nv_bfloat16*>(const_cast<void*>(p.Ko.ptr)) + b * p.Ko.sB + h * p.Ko.sH + i * p.Ko.sN + c;
  __nv_bfloat16* vo = static_cast<__nv_bfloat16*>(const_cast<void*>(p.Vo.ptr)) + b * p.Vo.sB + h * p.Vo.sH + i * p.Vo.sN + c;
  *reinterpret_cast<uint4*>(ko) = *reinterpret_cast<const uint4*>(k);
  *reinterpret_cast<uint4*>(vo) = *reinterpret_cast<const uint4*>(v);
  if (c == 0) p.mass_out[row * p.mass_out_stride + i] = p.mass[row * p.mass_stride + j];
}

}  // namespace

size_t evict_ws_bytes(const TensorDesc&) { return 0; }

cudaError_t launch_evict(const EvictParams& p, cudaStream_t s) {
  const unsigned rows = static_cast<unsigned>(p.K.B * p.K.H);
  evict_select_kernel<<<rows, kThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.budget) * (p.K.D / 8) + 255) / 256), rows);
  evict_gather_kernel<<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace pbs
