// pbs_evict: the kept positions of every cache, and the rows they hold.
//
// Selection, one CTA per (sequence, KV head).  The mass of a key that may be
// dropped is mapped to an unsigned integer of the same order (NaN lowest), keys
// that always stay to the largest one.  A radix select (digits of 11, 11 and 10
// bits from the top, histograms in shared memory) finds the budget-th largest
// value; everything above it stays, and of its equals the lowest positions that
// fill the budget.  The values are read once and held in shared memory where
// they fit (N <= 49152), else read again for each of the five passes.  Then the
// 32 warps, each over its own run of positions, count and write the kept ones in
// ascending order.
// The gather copies the kept rows of K and V, bound by HBM: 2 x 4 D bytes a row.
#include <math.h>

#include <algorithm>

#include "cache_common.cuh"

namespace pbs {
namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 2048;
constexpr int kHeldKeys = 49152;   // 192 KB of shared memory

// 1 .. 2^32 - 2 in the order of the mass; 0 for NaN, 2^32 - 1 for keys that
// always stay (no float maps to either: +inf gives 0xff800000).
__device__ __forceinline__ uint32_t mass_key(float x, int j, int L, int recent, int n_sink) {
  if (j < n_sink || j >= L - recent) return 0xffffffffu;
  return isnan(x) ? 0u : ordered_u32(x);
}

template <bool HELD>
__global__ void __launch_bounds__(kThreads, 1) evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t held[];
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t sh_digit, sh_need, wsum[kThreads / 32];
  __shared__ int above[kThreads / 32], equal[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  wait_for_previous_kernel();
  const int64_t row = blockIdx.x, b = row / p.K.H;
  const int L = cache_len(p.kv_len, b, p.K.N, p.err);
  const float* mass = p.mass + row * p.mass_stride;
  int32_t* keep = p.keep + row * p.budget;
  const int n_keep = min(L, p.budget);
  if (tid == 0 && p.new_len && row % p.K.H == 0) p.new_len[b] = n_keep;
  for (int i = n_keep + tid; i < p.budget; i += kThreads) keep[i] = -1;
  if (L <= p.budget) {
    for (int j = tid; j < L; j += kThreads) keep[j] = j;
    return;
  }
  auto value = [&](int j) { return HELD ? held[j] : mass_key(mass[j], j, L, p.recent, p.n_sink); };
  uint32_t prefix = 0, mask = 0;
  uint32_t need = static_cast<uint32_t>(n_keep);   // still to take among the values that match the prefix
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
    for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
    __syncthreads();
    if (pass == 0) {
#pragma unroll 4
      for (int j = tid; j < L; j += kThreads) {
        const uint32_t u = mass_key(mass[j], j, L, p.recent, p.n_sink);
        if (HELD) held[j] = u;
        atomicAdd(&hist[u >> 21], 1u);
      }
    } else {
#pragma unroll 4
      for (int j = tid; j < L; j += kThreads) {
        const uint32_t u = value(j);
        if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & digits], 1u);
      }
    }
    __syncthreads();
    // the digit whose values, from the top, reach `need`: thread t holds bins
    // 2047 - 2t and 2046 - 2t, summed from the top
    const uint32_t h0 = hist[kBins - 1 - 2 * tid], h1 = hist[kBins - 2 - 2 * tid];
    uint32_t incl = h0 + h1;
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    uint32_t before = incl - h0 - h1;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    if (before < need && before + h0 >= need) {
      sh_digit = kBins - 1 - 2 * tid;
      sh_need = need - before;
    } else if (before + h0 < need && before + h0 + h1 >= need) {
      sh_digit = kBins - 2 - 2 * tid;
      sh_need = need - before - h0;
    }
    __syncthreads();
    need = sh_need;
    prefix |= sh_digit << shift;
    mask |= digits << shift;
  }
  // each warp's run of positions, in steps of 32
  const int steps = (L + kThreads - 1) / kThreads;
  const int run = warp * steps * 32;
  int n_above = 0, n_equal = 0;
  for (int i = 0; i < steps; ++i) {
    const int j = run + i * 32 + lane;
    const uint32_t u = j < L ? value(j) : 0u;
    n_above += __popc(__ballot_sync(0xffffffffu, j < L && u > prefix));
    n_equal += __popc(__ballot_sync(0xffffffffu, j < L && u == prefix));
  }
  if (lane == 0) {
    above[warp] = n_above;
    equal[warp] = n_equal;
  }
  __syncthreads();
  int eq = 0, out = 0;                              // equals and kept positions before this warp's run
  for (int w = 0; w < warp; ++w) {
    out += above[w];
    eq += equal[w];
  }
  out += min(eq, static_cast<int>(need));
  for (int i = 0; i < steps; ++i) {
    const int j = run + i * 32 + lane;
    const uint32_t u = j < L ? value(j) : 0u;
    const bool is_eq = j < L && u == prefix;
    const uint32_t below = (1u << lane) - 1u, be = __ballot_sync(0xffffffffu, is_eq);
    const bool take = j < L && (u > prefix || (is_eq && eq + __popc(be & below) < static_cast<int>(need)));
    const uint32_t bt = __ballot_sync(0xffffffffu, take);
    if (take) keep[out + __popc(bt & below)] = j;
    eq += __popc(be);
    out += __popc(bt);
  }
}

// Kept rows in 16-byte chunks, four rows per thread with all their loads in
// flight before the first store.
constexpr int kGatherRows = 4;
template <int D>
__global__ void __launch_bounds__(256) evict_gather_kernel(const EvictParams p) {
  constexpr int CH = D / 8, RP = 256 / CH;          // chunks a row, rows a pass of the CTA
  wait_for_previous_kernel();
  const int blocks = (p.budget + RP * kGatherRows - 1) / (RP * kGatherRows);
  const int64_t row = blockIdx.x / blocks, b = row / p.K.H, h = row % p.K.H;
  const int c = threadIdx.x % CH * 8;
  const int i0 = static_cast<int>(blockIdx.x) % blocks * RP * kGatherRows + threadIdx.x / CH;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.K.ptr) + b * p.K.sB + h * p.K.sH + c;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.V.ptr) + b * p.V.sB + h * p.V.sH + c;
  __nv_bfloat16* ko = static_cast<__nv_bfloat16*>(const_cast<void*>(p.Ko.ptr)) + b * p.Ko.sB + h * p.Ko.sH + c;
  __nv_bfloat16* vo = static_cast<__nv_bfloat16*>(const_cast<void*>(p.Vo.ptr)) + b * p.Vo.sB + h * p.Vo.sH + c;
  int64_t j[kGatherRows];
#pragma unroll
  for (int q = 0; q < kGatherRows; ++q) j[q] = i0 + q * RP < p.budget ? p.keep[row * p.budget + i0 + q * RP] : -1;
  uint4 x[kGatherRows], y[kGatherRows];
#pragma unroll
  for (int q = 0; q < kGatherRows; ++q) {
    if (j[q] < 0) continue;
    x[q] = *reinterpret_cast<const uint4*>(k + j[q] * p.K.sN);
    y[q] = *reinterpret_cast<const uint4*>(v + j[q] * p.V.sN);
  }
#pragma unroll
  for (int q = 0; q < kGatherRows; ++q) {
    if (j[q] < 0) continue;
    const int64_t i = i0 + q * RP;
    *reinterpret_cast<uint4*>(ko + i * p.Ko.sN) = x[q];
    *reinterpret_cast<uint4*>(vo + i * p.Vo.sN) = y[q];
    if (c == 0) p.mass_out[row * p.mass_out_stride + i] = p.mass[row * p.mass_stride + j[q]];
  }
}

}  // namespace

size_t evict_ws_bytes(const TensorDesc&) { return 0; }

cudaError_t launch_evict(const EvictParams& p, cudaStream_t s) {
  const int64_t rows = p.K.B * p.K.H;
  const int per_cta = 256 / static_cast<int>(p.K.D / 8) * kGatherRows;
  const int64_t ctas = rows * ((p.budget + per_cta - 1) / per_cta);
  if (ctas >= (1ll << 31)) return cudaErrorInvalidValue;
  const bool held = p.K.N <= kHeldKeys;
  cudaError_t e = cudaSuccess;
  if (held) {
    static std::atomic<uint64_t> done{0};
    if ((e = allow_smem(evict_select_kernel<true>, kHeldKeys * 4, done)) != cudaSuccess) return e;
  }
  e = launch_after(held ? evict_select_kernel<true> : evict_select_kernel<false>, static_cast<unsigned>(rows), kThreads,
                   held ? static_cast<int>(p.K.N) * 4 : 0, 1, s, p);
  if (e != cudaSuccess) return e;
  return launch_after(p.K.D == 128 ? evict_gather_kernel<128> : evict_gather_kernel<64>, static_cast<unsigned>(ctas),
                      256, 0, 1, s, p);
}

}  // namespace pbs
