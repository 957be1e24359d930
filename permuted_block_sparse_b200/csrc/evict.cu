// pbs_evict: the kept positions of every cache, and the rows they hold.
//
// Selection, one cluster of up to eight CTAs per (sequence, KV head), each over its
// run of positions.  The mass of a key that may be dropped is mapped to an unsigned
// integer of the same order (NaN lowest), keys that always stay to the largest one.
// A radix select (digits of 11, 11 and 10 bits from the top, histograms in shared
// memory, added over the cluster) finds the budget-th largest value; everything above
// it stays, and of its equals the lowest positions that fill the budget.  The values
// are read once and held in shared memory where a CTA's run fits (40960 keys), else
// read again for each of the five passes.  Then the 32 warps of a CTA, each over its
// own run of positions, count and write the kept ones in ascending order, four
// consecutive positions a lane.
// Masses share their leading digits, so lanes meet on the same bin: there are four
// copies of the histogram, by lane.
// Bound: instructions, about 0.4 us per 1024 keys and CTA behind a fixed 7 us (three
// digits of a few barriers each).  Measured: 128 rows of 16384 to 32768 keys 22 us.
// The gather copies the kept rows of K and V, bound by HBM: 2 x 4 D bytes a row.
// Measured: 128 x 4097 rows of D = 128 84 us, 6.3 TB/s.
#include <math.h>

#include <algorithm>

#include "cache_common.cuh"

namespace pbs {
namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 2048;
constexpr int kCopies = 4;
constexpr int kBatch = 16;
constexpr int kHeldKeys = 40960;   // 160 KB of shared memory
constexpr int kMaxRank = 8;        // CTAs per cluster
constexpr int kHistBytes = kCopies * kBins * 4;

// 1 .. 2^32 - 2 in the order of the mass; 0 for NaN, 2^32 - 1 for keys that
// always stay (no float maps to either: +inf gives 0xff800000).
__device__ __forceinline__ uint32_t mass_key(float x, int j, int L, int recent, int n_sink) {
  if (j < n_sink || j >= L - recent) return 0xffffffffu;
  return isnan(x) ? 0u : ordered_u32(x);
}

__device__ __forceinline__ int ld_cluster_s32(uint32_t a) {
  int x;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(a));
  return x;
}

template <bool HELD>
__global__ void __launch_bounds__(kThreads, 1) evict_select_kernel(const EvictParams p, const int n_rank) {
  extern __shared__ __align__(16) int dyn[];
  int* hist = dyn;                                 // [copy][bin]
  uint32_t* held = reinterpret_cast<uint32_t*>(dyn + kCopies * kBins);
  __shared__ int total[2][kBins];                  // this CTA's histogram, by the parity of the pass
  __shared__ int sh_digit, sh_need, sh_ties, sh_above, sh_equal;
  __shared__ int warp_a[kThreads / 32], warp_b[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  wait_for_previous_kernel();
  const int rank = static_cast<int>(blockIdx.x) % n_rank;
  const int64_t row = blockIdx.x / n_rank, b = row / p.K.H;
  const int L = cache_len(p.kv_len, b, p.K.N, p.err);
  const float* mass = p.mass + row * p.mass_stride;
  int32_t* keep = p.keep + row * p.budget;
  const int n_keep = min(L, p.budget);
  if (rank == 0)
    for (int i = n_keep + tid; i < p.budget; i += kThreads) keep[i] = -1;
  if (L <= p.budget) {                             // (all of the cluster alike)
    for (int j = rank * kThreads + tid; j < L; j += kThreads * n_rank) keep[j] = j;
    return;
  }
  // this CTA's positions
  const int slice = (L + n_rank - 1) / n_rank;
  const int begin = min(L, rank * slice), end = min(L, begin + slice);
  auto value = [&](int j) { return HELD ? held[j - begin] : mass_key(mass[j], j, L, p.recent, p.n_sink); };
  // sum over the warps before this one, of one value per warp
  auto before_warp = [&](const int* per_warp) {
    int x = lane < warp ? per_warp[lane] : 0;
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
  };
  // sum of a shared-memory value over the CTAs of the cluster below `ranks`
  // (all reads in flight before the first is used)
  auto over_cluster = [&](const int* v, int ranks) {
    int x[kMaxRank], sum = 0;
#pragma unroll
    for (int q = 0; q < kMaxRank; ++q) x[q] = q < ranks ? ld_cluster_s32(mapa_shared(smem_u32(v), q)) : 0;
#pragma unroll
    for (int q = 0; q < kMaxRank; ++q) sum += x[q];
    return sum;
  };
  // The keys that always stay (n_sink + recent of them, as L > budget) are not
  // counted: they would all meet on one bin.
  uint32_t prefix = 0, mask = 0;
  int need = n_keep - p.n_sink - p.recent;         // still to take among the values that match the prefix
  int ties = need;                                 // values equal to the threshold, after the last pass
  if (need == 0) prefix = 0xfffffffeu;             // (above every mass, below the keys that always stay)
  for (int pass = need == 0 && !HELD ? 3 : 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
    for (int i = tid; i < kCopies * kBins; i += kThreads) hist[i] = 0;
    __syncthreads();
    int* mine = hist + (lane % kCopies) * kBins;
    if (pass == 0) {
      // all loads of a batch in flight before the first is used
      for (int j0 = begin + tid; j0 < end; j0 += kThreads * kBatch) {
        float x[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) x[q] = j0 + q * kThreads < end ? mass[j0 + q * kThreads] : 0.f;
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          const int j = j0 + q * kThreads;
          if (j >= end) break;
          const uint32_t u = mass_key(x[q], j, L, p.recent, p.n_sink);
          if (HELD) held[j - begin] = u;
          if (u != 0xffffffffu) atomicAdd(&mine[u >> 21], 1);
        }
      }
    } else {
#pragma unroll 8
      for (int j = begin + tid; j < end; j += kThreads) {
        const uint32_t u = value(j);
        if ((u & mask) == prefix) atomicAdd(&mine[(u >> shift) & digits], 1);
      }
    }
    __syncthreads();
    if (need == 0) break;                          // (the values are held now)
    // the digit whose values, from the top, reach `need`: thread t holds bins
    // 2047 - 2t and 2046 - 2t, summed from the top
    const int bin0 = kBins - 1 - 2 * tid, bin1 = bin0 - 1;
    int h0 = 0, h1 = 0;
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      h0 += hist[c * kBins + bin0];
      h1 += hist[c * kBins + bin1];
    }
    if (n_rank > 1) {
      // (two buffers: a CTA writes one again only two passes, and so two of these
      // barriers, after the others have read it)
      total[pass & 1][bin0] = h0;
      total[pass & 1][bin1] = h1;
      cluster_sync_all();
      h0 = over_cluster(&total[pass & 1][bin0], n_rank);
      h1 = over_cluster(&total[pass & 1][bin1], n_rank);
    }
    int incl = h0 + h1;
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (lane == 31) warp_a[warp] = incl;
    __syncthreads();
    const int before = incl - h0 - h1 + before_warp(warp_a);
    if (before < need && before + h0 >= need) {
      sh_digit = bin0;
      sh_need = need - before;
      sh_ties = h0;
    } else if (before + h0 < need && before + h0 + h1 >= need) {
      sh_digit = bin1;
      sh_need = need - before - h0;
      sh_ties = h1;
    }
    __syncthreads();
    need = sh_need;
    ties = sh_ties;
    prefix |= static_cast<uint32_t>(sh_digit) << shift;
    mask |= digits << shift;
  }
  // each warp's run of positions, in steps of 128
  const int steps = (end - begin + kThreads * 4 - 1) / (kThreads * 4);
  const int run = begin + warp * steps * 128;
  int n_above = 0, n_equal = 0;
  for (int i = 0; i < steps; ++i) {
    const int j = run + i * 128 + lane * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t u = j + e < end ? value(j + e) : 0u;
      n_above += j + e < end && u > prefix;
      n_equal += j + e < end && u == prefix;
    }
  }
  for (int off = 16; off > 0; off >>= 1) {
    n_above += __shfl_xor_sync(0xffffffffu, n_above, off);
    n_equal += __shfl_xor_sync(0xffffffffu, n_equal, off);
  }
  __syncthreads();                                  // (warp_a was the scan's)
  if (lane == 0) {
    warp_a[warp] = n_above;
    warp_b[warp] = n_equal;
  }
  __syncthreads();
  // equals and kept positions before this warp's run
  int out = before_warp(warp_a), eq = before_warp(warp_b);
  if (n_rank > 1) {
    if (tid == kThreads - 1) {
      sh_above = out + n_above;
      sh_equal = eq + n_equal;
    }
    cluster_sync_all();
    out += over_cluster(&sh_above, rank);
    eq += over_cluster(&sh_equal, rank);
  }
  out += min(eq, need);
  const bool all_ties = need == ties;
  const uint32_t lower = (1u << lane) - 1u;
  // lanes' counts of 0 .. 4 summed over the lanes below, and over all
  auto scan = [&](int c, int& sum) {
    const uint32_t b0 = __ballot_sync(0xffffffffu, c & 1), b1 = __ballot_sync(0xffffffffu, c & 2),
                   b2 = __ballot_sync(0xffffffffu, c & 4);
    sum = __popc(b0) + 2 * __popc(b1) + 4 * __popc(b2);
    return __popc(b0 & lower) + 2 * __popc(b1 & lower) + 4 * __popc(b2 & lower);
  };
  for (int i = 0; i < steps; ++i) {
    const int j = run + i * 128 + lane * 4;
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = j + e < end ? value(j + e) : 0u;
    bool take[4];
    if (all_ties) {
#pragma unroll
      for (int e = 0; e < 4; ++e) take[e] = j + e < end && u[e] >= prefix;
    } else {
      int c = 0, sum;
#pragma unroll
      for (int e = 0; e < 4; ++e) c += j + e < end && u[e] == prefix;
      int place = eq + scan(c, sum);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool is_eq = j + e < end && u[e] == prefix;
        take[e] = j + e < end && (u[e] > prefix || (is_eq && place < need));
        place += is_eq;
      }
      eq += sum;
    }
    int sum;
    int at = out + scan(take[0] + take[1] + take[2] + take[3], sum);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (take[e]) keep[at++] = j + e;
    out += sum;
  }
  if (n_rank > 1) cluster_sync_all();               // the others may still read this CTA's shared memory
}

// Kept rows in 16-byte chunks, two rows of K and V per thread with all their loads in
// flight before the first store.  Rows are read and written once: the streaming hints
// on both sides take 128 rows of 4097 keys (D 128) from 88 to 84 us (one
// side alone gains nothing; four rows per thread 85, eight without the hints 118).
constexpr int kGatherRows = 2;
template <int D>
__global__ void __launch_bounds__(256) evict_gather_kernel(const EvictParams p) {
  constexpr int CH = D / 8, RP = 256 / CH;          // chunks a row, rows a pass of the CTA
  wait_for_previous_kernel();
  const int blocks = (p.budget + RP * kGatherRows - 1) / (RP * kGatherRows);
  const int64_t row = blockIdx.x / blocks, b = row / p.K.H, h = row % p.K.H;
  // (here, as new_len may be kv_len, which every CTA of the selection reads; nothing else
  // reads it from here on)
  if (p.new_len && h == 0 && blockIdx.x % blocks == 0 && threadIdx.x == 0)
    p.new_len[b] = min(cache_len(p.kv_len, b, p.K.N, p.err), p.budget);
  const int c = threadIdx.x % CH * 8;
  const int i0 = static_cast<int>(blockIdx.x) % blocks * RP * kGatherRows + threadIdx.x / CH;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.K.ptr) + b * p.K.sB + h * p.K.sH + c;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.V.ptr) + b * p.V.sB + h * p.V.sH + c;
  __nv_bfloat16* ko = static_cast<__nv_bfloat16*>(const_cast<void*>(p.Ko.ptr)) + b * p.Ko.sB + h * p.Ko.sH + c;
  __nv_bfloat16* vo = static_cast<__nv_bfloat16*>(const_cast<void*>(p.Vo.ptr)) + b * p.Vo.sB + h * p.Vo.sH + c;
  int64_t j[kGatherRows];
#pragma unroll
  for (int q = 0; q < kGatherRows; ++q) {
    j[q] = i0 + q * RP < p.budget ? p.keep[row * p.budget + i0 + q * RP] : -1;
    if (j[q] >= p.K.N) j[q] = -1;                     // (never, unless something else wrote into keep)
  }
  uint4 x[kGatherRows], y[kGatherRows];
#pragma unroll
  for (int q = 0; q < kGatherRows; ++q) {
    if (j[q] < 0) continue;
    x[q] = __ldcs(reinterpret_cast<const uint4*>(k + j[q] * p.K.sN));
    y[q] = __ldcs(reinterpret_cast<const uint4*>(v + j[q] * p.V.sN));
  }
#pragma unroll
  for (int q = 0; q < kGatherRows; ++q) {
    if (j[q] < 0) continue;
    const int64_t i = i0 + q * RP;
    __stcs(reinterpret_cast<uint4*>(ko + i * p.Ko.sN), x[q]);
    __stcs(reinterpret_cast<uint4*>(vo + i * p.Vo.sN), y[q]);
    if (c == 0) p.mass_out[row * p.mass_out_stride + i] = p.mass[row * p.mass_stride + j[q]];
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t s) {
  const int64_t rows = p.K.B * p.K.H;
  const int per_cta = 256 / static_cast<int>(p.K.D / 8) * kGatherRows;
  const int64_t ctas = rows * ((p.budget + per_cta - 1) / per_cta);
  if (ctas >= (1ll << 31)) return cudaErrorInvalidValue;
  // CTAs per row: as many as leave each 16384 keys, while all rows run at once (one
  // CTA takes 19 us for 32768 keys, eight 23; for 131072 one takes 125, eight 28)
  int rank = 1;
  while (rank < kMaxRank && p.K.N / (2 * rank) >= 16384 && p.K.N > 32768 && rows * 2 * rank <= kSMs) rank *= 2;
  const int64_t slice = (p.K.N + rank - 1) / rank;
  const bool held = slice <= kHeldKeys;
  auto kernel = held ? evict_select_kernel<true> : evict_select_kernel<false>;
  static std::atomic<uint64_t> done[2];
  cudaError_t e = allow_smem(kernel, kHistBytes + (held ? kHeldKeys * 4 : 0), done[held]);
  if (e != cudaSuccess) return e;
  e = launch_after(kernel, static_cast<unsigned>(rows * rank), kThreads,
                   kHistBytes + (held ? static_cast<int>(slice) * 4 : 0), rank, s, p, rank);
  if (e != cudaSuccess) return e;
  return launch_after(p.K.D == 128 ? evict_gather_kernel<128> : evict_gather_kernel<64>, static_cast<unsigned>(ctas),
                      256, 0, 1, s, p);
}

}  // namespace pbs
