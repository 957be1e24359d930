// pbs_key_mass: attention weight per key,
//   mass[j] = decay prev[j] + sum over rows r that see j of 2^(x_rj - y_r),
// x_rj = scale log2(e) Q[r].K[j], y_r = log2(e) lse[r], over the query rows of
// all heads of a KV head.  Products and exponentials in fp32; the weights of up
// to 128 rows are added in fp32, those sums in fp64 (a prompt adds tens of
// thousands of small terms to one key), or in fp32 where there are at most eight: in
// launches of two, with the mass so far rounded to fp32 after each, which for weights
// that are never negative is 2^-24 of the result a launch.
// No atomics: a key's sum has one owner, or parts that a second kernel adds in order.
//
// The keys are the rows of the MMA in all kernels (S^T = K Q^T), so that a
// thread's values belong to one key and are summed in registers.
#include <math.h>

#include <algorithm>

#include "cache_common.cuh"
#include "mma_sync.cuh"

namespace pbs {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// What is written for key j of row `bh` of the outputs, given its sum.
__device__ __forceinline__ void write_mass(const KeyMassParams& p, int64_t bh, int64_t j, int L, double sum) {
  float x = 0.f;
  if (j < L) x = static_cast<float>(p.prev ? static_cast<double>(p.decay) * p.prev[bh * p.prev_stride + j] + sum : sum);
  p.mass[bh * p.mass_stride + j] = x;
}

// Sums 2^(scale s - y) over 32 columns of a product (`v`, one key a thread) into a2, the
// whole of it or the columns in `see`.  A column that is left out is taken out of the
// finished exponent: its own s or y may be NaN.
template <bool WHOLE>
__device__ __forceinline__ void add_weights(const uint32_t (&v)[32], const float* ny, unsigned long long sc2,
                                            uint32_t see, unsigned long long (&a2)[4]) {
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const ulonglong2 n2 = *reinterpret_cast<const ulonglong2*>(ny + e);
    float t[4];
    f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sc2, n2.x), t[0], t[1]);
    f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), sc2, n2.y), t[2], t[3]);
    if (!WHOLE) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (!(see & (1u << (e + q)))) t[q] = -INFINITY;
    }
    a2[(e / 2) & 3] = f2_add(a2[(e / 2) & 3], f2_pack(ex2(t[0]), ex2(t[1])));
    a2[(e / 2 + 1) & 3] = f2_add(a2[(e / 2 + 1) & 3], f2_pack(ex2(t[2]), ex2(t[3])));
  }
}
// Bits of the columns c .. c + 31 that lie in c_lo .. c_hi - 1.
__device__ __forceinline__ uint32_t columns_in(int c, int c_lo, int c_hi) {
  const int lo = c_lo - c, up = c_hi - c;
  return (up <= 0 ? 0u : up >= 32 ? ~0u : (1u << up) - 1u) & ~(lo <= 0 ? 0u : lo >= 32 ? ~0u : (1u << lo) - 1u);
}

// ------------------------------------------------------------------ few rows
// Up to 16 query rows per KV head (a decode step).  Four warps per CTA; each
// warp streams groups of 16 keys through a private cp.async ring and multiplies
// them as the A operand of m16n8k16 (keys x rows); the queries stay in registers
// as the B operand.  Groups that no row sees (outside a window) are not among them:
// their mass is carried over beside the first loads.  The CTAs take groups in turn.
// Bound: HBM, 2 D bytes per visible key.  Measured: 32 sequences of 4096 to 8192 keys
// (Hq 32, Hkv 8, D 128) 65 us, 6.4 TB/s; 200 rows of 30000 keys under a window of 1000
// 33 us (88 with the unseen groups in the loop).
// Sixteen warps per SM (four CTAs of 48 KB) hide the chain from a group's arrival
// to its sums; with eight the schedulers issued in 41% of the cycles.
constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr int kGroup = 16;
constexpr int kFewCtas = 4;                       // per SM

template <int D, int NG>
__global__ void __launch_bounds__(kWarps * 32, kFewCtas) mass_few_kernel(const KeyMassParams p, const int n_parts) {
  constexpr int kTile = kGroup * D * 2;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  wait_for_previous_kernel();
  const int M = static_cast<int>(p.Q.N), N = static_cast<int>(p.K.N), Hq = static_cast<int>(p.Q.H);
  const int Hkv = static_cast<int>(p.K.H), G = Hq / Hkv;
  const int part = static_cast<int>(blockIdx.x) % n_parts, bh = static_cast<int>(blockIdx.x) / n_parts;
  const int b = bh / Hkv, hk = bh % Hkv;
  const int nq = cache_len(p.mask.q_len, b, M, p.err), L = cache_len(p.mask.kv_len, b, N, p.err);
  const int window = static_cast<int>(p.mask.window), n_sink = p.mask.n_sink;
  const int first = L - nq;                       // position of row 0
  // keys that some row sees: j < n_sink or j >= lo_min (and j < L); keys that every row sees end at `first`
  const int lo_min = max(0, first - window + 1);
  const int lo_max = max(0, L - window);
  const int seen_end = nq > 0 ? L : 0;
  // groups of 16 keys that hold one of them: below g_sink, and g_low to g_end
  const int g_sink = (min(n_sink, seen_end) + kGroup - 1) / kGroup;
  const int g_end = max(g_sink, (seen_end + kGroup - 1) / kGroup), g_low = min(g_end, max(g_sink, lo_min / kGroup));
  const int n_group = g_sink + g_end - g_low, gap_groups = g_low - g_sink;
  constexpr int kNone = 0x7fffff00;               // past every key
  // first key of the v-th of them
  auto key_of = [&](int v) { return v < n_group ? (v + (v < g_sink ? 0 : gap_groups)) * kGroup : kNone; };

  uint32_t qb[NG][D / 16][2];                     // Q as B fragments: row lane / 4 of each eight
  float y[NG][2];                                 // and the lse of rows 2 (lane mod 4) + {0, 1}
  int pos[NG][2];                                 // their positions; -1: no query
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int i = g * 8 + lane / 4;
    const bool valid = i < nq * G;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.Q.ptr);
    if (valid) q += b * p.Q.sB + (hk * G + i % G) * p.Q.sH + i / G * p.Q.sN + (lane & 3) * 2;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      qb[g][k][0] = valid ? *reinterpret_cast<const uint32_t*>(q + k * 16) : 0u;
      qb[g][k][1] = valid ? *reinterpret_cast<const uint32_t*>(q + k * 16 + 8) : 0u;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = g * 8 + (lane & 3) * 2 + e;
      y[g][e] = INFINITY;                         // no query
      pos[g][e] = -1;
      if (c < nq * G) {
        const float x = p.lse[(static_cast<int64_t>(b) * Hq + hk * G + c % G) * M + c / G];
        if (x != -INFINITY) {
          y[g][e] = x * kLog2e;
          pos[g][e] = first + c / G;
        }
      }
    }
  }
  const uint32_t ring = smem_u32(smem + warp * kStages * kTile);
  constexpr int CH = D / 8, RPI = 32 / CH;
  const int lc = lane % CH, lr = lane / CH;
  // this lane's chunk of its rows of group 0, and from there to its next row
  const __nv_bfloat16* kb = static_cast<const __nv_bfloat16*>(p.K.ptr) + b * p.K.sB + hk * p.K.sH + lc * 8;
  const int64_t sN = p.K.sN;
  const int stride = n_parts * kWarps;
  auto load = [&](int j0, int st) {
    if (j0 < seen_end) {
      const uint32_t dst = ring + st * kTile;
      if (j0 + kGroup <= L && (j0 >= lo_min || j0 + kGroup <= n_sink)) {
        const __nv_bfloat16* src = kb + (j0 + lr) * sN;
#pragma unroll
        for (int it = 0; it < kGroup / RPI; ++it, src += RPI * sN)
          cp_async16(dst + rows_offset<D>(it * RPI + lr, lc), src);
      } else {
#pragma unroll
        for (int it = 0; it < kGroup / RPI; ++it) {
          const int j = j0 + it * RPI + lr;
          const bool ok = j < L && (j >= lo_min || j < n_sink);
          cp_async16_zfill(dst + rows_offset<D>(it * RPI + lr, lc), kb + (ok ? j : 0) * sN, ok);
        }
      }
    }
    cp_async_commit();
  };
  // the lanes (lane mod 4) < 2 write keys 8 (lane mod 4) + lane / 4; their earlier
  // mass is read a round ahead, or its latency would be paid every round
  const int mine = (lane & 3) * 8 + lane / 4;
  const float* prev = p.prev && (lane & 3) < 2 ? p.prev + bh * p.prev_stride + mine : nullptr;
  float* mass = p.mass + bh * p.mass_stride + mine;
  auto earlier = [&](int j0) { return prev && j0 + mine < L ? prev[j0] : 0.f; };
  // this warp's group, the next and the one after
  int v = part * kWarps + warp, j0 = key_of(v), j1 = key_of(v + stride), j2;
  static_assert(kStages == 3, "two groups ahead");
  load(j0, 0);
  load(j1, 1);
  // keys of the other groups, which no row sees, while those land
  {
    const float* old = p.prev ? p.prev + bh * p.prev_stride : nullptr;
    float* out = p.mass + bh * p.mass_stride;
    const int gap = gap_groups * kGroup, n = gap + max(0, N - g_end * kGroup);
    auto at = [&](int i) { return i < gap ? g_sink * kGroup + i : g_end * kGroup + i - gap; };
    constexpr int kAhead = 4, kStep = kWarps * 32;
    for (int i = part * kAhead * kStep + tid; i < n; i += n_parts * kAhead * kStep) {
      float x[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const int j = at(i + e * kStep);
        x[e] = old && i + e * kStep < n && j < L ? p.decay * old[j] : 0.f;
      }
#pragma unroll
      for (int e = 0; e < kAhead; ++e)
        if (i + e * kStep < n) out[at(i + e * kStep)] = x[e];
    }
  }
  int st = 0;
  float next_old = earlier(j0);
  for (; j0 < seen_end; j0 = j1, j1 = j2, v += stride) {
    j2 = key_of(v + 2 * stride);
    const float old = next_old;
    next_old = earlier(j1);
    cp_async_wait<kStages - 2>();
    __syncwarp();
    load(j2, st == 0 ? kStages - 1 : st - 1);
    const uint32_t sk = ring + st * kTile;
    st = st == kStages - 1 ? 0 : st + 1;
    float sum[2] = {0.f, 0.f};                    // keys lane / 4 and 8 + lane / 4
    float s[NG][4];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[g][e] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      // matrices: keys 0-7 | 8-15 | 0-7 | 8-15, chunks 2k | 2k | 2k+1 | 2k+1
      uint32_t f[4];
      ldsm4(f, sk + rows_offset<D>((lane & 7) + (((lane >> 3) & 1) << 3), 2 * k + (lane >> 4)));
#pragma unroll
      for (int g = 0; g < NG; ++g) mma_16816(s[g], f[0], f[1], f[2], f[3], qb[g][k][0], qb[g][k][1]);
    }
    const bool full = j0 + kGroup - 1 <= first && (j0 >= lo_max || j0 + kGroup <= n_sink);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float w = ex2(fmaf(s[g][e], p.scale_log2, -y[g][e & 1]));
        const int at = pos[g][e & 1];
        if (at < 0) w = 0.f;                      // (a NaN or infinity of the key makes w NaN without a query too)
        if (!full) {
          const int j = j0 + (e >> 1) * 8 + lane / 4;
          if (j > at || (j <= at - window && j >= n_sink)) w = 0.f;
        }
        sum[e >> 1] += w;
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
      sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
    }
    if ((lane & 3) < 2 && j0 + mine < N)
      mass[j0] = j0 + mine < L ? fmaf(p.decay, old, (lane & 3) ? sum[1] : sum[0]) : 0.f;
  }
  cp_async_wait_all();
}

// ------------------------------------------------------------------ many rows
// One CTA per (256 keys, KV head, sequence, part of the query rows), the heaviest
// key tiles (the first, which the most rows see) first.  Two tiles of 128 keys stay
// in tensor memory as A operands; the query rows stream past in TMA boxes packed as
// (position, head of the group), up to 128 a box, as the B operand of both.  (With
// A in shared memory too, a 128 x 128 product reads both operands from there and
// took 0.65 us of an SM, and with one tile a box its boxes 7 TB/s of L2.)
//   warp 0  issues S^T = K Q^T, box by box for both tiles, into a ring of three
//     tensor-memory buffers;
//   warp 1  loads K once and the query boxes and their lse into rings of four;
//   warps 2-17 copy K into tensor memory, then take 2^(x - y) of every column and
//     sum it: a thread has one key and 64 of the 128 columns.
// Bound: exponentials, 16 per clock and SM on the SFU.  Measured: a prompt of 8192
// (Hq 32, Hkv 8, D 128) 344 us, 3.1 T weights/s, of which the SFU needs 231; the
// products and hand-offs alone take 288.  A ring of four buffers with K in shared
// memory takes 396, products of 64 columns 458.
constexpr int kWideThreads = 576;
constexpr int kConsumerWarps = 16;
constexpr int kQStages = 4;

template <int D>
struct MassCfg {
  static constexpr int kTile = (D / 64) * 128 * 128;
  static constexpr int kBytes = (2 + kQStages) * kTile + 1024;
  static constexpr int kSmem = kBytes > 120 * 1024 ? kBytes : 120 * 1024;   // one CTA per SM: all of tensor memory
};

template <int D>
__global__ void __launch_bounds__(kWideThreads, 1) mass_wide_kernel(const KeyMassParams p, const int n_parts,
                                                                    const int pm, double* __restrict__ partial,
                                                                    const __grid_constant__ CUtensorMap mq,
                                                                    const __grid_constant__ CUtensorMap mk) {
  using C = MassCfg<D>;
  constexpr int NS = kQStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t bar_k, bar_q[NS], bar_qempty[NS], bar_y[NS], bar_yempty[NS], bar_a, bar_s[3], bar_sfree[3];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_sh;
  __shared__ __align__(16) float ny[NS][128];         // -log2(e) lse of the box's rows
  __shared__ uint2 live[NS][2];                       // bits of the rows that add something (lse not -inf)
  __shared__ double half_sum[256];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  wait_for_previous_kernel();
  const int M = static_cast<int>(p.Q.N), N = static_cast<int>(p.K.N), Hq = static_cast<int>(p.Q.H);
  const int Hkv = static_cast<int>(p.K.H), G = Hq / Hkv, BH = static_cast<int>(p.K.B) * Hkv;
  const int part = static_cast<int>(blockIdx.x) % n_parts, rest = static_cast<int>(blockIdx.x) / n_parts;
  const int bh = rest % BH, j0 = rest / BH * 256, b = bh / Hkv, hk = bh % Hkv;
  const int nq = cache_len(p.mask.q_len, b, M, p.err), L = cache_len(p.mask.kv_len, b, N, p.err);
  const int window = static_cast<int>(p.mask.window), n_sink = p.mask.n_sink;
  const int64_t first = L - nq;
  // query rows that see some key of these tiles: r0 <= r < r1, then this part's boxes of pm positions
  const int64_t last_key = min(j0 + 255, L - 1);
  int64_t r0 = max(static_cast<int64_t>(0), j0 - first), r1 = nq;
  if (j0 >= n_sink) r1 = min(r1, last_key + window - first);
  if (j0 >= L || r1 <= r0) r0 = r1 = 0;
  const int n_box = static_cast<int>((r1 - r0 + pm - 1) / pm);
  const int x0 = static_cast<int>(static_cast<int64_t>(n_box) * part / n_parts);
  const int x1 = static_cast<int>(static_cast<int64_t>(n_box) * (part + 1) / n_parts);
  const int cols = pm * G, n_mma = (cols + 15) / 16 * 16, n_tile = j0 + 128 < L ? 2 : 1;
  double* mine = n_parts > 1 ? partial + (static_cast<int64_t>(part) * BH + bh) * N : nullptr;
  if (x0 == x1) {                                 // nothing sees these keys here
    if (tid < 256 && j0 + tid < N) {
      if (mine) mine[j0 + tid] = 0.0;
      else write_mass(p, bh, j0 + tid, L, 0.0);
    }
    return;
  }

  const uint32_t sK = smem_u32(smem), sQ = smem_u32(smem + 2 * C::kTile);
  // MMA columns past the box: zero rows (the boxes never write them)
  for (int i = tid; i < NS * (n_mma - cols) * (D / 8); i += kWideThreads) {
    const int c = i % (D / 8), r = cols + i / (D / 8) % (n_mma - cols), s = i / (D / 8) / (n_mma - cols);
    *reinterpret_cast<uint4*>(smem + (2 + s) * C::kTile + (c / 8) * (128 * 128) + sw128_offset(r, c % 8)) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async();
  if (warp == 0) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    abort_sh = 0;
    mbar_init(&bar_k, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&bar_q[i], 1);
      mbar_init(&bar_qempty[i], 1);
      mbar_init(&bar_y[i], 32);
      mbar_init(&bar_yempty[i], 8 * n_tile);
    }
    mbar_init(&bar_a, 8 * n_tile);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&bar_s[i], 1);
      mbar_init(&bar_sfree[i], 8);
    }
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  volatile int* abort_flag = &abort_sh;

  if (warp == 1) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      mbar_expect_tx(&bar_k, static_cast<uint32_t>(n_tile * C::kTile));
      for (int h = 0; h < n_tile; ++h)
        for (int c = 0; c < D / 64; ++c)
          tma_rows_4d(sK + h * C::kTile + c * (128 * 128), &mk, c * 64, j0 + 128 * h, p.K.sH == 0 ? 0 : hk,
                      p.K.sB == 0 ? 0 : b, &bar_k);
    }
    auto load_box = [&](int x) {                  // (one lane)
      const int s = (x - x0) % NS;
      mbar_expect_tx(&bar_q[s], static_cast<uint32_t>(cols * D * 2));
      for (int c = 0; c < D / 64; ++c)
        tma_rows_4d(sQ + s * C::kTile + c * (128 * 128), &mq, c * 64, hk * G, static_cast<int>(r0 + x * pm), b,
                    &bar_q[s]);
    };
    int issued = min(x1, x0 + NS);
    if (lane == 0)
      for (int x = x0; x < issued; ++x) load_box(x);
    // The lse of this lane's rows lane, lane + 32, ... of box x, of four boxes at a
    // time and four boxes ahead: one at a time, one ahead, its latency was what
    // every box took.
    const float* lse[4];
    int in_box[4];                                // the row's position in the box; past its end: never a query
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = lane + 32 * e;
      in_box[e] = c < cols ? c / G : 0x40000000;
      lse[e] = p.lse + (static_cast<int64_t>(b) * Hq + hk * G + c % G) * M + r0 + c / G;
    }
    const int n_left = static_cast<int>(nq - r0);
    auto lse_of = [&](int x, float (&v)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = x < x1 && x * pm + in_box[e] < n_left ? lse[e][x * pm] : -INFINITY;    // -inf: the row adds nothing
      }
    };
    float v[NS][4], ahead[NS][4];
    bool ok = true;
#pragma unroll
    for (int q = 0; q < NS; ++q) lse_of(x0 + q, v[q]);
    for (int xb = x0; ok && xb < x1; xb += NS) {
#pragma unroll
      for (int q = 0; q < NS; ++q) lse_of(xb + NS + q, ahead[q]);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int x = xb + s, i = x - x0;
        if (x >= x1 || !ok) break;
        if (i >= NS) {
          ok = mbar_wait_or_abort(&bar_qempty[s], (i / NS - 1) & 1, p.err, abort_flag);
          if (ok = __all_sync(0xffffffffu, ok); !ok) break;
          if (lane == 0) load_box(x);
          issued = x + 1;
          ok = mbar_wait_or_abort(&bar_yempty[s], (i / NS - 1) & 1, p.err, abort_flag);
          if (ok = __all_sync(0xffffffffu, ok); !ok) break;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ny[s][lane + 32 * e] = -v[s][e] * kLog2e;
          const uint32_t some = __ballot_sync(0xffffffffu, v[s][e] != -INFINITY);
          if (lane == e) reinterpret_cast<uint32_t*>(live[s])[e] = some;
        }
        mbar_arrive(&bar_y[s]);
      }
#pragma unroll
      for (int q = 0; q < NS; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[q][e] = ahead[q][e];
    }
    // no copy may be in flight when the CTA ends; without an abort the other
    // roles have waited for all of them
    if (*abort_flag) {
      mbar_wait(&bar_k, 0, p.err);
      for (int x = max(x0, issued - NS); x < issued; ++x)
        mbar_wait(&bar_q[(x - x0) % NS], ((x - x0) / NS) & 1, p.err);
    }
  } else if (warp == 0) {
    // ---------------------------------------------------------------- MMA
    const uint32_t idesc = idesc_bf16(128, n_mma, false);
    bool ok = __all_sync(0xffffffffu, mbar_wait_or_abort(&bar_a, 0, p.err, abort_flag));
    int u = 0, d = 0, par = 0;                    // products so far; the next one's buffer and its parity
    for (int x = x0; ok && x < x1; ++x) {
      const int i = x - x0, s = i % NS;
      ok = mbar_wait_or_abort(&bar_q[s], (i / NS) & 1, p.err, abort_flag);
      const uint64_t b0 = sdesc_sw128(sQ + s * C::kTile, 16, 1024);
      for (int h = 0; h < n_tile; ++h, ++u) {
        if (ok && u >= 3) ok = mbar_wait_or_abort(&bar_sfree[d], par ^ 1, p.err, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * (128 * 128) + (kk % 4) * 32;
          if (elect_one())
            mma_ts(tmem + 128 + d * 128, tmem + h * 64 + kk * 8, sdesc_add(b0, off), idesc, kk > 0 ? 1u : 0u);
        }
        if (elect_one()) {
          tc_commit(&bar_s[d]);
          if (h == n_tile - 1) tc_commit(&bar_qempty[s]);
        }
        __syncwarp();
        if (++d == 3) {
          d = 0;
          par ^= 1;
        }
      }
    }
  } else {
    // ----------------------------------------------------------- consumers
    const int tile = (warp - 2) >> 3, half = ((warp - 2) >> 2) & 1;
    const int key = tile * 128 + (warp & 3) * 32 + lane;      // lane of tensor memory within the tile
    const int64_t j = j0 + key;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 128 + half * 64 + lanes;
    const unsigned long long sc2 = f2_pack(p.scale_log2, p.scale_log2);
    double sum = 0.0;
    if (tile < n_tile) {
      // this key's half of its row into tensor memory: column c holds elements 2c, 2c + 1
      mbar_wait_or_abort(&bar_k, 0, p.err, abort_flag);
      const unsigned char* row = smem + tile * C::kTile;
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {          // 32 elements at a time
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int chunk = half * (D / 16) + q * 4 + e;
          const uint4 v = *reinterpret_cast<const uint4*>(row + (chunk / 8) * (128 * 128) +
                                                          sw128_offset(key & 127, chunk % 8));
          w[4 * e] = v.x;
          w[4 * e + 1] = v.y;
          w[4 * e + 2] = v.z;
          w[4 * e + 3] = v.w;
        }
        tmem_st16(tmem + tile * 64 + half * (D / 4) + q * 16 + lanes, w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_a);
    }
    for (int x = x0; tile < n_tile && x < x1; ++x) {
      const int i = x - x0, s = i % NS, u = i * n_tile + tile, d = u % 3;
      // (after an abort the waits return at once; the sums are then meaningless
      // and the error word says so)
      mbar_wait_or_abort(&bar_y[s], (i / NS) & 1, p.err, abort_flag);
      mbar_wait_or_abort(&bar_s[d], (u / 3) & 1, p.err, abort_flag);
      tc_fence_after();
      // rows of the box that see this key: c_lo <= c < c_hi
      // (32 bits: at >= j0 from row r0 on, so -N <= j - at < 256 and window <= N)
      const int row = static_cast<int>(r0) + x * pm, at = static_cast<int>(first) + row;
      const int ahead = static_cast<int>(j) - at;
      const int hi = j < n_sink ? nq - row : min(nq - row, ahead + window);
      const int c_lo = min(pm, max(0, ahead)) * G, c_hi = j < L ? min(pm, max(0, hi)) * G : 0;
      const uint2 some = live[s][half];
      const bool full = __all_sync(0xffffffffu, c_lo == 0 && c_hi == 128 && (some.x & some.y) == ~0u);
      const bool none = __all_sync(0xffffffffu, c_lo >= c_hi);
      unsigned long long a2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1
      for (int c = half * 64; c < min(none ? 0 : n_mma, half * 64 + 64); c += 32) {
        uint32_t v[32];
        tmem_ld32(tS + d * 128 + (c & 32), v);
        if (full) add_weights<true>(v, &ny[s][c], sc2, ~0u, a2);
        else                                      // (columns past the box are past c_hi)
          add_weights<false>(v, &ny[s][c], sc2, columns_in(c, c_lo, c_hi) & (c & 32 ? some.y : some.x), a2);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar_sfree[d]);
        mbar_arrive(&bar_yempty[s]);
      }
      float s0, s1, s2, s3, s4, s5, s6, s7;
      f2_unpack(a2[0], s0, s1);
      f2_unpack(a2[1], s2, s3);
      f2_unpack(a2[2], s4, s5);
      f2_unpack(a2[3], s6, s7);
      sum += static_cast<double>(((s0 + s1) + (s2 + s3)) + ((s4 + s5) + (s6 + s7)));
    }
    if (half == 1) half_sum[key] = sum;
    named_sync(1, kConsumerWarps * 32);
    if (half == 0 && j < N) {
      sum += half_sum[key];
      if (mine) mine[j] = sum;
      else write_mass(p, bh, j, L, sum);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------- some hundred rows
// Up to 256 query rows per KV head (drafted tokens, the last rows of a prompt); in up to
// four launches, each adding to the one before, 1024 over many keys.  The other way
// round: the queries (one or two boxes) and their lse stay in shared memory and the
// key tiles stream past, through a ring of four, in pairs that two groups of eight
// consumer warps take.  Each group has two tensor-memory buffers.  CTAs are one per
// SM; those of one (sequence, KV head) share its visible tiles in turn.
// Bound: HBM for the keys, with many rows the exponentials and the products, which
// read both operands from shared memory.  Measured: 61 rows of two sequences (3 heads a
// group, D 64) over 9061 visible of 20011 keys 13 us; 256 rows (8 KV heads, D 128) over
// 32768 keys 33 us.
constexpr int kKStages = 4;

template <int D>
struct MidCfg {
  static constexpr int kTile = (D / 64) * 128 * 128;
  static constexpr int kBytes = (2 + kKStages) * kTile + 1024;
  static constexpr int kSmem = kBytes > 120 * 1024 ? kBytes : 120 * 1024;   // one CTA per SM: all of tensor memory
};

template <int D>
__global__ void __launch_bounds__(kWideThreads, 1) mass_mid_kernel(const KeyMassParams p, const int n_parts,
                                                                   const int pm, const int base,
                                                                   const __grid_constant__ CUtensorMap mq,
                                                                   const __grid_constant__ CUtensorMap mk) {
  using C = MidCfg<D>;
  constexpr int NS = kKStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t bar_q, bar_k[NS], bar_kempty[NS], bar_s[4], bar_sfree[4];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_sh;
  __shared__ __align__(16) float ny[2][128];          // -log2(e) lse of the boxes' rows
  __shared__ uint2 live[2][2];                        // bits of the rows that add something (lse not -inf)
  __shared__ float group_sum[2][2][128];              // [group][parity of the pair][key]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  wait_for_previous_kernel();
  const int M = static_cast<int>(p.Q.N), N = static_cast<int>(p.K.N), Hq = static_cast<int>(p.Q.H);
  const int Hkv = static_cast<int>(p.K.H), G = Hq / Hkv;
  const int part = static_cast<int>(blockIdx.x) % n_parts, bh = static_cast<int>(blockIdx.x) / n_parts;
  const int b = bh / Hkv, hk = bh % Hkv;
  // this launch's query rows: from row `base`
  const int nq_all = cache_len(p.mask.q_len, b, M, p.err), nq = min(2 * pm, max(0, nq_all - base));
  const int L = cache_len(p.mask.kv_len, b, N, p.err);
  const int window = static_cast<int>(p.mask.window), n_sink = p.mask.n_sink;
  const int first = L - nq_all + base;                // position of row `base`
  // tiles that some row sees: those of the sinks, then those of the window
  const int end_t = nq > 0 ? (L + 127) / 128 : 0;
  const int sink_t = min((n_sink + 127) / 128, end_t), low_t = max(sink_t, max(0, first - window + 1) / 128);
  const int n_tiles = sink_t + max(0, end_t - low_t), n_pairs = (n_tiles + 1) / 2;
  const int my_pairs = part < n_pairs ? (n_pairs - part + n_parts - 1) / n_parts : 0;
  auto tile_of = [&](int v) { return v < sink_t ? v : v - sink_t + low_t; };
  // does group g have a tile in the CTA's pair i, and which?
  auto has = [&](int i, int g) { return 2 * (part + i * n_parts) + g < n_tiles; };
  auto tile_at = [&](int i, int g) { return tile_of(2 * (part + i * n_parts) + g); };
  const int cols = pm * G, n_mma = (cols + 15) / 16 * 16, n_box = min(2, (nq + pm - 1) / pm);
  const float* prev = p.prev ? p.prev + bh * p.prev_stride : nullptr;
  float* mass = p.mass + bh * p.mass_stride;
  // keys that no row sees
  for (int64_t j = static_cast<int64_t>(part) * kWideThreads + tid; j < N; j += n_parts * kWideThreads) {
    const int t = static_cast<int>(j >> 7);
    if (t < sink_t || (t >= low_t && t < end_t)) continue;
    mass[j] = j < L && prev ? p.decay * prev[j] : 0.f;
  }
  if (my_pairs == 0) return;

  const uint32_t sQ = smem_u32(smem), sK = smem_u32(smem + 2 * C::kTile);
  // MMA columns past the box: zero rows (the boxes never write them)
  for (int i = tid; i < 2 * (n_mma - cols) * (D / 8); i += kWideThreads) {
    const int c = i % (D / 8), r = cols + i / (D / 8) % (n_mma - cols), s = i / (D / 8) / (n_mma - cols);
    *reinterpret_cast<uint4*>(smem + s * C::kTile + (c / 8) * (128 * 128) + sw128_offset(r, c % 8)) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async();
  if (tid < 256) {
    const int c = tid & 127, r = (tid >> 7) * pm + c / G;
    const int64_t at = (static_cast<int64_t>(b) * Hq + hk * G + c % G) * M + base + r;
    const float l = c < cols && r < nq ? p.lse[at] : -INFINITY;
    ny[tid >> 7][c] = -l * kLog2e;
    const uint32_t some = __ballot_sync(0xffffffffu, l != -INFINITY);      // (-inf: the row adds nothing)
    if (lane == 0) reinterpret_cast<uint32_t*>(live)[warp] = some;
  }
  if (warp == 0) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    abort_sh = 0;
    mbar_init(&bar_q, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&bar_k[i], 1);
      mbar_init(&bar_kempty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar_s[i], 1);
      mbar_init(&bar_sfree[i], 8);
    }
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  volatile int* abort_flag = &abort_sh;

  if (warp == 1) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      mbar_expect_tx(&bar_q, static_cast<uint32_t>(n_box * cols * D * 2));
      for (int x = 0; x < n_box; ++x)
        for (int c = 0; c < D / 64; ++c)
          tma_rows_4d(sQ + x * C::kTile + c * (128 * 128), &mq, c * 64, hk * G, base + x * pm, b, &bar_q);
      int f = 0;                                      // tiles issued
      bool ok = true;
      for (int i = 0; ok && i < my_pairs; ++i) {
        for (int g = 0; g < 2 && has(i, g); ++g) {
          const int s = f % NS;
          if (f >= NS) ok = mbar_wait_or_abort(&bar_kempty[s], (f / NS - 1) & 1, p.err, abort_flag);
          if (!ok) break;
          mbar_expect_tx(&bar_k[s], C::kTile);
          for (int c = 0; c < D / 64; ++c)
            tma_rows_4d(sK + s * C::kTile + c * (128 * 128), &mk, c * 64, tile_at(i, g) * 128, p.K.sH == 0 ? 0 : hk,
                        p.K.sB == 0 ? 0 : b, &bar_k[s]);
          ++f;
        }
      }
      // no copy may be in flight when the CTA ends; without an abort the MMA
      // role has waited for all of them
      if (*abort_flag) {
        mbar_wait(&bar_q, 0, p.err);
        for (int i = max(0, f - NS); i < f; ++i) mbar_wait(&bar_k[i % NS], (i / NS) & 1, p.err);
      }
    }
    __syncwarp();
  } else if (warp == 0) {
    // ---------------------------------------------------------------- MMA
    const uint32_t idesc = idesc_bf16(128, n_mma, false);
    bool ok = __all_sync(0xffffffffu, mbar_wait_or_abort(&bar_q, 0, p.err, abort_flag));
    int f = 0, n = 0;                                 // tiles before this pair; products per group
    for (int i = 0; ok && i < my_pairs; ++i) {
      const int n_g = has(i, 1) ? 2 : 1;
      for (int x = 0; ok && x < n_box; ++x, ++n) {
        for (int g = 0; g < n_g; ++g) {
          const int s = (f + g) % NS, d = g * 2 + (n & 1);
          if (x == 0) ok = mbar_wait_or_abort(&bar_k[s], ((f + g) / NS) & 1, p.err, abort_flag);
          if (ok && n >= 2) ok = mbar_wait_or_abort(&bar_sfree[d], (n / 2 - 1) & 1, p.err, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a0 = sdesc_sw128(sK + s * C::kTile, 16, 1024);
          const uint64_t b0 = sdesc_sw128(sQ + x * C::kTile, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk / 4) * (128 * 128) + (kk % 4) * 32;
            if (elect_one())
              mma_ss(tmem + d * 128, sdesc_add(a0, off), sdesc_add(b0, off), idesc, kk > 0 ? 1u : 0u);
          }
          if (elect_one()) {
            tc_commit(&bar_s[d]);
            if (x == n_box - 1) tc_commit(&bar_kempty[s]);
          }
          __syncwarp();
        }
      }
      f += n_g;
    }
  } else {
    // ----------------------------------------------------------- consumers
    const int g = (warp - 2) >> 3, half = ((warp - 2) >> 2) & 1, key = (warp & 3) * 32 + lane;
    const uint32_t tS = tmem + g * 256 + half * 64 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const unsigned long long sc2 = f2_pack(p.scale_log2, p.scale_log2);
    int n = 0;                                        // products of this group
    // (after an abort the waits return at once; the sums are then meaningless and
    // the error word says so)
    for (int i = 0; i < my_pairs; ++i) {
      if (!has(i, g)) continue;
      const int j = tile_at(i, g) * 128 + key;
      const float old = prev && half == 0 && j < L ? prev[j] : 0.f;
      float sum = 0.f;
      for (int x = 0; x < n_box; ++x, ++n) {
        const int d = n & 1;
        mbar_wait_or_abort(&bar_s[g * 2 + d], (n / 2) & 1, p.err, abort_flag);
        tc_fence_after();
        // rows of the box that see this key: c_lo <= c < c_hi
        const int row = x * pm, at = first + row;
        const int ahead = j - at;                     // at most 128 + 256, before the window is added
        const int hi = j < n_sink ? nq - row : min(nq - row, ahead + window);
        const int c_lo = min(pm, max(0, ahead)) * G, c_hi = j < L ? min(pm, max(0, hi)) * G : 0;
        const uint2 some = live[x][half];
        const bool full = __all_sync(0xffffffffu, c_lo == 0 && c_hi == 128 && (some.x & some.y) == ~0u);
        const bool none = __all_sync(0xffffffffu, c_lo >= c_hi);
        unsigned long long a2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1
        for (int c = half * 64; c < min(none ? 0 : n_mma, half * 64 + 64); c += 32) {
          uint32_t v[32];
          tmem_ld32(tS + d * 128 + (c & 32), v);
          if (full) add_weights<true>(v, &ny[x][c], sc2, ~0u, a2);
          else                                        // (columns past the box are past c_hi)
            add_weights<false>(v, &ny[x][c], sc2, columns_in(c, c_lo, c_hi) & (c & 32 ? some.y : some.x), a2);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_sfree[g * 2 + d]);
        float s0, s1, s2, s3, s4, s5, s6, s7;
        f2_unpack(a2[0], s0, s1);
        f2_unpack(a2[1], s2, s3);
        f2_unpack(a2[2], s4, s5);
        f2_unpack(a2[3], s6, s7);
        sum += ((s0 + s1) + (s2 + s3)) + ((s4 + s5) + (s6 + s7));
      }
      if (half == 1) group_sum[g][i & 1][key] = sum;
      named_sync(1 + g, 256);
      if (half == 0 && j < N) mass[j] = j < L ? fmaf(p.decay, old, sum + group_sum[g][i & 1][key]) : 0.f;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

__global__ void __launch_bounds__(256) mass_join_kernel(const KeyMassParams p, const int n_parts,
                                                        const double* __restrict__ partial) {
  wait_for_previous_kernel();
  const int64_t N = p.K.N, BH = p.K.B * p.K.H, blocks = (N + 255) / 256, bh = blockIdx.x / blocks;
  const int64_t j = blockIdx.x % blocks * 256 + threadIdx.x;
  if (j >= N) return;
  double sum = 0.0;
  for (int s = 0; s < n_parts; ++s) sum += partial[(s * BH + bh) * N + j];
  write_mass(p, bh, j, cache_len(p.mask.kv_len, bh / p.K.H, N, p.err), sum);
}

constexpr int kFewRows = 16;
constexpr int kMaxParts = 8;

// Launches of mass_mid_kernel, two boxes of query rows each, that take all rows, or
// 0 where mass_wide_kernel does: more than one launch where that kernel's key tiles
// would take several rounds of CTAs, each with its set-up, and at most four (sums of
// a launch are fp32).  512 rows over 32768 keys (8 KV heads, D 128) take 64 us in two
// launches, 85 there; 1024 rows of 8 sequences over 8192 233 in four, 256 there; but
// 400 rows over 2 x 2048 15.6 in two, 12.9 there.
int mid_launches(const TensorDesc& Q, const TensorDesc& K) {
  const int64_t per = 2 * (128 / (Q.H / K.H)), n = (Q.N + per - 1) / per;
  const bool rounds = (K.N + 255) / 256 * K.B * K.H > kSMs;
  return n == 1 || (rounds && n <= 4) ? static_cast<int>(n) : 0;
}

// Parts that the query rows are cut into: two where a CTA would run 256 boxes one
// after the other (the first keys of a prompt are seen by all its rows), more where
// there are fewer key tiles than SMs, at least four boxes each.  A prompt of 8192
// takes 358, 349 and 367 us in 1, 2 and 4 parts, one of 2048 95, 54 and 39.
int mass_parts(const TensorDesc& Q, const TensorDesc& K) {
  const int64_t G = Q.H / K.H, tiles = (K.N + 255) / 256 * K.B * K.H;
  if (mid_launches(Q, K) > 0) return 1;
  const int64_t boxes = (Q.N * G + 127) / 128;
  const int64_t parts = std::max(2 * kSMs / tiles, std::min<int64_t>(2, boxes / 128));
  return static_cast<int>(std::max<int64_t>(1, std::min({parts, boxes / 4, static_cast<int64_t>(kMaxParts)})));
}

template <int D>
cudaError_t launch(const KeyMassParams& p, cudaStream_t s) {
  const int64_t G = p.Q.H / p.K.H, rows = p.Q.N * G, BH = p.K.B * p.K.H;
  if (rows <= kFewRows) {
    const int64_t rounds = (p.K.N + kWarps * kGroup - 1) / (kWarps * kGroup);
    // One CTA for every place on the chip and no more, with two rounds of keys at
    // least; 16 rounds of visible keys a CTA where that makes more of them, so that sequences of
    // unequal length even out.  8 KV-head rows of 4096 keys take 4.0 us in 32 parts
    // (6.0 in 8); 64 rows of up to 8192 20.4 us in 9 (23.0 in 10, which take a second
    // round); 256 rows 66 us in 8 (73 in 3), of 2048 36 us in 2 (38 in 5).
    const int64_t seen = std::min(rounds, (p.mask.window + p.mask.n_sink + p.Q.N) / (kWarps * kGroup) + 2);
    const int64_t want = std::max(kFewCtas * kSMs / BH, seen / 16);
    const int parts = static_cast<int>(std::max<int64_t>(1, std::min(rounds / 2, want)));
    const int bytes = kWarps * kStages * kGroup * D * 2;
    static std::atomic<uint64_t> done[2];
    auto kernel = rows <= 8 ? mass_few_kernel<D, 1> : mass_few_kernel<D, 2>;
    const cudaError_t e = allow_smem(kernel, bytes, done[rows <= 8]);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, static_cast<unsigned>(BH * parts), kWarps * 32, bytes, 1, s, p, parts);
  }
  const int pm = static_cast<int>(std::min(p.Q.N, 128 / G));
  CUtensorMap mq, mk;
  if (!encode_queries_map(&mq, p.Q, static_cast<int>(G), pm, 1) || !encode_keys_map(&mk, p.K, 128))
    return cudaErrorNotSupported;
  if (mid_launches(p.Q, p.K) > 0) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(mass_mid_kernel<D>, MidCfg<D>::kSmem, done);
    if (e != cudaSuccess) return e;
    const int64_t pairs = (p.K.N + 255) / 256;
    const int parts = static_cast<int>(std::max<int64_t>(1, std::min(pairs, kSMs / BH)));
    KeyMassParams q = p;
    for (int base = 0; base < p.Q.N; base += 2 * pm) {
      const cudaError_t e = launch_after(mass_mid_kernel<D>, static_cast<unsigned>(BH * parts), kWideThreads,
                                         MidCfg<D>::kSmem, 1, s, q, parts, pm, base, mq, mk);
      if (e != cudaSuccess) return e;
      q.prev = p.mass;                                // the rows so far
      q.prev_stride = p.mass_stride;
      q.decay = 1.0f;
    }
    return cudaSuccess;
  }
  const int parts = mass_parts(p.Q, p.K);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(mass_wide_kernel<D>, MassCfg<D>::kSmem, done);
  if (e != cudaSuccess) return e;
  const int64_t ctas = (p.K.N + 255) / 256 * BH * parts;
  if (ctas >= (1ll << 31)) return cudaErrorInvalidValue;
  double* partial = static_cast<double*>(p.ws);
  e = launch_after(mass_wide_kernel<D>, static_cast<unsigned>(ctas), kWideThreads, MassCfg<D>::kSmem, 1, s, p, parts,
                   pm, partial, mq, mk);
  if (e != cudaSuccess || parts == 1) return e;
  return launch_after(mass_join_kernel, static_cast<unsigned>((p.K.N + 255) / 256 * BH), 256, 0, 1, s, p, parts,
                      partial);
}

}  // namespace

size_t key_mass_ws_bytes(const TensorDesc& Q, const TensorDesc& K) {
  const int parts = mass_parts(Q, K);
  return parts == 1 ? 0 : static_cast<size_t>(parts) * K.B * K.H * K.N * sizeof(double);
}

cudaError_t launch_key_mass(const KeyMassParams& p, cudaStream_t s) {
  return p.Q.D == 128 ? launch<128>(p, s) : launch<64>(p, s);
}

}  // namespace pbs
