// pbs_attn_window and pbs_attn_prefix: attention over a K/V cache.
//
//   O[r] = sum_j 2^(x_rj - m_r) V[j] / l_r,  x_rj = scale log2(e) Q[r].K[j],
//   m_r = max_j x_rj,  l_r = sum_j 2^(x_rj - m_r),  lse_r = ln 2 (m_r + log2 l_r)
//
// over the keys j that row r sees, in one pass with the running (m, l, O)
// rescaled whenever m grows.  The key axis may be cut into parts: the CTAs of a
// cluster join theirs through distributed shared memory; what several clusters
// (or several CTAs of the tcgen05 kernel) leave in fp32, attn_join_kernel adds.
//
// Query rows of one KV head that read the same keys run together: the G heads
// of the group, the M new tokens and, over a shared prefix, the sequences.  Up
// to 32 such rows (a decode step) are bound by the bytes of K and V and run in
// attn_few_kernel below, 8 or 16 rows a CTA (a second block of rows finds the keys
// in L2); more rows run on the tcgen05 kernel of cache_attn_wide.cu.  With a prefix
// of many rows the two kernels run side by side: one is bound by products, the other
// by HBM.
#include <math.h>

#include <algorithm>

#include "cache_attn.cuh"
#include "mma_sync.cuh"

namespace pbs {
namespace {

// ------------------------------------------------------------------ few rows
// One CTA of four warps per (KV head, sequence, part of the keys).  Each warp
// streams its own groups of 16 keys through a private ring of cp.async stages,
// so nothing but the end synchronises the CTA, and keeps its own (m, l, O):
//   S = Q K^T  mma m16n8k16, rows = queries (8 per row group), B = K by ldmatrix;
//   P = 2^(S - m) split into two bf16, P = hi + lo: the rows 8-15 of the tile
//   that the queries leave free carry lo, so one mma gives hi V and lo V in the
//   same thread and P is effectively held in 16 bits of mantissa;
//   O += P V   with V by ldmatrix.trans.
// 16 query rows are two such groups: one QK^T tile, two PV tiles.
// Bound: HBM, 4 D bytes per key.  Measured: 64 sequences with 4100 visible keys each
// (Hq 32, Hkv 8, D 128) 157 us, 6.9 TB/s; one sequence with 260 7.0 us, of which 2
// are the launch and the rest one chain of load, products and joins.
constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr int kGroup = 16;                      // keys per warp and stage
constexpr int kMaxRank = 8;                     // CTAs per cluster

template <int D>
struct FewCfg {
  static constexpr int kTile = kGroup * D * 2;                 // one K or V group
  static constexpr int kRing = kStages * 2 * kTile;            // per warp
  static constexpr int kBytes = kWarps * kRing;
};

// What each row of the CTA is, in shared memory.
struct FewRow {
  int lo, hi;          // bounds of its visible indices (see KeyRun); hi < 0: none
  int out;             // row (b * Hq + h) * M + r of the outputs, -1: not computed
};

// A group of keys that only some rows see and that holds NaN or infinities
// among its values (rare): add those entries to the rows that do see them --
// exp is never zero, so such an entry is what its column becomes -- and zero
// them for the product.  Whole warp; 8 j + 2 (lane mod 4) + {0, 1} are a
// thread's columns.  (Inline: out of line, `o` would live in local memory.)
template <int D, int NG>
__device__ __forceinline__ void few_nonfinite(unsigned char* v, const FewRow* row, int n_sink, int v0, int lane,
                                           float (&o)[NG][D / 8][4]) {
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const FewRow me = row[g * 8 + lane / 4];
#pragma unroll 1
    for (int k = 0; k < kGroup; ++k) {
      const int i = v0 + k;
      if (i > me.hi || (i < me.lo && i >= n_sink)) continue;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(v + rows_offset<D>(k, j) + (lane & 3) * 4);
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
        if (!isfinite(f.x)) o[g][j][0] += f.x;
        if (!isfinite(f.y)) o[g][j][1] += f.y;
      }
    }
  }
  __syncwarp();
  uint32_t* w = reinterpret_cast<uint32_t*>(v);
  for (int i = lane; i < kGroup * D / 2; i += 32) w[i] = finite_or_zero_bf16x2(w[i]);
  __syncwarp();
}

// hi V + lo V of a column.  Where a value is infinite or NaN, hi V is what its weight
// times the value is; lo V is NaN or of the wrong sign, as lo is zero or negative.
__device__ __forceinline__ float hi_and_lo(float hi, float lo) { return isfinite(hi) ? hi + lo : hi; }

template <int D, int NG>
__global__ void __launch_bounds__(kWarps * 32, 2) attn_few_kernel(const CacheAttnParams p, const AttnParts parts,
                                                                  const int prefix_ctas, const int n_rank) {
  using C = FewCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ FewRow row[NG * 8];
  __shared__ float sm_m[kWarps][NG * 8], sm_l[kWarps][NG * 8];
  __shared__ float2 sm_ml[NG * 8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int M = static_cast<int>(p.Q.N), Hq = static_cast<int>(p.Q.H), Hkv = static_cast<int>(p.K.H), G = Hq / Hkv;

  begin_in(parts.order);

  // this CTA's rows and keys
  const bool pre = static_cast<int>(blockIdx.x) < prefix_ctas;
  const int cta = pre ? blockIdx.x : blockIdx.x - prefix_ctas;
  const int n_clusters = pre ? parts.prefix : parts.own, n_parts = n_clusters * n_rank;
  const int rows = (pre ? static_cast<int>(p.Q.B) : 1) * M * G, n_block = (rows + NG * 8 - 1) / (NG * 8);
  const int part = cta % n_parts, block = cta / n_parts % n_block, unit = cta / n_parts / n_block;
  const int hk = unit % Hkv, b = pre ? 0 : unit / Hkv;
  const int row0 = block * NG * 8, R = min(NG * 8, rows - row0);     // this CTA's rows
  const int nq = pre ? M : cache_len(p.mask.q_len, b, M, p.err);
  if (nq == 0) return end_in(parts.order);
  const int L = pre ? static_cast<int>(p.Kp.N) : cache_len(p.mask.kv_len, b, p.K.N, p.err);
  const KeyRun run = pre ? KeyRun{0, 0, 0, L} : key_run<1>(L - nq, L - 1, p.mask.window, p.mask.n_sink);
  if (tid < NG * 8) {
    FewRow f{0, -1, -1};
    if (tid < R) {
      const int i = row0 + tid, bb = pre ? i / (M * G) : b, r = i / G % M, h = hk * G + i % G;
      const int pos = L - nq + r;
      if (pre ? r < cache_len(p.mask.q_len, bb, M, p.err) : r < nq) {
        f.out = (bb * Hq + h) * M + r;
        f.hi = pre ? L - 1 : run.hi(pos);
        f.lo = pre ? 0 : run.lo(pos, p.mask.window);
      }
    }
    row[tid] = f;
  }
  __syncthreads();
  // the part of the keys: whole rounds of the four warps, the rest to the last
  const int chunk = (run.n + n_parts * kWarps * kGroup - 1) / (n_parts * kWarps * kGroup) * (kWarps * kGroup);
  const int begin = static_cast<int>(min(static_cast<int64_t>(run.n), static_cast<int64_t>(part) * chunk));
  const int end = static_cast<int>(min(static_cast<int64_t>(run.n), static_cast<int64_t>(begin) + chunk));
  // indices seen by every row: full_lo <= v <= full_hi (or v < n_sink)
  int full_lo = 0, full_hi = 0x7fffffff;
  for (int i = 0; i < NG * 8; ++i) {
    if (row[i].out < 0) continue;
    full_lo = max(full_lo, row[i].lo);
    full_hi = min(full_hi, row[i].hi);
  }

  // Q as mma A fragments: rows lane/4 (and 8 + lane/4 with two groups),
  // columns 2 (lane mod 4) and + 8 of every 16
  uint32_t qa[D / 16][2 * NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int i = row0 + g * 8 + lane / 4;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.Q.ptr);
    const bool valid = row[g * 8 + lane / 4].out >= 0;
    if (valid) q += (pre ? i / (M * G) : b) * p.Q.sB + (hk * G + i % G) * p.Q.sH + i / G % M * p.Q.sN + (lane & 3) * 2;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      qa[k][g] = valid ? *reinterpret_cast<const uint32_t*>(q + k * 16) : 0u;
      qa[k][NG + g] = valid ? *reinterpret_cast<const uint32_t*>(q + k * 16 + 8) : 0u;
    }
  }

  const TensorDesc& Kt = pre ? p.Kp : p.K;
  const TensorDesc& Vt = pre ? p.Vp : p.V;
  const __nv_bfloat16* kb = static_cast<const __nv_bfloat16*>(Kt.ptr) + (pre ? 0 : b * Kt.sB) + hk * Kt.sH;
  const __nv_bfloat16* vb = static_cast<const __nv_bfloat16*>(Vt.ptr) + (pre ? 0 : b * Vt.sB) + hk * Vt.sH;
  const int64_t ksN = Kt.sN, vsN = Vt.sN;
  unsigned char* ring = smem + warp * C::kRing;
  const uint32_t ring_s = smem_u32(ring);
  constexpr int CH = D / 8, RPI = 32 / CH;        // chunks per row, rows per pass of the warp
  const int lc = lane % CH, lr = lane / CH;
  // group i of this warp: indices begin + (4 i + warp) 16 ...; past `end` zeros
  auto load = [&](int i, int st) {
    const int v0 = begin + (i * kWarps + warp) * kGroup;
    if (v0 < end) {
      const uint32_t dk = ring_s + st * 2 * C::kTile, dv = dk + C::kTile;
#pragma unroll
      for (int it = 0; it < kGroup / RPI; ++it) {
        const int r = it * RPI + lr, v = v0 + r;
        const bool ok = v < end;
        const int64_t key = ok ? run.key(v) : 0;
        cp_async16_zfill(dk + rows_offset<D>(r, lc), kb + key * ksN + lc * 8, ok);
        cp_async16_zfill(dv + rows_offset<D>(r, lc), vb + key * vsN + lc * 8, ok);
      }
    }
    cp_async_commit();
  };

  float o[NG][D / 8][4];
  float m[NG], l[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[g][j][e] = 0.f;
  }
  const int rounds = (end - begin + kWarps * kGroup - 1) / (kWarps * kGroup);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load(i, i);
  int st = 0;
  for (int i = 0; i < rounds; ++i) {
    cp_async_wait<kStages - 2>();
    __syncwarp();                                 // the other lanes' copies too; and stage st - 1 is read
    load(i + kStages - 1, st == 0 ? kStages - 1 : st - 1);
    const int v0 = begin + (i * kWarps + warp) * kGroup;
    if (v0 >= end) break;
    const uint32_t sk = ring_s + st * 2 * C::kTile, sv = sk + C::kTile;
    // S: two tiles of 8 keys
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      // matrices: keys 0-7 | 0-7 | 8-15 | 8-15, chunks 2k | 2k+1 | 2k | 2k+1
      uint32_t f[4];
      ldsm4(f, sk + rows_offset<D>((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
#pragma unroll
      for (int t = 0; t < 2; ++t)
        mma_16816(s[t], qa[k][0], NG > 1 ? qa[k][NG - 1] : 0u, qa[k][NG], NG > 1 ? qa[k][2 * NG - 1] : 0u, f[2 * t],
                  f[2 * t + 1]);
    }
    const bool full = v0 + kGroup <= end && v0 + kGroup - 1 <= full_hi &&
                      (v0 >= full_lo || v0 + kGroup <= run.n_sink);
    uint32_t ph[NG][2], pl[NG][2];                // P of this thread's row: keys 0-7, 8-15
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      // keys v0 + 8 t + 2 (lane mod 4) + e
      float x[4] = {s[0][2 * g], s[0][2 * g + 1], s[1][2 * g], s[1][2 * g + 1]};
      if (!full) {
        const FewRow me = row[g * 8 + lane / 4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int v = v0 + (e >> 1) * 8 + (lane & 3) * 2 + (e & 1);
          if (v >= end || v > me.hi || (v < me.lo && v >= run.n_sink)) x[e] = -INFINITY;
        }
      }
      float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * p.scale_log2;
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (__any_sync(0xffffffffu, mx > m[g])) {
        const float mn = fmaxf(m[g], mx);
        const float a = mn == -INFINITY ? 1.f : ex2(m[g] - mn);
        m[g] = mn;
        l[g] *= a;
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[g][j][e] *= a;
      }
      const float mu = m[g] == -INFINITY ? 0.f : m[g];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = ex2(fmaf(x[e], p.scale_log2, -mu));
      l[g] += (x[0] + x[1]) + (x[2] + x[3]);
      split_bf16x2(x[0], x[1], ph[g][0], pl[g][0]);
      split_bf16x2(x[2], x[3], ph[g][1], pl[g][1]);
    }
    if (!full) {
      bool bad = false;
      const uint4* w = reinterpret_cast<const uint4*>(ring + st * 2 * C::kTile + C::kTile);
#pragma unroll
      for (int k = lane; k < kGroup * CH; k += 32) {
        const uint4 x = w[k];
        bad |= nonfinite_bf16x2(x.x) | nonfinite_bf16x2(x.y) | nonfinite_bf16x2(x.z) | nonfinite_bf16x2(x.w);
      }
      if (__any_sync(0xffffffffu, bad))
        few_nonfinite<D, NG>(ring + st * 2 * C::kTile + C::kTile, row, run.n_sink, v0, lane, o);
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      // matrices: keys 0-7 | 8-15 | 0-7 | 8-15, chunks 2j | 2j | 2j+1 | 2j+1
      uint32_t f[4];
      ldsm4_t(f, sv + rows_offset<D>((lane & 7) + (((lane >> 3) & 1) << 3), 2 * j + (lane >> 4)));
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        mma_16816(o[g][2 * j], ph[g][0], pl[g][0], ph[g][1], pl[g][1], f[0], f[1]);
        mma_16816(o[g][2 * j + 1], ph[g][0], pl[g][0], ph[g][1], pl[g][1], f[2], f[3]);
      }
    }
    st = st == kStages - 1 ? 0 : st + 1;
  }

  // ---- join the warps: m and l by rows, then O through shared memory
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    l[g] += __shfl_xor_sync(0xffffffffu, l[g], 1);
    l[g] += __shfl_xor_sync(0xffffffffu, l[g], 2);
    if ((lane & 3) == 0) {
      sm_m[warp][g * 8 + lane / 4] = m[g];
      sm_l[warp][g * 8 + lane / 4] = l[g];
    }
  }
  cp_async_wait_all();
  __syncthreads();                                // rings are free
  float* so = reinterpret_cast<float*>(smem);     // [warp][row][D]
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int i = g * 8 + lane / 4;
    float mm = sm_m[0][i];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w][i]);
    const float a = m[g] == -INFINITY ? 0.f : ex2(m[g] - mm);
    if (a != 0.f || l[g] != 0.f) {
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
        *reinterpret_cast<float2*>(so + (warp * NG * 8 + i) * D + j * 8 + (lane & 3) * 2) =
            make_float2(hi_and_lo(o[g][j][0], o[g][j][2]) * a, hi_and_lo(o[g][j][1], o[g][j][3]) * a);
    } else {
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
        *reinterpret_cast<float2*>(so + (warp * NG * 8 + i) * D + j * 8 + (lane & 3) * 2) = make_float2(0.f, 0.f);
    }
  }
  __syncthreads();
  const int n_slots = parts.prefix + parts.own, slot = (pre ? 0 : parts.prefix) + part / n_rank;
  for (int id = tid; id < R * (D / 4); id += kWarps * 32) {
    const int i = id / (D / 4), c = id % (D / 4) * 4;
    if (row[i].out < 0) continue;
    float mm = sm_m[0][i], ll = 0.f;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w][i]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (sm_l[w][i] != 0.f) ll += sm_l[w][i] * (mm == -INFINITY ? 1.f : ex2(sm_m[w][i] - mm));
      const float4 x = *reinterpret_cast<const float4*>(so + (w * NG * 8 + i) * D + c);
      acc.x += x.x;
      acc.y += x.y;
      acc.z += x.z;
      acc.w += x.w;
    }
    if (n_rank == 1) {
      leave_row4(p, parts, n_slots, slot, row[i].out, c, D, acc, mm, ll);
    } else {
      *reinterpret_cast<float4*>(so + i * D + c) = acc;          // (this thread alone reads and writes it)
      if (c == 0) sm_ml[i] = make_float2(mm, ll);
    }
  }
  if (n_rank == 1) return end_in(parts.order);
  // ---- join the cluster: each CTA takes every n_rank-th piece of the rows
  cluster_sync_all();
  const uint32_t so_s = smem_u32(so), ml_s = smem_u32(sm_ml);
  for (int id = tid * n_rank + part % n_rank; id < R * (D / 4); id += kWarps * 32 * n_rank) {
    const int i = id / (D / 4), c = id % (D / 4) * 4;
    if (row[i].out < 0) continue;
    float2 ml[kMaxRank];
    float4 x[kMaxRank];
#pragma unroll
    for (int q = 0; q < kMaxRank; ++q) {
      if (q >= n_rank) break;
      ml[q] = ld_cluster_f2(mapa_shared(ml_s + i * 8, q));
      x[q] = ld_cluster_f4(mapa_shared(so_s + (i * D + c) * 4, q));
    }
    float mm = -INFINITY, ll = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < kMaxRank; ++q)
      if (q < n_rank) mm = fmaxf(mm, ml[q].x);
#pragma unroll
    for (int q = 0; q < kMaxRank; ++q) {
      if (q >= n_rank || ml[q].y == 0.f) continue;
      const float w = mm == -INFINITY ? 1.f : ex2(ml[q].x - mm);
      ll = fmaf(w, ml[q].y, ll);
      acc.x = fmaf(w, x[q].x, acc.x);
      acc.y = fmaf(w, x[q].y, acc.y);
      acc.z = fmaf(w, x[q].z, acc.z);
      acc.w = fmaf(w, x[q].w, acc.w);
    }
    leave_row4(p, parts, n_slots, slot, row[i].out, c, D, acc, mm, ll);
  }
  cluster_sync_all();                             // the others may still read this CTA's shared memory
  end_in(parts.order);
}

// ---------------------------------------------------------------- joining
constexpr int kMaxParts = 32;      // that the prefix and the own keys each leave to attn_join_kernel
// One warp per output row, lane s looking after part s, s + 32, ...: the largest
// maximum, then the parts' sums and accumulators rescaled to it and added in the
// order of the parts, sixteen accumulator rows in flight.  2048 rows of 19 parts
// take 7 us (20 MB read), small cases 3 to 5.
template <int D>
__global__ void __launch_bounds__(128) attn_join_kernel(const CacheAttnParams p, const AttnParts parts) {
  wait_for_previous_kernel();
  const int64_t out = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, n = parts.prefix + parts.own;
  const int64_t M = p.Q.N;
  if (out >= p.Q.B * p.Q.H * M) return;
  if (p.mask.q_len && out % M >= cache_len(p.mask.q_len, out / M / p.Q.H, M, p.err)) return;
  constexpr int kBatch = 16, E = D / 32, kHold = (2 * kMaxParts + 31) / 32;
  float2 ml[kHold];
  float mm = -INFINITY;
#pragma unroll
  for (int q = 0; q < kHold; ++q) {
    ml[q] = lane + 32 * q < n ? parts.ml[out * n + lane + 32 * q] : make_float2(-INFINITY, 0.f);
    mm = fmaxf(mm, ml[q].x);
  }
  for (int off = 16; off > 0; off >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, off));
  const float* acc = parts.acc + out * n * D + lane * E;
  float ll = 0.f, a[E];
#pragma unroll
  for (int e = 0; e < E; ++e) a[e] = 0.f;
#pragma unroll
  for (int q = 0; q < kHold; ++q) {
    if (q * 32 >= n) break;
    // (a part in which the row sees nothing has sum 0 and no accumulator)
    const float w = ml[q].y == 0.f ? 0.f : mm == -INFINITY ? 1.f : ex2(ml[q].x - mm);
    const float wl = ml[q].y == 0.f ? 0.f : w * ml[q].y;
    for (int s0 = 0; s0 < 32 && q * 32 + s0 < n; s0 += kBatch) {
      float x[kBatch][E];
#pragma unroll
      for (int s = 0; s < kBatch; ++s) {
        const bool some = q * 32 + s0 + s < n && __shfl_sync(0xffffffffu, ml[q].y, s0 + s) != 0.f;
        const float* at = acc + static_cast<int64_t>(q * 32 + s0 + s) * D;
        if constexpr (E == 4) {
          const float4 f = some ? *reinterpret_cast<const float4*>(at) : make_float4(0.f, 0.f, 0.f, 0.f);
          x[s][0] = f.x;
          x[s][1] = f.y;
          x[s][2] = f.z;
          x[s][3] = f.w;
        } else {
          const float2 f = some ? *reinterpret_cast<const float2*>(at) : make_float2(0.f, 0.f);
          x[s][0] = f.x;
          x[s][1] = f.y;
        }
      }
#pragma unroll
      for (int s = 0; s < kBatch; ++s) {
        const float ws = __shfl_sync(0xffffffffu, w, s0 + s);
        ll += __shfl_sync(0xffffffffu, wl, s0 + s);
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] = fmaf(ws, x[s][e], a[e]);
      }
    }
  }
  const float inv = ll == 0.f ? 0.f : 1.f / ll;
  const int64_t b = out / M / p.Q.H, h = out / M % p.Q.H, r = out % M;
  __nv_bfloat16* o =
      static_cast<__nv_bfloat16*>(const_cast<void*>(p.O.ptr)) + b * p.O.sB + h * p.O.sH + r * p.O.sN + lane * E;
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(a[0] * inv, a[1] * inv), pack_bf16x2(a[2] * inv, a[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(o) = pack_bf16x2(a[0] * inv, a[1] * inv);
  if (lane == 0 && p.lse) p.lse[out] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994531f;
}

template <int D, int NG>
cudaError_t run_few(const CacheAttnParams& p, const AttnParts& parts, int prefix_ctas, int ctas, int rank,
                    cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(attn_few_kernel<D, NG>, FewCfg<D>::kBytes, done);
  if (e != cudaSuccess) return e;
  return launch_after(attn_few_kernel<D, NG>, static_cast<unsigned>(ctas), kWarps * 32, FewCfg<D>::kBytes, rank, s, p,
                      parts, prefix_ctas, rank);
}

constexpr int kFewRows = 32;
// One CTA for every place on the chip, with 128 keys each at least.  8 KV-head rows
// of 32768 keys take 27 us in 256 CTAs, 34 in 576 (two rounds of clusters), 33 in
// 128; 8 rows of 1024 keys 7.9 us in 64 CTAs and one kernel, 9.5 in 128 and two.
constexpr int kFewCtas = 2 * kSMs;
constexpr int kFewKeys = 128;
// ... and 512 beside attn_wide_kernel, which takes longer than such a part: 17
// sequences of 333 keys over 10007 (5 rows, D 64) take 21.7 us, 25.9 with 128.
constexpr int kBesideKeys = 512;

// Parts that `units` independent pieces of work of at most `keys` keys are cut
// into: enough for `ctas` CTAs, none shorter than `shortest` keys.
int cut(int64_t units, int64_t keys, int64_t ctas, int64_t shortest, int64_t most) {
  return static_cast<int>(std::max<int64_t>(1, std::min({keys / shortest, ctas / units, most})));
}
int power_of_two_up_to(int n) {
  int x = 1;
  while (2 * x <= n) x *= 2;
  return x;
}

// Blocks of rows that attn_few_kernel runs in different CTAs.
int64_t row_blocks(int64_t rows) { return (rows + 15) / 16; }

// Parts of a prefix that attn_wide_kernel takes (one CTA of the `units` each) while
// attn_few_kernel streams the sequences' own keys on the other SMs: the most, up to
// `most`, that leave those `blocks` of 16 rows enough SM time, by what the two take
// alone: 15 us and 2 us for every 128 keys of the prefix; 1 us and 0.9 us for 128
// own keys of D 128, with more than 8 rows 2.5 times that.  The lengths are not
// known here, only the most that they may be, so the prefix keeps half the SMs at
// least.  64 sequences (Hq 32, Hkv 8, D 128), 1024 keys over 32768: 79 to 84 us in
// 10 to 12 parts, 101 in all 18; 9 sequences, 4096 over 32768: 63 in 12 parts, 94 in
// 18; D 64, 256 over 32768: 53 in 16 parts, 57 in 18.
int beside_own(int most, bool few_own, int64_t units, int64_t P, int64_t blocks, int64_t rows, int64_t keys,
               int64_t D) {
  if (!few_own) return most;
  const double own = static_cast<double>(blocks) * (0.9 * keys / 128 + 1) * D / 128 * (rows > 8 ? 2.5 : 1);
  int parts = most;
  while (parts > (most + 1) / 2 && own > (kSMs - units * parts) * (15 + 2 * (P / 128.0) / parts)) --parts;
  return parts;
}

struct Plan {
  bool few_own, few_prefix;
  int rank;                        // CTAs per cluster of the few-row kernel
  int own, prefix;                 // parts left to attn_join_kernel
};
Plan plan(const TensorDesc& Q, const TensorDesc& K, int64_t keys, bool has_prefix, int64_t P) {
  const int64_t G = Q.H / K.H, rows = Q.N * G;
  Plan w{};
  w.few_own = rows <= kFewRows;
  w.few_prefix = has_prefix && Q.B * rows <= kFewRows;
  w.rank = 1;
  int own = 0, prefix = 0;
  const int64_t own_units = K.B * K.H * row_blocks(rows), prefix_units = K.H * row_blocks(Q.B * rows);
  const int64_t ctas = w.few_own && w.few_prefix ? kFewCtas / 2 : kFewCtas;
  const int shortest = has_prefix && !w.few_prefix ? kBesideKeys : kFewKeys;
  if (w.few_own) own = cut(own_units, keys, ctas, shortest, kMaxParts * kMaxRank);
  if (w.few_prefix) prefix = cut(prefix_units, P, ctas, kFewKeys, kMaxParts * kMaxRank);
  w.rank = power_of_two_up_to(std::min(std::max({own, prefix, 1}), kMaxRank));
  // (clusters as large as the prefix's parts want them, but not so large that the
  // sequences' own keys, which may want one CTA each, take more than their places)
  while (w.rank > 1 && own < w.rank && w.few_own && own_units * w.rank > ctas) w.rank /= 2;
  w.own = w.few_own ? std::max(own / w.rank, 1) : cut(wide_units(Q, K, false), keys, kSMs, 256, kMaxParts);
  if (has_prefix)
    w.prefix = w.few_prefix ? std::max(prefix / w.rank, 1)
                            : beside_own(cut(wide_units(Q, K, true), P, kSMs, 256, kMaxParts), w.few_own,
                                         wide_units(Q, K, true), P, own_units, rows, keys, Q.D);
  return w;
}

}  // namespace

size_t cache_attn_ws_bytes(const TensorDesc& Q, const TensorDesc& K, bool prefix) {
  // a window only makes for fewer parts; the prefix's length is not known here
  const Plan w = plan(Q, K, K.N, prefix, 1ll << 31);
  const int64_t n = w.own + w.prefix;
  return n == 1 ? 0 : static_cast<size_t>(Q.B * Q.H * Q.N * n) * (Q.D * 4 + 8);
}

cudaError_t launch_cache_attn(const CacheAttnParams& p, cudaStream_t s) {
  const bool pre = p.Kp.ptr != nullptr;
  const int64_t keys = std::min(p.K.N, p.mask.window + p.mask.n_sink + p.Q.N);
  const Plan w = plan(p.Q, p.K, keys, pre, p.Kp.N);
  // (the workspace was sized without the window and the prefix's length, for at
  // least as many parts)
  const Plan most = plan(p.Q, p.K, p.K.N, pre, 1ll << 31);
  if (w.own + w.prefix > most.own + most.prefix) return cudaErrorInvalidValue;
  AttnParts parts;
  parts.own = w.own;
  parts.prefix = w.prefix;
  parts.order = Order::kAlone;
  const int64_t rows = p.Q.B * p.Q.H * p.Q.N, n = w.own + w.prefix;
  parts.acc = static_cast<float*>(p.ws);
  parts.ml = reinterpret_cast<float2*>(parts.acc + rows * n * p.Q.D);
  const bool two = std::max(w.few_own ? p.Q.N * (p.Q.H / p.K.H) : 0,
                            w.few_prefix ? p.Q.B * p.Q.N * (p.Q.H / p.K.H) : 0) > 8;
  const int64_t own_rows = p.Q.N * (p.Q.H / p.K.H);
  const int prefix_ctas =
      w.few_prefix ? static_cast<int>(p.K.H * row_blocks(p.Q.B * own_rows)) * w.prefix * w.rank : 0;
  const int ctas =
      prefix_ctas + (w.few_own ? static_cast<int>(p.K.B * p.K.H * row_blocks(own_rows)) * w.own * w.rank : 0);
  cudaError_t e = cudaSuccess;
  if (pre && !w.few_prefix) {
    parts.order = Order::kFirst;
    if ((e = launch_attn_wide(p, parts, true, s)) != cudaSuccess) return e;
    parts.order = Order::kSecond;
  }
  if (!w.few_own && (e = launch_attn_wide(p, parts, false, s)) != cudaSuccess) return e;
  if (ctas > 0) {
    auto run = p.Q.D == 128 ? (two ? run_few<128, 2> : run_few<128, 1>) : (two ? run_few<64, 2> : run_few<64, 1>);
    if ((e = run(p, parts, prefix_ctas, ctas, w.rank, s)) != cudaSuccess) return e;
  }
  if (n == 1) return cudaSuccess;
  return launch_after(p.Q.D == 128 ? attn_join_kernel<128> : attn_join_kernel<64>,
                      static_cast<unsigned>((rows + 3) / 4), 128, 0, 1, s, p, parts);
}

}  // namespace pbs
