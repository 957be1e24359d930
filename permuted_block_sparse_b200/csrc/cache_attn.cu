// pbs_attn_window and pbs_attn_prefix: attention over a K/V cache.
//
//   O[r] = sum_j 2^(x_rj - m_r) V[j] / l_r,  x_rj = scale log2(e) Q[r].K[j],
//   m_r = max_j x_rj,  l_r = sum_j 2^(x_rj - m_r),  lse_r = ln 2 (m_r + log2 l_r)
//
// over the keys j that row r sees, in one pass with the running (m, l, O)
// rescaled whenever m grows.  The key axis may be cut into parts that different
// CTAs run; a part leaves its (m, l, O) in fp32 and attn_join_kernel adds them.
//
// Query rows of one KV head that read the same keys run together: the G heads
// of the group, the M new tokens and, over a shared prefix, the sequences.  Up
// to 16 such rows (a decode step) are bound by the bytes of K and V and run in
// attn_few_kernel below; more rows run on the tcgen05 kernel of
// cache_attn_wide.cu.
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
// Bound: HBM, 4 D bytes per key.
constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr int kGroup = 16;                      // keys per warp and stage

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
// them for the product.  Whole warp; col0 + 8 j + {0, 1} are a thread's columns.
template <int D, int NG>
__device__ __noinline__ void few_nonfinite(unsigned char* v, const FewRow* row, int n_sink, int v0, int lane,
                                           float (&o)[NG][D / 8][4]) {
  for (int g = 0; g < NG; ++g) {
    const FewRow me = row[g * 8 + lane / 4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      for (int k = 0; k < kGroup; ++k) {
        const int i = v0 + k;
        if (i > me.hi || (i < me.lo && i >= n_sink)) continue;
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

template <int D, int NG>
__global__ void __launch_bounds__(kWarps * 32, 2) attn_few_kernel(const CacheAttnParams p, const AttnParts parts,
                                                                  const int prefix_ctas) {
  using C = FewCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ FewRow row[NG * 8];
  __shared__ float sm_m[kWarps][NG * 8], sm_l[kWarps][NG * 8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int M = static_cast<int>(p.Q.N), Hq = static_cast<int>(p.Q.H), Hkv = static_cast<int>(p.K.H), G = Hq / Hkv;

  // this CTA's rows and keys
  const bool pre = static_cast<int>(blockIdx.x) < prefix_ctas;
  const int cta = pre ? blockIdx.x : blockIdx.x - prefix_ctas;
  const int n_parts = pre ? parts.prefix : parts.own;
  const int part = cta % n_parts, unit = cta / n_parts;
  const int hk = unit % Hkv, b = pre ? 0 : unit / Hkv;
  const int R = (pre ? static_cast<int>(p.Q.B) : 1) * M * G;
  const int nq = pre ? M : cache_len(p.mask.q_len, b, M, p.err);
  if (nq == 0) return;
  const int L = pre ? static_cast<int>(p.Kp.N) : cache_len(p.mask.kv_len, b, p.K.N, p.err);
  const KeyRun run = pre ? KeyRun{0, 0, 0, L} : key_run<1>(L - nq, L - 1, p.mask.window, p.mask.n_sink);
  if (tid < NG * 8) {
    FewRow f{0, -1, -1};
    if (tid < R) {
      const int bb = pre ? tid / (M * G) : b, r = tid / G % M, h = hk * G + tid % G;
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
    const int i = g * 8 + lane / 4;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.Q.ptr);
    const bool valid = row[i].out >= 0;
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
            make_float2((o[g][j][0] + o[g][j][2]) * a, (o[g][j][1] + o[g][j][3]) * a);
    } else {
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
        *reinterpret_cast<float2*>(so + (warp * NG * 8 + i) * D + j * 8 + (lane & 3) * 2) = make_float2(0.f, 0.f);
    }
  }
  __syncthreads();
  const int slot = pre ? part : parts.prefix + part, n_slots = parts.prefix + parts.own;
  for (int id = tid; id < R * (D / 4); id += kWarps * 32) {
    const int i = id / (D / 4), c = id % (D / 4) * 4;
    if (row[i].out < 0) continue;
    float mm = sm_m[0][i], ll = 0.f;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w][i]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (sm_m[w][i] != -INFINITY || sm_l[w][i] != 0.f) ll += sm_l[w][i] * (mm == -INFINITY ? 1.f : ex2(sm_m[w][i] - mm));
      const float4 x = *reinterpret_cast<const float4*>(so + (w * NG * 8 + i) * D + c);
      acc.x += x.x;
      acc.y += x.y;
      acc.z += x.z;
      acc.w += x.w;
    }
    if (n_slots == 1) {
      write_row4(p, row[i].out, c, acc, mm, ll);
    } else {
      const int64_t at = static_cast<int64_t>(row[i].out) * n_slots + slot;
      if (ll != 0.f) *reinterpret_cast<float4*>(parts.acc + at * D + c) = acc;
      if (c == 0) parts.ml[at] = make_float2(mm, ll);
    }
  }
}

// ---------------------------------------------------------------- joining
// One warp per output row: the largest maximum, then the parts' sums and
// accumulators rescaled to it, in the order of the parts.
template <int D>
__global__ void __launch_bounds__(128) attn_join_kernel(const CacheAttnParams p, const AttnParts parts) {
  const int64_t out = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, n = parts.prefix + parts.own;
  const int64_t M = p.Q.N;
  if (out >= p.Q.B * p.Q.H * M) return;
  if (p.mask.q_len && out % M >= cache_len(p.mask.q_len, out / M / p.Q.H, M, p.err)) return;
  const float2* ml = parts.ml + out * n;
  float mm = -INFINITY;
  for (int s = lane; s < n; s += 32) mm = fmaxf(mm, ml[s].x);
  for (int off = 16; off > 0; off >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, off));
  const float* acc = parts.acc + out * n * D + lane * (D / 32);
  float ll = 0.f, a[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) a[e] = 0.f;
#pragma unroll 4
  for (int s = 0; s < n; ++s) {
    const float2 x = ml[s];
    if (x.y == 0.f) continue;                     // a part in which the row sees nothing
    const float w = x.x == mm ? 1.f : ex2(x.x - mm);
    ll += w * x.y;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) a[e] = fmaf(w, acc[static_cast<int64_t>(s) * D + e], a[e]);
  }
  const float inv = ll == 0.f ? 0.f : 1.f / ll;
  const int64_t b = out / M / p.Q.H, h = out / M % p.Q.H, r = out % M;
  __nv_bfloat16* o =
      static_cast<__nv_bfloat16*>(const_cast<void*>(p.O.ptr)) + b * p.O.sB + h * p.O.sH + r * p.O.sN + lane * (D / 32);
#pragma unroll
  for (int e = 0; e < D / 32; e += 2) *reinterpret_cast<uint32_t*>(o + e) = pack_bf16x2(a[e] * inv, a[e + 1] * inv);
  if (lane == 0 && p.lse) p.lse[out] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994531f;
}

template <int D, int NG>
cudaError_t run_few(const CacheAttnParams& p, const AttnParts& parts, int prefix_ctas, int own_ctas, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(attn_few_kernel<D, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       FewCfg<D>::kBytes);
  if (e != cudaSuccess) return e;
  attn_few_kernel<D, NG><<<prefix_ctas + own_ctas, kWarps * 32, FewCfg<D>::kBytes, s>>>(p, parts, prefix_ctas);
  return cudaGetLastError();
}

constexpr int kFewRows = 16;
constexpr int kMaxParts = 64;      // of the prefix and of the own keys each

// Parts that `units` independent pieces of work of at most `keys` keys are cut
// into: enough for `ctas` CTAs, none shorter than `shortest` keys.
int cut(int64_t units, int64_t keys, int64_t ctas, int64_t shortest) {
  const int64_t most = std::max<int64_t>(1, keys / shortest);
  return static_cast<int>(std::max<int64_t>(1, std::min({most, ctas / units, static_cast<int64_t>(kMaxParts)})));
}

struct Plan {
  bool few_own, few_prefix;
  int own, prefix;                 // parts
};
Plan plan(const TensorDesc& Q, const TensorDesc& K, int64_t keys, bool has_prefix, int64_t P) {
  const int64_t G = Q.H / K.H, rows = Q.N * G;
  Plan w{};
  w.few_own = rows <= kFewRows;
  w.own = w.few_own ? cut(K.B * K.H, keys, 4 * kSMs, 256) : cut(wide_units(Q, K, false), keys, kSMs, 256);
  if (has_prefix) {
    w.few_prefix = Q.B * rows <= kFewRows;
    w.prefix = w.few_prefix ? cut(K.H, P, 2 * kSMs, 64) : cut(wide_units(Q, K, true), P, kSMs, 256);
  }
  return w;
}

}  // namespace

size_t cache_attn_ws_bytes(const TensorDesc& Q, const TensorDesc& K, bool prefix) {
  if (Q.H % K.H || K.H > Q.H) return 0;
  // a window only makes for fewer parts; the prefix's length is not known here
  const Plan w = plan(Q, K, K.N, prefix, 1ll << 31);
  const int64_t n = w.own + w.prefix;
  return n == 1 ? 0 : static_cast<size_t>(Q.B * Q.H * Q.N * n) * (Q.D * 4 + 8);
}

cudaError_t launch_cache_attn(const CacheAttnParams& p, cudaStream_t s) {
  const bool pre = p.Kp.ptr != nullptr;
  const int64_t keys = std::min(p.K.N, p.mask.window + p.mask.n_sink + p.Q.N);
  const Plan w = plan(p.Q, p.K, keys, pre, p.Kp.N);
  AttnParts parts;
  parts.own = w.own;
  parts.prefix = w.prefix;
  const int64_t rows = p.Q.B * p.Q.H * p.Q.N, n = w.own + w.prefix;
  parts.acc = static_cast<float*>(p.ws);
  parts.ml = reinterpret_cast<float2*>(parts.acc + rows * n * p.Q.D);
  const bool two = std::max(w.few_own ? p.Q.N * (p.Q.H / p.K.H) : 0,
                            w.few_prefix ? p.Q.B * p.Q.N * (p.Q.H / p.K.H) : 0) > 8;
  const int prefix_ctas = w.few_prefix ? static_cast<int>(p.K.H) * w.prefix : 0;
  const int own_ctas = w.few_own ? static_cast<int>(p.K.B * p.K.H) * w.own : 0;
  cudaError_t e = cudaSuccess;
  if (pre && !w.few_prefix && (e = launch_attn_wide(p, parts, true, s)) != cudaSuccess) return e;
  if (!w.few_own && (e = launch_attn_wide(p, parts, false, s)) != cudaSuccess) return e;
  if (prefix_ctas + own_ctas > 0) {
    if (p.Q.D == 128)
      e = two ? run_few<128, 2>(p, parts, prefix_ctas, own_ctas, s) : run_few<128, 1>(p, parts, prefix_ctas, own_ctas, s);
    else
      e = two ? run_few<64, 2>(p, parts, prefix_ctas, own_ctas, s) : run_few<64, 1>(p, parts, prefix_ctas, own_ctas, s);
    if (e != cudaSuccess) return e;
  }
  if (n > 1) {
    const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
    if (p.Q.D == 128)
      attn_join_kernel<128><<<grid, 128, 0, s>>>(p, parts);
    else
      attn_join_kernel<64><<<grid, 128, 0, s>>>(p, parts);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace pbs
