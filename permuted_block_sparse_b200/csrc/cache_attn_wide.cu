// Attention over a K/V cache for many query rows (prompts, chunks, and a
// batch's rows over a shared prefix): the tcgen05 kernel of pbs_attn_window
// and pbs_attn_prefix.
//
// Tile layout.  128 MMA rows are query rows of ONE KV head packed as (sequence,
// position, head of the group), head innermost: one TMA box {64 columns, G
// heads, positions, sequences} lands them in that order.  So a tile spans only
// 128 / G positions, and with a window of W keys it reads W + 128 / G keys where
// a tile of 128 positions of one head would read W + 128; every K/V tile serves
// the whole head group.  A CTA runs two such tiles (slots) over the union of
// their keys, so each K/V tile is loaded once for 256 rows and one slot's
// softmax runs while the tensor core works for the other.
//
// The keys a CTA needs are a run of virtual indices (KeyRun): sinks, then the
// window, without the gap between them; the tile in which they meet is loaded
// as 16-row boxes.  Tiles start at the first needed key, not at a multiple of
// 128.
//
// Roles (640 threads): warp 0 issues tcgen05.mma and owns tensor memory; warp
// 1 issues the TMA loads of Q and of the K and V rings, the first ones before the
// rest of the CTA is set up; warps 2-3 clean the V tiles that some row must not
// see in full (below); warps 4-11 and 12-19 run the softmax of slot 0 and 1, two
// threads per row with half of the tile's columns each, which agree on the row's
// maximum through shared memory (one 64-thread barrier a tile).  One thread per
// row left a scheduler with one softmax warp per slot, and that warp's chain of
// maximum, exponentials and stores took 1.3 us a tile where the exponentials
// alone take 0.5.  Tensor memory (512 columns): S0 | S1 | O0 | O1; P (bf16)
// overwrites S and is the A operand of PV.  The order of MMAs is fixed: PV of a
// slot's tile, then QK^T of its next tile, slots in turn.
//
// A masked key has weight 0, but 0 * NaN is NaN: where a tile holds a key that
// some row of the CTA does not see, warps 2-3 replace NaN and infinities in V
// by 0 before the product and note the key; at the end each row that does see
// such a key takes those entries from global memory.
//
// Roundings: statistics, sums and O in fp32; P to bf16 for its product, the only type
// that goes with V (the row's sum is of P before the rounding).  Each weight is off by
// 2^-8 at most, which leaves O 2.3e-3 from fp64 (2-norm) where the bf16 of O alone is
// 1.65e-3; P as two bf16, as attn_few_kernel has it where HBM is the bound, would be
// half as many products again where products are: 2.27 us a tile pair for 1.51.
//
// Bound: the tensor core; with few rows per CTA, HBM.  Measured (a 32K prompt, Hq 32,
// Hkv 8, D 128, window 2048, 128 sinks): 1.36 ms, 831 TFLOP/s of visible products.
// One more tile for both slots costs 1.82 us, 1.60 with the softmax arithmetic left
// out, 1.51 at the measured matrix rate; each CTA adds 13 us to its 18 tiles (set-up
// and first loads 3.6, the two slots' ends 4.7, masked and cleaned tiles).  A
// persistent form that overlaps those with the next item ran at 1.73 ms: its roles
// no longer fit 96 registers.  Moving the exponentials to the FMA pipe, or taking them
// against an older maximum, gained nothing.
#include <math.h>

#include <algorithm>

#include "cache_attn.cuh"
#include "wide_order.h"

namespace pbs {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();   // (select_sample.cu)

namespace {

constexpr int kThreads = 640;
constexpr float kRescaleSlack = 8.0f;   // keep the running max while within 2^8
// Tiles of a CTA that some row does not see in full: two per slot at the causal
// end and two at the window's start (a slot spans at most 128 positions), one
// at the end of the sinks.
constexpr int kMaxDirty = 9;

template <int D>
struct WideCfg {
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kTile = (D / 64) * 128 * 128;   // Q, K or V tile: 64-column halves of 128-byte rows
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kTile;
  static constexpr int kV = kK + kStages * kTile;
  static constexpr int kBytes = kV + kStages * kTile + 1024;   // alignment slack
};

// How query rows are packed into tiles.
struct WideRows {
  int pos_per_tile, seqs_per_tile, tiles;   // tiles per sequence, or in all over a prefix
};

__host__ __device__ __forceinline__ WideRows wide_rows(int64_t B, int64_t M, int64_t G, bool prefix) {
  WideRows w;
  const int64_t most = 128 / G;
  w.pos_per_tile = static_cast<int>(M < most ? M : most);
  w.seqs_per_tile = 1;
  if (prefix && M <= most) {
    const int64_t n = 128 / (G * M);
    w.seqs_per_tile = static_cast<int>(n < B ? n : B);
    w.tiles = static_cast<int>((B + w.seqs_per_tile - 1) / w.seqs_per_tile);
  } else {
    w.tiles = static_cast<int>((M + w.pos_per_tile - 1) / w.pos_per_tile * (prefix ? B : 1));
  }
  return w;
}

// Rescale a thread's half of its row of O by alpha (rare; whole warps).
template <int D>
__device__ __noinline__ void rescale_o(uint32_t tO, float alpha) {
#pragma unroll 1
  for (int c = 0; c < D / 64; ++c) {
    uint32_t u[32];
    tmem_ld32(tO + c * 32, u);
#pragma unroll
    for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * alpha);
    tmem_st32(tO + c * 32, u);
  }
}

template <int NS>
struct Shared {
  uint64_t bar_q, bar_k[NS], bar_v[NS], bar_vraw[NS], bar_kempty[NS], bar_vempty[NS];
  uint64_t bar_s[2], bar_p[2], bar_o[2], bar_fin;
  uint32_t tmem_base;
  int abort;
  int n_dirty;                            // tiles cleaned, and whether any held something
  int any_bad;
  int dirty_tile[kMaxDirty];
  uint32_t bad[kMaxDirty][4];             // their keys with NaN or infinities in V
  float row_max[2][2][2][128];            // [tile parity][slot][half][row]; then the sums
};

struct WideMaps {
  CUtensorMap q, k, v, k16, v16;          // boxes of 128 key rows, and of 16
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_wide_kernel(const CacheAttnParams p, const AttnParts parts,
                                                                const bool prefix, const WideRows wr,
                                                                const __grid_constant__ WideMaps maps) {
  using C = WideCfg<D>;
  constexpr int NS = C::kStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  __shared__ Shared<NS> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int M = static_cast<int>(p.Q.N), Hq = static_cast<int>(p.Q.H), Hkv = static_cast<int>(p.K.H), G = Hq / Hkv;
  const int B = static_cast<int>(p.Q.B);

  begin_in(parts.order);

  // ---- this CTA's work: a pair of tiles, a KV head (and sequence), a part of the keys
  const int n_parts = prefix ? parts.prefix : parts.own;
  const int pairs = (wr.tiles + 1) / 2;
  const int part = static_cast<int>(blockIdx.x) % n_parts;
  // (without a window later positions have more keys: first)
  const int pair = pairs - 1 - static_cast<int>(blockIdx.x) / n_parts;
  const int hk = static_cast<int>(blockIdx.y) % Hkv;
  const int b_own = prefix ? 0 : static_cast<int>(blockIdx.y) / Hkv;
  const int nq_own = prefix ? M : cache_len(p.mask.q_len, b_own, M, p.err);
  const int L = prefix ? static_cast<int>(p.Kp.N) : cache_len(p.mask.kv_len, b_own, p.K.N, p.err);
  const int n_pos_tiles = (M + wr.pos_per_tile - 1) / wr.pos_per_tile;   // per sequence
  // first sequence and first row of each slot's tile
  auto tile_seq = [&](int h) {
    const int t = 2 * pair + h;
    return prefix ? (wr.seqs_per_tile > 1 || n_pos_tiles == 1 ? t * wr.seqs_per_tile : t / n_pos_tiles) : b_own;
  };
  auto tile_row = [&](int h) {
    const int t = 2 * pair + h;
    return (prefix ? (n_pos_tiles == 1 ? 0 : t % n_pos_tiles) : t) * wr.pos_per_tile;
  };
  auto has_rows = [&](int h) { return 2 * pair + h < wr.tiles && tile_row(h) < nq_own; };
  if (!has_rows(0)) return end_in(parts.order);   // (slot 1 then has none either)
  const int n_slot = has_rows(1) ? 2 : 1;
  // positions of the slots' first and last rows (own keys)
  auto first_pos = [&](int h) { return L - nq_own + tile_row(h); };
  auto last_pos = [&](int h) { return L - nq_own + min(tile_row(h) + wr.pos_per_tile, nq_own) - 1; };
  const KeyRun run = prefix ? KeyRun{0, 0, 0, L}
                            : key_run<16>(first_pos(0), last_pos(n_slot - 1), p.mask.window, p.mask.n_sink);
  const int T = (run.n + 127) / 128;
  const int t0 = static_cast<int>(static_cast<int64_t>(T) * part / n_parts);
  const int t1 = static_cast<int>(static_cast<int64_t>(T) * (part + 1) / n_parts);
  // does slot h see any key of tile t, and do all its rows see all of them?
  // (bounds of each slot's first and last rows, chosen without indexing so that
  // they stay in registers)
  int hi_first0 = L - 1, hi_last0 = L - 1, lo_first0 = 0, lo_last0 = 0;
  int hi_first1 = L - 1, hi_last1 = L - 1, lo_first1 = 0, lo_last1 = 0;
  if (!prefix) {
    hi_first0 = run.hi(first_pos(0));
    hi_last0 = run.hi(last_pos(0));
    lo_first0 = run.lo(first_pos(0), p.mask.window);
    lo_last0 = run.lo(last_pos(0), p.mask.window);
    hi_first1 = run.hi(first_pos(1));
    hi_last1 = run.hi(last_pos(1));
    lo_first1 = run.lo(first_pos(1), p.mask.window);
    lo_last1 = run.lo(last_pos(1), p.mask.window);
  }
  auto active = [&](int h, int t) {
    return h < n_slot && slot_uses(t, h ? hi_last1 : hi_last0, h ? lo_first1 : lo_first0, run.n_sink);
  };
  auto full = [&](int h, int t) {
    const int up = h ? hi_first1 : hi_first0, low = h ? lo_last1 : lo_last0;
    return 128 * t + 127 <= up && (128 * t >= low || 128 * t + 127 < run.n_sink);
  };
  // (rows past the prefix are zeros, never NaN: no cleaning there)
  auto dirty = [&](int t) {
    return !prefix && ((active(0, t) && !full(0, t)) || (active(1, t) && !full(1, t)));
  };

  const uint32_t sQ = smem_u32(smem + C::kQ), sK = smem_u32(smem + C::kK), sV = smem_u32(smem + C::kV);
  // ---- loads (warp 1, one thread): a K or V tile is one box per 64 columns, or
  // 16-row boxes where it spans the end of the sinks
  int raw[NS] = {};                                   // V tiles through bar_vraw, per stage
  auto load_tile = [&](uint32_t dst, const CUtensorMap* one, const CUtensorMap* rows16, int head, int seq, int t,
                       uint64_t* bar) {
    mbar_expect_tx(bar, static_cast<uint32_t>(C::kTile));
    const int v0 = 128 * t;
    const bool mixed = run.delta > 0 && v0 < run.sink_end && v0 + 128 > run.sink_end;
    for (int c = 0; c < D / 64; ++c) {
      const uint32_t d = dst + c * (128 * 128);
      if (!mixed) {
        tma_rows_4d(d, one, c * 64, run.key(v0), head, seq, bar);
      } else {
        for (int r = 0; r < 128; r += 16) tma_rows_4d(d + r * 128, rows16, c * 64, run.key(v0 + r), head, seq, bar);
      }
    }
  };
  // (broadcast heads or sequences are one in the map)
  auto load_k = [&](int t) {
    const int st = (t - t0) % NS;
    load_tile(sK + st * C::kTile, &maps.k, &maps.k16, (prefix ? p.Kp.sH : p.K.sH) == 0 ? 0 : hk,
              p.K.sB == 0 ? 0 : b_own, t, &sh.bar_k[st]);
  };
  auto load_v = [&](int t) {
    const int st = (t - t0) % NS;
    const bool d = dirty(t);
#pragma unroll
    for (int q = 0; q < NS; ++q) raw[q] += d && q == st;
    load_tile(sV + st * C::kTile, &maps.v, &maps.v16, (prefix ? p.Vp.sH : p.V.sH) == 0 ? 0 : hk,
              p.V.sB == 0 ? 0 : b_own, t, d ? &sh.bar_vraw[st] : &sh.bar_v[st]);
  };
  if (tid == 32) {
    sh.abort = 0;
    sh.n_dirty = 0;
    sh.any_bad = 0;
    mbar_init(&sh.bar_q, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sh.bar_k[i], 1);
      mbar_init(&sh.bar_v[i], 1);
      mbar_init(&sh.bar_vraw[i], 1);
      mbar_init(&sh.bar_kempty[i], 1);
      mbar_init(&sh.bar_vempty[i], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&sh.bar_s[h], 1);
      mbar_init(&sh.bar_p[h], 8);
      mbar_init(&sh.bar_o[h], 1);
    }
    mbar_init(&sh.bar_fin, 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
  }
  if (tid >= 64 && tid < 64 + kMaxDirty * 4) sh.bad[(tid - 64) / 4][(tid - 64) % 4] = 0u;
  tc_fence_before();
  // warp 1 has nothing to wait for: it goes on to the first loads
  if (warp == 1) {
    __syncwarp();
    asm volatile("bar.arrive 15, %0;" ::"n"(kThreads) : "memory");
  } else {
    named_sync(15, kThreads);
  }
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;                 // (not warp 1's)
  volatile int* abort_flag = &sh.abort;

  if (warp == 1) {
    // ============================================================ producer
    if (lane == 0) {
      const int box = wr.pos_per_tile * wr.seqs_per_tile * G * 128;     // bytes of a 64-column Q box
      mbar_expect_tx(&sh.bar_q, static_cast<uint32_t>(n_slot * (D / 64) * box));
      for (int h = 0; h < n_slot; ++h)
        for (int c = 0; c < D / 64; ++c)
          tma_rows_4d(sQ + h * C::kTile + c * (128 * 128), &maps.q, c * 64, hk * G, tile_row(h), tile_seq(h), &sh.bar_q);
      for (int t = t0; t < min(t0 + NS, t1); ++t) {
        load_k(t);
        load_v(t);
      }
      int nk = min(t0 + NS, t1), nv = nk;             // tiles issued
      for (int t = t0 + NS; t < t1; ++t) {
        const int st = (t - t0) % NS;
        const uint32_t again = ((t - t0) / NS - 1) & 1;
        if (!mbar_wait_or_abort(&sh.bar_kempty[st], again, p.err, abort_flag)) break;
        load_k(t);
        ++nk;
        if (!mbar_wait_or_abort(&sh.bar_vempty[st], again, p.err, abort_flag)) break;
        load_v(t);
        ++nv;
      }
      // no copy may be in flight when the CTA ends; without an abort the MMA
      // role has waited for all of them
      if (*abort_flag) {
        mbar_wait(&sh.bar_q, 0, p.err);
        for (int t = max(t0, nk - NS); t < nk; ++t) mbar_wait(&sh.bar_k[(t - t0) % NS], ((t - t0) / NS) & 1, p.err);
        for (int t = max(t0, nv - NS); t < nv; ++t) {
          const int st = (t - t0) % NS;
          int fills = 0;
#pragma unroll
          for (int q = 0; q < NS; ++q)
            if (q == st) fills = raw[q];
          if (dirty(t)) mbar_wait(&sh.bar_vraw[st], (fills - 1) & 1, p.err);
          else mbar_wait(&sh.bar_v[st], ((t - t0) / NS) & 1, p.err);
        }
      }
    }
    __syncwarp();
  } else if (warp == 0) {
    // ========================================================= MMA issuer
    // (all lanes wait, so that each has acquired what it issues on)
    constexpr uint32_t idesc_qk = idesc_bf16(128, 128, false), idesc_pv = idesc_bf16(128, D, true);
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_or_abort(bar, parity, p.err, abort_flag));
      tc_fence_after();
    };
    wait(&sh.bar_q, 0);
    int k_seen = t0, v_seen = t0;           // tiles below have landed (waited for in order)
    auto landed = [&](uint64_t* bars, int& seen, int t) {
      for (; ok && seen <= t; ++seen) wait(&bars[(seen - t0) % NS], ((seen - t0) / NS) & 1);
    };
    int done0 = 0, done1 = 0;               // tiles whose QK^T has been issued, per slot
    int on0 = t0 - 1, on1 = t0 - 1;         // and the last of them
    auto qk = [&](int h, int t) {
      landed(sh.bar_k, k_seen, t);
      if (!ok) return;
      const int st = (t - t0) % NS;
      const uint64_t a0 = sdesc_sw128(sQ + h * C::kTile, 16, 1024);
      const uint64_t b0 = sdesc_sw128(sK + st * C::kTile, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk / 4) * (128 * 128) + (kk % 4) * 32;
        if (elect_one()) mma_ss(tmem + h * 128, sdesc_add(a0, off), sdesc_add(b0, off), idesc_qk, kk > 0 ? 1u : 0u);
      }
      if (elect_one()) {
        tc_commit(&sh.bar_s[h]);
        if (k_free(t, active(h ^ 1, t), h ? on0 : on1)) tc_commit(&sh.bar_kempty[st]);
      }
      __syncwarp();
      ++(h ? done1 : done0);
      (h ? on1 : on0) = t;
    };
    auto next = [&](int h, int t) {
      while (t < t1 && !active(h, t)) ++t;
      return t;
    };
    // (a host test replays this order)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = next(h, t0);
      if (h < n_slot && t < t1) qk(h, t);
    }
    bool o_init[2] = {false, false};
    for (int t = t0; ok && t < t1; ++t) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!ok || !active(h, t)) continue;
        wait(&sh.bar_p[h], ((h ? done1 : done0) - 1) & 1);
        landed(sh.bar_v, v_seen, t);
        if (!ok) break;
        const int st = (t - t0) % NS;
        const uint64_t b0 = sdesc_sw128(sV + st * C::kTile, 128 * 128, 1024);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          if (elect_one())
            mma_ts(tmem + 256 + h * 128, tmem + h * 128 + kk * 8, sdesc_add(b0, kk * 2048), idesc_pv,
                   kk > 0 || o_init[h] ? 1u : 0u);
        o_init[h] = true;
        if (v_free(h, active(h ^ 1, t)) && elect_one()) tc_commit(&sh.bar_vempty[st]);
        __syncwarp();
        const int tn = next(h, t + 1);
        if (tn < t1) qk(h, tn);
      }
    }
    if (elect_one()) {
      tc_commit(&sh.bar_o[0]);
      tc_commit(&sh.bar_o[1]);
      tc_commit(&sh.bar_fin);
    }
    __syncwarp();
    mbar_wait(&sh.bar_fin, 0, p.err);       // every MMA has completed before tensor memory is freed
  } else if (warp < 4) {
    // ===================================================== cleaning of V tiles
    const int x = tid - 64;
    int seen[NS] = {}, n_dirty = 0;
    for (int t = t0; t < t1 && n_dirty < kMaxDirty; ++t) {
      if (!dirty(t)) continue;
      const int st = (t - t0) % NS;
      int fill = 0;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (i == st) fill = seen[i]++;
      const bool got = mbar_wait_or_abort(&sh.bar_vraw[st], fill & 1, p.err, abort_flag);
      if (named_sync_or(9, 64, !got)) break;
      uint4* v = reinterpret_cast<uint4*>(smem + C::kV + st * C::kTile);
      // adding 1 to an exponent of all ones carries into the sign bit
      uint32_t bad = 0;
#pragma unroll 1
      for (int i = x; i < C::kTile / 16; i += 64 * 8) {
        uint4 w[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = v[i + 64 * q];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          bad |= ((w[q].x & 0x7f807f80u) + 0x00800080u) | ((w[q].y & 0x7f807f80u) + 0x00800080u) |
                 ((w[q].z & 0x7f807f80u) + 0x00800080u) | ((w[q].w & 0x7f807f80u) + 0x00800080u);
      }
      if (bad & 0x80008000u) {
#pragma unroll 1
        for (int i = x; i < C::kTile / 16; i += 64) {
          uint4 w = v[i];
          if (nonfinite_bf16x2(w.x) | nonfinite_bf16x2(w.y) | nonfinite_bf16x2(w.z) | nonfinite_bf16x2(w.w)) {
            w.x = finite_or_zero_bf16x2(w.x);
            w.y = finite_or_zero_bf16x2(w.y);
            w.z = finite_or_zero_bf16x2(w.z);
            w.w = finite_or_zero_bf16x2(w.w);
            v[i] = w;
            const int row = i / 8 % 128;
            if (128 * t + row < run.n) {
              atomicOr(&sh.bad[n_dirty][row >> 5], 1u << (row & 31));
              sh.any_bad = 1;
            }
          }
        }
      }
      if (x == 0) {
        sh.dirty_tile[n_dirty] = t;
        sh.n_dirty = n_dirty + 1;
      }
      ++n_dirty;
      fence_proxy_async();
      named_sync(9, 64);
      if (x == 0) mbar_arrive(&sh.bar_v[st]);
    }
  } else {
    // ============================================================ softmax
    const int h = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1, quad = warp & 3;
    const int i = quad * 32 + lane;                   // row of the tile = tensor-memory lane
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem + h * 128 + lane_off, tO = tmem + 256 + h * 128 + half * (D / 2) + lane_off;
    const uint32_t pair_bar = 1 + h * 4 + quad;       // the two warps of these 32 rows
    // the query row of this thread
    const int bb = tile_seq(h) + i / (wr.pos_per_tile * G), r = tile_row(h) + i / G % wr.pos_per_tile;
    bool valid = h < n_slot && i < wr.pos_per_tile * wr.seqs_per_tile * G && bb < B && r < M;
    if (valid) valid = r < (prefix ? cache_len(p.mask.q_len, bb, M, p.err) : nq_own);
    const int pos = L - nq_own + r;
    const int hi = prefix ? L - 1 : run.hi(pos), lo = prefix ? 0 : run.lo(pos, p.mask.window);
    float m_run = -INFINITY, l_run = 0.f;
    int k = 0;
    for (int t = t0; t < t1; ++t) {
      if (!active(h, t)) continue;
      // (after an abort the waits return at once; the loop still runs to its end,
      // so that both warps take the same barriers)
      mbar_wait_or_abort(&sh.bar_s[h], k & 1, p.err, abort_flag);
      tc_fence_after();
      uint32_t x[64];
      tmem_ld64(tS + half * 64, x);
      if (!full(h, t)) {
        // columns e <= e_hi with e < e_s or e >= e_lo, as bits
        const int v0 = 128 * t + half * 64, e_hi = hi - v0, e_lo = lo - v0, e_s = run.n_sink - v0;
        auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; };   // bits 0 .. n-1
        const unsigned long long see = below(e_hi + 1) & (below(e_s) | ~below(e_lo));
        const uint32_t see0 = static_cast<uint32_t>(see), see1 = static_cast<uint32_t>(see >> 32);
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (!((e < 32 ? see0 : see1) & (1u << (e & 31)))) x[e] = __float_as_uint(-INFINITY);
      }
      float mm[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        mm[q] = fmax3(__uint_as_float(x[q]), __uint_as_float(x[8 + q]), __uint_as_float(x[16 + q]));
        mm[q] = fmax3(mm[q], __uint_as_float(x[24 + q]), __uint_as_float(x[32 + q]));
        mm[q] = fmax3(mm[q], __uint_as_float(x[40 + q]), __uint_as_float(x[48 + q]));
        mm[q] = fmaxf(mm[q], __uint_as_float(x[56 + q]));
      }
      float cm = fmax3(fmax3(mm[0], mm[1], mm[2]), fmax3(mm[3], mm[4], mm[5]), fmaxf(mm[6], mm[7])) * p.scale_log2;
      // the other half's maximum; past this barrier both halves of S are read,
      // so P may overwrite them
      sh.row_max[k & 1][h][half][i] = cm;
      named_sync(pair_bar, 64);
      cm = fmaxf(cm, sh.row_max[k & 1][h][half ^ 1][i]);
      // The running maximum moves only when the row's grows by more than 2^8, so
      // P stays below 2^8 and O is rarely rescaled.  (PV of this slot's previous
      // tile has completed: the S-ready barrier tracks every MMA before this QK^T.)
      const bool up = cm > (m_run == -INFINITY ? -INFINITY : m_run + kRescaleSlack);
      if (__any_sync(0xffffffffu, up)) {
        const float m_new = up ? cm : m_run;
        const float alpha = m_new == -INFINITY ? 1.0f : ex2(m_run - m_new);
        if (k > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) rescale_o<D>(tO, alpha);
        l_run *= alpha;
        m_run = m_new;
      }
      const float m_use = m_run == -INFINITY ? 0.f : m_run;
      unsigned long long ps2[4] = {0ull, 0ull, 0ull, 0ull};
      const unsigned long long sc2 = f2_pack(p.scale_log2, p.scale_log2), nm2 = f2_pack(-m_use, -m_use);
      uint32_t u[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const unsigned long long y =
            f2_fma(f2_pack(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), sc2, nm2);
        float y0, y1;
        f2_unpack(y, y0, y1);
        const float a0 = ex2(y0), a1 = ex2(y1);
        ps2[e & 3] = f2_add(ps2[e & 3], f2_pack(a0, a1));
        u[e] = cvt_bf16x2(a0, a1);
      }
      tmem_st32(tS + half * 32, u);
      float s0, s1, s2, s3, s4, s5, s6, s7;
      f2_unpack(ps2[0], s0, s1);
      f2_unpack(ps2[1], s2, s3);
      f2_unpack(ps2[2], s4, s5);
      f2_unpack(ps2[3], s6, s7);
      l_run += ((s0 + s1) + (s2 + s3)) + ((s4 + s5) + (s6 + s7));
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.bar_p[h]);
      ++k;
    }
    // ---- epilogue
    if (h < n_slot) {
      // (also where the slot has had no tile: the staging below overwrites tiles that
      // the other slot's MMAs read, and Q may still be landing)
      bool ok = mbar_wait_or_abort(&sh.bar_o[h], 0, p.err, abort_flag);
      tc_fence_after();
      // the row's sum over both halves (the maxima of both parities may still be
      // read: a barrier before and after)
      named_sync(pair_bar, 64);
      sh.row_max[0][h][half][i] = l_run;
      named_sync(pair_bar, 64);
      l_run += sh.row_max[0][h][half ^ 1][i];
      if (!valid || k == 0) l_run = 0.f;
      ok = __all_sync(0xffffffffu, ok && !*abort_flag);
      const int n_all = parts.prefix + parts.own, slot = prefix ? part : parts.prefix + part;
      const int64_t out = (static_cast<int64_t>(bb) * Hq + hk * G + i % G) * M + r;
      const int n_dirty = sh.any_bad ? sh.n_dirty : 0;
      const bool last = n_all == 1;                   // write the result, else this part's sums
      const float inv = l_run == 0.f ? 0.f : last ? 1.0f / l_run : 1.0f;
      unsigned char* dst =
          last ? reinterpret_cast<unsigned char*>(static_cast<__nv_bfloat16*>(const_cast<void*>(p.O.ptr)) +
                                                  bb * p.O.sB + (hk * G + i % G) * p.O.sH + r * p.O.sN + half * (D / 2))
               : reinterpret_cast<unsigned char*>(parts.acc + (out * n_all + slot) * D + half * (D / 2));
      // Rows go through shared memory (every MMA has completed, so the tiles are
      // free), 32 columns of the warp's 32 rows at a time, so that a store covers
      // whole runs of a row: 16-byte chunk c of row i lies at chunk c ^ (i mod 8).
      uint4* stage = reinterpret_cast<uint4*>(smem + (warp - 4) * 4096);
      const bool write = valid && (last || l_run != 0.f);
#pragma unroll 1
      for (int c = 0; ok && c < D / 64; ++c) {
        uint32_t u[32];
        if (k > 0) tmem_ld32(tO + c * 32, u);
        if (l_run == 0.f) {
#pragma unroll
          for (int e = 0; e < 32; ++e) u[e] = 0u;
        }
        for (int q = 0; q < n_dirty * 128; ++q) {
          if (!valid || !((sh.bad[q / 128][q / 32 % 4] >> (q % 32)) & 1u)) continue;
          const int v = 128 * sh.dirty_tile[q / 128] + q % 128;
          if (v > hi || (v < lo && v >= run.n_sink)) continue;
          const __nv_bfloat16* vr = static_cast<const __nv_bfloat16*>(p.V.ptr) + b_own * p.V.sB + hk * p.V.sH +
                                    static_cast<int64_t>(run.key(v)) * p.V.sN + half * (D / 2) + c * 32;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float f = __bfloat162float(vr[e]);
            if (!isfinite(f)) u[e] = __float_as_uint(__uint_as_float(u[e]) + f);
          }
        }
        const int chunks = last ? 4 : 8;              // of 16 bytes a row
        if (last) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(u[8 * e + 0]) * inv, __uint_as_float(u[8 * e + 1]) * inv);
            w.y = pack_bf16x2(__uint_as_float(u[8 * e + 2]) * inv, __uint_as_float(u[8 * e + 3]) * inv);
            w.z = pack_bf16x2(__uint_as_float(u[8 * e + 4]) * inv, __uint_as_float(u[8 * e + 5]) * inv);
            w.w = pack_bf16x2(__uint_as_float(u[8 * e + 6]) * inv, __uint_as_float(u[8 * e + 7]) * inv);
            stage[lane * 8 + (e ^ (lane & 7))] = w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            stage[lane * 8 + (e ^ (lane & 7))] = make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
        }
        __syncwarp();
#pragma unroll 4
        for (int q = lane; q < 32 * chunks; q += 32) {
          const int row = q / chunks, e = q % chunks;
          const uint4 w = stage[row * 8 + (e ^ (row & 7))];
          unsigned char* to = reinterpret_cast<unsigned char*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), row));
          if (__shfl_sync(0xffffffffu, write, row)) *reinterpret_cast<uint4*>(to + c * chunks * 16 + e * 16) = w;
        }
        __syncwarp();
      }
      if (valid && ok && half == 0) {
        if (!last)
          parts.ml[out * n_all + slot] = make_float2(l_run == 0.f ? -INFINITY : m_run, l_run);
        else if (p.lse)
          p.lse[out] = l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * 0.69314718055994531f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  end_in(parts.order);
}

template <int D>
cudaError_t launch(const CacheAttnParams& p, const AttnParts& parts, bool prefix, cudaStream_t s) {
  const TensorDesc& K = prefix ? p.Kp : p.K;
  const TensorDesc& V = prefix ? p.Vp : p.V;
  const int G = static_cast<int>(p.Q.H / p.K.H);
  const WideRows wr = wide_rows(p.Q.B, p.Q.N, G, prefix);
  WideMaps maps;
  if (!encode_queries_map(&maps.q, p.Q, G, wr.pos_per_tile, wr.seqs_per_tile) ||
      !encode_keys_map(&maps.k, K, 128) || !encode_keys_map(&maps.v, V, 128) || !encode_keys_map(&maps.k16, K, 16) ||
      !encode_keys_map(&maps.v16, V, 16))
    return cudaErrorNotSupported;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(attn_wide_kernel<D>, WideCfg<D>::kBytes, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((wr.tiles + 1) / 2 * (prefix ? parts.prefix : parts.own)),
                  static_cast<unsigned>(p.K.H * (prefix ? 1 : p.K.B)));
  return launch_after(attn_wide_kernel<D>, grid, kThreads, WideCfg<D>::kBytes, 1, s, p, parts, prefix, wr, maps);
}

}  // namespace

// Tensor map over dims (D, d1, d2, d3) of a bf16 tensor with the given element
// strides; extents of broadcast (zero-stride) dimensions are 1.  Strides of
// extent-1 dimensions are never used and replaced by valid ones.
static bool encode_map(CUtensorMap* map, const void* ptr, int64_t D, const int64_t (&ext)[3], const int64_t (&str)[3],
            const int (&box)[3]) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), 1, 1, 1}, strides[3];
  cuuint32_t boxes[4] = {64, 1, 1, 1}, ones[4] = {1, 1, 1, 1};
  for (int i = 0; i < 3; ++i) {
    dims[i + 1] = str[i] == 0 ? 1 : static_cast<cuuint64_t>(ext[i]);
    strides[i] = 2 * static_cast<cuuint64_t>(dims[i + 1] == 1 ? D : str[i]);
    boxes[i + 1] = static_cast<cuuint32_t>(box[i]);
  }
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, boxes, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool encode_keys_map(CUtensorMap* map, const TensorDesc& t, int rows) {
  return encode_map(map, t.ptr, t.D, {t.N, t.H, t.B}, {t.sN, t.sH, t.sB}, {rows, 1, 1});
}

bool encode_queries_map(CUtensorMap* map, const TensorDesc& t, int heads, int positions, int seqs) {
  return encode_map(map, t.ptr, t.D, {t.H, t.N, t.B}, {t.sH, t.sN, t.sB}, {heads, positions, seqs});
}

int64_t wide_units(const TensorDesc& Q, const TensorDesc& K, bool prefix) {
  const WideRows w = wide_rows(Q.B, Q.N, Q.H / K.H, prefix);
  return (w.tiles + 1) / 2 * K.H * (prefix ? 1 : K.B);
}

cudaError_t launch_attn_wide(const CacheAttnParams& p, const AttnParts& parts, bool prefix, cudaStream_t s) {
  return p.Q.D == 128 ? launch<128>(p, parts, prefix, s) : launch<64>(p, parts, prefix, s);
}

}  // namespace pbs
