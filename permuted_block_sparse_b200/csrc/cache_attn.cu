// pbs_attn_window and pbs_attn_prefix: attention over a K/V cache.
//
//   O[r] = sum_j 2^(x_rj - m_r) V[j] / l_r,  x_rj = scale log2(e) Q[r].K[j],
//   m_r = max_j x_rj,  l_r = sum_j 2^(x_rj - m_r),  lse_r = ln 2 (m_r + log2 l_r)
//
// over the keys j that row r sees, in one pass with the running (m, l, O)
// rescaled whenever m grows.  fp32 throughout.
#include <math.h>

#include "cache_common.cuh"

namespace pbs {
namespace {

constexpr int kThreads = 128;

// One CTA per (row, query head, batch): 128 keys at a time, one per thread
// for the logits, then one output column per thread for the values.
__global__ void __launch_bounds__(kThreads) cache_attn_row_kernel(CacheAttnParams p) {
  __shared__ float q[128], w[kThreads], red[4];
  __shared__ int seen[kThreads];
  const int tid = threadIdx.x, D = static_cast<int>(p.Q.D);
  const int64_t M = p.Q.N, N = p.K.N, P = p.Kp.N;
  const int64_t r = blockIdx.x % M, h = blockIdx.x / M % p.Q.H, b = blockIdx.x / M / p.Q.H;
  const int64_t hk = h / (p.Q.H / p.K.H);
  const int64_t L = cache_len(p.mask.kv_len, b, N, p.err), n_rows = cache_len(p.mask.q_len, b, M, p.err);
  if (r >= n_rows) return;
  const int64_t pos = L - n_rows + r;
  if (tid < D)
    q[tid] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.Q.ptr)[b * p.Q.sB + h * p.Q.sH + r * p.Q.sN + tid]);
  float m = -INFINITY, l = 0.f, acc = 0.f;
  const int64_t own = pos < 0 ? 0 : pos + 1;
  for (int64_t v0 = 0; v0 < P + own; v0 += kThreads) {
    __syncthreads();
    const int64_t v = v0 + tid;
    const bool vis = v < P + own && (v < P || key_visible(v - P, pos, p.mask.window, p.mask.n_sink));
    float x = -INFINITY;
    if (vis) {
      const TensorDesc& t = v < P ? p.Kp : p.K;
      const __nv_bfloat16* k =
          static_cast<const __nv_bfloat16*>(t.ptr) + (v < P ? 0 : b * t.sB) + hk * t.sH + (v < P ? v : v - P) * t.sN;
      float s = 0.f;
      for (int c = 0; c < D; ++c) s = fmaf(q[c], __bfloat162float(k[c]), s);
      x = s * p.scale_log2;
    }
    float mx = x;
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float a = mn == -INFINITY ? 1.f : exp2f(m - mn);
    const float e = mn == -INFINITY ? 0.f : exp2f(x - mn);
    m = mn;
    w[tid] = e;
    seen[tid] = vis;
    __syncthreads();
    l *= a;
    acc *= a;
    const int n = static_cast<int>(min(static_cast<int64_t>(kThreads), P + own - v0));
    for (int i = 0; i < n; ++i) {
      l += w[i];
      const int64_t j = v0 + i;
      if (seen[i] && tid < D) {
        const TensorDesc& t = j < P ? p.Vp : p.V;
        acc = fmaf(w[i],
                   __bfloat162float(static_cast<const __nv_bfloat16*>(
                       t.ptr)[(j < P ? 0 : b * t.sB) + hk * t.sH + (j < P ? j : j - P) * t.sN + tid]),
                   acc);
      }
    }
  }
  if (tid < D)
    static_cast<__nv_bfloat16*>(const_cast<void*>(p.O.ptr))[b * p.O.sB + h * p.O.sH + r * p.O.sN + tid] =
        __float2bfloat16(l == 0.f ? 0.f : acc / l);
  if (tid == 0 && p.lse)
    p.lse[(b * p.Q.H + h) * M + r] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

size_t cache_attn_ws_bytes(const TensorDesc&, const TensorDesc&, bool) { return 0; }

cudaError_t launch_cache_attn(const CacheAttnParams& p, cudaStream_t s) {
  cache_attn_row_kernel<<<static_cast<unsigned>(p.Q.B * p.Q.H * p.Q.N), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace pbs
