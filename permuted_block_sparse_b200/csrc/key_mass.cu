// pbs_key_mass: attention weight per key,
//   mass[j] = decay prev[j] + sum over rows r that see j of 2^(x_rj - y_r),
// x_rj = scale log2(e) Q[r].K[j], y_r = log2(e) lse[r], over the query rows of
// all heads of a KV head.  fp32 products, the sum in fp64.
#include <math.h>

#include "cache_common.cuh"

namespace pbs {
namespace {

constexpr int kThreads = 128;

// One thread per key; the query rows pass by in shared memory.
__global__ void __launch_bounds__(kThreads) key_mass_row_kernel(KeyMassParams p) {
  __shared__ float q[8][128];
  const int tid = threadIdx.x, D = static_cast<int>(p.Q.D), G = static_cast<int>(p.Q.H / p.K.H);
  const int64_t M = p.Q.N, N = p.K.N, b = blockIdx.y / p.K.H, hk = blockIdx.y % p.K.H;
  const int64_t L = cache_len(p.mask.kv_len, b, N, p.err), n_rows = cache_len(p.mask.q_len, b, M, p.err);
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kThreads + tid;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.K.ptr) + b * p.K.sB + hk * p.K.sH + j * p.K.sN;
  double sum = 0.0;
  for (int64_t i0 = 0; i0 < n_rows * G; i0 += 8) {
    __syncthreads();
    for (int i = tid; i < 8 * D; i += kThreads) {
      const int64_t row = i0 + i / D;
      if (row < n_rows * G)
        q[i / D][i % D] = __bfloat162float(static_cast<const __nv_bfloat16*>(
            p.Q.ptr)[b * p.Q.sB + (hk * G + row % G) * p.Q.sH + row / G * p.Q.sN + i % D]);
    }
    __syncthreads();
    if (j >= L) continue;
    for (int i = 0; i < 8 && i0 + i < n_rows * G; ++i) {
      const int64_t r = (i0 + i) / G, h = hk * G + (i0 + i) % G;
      const int64_t pos = L - n_rows + r;
      if (j > pos || (j <= pos - p.mask.window && j >= p.mask.n_sink)) continue;
      const float y = p.lse[(b * p.Q.H + h) * M + r];
      if (y == -INFINITY) continue;
      float s = 0.f;
      for (int c = 0; c < D; ++c) s = fmaf(q[i][c], __bfloat162float(k[c]), s);
      sum += exp2f(fmaf(s, p.scale_log2, -y * 1.4426950408889634f));
    }
  }
  if (j >= N) return;
  const float old = p.prev && j < L ? p.decay * p.prev[blockIdx.y * p.prev_stride + j] : 0.f;
  p.mass[blockIdx.y * p.mass_stride + j] = old + static_cast<float>(sum);
}

}  // namespace

size_t key_mass_ws_bytes(const TensorDesc&, const TensorDesc&) { return 0; }

cudaError_t launch_key_mass(const KeyMassParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.K.N + kThreads - 1) / kThreads), static_cast<unsigned>(p.K.B * p.K.H));
  key_mass_row_kernel<<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace pbs
