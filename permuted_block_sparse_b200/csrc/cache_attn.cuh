// Shared by the two attention kernels of the cache operators (cache_attn.cu,
// cache_attn_wide.cu): where a part of the keys leaves its result.
#pragma once

#include "cache_common.cuh"

namespace pbs {

// Parts that the prefix and the own keys are cut into (0: there is no prefix).
// With more than one in all, part s of output row i = (b Hq + h) M + r leaves
// its maximum and sum in ml[i n + s] (n parts in all) and, where the row sees a
// key in it, its accumulator in acc[(i n + s) D ...].
struct AttnParts {
  int prefix, own;
  float* acc;
  float2* ml;
  Order order;                     // of the kernel that gets this
};

// Four columns of output row `out`, and with the first ones its lse.
__device__ __forceinline__ void write_row4(const CacheAttnParams& p, int64_t out, int c, float4 acc, float m, float l) {
  const int64_t M = p.Q.N, b = out / M / p.Q.H, h = out / M % p.Q.H, r = out % M;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(const_cast<void*>(p.O.ptr)) + b * p.O.sB + h * p.O.sH + r * p.O.sN + c;
  *reinterpret_cast<uint2*>(o) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (c == 0 && p.lse) p.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// Four columns of one of n parts of output row `out`: the result itself where
// there is one part.
__device__ __forceinline__ void leave_row4(const CacheAttnParams& p, const AttnParts& parts, int n, int part,
                                           int64_t out, int c, int D, float4 acc, float m, float l) {
  if (n == 1) {
    write_row4(p, out, c, acc, m, l);
    return;
  }
  const int64_t at = out * n + part;
  if (l != 0.f) *reinterpret_cast<float4*>(parts.acc + at * D + c) = acc;
  if (c == 0) parts.ml[at] = make_float2(m, l);
}

// Pieces of work of the wide kernel before the keys are cut, and its launch
// over the prefix or the own keys.
int64_t wide_units(const TensorDesc& Q, const TensorDesc& K, bool prefix);
cudaError_t launch_attn_wide(const CacheAttnParams& p, const AttnParts& parts, bool prefix, cudaStream_t s);

}  // namespace pbs
