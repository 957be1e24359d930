// C-ABI entry points of the cache operators (pbs_attn_window,
// pbs_attn_prefix, pbs_key_mass, pbs_evict): argument checks and launches.
// See include/pbs.h for their contracts.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "pbs_internal.h"

namespace {

using pbs::TensorDesc;

int fail(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return pbs::api_fail(code, buf);
}

int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return pbs::api_ok();
  return fail(PBS_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

// The sizes that pbs_workspace_size gives.
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

bool broadcast(const TensorDesc& t) { return (t.H > 1 && t.sH == 0) || (t.B > 1 && t.sB == 0); }

// Queries against a cache: shapes, head groups and the mask's numbers.
int check_pair(const TensorDesc& Q, const TensorDesc& K, int64_t window, int n_sink, float scale) {
  if (const int rc = pbs::api_check_cache_shapes(Q, K)) return rc;
  if (broadcast(Q)) return fail(PBS_ERR_UNSUPPORTED, "Q may not be a broadcast view (zero head or batch stride)");
  if (window < 0 || n_sink < 0) return fail(PBS_ERR_INVALID_ARG, "window/n_sink negative");
  if (!(scale > 0.0f) || !std::isfinite(scale * 1.4426950408889634f))
    return fail(PBS_ERR_INVALID_ARG, "softmax_scale must be positive and finite");
  return PBS_OK;
}

int check_same(const TensorDesc& V, const TensorDesc& K, const char* v, const char* k) {
  if (V.B != K.B || V.H != K.H || V.N != K.N || V.D != K.D)
    return fail(PBS_ERR_INVALID_ARG, "%s shape differs from %s", v, k);
  return PBS_OK;
}

pbs::CacheMask mask_of(const TensorDesc& K, const int32_t* kv_len, const int32_t* q_len, int64_t window, int n_sink) {
  pbs::CacheMask m;
  m.kv_len = kv_len;
  m.q_len = q_len;
  m.window = window == 0 || window > K.N ? K.N : window;
  m.n_sink = static_cast<int>(n_sink < K.N ? n_sink : K.N);
  return m;
}

// One axis of two arrays of elements: sizes and strides (in elements) in each.
struct Axis {
  int64_t n_a, n_b, s_a, s_b;
};

// Do arrays over axes of the same strides, largest first, share an element, where
// the second begins `delta` elements after the first?  They do if delta = sum of
// d_k s_k for differences d_k of their indices.
bool meet(int64_t delta, const Axis* x, int n) {
  if (n == 0) return delta == 0;
  int64_t lo = 0, hi = 0;                             // what the other axes can make up
  for (int k = 1; k < n; ++k) {
    lo -= (x[k].n_b - 1) * x[k].s_a;
    hi += (x[k].n_a - 1) * x[k].s_a;
  }
  const int64_t s = x[0].s_a;
  auto down = [s](int64_t v) { return v >= 0 ? v / s : -((-v + s - 1) / s); };
  const int64_t first = std::max(-(x[0].n_b - 1), -down(hi - delta)), last = std::min(x[0].n_a - 1, down(delta - lo));
  if (last - first > 8) return true;                  // (strides that do not nest: taken to overlap)
  for (int64_t d = first; d <= last; ++d)
    if (meet(delta - d * s, x + 1, n - 1)) return true;
  return false;
}

// Do two arrays of elements of `size` bytes overlap?  Exact where their strides are
// the same (the halves of one buffer do not), else by their first and last bytes.
bool overlap(const void* a, const void* b, int64_t size, std::initializer_list<Axis> axes) {
  const int64_t delta = static_cast<const char*>(b) - static_cast<const char*>(a);
  Axis x[4];
  int n = 0;
  int64_t end_a = 1, end_b = 1;
  bool exact = delta % size == 0;
  for (Axis y : axes) {
    end_a += (y.n_a - 1) * y.s_a;
    end_b += (y.n_b - 1) * y.s_b;
    if (y.n_a == 1) y.s_a = y.s_b;
    if (y.n_b == 1) y.s_b = y.s_a;
    if (y.s_a != y.s_b) exact = false;
    if ((y.n_a > 1 || y.n_b > 1) && y.s_a != 0) x[n++] = y;
  }
  if (delta >= end_a * size || -delta >= end_b * size) return false;
  if (!exact) return true;
  std::sort(x, x + n, [](const Axis& l, const Axis& r) { return l.s_a > r.s_a; });
  return meet(delta / size, x, n);
}
bool overlap(const TensorDesc& a, const TensorDesc& b) {
  return overlap(a.ptr, b.ptr, 2,
                 {{a.B, b.B, a.sB, b.sB}, {a.H, b.H, a.sH, b.sH}, {a.N, b.N, a.sN, b.sN}, {a.D, b.D, 1, 1}});
}

// Rows of fp32, `stride` elements apart.
bool rows_overlap(const float* a, int64_t a_stride, int64_t a_len, const float* b, int64_t b_stride, int64_t b_len,
                  int64_t rows) {
  return overlap(a, b, 4, {{rows, rows, a_stride, b_stride}, {a_len, b_len, 1, 1}});
}

// Two arrays of int32 (NULL: none).
bool ints_overlap(const int32_t* a, int64_t n_a, const int32_t* b, int64_t n_b) {
  return a && b && overlap(a, b, 4, {{n_a, n_b, 1, 1}});
}

int attn(const pbs_tensor* Qt, const pbs_tensor* Kpt, const pbs_tensor* Vpt, bool prefix, const pbs_tensor* Kt,
         const pbs_tensor* Vt, const int32_t* kv_len, const int32_t* q_len, int64_t window, int n_sink,
         float softmax_scale, pbs_tensor* Ot, float* lse, void* ws, size_t ws_bytes, void* stream, const char* what) {
  pbs::CacheAttnParams p;
  int rc;
  if ((rc = pbs::api_check_tensor(Qt, "Q", &p.Q)) || (rc = pbs::api_check_tensor(Kt, "K", &p.K)) ||
      (rc = pbs::api_check_tensor(Vt, "V", &p.V)) || (rc = pbs::api_check_tensor(Ot, "O", &p.O)))
    return rc;
  if ((rc = check_pair(p.Q, p.K, window, n_sink, softmax_scale)) || (rc = check_same(p.V, p.K, "V", "K")) ||
      (rc = check_same(p.O, p.Q, "O", "Q")))
    return rc;
  if (broadcast(p.O)) return fail(PBS_ERR_UNSUPPORTED, "O may not be a broadcast view (zero head or batch stride)");
  p.Kp = p.Vp = TensorDesc{};
  if (prefix) {
    if ((rc = pbs::api_check_tensor(Kpt, "Kp", &p.Kp)) || (rc = pbs::api_check_tensor(Vpt, "Vp", &p.Vp)) ||
        (rc = check_same(p.Vp, p.Kp, "Vp", "Kp")))
      return rc;
    if (p.Kp.B != 1 || p.Kp.H != p.K.H || p.Kp.D != p.K.D)
      return fail(PBS_ERR_INVALID_ARG, "Kp must be [1, Hkv, P, D] with K's Hkv and D");
  }
  if ((rc = pbs::api_check_ws(ws, ws_bytes, align256(pbs::cache_attn_ws_bytes(p.Q, p.K, prefix))))) return rc;
  p.mask = mask_of(p.K, kv_len, q_len, window, n_sink);
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.lse = lse;
  p.ws = ws;
  p.err = pbs::api_device_error_word();
  if (!p.err) return fail(PBS_ERR_CUDA, "cannot resolve the device error word");
  return launched(pbs::launch_cache_attn(p, static_cast<cudaStream_t>(stream)), what);
}

}  // namespace

namespace pbs {

// (the plans of the kernels divide by the rows that fit a tile: they are only made for
// shapes that pass)
int api_check_cache_shapes(const TensorDesc& Q, const TensorDesc& K) {
  if (Q.B != K.B || Q.D != K.D) return fail(PBS_ERR_INVALID_ARG, "Q and K disagree on B or D");
  if (Q.H % K.H)
    return fail(PBS_ERR_INVALID_ARG, "Hq %lld not a multiple of Hkv %lld", (long long)Q.H, (long long)K.H);
  if (Q.H / K.H > 64) return fail(PBS_ERR_UNSUPPORTED, "Hq / Hkv %lld > 64", (long long)(Q.H / K.H));
  if (Q.B > 65535 || K.H > 65535 || Q.B * K.H > 65535)
    return fail(PBS_ERR_UNSUPPORTED, "B * Hkv above 65535");
  if (Q.B * Q.H * Q.N >= (1ll << 31)) return fail(PBS_ERR_UNSUPPORTED, "B * Hq * M above 2^31");
  return PBS_OK;
}

}  // namespace pbs

extern "C" {

int pbs_attn_window(const pbs_tensor* Qt, const pbs_tensor* Kt, const pbs_tensor* Vt, const int32_t* kv_len,
                    const int32_t* q_len, int64_t window, int n_sink, float softmax_scale, pbs_tensor* Ot, float* lse,
                    void* ws, size_t ws_bytes, void* stream) {
  return attn(Qt, nullptr, nullptr, false, Kt, Vt, kv_len, q_len, window, n_sink, softmax_scale, Ot, lse, ws, ws_bytes,
              stream, "attn_window");
}

int pbs_attn_prefix(const pbs_tensor* Qt, const pbs_tensor* Kpt, const pbs_tensor* Vpt, const pbs_tensor* Kt,
                    const pbs_tensor* Vt, const int32_t* kv_len, const int32_t* q_len, float softmax_scale,
                    pbs_tensor* Ot, float* lse, void* ws, size_t ws_bytes, void* stream) {
  return attn(Qt, Kpt, Vpt, true, Kt, Vt, kv_len, q_len, 0, 0, softmax_scale, Ot, lse, ws, ws_bytes, stream,
              "attn_prefix");
}

int pbs_key_mass(const pbs_tensor* Qt, const pbs_tensor* Kt, const float* lse, const int32_t* kv_len,
                 const int32_t* q_len, int64_t window, int n_sink, float decay, float softmax_scale,
                 const float* prev, int64_t prev_stride, float* mass, int64_t mass_stride, void* ws, size_t ws_bytes,
                 void* stream) {
  pbs::KeyMassParams p;
  int rc;
  if ((rc = pbs::api_check_tensor(Qt, "Q", &p.Q)) || (rc = pbs::api_check_tensor(Kt, "K", &p.K))) return rc;
  if ((rc = check_pair(p.Q, p.K, window, n_sink, softmax_scale))) return rc;
  if (!lse || !mass) return fail(PBS_ERR_INVALID_ARG, "lse or mass is null");
  if (mass_stride < p.K.N || (prev && prev_stride < p.K.N))
    return fail(PBS_ERR_INVALID_ARG, "mass and prev rows must be at least N = %lld elements apart", (long long)p.K.N);
  if (prev && !(prev == mass && prev_stride == mass_stride) &&
      rows_overlap(prev, prev_stride, p.K.N, mass, mass_stride, p.K.N, p.K.B * p.K.H))
    return fail(PBS_ERR_INVALID_ARG, "prev and mass overlap without being the same");
  if (prev && (!(decay >= 0.0f) || !std::isfinite(decay)))
    return fail(PBS_ERR_INVALID_ARG, "decay must be finite and >= 0");
  if ((rc = pbs::api_check_ws(ws, ws_bytes, align256(pbs::key_mass_ws_bytes(p.Q, p.K))))) return rc;
  p.mask = mask_of(p.K, kv_len, q_len, window, n_sink);
  p.lse = lse;
  p.prev = prev;
  p.prev_stride = prev_stride;
  p.mass_stride = mass_stride;
  p.decay = prev ? decay : 1.0f;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.mass = mass;
  p.ws = ws;
  p.err = pbs::api_device_error_word();
  if (!p.err) return fail(PBS_ERR_CUDA, "cannot resolve the device error word");
  return launched(pbs::launch_key_mass(p, static_cast<cudaStream_t>(stream)), "key_mass");
}

int pbs_evict(const float* mass, int64_t mass_stride, const pbs_tensor* Kt, const pbs_tensor* Vt,
              const int32_t* kv_len, int budget, int recent, int n_sink, int32_t* keep, int32_t* new_len,
              pbs_tensor* Kot, pbs_tensor* Vot, float* mass_out, int64_t mass_out_stride, void* /*ws*/,
              size_t /*ws_bytes*/, void* stream) {
  pbs::EvictParams p;
  int rc;
  if ((rc = pbs::api_check_tensor(Kt, "K", &p.K)) || (rc = pbs::api_check_tensor(Vt, "V", &p.V)) ||
      (rc = pbs::api_check_tensor(Kot, "K_out", &p.Ko)) || (rc = pbs::api_check_tensor(Vot, "V_out", &p.Vo)))
    return rc;
  if ((rc = check_same(p.V, p.K, "V", "K")) || (rc = check_same(p.Vo, p.Ko, "V_out", "K_out"))) return rc;
  if (p.Ko.B != p.K.B || p.Ko.H != p.K.H || p.Ko.D != p.K.D)
    return fail(PBS_ERR_INVALID_ARG, "K_out and K disagree on B, Hkv or D");
  if (p.K.B * p.K.H > 65535) return fail(PBS_ERR_UNSUPPORTED, "B * Hkv above 65535");
  if (!mass || !keep || !mass_out) return fail(PBS_ERR_INVALID_ARG, "mass, keep or mass_out is null");
  if (budget < 1 || budget > p.K.N || p.Ko.N < budget)
    return fail(PBS_ERR_INVALID_ARG, "budget %d must be in [1, N] and fit K_out", budget);
  if (recent < 0 || n_sink < 0 || static_cast<int64_t>(recent) + n_sink > budget)
    return fail(PBS_ERR_INVALID_ARG, "recent and n_sink must be >= 0 and fit the budget together");
  if (mass_stride < p.K.N || mass_out_stride < budget)
    return fail(PBS_ERR_INVALID_ARG, "mass or mass_out rows too close together");
  if (broadcast(p.Ko) || broadcast(p.Vo))
    return fail(PBS_ERR_UNSUPPORTED, "K_out and V_out may not be broadcast views");
  if (overlap(p.Ko, p.K) || overlap(p.Ko, p.V) || overlap(p.Vo, p.K) || overlap(p.Vo, p.V) || overlap(p.Ko, p.Vo) ||
      rows_overlap(mass, mass_stride, p.K.N, mass_out, mass_out_stride, budget, p.K.B * p.K.H))
    return fail(PBS_ERR_INVALID_ARG, "outputs overlap inputs or each other");
  const int64_t n_kept = p.K.B * p.K.H * budget;
  if (ints_overlap(keep, n_kept, kv_len, p.K.B) || ints_overlap(keep, n_kept, new_len, p.K.B) ||
      (new_len != kv_len && ints_overlap(new_len, p.K.B, kv_len, p.K.B)))
    return fail(PBS_ERR_INVALID_ARG, "keep or new_len overlap kv_len or each other");
  p.mass = mass;
  p.mass_stride = mass_stride;
  p.mass_out_stride = mass_out_stride;
  p.kv_len = kv_len;
  p.budget = budget;
  p.recent = recent;
  p.n_sink = n_sink;
  p.keep = keep;
  p.new_len = new_len;
  p.mass_out = mass_out;
  p.err = pbs::api_device_error_word();
  if (!p.err) return fail(PBS_ERR_CUDA, "cannot resolve the device error word");
  return launched(pbs::launch_evict(p, static_cast<cudaStream_t>(stream)), "evict");
}

}  // extern "C"
