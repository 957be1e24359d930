// The two slots of a CTA of attn_wide_kernel: which tiles of its keys a slot uses, and
// when a K or V stage is free again.  Plain C++, so that a host test can replay the
// order in which the kernel issues its products.
#pragma once

#ifdef __CUDACC__
#define PBS_ORDER __device__ __forceinline__
#else
#define PBS_ORDER inline
#endif

namespace pbs {

// Does a slot see any key of tile t (indices 128 t .. 128 t + 127)?  `up` is the last
// index that its last row sees, `low` the first of its first row's window.
PBS_ORDER bool slot_uses(int t, int up, int low, int n_sink) {
  return 128 * t <= up && (128 * t + 127 >= low || 128 * t < n_sink);
}

// A slot's Q K^T on tile t has been issued; the other slot uses the tile or not, and
// its last one was on tile `other`.  Are all products on this K tile issued, so that
// its stage is free once they complete?  Either slot may be the later one: where slot 1
// skips a tile that slot 0 uses it runs a tile ahead.
PBS_ORDER bool k_free(int t, bool other_uses, int other) { return !other_uses || other >= t; }

// The same of PV, which slot 0 issues first on every tile.
PBS_ORDER bool v_free(int h, bool other_uses) { return h == 1 || !other_uses; }

}  // namespace pbs
