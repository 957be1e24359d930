// Replays the order in which attn_wide_kernel issues its products and frees the K
// stages, over causal windows of many shapes: a stage is freed once per tile, and only
// when the products of both slots on that tile have been issued; and no product waits
// for a tile whose load waits for a later product (tiles are loaded K, V, K, V ...,
// each into the stage that the tile kStages before it has freed).
#include <algorithm>
#include <cstdio>
#include <vector>

#include "wide_order.h"

namespace {

struct Slots {
  int n_slot, n_sink, up0, up1, low0, low1;
  bool active(int h, int t) const {
    return h < n_slot && pbs::slot_uses(t, h ? up1 : up0, h ? low1 : low0, n_sink);
  }
  int next(int h, int t, int t1) const {
    while (t < t1 && !active(h, t)) ++t;
    return t;
  }
};

// The kernel's order over tiles t0 .. t1 - 1: qk(h, t) for S = Q K^T of a slot's first
// tile, then for each tile and slot pv(h, t) and the qk of the slot's next tile.
template <typename Qk, typename Pv>
void issue(const Slots& s, int t0, int t1, Qk qk, Pv pv) {
  for (int h = 0; h < 2; ++h) {
    const int t = s.next(h, t0, t1);
    if (h < s.n_slot && t < t1) qk(h, t);
  }
  for (int t = t0; t < t1; ++t) {
    for (int h = 0; h < 2; ++h) {
      if (!s.active(h, t)) continue;
      pv(h, t);
      const int tn = s.next(h, t + 1, t1);
      if (tn < t1) qk(h, tn);
    }
  }
}

int failures = 0;
long long shapes = 0, ahead = 0;   // shapes replayed; tiles on which slot 1's product comes first

// One CTA: rows at positions first .. first + n - 1 of each slot, one part of the keys.
void replay(int first0, int n0, int first1, int n1, int window, int n_sink, int n_parts) {
  const int last = n1 ? first1 + n1 - 1 : first0 + n0 - 1;
  if (last < 0) return;
  // the run of virtual indices (sinks rounded up to 16, then the window)
  const int low = std::max(0, first0 - window + 1), sinks = std::min(n_sink, last + 1);
  const int sink_end = (sinks + 15) / 16 * 16, delta = std::max(0, low - sink_end), n = last + 1 - delta;
  auto lo = [&](int pos) { return std::max(0, pos - window + 1) - delta; };
  const Slots s{n1 ? 2 : 1, sinks, first0 + n0 - 1 - delta, first1 + n1 - 1 - delta, lo(first0), lo(first1)};
  const int tiles = (n + 127) / 128;
  for (int part = 0; part < n_parts; ++part) {
    const int t0 = static_cast<int>(static_cast<long long>(tiles) * part / n_parts);
    const int t1 = static_cast<int>(static_cast<long long>(tiles) * (part + 1) / n_parts);
    std::vector<int> issued[2], freed(tiles, 0), v_freed(tiles, 0);
    int last_issued[2] = {t0 - 1, t0 - 1};
    for (auto& v : issued) v.assign(tiles, 0);
    bool ok = true;
    // the tile kStages (2 or 4) before t has been freed by now
    auto room = [&](const std::vector<int>& f, int t) { return t - 2 < t0 || (f[t - 2] && (t - 4 < t0 || f[t - 4])); };
    issue(
        s, t0, t1,
        [&](int h, int t) {
          ok = ok && s.active(h, t) && t > last_issued[h] && !freed[t];
          ok = ok && room(freed, t) && (t == t0 || room(v_freed, t - 1));
          issued[h][t] = 1;
          last_issued[h] = t;
          if (pbs::k_free(t, s.active(h ^ 1, t), last_issued[h ^ 1])) {
            for (int q = 0; q < 2; ++q) ok = ok && (!s.active(q, t) || issued[q][t]);
            ++freed[t];
          }
          if (h == 1 && s.active(0, t) && !issued[0][t]) ++ahead;
        },
        [&](int h, int t) {
          ok = ok && issued[h][t] && room(v_freed, t);
          if (pbs::v_free(h, s.active(h ^ 1, t))) {
            ok = ok && !v_freed[t];
            v_freed[t] = 1;
          }
        });
    for (int t = t0; t < t1; ++t) ok = ok && freed[t] == 1 && v_freed[t];
    if (!ok && ++failures <= 5)
      std::printf("slots at %d (%d rows) and %d (%d), window %d, sinks %d, part %d of %d\n", first0, n0, first1, n1,
                  window, n_sink, part, n_parts);
  }
  ++shapes;
}

}  // namespace

int main() {
  for (int span : {128, 64, 32, 25, 2})                       // positions of a slot
    for (int window : {1, 17, 100, 128, 384, 512, 700, 1 << 20})
      for (int n_sink : {0, 1, 16, 100, 112, 113, 128, 129, 256, 300})
        for (int first = -150; first < 1700; first += first < 0 ? 37 : 64)
          for (int n1 : {0, 1, span})
            for (int parts : {1, 3}) replay(first, span, first + span, n1, window, n_sink, parts);
  std::printf("%lld shapes, %lld tiles with slot 1 first, %d failures\n", shapes, ahead, failures);
  return failures || !ahead;
}
