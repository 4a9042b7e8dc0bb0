// mla_int4_shape.h - how many clusters of how many pairs the attention over packed rows
// is launched with (host only, no CUDA: compiled alone by its test).
#pragma once

#include <atomic>

namespace dsa {

// A number looked up once per slot.  A look-up that fails (a negative answer) is not
// kept: the next call asks again.
struct OnceAsked {
  std::atomic<int> kept{0};            // answer + 1
  template <class Ask>
  int get(Ask&& ask) {
    const int have = kept.load(std::memory_order_relaxed);
    if (have > 0) return have - 1;
    const int n = ask();
    if (n >= 0) kept.store(n + 1, std::memory_order_relaxed);
    return n;
  }
};

struct Int4Shape {
  int splits, clusters;                // key splits of a row = pairs of a cluster
};

// resident(s): clusters of s pairs that can be resident at once, negative where that
// is not known.  Key splits: the most whose clusters are all resident (a second wave
// costs more than a split saves), where the selection has a block of `block` keys for
// each.  Without splits one resident wave of pairs shares the rows, a pair for every two
// SMs where residency is not known: clusters never wait for one another, so that a
// number too large costs a second wave and nothing else.
template <class Resident>
Int4Shape int4_shape(int rows, int topk, int block, int sms, Resident&& resident) {
  if (topk > 2 * block && rows <= resident(4)) return {4, rows};
  if (topk > block && rows <= resident(2)) return {2, rows};
  const int known = resident(1), pairs = known > 0 ? known : sms / 2 > 0 ? sms / 2 : 1;
  return {1, rows < pairs ? rows : pairs};
}

}  // namespace dsa
