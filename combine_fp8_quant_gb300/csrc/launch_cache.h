// launch_cache.h -- what the host remembers of its launch queries (host code only).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace moeperm {

struct LaunchKey {
  const void* kernel;
  size_t smem;      // dynamic shared memory
  int32_t threads;  // of a CTA, or CTAs of a cluster
  int32_t dev;
  bool operator==(const LaunchKey& o) const {
    return kernel == o.kernel && smem == o.smem && threads == o.threads && dev == o.dev;
  }
  uint64_t hash() const {
    uint64_t h = (uint64_t)(uintptr_t)kernel ^ ((uint64_t)smem << 20) ^ ((uint64_t)(uint32_t)threads << 44) ^ ((uint64_t)(uint32_t)dev << 56);
    h *= 0x9E3779B97F4A7C15ull;  // 2^64 over the golden ratio: the high bits depend on all
    return h ^ (h >> 32);
  }
};

// Answers of queries, in sets of four entries, of which a new one replaces the oldest.
// Sizes that data decide (tokens of a batch, groups of a loss) make new keys for as long as a
// program runs: they displace one another, and whatever is asked for again is found again. Not
// synchronised.
template <int SETS>
class QueryCache {
  static_assert((SETS & (SETS - 1)) == 0, "a power of two");
  struct Entry { LaunchKey key; int value; };
  struct Set { Entry e[4]; int held, next; };
  Set sets_[SETS] = {};
  Set& set_of(const LaunchKey& k) { return sets_[k.hash() % SETS]; }

 public:
  bool find(const LaunchKey& k, int* value) {
    const Set& s = set_of(k);
    for (int i = 0; i < s.held; ++i)
      if (s.e[i].key == k) {
        *value = s.e[i].value;
        return true;
      }
    return false;
  }
  void keep(const LaunchKey& k, int value) {
    int there;
    if (find(k, &there)) return;  // (another thread asked, too)
    Set& s = set_of(k);
    s.e[s.next] = {k, value};
    s.next = (s.next + 1) % 4;
    if (s.held < 4) ++s.held;
  }
};

}  // namespace moeperm
