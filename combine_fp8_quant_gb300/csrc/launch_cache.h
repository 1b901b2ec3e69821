// launch_cache.h -- what the host remembers of its launch queries (host code only).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <mutex>

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

// How much dynamic shared memory each kernel may take in each context. It only ever rises: of
// two threads whose launches need different sizes, neither may lower what the other has set
// and is about to launch with, so a size is compared and set under one lock.
template <int ENTRIES>
class SmemOptIns {
  struct Entry { const void* kernel; unsigned long long ctx; size_t dyn; };
  std::mutex mu_;
  Entry e_[ENTRIES] = {};
  // The entry of a kernel in a context, or a free one; nullptr: none is free.
  Entry* entry(const void* kernel, unsigned long long ctx) {
    const uint64_t h = LaunchKey{kernel, (size_t)ctx, 0, 0}.hash();
    for (uint64_t i = 0; i < ENTRIES; ++i) {
      Entry& e = e_[(h + i) % ENTRIES];
      if (e.kernel == nullptr || (e.kernel == kernel && e.ctx == ctx)) return &e;
    }
    return nullptr;
  }

 public:
  // Calls set(bytes) unless as much was set for the kernel before in the context; bytes: the
  // most that was ever asked for. ctx 0: the context is not known (none is current yet), so
  // that every call sets it, and what was set so holds in a context that is known later.
  // Returns what set returned, or 0.
  template <typename SET>
  int raise(const void* kernel, unsigned long long ctx, size_t dyn, SET set) {
    std::lock_guard<std::mutex> lock(mu_);
    Entry* e = entry(kernel, ctx);
    if (e != nullptr && e->kernel != nullptr && ctx != 0 && e->dyn >= dyn) return 0;
    const Entry* u = entry(kernel, 0);
    if (e != nullptr && e->kernel != nullptr && e->dyn > dyn) dyn = e->dyn;
    if (u != nullptr && u->kernel != nullptr && u->dyn > dyn) dyn = u->dyn;
    const int err = set(dyn);
    if (err == 0 && e != nullptr) *e = {kernel, ctx, dyn};
    return err;
  }
};

}  // namespace moeperm
