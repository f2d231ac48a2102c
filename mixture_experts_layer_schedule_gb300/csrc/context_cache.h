// context_cache.h -- values that belong to one CUDA context (a kernel's raised
// shared-memory limit, what an occupancy query said), kept by the context's id.
// No CUDA calls here.
#pragma once
#include <mutex>

namespace moe {

// The values of the last kSlots contexts. A process has one context per GPU;
// one that is destroyed and made again has a new id and so a new entry.
template <class V>
class ContextCache {
 public:
  // The current context's value in `out`: the one kept, or a new one from
  // make(V&). Where make returns false nothing is kept and the next call tries
  // again. id() is the unique id of the current context, or 0 if there is none
  // yet; make may bring it about, so it is asked again afterwards.
  template <class Id, class Make>
  bool get(Id&& id, Make&& make, V& out) {
    std::lock_guard<std::mutex> lock(mu_);
    if (find(id(), out)) return true;
    V v{};
    if (!make(v)) return false;
    const unsigned long long now = id();
    V kept;
    if (now != 0 && !find(now, kept)) {
      at_[next_] = Entry{now, v};
      next_ = (next_ + 1) % kSlots;
    }
    out = v;
    return true;
  }

  static constexpr int kSlots = 16;

 private:
  struct Entry {
    unsigned long long id;
    V v;
  };
  bool find(unsigned long long id, V& out) const {
    if (id == 0) return false;
    for (const Entry& e : at_)
      if (e.id == id) {
        out = e.v;
        return true;
      }
    return false;
  }
  std::mutex mu_;
  Entry at_[kSlots] = {};
  int next_ = 0;
};

}  // namespace moe
