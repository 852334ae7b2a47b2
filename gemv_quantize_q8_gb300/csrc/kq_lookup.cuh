// kq_lookup.cuh -- host values that are looked up once and kept (internal; plain C++).
#pragma once
#include <atomic>

namespace kq {

// A value looked up once (zero: not yet).  Any thread may be the first to ask, several at once too: all find the same.
template <typename F>
inline int looked_up(std::atomic<int> &slot, F find) {
    int n = slot.load(std::memory_order_relaxed);
    if (!n) slot.store(n = find(), std::memory_order_relaxed);
    return n;
}

}  // namespace kq
