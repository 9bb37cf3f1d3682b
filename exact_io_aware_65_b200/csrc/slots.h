// slots.h -- slots that are lent one at a time, each to one owner until it gives
// it back.
#pragma once

#include <stdint.h>

#include <atomic>

namespace fa {

// N slots (a multiple of 64), a bit each; free of locks, and without a destructor,
// since owners may give back while the process ends.
template <uint32_t N>
class OwnedSlots {
  static_assert(N % 64 == 0, "whole words of bits");
  std::atomic<uint64_t> used_[N / 64];
  std::atomic<uint32_t> last_;  // word of the slot lent last: the search starts there

 public:
  // A slot that nobody has; -1 if all are lent.
  int take() {
    const uint32_t first = last_.load(std::memory_order_relaxed);
    for (uint32_t i = 0; i < N / 64; ++i) {
      const uint32_t w = (first + i) % (N / 64);
      uint64_t u = used_[w].load(std::memory_order_relaxed);
      while (~u != 0) {
        const int bit = __builtin_ctzll(~u);
        if (used_[w].compare_exchange_weak(u, u | 1ull << bit, std::memory_order_acquire, std::memory_order_relaxed)) {
          last_.store(w, std::memory_order_relaxed);
          return (int)(w * 64 + (uint32_t)bit);
        }
      }
    }
    return -1;
  }
  void give(int slot) { used_[slot / 64].fetch_and(~(1ull << (slot % 64)), std::memory_order_release); }
};

}  // namespace fa
