// Places that are taken for as long as somebody needs them.
#pragma once

#include <cstdint>
#include <mutex>

namespace slope {

// N places, taken in turn: one that is given back is the last to be taken again.  (Nothing is destroyed at the process's end,
// when places may still be given back.)
template <uint32_t N>
class SlotPool {
  static_assert(N % 64 == 0, "whole words");

 public:
  // A free place; N if there is none.
  uint32_t take() {
    const std::lock_guard<std::mutex> lock(mutex_);
    for (uint32_t i = 0; i <= N / 64; ++i) {  // (the first word twice: its places before next_ come last)
      const uint32_t word = (next_ / 64 + i) % (N / 64);
      uint64_t free = ~taken_[word];
      if (i == 0) free &= ~uint64_t(0) << (next_ % 64);
      if (free == 0) continue;
      const uint32_t k = word * 64 + static_cast<uint32_t>(__builtin_ctzll(free));
      taken_[word] |= uint64_t(1) << (k % 64);
      next_ = (k + 1) % N;
      return k;
    }
    return N;
  }
  void give_back(uint32_t k) {
    const std::lock_guard<std::mutex> lock(mutex_);
    taken_[k / 64] &= ~(uint64_t(1) << (k % 64));
  }

 private:
  std::mutex mutex_;
  uint64_t taken_[N / 64] = {};
  uint32_t next_ = 0;
};

}  // namespace slope
