// Which give-ups of bounded device waits callers have not been told of yet. A wait that gives up writes the
// time into its kernel's word, which nothing clears: what is written while a caller reads differs from
// what it has read, and is told of by the next call.
#pragma once
#include <stdint.h>

#include <array>
#include <map>
#include <mutex>

namespace s1 {

template <int N>
class GiveUps {
 public:
  // read(words) reads the device's words and returns 0, or an error that is passed on (nothing is told of
  // then). *any: they differ from what the calls before told of. One caller reads at a time, so that words read
  // earlier never come in after newer ones.
  template <typename Read>
  int news(int device, Read&& read, bool* any) {
    std::lock_guard<std::mutex> lk(mu_);
    std::array<uint64_t, N> now{};
    if (const int e = read(now.data())) return e;
    std::array<uint64_t, N>& told = told_[device];     // (zeros at first, as the device's words)
    *any = now != told;
    told = now;
    return 0;
  }

 private:
  std::mutex mu_;
  std::map<int, std::array<uint64_t, N>> told_;
};

}  // namespace s1
