// Answers of a device that are asked for once and kept: how many clusters of n CTAs of a kernel it runs at one time.
#pragma once

#include <atomic>

namespace msa {

// Shared by all host threads: two that ask at one time keep the same answer.
class AtOnce {
 public:
  static constexpr int kDevices = 64, kSizes = 9;
  // ask(): the answer, 0 where no such cluster fits, negative where the question failed. A failure is not kept: the next
  // call asks again.
  template <typename Ask>
  int get(int dev, int n, Ask ask) {
    const bool known = dev >= 0 && dev < kDevices && n >= 0 && n < kSizes;
    if (known) {
      const int v = of_[dev][n].load();
      if (v > 0) return v - 1;
    }
    const int v = ask();
    if (known && v >= 0) of_[dev][n].store(v + 1);
    return v;
  }

 private:
  std::atomic<int> of_[kDevices][kSizes] = {};           // the answer + 1; 0: not asked
};

// The cheapest number of CTAs (or pairs) from 1 to `most` that share a tile's K, and its cost. room(s): clusters at one time, below 1 where
// s is not to be had; cost(s, room); `forced`: that one, if it is to be had. 0: none is.
template <typename Room, typename Cost>
int cheapest_split(int most, int forced, bool later_of_equals, Room room, Cost cost, float& us) {
  if (forced >= 1 && forced <= most) {
    const int r = room(forced);
    if (r >= 1) {
      us = cost(forced, r);
      return forced;
    }
  }
  int split = 0;
  for (int s = 1; s <= most; ++s) {
    const int r = room(s);
    if (r < 1) continue;
    const float t = cost(s, r);
    if (split == 0 || t < us || (later_of_equals && t == us)) {
      split = s;
      us = t;
    }
  }
  return split;
}

}  // namespace msa
