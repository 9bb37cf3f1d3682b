// OwnedSlots (slots.h) on the host: no slot has two owners, whatever the threads
// do; with all lent there is none; what was given back is lent again.
#include <stdio.h>

#include <atomic>
#include <set>
#include <thread>
#include <vector>

#include "slots.h"

static fa::OwnedSlots<128> few;
static fa::OwnedSlots<65536> many;
static std::atomic<int> owners[128];

static int fail(const char* what, int a) {
  printf("FAILED %s (%d)\n", what, a);
  return 1;
}

int main() {
  for (int round = 0; round < 3; ++round) {
    std::set<int> got;
    for (int i = 0; i < 128; ++i) {
      const int s = few.take();
      if (s < 0 || s >= 128 || !got.insert(s).second) return fail("lent twice", s);
    }
    if (few.take() != -1) return fail("more than there are", round);
    for (int s : {127, 0, 64, 63}) few.give(s);
    std::set<int> again;
    for (int i = 0; i < 4; ++i) again.insert(few.take());
    if (again != std::set<int>{0, 63, 64, 127}) return fail("given back", (int)again.size());
    if (few.take() != -1) return fail("more than there are", round);
    for (int s = 0; s < 128; ++s) few.give(s);
  }
  std::atomic<int> bad{0};
  std::vector<std::thread> t;
  for (int k = 0; k < 8; ++k)
    t.emplace_back([&, k] {
      std::vector<int> mine;
      unsigned r = 12345u + (unsigned)k;
      for (int i = 0; i < 200000; ++i) {
        r = r * 1664525u + 1013904223u;
        if (mine.size() < 20 && (r >> 20 & 1u)) {
          const int s = few.take();
          if (s < 0) continue;
          if (owners[s].fetch_add(1) != 0) ++bad;
          mine.push_back(s);
        } else if (!mine.empty()) {
          const size_t at = r % mine.size();
          const int s = mine[at];
          mine[at] = mine.back();
          mine.pop_back();
          owners[s].fetch_sub(1);
          few.give(s);
        }
      }
      for (int s : mine) {
        owners[s].fetch_sub(1);
        few.give(s);
      }
    });
  for (auto& x : t) x.join();
  if (bad) return fail("two owners", bad);
  for (int i = 0; i < 128; ++i)
    if (few.take() < 0) return fail("lost", i);
  std::vector<bool> seen(65536, false);
  for (int i = 0; i < 65536; ++i) {
    const int s = many.take();
    if (s < 0 || seen[s]) return fail("of many", s);
    seen[s] = true;
  }
  if (many.take() != -1) return fail("of many, more", 0);
  printf("ok\n");
  return 0;
}
