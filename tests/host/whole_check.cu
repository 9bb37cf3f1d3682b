// whole_check.cu -- the decode call's walk where units are not divided: every
// unit of every sequence with keys is taken by one CTA, from its first block to
// its last.  Prints "ok <walks>", or the first mismatch and exits 1.
#include <stdio.h>
#include <stdlib.h>

#include <set>
#include <utility>
#include <vector>

#include "paged.cuh"

using namespace fa::paged;

static int check(const std::vector<int>& lens, int HU, int gpu) {
  const int B = (int)lens.size();
  Cache c{};
  c.page_size = 16;
  c.max_pages = 1 << 20;
  std::vector<int> prefix(B);
  int sum = 0, units = 0;
  for (int b = 0; b < B; ++b) {
    prefix[b] = sum += blocks_of(clamp_len(c, lens[b]));
    units += clamp_len(c, lens[b]) > 0 ? HU : 0;
  }
  const long long total = (long long)sum * HU;
  const int grid = (int)(gpu < total ? gpu : total);
  const Work k{&c, lens.data(), B, HU};
  std::set<std::pair<int, int>> seen;
  for (int cta = 0; cta < gpu; ++cta) {
    const int b0 = cta < grid ? sequence_of(prefix.data(), B, HU, share(total, grid, cta)) : 0;
    const int b1 = cta + 1 < grid ? sequence_of(prefix.data(), B, HU, share(total, grid, cta + 1)) : 0;
    Walk w = whole_units(k, start_walk(k, prefix.data(), b0, total, grid, cta),
                         start_walk(k, prefix.data(), b1, total, grid, cta + 1), grid, cta);
    while (w.at < w.end) {
      if (w.blk != 0 || w.nblk <= 0 || w.at + w.nblk > w.end || !seen.insert({w.b, w.hu}).second) {
        printf("MISMATCH cta %d of %d: sequence %d unit %d block %d of %d, at %lld, end %lld\n", cta, gpu, w.b, w.hu, w.blk,
               w.nblk, w.at, w.end);
        return 1;
      }
      w.at += w.nblk;
      w.blk = w.nblk;
      next_unit(k, w);
    }
  }
  if ((int)seen.size() != units) {
    printf("MISMATCH %d units of %d taken\n", (int)seen.size(), units);
    return 1;
  }
  return 0;
}

int main() {
  int walks = 0;
  for (int gpu : {1, 2, 5, 148})
    for (int HU : {1, 2, 3, 8, 24})
      for (int r = 0; r < 80; ++r) {
        std::vector<int> l(1 + rand() % 40);
        const int most = 1 << (rand() % 14);
        for (int& x : l) x = rand() % 4 ? rand() % most : 0;
        if (check(l, HU, gpu)) return 1;
        ++walks;
      }
  if (check({777}, 8, 148) || check({0, 0}, 4, 148) || check({1}, 1, 148)) return 1;
  printf("ok %d walks\n", walks + 3);
  return 0;
}
