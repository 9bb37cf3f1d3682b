// The decode kernel's walk (paged.cuh) over lengths that change while it reads them:
// whatever it then computes, it ends, and it names only sequences, head units and
// blocks that exist.
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "paged.cuh"

using namespace fa::paged;

static const int GUARD = 8;  // entries around the lengths that no walk may read

static int walk(std::vector<int>& room, int B, int HU, int grid_max, int whole, Cache& c) {
  int* lens = room.data() + GUARD;
  std::vector<int> prefix(B);
  int sum = 0;
  for (int b = 0; b < B; ++b) prefix[b] = sum += blocks_of(clamp_len(c, lens[b]));
  const long long total = (long long)sum * HU;
  const int grid = (int)(grid_max < total ? grid_max : total);
  const Work k{&c, lens, B, HU};
  auto change = [&] {
    for (int n = rand() % 3; n > 0; --n) lens[rand() % B] = rand() % 3 ? rand() % 3000 : 0;
  };
  for (int cta = 0; cta < grid; ++cta) {
    const int b0 = sequence_of(prefix.data(), B, HU, share(total, grid, cta));
    change();
    Walk w = start_walk(k, prefix.data(), b0, total, grid, cta);
    change();
    if (whole) {
      const int b1 = cta + 1 < grid ? sequence_of(prefix.data(), B, HU, share(total, grid, cta + 1)) : 0;
      w = whole_units(k, w, start_walk(k, prefix.data(), b1, total, grid, cta + 1), grid, cta);
    }
    long long steps = 0;
    while (at_hand(w)) {
      if (w.b < 0 || w.b >= B || w.hu < 0 || w.hu >= HU || w.blk < 0 || w.blk >= w.nblk ||
          (long long)(w.nblk - 1) * BLOCK >= (long long)c.max_pages * c.page_size) {
        printf("FAILED sequence %d of %d, unit %d of %d, block %d of %d\n", w.b, B, w.hu, HU, w.blk, w.nblk);
        return 1;
      }
      const long long rest = w.nblk - w.blk, room_left = w.end - w.at;
      const int n = (int)(rest < room_left ? rest : room_left);
      if (n <= 0 || ++steps > 1000000) {
        printf("FAILED a walk that does not end (%lld of %lld)\n", w.at, w.end);
        return 1;
      }
      const int first = owner(total, grid, w.at - w.blk), last = owner(total, grid, w.at - w.blk + w.nblk - 1);
      if (first < 0 || last < first || last >= grid) {
        printf("FAILED parts in CTAs %d to %d of %d\n", first, last, grid);
        return 1;
      }
      change();
      w.at += n;
      w.blk += n;
      if (w.blk == w.nblk) next_unit(k, w);
      if (w.b < 0 || w.b >= B) {
        printf("FAILED sequence %d of %d\n", w.b, B);
        return 1;
      }
    }
  }
  return 0;
}

int main() {
  srand(11);
  int walks = 0;
  for (int r = 0; r < 40000; ++r) {
    const int B = 1 + rand() % (r % 10 ? 6 : 50), HU = 1 + rand() % 9;
    Cache c{};
    c.page_size = 16;
    c.max_pages = r % 2 ? 200 : 32;
    std::vector<int> room(B + 2 * GUARD, 1 << 30);
    for (int b = 0; b < B; ++b) room[GUARD + b] = rand() % 4 ? rand() % 3000 : 0;
    if (walk(room, B, HU, 1 + rand() % 148, r % 2 == 0, c)) return 1;
    ++walks;
  }
  printf("ok %d walks\n", walks);
  return 0;
}
