// Walks, on the host, the functions that the paged-cache kernels find rows and
// divide work by (paged.cuh): every page index, good or bad, must end in a row
// of the pool or in -1; every block of every head unit must be walked by
// exactly one CTA; and the parts that a unit's CTAs leave must be the ones that
// its join reads, each slot used once.
#include <stdio.h>
#include <stdlib.h>

#include <limits>
#include <set>
#include <tuple>
#include <vector>

#include "paged.cuh"

using namespace fa::paged;

static int fail(const char* what, long long a, long long b) {
  printf("FAILED %s (%lld, %lld)\n", what, a, b);
  return 1;
}

static int check_rows() {
  const int lo = std::numeric_limits<int>::min(), hi = std::numeric_limits<int>::max();
  for (int page_size : {1, 7, 16, 128}) {
    const int pages = 37, width = 5;
    std::vector<int> table(2 * width, 3);
    Cache c{};
    c.row_stride = 256;
    c.head_stride = 256LL * page_size;
    c.page_stride = 4 * c.head_stride;
    c.num_pages = pages;
    c.page_size = page_size;
    c.table = table.data();
    c.max_pages = width;
    c.table_stride = width;
    const long long pool = pages * c.page_stride;
    for (int page : {lo, -1, 0, 1, pages - 1, pages, hi})
      for (int slot : {0, page_size - 1}) {
        const long long off = row_offset(c, page, slot);
        const bool good = page >= 0 && page < pages;
        if (good ? off < 0 || off + 3 * c.head_stride + 256 > pool : off != -1) return fail("row", page, slot);
      }
    for (long long pos : {-1LL, (long long)lo, 0LL, 1LL, (long long)width * page_size - 1, (long long)width * page_size,
                          (long long)hi, 3LL * hi}) {
      const bool in = pos >= 0 && pos < (long long)width * page_size;
      if (page_of(c, 1, pos) != (in ? 3 : -1)) return fail("page", pos, page_size);
    }
    for (int len : {lo, -1, 0, 1, width * page_size, width * page_size + 1, hi}) {
      const int n = clamp_len(c, len);
      if (n < 0 || n > width * page_size || (len >= 0 && len <= width * page_size && n != len)) return fail("len", len, n);
    }
  }
  // strides whose products pass 32 bits
  Cache c{};
  c.page_stride = 1 << 20;
  c.row_stride = 256;
  c.num_pages = 1 << 20;
  if (row_offset(c, (1 << 20) - 1, 15) != (((1LL << 20) - 1) << 20) + 15 * 256) return fail("wide", 0, 0);
  return 0;
}

static int check_walk(const std::vector<int>& lens, int HU, int gpu) {
  const int B = (int)lens.size();
  Cache c{};
  c.page_size = 16;
  c.max_pages = 1 << 20;
  std::vector<int> prefix(B);
  int sum = 0;
  for (int b = 0; b < B; ++b) prefix[b] = sum += blocks_of(clamp_len(c, lens[b]));
  const long long total = (long long)sum * HU;
  const int grid = (int)(gpu < total ? gpu : total);
  const Work k{&c, lens.data(), B, HU};
  std::set<std::tuple<int, int, int>> seen;
  std::vector<std::tuple<int, int>> slot_unit(2 * gpu, std::make_tuple(-1, -1));
  struct Join { int b, hu, first, n, cta; };
  std::vector<Join> joins;
  std::set<std::tuple<int, int>> open;
  for (int cta = 0; cta < gpu; ++cta) {
    const int b0 = cta < grid ? sequence_of(prefix.data(), B, HU, share(total, grid, cta)) : 0;
    Walk w = start_walk(k, prefix.data(), b0, total, grid, cta);
    const long long begin = w.at;
    int begun = 0;
    while (w.at < w.end) {
      const long long unit_begin = w.at - w.blk;
      const long long rest = w.nblk - w.blk, room = w.end - w.at;
      const int nseg = (int)(rest < room ? rest : room);
      if (nseg <= 0) return fail("empty segment", cta, w.at);
      for (int i = 0; i < nseg; ++i)
        if (!seen.insert(std::make_tuple(w.b, w.hu, w.blk + i)).second) return fail("block twice", cta, w.blk + i);
      if (nseg != w.nblk) {
        const int slot = part_slot(cta, begin, unit_begin);
        if (std::get<0>(slot_unit[slot]) >= 0) return fail("slot twice", cta, slot);
        slot_unit[slot] = std::make_tuple(w.b, w.hu);
        open.insert(std::make_tuple(w.b, w.hu));
        if (w.blk == 0) {
          if (begun++) return fail("two joins", cta, w.b);
          joins.push_back({w.b, w.hu, slot, owner(total, grid, unit_begin + w.nblk - 1) - cta + 1, cta});
        }
      }
      w.at += nseg;
      w.blk += nseg;
      if (w.blk == w.nblk) next_unit(k, w);
    }
  }
  if ((long long)seen.size() != total) return fail("blocks missed", (long long)seen.size(), total);
  size_t parts = 0;
  for (const Join& j : joins) {
    for (int i = 0; i < j.n; ++i) {
      const int slot = i ? 2 * (j.cta + i) : j.first;
      if (slot >= 2 * gpu || slot_unit[slot] != std::make_tuple(j.b, j.hu)) return fail("join", j.cta, slot);
      ++parts;
    }
    open.erase(std::make_tuple(j.b, j.hu));
  }
  if (!open.empty()) return fail("unit without a join", std::get<0>(*open.begin()), std::get<1>(*open.begin()));
  size_t left = 0;
  for (auto& u : slot_unit) left += std::get<0>(u) >= 0;
  if (left != parts) return fail("parts unread", (long long)left, (long long)parts);
  return 0;
}

int main() {
  if (check_rows()) return 1;
  int walks = 0;
  srand(1);
  const std::vector<std::vector<int>> fixed = {
      {0}, {1}, {128}, {129}, {777}, {0, 0, 1, 0}, {100000}, {1, 1, 1, 1, 1, 1}, {-3, 2147483647 / 8, 5}, {0, 0, 300, 0, 0}};
  for (int gpu : {1, 2, 5, 148})
    for (int HU : {1, 2, 3, 8, 24}) {
      for (const auto& l : fixed) {
        if (check_walk(l[0] < 0 ? std::vector<int>{-3, 16777, 5} : l, HU, gpu)) return 1;
        ++walks;
      }
      for (int r = 0; r < 60; ++r) {
        std::vector<int> l(1 + rand() % 40);
        const int most = 1 << (rand() % 14);
        for (int& x : l) x = rand() % 4 ? rand() % most : 0;
        if (check_walk(l, HU, gpu)) return 1;
        ++walks;
      }
    }
  printf("ok %d walks\n", walks);
  return 0;
}
