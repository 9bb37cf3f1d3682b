// Where the append kernel finds a position's row (paged.cuh): the page
// by the launch's division, then the row in the pool.  Any position must end in the
// row that the definition names or, where the table has none, in -1, with no read
// outside the table.
#include <limits.h>
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "paged.cuh"

using namespace fa::paged;

int main() {
  int checks = 0;
  srand(5);
  for (int page_size : {1, 2, 7, 16, 24, 64, 128, 1000, 1 << 20, INT_MAX})
    for (int width : {1, 2, 5, 333}) {
      if ((long long)page_size * width > (1ll << 30) && width > 1) continue;
      const Divider by_page = make_divider(page_size);
      const int pages = 50;
      // entries outside of the pool to both sides of the row
      std::vector<int> table(3 * width + 2, pages);
      for (int i = 0; i < width; ++i) table[width + 1 + i] = (i * 7 + 3) % pages;
      Cache c{};
      c.row_stride = 128;
      c.head_stride = 128;
      c.page_stride = 1 << 10;
      c.num_pages = pages;
      c.page_size = page_size;
      c.table = table.data() + 1;
      c.max_pages = width;
      c.table_stride = width;
      const long long cap = (long long)page_size * width;
      std::vector<long long> at = {INT_MIN, -1, 0, 1, page_size - 1, page_size, cap - 1, cap, cap + 1, INT_MAX, INT_MAX - 1};
      for (int i = 0; i < 50; ++i) at.push_back((long long)(rand() % 1000) * cap / 900);
      for (long long x : at) {
        if (x > INT_MAX) continue;
        const int pos = (int)x, i = by_page(pos);
        const bool in = pos >= 0 && pos < cap;
        const int page = page_of(c, c.table + width, pos, i);
        const int want = in ? table[width + 1 + pos / page_size] : -1;
        const long long off = row_offset(c, page, in ? pos - i * page_size : 0);
        if (page != want || page != page_of(c, 1, pos) || (off < 0) != !in ||
            (in && off != want * c.page_stride + pos % page_size * c.row_stride)) {
          printf("FAILED position %d of pages of %d, table of %d: %d, not %d\n", pos, page_size, width, page, want);
          return 1;
        }
        ++checks;
      }
    }
  printf("ok %d positions\n", checks);
  return 0;
}
