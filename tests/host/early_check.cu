// Rows that idle SMs move during the selections of an eviction (early_most of
// paged.cuh): never more than the last rows that stay in any case, and no SM has more
// than a few heads' rows to wait for, however few SMs are idle.
#include <stdio.h>

#include "paged.cuh"

using namespace fa::paged;

int main() {
  int some = 0;
  for (int sms : {1, 2, 84, 148, 160})
    for (int heads = 1; heads <= 2 * sms; ++heads)
      for (int recent : {0, 1, 64, 256, 5000, 1 << 30})
        for (int width : {64, 128, 256}) {
          const int idle = sms - heads, early = early_most(heads, idle, recent, width);
          if (early < 0 || early > recent || (idle <= 0 && early != 0)) {
            printf("FAILED %d rows for %d heads on %d SMs, %d recent\n", early, heads, sms, recent);
            return 1;
          }
          if (early == 0) continue;
          ++some;
          const int per = SEL_THREADS / (width / 16) * SEL_ROWS;
          const long long units = (long long)heads * ((early + per - 1) / per);
          const long long each = (units + idle - 1) / idle;
          if (each > 3) {
            printf("FAILED %lld heads' rows for each of %d idle SMs (%d heads, %d rows each)\n", each, idle, heads, early);
            return 1;
          }
        }
  printf("ok %d\n", some);
  return some > 0 ? 0 : 1;
}
