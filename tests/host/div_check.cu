// div_check.cu -- Divider (paged.cuh) against the language's division, at the
// ends of every quotient and over random operands.  Prints "ok", or the first
// mismatch and exits 1.
#include <stdio.h>
#include <stdlib.h>

#include "paged.cuh"

static int check(int n, int d) {
  if (fa::paged::make_divider(d)(n) == n / d) return 0;
  printf("MISMATCH %d / %d\n", n, d);
  return 1;
}

int main() {
  const int top = 0x7fffffff;
  for (int i = 1; i < 3000; ++i) {
    const int d = i < 1500 ? i : i < 2900 ? 1 + (int)(((unsigned)rand() * 32771u + rand()) % (1u << 30)) : (1 << 30) - (2999 - i);
    for (int k = 0; k < 2000; ++k) {
      const int q = k < 1000 ? k : (int)(((long long)rand() * top / RAND_MAX) / d);
      for (int n = -1; n <= 1; ++n) {
        const long long x = (long long)q * d + n;
        if (x >= 0 && x <= top && check((int)x, d)) return 1;
      }
    }
    if (check(top, d) || check(0, d)) return 1;
  }
  printf("ok\n");
  return 0;
}
