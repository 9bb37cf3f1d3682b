// The counter of a divided unit's parts (paged.cuh) on the host, with threads as
// the CTAs: over any contents of the word, n parts must get the numbers 0 .. n - 1,
// each once, and the last one alone the number n - 1; and the word that it leaves
// must serve the next call.
#include <stdio.h>
#include <stdlib.h>

#include <atomic>
#include <thread>
#include <vector>

#include "paged.cuh"

using namespace fa::paged;

struct Word {
  std::atomic<unsigned long long>* p;
  unsigned long long add(unsigned long long n) { return p->fetch_add(n); }
  unsigned long long cas(unsigned long long expected, unsigned long long desired) {
    p->compare_exchange_strong(expected, desired);
    return expected;
  }
};

// A word that another part's operation reaches first, on each of the first operations.
struct Crossed {
  unsigned long long word, tag;
  int others;  // parts that come in between, each by its own first addition and no more
  void other() {
    if (others > 0) {
      --others;
      ++word;
    }
  }
  unsigned long long add(unsigned long long n) {
    const unsigned long long was = word;
    word += n;
    other();
    return was;
  }
  unsigned long long cas(unsigned long long expected, unsigned long long desired) {
    const unsigned long long was = word;
    if (word == expected) word = desired;
    other();
    return was;
  }
};

static int run(unsigned long long start, unsigned long long tag, int n, int calls) {
  std::atomic<unsigned long long> word{start};
  for (int call = 0; call < calls; ++call) {
    std::vector<int> got(n, -1);
    std::atomic<int> go{0};
    std::vector<std::thread> parts;
    for (int i = 0; i < n; ++i)
      parts.emplace_back([&, i] {
        go.fetch_add(1);
        while (go.load() < n) {
        }
        Word w{&word};
        got[i] = count_part(w, tag);
        if (got[i] == n - 1) word.store(tag);
      });
    for (auto& t : parts) t.join();
    std::vector<int> seen(n, 0);
    for (int x : got) {
      if (x < 0 || x >= n || seen[x]++) {
        printf("FAILED number %d of %d parts over %llx (tag %llx)\n", x, n, start, tag);
        return 1;
      }
    }
    if (word.load() != tag) {
      printf("FAILED %llx left over %llx\n", word.load(), start);
      return 1;
    }
  }
  return 0;
}

int main() {
  const unsigned long long tags[] = {0x123456789abcde00ull, 0x0ull, 0xffffffffffffff00ull, 0x8000000000000100ull};
  int runs = 0;
  srand(3);
  for (unsigned long long tag : tags) {
    std::vector<unsigned long long> words = {tag, tag - 1, tag - 2, tag - 7, tag + 256, tag ^ (1ull << 63), ~tag};
    for (unsigned long long w : {0ull, ~0ull, 0x0101010101010101ull, 0x7f7f7f7f7f7f7f7full, 0xffffffffffffff00ull})
      if (((w ^ tag) >> COUNT_BITS) != 0 || w == tag) words.push_back(w);
    for (int i = 0; i < 20; ++i) words.push_back((unsigned long long)rand() << 33 | (unsigned long long)rand());
    for (unsigned long long w : words)
      for (int n : {1, 2, 3, 7, 16}) {
        if (((w ^ tag) >> COUNT_BITS) == 0 && w != tag) continue;  // the chance that paged.cuh names
        if (run(w, tag, n, 3)) return 1;
        ++runs;
      }
    // the most parts, in an order that makes every replacement fail at first
    for (int others : {0, 1, 2, 158}) {
      Crossed w{tag ^ 0x5500, tag, others};
      if (count_part(w, tag) != 0 || w.word < tag + 1) {
        printf("FAILED crossed by %d\n", others);
        return 1;
      }
      ++runs;
    }
  }
  if (run(0xdeadbeefull, tags[0], 160, 2)) return 1;
  printf("ok %d runs\n", runs + 1);
  return 0;
}
