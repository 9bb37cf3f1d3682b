// pack_check.cu -- the packed attention's schedules, walked on the host: every
// (head, query tile) is in one forward item and every (key head, part, key tile)
// one backward item; with the masks as the kernels apply them, a tile visit at
// a time, a query row meets exactly the keys that the rule j <= i + Lk - Lq (or
// no mask) shows it; tile slots are distinct and inside the workspace, and so
// are the rows that tiles read and write, for any cu.
//
// Usage: pack_check -> prints "ok <cases>" and exits 0, or the first mismatch and 1.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <set>
#include <vector>

#include "bwd_sched.cuh"
#include "fwd_sched.cuh"

namespace {

int g_fail = 0;
void fail(const char* what, int a, int b, int c, int d) {
  if (g_fail++ == 0) printf("MISMATCH %s at (%d, %d, %d, %d)\n", what, a, b, c, d);
}
unsigned g_rng = 1;
int rnd(int n) {
  g_rng = g_rng * 1664525u + 1013904223u;
  return (int)((g_rng >> 8) % (unsigned)n);
}

using fa::Pack;
using fa::PACKED;

// the kernels' element masks, in the tiles' rows
bool shown(int causal, int i_tile, int j_tile, int off, int r, int c, int Lk) {
  if (j_tile == 0 && c < fa::pack::pad(Lk)) return false;
  return !(causal && j_tile == i_tile + off) || c <= r;
}

void check(const Pack& k, int d, int kind, int parts) {
  namespace P = fa::pack;
  fa::fwd::PackedParams f = {};
  f.pk = k;
  f.d = d;
  f.mask_kind = kind;
  f.tiles_per_item = d == 64 ? 1 : 2;
  f.by_heads = d == 128 && k.G % 2 == 0;
  f.parts = 1;
  fa::bwd::PackedParams w = {};
  w.pk = k;
  w.d = d;
  w.mask_kind = kind;
  w.parts = parts;
  std::set<long long> used;
  long long f_items = 0, w_items = 0;
  for (int b = 0; b < k.B; ++b) {
    const P::Seq s = P::seq_at(k, b);
    if (s.sq < 0 || s.Lq < 0 || s.sq + s.Lq > k.Tq || s.sk < 0 || s.Lk < 0 || s.sk + s.Lk > k.Tk) fail("rows", b, s.sq, s.Lq, s.Lk);
    const int nq = P::tiles(s.Lq), nk = P::tiles(s.Lk), pq = P::pad(s.Lq), pk = P::pad(s.Lk);
    for (int i = 0; i < nq; ++i) {
      const long long slot = P::slot_base(s.sq, b) + i;
      if (slot < 0 || slot >= P::slots(k.Tq, k.B) || !used.insert(slot).second) fail("slot", b, i, (int)slot, 0);
    }
    // ---- forward: visits of each (head, query tile)
    std::vector<int> seen((size_t)k.Hq * nq, 0);
    const P::Units u = fa::fwd::packed_units(f, s);
    f_items += (long long)u.tiles * u.heads;
    int last = 1 << 30;
    for (int r = 0; r < u.tiles * u.heads; ++r) {
      const P::Place at = P::place_of(u, r);
      const fa::fwd::Item it = fa::fwd::packed_item(f, s, at);
      const int e = fa::fwd::kv_end<PACKED>(f, it);
      if (u.group >= u.heads && e > last) fail("order", b, r, e, last);  // longest first within a group
      last = e;
      for (int t = 0; t < (it.has1 ? 2 : 1); ++t) {
        const int q = t ? it.q1 : it.q0, h = t ? it.h1 : it.h0;
        if (q < 0 || q >= nq || h < 0 || h >= k.Hq || h / k.G != it.h0 / k.G) {
          fail("tile", b, r, q, h);
          continue;
        }
        if (seen[(size_t)h * nq + q]++) fail("tile twice", b, r, q, h);
        if (h % std::max(1, k.Hq / 2)) continue;  // the masks do not depend on the head
        for (int j = 0; j < nk; ++j) {
          const bool member = j < e && fa::fwd::member<PACKED>(f, it, q, j);
          for (int x = 0; x < 128; x += (x < 3 || x > 124) ? 1 : 7)
            for (int c = 0; c < 128; c += (c < 3 || c > 124) ? 1 : 5) {
              const int i = q * 128 + x - pq, key = j * 128 + c - pk;
              if (i < 0) continue;  // a row before the sequence: not written
              const bool want = key >= 0 && (kind == FA_MASK_NONE || key <= i + s.Lk - s.Lq);
              if ((member && shown(kind == FA_MASK_CAUSAL, q, j, it.off, x, c, s.Lk)) != want) fail("fwd mask", b, i, key, nk);
            }
        }
      }
    }
    for (int x : seen)
      if (x != 1) fail("tile missed", b, x, 0, 0);
    // ---- forward with divided keys: an item's parts cover its key tiles once,
    // and the join counts the parts that the items have
    fa::fwd::PackedParams g = f;
    g.parts = 1 + rnd(6);
    std::vector<int> visits((size_t)k.Hq * nq * std::max(nk, 1), 0), parts_seen((size_t)k.Hq * nq, 0);
    const P::Units ug = fa::fwd::packed_units(g, s);
    for (int r = 0; r < ug.tiles * ug.heads; ++r) {
      fa::fwd::Item it = fa::fwd::packed_item(g, s, P::place_of(ug, r));
      fa::fwd::take_part(g, it);
      if (it.part >= it.parts) {
        if (it.j0 < it.j1) fail("part past the parts", b, r, it.part, it.parts);
        continue;
      }
      for (int t = 0; t < (it.has1 ? 2 : 1); ++t) {
        const int q = t ? it.q1 : it.q0, h = t ? it.h1 : it.h0;
        parts_seen[(size_t)h * nq + q]++;
        for (int j = fa::fwd::kv_begin<fa::SPLIT>(it); j < fa::fwd::kv_end<fa::SPLIT>(g, it); ++j) {
          if (j >= nk) fail("part's key tile", b, r, j, nk);
          else visits[((size_t)h * nq + q) * nk + j]++;
        }
      }
    }
    for (int h = 0; h < k.Hq; ++h)
      for (int q = 0; q < nq; ++q) {
        const int e = fa::fwd::packed_end(g, nk, nk - nq, fa::fwd::last_tile(g, nq, q));
        if (parts_seen[(size_t)h * nq + q] != fa::fwd::parts_of(g, e)) fail("parts", b, h, q, parts_seen[(size_t)h * nq + q]);
        for (int j = 0; j < nk; ++j)
          if (visits[((size_t)h * nq + q) * nk + j] != (j < e)) fail("divided keys", b, h, q, j);
      }
    // ---- backward
    std::vector<int> done((size_t)k.Hkv * parts * nk, 0), pairs((size_t)k.Hq * nq * nk, 0);
    const P::Units v = fa::bwd::packed_units(w, s);
    w_items += (long long)v.tiles * v.heads;
    for (int r = 0; r < v.tiles * v.heads; ++r) {
      const fa::bwd::Item it = fa::bwd::packed_item(w, s, b, P::place_of(v, r));
      if (it.j < 0 || it.j >= nk || it.hk < 0 || it.hk >= k.Hkv || it.part < 0 || it.part >= parts) {
        fail("key tile", b, r, it.j, it.hk);
        continue;
      }
      done[((size_t)it.hk * parts + it.part) * nk + it.j]++;
      using fa::bwd::Step;
      for (Step q = fa::bwd::first_step<PACKED>(w, it); fa::bwd::more<PACKED>(w, it, q); q = fa::bwd::next_step<PACKED>(w, it, q)) {
        const int h = it.hk * k.G + q.g;
        if (q.i < 0 || q.i >= nq || h >= k.Hq || q.g >= k.G) {
          fail("step", b, r, q.i, h);
          break;
        }
        pairs[((size_t)h * nq + q.i) * nk + it.j]++;
      }
    }
    for (int x : done)
      if (x != 1) fail("key tile count", b, x, 0, 0);
    for (int h = 0; h < k.Hq; ++h)
      for (int i = 0; i < nq; ++i)
        for (int j = 0; j < nk; ++j) {
          const int off = nk - nq;
          const int need = kind == FA_MASK_NONE || j <= i + off;  // some pair of the tiles can be seen
          if (pairs[((size_t)h * nq + i) * nk + j] != need) fail("bwd pair", b, h, i, j);
          if (need && h == 0)
            for (int x = 0; x < 128; x += (x < 3 || x > 124) ? 1 : 7)
              for (int c = 0; c < 128; c += (c < 3 || c > 124) ? 1 : 5) {
                const int row = i * 128 + x - pq, key = j * 128 + c - pk;
                if (row < 0) continue;  // its P is zero by its LSE
                const bool want = key >= 0 && (kind == FA_MASK_NONE || key <= row + s.Lk - s.Lq);
                if (shown(kind == FA_MASK_CAUSAL, i, j, off, x, c, s.Lk) != want) fail("bwd mask", b, row, key, nk);
              }
        }
  }
  const long long per = f.by_heads ? k.Hq / 2 : k.Hq;
  if (f_items > P::slots(k.Tq, k.B) * per) fail("forward items", (int)f_items, 0, 0, 0);
  if (w_items > P::slots(k.Tk, k.B) * k.Hkv * parts) fail("backward items", (int)w_items, 0, 0, 0);
}

}  // namespace

int main() {
  static const int lens[] = {0, 1, 2, 63, 64, 127, 128, 129, 200, 255, 256, 257, 300, 500};
  static const int heads[][2] = {{1, 1}, {4, 4}, {8, 2}, {6, 2}, {5, 1}, {16, 1}, {10, 2}};
  int cases = 0;
  for (int n = 0; n < 30; ++n) {  // long enough to be divided
    std::vector<int> cq(1, 0), ck(1, 0);
    cq.push_back(1 + rnd(3000));
    ck.push_back(1 + rnd(6000));
    const int* h = heads[rnd(7)];
    Pack k{cq.data(), ck.data(), 1, cq.back(), ck.back(), h[0], h[1], h[0] / h[1]};
    check(k, rnd(2) ? 64 : 128, rnd(2) ? FA_MASK_CAUSAL : FA_MASK_NONE, 1 + rnd(k.G));
    ++cases;
  }
  for (int n = 0; n < 400; ++n) {
    const int B = 1 + rnd(5);
    std::vector<int> cq(1, rnd(2) ? rnd(200) : 0), ck(1, rnd(2) ? rnd(200) : 0);
    for (int b = 0; b < B; ++b) {
      cq.push_back(cq.back() + lens[rnd(14)]);
      ck.push_back(ck.back() + (rnd(3) ? cq[b + 1] - cq[b] + rnd(200) : lens[rnd(14)]));
    }
    const int* h = heads[rnd(7)];
    Pack k{cq.data(), ck.data(), B, cq.back() + rnd(3), ck.back() + rnd(3), h[0], h[1], h[0] / h[1]};
    check(k, rnd(2) ? 64 : 128, rnd(2) ? FA_MASK_CAUSAL : FA_MASK_NONE, 1 + rnd(k.G));
    ++cases;
  }
  // the places of a sequence's items, at every size of the heads' groups
  for (int tiles = 1; tiles <= 4; ++tiles)
    for (int heads = 1; heads <= 7; ++heads)
      for (int group = 1; group <= heads; ++group) {
        const fa::pack::Units u{tiles, heads, group};
        std::set<int> at;
        for (int r = 0; r < tiles * heads; ++r) {
          const fa::pack::Place x = fa::pack::place_of(u, r);
          if (x.tile < 0 || x.tile >= tiles || x.head < 0 || x.head >= heads || !at.insert(x.tile * 8 + x.head).second)
            fail("place", tiles, heads, group, r);
        }
        ++cases;
      }
  // any cu at all: rows, tiles and slots stay inside (slots may then be shared)
  for (int n = 0; n < 2000; ++n) {
    const int B = 1 + rnd(4);
    std::vector<int> cq, ck;
    for (int b = 0; b <= B; ++b) {
      cq.push_back(rnd(8) ? rnd(3000) - 500 : (rnd(2) ? 0x7fffffff : (int)0x80000000));
      ck.push_back(rnd(8) ? rnd(3000) - 500 : (rnd(2) ? 0x7fffffff : (int)0x80000000));
    }
    const Pack k{cq.data(), ck.data(), B, rnd(2000), rnd(2000), 4, 2, 2};
    for (int b = 0; b < B; ++b) {
      const fa::pack::Seq s = fa::pack::seq_at(k, b);
      if (s.sq < 0 || s.Lq < 0 || s.sq + s.Lq > k.Tq || s.sk < 0 || s.Lk < 0 || s.sk + s.Lk > k.Tk) fail("any cu: rows", b, s.sq, s.Lq, 0);
      if (s.Lq > 0 && fa::pack::slot_base(s.sq, b) + fa::pack::tiles(s.Lq) > fa::pack::slots(k.Tq, k.B))
        fail("any cu: slots", b, s.sq, s.Lq, k.Tq);
    }
    ++cases;
  }
  if (g_fail) return 1;
  printf("ok %d\n", cases);
  return 0;
}
