// pack.cuh -- packed sequences as the attention kernels see them: where the
// tiles of a sequence lie, and the order of the work.  The functions are
// host-callable too (the warp's search apart), so that a host test can walk the
// schedule of any batch.
//
// Tiles are counted back from a sequence's END: row r of L rows is row
// r + pad(L) of its ceil(L / 128) tiles, so the rows that a tile lacks stand
// before the sequence's first.  A tensor map with one dimension that starts at
// the sequence's first row (its stride the row's, like the next dimension's)
// then reads a tile at y = 128 tile - pad, and what lies before row 0 of the
// sequence is out of bounds and reads as zeros: no row of another sequence, or
// behind the last, is ever read, whatever it holds.  A causal mask aligned at
// the last query and key crosses such tiles on their diagonals only.
#pragma once

#include <stdint.h>

#include "fa.h"
#include "sm100.cuh"

namespace fa {

// Instantiations of the attention kernels: one length for all sequences,
// padded storage with a length each, packed rows, and (forward) packed rows whose
// keys are divided into parts.
enum : int { FIXED = 0, PADDED = 1, PACKED = 2, SPLIT = 3 };

struct Pack {
  const int* cu_q;  // [B + 1] first rows of the sequences
  const int* cu_k;
  int B, Tq, Tk;    // sequences, rows of the query and key tensors
  int Hq, Hkv, G;   // heads, and query heads of a key head
};

namespace pack {

// A sequence's rows, held to the tensors whatever cu says.
struct Seq {
  int sq, Lq, sk, Lk;
};
__host__ __device__ __forceinline__ Seq seq_at(const Pack& k, int b) {
  Seq s;
  s.sq = min(max(ld_ro(k.cu_q + b), 0), k.Tq);
  s.Lq = min(max(ld_ro(k.cu_q + b + 1), s.sq), k.Tq) - s.sq;
  s.sk = min(max(ld_ro(k.cu_k + b), 0), k.Tk);
  s.Lk = min(max(ld_ro(k.cu_k + b + 1), s.sk), k.Tk) - s.sk;
  return s;
}
__host__ __device__ __forceinline__ int tiles(int L) { return (L + 127) >> 7; }
__host__ __device__ __forceinline__ int pad(int L) { return -L & 127; }

// Tile slots: query tile i of sequence b owns slot slot_base(b) + i of the
// backward's workspace.  The tiles before b number at most sq / 128 + b, so the
// slots of different sequences differ, without a sum over the lengths.
__host__ __device__ __forceinline__ int slot_base(int sq, int b) { return (sq >> 7) + b; }
__host__ __device__ __forceinline__ long long slots(int T, int B) { return (long long)(T >> 7) + B; }

// The sequence that owns a slot: the last b with slot_base <= slot (a warp looks
// at 32 sequences at a time), -1 if none.  Warp-collective.
__device__ __forceinline__ int sequence_of_slot(const Pack& k, int slot) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = k.B;
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    bool le = false;
    if (i < lo + n) le = slot_base(min(max(__ldg(k.cu_q + i), 0), k.Tq), i) <= slot;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    if (m == 0) break;
    const int last = 31 - __clz(m);
    const int end = min(lo + n, lo + (last + 1) * step);
    lo += last * step + 1;
    n = end - lo;
  }
  return lo - 1;
}

// A slot's query rows and tile (-1: no tile uses the slot).  Warp-collective.
struct Slot {
  int sq, Lq, tile;
};
__device__ __forceinline__ Slot find_slot(const Pack& k, int slot) {
  Slot s{0, 0, -1};
  int b;
  if (k.B <= 32) {  // a lane a sequence: no load waits for another
    const int lane = threadIdx.x & 31;
    const int from = min(max(__ldg(k.cu_q + min(lane, k.B)), 0), k.Tq);
    const int to = min(max(__ldg(k.cu_q + min(lane + 1, k.B)), from), k.Tq);
    const unsigned m = __ballot_sync(0xffffffffu, lane < k.B && slot_base(from, lane) <= slot);
    b = 31 - __clz(m);
    s.sq = __shfl_sync(0xffffffffu, from, max(b, 0));
    s.Lq = __shfl_sync(0xffffffffu, to, max(b, 0)) - s.sq;
  } else {
    b = sequence_of_slot(k, slot);
    if (b >= 0) {
      const Seq x = seq_at(k, b);
      s.sq = x.sq;
      s.Lq = x.Lq;
    }
  }
  if (b >= 0 && slot - slot_base(s.sq, b) < tiles(s.Lq)) s.tile = slot - slot_base(s.sq, b);
  return s;
}

// Work items.  A sequence's items are `tiles` x `heads` (tiles of queries or of
// pairs of them, or of keys; heads, pairs of them, or key heads): heads in
// groups of `group`, so that what a group's items share stays in L2, and within
// a group tile by tile.
struct Units {
  int tiles, heads, group;
};
struct Place {
  int tile, head;
};
__host__ __device__ __forceinline__ Place place_of(const Units& u, int r) {
  const int per_group = u.group * u.tiles;
  const int g = r / per_group, rr = r % per_group;
  const int gsize = min(u.group, u.heads - g * u.group);
  return Place{rr / gsize, g * u.group + rr % gsize};
}

// The order of the sequences: 32 at a time, the longest of each 32 first, so
// that the items claimed last are short ones.  Warp-collective; lane L keeps
// the sequence of rank L.  Claims only grow, so the walk never turns back.
struct Walker {
  int chunk = -32;  // first sequence of the 32 at hand
  int base = 0;     // items before them
  int seq = -1;     // this lane's sequence,
  int from = 0;     // the chunk's items of the ranks before it,
  int upto = 0;     // and with its own (lane 31: all)
};

// UnitsOf: (Seq) -> Units; Weight: (Seq) -> the length they are ranked by; most:
// the items that the launch's sizes allow (a cu that is not ascending could
// describe more, which are not done).
template <typename UnitsOf, typename Weight>
__device__ __forceinline__ void next_chunk(const Pack& k, Walker& w, int most, UnitsOf units_of, Weight weight) {
  const int lane = threadIdx.x & 31;
  w.base += __shfl_sync(0xffffffffu, w.upto, 31);
  w.chunk += 32;
  const int b = w.chunk + lane;
  int items = 0, wt = -1;
  if (b < k.B) {
    const Seq s = seq_at(k, b);
    const Units u = units_of(s);
    items = u.tiles * u.heads;
    wt = weight(s);
  }
  const int n = min(32, k.B - w.chunk);
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const int o = __shfl_sync(0xffffffffu, wt, i);
    rank += o > wt || (o == wt && i < lane);
  }
  w.seq = -1;
  int mine = 0;
  for (int i = 0; i < n; ++i) {
    const int r = __shfl_sync(0xffffffffu, rank, i), x = __shfl_sync(0xffffffffu, items, i);
    if (r == lane) {
      w.seq = w.chunk + i;
      mine = x;
    }
  }
  long long sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  w.upto = (int)min(sum, (long long)(most - w.base));
  w.from = (int)min(sum - mine, (long long)(most - w.base));
}

// The sequence and place of item idx; false past the last.
template <typename UnitsOf, typename Weight>
__device__ __forceinline__ bool locate(const Pack& k, Walker& w, int idx, int most, UnitsOf units_of, Weight weight, int& b,
                                       Seq& s, Place& at) {
  while (idx - w.base >= __shfl_sync(0xffffffffu, w.upto, 31)) {
    if (w.chunk + 32 >= k.B) return false;
    next_chunk(k, w, most, units_of, weight);
  }
  const int r = idx - w.base;
  const int src = __ffs(__ballot_sync(0xffffffffu, r < w.upto)) - 1;
  b = __shfl_sync(0xffffffffu, w.seq, src);
  const int in = r - __shfl_sync(0xffffffffu, w.from, src);
  s = seq_at(k, b);
  at = place_of(units_of(s), in);
  return true;
}

}  // namespace pack
}  // namespace fa
