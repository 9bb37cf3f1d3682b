// paged.cuh -- the paged key/value cache as the kernels see it: where the row
// of a position lies, which packed token a row of the input is, and how the
// decode call divides its work.  The functions are host-callable too, so that
// a host test can walk them over any table, good or bad.
#pragma once

#include <stdint.h>

#include "fa.h"
#include "fa_internal.h"
#include "sm100.cuh"

namespace fa {
namespace paged {

// Device view of an fa_paged_cache.  Strides count bytes.
struct Cache {
  uint8_t* K;
  uint8_t* V;
  long long page_stride, head_stride, row_stride;
  int num_pages, page_size;
  const int* table;  // [B, max_pages], rows table_stride apart
  int max_pages;
  long long table_stride;
  const float* k_scale;  // [Hkv], 8-bit pools only
  const float* v_scale;
};

// Byte offset, in either pool, of head 0's row of a page's slot; -1 for a page
// index outside the pool (the caller records FA_ERR_BOUNDS and skips the row).
__host__ __device__ __forceinline__ long long row_offset(const Cache& c, int page, int slot) {
  if (page < 0 || page >= c.num_pages) return -1;
  return page * c.page_stride + slot * c.row_stride;
}

// The page index of position `pos`, entry i = pos / page_size of a sequence's row of
// the table; -1 for a position that the table does not span (i is then not used).
template <class Int>
__host__ __device__ __forceinline__ int page_of(const Cache& c, const int* row, Int pos, Int i) {
  if (pos < 0 || i >= c.max_pages) return -1;
  return ld_ro(row + i);
}
// The same of sequence b, by division.
__host__ __device__ __forceinline__ int page_of(const Cache& c, int b, long long pos) {
  return page_of(c, c.table + b * c.table_stride, pos, pos / c.page_size);
}

// Division of n < 2^31 by a number fixed for the launch: with 2^(s-1) < d <= 2^s
// and mul = ceil(2^(31+s) / d), n mul / 2^(31+s) exceeds n / d by less than
// n d / (d 2^(31+s)) < 1 / d, and so has the same whole part.
struct Divider {
  uint32_t mul;
  int shift;
  __host__ __device__ __forceinline__ int operator()(int n) const {
    return (int)(((unsigned long long)(uint32_t)n * mul) >> shift);
  }
};
inline Divider make_divider(int d) {
  int s = 0;
  while ((1ll << s) < d) ++s;
  return Divider{(uint32_t)(((1ull << (31 + s)) + d - 1) / d), 31 + s};
}

// Records a page index outside the pool.
__device__ __forceinline__ void bad_page(uint32_t* status) { atomicCAS(status, FA_DEV_OK, FA_DEV_ERR_BOUNDS); }

// A sequence's length as the kernels use it: at most what its table can hold.
__host__ __device__ __forceinline__ int clamp_len(const Cache& c, int len) {
  const long long cap = (long long)c.max_pages * c.page_size;
  return len < 0 ? 0 : (int)(len < cap ? len : cap);
}

// ------------------------------------------------------------------ decode ---
// The keys of each (sequence, head unit) form blocks of BLOCK keys, and the
// blocks of all of them one row: sequence by sequence, unit by unit, in key
// order.  CTA c of `grid` takes blocks [share(c), share(c + 1)), whatever
// sequences these belong to, so that every CTA reads the same amount of cache
// (to one block) however the lengths are spread.
constexpr int WARPS = 8;
constexpr int STEP = 16;             // keys a warp handles at a time
constexpr int BLOCK = WARPS * STEP;  // keys of one block

__host__ __device__ __forceinline__ int blocks_of(int len) { return (len + BLOCK - 1) / BLOCK; }
// a / b for a >= 0, b > 0: in 32 bits where they do (a 64-bit division takes about
// a hundred instructions).
__host__ __device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}
__host__ __device__ __forceinline__ long long share(long long total, int grid, int c) { return quotient(total * c, grid); }

// The CTA that holds block x: the largest c with share(c) <= x.
__host__ __device__ __forceinline__ int owner(long long total, int grid, long long x) {
  int c = (int)quotient(x * grid, total);
  if (c >= grid) c = grid - 1;  // x past the last block
  while (c + 1 < grid && share(total, grid, c + 1) <= x) ++c;
  while (c > 0 && share(total, grid, c) > x) --c;
  return c;
}

// A CTA leaves at most two partial results: of the unit that began before its
// first block (or with it), slot 2c, and of the one that goes on past its
// last, slot 2c + 1; units between these are complete in it.
__host__ __device__ __forceinline__ int part_slot(int c, long long cta_begin, long long unit_begin) {
  return 2 * c + (cta_begin >= unit_begin ? 0 : 1);
}

// The parts of a unit that is divided between CTAs are counted, and the CTA that
// brings the last one joins them.  The counter of the unit that begins in CTA c is
// word c at the head of the call's workspace, which calls that may overlap do not
// share.  Whatever the workspace holds on entry, a word counts only under the
// process's tag, 56 random bits above an 8-bit count: a part that meets other
// contents puts the tag there, and the last one leaves the tag with a count of
// zero, so that later calls on the same workspace need one addition a part and
// none has to clear the words first (a launch of its own would cost 2 us of 10).
// (Other contents pass for the tag with a chance of 2^-56.)
constexpr int COUNT_BITS = 8;
// Parts of the unit counted before this one.  Word: add(n) and cas(expected,
// desired), both atomic, return the word as it was.  A part adds to other contents
// once at most, so that each of the n parts fails at most n times to replace them.
#pragma nv_exec_check_disable
template <class Word>
__host__ __device__ __forceinline__ int count_part(Word& w, unsigned long long tag) {
  constexpr unsigned long long COUNT = (1ull << COUNT_BITS) - 1;
  unsigned long long seen = w.add(1);
  if (((seen ^ tag) & ~COUNT) == 0) return (int)(seen & COUNT);
  for (++seen;;) {
    const unsigned long long was = w.cas(seen, tag | 1u);
    if (was == seen) return 0;
    if (((was ^ tag) & ~COUNT) == 0) return (int)(w.add(1) & COUNT);
    seen = was;
  }
}

// What the walk goes by.  (Lengths are read again at each sequence.  Should they
// change during the launch, the results are undefined, but the walk ends, in
// sequences and head units that exist.)
struct Work {
  const Cache* c;
  const int* lens;
  int B, HU;  // sequences, head units of each
};

// A CTA's place in its blocks.
struct Walk {
  int b, hu, blk, nblk;  // sequence, head unit, block and blocks of the unit
  int len;
  long long at, end;     // place in the row of all blocks, and where the CTA stops
};

__host__ __device__ __forceinline__ void enter_sequence(const Work& k, Walk& w) {
  w.len = clamp_len(*k.c, ld_ro(k.lens + w.b));
  w.nblk = blocks_of(w.len);
}

// The start of CTA `cta` of `grid` <= total, in sequence b; before: blocks of one
// head unit in the sequences before it.
__host__ __device__ __forceinline__ Walk start_walk_at(const Work& k, int before, int b, long long total, int grid,
                                                       int cta) {
  Walk w;
  w.at = cta < grid ? share(total, grid, cta) : total;
  w.end = cta < grid ? share(total, grid, cta + 1) : total;
  w.b = b;
  w.hu = w.blk = w.nblk = w.len = 0;
  if (w.at < w.end) {
    enter_sequence(k, w);
    const long long into = w.at - (long long)before * k.HU;
    w.hu = w.nblk > 0 ? (int)quotient(into, w.nblk) : k.HU;
    w.blk = (int)(into - (long long)w.hu * w.nblk);
    if (w.hu >= k.HU) w.at = w.end;  // the length is another by now
  }
  return w;
}
// The same from prefix[b], the blocks of one head unit in sequences 0 .. b.
__host__ __device__ __forceinline__ Walk start_walk(const Work& k, const int* prefix, int b, long long total, int grid,
                                                    int cta) {
  return start_walk_at(k, b > 0 ? prefix[b - 1] : 0, b, total, grid, cta);
}

// The sequence that holds block x: the first b with prefix[b] * HU > x.
__host__ __device__ __forceinline__ int sequence_of(const int* prefix, int B, int HU, long long x) {
  int lo = 0, hi = B;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if ((long long)prefix[mid] * HU > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// From the last block of a unit, `at` already past it, to the next unit.
__host__ __device__ __forceinline__ void next_unit(const Work& k, Walk& w) {
  w.blk = 0;
  if (++w.hu < k.HU) return;
  w.hu = 0;
  if (w.at >= w.end) return;
  if (w.b + 1 >= k.B) return;  // (the lengths are others by now: the last sequence again)
  do {  // at < end <= total: a sequence with blocks is ahead
    ++w.b;
    enter_sequence(k, w);
  } while (w.nblk == 0 && w.b + 1 < k.B);
}
// Whether the walk has a unit, or a part of one, at hand.
__host__ __device__ __forceinline__ bool at_hand(const Walk& w) { return w.at < w.end && w.nblk > 0; }

// Whole units only: a CTA takes the units that begin in its share.  w: its walk;
// next: the walk that the next CTA starts with.
__host__ __device__ __forceinline__ long long unit_boundary(const Walk& w) { return w.blk > 0 ? w.at + (w.nblk - w.blk) : w.at; }
__host__ __device__ __forceinline__ Walk whole_units(const Work& k, Walk w, const Walk& next, int grid, int cta) {
  if (w.at >= w.end) return w;
  if (cta + 1 < grid) w.end = unit_boundary(next);
  if (w.blk > 0) {
    w.at = unit_boundary(w);
    next_unit(k, w);
  }
  return w;
}

// ------------------------------------------------------------------- evict ---
constexpr int SEL_THREADS = 1024;  // of a selecting CTA
constexpr int SEL_ROWS = 4;        // rows of K and V that a lane has on their way in one

// SMs without a selection (idle, next to one for each of `heads` (sequence, head)s)
// move rows meanwhile that need none: of each head this many at most, 256 KB read and
// written by each SM, which takes about as long as the selection.  Not where an SM
// would go through more than two heads, since it waits for the rows of each in turn.
// 64 heads of 4000-8192 rows: 32.6 us without, 30.3 with; 96: 45.0, 42.7; 112: 50.4,
// 50.6; 128: 56.6, 60.6; 144: 62, 114; 147: 63, 352.
__host__ __device__ __forceinline__ int early_most(int heads, int idle, int recent, int row_bytes) {
  if (heads > 2 * idle) return 0;
  const long long fit = idle * (256LL << 10) / ((long long)heads * 4 * row_bytes);
  return (int)(fit < recent ? fit : recent);
}

}  // namespace paged

inline paged::Cache cache_view(const PagedCache& c) {
  paged::Cache v;
  v.K = static_cast<uint8_t*>(c.K);
  v.V = static_cast<uint8_t*>(c.V);
  v.page_stride = c.page_stride * c.elem;
  v.head_stride = c.head_stride * c.elem;
  v.row_stride = c.row_stride * c.elem;
  v.num_pages = c.num_pages;
  v.page_size = c.page_size;
  v.table = c.table;
  v.max_pages = c.max_pages;
  v.table_stride = c.table_stride;
  v.k_scale = c.k_scale;
  v.v_scale = c.v_scale;
  return v;
}

}  // namespace fa
