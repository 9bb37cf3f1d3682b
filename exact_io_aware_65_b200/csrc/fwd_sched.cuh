// fwd_sched.cuh -- the forward's launch parameters and its work schedule:
// which (head, query-tile pair) a work item is, and which key tiles each
// query tile of it visits.  The kernel in fa_fwd.cu runs these functions in
// every role; they are host-callable too, so that a host test can walk the
// schedule of any problem and compare it with the visibility rule.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include <type_traits>

#include "fa.h"
#include "pack.cuh"
#include "sm100.cuh"

namespace fa {
namespace fwd {

constexpr int BM = 128;              // query rows per tile
constexpr int BN = 128;              // keys per tile

struct Params {
  int BH, N, nq, n_pairs, n_items, mask_kind;  // N, nq: query rows and tiles
  // Query tiles per work item: 2 (a pair, n_pairs = ceil(nq / 2)) or 1
  // (n_pairs = nq: one tile per item).
  int tiles_per_item;
  int Nk, nk, off;  // key rows and tiles; causal: query i sees keys j <= i + off
  int H;            // heads per batch element (a head's batch element is bh / H)
  // Optional per-batch-element lengths (device int [B], nullptr: N and Nk):
  // query rows and keys at or past them are padding.
  const int* seqlens_q;
  const int* seqlens_k;
  int group;  // heads per scheduling group
  const uint8_t* block_mask;
  float scale_log2;
  __nv_bfloat16* O;
  float* LSE;
  uint64_t timeout_ns;
  uint32_t* status;
  uint32_t slot;  // scheduler counter slot of this launch
};

// What the packed launches have besides.  (Of its own type: with these fields in
// Params, nvcc spilled other registers of the fixed-size kernels, which took 4%
// longer at d = 128 for it.)
struct PackedParams : Params {
  Pack pk;
  int by_heads;  // an item's two tiles are two heads' of one query tile
  int d;
  long long o_row, o_head;  // strides of O, elements
  // SPLIT: parts of an item's key tiles, at most; each leaves its unnormalised O
  // [parts][Hq][Tq][d] and (m, l) [parts][Hq][Tq].
  int parts;
  float* part_o;
  float2* part_ml;
};
template <int MODE>
using ParamsOf = std::conditional_t<(MODE >= PACKED), PackedParams, Params>;
// The packed launch's parameters, for branches that only MODE >= PACKED takes.
__host__ __device__ __forceinline__ const PackedParams& packed(const Params& p) { return static_cast<const PackedParams&>(p); }

// Heads per scheduling group.  The group's K and V tiles are the forward's
// working set in L2, kept to about 32 MiB; above that, more heads per group
// spread the longest-first order over more items, which evens out the CTAs'
// work under a causal mask (short sequences: all heads in one group).  At
// least 8 heads, or all of them.
__host__ __device__ inline int sched_group(int BH, int Nk, int d) {
  const long long per_head = 4LL * (Nk > 0 ? Nk : 1) * d;  // K and V, bf16
  const long long fit = (32LL << 20) / per_head;
  const long long g = fit > 8 ? fit : 8;
  return (int)(g < BH ? g : BH);
}

struct Item {
  int bh, q0, q1;
  bool has1;
  int Lq, Lk, off, nkb;  // this sequence's query rows and keys, causal offset, key tiles
  // PACKED: the heads of the item's tiles, the sequence's first query row and
  // key; off counts tiles.
  int h0, h1, sq, sk;
  int part, parts, j0, j1;  // SPLIT: the item's part of its parts, and its key tiles
};

// Work item idx -> (head, pair of query tiles, or one query tile).  Heads are taken in groups
// of p.group so that the K/V tiles in flight belong to a few heads and stay
// in L2; within a group later query tiles come first, so that under a causal
// mask the longest items start earliest (and, claimed dynamically, the short
// ones fill in at the end).
template <int MODE>
__host__ __device__ __forceinline__ Item item_at(const Params& p, int idx) {
  Item it;
  const int per_group = p.group * p.n_pairs;
  const int g = idx / per_group, r = idx % per_group;
  const int gsize = min(p.group, p.BH - g * p.group);
  const int c = p.n_pairs - 1 - r / gsize;
  it.bh = g * p.group + r % gsize;
  it.q0 = p.tiles_per_item * c;
  it.q1 = it.q0 + 1;
  it.has1 = p.tiles_per_item == 2 && it.q1 < p.nq;
  if (MODE == PADDED) {
    const int b = it.bh / p.H;
    const bool bok = FA_IN_BOUNDS(p.status, b, 1, p.BH / p.H);
    it.Lq = p.seqlens_q ? (bok ? min(max(ld_ro(p.seqlens_q + b), 0), p.N) : 0) : p.N;
    it.Lk = p.seqlens_k ? (bok ? min(max(ld_ro(p.seqlens_k + b), 0), p.Nk) : 0) : p.Nk;
    it.off = it.Lk - it.Lq;
    it.nkb = (it.Lk + BN - 1) / BN;
  } else {  // every sequence fills its slice: the launch's own sizes
    it.Lq = p.N;
    it.Lk = p.Nk;
    it.off = p.off;
    it.nkb = p.nk;
  }
  return it;
}

// One past the last key tile that query tile qt of a packed sequence sees.
__host__ __device__ __forceinline__ int packed_end(const Params& p, int nkb, int off, int qt) {
  return p.mask_kind == FA_MASK_CAUSAL ? max(0, min(nkb, qt + off + 1)) : nkb;
}

// SPLIT: the parts that `tiles` key tiles are divided into: at least eight tiles
// each, since a part costs about two tiles' time before and after them.
__host__ __device__ __forceinline__ int parts_of(const PackedParams& p, int tiles) { return max(1, min(p.parts, tiles / 8)); }
// The later query tile of the item that query tile qt of nq belongs to.
__host__ __device__ __forceinline__ int last_tile(const PackedParams& p, int nq, int qt) {
  return p.tiles_per_item == 2 && !p.by_heads ? nq - 1 - (nq - 1 - qt) / 2 * 2 : qt;
}
// The part's key tiles (none for a part past the item's parts).
__host__ __device__ __forceinline__ void take_part(const PackedParams& p, Item& it) {
  const int e = packed_end(p, it.nkb, it.off, it.has1 ? it.q1 : it.q0);
  it.parts = parts_of(p, e);
  it.j0 = it.part < it.parts ? e * it.part / it.parts : 0;
  it.j1 = it.part < it.parts ? e * (it.part + 1) / it.parts : 0;
}

// Packed sequences.  An item's one or two query tiles: at d = 64 one; at
// d = 128 one query tile of two heads that share their keys where the heads of
// a key head come in pairs (both see the same keys, and a sequence of one tile
// still fills the item), else two neighbouring tiles, from the end.
__host__ __device__ __forceinline__ pack::Units packed_units(const PackedParams& p, const pack::Seq& s) {
  pack::Units u;
  const int nq = pack::tiles(s.Lq), per = p.by_heads ? 2 : 1;
  u.tiles = p.tiles_per_item == 2 && !p.by_heads ? (nq + 1) / 2 : nq;
  u.heads = p.pk.Hq / per * p.parts;
  // the heads of whole key heads, their K and V kept to about 32 MiB (as sched_group)
  const long long fit = (32LL << 20) / (4LL * max(s.Lk, 1) * p.d);
  const long long least = (8 + p.pk.G - 1) / p.pk.G;  // 8 query heads
  u.group = (int)min((long long)p.pk.Hkv, max(fit, least)) * p.pk.G / per * p.parts;
  return u;
}

__host__ __device__ __forceinline__ Item packed_item(const PackedParams& p, const pack::Seq& s, const pack::Place& place) {
  Item it;
  const pack::Place at{place.tile, place.head / p.parts};
  it.part = place.head % p.parts;
  const int nq = pack::tiles(s.Lq);
  it.bh = 0;
  it.Lq = s.Lq;
  it.Lk = s.Lk;
  it.nkb = pack::tiles(s.Lk);
  it.off = it.nkb - nq;
  it.sq = s.sq;
  it.sk = s.sk;
  if (p.tiles_per_item == 1 || p.by_heads) {
    it.q0 = it.q1 = nq - 1 - at.tile;
    it.has1 = p.by_heads;
    it.h0 = p.by_heads ? 2 * at.head : at.head;
    it.h1 = it.h0 + 1;
  } else {
    it.h0 = it.h1 = at.head;
    it.q1 = nq - 1 - 2 * at.tile;
    it.has1 = it.q1 > 0;
    it.q0 = it.has1 ? it.q1 - 1 : 0;
  }
  return it;
}

// Last key a query row of tile qt may see under the causal mask (the tile's
// last row of the sequence, shifted by the alignment; negative: none).
__host__ __device__ __forceinline__ int causal_last_key(const Item& it, int qt) {
  return min(qt * BM + BM - 1, it.Lq - 1) + it.off;
}

// Does query tile qt attend to key tile j?  (With per-sequence lengths,
// tiles past the sequence's query rows or keys attend to nothing; without,
// every tile an item or a key loop reaches is inside.)
template <int MODE>
__host__ __device__ __forceinline__ bool member(const Params& p, const Item& it, int qt, int j) {
  if (MODE == PADDED && (qt * BM >= it.Lq || j >= it.nkb)) return false;
  if (MODE >= PACKED) return j < it.nkb && (p.mask_kind != FA_MASK_CAUSAL || j <= qt + it.off);
  if (p.mask_kind == FA_MASK_CAUSAL) return j * BN <= causal_last_key(it, qt);
  if (p.mask_kind == FA_MASK_BLOCK)
    return FA_IN_BOUNDS(p.status, (size_t)qt * p.nk + j, 1, (size_t)p.nq * p.nk) &&
           ld_ro(p.block_mask + (size_t)qt * p.nk + j) != 0;
  return true;
}

// One past the last key tile either query tile of the item may need.
template <int MODE>
__host__ __device__ __forceinline__ int kv_end(const Params& p, const Item& it) {
  if (MODE == PADDED && it.q0 * BM >= it.Lq) return 0;
  if (MODE == SPLIT) return it.j1;
  if (MODE >= PACKED) return packed_end(p, it.nkb, it.off, it.has1 ? it.q1 : it.q0);
  if (p.mask_kind == FA_MASK_CAUSAL) {
    const int last = causal_last_key(it, (it.has1 && (MODE != PADDED || it.q1 * BM < it.Lq)) ? it.q1 : it.q0);
    return last < 0 ? 0 : min(it.nkb, last / BN + 1);
  }
  return it.nkb;
}

// The first key tile of the item's key loop.
template <int MODE>
__host__ __device__ __forceinline__ int kv_begin(const Item& it) {
  return MODE == SPLIT ? it.j0 : 0;
}

// Next key tile >= j needed by either query tile of the item (kv_end if none).
template <int MODE>
__host__ __device__ __forceinline__ int next_union(const Params& p, const Item& it, int j) {
  const int e = kv_end<MODE>(p, it);
  if (p.mask_kind != FA_MASK_BLOCK) return j < e ? j : e;
  for (; j < e; ++j)
    if (member<MODE>(p, it, it.q0, j) || (it.has1 && member<MODE>(p, it, it.q1, j))) return j;
  return e;
}

}  // namespace fwd
}  // namespace fa
