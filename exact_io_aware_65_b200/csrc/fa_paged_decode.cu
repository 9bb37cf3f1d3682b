// fa_paged_decode.cu -- attention of one new token per sequence over a paged
// key/value cache with grouped heads.
//
// For query head h of sequence b, over the keys j < lens[b] of key head
// h / G (G = Hq / Hkv):  s_j = scale q . k_j,  O = sum_j 2^(s_j - m) v_j / l with
// the running maximum m and sum l of an online softmax (in log2 units), and
// LSE = (m + log2 l) ln 2.  A key is used by G query heads and read once for each 16
// of them (a unit): up to G = 16 the call is bound by one read of the cache, 4 Nk d
// bytes a key head in bf16 and half of that in 8 bits.
//
// Kernel 1 (partial).  One CTA per SM; every CTA takes the same number of
// 128-key blocks of the batch, in order, whatever sequences they belong to
// (paged.cuh).  A warp takes 16 keys of each block: it copies their rows into
// its own ring in shared memory (cp.async, 16 bytes a lane, the row's place
// looked up in the page table a step before), and no warp waits for another
// until the unit ends.  Keys are the rows of both matrix products (m16n8k16),
// S^T = K Q^T and O^T = V^T P^T, and the query heads the eight columns: G <= 8
// heads fill half as much of the products as they would as rows, O takes half
// the registers, and the maxima and sums of a head stay in its lanes.  (On the
// CUDA cores G multiply-adds a cache element would take longer than the
// element's read from G = 8 on; the 128-row tiles of the tensor-memory products
// would be mostly empty.)  8-bit rows are widened to fp16 in registers (exact),
// the queries are then scaled by a power of two into fp16's range, and P is
// rounded to fp16 (2^-12 relative) rather than bf16.
// The running maximum is lazy: a head takes it from its first keys and moves it
// only when a score lies more than 8 (in log2 units) above it, so that a step
// usually has no reduction over lanes; O / l does not depend on it, and 2^8
// leaves fp16 room.
// At the end of a unit the eight warps join their (O, m, l) in shared memory;
// a unit that lies in one CTA is finished there, a part of one goes to the
// workspace, and the CTA that brings a unit's last part joins its parts, in their
// order (the same bits each run): a second kernel for that cost 2 us more (one
// sequence of 777 keys, 32 over 8 heads: 14.4 us against 12.4, then; now 10.3).
// What it comes to: 4 sequences of 30001-32768 keys, 8 key heads of 128, in 8 bits
// 55 us, 4.6 TB/s (bound by the instructions that widen 8 bits); the same in bf16
// 91 us, 5.6 TB/s, near the rate of a plain copy.
// Kernel 2 (weights), on request: P = 2^(s - LSE log2 e) from the scores that
// kernel 1 left in the workspace, summed over the group in head order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <sys/random.h>
#include <time.h>

#include <type_traits>

#include "fa_internal.h"
#include "sm100.cuh"
#include "paged.cuh"

namespace fa {
namespace paged {

constexpr int ROWS = 16;  // query heads of a unit, at most: 8 in a tile, NB tiles
constexpr int THREADS = WARPS * 32;
constexpr int MAX_GRID = 160;
static_assert(MAX_GRID < 1 << COUNT_BITS, "a unit's parts are counted in this many bits");

constexpr float SLACK = 8.0f;  // log2 units a score may lie above the reference maximum
constexpr int MAX_BATCH = 4096;                 // sequences per launch (prefix of their blocks in shared memory)
constexpr float LN2 = 0.69314718055994530942f;
constexpr float LOG2E = 1.4426950408889634074f;

struct DecodeParams {
  Cache c;
  const __nv_bfloat16* Q;
  long long q_row, q_head;  // elements
  const int* lens;
  int B, Hq, Hkv, G, HB;    // HB: units of a key head's group
  int R;                    // query heads of a unit
  Divider page;
  int whole;                // a unit is never divided between CTAs
  int wide;                 // rows lie 2^36 bytes or more from the pool's start
  float sl2;                // scale * log2(e)
  float* part;              // [2 grid][ROWS][D] unnormalised O
  float2* ml;               // [2 grid][ROWS] (m, l)
  unsigned long long* came; // [grid] counters of the parts of the unit that begins in a CTA (paged.cuh)
  unsigned long long tag;   // above their counts
  float* scores;            // [B, Hq, pitch] scaled log2 scores, or nullptr
  long long pitch;
  __nv_bfloat16* O;         // [B, Hq, D]
  float* LSE;               // [B, Hq]
  uint32_t* status;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
// c += a b (16 x 8 x 16); HALF: fp16 operands, else bf16.
template <bool HALF>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (HALF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two 8-bit values to two fp16 (exact).
__device__ __forceinline__ uint32_t widen(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
template <bool HALF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (HALF)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A step's rows in a ring stage: 16-byte piece c of row r.  The pieces are
// exchanged so that the eight rows an ldmatrix reads at one piece index fall
// in eight different bank groups.
template <int ROWB>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  if (ROWB == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) * 16);
  return r * ROWB + ((c ^ (r & 7)) * 16);
}

// A counter of parts: each operation releases what the CTA has stored before, and
// acquires what the others had stored before theirs.
struct Counter {
  unsigned long long* p;
  __device__ __forceinline__ unsigned long long add(unsigned long long n) {
    unsigned long long r;
    asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], %2;" : "=l"(r) : "l"(p), "l"(n) : "memory");
    return r;
  }
  __device__ __forceinline__ unsigned long long cas(unsigned long long expected, unsigned long long desired) {
    unsigned long long r;
    asm volatile("atom.acq_rel.gpu.global.cas.b64 %0, [%1], %2, %3;" : "=l"(r) : "l"(p), "l"(expected), "l"(desired) : "memory");
    return r;
  }
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Shared memory: the warps' rings of units (16 keys' rows of K or of V), the
// queries (fp16 or bf16, rows a piece longer so that ldmatrix meets no bank
// twice), and the warps' O at the end (rows four floats longer, likewise).
template <int D, bool E4M3, int NB>
struct DCfg {
  static constexpr int R = 8 * NB;
  static constexpr int ROWB = E4M3 ? D : 2 * D;  // bytes of a cache row
  static constexpr int UNIT = STEP * ROWB;
  static constexpr int QPITCH = 2 * D + 16;
  static constexpr int JPITCH = D + 4;
  // (also the parts' (m, l) of a divided unit, and the sequences' prefix)
  static_assert(MAX_GRID * R * 8 <= WARPS * R * JPITCH * 4, "shared memory for the join");
  static constexpr int JOIN_BYTES = WARPS * R * JPITCH * 4 > MAX_BATCH * 4 ? WARPS * R * JPITCH * 4 : MAX_BATCH * 4;
  static constexpr int FIT = (224 * 1024 - R * QPITCH - JOIN_BYTES) / (WARPS * UNIT);
  // Units of a ring: an odd number, so that a step frees the places of the K and
  // V of one later step, whose rows are looked up once.
  static constexpr int NU = FIT < 7 ? (FIT - 1) / 2 * 2 + 1 : 7;
  static_assert(NU >= 3, "shared memory");
  static constexpr int SMEM_BYTES = WARPS * NU * UNIT + R * QPITCH + JOIN_BYTES;
};

template <int D, bool E4M3, int NB>
__global__ void __launch_bounds__(THREADS, 1) partial_kernel(const DecodeParams p) {
  using C = DCfg<D, E4M3, NB>;
  constexpr int ROWB = C::ROWB, R = C::R, NU = C::NU;
  constexpr int PIECES = ROWB / 16;
  constexpr int RPI = 32 / PIECES;  // rows a warp copies per instruction
  constexpr int KS = D / 16;        // 16-column steps of a row
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* sQ = smem + WARPS * NU * C::UNIT;
  float* join = reinterpret_cast<float*>(sQ + R * C::QPITCH);  // the prefix at the start
  __shared__ float sm_m[WARPS][ROWS], sm_l[WARPS][ROWS], sm_sl2[ROWS];
  __shared__ int warp_sum[WARPS];
  __shared__ int start_b, end_b, join_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int HU = p.Hkv * p.HB, cta = blockIdx.x;

  // ---- this CTA's blocks
  const Work work{&p.c, p.lens, p.B, HU};
  Walk w;
  long long total;  // blocks of all units
  int grid;         // CTAs with blocks (with fewer blocks than CTAs the first `total` take one each, so that no CTA
                    // between a unit's first and last is without a part)
  if (p.B <= 32) {
    // every warp for itself: a lane a sequence
    const int mine = lane < p.B ? blocks_of(clamp_len(p.c, __ldg(p.lens + lane))) : 0;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    total = (long long)__shfl_sync(0xffffffffu, upto, 31) * HU;
    grid = (int)min((long long)gridDim.x, total);
    auto start = [&](int c) {
      const unsigned past = __ballot_sync(0xffffffffu, c < grid && (long long)upto * HU > share(total, grid, c));
      const int b = past ? __ffs(past) - 1 : 0;
      return start_walk_at(work, __shfl_sync(0xffffffffu, upto - mine, b), b, total, grid, c);
    };
    w = start(cta);
    if (p.whole) w = whole_units(work, w, start(cta + 1), grid, cta);
  } else {
    int* prefix = reinterpret_cast<int*>(join);  // [b]: blocks of a head unit in the sequences up to b
    int carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
      const int b = b0 + tid;
      int x = b < p.B ? blocks_of(clamp_len(p.c, __ldg(p.lens + b))) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) warp_sum[warp] = x;
      __syncthreads();
      int before = carry;
      for (int v = 0; v < warp; ++v) before += warp_sum[v];
      if (b < p.B) prefix[b] = before + x;
      for (int v = 0; v < WARPS; ++v) carry += warp_sum[v];
      __syncthreads();
    }
    total = (long long)carry * HU;
    grid = (int)min((long long)gridDim.x, total);
    if (tid == 0) {
      start_b = cta < grid ? sequence_of(prefix, p.B, HU, share(total, grid, cta)) : 0;
      end_b = p.whole && cta + 1 < grid ? sequence_of(prefix, p.B, HU, share(total, grid, cta + 1)) : 0;
    }
    __syncthreads();
    w = start_walk(work, prefix, start_b, total, grid, cta);
    if (p.whole) w = whole_units(work, w, start_walk(work, prefix, end_b, total, grid, cta + 1), grid, cta);
    __syncthreads();  // prefix has been read
  }
  const long long begin = w.at;
  // sequences without keys: nothing else writes their rows
  for (int b = cta; b < p.B; b += gridDim.x) {
    if (__ldg(p.lens + b) > 0) continue;
    for (int i = tid; i < p.Hq * (D / 8); i += THREADS)
      reinterpret_cast<uint4*>(p.O + (long long)b * p.Hq * D)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = tid; i < p.Hq; i += THREADS) p.LSE[(long long)b * p.Hq + i] = -INFINITY;
  }
  if (!at_hand(w)) return;

  // ---- the copies run up to NU units ahead of the products (K, V, K, V, ...),
  // the page lookups a step ahead of the copies.  Lane r (and r + 16) looks up
  // row r of a step.
  const uint32_t ring = smem_u32(smem) + warp * (NU * C::UNIT);
  const int piece = lane % PIECES, row_of_lane = lane / PIECES;
  Walk f = w;  // the next step to look up
  long long looked = f.at;
  int f_hk = f.hu / p.HB;
  const int* f_table = p.c.table + f.b * p.c.table_stride;
  int page = 0, slot = 0, page_hk = 0;  // of the step looked up last
  bool asked = false;                   // the row exists
  auto look_up = [&]() {
    asked = false;
    if (looked < f.end) {
      const int key = f.blk * BLOCK + warp * STEP + (lane & 15);
      page_hk = f_hk;
      if (key < f.len) {
        const int i = p.page(key);
        slot = key - i * p.c.page_size;
        page = __ldg(f_table + i);  // i < max_pages: len is held to what the table spans
        asked = true;
      }
      ++looked;
      if (++f.blk == f.nblk) {
        f.at = looked;
        next_unit(work, f);
        f_hk = f.hu / p.HB;
        f_table = p.c.table + f.b * p.c.table_stride;
      }
    }
  };
  uint32_t off_lo = 0, off_hi = 0, real = 0;  // of the step to copy: the row's place (16-byte pieces), which rows are read
  long long head_off = 0;
  auto next_rows = [&]() {
    const bool good = asked && page >= 0 && page < p.c.num_pages;
    if (asked && !good) bad_page(p.status);
    const unsigned long long off = good ? (unsigned long long)(page * p.c.page_stride + slot * p.c.row_stride) >> 4 : 0ull;
    off_lo = (uint32_t)off;
    off_hi = (uint32_t)(off >> 32);
    real = __ballot_sync(0xffffffffu, good);
    head_off = page_hk * p.c.head_stride + piece * 16;
  };
  auto after = [](uint32_t slot) { return slot + 1 == NU ? 0u : slot + 1; };
  uint32_t put = 0;  // ring slot of the next unit
  // K, V or both of the step at hand, a group each; after its V the next step
  // is at hand.
  auto copy_rows = [&](bool k, bool v) {
    uint32_t lo[STEP / RPI], hi[STEP / RPI];
#pragma unroll
    for (int i = 0; i < STEP / RPI; ++i) {
      lo[i] = __shfl_sync(0xffffffffu, off_lo, i * RPI + row_of_lane);
      hi[i] = p.wide ? __shfl_sync(0xffffffffu, off_hi, i * RPI + row_of_lane) : 0u;
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      if (kv == 0 ? !k : !v) continue;
      const uint32_t dst = ring + put * C::UNIT;
      const uint8_t* src = (kv == 0 ? p.c.K : p.c.V) + head_off;
#pragma unroll
      for (int i = 0; i < STEP / RPI; ++i) {
        const int r = i * RPI + row_of_lane;
        const unsigned long long off = ((unsigned long long)hi[i] << 32 | lo[i]) << 4;
        cp16(dst + piece_at<ROWB>(r, piece), src + off, (real >> r) & 1u);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      put = after(put);
    }
    if (v) {
      next_rows();
      look_up();
    }
  };
  look_up();
  next_rows();
  look_up();
  // (steps that do not exist are left out here; in the loop below that check cost
  // 7% of a long 8-bit call)
#pragma unroll
  for (int i = 0; i < NU; i += 2) {
    if (w.at + i / 2 < w.end) {
      copy_rows(true, i + 1 < NU);
    } else {
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (i + 1 < NU) asm volatile("cp.async.commit_group;" ::: "memory");
      put = after(put);
      if (i + 1 < NU) put = after(put);
    }
  }

  uint32_t got = 0;  // ring slot of the next unit to use
  while (at_hand(w)) {
    // ---- a unit, or this CTA's part of it
    const int hk = w.hu / p.HB, row0 = (w.hu % p.HB) * R;
    const int heads = min(R, p.G - row0);  // query heads in use
    const int b = w.b;
    const long long unit_begin = w.at - w.blk;
    const int nseg = (int)min((long long)(w.nblk - w.blk), w.end - w.at);
    const long long q_first = (long long)b * p.Hq + hk * p.G + row0;  // output row of the unit's first head
    // ---- the queries: a row per warp into shared memory
    for (int r = warp; r < R; r += WARPS) {
      constexpr int E = D / 32;  // values a lane
      float x[E];
      const __nv_bfloat16* src = p.Q + b * p.q_row + (hk * p.G + row0 + r) * p.q_head + lane * E;
      if (r < heads) {
        if (E == 4) {
          const uint2 v = *reinterpret_cast<const uint2*>(src);
          const uint32_t u[2] = {v.x, v.y};
#pragma unroll
          for (int e = 0; e < E; ++e) x[e] = __uint_as_float(e & 1 ? u[e / 2] & 0xffff0000u : u[e / 2] << 16);
        } else {
          const uint32_t u = *reinterpret_cast<const uint32_t*>(src);
          x[0] = __uint_as_float(u << 16);
          x[1] = __uint_as_float(u & 0xffff0000u);
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = 0.0f;
      }
      float sl2 = p.sl2;
      if (E4M3) {
        // bf16 reaches further than fp16: each row is scaled by the power of
        // two that brings its largest entry into [1, 2).  Entries below 2^-14 of
        // that lose bits that the row's sum cannot show.
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int e2 = max(-126, min(126, (int)(__float_as_uint(amax) >> 23) - 127));
        const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
        sl2 = p.sl2 * __ldg(p.c.k_scale + hk) * __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] *= down;
      }
      if (lane == 0) sm_sl2[r] = sl2;
      // 8 bits: within 16 columns in the order in which a lane finds its four
      // values of a piece (columns 4 t, 4 t + 1 at 2 t, and 4 t + 2, 4 t + 3 at 2 t + 8)
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const int col = lane * E + e, in = col & 15;
        const int at = E4M3 ? (col & ~15) + ((in & 2) ? 8 : 0) + (in >> 2) * 2 : col;
        *reinterpret_cast<uint32_t*>(sQ + r * C::QPITCH + at * 2) = pack2<E4M3>(x[e], x[e + 1]);
      }
    }
    __syncthreads();
    // B operands: head g, columns 2 t, 2 t + 1 (+ 8) of each 16
    const uint32_t q_at = smem_u32(sQ) + (lane & 7) * C::QPITCH + (lane >> 3) * 16;
    uint32_t qb[NB == 1 ? KS / 2 : 1][4];
    if (NB == 1) {
#pragma unroll
      for (int s = 0; s < KS / 2; ++s) ldsm4(qb[NB == 1 ? s : 0], q_at + s * 64);
    }
    float sl2[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      sl2[n][0] = sm_sl2[n * 8 + 2 * t];
      sl2[n][1] = sm_sl2[n * 8 + 2 * t + 1];
    }
    // O^T: tile i, rows g and g + 8 (bf16: columns 16 i + g, + 8 of the head; 8
    // bits: 16 i + 2 g, + 1), heads 8 n + 2 t, + 1
    float o[KS][NB][4];
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int n = 0; n < NB; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.0f;
    float m[NB][2], l[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }

    // Products of 32 columns (i, i + 1 of the 16-column steps).  S^T += K Q^T, two
    // chains of products:
    float c[NB][2][4];
    const int mi = lane >> 3, lr = lane & 7;  // ldmatrix: matrix and row of this lane's address
    auto clear = [&]() {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[n][0][e] = c[n][1][e] = 0.0f;
    };
    auto mul_k = [&](uint32_t sK, int s) {
      uint32_t q4[NB][4];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        if (NB == 1) {
#pragma unroll
          for (int e = 0; e < 4; ++e) q4[n][e] = qb[NB == 1 ? s / 2 : 0][e];
        } else {
          ldsm4(q4[n], q_at + n * 8 * C::QPITCH + s * 32);
        }
      }
      const int kr = (mi & 1) * 8 + lr;
      uint32_t a0[4], a1[4];
      if (E4M3) {  // a piece is 16 columns
        uint32_t r[4];
        ldsm4(r, sK + piece_at<ROWB>(kr, s + (mi >> 1)));
        a0[0] = widen(r[0]);
        a0[1] = widen(r[1]);
        a0[2] = widen(r[0] >> 16);
        a0[3] = widen(r[1] >> 16);
        a1[0] = widen(r[2]);
        a1[1] = widen(r[3]);
        a1[2] = widen(r[2] >> 16);
        a1[3] = widen(r[3] >> 16);
      } else {
        ldsm4(a0, sK + piece_at<ROWB>(kr, 2 * s + (mi >> 1)));
        ldsm4(a1, sK + piece_at<ROWB>(kr, 2 * s + 2 + (mi >> 1)));
      }
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        mma<E4M3>(c[n][0], a0, q4[n][0], q4[n][1]);
        mma<E4M3>(c[n][1], a1, q4[n][2], q4[n][3]);
      }
    };
    // O^T += V^T P^T (ldmatrix transposed):
    uint32_t pb[NB][2];  // P^T as B operand
    auto mul_v = [&](uint32_t sV, int i) {
      uint32_t a0[4], a1[4];
      if (E4M3) {
        // bytes (key, col), (key, col + 1), (key + 1, col), (key + 1, col + 1): the
        // even columns are rows g of the tile, the odd ones rows g + 8
        uint32_t r[4];
        ldsm4_t(r, sV + piece_at<ROWB>((mi & 1) * 8 + lr, i + (mi >> 1)));
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = __byte_perm(r[e], 0, 0x3120);
        a0[0] = widen(r[0]);
        a0[1] = widen(r[0] >> 16);
        a0[2] = widen(r[1]);
        a0[3] = widen(r[1] >> 16);
        a1[0] = widen(r[2]);
        a1[1] = widen(r[2] >> 16);
        a1[2] = widen(r[3]);
        a1[3] = widen(r[3] >> 16);
      } else {
        const int kr = (mi >> 1) * 8 + lr;
        ldsm4_t(a0, sV + piece_at<ROWB>(kr, 2 * i + (mi & 1)));
        ldsm4_t(a1, sV + piece_at<ROWB>(kr, 2 * i + 2 + (mi & 1)));
      }
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        mma<E4M3>(o[i][n], a0, pb[n][0], pb[n][1]);
        mma<E4M3>(o[i + 1][n], a1, pb[n][0], pb[n][1]);
      }
    };
    // Online softmax of step `step`'s scores; a lane has keys g, g + 8 of heads 2 t, 2 t + 1.
    auto softmax = [&](int step) {
      const int key0 = (w.blk + step) * BLOCK + warp * STEP;
      const int valid = w.len - key0;  // keys of this step that exist (may be <= 0: then P = 0)
      float x[NB][4];
      bool above = false;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[n][e] = g + (e >> 1) * 8 < valid ? (c[n][0][e] + c[n][1][e]) * sl2[n][e & 1] : -INFINITY;
        if (p.scores && valid > 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int h = n * 8 + 2 * t + e;
            if (h < heads) {
              float* row = p.scores + (q_first + h) * p.pitch + key0 + g;
              row[0] = x[n][e];
              row[8] = x[n][e + 2];
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) above |= fmaxf(x[n][e], x[n][e + 2]) > m[n][e] + SLACK;
      }
      if (__any_sync(0xffffffffu, above)) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(x[n][e], x[n][e + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            mx = fmaxf(mx, m[n][e]);
            const float down = ex2_approx(m[n][e] - (mx == -INFINITY ? 0.0f : mx));
            m[n][e] = mx;
            l[n][e] *= down;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              o[i][n][e] *= down;
              o[i][n][e + 2] *= down;
            }
          }
      }
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const float r0 = m[n][0] == -INFINITY ? 0.0f : m[n][0];  // every score so far -inf: P = 0
        const float r1 = m[n][1] == -INFINITY ? 0.0f : m[n][1];
        const float p0 = ex2_approx(x[n][0] - r0), p1 = ex2_approx(x[n][1] - r1);
        const float p2 = ex2_approx(x[n][2] - r0), p3 = ex2_approx(x[n][3] - r1);
        l[n][0] += p0 + p2;
        l[n][1] += p1 + p3;
        pb[n][0] = transpose8x8(pack2<E4M3>(p0, p1));
        pb[n][1] = transpose8x8(pack2<E4M3>(p2, p3));
      }
    };
    // The place of the next unit to use.  At every wait below NU units behind the
    // last used one are on their way, so that all but NU - 1 (or, where two are
    // used, NU - 2) of them having landed means that it has; once used, a unit's
    // place goes to the one NU later.
    auto use = [&]() {
      const uint32_t at = ring + got * C::UNIT;
      got = after(got);
      return at;
    };

    // S of the first step; then S of a step together with P V of the step before
    // (independent products side by side: the two warps of a scheduler do not
    // hide each other's latencies); at last P V of the last.
    {
      asm volatile("cp.async.wait_group %0;" ::"n"(NU - 1) : "memory");
      __syncwarp();
      const uint32_t sK = use();
      clear();
#pragma unroll
      for (int i = 0; i < KS; i += 2) mul_k(sK, i);
      __syncwarp();
      copy_rows(false, true);
      softmax(0);
    }
    for (int step = 1; step < nseg; ++step) {
      asm volatile("cp.async.wait_group %0;" ::"n"(NU - 2) : "memory");
      __syncwarp();
      const uint32_t sV = use(), sK = use();
      clear();
#pragma unroll
      for (int i = 0; i < KS; i += 2) {
        mul_k(sK, i);
        mul_v(sV, i);
      }
      __syncwarp();
      copy_rows(true, true);
      softmax(step);
    }
    {
      asm volatile("cp.async.wait_group %0;" ::"n"(NU - 1) : "memory");
      __syncwarp();
      const uint32_t sV = use();
#pragma unroll
      for (int i = 0; i < KS; i += 2) mul_v(sV, i);
      __syncwarp();
      copy_rows(true, false);
    }

    // ---- join the eight warps, in their order
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
        if (g == 0) {
          sm_m[warp][n * 8 + 2 * t + e] = m[n][e];
          sm_l[warp][n * 8 + 2 * t + e] = l[n][e];
        }
      }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = n * 8 + 2 * t + e;
        float M = -INFINITY;
#pragma unroll
        for (int v = 0; v < WARPS; ++v) M = fmaxf(M, sm_m[v][h]);
        const float f0 = ex2_approx(m[n][e] - (M == -INFINITY ? 0.0f : M));
        float* row = join + (warp * R + h) * C::JPITCH;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          if (E4M3) {
            *reinterpret_cast<float2*>(row + 16 * i + 2 * g) = make_float2(o[i][n][e] * f0, o[i][n][e + 2] * f0);
          } else {
            row[16 * i + g] = o[i][n][e] * f0;
            row[16 * i + g + 8] = o[i][n][e + 2] * f0;
          }
        }
      }
    __syncthreads();
    const bool whole = nseg == w.nblk;
    {
      const float vs = E4M3 ? __ldg(p.c.v_scale + hk) : 1.0f;
      const int part = part_slot(cta, begin, unit_begin);
      for (int k = tid; k < heads * (D / 4); k += THREADS) {
        const int h = k / (D / 4), col = k % (D / 4) * 4;
        float M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int v = 0; v < WARPS; ++v) M = fmaxf(M, sm_m[v][h]);
        const float ref = M == -INFINITY ? 0.0f : M;
#pragma unroll
        for (int v = 0; v < WARPS; ++v) L += sm_l[v][h] * ex2_approx(sm_m[v][h] - ref);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int v = 0; v < WARPS; ++v) {
          const float4 y = *reinterpret_cast<const float4*>(join + (v * R + h) * C::JPITCH + col);
          x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
        if (whole) {
          const float inv = L > 0.0f ? vs / L : L == 0.0f ? 0.0f : L;
          *reinterpret_cast<uint2*>(p.O + (q_first + h) * D + col) =
              make_uint2(pack2<false>(x.x * inv, x.y * inv), pack2<false>(x.z * inv, x.w * inv));
          if (col == 0) p.LSE[q_first + h] = (M + log2f(L)) * LN2;
        } else {
          *reinterpret_cast<float4*>(p.part + ((long long)part * ROWS + h) * D + col) =
              make_float4(x.x * vs, x.y * vs, x.z * vs, x.w * vs);
          if (col == 0) p.ml[(long long)part * ROWS + h] = make_float2(M, L);
        }
      }
    }
    if (!whole) {
      // The CTA whose part of the unit comes last joins them all.  (A CTA's barrier
      // orders its threads' stores before thread 0's addition, and that before
      // their loads.)
      const int c0 = owner(total, grid, unit_begin), n = owner(total, grid, unit_begin + w.nblk - 1) - c0 + 1;
      __syncthreads();
      if (tid == 0) {
        Counter came{p.came + c0};
        const bool last = count_part(came, p.tag) == n - 1;
        if (last) p.came[c0] = p.tag;
        join_last = last;
      }
      __syncthreads();
      if (join_last) {
        // in CTAs after c0 the unit comes first: slot 2 c
        const int first = part_slot(c0, share(total, grid, c0), unit_begin);
        auto slot_of = [&](int i) { return (long long)(i ? 2 * (c0 + i) : first) * ROWS; };
        float2* ml = reinterpret_cast<float2*>(join);  // [n][R]: (m, l) of the parts
        for (int k = tid; k < n * R; k += THREADS) ml[k] = __ldcg(p.ml + slot_of(k / R) + k % R);
        for (int k0 = 0; k0 < heads * (D / 4); k0 += THREADS) {
          const int k = k0 + tid, h = k / (D / 4), col = k % (D / 4) * 4;
          const bool mine = h < heads;
          auto load = [&](int i) {
            return mine && i < n ? __ldcg(reinterpret_cast<const float4*>(p.part + (slot_of(i) + h) * D + col))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
          };
          constexpr int U = 8;  // parts on their way while the maxima are
          float4 y[U];
#pragma unroll
          for (int i = 0; i < U; ++i) y[i] = load(i);
          __syncthreads();
          if (!mine) continue;
          float M = -INFINITY;
          for (int i = 0; i < n; ++i) M = fmaxf(M, ml[i * R + h].x);
          const float ref = M == -INFINITY ? 0.0f : M;
          float L = 0.0f;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int i0 = 0; i0 < n; i0 += U) {
            if (i0 > 0) {
#pragma unroll
              for (int i = 0; i < U; ++i) y[i] = load(i0 + i);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
              if (i0 + i >= n) break;
              const float2 z = ml[(i0 + i) * R + h];
              const float f = ex2_approx(z.x - ref);
              L = fmaf(z.y, f, L);
              x = make_float4(fmaf(y[i].x, f, x.x), fmaf(y[i].y, f, x.y), fmaf(y[i].z, f, x.z), fmaf(y[i].w, f, x.w));
            }
          }
          const float inv = L > 0.0f ? 1.0f / L : L == 0.0f ? 0.0f : L;
          *reinterpret_cast<uint2*>(p.O + (q_first + h) * D + col) =
              make_uint2(pack2<false>(x.x * inv, x.y * inv), pack2<false>(x.z * inv, x.w * inv));
          if (col == 0) p.LSE[q_first + h] = (M + log2f(L)) * LN2;
        }
        __syncthreads();  // ml, which the next unit's join overwrites
      }
    }
    // (sm_m, sm_l and the joined rows are written again only after the next
    // unit's barrier behind its queries, or behind its products)
    w.at += nseg;
    w.blk += nseg;
    if (w.blk == w.nblk) next_unit(work, w);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// A[b, hk, j] (+)= sum over the group of 2^(s_j - LSE log2 e): four keys a
// thread, four heads' scores in flight.
constexpr int W_THREADS = 256;
__global__ void __launch_bounds__(W_THREADS) weights_kernel(const DecodeParams p, float* A, long long a_batch,
                                                            long long a_head, int accumulate, int chunks) {
  const int bh = blockIdx.x / chunks, b = bh / p.Hkv, hk = bh % p.Hkv;
  const int len = clamp_len(p.c, __ldg(p.lens + b));
  const long long first = (long long)b * p.Hq + hk * p.G;
  for (long long j = 4 * ((long long)(blockIdx.x % chunks) * W_THREADS + threadIdx.x); j < len;
       j += 4LL * chunks * W_THREADS) {
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int r = 0; r < p.G; ++r) {
      // (rows are 16-byte aligned, and end on a whole step behind the last key)
      const float4 s = *reinterpret_cast<const float4*>(p.scores + (first + r) * p.pitch + j);
      // (a head all of whose scores are -inf draws nothing, as its O is zero)
      const float l = __ldg(p.LSE + first + r), lse = l == -INFINITY ? 0.0f : l * LOG2E;
      sum.x += ex2_approx(s.x - lse);
      sum.y += ex2_approx(s.y - lse);
      sum.z += ex2_approx(s.z - lse);
      sum.w += ex2_approx(s.w - lse);
    }
    float* a = A + b * a_batch + hk * a_head + j;
    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e < len) a[e] = accumulate ? a[e] + v[e] : v[e];
  }
}

// The process's tag of the counters.
static unsigned long long join_tag() {
  static const unsigned long long tag = [] {
    unsigned long long x = 0;
    if (getrandom(&x, sizeof(x), GRND_NONBLOCK) != (ssize_t)sizeof(x)) {
      timespec now;  // no random source: the time in nanoseconds, above the place of this stack
      clock_gettime(CLOCK_REALTIME, &now);
      x = ((unsigned long long)now.tv_sec * 1000000000ull + (unsigned long long)now.tv_nsec) << 24 ^ reinterpret_cast<uintptr_t>(&x);
    }
    return x >> COUNT_BITS << COUNT_BITS;
  }();
  return tag;
}

// One CTA per SM, at most as many as there are counters.
static int decode_grid() { return num_sms() < MAX_GRID ? num_sms() : MAX_GRID; }

static size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct DecodeLayout {
  size_t came, part, ml, scores, total;
};
static DecodeLayout layout(int B, int Hq, int d, long long cap, bool weights, int grid) {
  DecodeLayout w;
  w.came = 0;  // first, where every call finds what the last one left
  w.part = align256((size_t)grid * sizeof(unsigned long long));
  w.ml = w.part + align256((size_t)2 * grid * ROWS * d * sizeof(float));
  w.scores = w.ml + align256((size_t)2 * grid * ROWS * sizeof(float2));
  w.total = w.scores + (weights ? align256((size_t)B * Hq * ((cap + STEP - 1) / STEP * STEP) * sizeof(float)) : 0);
  return w;
}

}  // namespace paged

size_t paged_decode_workspace_bytes(int B, int Hq, int d, long long cap, bool weights) {
  return paged::layout(B, Hq, d, cap, weights, paged::decode_grid()).total;
}

template <int D, bool E4M3, int NB>
static fa_status launch_d(paged::DecodeParams p, int B, const PagedDecode& a, int grid, cudaStream_t s) {
  using namespace paged;
  constexpr int smem = DCfg<D, E4M3, NB>::SMEM_BYTES;
  static_assert(smem + 2048 <= 227 * 1024, "shared memory");
  auto kern = partial_kernel<D, E4M3, NB>;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(done, (const void*)kern, smem)) return FA_ERR_CUDA;
  const int* lens = p.lens;
  const int* table = p.c.table;
  const __nv_bfloat16* Q = p.Q;
  __nv_bfloat16* O = p.O;
  float* LSE = p.LSE;
  float* scores = p.scores;
  for (int b0 = 0; b0 < B; b0 += MAX_BATCH) {
    p.B = B - b0 < MAX_BATCH ? B - b0 : MAX_BATCH;
    p.lens = lens + b0;
    p.c.table = table + b0 * p.c.table_stride;
    p.Q = Q + b0 * p.q_row;
    p.O = O + (long long)b0 * p.Hq * D;
    p.LSE = LSE + (long long)b0 * p.Hq;
    if (scores) p.scores = scores + (long long)b0 * p.Hq * p.pitch;
    if (!launch(kern, (unsigned)grid, THREADS, smem, s, p)) return FA_ERR_CUDA;
    if (scores) {
      long long chunks = (p.pitch + 4 * W_THREADS - 1) / (4 * W_THREADS);  // four keys a thread
      if (chunks > 64) chunks = 64;
      if (!launch(weights_kernel, (unsigned)(p.B * p.Hkv * chunks), W_THREADS, 0, s, p, a.W + b0 * a.w_batch,
                        a.w_batch, a.w_head, a.accumulate, (int)chunks))
        return FA_ERR_CUDA;
    }
  }
  return FA_OK;
}

fa_status launch_paged_decode(const PagedCache& c, const PagedDecode& a, cudaStream_t s) {
  uint32_t* st = status_word();
  if (!st) return FA_ERR_CUDA;
  const int grid = paged::decode_grid();
  const long long cap = (long long)c.max_pages * c.page_size;
  const paged::DecodeLayout w = paged::layout(c.B, a.Hq, c.d, cap, a.W != nullptr, grid);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  paged::DecodeParams p;
  p.c = cache_view(c);
  p.Q = static_cast<const __nv_bfloat16*>(a.Q.data);
  p.q_row = a.Q.row_stride;
  p.q_head = a.Q.head_stride;
  p.lens = a.lens;
  p.Hq = a.Hq;
  p.Hkv = c.Hkv;
  p.G = a.Hq / c.Hkv;
  p.R = p.G <= 8 ? 8 : 16;
  p.HB = (p.G + p.R - 1) / p.R;
  p.page = paged::make_divider(c.page_size);
  // Short caches (by the width of the page table): a unit's few blocks one after the other take less time than
  // their parts' join (16 sequences of 500 keys, 32 over 8 heads of 128: 10.2
  // against 16.5 us; 64 of 250, 16 heads: 35.0 against 42.1; one of 500: 9.9
  // against 9.4).
  p.whole = cap <= 4 * paged::BLOCK;
  p.wide = ((c.num_pages - 1) * c.page_stride + (c.page_size - 1) * c.row_stride) * c.elem >= (1ll << 36);
  p.sl2 = a.scale_log2;
  p.came = reinterpret_cast<unsigned long long*>(ws + w.came);
  p.tag = paged::join_tag();
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.ml = reinterpret_cast<float2*>(ws + w.ml);
  p.scores = a.W ? reinterpret_cast<float*>(ws + w.scores) : nullptr;
  p.pitch = (cap + paged::STEP - 1) / paged::STEP * paged::STEP;
  p.O = static_cast<__nv_bfloat16*>(a.O);
  p.LSE = a.LSE;
  p.status = st;
  auto run = [&](auto nb) {
    constexpr int NB = decltype(nb)::value;
    if (c.elem == 1)
      return c.d == 64 ? launch_d<64, true, NB>(p, c.B, a, grid, s) : launch_d<128, true, NB>(p, c.B, a, grid, s);
    return c.d == 64 ? launch_d<64, false, NB>(p, c.B, a, grid, s) : launch_d<128, false, NB>(p, c.B, a, grid, s);
  };
  return p.R == 8 ? run(std::integral_constant<int, 1>()) : run(std::integral_constant<int, 2>());
}

}  // namespace fa
