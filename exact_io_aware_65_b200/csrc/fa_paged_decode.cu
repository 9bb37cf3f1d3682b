// fa_paged_decode.cu -- attention of one new token per sequence over a paged
// key/value cache with grouped heads.
//
// For query head h of sequence b, over the keys j < lens[b] of key head
// h / G (G = Hq / Hkv):  s_j = scale q . k_j,  O = sum_j 2^(s_j - m) v_j / l with
// the running maximum m and sum l of an online softmax (in log2 units), and
// LSE = (m + log2 l) ln 2.  A key is used by G query heads and read once: the
// call is bound by the read of the cache, 4 Nk d bytes a key head in bf16 and
// half of that in 8 bits.
//
// Kernel 1 (partial).  One CTA per SM; every CTA takes the same number of
// 128-key blocks of the batch, in order, whatever sequences they belong to
// (paged.cuh).  A warp takes 16 keys of each block: it copies their rows into
// its own ring in shared memory (cp.async, 16 bytes a lane, the row's place
// looked up in the page table two steps ahead), and no warp waits for
// another until the unit ends.  The G <= 16 query heads are the rows of
// m16n8k16 matrix products: on the CUDA cores G multiply-adds a cache element
// would take longer than the element's read from G = 8 on, and the 128-row
// tiles of the tensor-memory products would be an eighth full.  The products
// take their B operand with ldmatrix; 8-bit rows are widened to fp16 in
// registers (exact), the queries are then scaled by a power of two into fp16's
// range, and P is rounded to fp16 (2^-12 relative) rather than bf16.
// At the end of a unit the eight warps join their (O, m, l) in shared memory;
// a unit that lies in one CTA is finished there, a part of one goes to the
// workspace.
// Kernel 2 (join): joins a unit's parts in CTA order (the same bits each run).
// Kernel 3 (weights), on request: P = 2^(s - LSE log2 e) from the scores that
// kernel 1 left in the workspace, summed over the group in head order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "fa_internal.h"
#include "sm100.cuh"
#include "paged.cuh"

namespace fa {
namespace paged {

constexpr int ROWS = 16;  // query heads of a unit
constexpr int THREADS = WARPS * 32;
constexpr int RING_BYTES = 192 * 1024 / WARPS;  // of each warp
constexpr int MAX_BATCH = 4096;                 // sequences per launch (prefix of their blocks in shared memory)
constexpr float LN2 = 0.69314718055994530942f;
constexpr float LOG2E = 1.4426950408889634074f;

struct DecodeParams {
  Cache c;
  const __nv_bfloat16* Q;
  long long q_row, q_head;  // elements
  const int* lens;
  int B, Hq, Hkv, G, HB;    // HB: 16-head units of a key head's group
  float sl2;                // scale * log2(e)
  float* part;              // [2 grid][ROWS][D] unnormalised O
  float2* ml;               // [2 grid][ROWS] (m, l)
  int4* desc;               // [grid] (sequence, head unit, first part, parts) of the unit a CTA begins and does not end
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

template <int D, bool E4M3>
__global__ void __launch_bounds__(THREADS, 1) partial_kernel(const DecodeParams p) {
  constexpr int ROWB = E4M3 ? D : 2 * D;   // bytes of a cache row
  constexpr int PIECES = ROWB / 16;
  constexpr int RPI = 32 / PIECES;         // rows a warp copies per instruction
  constexpr int STAGE = 2 * STEP * ROWB;   // K rows, then V rows
  constexpr int NST = RING_BYTES / STAGE < 6 ? RING_BYTES / STAGE : 6;
  constexpr int NT = D / 8;                // O column tiles
  constexpr int KS = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  float* join = reinterpret_cast<float*>(smem + WARPS * NST * STAGE);  // 4 warps' O; the prefix at the start
  __shared__ float sm_m[WARPS][ROWS], sm_l[WARPS][ROWS];
  __shared__ int warp_sum[WARPS];
  __shared__ int start_b;
  __shared__ long long sh_total;

  pdl_wait();
  pdl_next();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int HU = p.Hkv * p.HB, cta = blockIdx.x;

  // ---- this CTA's blocks.  prefix[b]: blocks of a head unit in the sequences
  // up to b.
  int* prefix = reinterpret_cast<int*>(join);
  {
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
    if (tid == 0) {
      const long long all = (long long)carry * HU;
      const int n = (int)min((long long)gridDim.x, all);
      sh_total = all;
      start_b = cta < n ? sequence_of(prefix, p.B, HU, share(all, n, cta)) : 0;
    }
    __syncthreads();
  }
  // (with fewer blocks than CTAs the first `total` CTAs take one each, so that
  // no CTA between a unit's first and last is without a part)
  const long long total = sh_total;
  const int grid = (int)min((long long)gridDim.x, total);
  const Work work{&p.c, p.lens, p.B, HU};
  Walk w = start_walk(work, prefix, start_b, total, grid, cta);
  const long long begin = w.at;
  // sequences without keys: nothing else writes their rows
  for (int b = cta; b < p.B; b += gridDim.x) {
    if (__ldg(p.lens + b) > 0) continue;
    for (int i = tid; i < p.Hq * (D / 8); i += THREADS)
      reinterpret_cast<uint4*>(p.O + (long long)b * p.Hq * D)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = tid; i < p.Hq; i += THREADS) p.LSE[(long long)b * p.Hq + i] = -INFINITY;
  }
  if (tid == 0) p.desc[cta] = make_int4(-1, 0, 0, 0);
  __syncthreads();  // prefix has been read
  if (w.at >= w.end) return;

  // ---- the copies run NST - 1 steps ahead, the page lookups one more
  const uint32_t ring = smem_u32(smem) + warp * (NST * STAGE);
  Walk f = w;          // the next step to look up
  long long row_next;  // its rows' offsets (lane r < 16: row r; -1: not read)
  int hk_next = 0;
  long long looked = f.at;
  auto look_up = [&]() {
    row_next = -1;
    if (looked < f.end) {
      const int key = f.blk * BLOCK + warp * STEP + (lane & 15);
      hk_next = f.hu / p.HB;
      if (key < f.len) {
        row_next = row_offset(p.c, page_of(p.c, f.b, key), key % p.c.page_size);
        if (row_next < 0) bad_page(p.status);
      }
      f.at = ++looked;
      if (++f.blk == f.nblk) next_unit(work, f);
    }
  };
  uint32_t put = 0;
  auto copy_step = [&]() {
    const uint32_t dst = ring + (put % NST) * STAGE;
    const int c = lane % PIECES;
    const long long head = hk_next * p.c.head_stride + c * 16;
#pragma unroll
    for (int i = 0; i < STEP / RPI; ++i) {
      const int r = i * RPI + lane / PIECES;
      const long long off = __shfl_sync(0xffffffffu, row_next, r);
      const bool real = off >= 0;
      const long long at = real ? off + head : 0;
      cp16(dst + piece_at<ROWB>(r, c), p.c.K + at, real);
      cp16(dst + STEP * ROWB + piece_at<ROWB>(r, c), p.c.V + at, real);
    }
    ++put;
  };
  look_up();
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) {
    copy_step();
    asm volatile("cp.async.commit_group;" ::: "memory");
    look_up();
  }

  uint32_t got = 0;
  while (w.at < w.end) {
    // ---- a unit, or this CTA's part of it
    const int hk = w.hu / p.HB, row0 = (w.hu % p.HB) * ROWS;
    const int heads = min(ROWS, p.G - row0);  // rows in use
    const int b = w.b;
    const long long unit_begin = w.at - w.blk;
    const int nseg = (int)min((long long)(w.nblk - w.blk), w.end - w.at);
    const long long q_first = (long long)b * p.Hq + hk * p.G + row0;  // output row of the unit's row 0
    // queries as A fragments: rows g and g + 8
    uint32_t qa[KS][4];
    float sl2[2];
    {
      float amax[2] = {0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = g + (e & 1) * 8;
          // bf16: columns 16 s + 2 t and + 8; 8 bits: 16 s + 4 t and + 2 (the
          // order in which a lane finds its four values of a 16-byte piece)
          const int col = E4M3 ? 16 * s + 4 * t + (e >> 1) * 2 : 16 * s + 2 * t + (e >> 1) * 8;
          qa[s][e] = r < heads ? *reinterpret_cast<const uint32_t*>(p.Q + b * p.q_row +
                                                                    (hk * p.G + row0 + r) * p.q_head + col)
                               : 0u;
          if (E4M3)
            amax[e & 1] = fmaxf(amax[e & 1], fmaxf(fabsf(__uint_as_float(qa[s][e] << 16)),
                                                   fabsf(__uint_as_float(qa[s][e] & 0xffff0000u))));
        }
      sl2[0] = sl2[1] = p.sl2;
      if (E4M3) {
        // bf16 reaches further than fp16: each row is scaled by the power of
        // two that brings its largest entry into [1, 2).  Entries below 2^-14 of
        // that lose bits that the row's sum cannot show.
        const float ks = __ldg(p.c.k_scale + hk);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          amax[z] = fmaxf(amax[z], __shfl_xor_sync(0xffffffffu, amax[z], 1));
          amax[z] = fmaxf(amax[z], __shfl_xor_sync(0xffffffffu, amax[z], 2));
          const int e = max(-126, min(126, (int)(__float_as_uint(amax[z]) >> 23) - 127));
          const float down = __uint_as_float((uint32_t)(127 - e) << 23);
          sl2[z] = p.sl2 * ks * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
          for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
              const uint32_t x = qa[s][z + 2 * e2];
              qa[s][z + 2 * e2] = pack2<true>(__uint_as_float(x << 16) * down, __uint_as_float(x & 0xffff0000u) * down);
            }
        }
      }
    }
    float o[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    for (int step = 0; step < nseg; ++step, ++got) {
      asm volatile("cp.async.wait_group %0;" ::"n"(NST - 2) : "memory");
      __syncwarp();
      // the stage this step's copies go to was read out in the step before
      copy_step();
      asm volatile("cp.async.commit_group;" ::: "memory");
      look_up();
      const uint32_t sK = ring + (got % NST) * STAGE, sV = sK + STEP * ROWB;
      const int key0 = (w.blk + step) * BLOCK + warp * STEP;
      const int valid = w.len - key0;  // keys of this step that exist (may be <= 0)
      if (valid <= 0) continue;
      // ---- S = Q K^T: two tiles of eight keys
      float s[2][4] = {};
      {
        const int mi = lane >> 3, kr = (mi >> 1) * 8 + (lane & 7);  // ldmatrix: key half, piece parity
#pragma unroll
        for (int c = 0; c < PIECES; c += 2) {
          uint32_t r[4];
          ldsm4(r, sK + piece_at<ROWB>(kr, c + (mi & 1)));
          if (E4M3) {  // a piece is 16 columns: one product each
            mma<true>(s[0], qa[c], widen(r[0]), widen(r[0] >> 16));
            mma<true>(s[1], qa[c], widen(r[2]), widen(r[2] >> 16));
            mma<true>(s[0], qa[c + 1], widen(r[1]), widen(r[1] >> 16));
            mma<true>(s[1], qa[c + 1], widen(r[3]), widen(r[3] >> 16));
          } else {
            mma<false>(s[0], qa[c / 2], r[0], r[1]);
            mma<false>(s[1], qa[c / 2], r[2], r[3]);
          }
        }
      }
      // ---- online softmax; a lane has keys 2t, 2t + 1 (+ 8) of rows g, g + 8
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[j][e] = j * 8 + 2 * t + (e & 1) < valid ? s[j][e] * sl2[e >> 1] : -INFINITY;
      if (p.scores) {
#pragma unroll
        for (int z = 0; z < 2; ++z)
          if (g + 8 * z < heads) {
            float* row = p.scores + (q_first + g + 8 * z) * p.pitch + key0 + 2 * t;
            *reinterpret_cast<float2*>(row) = make_float2(s[0][2 * z], s[0][2 * z + 1]);
            *reinterpret_cast<float2*>(row + 8) = make_float2(s[1][2 * z], s[1][2 * z + 1]);
          }
      }
      float alpha[2];
      uint32_t pa[4];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        float mx = fmaxf(fmaxf(s[0][2 * z], s[0][2 * z + 1]), fmaxf(s[1][2 * z], s[1][2 * z + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        mx = fmaxf(mx, m[z]);
        const float ref = mx == -INFINITY ? 0.0f : mx;  // every score so far -inf: P = 0
        alpha[z] = ex2_approx(m[z] - ref);
        m[z] = mx;
        const float p0 = ex2_approx(s[0][2 * z] - ref), p1 = ex2_approx(s[0][2 * z + 1] - ref);
        const float p2 = ex2_approx(s[1][2 * z] - ref), p3 = ex2_approx(s[1][2 * z + 1] - ref);
        l[z] = l[z] * alpha[z] + ((p0 + p1) + (p2 + p3));
        pa[z] = pack2<E4M3>(p0, p1);
        pa[z + 2] = pack2<E4M3>(p2, p3);
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][0] *= alpha[0];
          o[n][1] *= alpha[0];
          o[n][2] *= alpha[1];
          o[n][3] *= alpha[1];
        }
      }
      // ---- O += P V (ldmatrix transposed: keys 0..7 and 8..15 of two pieces)
      {
        const int mi = lane >> 3, kr = (mi & 1) * 8 + (lane & 7);
#pragma unroll
        for (int c = 0; c < PIECES; c += 2) {
          uint32_t r[4];
          ldsm4_t(r, sV + piece_at<ROWB>(kr, c + (mi >> 1)));
          if (E4M3) {
            // bytes (key, col), (key, col + 1), (key + 1, col), (key + 1, col + 1):
            // even columns make one tile, odd ones the next
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t x0 = __byte_perm(r[2 * u], 0, 0x3120), x1 = __byte_perm(r[2 * u + 1], 0, 0x3120);
              mma<true>(o[2 * (c + u)], pa, widen(x0), widen(x1));
              mma<true>(o[2 * (c + u) + 1], pa, widen(x0 >> 16), widen(x1 >> 16));
            }
          } else {
            mma<false>(o[c], pa, r[0], r[1]);
            mma<false>(o[c + 1], pa, r[2], r[3]);
          }
        }
      }
    }

    // ---- join the eight warps
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      l[z] += __shfl_xor_sync(0xffffffffu, l[z], 1);
      l[z] += __shfl_xor_sync(0xffffffffu, l[z], 2);
      if (t == 0) {
        sm_m[warp][g + 8 * z] = m[z];
        sm_l[warp][g + 8 * z] = l[z];
      }
    }
    __syncthreads();
    float M[2], L[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      M[z] = -INFINITY;
#pragma unroll
      for (int v = 0; v < WARPS; ++v) M[z] = fmaxf(M[z], sm_m[v][g + 8 * z]);
      const float ref = M[z] == -INFINITY ? 0.0f : M[z];
      L[z] = 0.0f;
#pragma unroll
      for (int v = 0; v < WARPS; ++v) L[z] += sm_l[v][g + 8 * z] * ex2_approx(sm_m[v][g + 8 * z] - ref);
      const float f0 = ex2_approx(m[z] - ref);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        o[n][2 * z] *= f0;
        o[n][2 * z + 1] *= f0;
      }
    }
    // columns of a lane in tile n: bf16 8 n + 2 t, + 1; 8 bits: tiles 2i and
    // 2i + 1 hold the even and odd columns of piece i, 16 i + 2 (2t, 2t + 1) (+ 1)
#pragma unroll
    for (int half = WARPS / 2; half > 0; half >>= 1) {
      float4* buf = reinterpret_cast<float4*>(join) + (warp % half) * (NT * 32) + lane;
      if (warp >= half && warp < 2 * half)
#pragma unroll
        for (int n = 0; n < NT; ++n) buf[n * 32] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
      __syncthreads();
      if (warp < half)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float4 x = buf[n * 32];
          o[n][0] += x.x;
          o[n][1] += x.y;
          o[n][2] += x.z;
          o[n][3] += x.w;
        }
      __syncthreads();
    }
    if (warp == 0) {
      const bool whole = nseg == w.nblk;
      const float vs = E4M3 ? __ldg(p.c.v_scale + hk) : 1.0f;
      const int slot = part_slot(cta, begin, unit_begin);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int r = g + 8 * z;
        if (r >= heads) continue;
        const float inv = L[z] > 0.0f ? vs / L[z] : L[z] == 0.0f ? 0.0f : L[z];
        float* prow = p.part + ((long long)slot * ROWS + r) * D;
        __nv_bfloat16* orow = p.O + (q_first + r) * D;
#pragma unroll
        for (int n = 0; n < NT; n += E4M3 ? 2 : 1) {
          if (E4M3) {
            // four neighbouring columns: even, odd, even, odd
            const float x0 = o[n][2 * z], x1 = o[n + 1][2 * z], x2 = o[n][2 * z + 1], x3 = o[n + 1][2 * z + 1];
            const int col = 8 * n + 4 * t;
            if (whole)
              *reinterpret_cast<uint2*>(orow + col) = make_uint2(pack2<false>(x0 * inv, x1 * inv), pack2<false>(x2 * inv, x3 * inv));
            else
              *reinterpret_cast<float4*>(prow + col) = make_float4(x0 * vs, x1 * vs, x2 * vs, x3 * vs);
          } else {
            const int col = 8 * n + 2 * t;
            if (whole)
              *reinterpret_cast<uint32_t*>(orow + col) = pack2<false>(o[n][2 * z] * inv, o[n][2 * z + 1] * inv);
            else
              *reinterpret_cast<float2*>(prow + col) = make_float2(o[n][2 * z], o[n][2 * z + 1]);
          }
        }
        if (t == 0) {
          if (whole) p.LSE[q_first + r] = (M[z] + log2f(L[z])) * LN2;
          else p.ml[(long long)slot * ROWS + r] = make_float2(M[z], L[z]);
        }
      }
      // the unit begins here and goes on: the join kernel's block `cta` joins it
      if (lane == 0 && !whole && w.blk == 0) {
        const int last = owner(total, grid, unit_begin + w.nblk - 1);
        p.desc[cta] = make_int4(b, w.hu, slot, last - cta + 1);
      }
    }
    __syncthreads();  // sm_m, sm_l
    w.at += nseg;
    w.blk += nseg;
    if (w.blk == w.nblk) next_unit(work, w);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Block (c, r): row r of the unit that begins in CTA c and ends in another.
template <int D>
__global__ void __launch_bounds__(D) join_kernel(const DecodeParams p, int rows) {
  pdl_wait();
  pdl_next();
  const int c0 = blockIdx.x / rows, r = blockIdx.x % rows, col = threadIdx.x;
  const int4 u = p.desc[c0];
  if (u.x < 0) return;
  const int hk = u.y / p.HB, row0 = (u.y % p.HB) * ROWS;
  if (r >= min(ROWS, p.G - row0)) return;
  // in CTAs after c0 the unit comes first: slot 2 c
  const int first = u.z;
  float M = -INFINITY;
  for (int i = 0; i < u.w; ++i) M = fmaxf(M, p.ml[(long long)(i ? 2 * (c0 + i) : first) * ROWS + r].x);
  const float ref = M == -INFINITY ? 0.0f : M;
  float L = 0.0f, acc = 0.0f;
#pragma unroll 4
  for (int i = 0; i < u.w; ++i) {
    const long long slot = (long long)(i ? 2 * (c0 + i) : first) * ROWS + r;
    const float2 ml = p.ml[slot];
    const float f = ex2_approx(ml.x - ref);
    L = fmaf(ml.y, f, L);
    acc = fmaf(p.part[slot * D + col], f, acc);
  }
  const long long row = (long long)u.x * p.Hq + hk * p.G + row0 + r;
  p.O[row * D + col] = __float2bfloat16(L == 0.0f ? 0.0f : acc / L);
  if (col == 0) p.LSE[row] = (M + log2f(L)) * LN2;
}

// A[b, hk, j] (+)= sum over the group of 2^(s_j - LSE log2 e).
constexpr int W_THREADS = 256;
__global__ void __launch_bounds__(W_THREADS) weights_kernel(const DecodeParams p, float* A, long long a_batch,
                                                            long long a_head, int accumulate, int chunks) {
  pdl_wait();
  pdl_next();
  const int bh = blockIdx.x / chunks, b = bh / p.Hkv, hk = bh % p.Hkv;
  const int len = clamp_len(p.c, __ldg(p.lens + b));
  const long long first = (long long)b * p.Hq + hk * p.G;
  for (long long j = (long long)(blockIdx.x % chunks) * W_THREADS + threadIdx.x; j < len;
       j += (long long)chunks * W_THREADS) {
    float sum = 0.0f;
#pragma unroll 4
    for (int r = 0; r < p.G; ++r)
      sum += ex2_approx(p.scores[(first + r) * p.pitch + j] - __ldg(p.LSE + first + r) * LOG2E);
    float* a = A + b * a_batch + hk * a_head + j;
    *a = accumulate ? *a + sum : sum;
  }
}

static size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct DecodeLayout {
  size_t part, ml, desc, scores, total;
};
static DecodeLayout layout(int B, int Hq, int d, long long cap, bool weights, int grid) {
  DecodeLayout w;
  w.part = 0;
  w.ml = align256((size_t)2 * grid * ROWS * d * sizeof(float));
  w.desc = w.ml + align256((size_t)2 * grid * ROWS * sizeof(float2));
  w.scores = w.desc + align256((size_t)grid * sizeof(int4));
  w.total = w.scores + (weights ? align256((size_t)B * Hq * ((cap + STEP - 1) / STEP * STEP) * sizeof(float)) : 0);
  return w;
}

}  // namespace paged

size_t paged_decode_workspace_bytes(int B, int Hq, int d, long long cap, bool weights) {
  return paged::layout(B, Hq, d, cap, weights, num_sms()).total;
}

template <int D, bool E4M3>
static fa_status launch_d(paged::DecodeParams p, int B, const PagedDecode& a, int grid, cudaStream_t s) {
  using namespace paged;
  constexpr int STAGE = 2 * STEP * (E4M3 ? D : 2 * D);
  constexpr int NST = RING_BYTES / STAGE < 6 ? RING_BYTES / STAGE : 6;
  constexpr int smem = WARPS * NST * STAGE + WARPS / 2 * ROWS * D * 4;
  static_assert(smem + 2048 <= 227 * 1024 && WARPS / 2 * ROWS * D * 4 >= MAX_BATCH * 4, "shared memory");
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(done, (const void*)partial_kernel<D, E4M3>, smem)) return FA_ERR_CUDA;
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
    if (!launch_early(partial_kernel<D, E4M3>, (unsigned)grid, THREADS, smem, s, p)) return FA_ERR_CUDA;
    const int rows = p.G < ROWS ? p.G : ROWS;
    if (!launch_early(join_kernel<D>, (unsigned)(grid * rows), D, 0, s, p, rows)) return FA_ERR_CUDA;
    if (scores) {
      long long chunks = (p.pitch + 4 * W_THREADS - 1) / (4 * W_THREADS);
      if (chunks > 64) chunks = 64;
      if (!launch_early(weights_kernel, (unsigned)(p.B * p.Hkv * chunks), W_THREADS, 0, s, p, a.W + b0 * a.w_batch,
                        a.w_batch, a.w_head, a.accumulate, (int)chunks))
        return FA_ERR_CUDA;
    }
  }
  return FA_OK;
}

fa_status launch_paged_decode(const PagedCache& c, const PagedDecode& a, cudaStream_t s) {
  uint32_t* st = status_word();
  if (!st) return FA_ERR_CUDA;
  const int grid = num_sms();
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
  p.HB = (p.G + paged::ROWS - 1) / paged::ROWS;
  p.sl2 = a.scale_log2;
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.ml = reinterpret_cast<float2*>(ws + w.ml);
  p.desc = reinterpret_cast<int4*>(ws + w.desc);
  p.scores = a.W ? reinterpret_cast<float*>(ws + w.scores) : nullptr;
  p.pitch = (cap + paged::STEP - 1) / paged::STEP * paged::STEP;
  p.O = static_cast<__nv_bfloat16*>(a.O);
  p.LSE = a.LSE;
  p.status = st;
  if (c.elem == 1)
    return c.d == 64 ? launch_d<64, true>(p, c.B, a, grid, s) : launch_d<128, true>(p, c.B, a, grid, s);
  return c.d == 64 ? launch_d<64, false>(p, c.B, a, grid, s) : launch_d<128, false>(p, c.B, a, grid, s);
}

}  // namespace fa
