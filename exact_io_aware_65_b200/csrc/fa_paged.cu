// fa_paged.cu -- writing new keys and values into a paged cache, and evicting
// from it by accumulated attention weight.
//
// Append.  Row t of the packed input belongs to the sequence b with
// cu[b] <= t < cu[b + 1] and goes to position lens[b] + t - cu[b], that is to
// slot position % page_size of page table[b, position / page_size]: a copy in
// bf16, or the nearest 8-bit value (4 exponent bits, 3 of fraction) of
// x / scale, ties to even, magnitudes above the type's largest (448) held
// there.  Bound by the conversion's instructions (8476 tokens of 8 heads of 128
// into 8 bits: 14.4 us, of which HBM needs 8) or by the chain of dependent loads
// that finds the row (a step of 64 sequences: 2.2 us in a graph, most of it the launch).
// Evict.  Bound by the chain of its passes (small caches: 8 us) or by HBM (eight
// caches of 7000-8192 rows cut to 2048, 137 MB read and written: 36 us, 30 in a
// graph, the selection's 11 of them with an eighth of the moves beside it).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <limits.h>
#include <math.h>

#include <type_traits>

#include "fa_internal.h"
#include "sm100.cuh"
#include "paged.cuh"

namespace fa {
namespace paged {

constexpr int APPEND_THREADS = 128;

struct AppendParams {
  Cache c;
  const __nv_bfloat16* K;
  const __nv_bfloat16* V;
  long long k_row, k_head, v_row, v_head;  // strides of the new rows, elements
  const int* cu;
  const int* lens;
  int B, T, Hkv;
  Divider page;
  uint32_t* status;
};

// The sequence of packed row t: the last b with cu[b] <= t (a warp looks at 32
// entries at a time); -1 if none.  Any cu gives an answer in [-1, B).
__device__ __forceinline__ int find_sequence(const int* cu, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // candidates [lo, lo + n)
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, i < lo + n && __ldg(cu + min(i, B - 1)) <= t);
    if (le == 0) return lo - 1;
    const int last = 31 - __clz(le);
    const int end = min(lo + n, lo + (last + 1) * step);
    lo += last * step + 1;
    n = end - lo;
  }
  return lo - 1;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Keeps x within +-top; NaN stays.
__device__ __forceinline__ float hold(float x, float top) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(top));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(r), "f"(-top));
  return r;
}

// x / s from r, the correctly rounded 1 / s: with the remainder of the first
// quotient, the second is x / s correctly rounded but for rare last bits
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000",
// 1990, proves it for a first quotient within a unit of its last place; where it
// is exact, as on the borders between 8-bit values, so is the second).  For
// scales between 2^-60 and 2^60 and |x| <= 512 s nothing overflows on the way,
// and what underflows rounds to zero in 8 bits anyway.
__device__ __forceinline__ float divide(float x, float s, float r) {
  const float q = __fmul_rn(x, r);
  return q == 0.0f ? q : __fmaf_rn(__fmaf_rn(-q, s, x), r, q);  // (a zero keeps its sign)
}

// Eight bf16 to eight 8-bit values of x / s.
__device__ __forceinline__ uint2 encode(const uint4& x, float s) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t q[4];
  if (s > 0x1p-60f && s < 0x1p60f) {
    const float r = __frcp_rn(s), top = 512.0f * s;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      q[e] = e4m3x2(divide(hold(__uint_as_float(w[e] << 16), top), s, r),
                    divide(hold(__uint_as_float(w[e] & 0xffff0000u), top), s, r));
  } else {
#pragma unroll 1
    for (int e = 0; e < 4; ++e)
      q[e] = e4m3x2(__fdiv_rn(__uint_as_float(w[e] << 16), s), __fdiv_rn(__uint_as_float(w[e] & 0xffff0000u), s));
  }
  return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}

// A warp per (token, K or V): 16 bytes of the input a lane, four pieces of it in
// flight while the row's place is looked up (a chain of dependent loads: the
// sequence, its length, the page).
template <int D, bool E4M3>
__global__ void __launch_bounds__(APPEND_THREADS) append_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * (APPEND_THREADS / 32) + (threadIdx.x >> 5);
  const int t = (int)(unit >> 1), kv = (int)(unit & 1);
  if (t >= p.T) return;
  constexpr int CH = D / 8;  // 16-byte pieces of a head's row
  constexpr int N = 4;
  const int pieces = p.Hkv * CH;
  const __nv_bfloat16* src = kv ? p.V + t * p.v_row : p.K + t * p.k_row;
  const long long src_head = kv ? p.v_head : p.k_head;
  const float* scale = kv ? p.c.v_scale : p.c.k_scale;
  uint4 x[N];
  float s[N];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = i0 + 32 * k, h = i / CH, c = i % CH;
      if (i < pieces) {
        x[k] = *reinterpret_cast<const uint4*>(src + h * src_head + c * 8);
        if (E4M3) s[k] = __ldg(scale + h);
      }
    }
  };
  load(lane);
  const int b = find_sequence(p.cu, p.B, t);
  if (b < 0 || t >= __ldg(p.cu + b + 1)) return;  // behind the last sequence
  const int held = __ldg(p.lens + b);
  const long long pos = held + (long long)t - __ldg(p.cu + b);
  long long off = -1;
  if (held >= 0) {
    // (the table spans at most 2^30 positions)
    const int at = (int)min(pos, (long long)INT_MAX), i = p.page(at);
    off = row_offset(p.c, page_of(p.c, p.c.table + b * p.c.table_stride, at, i), at - i * p.c.page_size);
  }
  if (off < 0) {
    if (lane == 0) bad_page(p.status);
    return;
  }
  uint8_t* dst = (kv ? p.c.V : p.c.K) + off;
  for (int i0 = lane; i0 < pieces; i0 += 32 * N) {
    if (i0 != lane) load(i0);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = i0 + 32 * k, h = i / CH, c = i % CH;
      if (i >= pieces) break;
      if (E4M3) {
        *reinterpret_cast<uint2*>(dst + h * p.c.head_stride + c * 8) = encode(x[k], s[k]);
      } else {
        *reinterpret_cast<uint4*>(dst + h * p.c.head_stride + c * 16) = x[k];
      }
    }
  }
}

// ------------------------------------------------------------------- evict ---
// Of a sequence's n rows and for each head: the last `recent`, and of those
// before them the budget - recent with the largest weights (equal weights: the
// lowest position; NaN counts as less than every number), kept in their order.
// Selection runs on the weights' bits mapped so that unsigned order is the
// order of the numbers: histograms of 11, 11 and 10 bits narrow down the
// smallest key that stays and how many of its equals do (one histogram is
// enough where all of its last bin stay), and two more passes count and place
// what stays.  One CTA per (sequence, head); the passes after the first find the
// keys in shared memory when they fit.  11 bits are a float's sign, exponent and
// two bits of fraction: weights spread over a few powers of two share no bin
// with most lanes of a warp, and its additions go to shared memory one by one
// without waiting for each other (8 bits at a time needed the lanes of equal
// digit matched first: 38.7 us against 13, then, for 64 heads of 7000-8192 keys).
constexpr int SEL_SMEM_KEYS = 48 * 1024;  // 192 KB
constexpr int SEL_BINS = 2048;

struct EvictParams {
  Cache c;         // source rows
  const int* lens;
  const int* table_out;
  long long table_out_stride;
  const float* W;     // [B, Hkv, *], rows w_stride apart (heads), B * w_batch
  long long w_head, w_batch;
  float* Wout;
  long long wo_head, wo_batch;
  int wo_len;         // length of Wout's rows
  int* kept;          // [B, Hkv, budget]
  int* lens_out;      // [B]
  int B, Hkv, budget, recent, max_out;
  int chunks;         // blocks of the move kernel for one (sequence, head)
  int early;          // rows of each that move while others are selected, at most
  Divider page;
  uint32_t* status;
};

// Order of the floats as unsigned numbers, -0 = +0, NaN lowest.
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  if (w != w) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The rows that stay in any case are the last ones; this many of them, kept rows
// [left - n, left), need no selection before they move.  (p.early <= recent.)
__device__ __forceinline__ int early_rows(const EvictParams& p, int left) { return min(p.early, left); }

// Moves kept rows [r0, r0 + step) of head h of sequence b, then their weights:
// a group of ROWB / 16 lanes per row and pool, ROWS rows of K and of V in
// flight per lane.  Row r, of position pos_of(r), goes to position r of the table
// of destination pages.  (0 <= pos_of(r) < max_pages * page_size for r < left: the
// selection sees to that, whatever happens to lens and weights meanwhile.  A test
// here instead cost 0.5-1.4 of 30 us.)
template <int ROWB, int ROWS, class Pos>
__device__ __forceinline__ void move_rows(const EvictParams& p, int b, int h, int left, int r0, int step, Pos pos_of) {
  constexpr int LPR = ROWB / 16;
  const int groups = blockDim.x / LPR;
  const int sub = threadIdx.x / LPR, piece = threadIdx.x % LPR;
  const int end = min(left, r0 + step);
  for (int r1 = r0; r1 < end; r1 += groups * ROWS) {
    uint4 k[ROWS], v[ROWS];
    long long dst[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int r = r1 + i * groups + sub;
      dst[i] = -1;
      if (r < end) {
        // (rows past the destination table were refused)
        const int pos = pos_of(r), from = p.page(pos), to = p.page(r);
        const int page = to < p.max_out ? __ldg(p.table_out + b * p.table_out_stride + to) : -1;
        const long long src =
            row_offset(p.c, __ldg(p.c.table + b * p.c.table_stride + from), pos - from * p.c.page_size);
        dst[i] = row_offset(p.c, page, r - to * p.c.page_size);
        if (src < 0 || dst[i] < 0) {
          bad_page(p.status);
          dst[i] = -1;
        } else {
          const long long at = h * p.c.head_stride + piece * 16;
          k[i] = *reinterpret_cast<const uint4*>(p.c.K + src + at);
          v[i] = *reinterpret_cast<const uint4*>(p.c.V + src + at);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (dst[i] < 0) continue;
      const long long at = dst[i] + h * p.c.head_stride + piece * 16;
      *reinterpret_cast<uint4*>(p.c.K + at) = k[i];
      *reinterpret_cast<uint4*>(p.c.V + at) = v[i];
    }
  }
  const float* w = p.W + b * p.w_batch + h * p.w_head;
  float* wo = p.Wout + b * p.wo_batch + h * p.wo_head;
  for (int r = r0 + threadIdx.x; r < end; r += blockDim.x) wo[r] = __ldg(w + pos_of(r));
}

// The sum of what the warps before this one put into v[32].
template <typename T>
__device__ __forceinline__ T sum_before(const T* v, int warp, int lane) {
  return __reduce_add_sync(0xffffffffu, lane < warp ? v[lane] : T(0));
}

// The positions that stay; the CTA's (sequence, head) in p.kept, and how many.
__device__ __forceinline__ int select_rows(const EvictParams& p, uint32_t* keys) {
  __shared__ uint32_t hist[SEL_BINS];
  __shared__ int above_w[32];
  __shared__ uint32_t both_w[32];
  __shared__ uint32_t sh_digit;
  __shared__ int sh_need, sh_count;
  const int bh = blockIdx.x, b = bh / p.Hkv, h = bh % p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = clamp_len(p.c, __ldg(p.lens + b));
  const int left = min(n, p.budget);
  int* kept = p.kept + (long long)bh * p.budget;
  if (h == 0 && tid == 0) p.lens_out[b] = left;
  for (int i = left + tid; i < p.budget; i += SEL_THREADS) kept[i] = -1;
  if (n <= p.budget) {
    for (int i = tid; i < n; i += SEL_THREADS) kept[i] = i;
    return left;
  }
  const int old = n - p.recent, pick = p.budget - p.recent;  // old > pick >= 0
  for (int i = tid; i < p.recent; i += SEL_THREADS) kept[pick + i] = old + i;
  if (pick == 0) return left;
  const float* w = p.W + b * p.w_batch + h * p.w_head;
  const bool cached = old <= SEL_SMEM_KEYS;
  // the keys from position i on, four a load where i is a multiple of 4 (any
  // value past the last one)
  auto keys_at = [&](int i, auto& k) {
    constexpr int N = sizeof(k) / 4;
    if (cached && N == 1) {
      k[0] = i < old ? keys[i] : 0u;
    } else if (cached) {
#pragma unroll
      for (int u = 0; u < N / 4; ++u) {
        const uint4 x = i + 4 * u < old ? *reinterpret_cast<const uint4*>(keys + i + 4 * u) : make_uint4(0u, 0u, 0u, 0u);
        k[4 * u] = x.x;
        k[4 * u + 1] = x.y;
        k[4 * u + 2] = x.z;
        k[4 * u + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int u = 0; u < N; ++u) k[u] = i + u < old ? order_key(__ldg(w + i + u)) : 0u;
    }
  };
  hist[tid] = hist[tid + SEL_THREADS] = 0u;
  __syncthreads();
  auto count = [&](uint32_t digit, bool in) {
    // one addition for a warp of one digit, else one a lane
    const unsigned who = __ballot_sync(0xffffffffu, in);
    if (who == 0) return;
    const uint32_t first = __shfl_sync(0xffffffffu, digit, __ffs(who) - 1);
    if (__all_sync(0xffffffffu, !in || digit == first)) {
      if (lane == 0) atomicAdd(&hist[first], (uint32_t)__popc(who));
    } else if (in) {
      atomicAdd(&hist[digit], 1u);
    }
  };
  // the pick-th largest key: its upper bits `digits`, and how many of the keys
  // that share these stay
  uint32_t digits = 0;
  int need = pick, shift = 21;
  for (;;) {
    if (shift == 21) {
      constexpr int U = 8;  // loads in flight
      for (int i0 = warp * 32; i0 < old; i0 += SEL_THREADS * U) {
        float v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * SEL_THREADS + lane;
          v[u] = i < old ? __ldg(w + i) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * SEL_THREADS + lane;
          if (i - lane >= old) break;
          const uint32_t k = order_key(v[u]);
          if (cached && i < old) keys[i] = k;
          count(k >> 21, i < old);
        }
      }
    } else {
      const int up = shift == 10 ? 21 : 10;  // bits already known
      auto count_keys = [&](auto per) {
        constexpr int N = decltype(per)::value;
        for (int i0 = warp * 32 * N; i0 < old; i0 += SEL_THREADS * N) {
          const int i = i0 + N * lane;
          uint32_t k[N];
          keys_at(i, k);
          bool in[N], all = true;
#pragma unroll
          for (int u = 0; u < N; ++u) {
            in[u] = i + u < old && (k[u] >> up) == digits;
            k[u] = shift == 10 ? (k[u] >> 10) & 2047u : k[u] & 1023u;
            all = all && in[u] && k[u] == k[0];
          }
          const uint32_t first = __shfl_sync(0xffffffffu, k[0], 0);
          if (__all_sync(0xffffffffu, all && k[0] == first)) {
            if (lane == 0) atomicAdd(&hist[first], 32u * N);
            continue;
          }
#pragma unroll
          for (int u = 0; u < N; ++u)
            if (in[u]) atomicAdd(&hist[k[u]], 1u);
        }
      };
      if (old <= SEL_THREADS) count_keys(std::integral_constant<int, 1>());
      else count_keys(std::integral_constant<int, 4>());
    }
    __syncthreads();
    // thread T has the bins 2047 - 2 T and 2046 - 2 T, so that threads go down
    const int top = SEL_BINS - 1 - 2 * tid;
    const uint32_t c0 = hist[top], c1 = hist[top - 1];
    uint32_t before = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += v;
    }
    if (lane == 31) above_w[warp] = (int)before;
    before -= c0 + c1;
    __syncthreads();
    hist[top] = hist[top - 1] = 0u;  // for the next digits
    before += (uint32_t)sum_before(above_w, warp, lane);
    if (before < (uint32_t)need && before + c0 + c1 >= (uint32_t)need) {  // one thread
      const bool second = before + c0 < (uint32_t)need;
      sh_digit = (uint32_t)(second ? top - 1 : top);
      sh_need = need - (int)(second ? before + c0 : before);
      sh_count = (int)(second ? c1 : c0);
    }
    __syncthreads();
    digits = shift == 21 ? sh_digit : shift == 10 ? (digits << 11) | sh_digit : (digits << 10) | sh_digit;
    need = sh_need;
    if (shift == 0 || need == sh_count) break;
    shift = shift == 21 ? 10 : 0;
  }
  // Keys above `digits` stay, and the first `need` that share them.  A thread
  // takes N neighbouring positions at a time, and a sum over the block of both
  // counts (at most 8192 each, in halves of a word) gives it its place.  N = 8
  // where there are that many: the SM's four schedulers issue for 32 warps, and
  // with a position a lane, placed by ballots, this took 6300 of the selection's
  // 21000 cycles for 7500 keys.  Keys that do not fit on chip are read again here;
  // where they are no longer those that were counted, what is placed still stays
  // within the row, and the row is filled.
  auto place = [&](auto per, auto again) {
    constexpr int N = decltype(per)::value;
    constexpr bool AGAIN = decltype(again)::value;
    int at0 = 0, tie0 = 0;  // what stays of the positions before these, and their ties
    for (int i0 = 0; i0 < old; i0 += SEL_THREADS * N) {
      const int i = i0 + N * tid;
      uint32_t k[N];
      keys_at(i, k);
      uint32_t over = 0, tie = 0;
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const uint32_t x = k[u] >> shift;
        over |= (uint32_t)(i + u < old && x > digits) << u;
        tie |= (uint32_t)(i + u < old && x == digits) << u;
      }
      const uint32_t mine = (uint32_t)__popc(over) | (uint32_t)__popc(tie) << 16;
      uint32_t before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      if (i0 > 0) __syncthreads();  // both_w of the last round has been read
      if (lane == 31) both_w[warp] = before;
      __syncthreads();
      before += sum_before(both_w, warp, lane) - mine;
      int ties = tie0 + (int)(before >> 16);
      int at = at0 + (int)(before & 0xffffu) + min(ties, need) - min(tie0, need);
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const bool is_tie = (tie >> u) & 1u;
        if ((((over >> u) & 1u) || (is_tie && ties < need)) && (!AGAIN || at < pick)) kept[at++] = i + u;
        ties += is_tie;
      }
      if (AGAIN || i0 + SEL_THREADS * N < old) {
        const uint32_t all = sum_before(both_w, 32, lane);
        at0 += (int)(all & 0xffffu) + min(tie0 + (int)(all >> 16), need) - min(tie0, need);
        tie0 += (int)(all >> 16);
      }
    }
    if (AGAIN) {
      for (int i = at0 + tid; i < pick; i += SEL_THREADS) kept[i] = 0;
    }
  };
  if (old <= SEL_THREADS) place(std::integral_constant<int, 1>(), std::false_type());
  else if (cached) place(std::integral_constant<int, 8>(), std::false_type());
  else place(std::integral_constant<int, 8>(), std::true_type());
  return left;
}

// FUSED: the CTA moves its rows too.  Else the CTAs behind those of the (sequence,
// head)s, on SMs that had nothing to do, move the rows that need no selection.
template <int ROWB, bool FUSED>
__global__ void __launch_bounds__(SEL_THREADS, 1) select_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  const int heads = p.B * p.Hkv;
  if (!FUSED && (int)blockIdx.x >= heads) {
    constexpr int PER = SEL_THREADS / (ROWB / 16) * SEL_ROWS;
    const int chunks = (p.early + PER - 1) / PER;
    for (int u = (int)blockIdx.x - heads; u < heads * chunks; u += (int)gridDim.x - heads) {
      const int b = u / chunks / p.Hkv, h = u / chunks % p.Hkv;
      const int n = clamp_len(p.c, __ldg(p.lens + b)), left = min(n, p.budget);
      move_rows<ROWB, SEL_ROWS>(p, b, h, left, left - early_rows(p, left) + u % chunks * PER, PER,
                      [&](int r) { return n - left + r; });
    }
    return;
  }
  const int left = select_rows(p, keys);
  if constexpr (FUSED) {
    __syncthreads();  // kept
    const int b = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
    const int* kept = p.kept + (long long)blockIdx.x * p.budget;
    move_rows<ROWB, SEL_ROWS>(p, b, h, left, 0, left, [&](int r) { return kept[r]; });
    float* wo = p.Wout + b * p.wo_batch + h * p.wo_head;
    for (int r = left + threadIdx.x; r < p.wo_len; r += SEL_THREADS) wo[r] = 0.0f;
  }
}

// The other rows: p.chunks blocks a (sequence, head).  Eight blocks on an SM with two
// rows a lane: one block's chain of positions and pages hides behind the others'
// rows (four rows a lane and four blocks: 34.3 us for the call's 30.9, then).
constexpr int MOVE_THREADS = 256, MOVE_ROWS = 2;
template <int ROWB>
__global__ void __launch_bounds__(MOVE_THREADS, 8) move_kernel(const EvictParams p) {
  constexpr int PER = MOVE_THREADS / (ROWB / 16) * MOVE_ROWS;
  const int bh = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
  const int b = bh / p.Hkv, h = bh % p.Hkv;
  const int left = p.lens_out[b];  // of the selection, as the positions are
  const int* kept = p.kept + (long long)bh * p.budget;
  move_rows<ROWB, MOVE_ROWS>(p, b, h, left - early_rows(p, left), chunk * PER, PER, [&](int r) { return kept[r]; });
  float* wo = p.Wout + b * p.wo_batch + h * p.wo_head;
  // the rest of the weights' row, shared by the blocks, is zero
  for (long long r = left + (long long)chunk * MOVE_THREADS + threadIdx.x; r < p.wo_len;
       r += (long long)p.chunks * MOVE_THREADS)
    wo[r] = 0.0f;
}

}  // namespace paged

fa_status launch_paged_append(const PagedCache& c, const Rows& K, const Rows& V, const int* cu, const int* lens, int T,
                              cudaStream_t s) {
  uint32_t* st = status_word();
  if (!st) return FA_ERR_CUDA;
  paged::AppendParams p;
  p.c = cache_view(c);
  p.K = static_cast<const __nv_bfloat16*>(K.data);
  p.V = static_cast<const __nv_bfloat16*>(V.data);
  p.k_row = K.row_stride;
  p.k_head = K.head_stride;
  p.v_row = V.row_stride;
  p.v_head = V.head_stride;
  p.cu = cu;
  p.lens = lens;
  p.B = c.B;
  p.T = T;
  p.Hkv = c.Hkv;
  p.page = paged::make_divider(c.page_size);
  p.status = st;
  constexpr int WARPS = paged::APPEND_THREADS / 32;
  const unsigned grid = (unsigned)((2LL * T + WARPS - 1) / WARPS);
  const bool e4m3 = c.elem == 1;
  auto* kern = c.d == 64 ? (e4m3 ? paged::append_kernel<64, true> : paged::append_kernel<64, false>)
                         : (e4m3 ? paged::append_kernel<128, true> : paged::append_kernel<128, false>);
  return launch(kern, grid, paged::APPEND_THREADS, 0, s, p) ? FA_OK : FA_ERR_CUDA;
}

fa_status launch_paged_evict(const PagedCache& c, const Evict& e, cudaStream_t s) {
  uint32_t* st = status_word();
  if (!st) return FA_ERR_CUDA;
  paged::EvictParams p;
  p.c = cache_view(c);
  p.lens = e.lens;
  p.table_out = e.table_out;
  p.table_out_stride = e.table_out_stride;
  p.W = e.W;
  p.w_head = e.w_head;
  p.w_batch = e.w_batch;
  p.Wout = e.Wout;
  p.wo_head = e.wo_head;
  p.wo_batch = e.wo_batch;
  p.wo_len = e.wo_len;
  p.kept = e.kept;
  p.lens_out = e.lens_out;
  p.B = c.B;
  p.Hkv = c.Hkv;
  p.budget = e.budget;
  p.recent = e.recent;
  p.max_out = e.max_out;
  p.page = paged::make_divider(c.page_size);
  p.status = st;
  // shared memory for the keys a head can have to choose from, when they fit
  const long long most = (long long)c.max_pages * c.page_size - e.recent;
  const int smem = 4 * (int)(most < 0 ? 0 : most < paged::SEL_SMEM_KEYS ? (most + 3) / 4 * 4 : paged::SEL_SMEM_KEYS);
  // A CTA moves the rows it has selected where that is little (sequences
  // of 500 and 1000 rows cut to 250: 10.3 against 13.3 us); else a second kernel
  // moves them with all SMs, also where every SM has a CTA: a selecting CTA fills its
  // SM, and the last ones then moved alone (caches of 4000-8192 rows cut to 2048,
  // 152 heads: 70 us, 91 in the selecting CTAs; 200: 87, 93; 256: 105, 107; 320: 132,
  // 146; of 900-1800 rows cut to 450, 256 heads: 33, 32).
  const int rowb = c.d * c.elem;
  const long long rows = most + e.recent < e.budget ? most + e.recent : e.budget;
  const bool fused = 4 * rows * rowb <= 256 * 1024;
  auto run = [&](auto width) -> bool {
    constexpr int W = decltype(width)::value;
    static std::atomic<uint64_t> done[2];
    auto kern = fused ? paged::select_kernel<W, true> : paged::select_kernel<W, false>;
    const int heads = c.B * c.Hkv, idle = num_sms() - heads;
    p.early = fused ? 0 : paged::early_most(heads, idle, e.recent, W);
    if (!allow_smem(done[fused], (const void*)kern, 4 * paged::SEL_SMEM_KEYS) ||
        !launch(kern, (unsigned)(heads + (p.early > 0 ? idle : 0)), paged::SEL_THREADS, smem, s, p))
      return false;
    if (fused) return true;
    constexpr int PER = paged::MOVE_THREADS / (W / 16) * paged::MOVE_ROWS;
    p.chunks = (e.budget + PER - 1) / PER;
    return launch(paged::move_kernel<W>, (unsigned)(heads * p.chunks), paged::MOVE_THREADS, 0, s, p);
  };
  const bool ok = rowb == 64    ? run(std::integral_constant<int, 64>())
                  : rowb == 128 ? run(std::integral_constant<int, 128>())
                                : run(std::integral_constant<int, 256>());
  return ok ? FA_OK : FA_ERR_CUDA;
}

}  // namespace fa
