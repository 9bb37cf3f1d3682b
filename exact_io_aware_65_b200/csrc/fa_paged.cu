// fa_paged.cu -- writing new keys and values into a paged cache, and evicting
// from it by accumulated attention weight.
//
// Append.  Row t of the packed input belongs to the sequence b with
// cu[b] <= t < cu[b + 1] and goes to position lens[b] + t - cu[b], that is to
// slot position % page_size of page table[b, position / page_size]: a copy in
// bf16, or the nearest 8-bit value (4 exponent bits, 3 of fraction) of
// x / scale, ties to even, magnitudes above the type's largest (448) held
// there.  Bound by HBM (prompts) or by the chain of dependent loads that finds
// the row (single tokens).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math.h>

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

// A warp per (token, K or V): 16 bytes of the input a lane.
template <int D, bool E4M3>
__global__ void __launch_bounds__(APPEND_THREADS) append_kernel(const AppendParams p) {
  pdl_wait();
  pdl_next();
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * (APPEND_THREADS / 32) + (threadIdx.x >> 5);
  const int t = (int)(unit >> 1), kv = (int)(unit & 1);
  if (t >= p.T) return;
  const int b = find_sequence(p.cu, p.B, t);
  if (b < 0 || t >= __ldg(p.cu + b + 1)) return;  // behind the last sequence
  const int held = __ldg(p.lens + b);
  const long long pos = held + (long long)t - __ldg(p.cu + b);
  const long long off = held < 0 ? -1 : row_offset(p.c, page_of(p.c, b, pos), (int)(pos % p.c.page_size));
  if (off < 0) {
    if (lane == 0) bad_page(p.status);
    return;
  }
  constexpr int CH = D / 8;  // 16-byte pieces of a head's row
  const __nv_bfloat16* src = kv ? p.V + t * p.v_row : p.K + t * p.k_row;
  const long long src_head = kv ? p.v_head : p.k_head;
  uint8_t* dst = (kv ? p.c.V : p.c.K) + off;
  const float* scale = kv ? p.c.v_scale : p.c.k_scale;
#pragma unroll 4
  for (int i = lane; i < p.Hkv * CH; i += 32) {
    const int h = i / CH, c = i % CH;
    const uint4 x = *reinterpret_cast<const uint4*>(src + h * src_head + c * 8);
    if (E4M3) {
      const float s = __ldg(scale + h);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        q[e] = e4m3x2(__fdiv_rn(__uint_as_float(w[e] << 16), s), __fdiv_rn(__uint_as_float(w[e] & 0xffff0000u), s));
      *reinterpret_cast<uint2*>(dst + h * p.c.head_stride + c * 8) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
    } else {
      *reinterpret_cast<uint4*>(dst + h * p.c.head_stride + c * 16) = x;
    }
  }
}

// ------------------------------------------------------------------- evict ---
// Of a sequence's n rows and for each head: the last `recent`, and of those
// before them the budget - recent with the largest weights (equal weights: the
// lowest position; NaN counts as less than every number), kept in their order.
// Selection runs on the weights' bits mapped so that unsigned order is the
// order of the numbers: four passes of an 8-bit histogram narrow down the
// smallest key that stays and how many of its equals do, and two more passes
// count and place what stays.  One CTA per (sequence, head); the passes after
// the first find the keys in shared memory when they fit.
constexpr int SEL_THREADS = 1024;
constexpr int SEL_SMEM_KEYS = 48 * 1024;  // 192 KB

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
  uint32_t* status;
};

// Order of the floats as unsigned numbers, -0 = +0, NaN lowest.
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  if (w != w) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(SEL_THREADS, 1) select_kernel(const EvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[256];
  __shared__ int above_w[32], tie_w[32];
  __shared__ uint32_t sh_prefix;
  __shared__ int sh_need;
  pdl_wait();
  pdl_next();
  const int bh = blockIdx.x, b = bh / p.Hkv, h = bh % p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = clamp_len(p.c, __ldg(p.lens + b));
  const int left = min(n, p.budget);
  int* kept = p.kept + (long long)bh * p.budget;
  if (h == 0 && tid == 0) p.lens_out[b] = left;
  for (int i = left + tid; i < p.budget; i += SEL_THREADS) kept[i] = -1;
  if (n <= p.budget) {
    for (int i = tid; i < n; i += SEL_THREADS) kept[i] = i;
    return;
  }
  const int old = n - p.recent, pick = p.budget - p.recent;  // old > pick >= 0
  for (int i = tid; i < p.recent; i += SEL_THREADS) kept[pick + i] = old + i;
  if (pick == 0) return;
  const float* w = p.W + b * p.w_batch + h * p.w_head;
  const bool cached = old <= SEL_SMEM_KEYS;
  auto key_at = [&](int i) { return cached ? keys[i] : order_key(__ldg(w + i)); };
  if (cached)
    for (int i = tid; i < old; i += SEL_THREADS) keys[i] = order_key(__ldg(w + i));
  // the pick-th largest key, eight bits at a time
  uint32_t prefix = 0;
  int need = pick;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0u;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int i0 = warp * 32; i0 < old; i0 += SEL_THREADS) {
      const int i = i0 + lane;
      const uint32_t k = i < old ? key_at(i) : 0u;
      const bool in = i < old && (k & mask) == prefix;
      const uint32_t digit = (k >> shift) & 255u;
      // one addition for all lanes of equal digit
      const unsigned peers = __match_any_sync(0xffffffffu, in ? digit : 256u + lane);
      if (in && lane == __ffs(peers) - 1) atomicAdd(&hist[digit], (uint32_t)__popc(peers));
    }
    __syncthreads();
    if (warp == 0) {
      // lane L holds the digits 255 - 8L .. 248 - 8L, so that lanes go down
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += c[e] = hist[255 - 8 * lane - e];
      uint32_t before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      before -= sum;
      if (before < (uint32_t)need && before + sum >= (uint32_t)need) {  // one lane
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (before < (uint32_t)need && before + c[e] >= (uint32_t)need) {
            sh_prefix = prefix | ((uint32_t)(255 - 8 * lane - e) << shift);
            sh_need = need - (int)before;
            break;
          }
          before += c[e];
        }
      }
    }
    __syncthreads();
    prefix = sh_prefix;
    need = sh_need;
  }
  // Keys above `prefix` stay, and the first `need` that equal it.  Each warp
  // takes a stretch of positions, counts, and then places.
  const int per = ((old + 31) / 32 + 31) / 32 * 32;
  const int i0 = min(old, warp * per), i1 = min(old, i0 + per);
  int above = 0, ties = 0;
  for (int i = i0 + lane; i - lane < i1; i += 32) {
    const uint32_t k = i < i1 ? key_at(i) : 0u;
    above += __popc(__ballot_sync(0xffffffffu, i < i1 && k > prefix));
    ties += __popc(__ballot_sync(0xffffffffu, i < i1 && k == prefix));
  }
  if (lane == 0) {
    above_w[warp] = above;
    tie_w[warp] = ties;
  }
  __syncthreads();
  int at = 0, tie_at = 0;  // what the warps before keep, and how many ties they have
  for (int v = 0; v < warp; ++v) {
    at += above_w[v];
    tie_at += tie_w[v];
  }
  at += min(tie_at, need);
  const unsigned before_me = (1u << lane) - 1u;
  for (int i = i0 + lane; i - lane < i1; i += 32) {
    const uint32_t k = i < i1 ? key_at(i) : 0u;
    const unsigned tie = __ballot_sync(0xffffffffu, i < i1 && k == prefix);
    const bool stays = i < i1 && (k > prefix || (k == prefix && tie_at + __popc(tie & before_me) < need));
    const unsigned keep = __ballot_sync(0xffffffffu, stays);
    if (stays) kept[at + __popc(keep & before_me)] = i;
    at += __popc(keep);
    tie_at += __popc(tie);
  }
}

// Moves the kept rows: a group of ROWB / 16 lanes per row and pool, four rows
// of K and of V in flight per lane.  Row r goes to position r of the table of
// destination pages.
constexpr int MOVE_THREADS = 256;
constexpr int MOVE_ROWS = 4;

template <int ROWB>
__global__ void __launch_bounds__(MOVE_THREADS) move_kernel(const EvictParams p) {
  pdl_wait();
  pdl_next();
  constexpr int LPR = ROWB / 16, GROUPS = MOVE_THREADS / LPR, PER = GROUPS * MOVE_ROWS;
  const int bh = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
  const int b = bh / p.Hkv, h = bh % p.Hkv;
  const int left = min(clamp_len(p.c, __ldg(p.lens + b)), p.budget);
  const int sub = threadIdx.x / LPR, piece = threadIdx.x % LPR;
  const int* kept = p.kept + (long long)bh * p.budget;
  const int r0 = chunk * PER;
  uint4 k[MOVE_ROWS], v[MOVE_ROWS];
  long long dst[MOVE_ROWS];
#pragma unroll
  for (int i = 0; i < MOVE_ROWS; ++i) {
    const int r = r0 + i * GROUPS + sub;
    dst[i] = -1;
    if (r < left) {
      const int pos = __ldg(kept + r);
      const long long src = row_offset(p.c, page_of(p.c, b, pos), pos % p.c.page_size);
      const int slot = r / p.c.page_size;
      const int page = slot < p.max_out ? __ldg(p.table_out + b * p.table_out_stride + slot) : -1;
      dst[i] = row_offset(p.c, page, r % p.c.page_size);
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
  for (int i = 0; i < MOVE_ROWS; ++i) {
    if (dst[i] < 0) continue;
    const long long at = dst[i] + h * p.c.head_stride + piece * 16;
    *reinterpret_cast<uint4*>(p.c.K + at) = k[i];
    *reinterpret_cast<uint4*>(p.c.V + at) = v[i];
  }
  // the weights of these rows; the rest of the row, shared by the blocks, is zero
  const float* w = p.W + b * p.w_batch + h * p.w_head;
  float* wo = p.Wout + b * p.wo_batch + h * p.wo_head;
  for (int r = r0 + threadIdx.x; r < min(left, r0 + PER); r += MOVE_THREADS) wo[r] = __ldg(w + __ldg(kept + r));
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
  p.status = st;
  constexpr int WARPS = paged::APPEND_THREADS / 32;
  const unsigned grid = (unsigned)((2LL * T + WARPS - 1) / WARPS);
  const bool e4m3 = c.elem == 1;
  auto* kern = c.d == 64 ? (e4m3 ? paged::append_kernel<64, true> : paged::append_kernel<64, false>)
                         : (e4m3 ? paged::append_kernel<128, true> : paged::append_kernel<128, false>);
  return launch_early(kern, grid, paged::APPEND_THREADS, 0, s, p) ? FA_OK : FA_ERR_CUDA;
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
  p.status = st;
  // shared memory for the keys a head can have to choose from, when they fit
  const long long most = (long long)c.max_pages * c.page_size - e.recent;
  const int smem = 4 * (int)(most < 0 ? 0 : most < paged::SEL_SMEM_KEYS ? most : paged::SEL_SMEM_KEYS);
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(done, (const void*)paged::select_kernel, 4 * paged::SEL_SMEM_KEYS) ||
      !launch_early(paged::select_kernel, (unsigned)(c.B * c.Hkv), paged::SEL_THREADS, smem, s, p))
    return FA_ERR_CUDA;
  bool ok;
  auto move = [&](auto kern, int rowb) {
    const int per = paged::MOVE_THREADS / (rowb / 16) * paged::MOVE_ROWS;
    p.chunks = (e.budget + per - 1) / per;
    ok = launch_early(kern, (unsigned)(c.B * c.Hkv * p.chunks), paged::MOVE_THREADS, 0, s, p);
  };
  const int rowb = c.d * c.elem;
  if (rowb == 64) move(paged::move_kernel<64>, 64);
  else if (rowb == 128) move(paged::move_kernel<128>, 128);
  else move(paged::move_kernel<256>, 256);
  return ok ? FA_OK : FA_ERR_CUDA;
}

}  // namespace fa
