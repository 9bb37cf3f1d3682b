// fa_api.cu -- the extern "C" entry points of libfa.so: argument checks,
// TMA map encoding, the device status word, and dispatch to the kernels.
#include <cudaTypedefs.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include "fa.h"
#include "fa_internal.h"
#include "sm100.cuh"

namespace fa {

__device__ uint32_t g_status = 0;

uint32_t* status_word() {
  static std::atomic<uint32_t*> addr[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  uint32_t* known = addr[dev].load(std::memory_order_acquire);
  if (known) return known;
  void* p = nullptr;  // (two threads may both look it up: they find the same)
  if (cudaGetSymbolAddress(&p, g_status) != cudaSuccess) return nullptr;
  addr[dev].store(static_cast<uint32_t*>(p), std::memory_order_release);
  return static_cast<uint32_t*>(p);
}

static std::atomic<uint64_t> g_wait_timeout_ns{4000000000ull};
uint64_t wait_timeout_ns() { return g_wait_timeout_ns.load(); }

bool allow_smem(std::atomic<uint64_t>& done, const void* kernel, int bytes) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (done.load(std::memory_order_relaxed) >> dev & 1) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return true;
}

int num_sms() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev >= 0 && dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  if (dev >= 0 && dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// cuTensorMapEncodeTiled is fetched through the runtime so the library does
// not link against libcuda directly.
static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

bool make_map_bf16(CUtensorMap* map, const void* base, int BH, int N, int d, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)BH};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)d * 2 * (cuuint64_t)N};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool make_map_bf16_box(CUtensorMap* map, const void* base, int BH, int N, int d, int box_cols, int box_rows) {
  auto fn = encode_fn();
  if (!fn || (box_cols != 32 && box_cols != 64)) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)BH};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)d * 2 * (cuuint64_t)N};
  cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  // the box's rows are 64 or 128 bytes: the swizzle of that width
  const CUtensorMapSwizzle sw = box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool make_map_rows(CUtensorMap* map, const Rows& t, int T, int heads, int d, int box_cols, int box_rows) {
  auto fn = encode_fn();
  if (!fn || (box_cols != 32 && box_cols != 64)) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)heads};
  cuuint64_t strides[2] = {(cuuint64_t)t.row_stride * 2, (cuuint64_t)t.head_stride * 2};
  cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapSwizzle sw = box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, t.data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            sw, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_map_packed(CUtensorMap* map, const Rows& t, int T, int heads, int d) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)T, (cuuint64_t)heads};
  const cuuint64_t row = (cuuint64_t)t.row_stride * 2;
  cuuint64_t strides[3] = {row, row, (cuuint64_t)t.head_stride * 2};
  cuuint32_t box[4] = {64, 128, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, t.data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_map_bf16_2d(CUtensorMap* map, const void* base, int rows, int cols, int box_rows) {
  return make_map_bf16(map, base, 1, rows, cols, box_rows);
}

}  // namespace fa

using namespace fa;

static bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The kernels count work items (heads x 128-row tiles) and tile rows in
// 32-bit ints: B*H*N up to 2^37 keeps both below 2^31 (and is far beyond
// what fits in device memory at d = 64).
static bool sizes_supported(long long bh, int N) {
  return bh <= (1ll << 30) && N <= (1 << 30) && bh * (long long)N <= (1ll << 37);
}

static fa_status check_common(const void* Q, const void* K, const void* V, int B, int H, int N, int Nk, int d,
                              int mask_kind, const uint8_t* block_mask, float scale, Problem* p) {
  if (!Q || !K || !V) return FA_ERR_INVALID_ARG;
  if (B <= 0 || H <= 0 || N <= 0 || Nk <= 0 || d <= 0) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || !isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (mask_kind != FA_MASK_NONE && mask_kind != FA_MASK_CAUSAL && mask_kind != FA_MASK_BLOCK)
    return FA_ERR_INVALID_ARG;
  if (mask_kind == FA_MASK_BLOCK && !block_mask) return FA_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  const long long bh = (long long)B * H;
  if (!sizes_supported(bh, N) || !sizes_supported(bh, Nk)) return FA_ERR_UNSUPPORTED;
  p->B = B; p->H = H; p->N = N; p->Nk = Nk; p->d = d;
  p->BH = (int)bh;
  p->nq = (N + 127) / 128;
  p->nk = (Nk + 127) / 128;
  p->off = Nk - N;
  p->mask_kind = mask_kind;
  p->block_mask = mask_kind == FA_MASK_BLOCK ? block_mask : nullptr;
  p->scale = scale;
  p->scale_log2 = (float)((double)scale * 1.4426950408889634074);
  return FA_OK;
}

extern "C" {

fa_status fa_fwd_qk(const void* Q, const void* K, const void* V, int B, int H, int Nq, int Nk, int d,
                    int mask_kind, const uint8_t* block_mask, float scale, void* O, float* LSE, void* stream) {
  Problem p;
  fa_status st = check_common(Q, K, V, B, H, Nq, Nk, d, mask_kind, block_mask, scale, &p);
  if (st != FA_OK) return st;
  if (!O || !LSE || !aligned(O, 16) || !aligned(LSE, 4)) return FA_ERR_INVALID_ARG;
  return launch_fwd(p, Q, K, V, O, LSE, (cudaStream_t)stream);
}

fa_status fa_fwd_varlen(const void* Q, const void* K, const void* V, int B, int H, int Nq, int Nk, int d,
                        int mask_kind, const uint8_t* block_mask, float scale, const int* seqlens_q,
                        const int* seqlens_k, void* O, float* LSE, void* stream) {
  if (!aligned(seqlens_q, 4) || !aligned(seqlens_k, 4)) return FA_ERR_INVALID_ARG;
  Problem p;
  fa_status st = check_common(Q, K, V, B, H, Nq, Nk, d, mask_kind, block_mask, scale, &p);
  if (st != FA_OK) return st;
  if (!O || !LSE || !aligned(O, 16) || !aligned(LSE, 4)) return FA_ERR_INVALID_ARG;
  p.seqlens_q = seqlens_q;
  p.seqlens_k = seqlens_k;
  return launch_fwd(p, Q, K, V, O, LSE, (cudaStream_t)stream);
}

fa_status fa_fwd(const void* Q, const void* K, const void* V, int B, int H, int N, int d, int mask_kind,
                 const uint8_t* block_mask, float scale, void* O, float* LSE, void* stream) {
  return fa_fwd_qk(Q, K, V, B, H, N, N, d, mask_kind, block_mask, scale, O, LSE, stream);
}

size_t fa_bwd_workspace_size(int B, int H, int N, int d) {
  if (B <= 0 || H <= 0 || N <= 0 || (d != 64 && d != 128)) return 0;
  if (!sizes_supported((long long)B * H, N)) return 0;
  return bwd_workspace_bytes(B, H, N, d);
}

size_t fa_bwd_workspace_size_qk(int B, int H, int Nq, int Nk, int d) {
  if (Nk <= 0 || !sizes_supported((long long)B * H, Nk)) return 0;
  return fa_bwd_workspace_size(B, H, Nq, d);  // the workspace is per query row
}

static fa_status bwd_common(int stage, const void* Q, const void* K, const void* V, const void* O, const void* dO,
                            const float* LSE, int B, int H, int N, int Nk, int d, int mask_kind,
                            const uint8_t* block_mask, float scale, void* dQ, void* dK, void* dV, void* workspace,
                            size_t workspace_bytes, void* stream, int deterministic = 0,
                            const int* seqlens_q = nullptr, const int* seqlens_k = nullptr) {
  Problem p;
  fa_status st = check_common(Q, K, V, B, H, N, Nk, d, mask_kind, block_mask, scale, &p);
  p.deterministic = deterministic;
  p.seqlens_q = seqlens_q;
  p.seqlens_k = seqlens_k;
  if (st != FA_OK) return st;
  if (!O || !dO || !LSE || !dQ || !dK || !dV) return FA_ERR_INVALID_ARG;
  if (!aligned(O, 16) || !aligned(dO, 16) || !aligned(LSE, 4) || !aligned(dQ, 16) || !aligned(dK, 16) ||
      !aligned(dV, 16))
    return FA_ERR_INVALID_ARG;
  const size_t need = bwd_workspace_bytes(B, H, N, d);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return FA_ERR_WORKSPACE;
  return launch_bwd(p, Q, K, V, O, dO, LSE, dQ, dK, dV, workspace, (cudaStream_t)stream, stage);
}

fa_status fa_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO, const float* LSE,
                 int B, int H, int N, int d, int mask_kind, const uint8_t* block_mask, float scale, void* dQ,
                 void* dK, void* dV, void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_common(-1, Q, K, V, O, dO, LSE, B, H, N, N, d, mask_kind, block_mask, scale, dQ, dK, dV, workspace,
                    workspace_bytes, stream);
}

fa_status fa_bwd_qk(const void* Q, const void* K, const void* V, const void* O, const void* dO, const float* LSE,
                    int B, int H, int Nq, int Nk, int d, int mask_kind, const uint8_t* block_mask, float scale,
                    void* dQ, void* dK, void* dV, void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_common(-1, Q, K, V, O, dO, LSE, B, H, Nq, Nk, d, mask_kind, block_mask, scale, dQ, dK, dV, workspace,
                    workspace_bytes, stream);
}

fa_status fa_bwd_varlen(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                        const float* LSE, int B, int H, int Nq, int Nk, int d, int mask_kind,
                        const uint8_t* block_mask, float scale, const int* seqlens_q, const int* seqlens_k,
                        int deterministic, void* dQ, void* dK, void* dV, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (!aligned(seqlens_q, 4) || !aligned(seqlens_k, 4)) return FA_ERR_INVALID_ARG;
  return bwd_common(-1, Q, K, V, O, dO, LSE, B, H, Nq, Nk, d, mask_kind, block_mask, scale, dQ, dK, dV, workspace,
                    workspace_bytes, stream, deterministic ? 1 : 0, seqlens_q, seqlens_k);
}

fa_status fa_bwd_qk_deterministic(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                                  const float* LSE, int B, int H, int Nq, int Nk, int d, int mask_kind,
                                  const uint8_t* block_mask, float scale, void* dQ, void* dK, void* dV,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_common(-1, Q, K, V, O, dO, LSE, B, H, Nq, Nk, d, mask_kind, block_mask, scale, dQ, dK, dV, workspace,
                    workspace_bytes, stream, 1);
}

fa_status fa_bwd_stage(int stage, const void* Q, const void* K, const void* V, const void* O, const void* dO,
                       const float* LSE, int B, int H, int N, int d, int mask_kind, const uint8_t* block_mask,
                       float scale, void* dQ, void* dK, void* dV, void* workspace, size_t workspace_bytes,
                       void* stream) {
  if (stage < 0 || stage > 2) return FA_ERR_INVALID_ARG;
  return bwd_common(stage, Q, K, V, O, dO, LSE, B, H, N, N, d, mask_kind, block_mask, scale, dQ, dK, dV, workspace,
                    workspace_bytes, stream);
}

// fa_decode hands problems with at least this many queries per head (and at
// least one head per SM) to the tensor-core forward.
constexpr int DECODE_TC_MIN_NQ = 4;

size_t fa_decode_workspace_size(int B, int H, int Nq, int Nk, int d) {
  if (B <= 0 || H <= 0 || Nq <= 0 || Nq > 16 || Nk <= 0 || (d != 64 && d != 128)) return 0;
  const long long bh = (long long)B * H;
  if (!sizes_supported(bh, Nk)) return 0;
  return decode_workspace_bytes((int)bh, Nq, Nk, d);
}

fa_status fa_decode(const void* Q, const void* K, const void* V, int B, int H, int Nq, int Nk, int d, int mask_kind,
                    float scale, void* O, float* LSE, void* workspace, size_t workspace_bytes, void* stream) {
  if (mask_kind == FA_MASK_BLOCK) return FA_ERR_UNSUPPORTED;
  Problem p;
  fa_status st = check_common(Q, K, V, B, H, Nq, Nk, d, mask_kind, nullptr, scale, &p);
  if (st != FA_OK) return st;
  if (Nq > 16) return FA_ERR_UNSUPPORTED;
  if (!O || !LSE || !aligned(O, 16) || !aligned(LSE, 4)) return FA_ERR_INVALID_ARG;
  const size_t need = decode_workspace_bytes(p.BH, Nq, Nk, d);
  if (need == 0) return FA_ERR_CUDA;
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return FA_ERR_WORKSPACE;
  // With several queries per head and a head for every SM, the tensor-core
  // forward (one work item per head, the cache read once per head) fills the
  // GPU and outruns the split-key kernel, whose per-query work runs on the
  // CUDA cores.
  if (Nq >= DECODE_TC_MIN_NQ && p.BH >= num_sms()) return launch_fwd(p, Q, K, V, O, LSE, (cudaStream_t)stream);
  return launch_decode(p, Q, K, V, O, LSE, workspace, workspace_bytes, (cudaStream_t)stream);
}

size_t fa_standard_fwd_workspace_size(int B, int H, int N, int d) {
  if (B <= 0 || H <= 0 || N <= 0 || N > 16384 || (d != 64 && d != 128)) return 0;
  const long long bh = (long long)B * H;
  if (!sizes_supported(bh, N) || bh > (1 << 30) / 16) return 0;
  return standard_workspace_bytes((int)bh, N);
}

fa_status fa_standard_fwd(const void* Q, const void* K, const void* V, int B, int H, int N, int d, int mask_kind,
                          const uint8_t* block_mask, float scale, void* O, float* LSE, void* workspace,
                          size_t workspace_bytes, void* stream) {
  Problem p;
  fa_status st = check_common(Q, K, V, B, H, N, N, d, mask_kind, block_mask, scale, &p);
  if (st != FA_OK) return st;
  if (N > 16384) return FA_ERR_UNSUPPORTED;
  if (!O || !LSE || !aligned(O, 16) || !aligned(LSE, 4)) return FA_ERR_INVALID_ARG;
  const size_t need = fa_standard_fwd_workspace_size(B, H, N, d);
  if (need == 0) return FA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return FA_ERR_WORKSPACE;
  return launch_standard_fwd(p, Q, K, V, O, LSE, workspace, (cudaStream_t)stream);
}

// ---- packed sequences ----
static bool valid_rows(const fa_rows* r, int d) {
  return r && r->data && aligned(r->data, 16) && r->row_stride >= 0 && r->head_stride >= 0 && r->row_stride % 8 == 0 &&
         r->head_stride % 8 == 0 && r->row_stride < (1ll << 40) && r->head_stride < (1ll << 40) && d > 0;
}
static Rows rows_of(const fa_rows* r) { return Rows{r->data, (long long)r->row_stride, (long long)r->head_stride}; }

// Rows that the tensor maps take: strides above zero (of one row or head: never used).
static bool valid_packed(const fa_rows* r, int T, int heads, int d, Rows* out) {
  if (T == 0) {  // nothing to read: no data, any strides
    *out = Rows{nullptr, d, d};
    return true;
  }
  if (!valid_rows(r, d) || (T > 1 && r->row_stride == 0) || (heads > 1 && r->head_stride == 0)) return false;
  *out = rows_of(r);
  if (out->row_stride == 0) out->row_stride = d;
  if (out->head_stride == 0) out->head_stride = d;
  return true;
}

static bool packed_sizes_supported(int B, int Tq, int Tk, int Hq, int Hkv) {
  // tiles x heads, and rows x heads of LSE, in 32 bits
  return Tq <= (1 << 28) && Tk <= (1 << 28) && B <= (1 << 24) && Hkv <= Hq &&
         (pack::slots(Tq, B) + 1) * Hq <= (1ll << 29) && (pack::slots(Tk, B) + 1) * Hq <= (1ll << 29);
}

static fa_status check_packed(const int* cu_q, const int* cu_k, int B, int Tq, int Tk, int Hq, int Hkv, int d,
                              int mask_kind, float scale, PackedProblem* p) {
  if (B <= 0 || Tq < 0 || Tk < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || d <= 0) return FA_ERR_INVALID_ARG;
  if (!cu_q || !cu_k || !aligned(cu_q, 4) || !aligned(cu_k, 4)) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || !isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (mask_kind == FA_MASK_BLOCK) return FA_ERR_UNSUPPORTED;
  if (mask_kind != FA_MASK_NONE && mask_kind != FA_MASK_CAUSAL) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || !packed_sizes_supported(B, Tq, Tk, Hq, Hkv)) return FA_ERR_UNSUPPORTED;
  p->pk = Pack{cu_q, cu_k, B, Tq, Tk, Hq, Hkv, Hq / Hkv};
  p->d = d;
  p->mask_kind = mask_kind;
  p->scale = scale;
  p->scale_log2 = (float)((double)scale * 1.4426950408889634074);
  return FA_OK;
}

fa_status fa_fwd_packed(const fa_rows* Q, const fa_rows* K, const fa_rows* V, const int* cu_q, const int* cu_k, int B,
                        int Tq, int Tk, int Hq, int Hkv, int d, int mask_kind, float scale, const fa_rows* O,
                        float* LSE, void* workspace, size_t workspace_bytes, void* stream) {
  PackedProblem p;
  const fa_status st = check_packed(cu_q, cu_k, B, Tq, Tk, Hq, Hkv, d, mask_kind, scale, &p);
  if (st != FA_OK) return st;
  Rows q, k, v, o;
  if (!valid_packed(Q, Tq, Hq, d, &q) || !valid_packed(K, Tk, Hkv, d, &k) || !valid_packed(V, Tk, Hkv, d, &v) ||
      !valid_packed(O, Tq, Hq, d, &o))
    return FA_ERR_INVALID_ARG;
  if (Tq == 0) return FA_OK;
  if (!LSE || !aligned(LSE, 4)) return FA_ERR_INVALID_ARG;
  const size_t need = fwd_packed_workspace_bytes(B, Tq, Hq, d);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return FA_ERR_WORKSPACE;
  return launch_fwd_packed(p, q, k, v, o, LSE, workspace, (cudaStream_t)stream);
}

size_t fa_fwd_packed_workspace_size(int B, int Tq, int Hq, int Hkv, int d) {
  if (B <= 0 || Tq <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || (d != 64 && d != 128)) return 0;
  if (!packed_sizes_supported(B, Tq, 0, Hq, Hkv)) return 0;
  return fwd_packed_workspace_bytes(B, Tq, Hq, d);
}

size_t fa_bwd_packed_workspace_size(int B, int Tq, int Tk, int Hq, int Hkv, int d) {
  if (B <= 0 || Tq < 0 || Tk < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || (d != 64 && d != 128)) return 0;
  if (!packed_sizes_supported(B, Tq, Tk, Hq, Hkv)) return 0;
  return bwd_packed_workspace_bytes(Pack{nullptr, nullptr, B, Tq, Tk, Hq, Hkv, Hq / Hkv}, d);
}

fa_status fa_bwd_packed(const fa_rows* Q, const fa_rows* K, const fa_rows* V, const fa_rows* O, const fa_rows* dO,
                        const float* LSE, const int* cu_q, const int* cu_k, int B, int Tq, int Tk, int Hq, int Hkv,
                        int d, int mask_kind, float scale, int deterministic, const fa_rows* dQ, const fa_rows* dK,
                        const fa_rows* dV, void* workspace, size_t workspace_bytes, void* stream) {
  PackedProblem p;
  const fa_status st = check_packed(cu_q, cu_k, B, Tq, Tk, Hq, Hkv, d, mask_kind, scale, &p);
  if (st != FA_OK) return st;
  p.deterministic = deterministic ? 1 : 0;
  Rows q, k, v, o, g, dq, dk, dv;
  if (!valid_packed(Q, Tq, Hq, d, &q) || !valid_packed(K, Tk, Hkv, d, &k) || !valid_packed(V, Tk, Hkv, d, &v) ||
      !valid_packed(O, Tq, Hq, d, &o) || !valid_packed(dO, Tq, Hq, d, &g) || !valid_packed(dQ, Tq, Hq, d, &dq) ||
      !valid_packed(dK, Tk, Hkv, d, &dk) || !valid_packed(dV, Tk, Hkv, d, &dv))
    return FA_ERR_INVALID_ARG;
  if (Tq > 0 && (!LSE || !aligned(LSE, 4))) return FA_ERR_INVALID_ARG;
  if (Tq == 0 && Tk == 0) return FA_OK;
  const size_t need = bwd_packed_workspace_bytes(p.pk, d);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return FA_ERR_WORKSPACE;
  return launch_bwd_packed(p, q, k, v, o, g, LSE, dq, dk, dv, workspace, (cudaStream_t)stream);
}

// ---- paged cache ----
static fa_status check_cache(const fa_paged_cache* c, bool scales, PagedCache* p) {
  if (!c || !c->K || !c->V || !c->page_table) return FA_ERR_INVALID_ARG;
  if (c->dtype != FA_CACHE_BF16 && c->dtype != FA_CACHE_E4M3) return FA_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->page_size <= 0 || c->Hkv <= 0 || c->d <= 0 || c->B <= 0 || c->max_pages <= 0)
    return FA_ERR_INVALID_ARG;
  const int elem = c->dtype == FA_CACHE_E4M3 ? 1 : 2;
  const int64_t unit = 16 / elem;  // every row starts on a 16-byte boundary
  for (int64_t st : {c->page_stride, c->head_stride, c->row_stride})
    if (st < 0 || st % unit != 0 || st >= (1ll << 40)) return FA_ERR_INVALID_ARG;
  if (!aligned(c->K, 16) || !aligned(c->V, 16) || !aligned(c->page_table, 4) || c->table_stride < 0)
    return FA_ERR_INVALID_ARG;
  if (scales && elem == 1 && (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)))
    return FA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED;
  // positions fit an int; rows of (sequence, head) and blocks of 128 keys too
  const long long cap = (long long)c->max_pages * c->page_size;
  if (cap > (1ll << 30) || (long long)c->B * c->Hkv > (1ll << 24) || c->B * (cap / 128 + 1) > (1ll << 30))
    return FA_ERR_UNSUPPORTED;
  *p = PagedCache{c->K, c->V, elem, c->num_pages, c->page_size, c->Hkv, c->d, (long long)c->page_stride,
                  (long long)c->head_stride, (long long)c->row_stride, c->k_scale, c->v_scale, c->page_table, c->B,
                  c->max_pages, (long long)c->table_stride};
  return FA_OK;
}

// Rows that are written may not lie on top of each other.
static bool cache_rows_apart(const PagedCache& c) {
  return (c.num_pages == 1 || c.page_stride > 0) && (c.Hkv == 1 || c.head_stride > 0) && (c.page_size == 1 || c.row_stride > 0);
}
static bool weight_rows_apart(const PagedCache& c, int64_t batch, int64_t head) {
  return (c.B == 1 || batch > 0) && (c.Hkv == 1 || head > 0);
}

fa_status fa_paged_append(const fa_paged_cache* cache, const fa_rows* K, const fa_rows* V, const int* cu_seqlens,
                          const int* lens, int T, void* stream) {
  PagedCache c;
  const fa_status st = check_cache(cache, true, &c);
  if (st != FA_OK) return st;
  if (T < 0 || !cu_seqlens || !lens || !aligned(cu_seqlens, 4) || !aligned(lens, 4)) return FA_ERR_INVALID_ARG;
  if (!cache_rows_apart(c)) return FA_ERR_INVALID_ARG;
  if (T > (1 << 30)) return FA_ERR_UNSUPPORTED;
  if (T == 0) return FA_OK;
  if (!valid_rows(K, c.d) || !valid_rows(V, c.d)) return FA_ERR_INVALID_ARG;
  return launch_paged_append(c, rows_of(K), rows_of(V), cu_seqlens, lens, T, (cudaStream_t)stream);
}

size_t fa_paged_decode_workspace_size(int B, int Hq, int Hkv, int d, int64_t max_len, int weights) {
  if (B <= 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv != 0 || (d != 64 && d != 128) || max_len <= 0) return 0;
  if (max_len > (1ll << 30) || (long long)B * Hq > (1ll << 24)) return 0;
  return paged_decode_workspace_bytes(B, Hq, d, max_len, weights != 0);
}

fa_status fa_paged_decode(const fa_paged_cache* cache, const fa_rows* Q, int Hq, const int* lens, float scale,
                          float* weights, int64_t w_batch_stride, int64_t w_head_stride, int accumulate, void* O,
                          float* LSE, void* workspace, size_t workspace_bytes, void* stream) {
  PagedCache c;
  const fa_status st = check_cache(cache, true, &c);
  if (st != FA_OK) return st;
  if (!valid_rows(Q, c.d) || Hq <= 0 || Hq % c.Hkv != 0 || !lens || !aligned(lens, 4)) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || !isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (!O || !LSE || !aligned(O, 16) || !aligned(LSE, 4)) return FA_ERR_INVALID_ARG;
  if (weights && (!aligned(weights, 4) || w_batch_stride < 0 || w_head_stride < 0))
    return FA_ERR_INVALID_ARG;
  if ((long long)c.B * Hq > (1ll << 24)) return FA_ERR_UNSUPPORTED;
  const size_t need = paged_decode_workspace_bytes(c.B, Hq, c.d, (long long)c.max_pages * c.page_size, weights != nullptr);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return FA_ERR_WORKSPACE;
  if (weights && !weight_rows_apart(c, w_batch_stride, w_head_stride)) return FA_ERR_INVALID_ARG;
  PagedDecode a;
  a.Q = rows_of(Q);
  a.Hq = Hq;
  a.lens = lens;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634074);
  a.W = weights;
  a.w_batch = w_batch_stride;
  a.w_head = w_head_stride;
  a.accumulate = accumulate != 0;
  a.O = O;
  a.LSE = LSE;
  a.workspace = workspace;
  return launch_paged_decode(c, a, (cudaStream_t)stream);
}

fa_status fa_paged_evict(const fa_paged_cache* cache, const int* lens, const int* table_out, int64_t table_out_stride,
                         int max_pages_out, const float* weights, int64_t w_batch_stride, int64_t w_head_stride,
                         int budget, int recent, float* weights_out, int64_t wo_batch_stride, int64_t wo_head_stride,
                         int64_t wo_len, int* kept, int* lens_out, void* stream) {
  PagedCache c;
  const fa_status st = check_cache(cache, false, &c);
  if (st != FA_OK) return st;
  if (!lens || !table_out || !weights || !weights_out || !kept || !lens_out) return FA_ERR_INVALID_ARG;
  for (const void* q : {(const void*)lens, (const void*)table_out, (const void*)weights, (const void*)weights_out,
                        (const void*)kept, (const void*)lens_out})
    if (!aligned(q, 4)) return FA_ERR_INVALID_ARG;
  if (table_out_stride < 0 || w_batch_stride < 0 || w_head_stride < 0 || wo_batch_stride < 0 || wo_head_stride < 0)
    return FA_ERR_INVALID_ARG;
  if (budget <= 0 || recent < 0 || recent > budget || max_pages_out <= 0) return FA_ERR_INVALID_ARG;
  if (!cache_rows_apart(c) || !weight_rows_apart(c, wo_batch_stride, wo_head_stride)) return FA_ERR_INVALID_ARG;
  const long long cap = (long long)c.max_pages * c.page_size;
  const long long most = cap < budget ? cap : budget;  // rows a sequence can be left with
  if ((long long)max_pages_out * c.page_size < most || wo_len < most) return FA_ERR_INVALID_ARG;
  if (wo_len > (1ll << 30) || budget > (1 << 30) || (long long)c.B * c.Hkv * (budget / 32 + 1) > (1ll << 30))
    return FA_ERR_UNSUPPORTED;
  // in place, blocks would read what others have written (partly overlapping
  // buffers are the caller's to avoid)
  if (lens_out == lens || weights_out == weights || table_out == cache->page_table) return FA_ERR_INVALID_ARG;
  Evict e{lens, table_out, (long long)table_out_stride, max_pages_out, weights, (long long)w_batch_stride,
          (long long)w_head_stride, budget, recent, weights_out, (long long)wo_batch_stride,
          (long long)wo_head_stride, (int)wo_len, kept, lens_out};
  return launch_paged_evict(c, e, (cudaStream_t)stream);
}

fa_status fa_device_status(void* stream) {
  if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return FA_ERR_CUDA;
  uint32_t v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(v)) != cudaSuccess) return FA_ERR_CUDA;
  if (v != 0 && cudaMemcpyToSymbol(g_status, &zero, sizeof(zero)) != cudaSuccess) return FA_ERR_CUDA;
  if (v == 0) return FA_OK;
  if (v == FA_DEV_ERR_TIMEOUT) return FA_ERR_TIMEOUT;
  return v == FA_DEV_ERR_BOUNDS ? FA_ERR_BOUNDS : FA_ERR_CUDA;
}

void fa_set_wait_timeout_ns(uint64_t ns) { g_wait_timeout_ns.store(ns ? ns : 4000000000ull); }

const char* fa_status_string(fa_status s) {
  switch (s) {
    case FA_OK: return "ok";
    case FA_ERR_INVALID_ARG: return "invalid argument";
    case FA_ERR_UNSUPPORTED: return "unsupported problem";
    case FA_ERR_CUDA: return "CUDA error";
    case FA_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
    case FA_ERR_TIMEOUT: return "a bounded device-side wait timed out";
    case FA_ERR_BOUNDS: return "an index lay outside its buffer, and the access was skipped";
  }
  return "unknown status";
}

fa_status fa_selftest_bounded_wait(uint64_t timeout_ns, void* stream) {
  if (timeout_ns == 0 || timeout_ns > 10000000000ull) return FA_ERR_INVALID_ARG;
  return launch_selftest_wait(timeout_ns, (cudaStream_t)stream);
}

fa_status fa_selftest_mma_tile(const void* A, const void* B, float* C, int n, int k, int mode, void* stream) {
  if (!A || !B || !C) return FA_ERR_INVALID_ARG;
  if ((n != 64 && n != 128) || (k != 64 && k != 128) || (mode != 0 && mode != 1)) return FA_ERR_INVALID_ARG;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(C, 16)) return FA_ERR_INVALID_ARG;
  return launch_selftest_mma(A, B, C, n, k, mode, (cudaStream_t)stream);
}

}  // extern "C"
