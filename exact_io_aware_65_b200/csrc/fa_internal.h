// fa_internal.h -- host-side declarations shared by the library's .cu files.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "fa.h"
#include "pack.cuh"

namespace fa {

// Problem description after validation.
struct Problem {
  int B, H, N, d;  // N: query rows
  int Nk;          // key rows (N for self-attention)
  int BH;          // B * H
  int nq, nk;      // ceil(N / 128) query tiles, ceil(Nk / 128) key tiles
  int off;         // Nk - N: causal alignment (query i sees keys j <= i + off)
  int mask_kind;
  const uint8_t* block_mask;  // device [nq, nk] or nullptr
  int deterministic = 0;      // backward: fixed order of the dQ additions
  // Optional per-batch-element lengths (device int [B]; nullptr: N, Nk).
  const int* seqlens_q = nullptr;
  const int* seqlens_k = nullptr;
  float scale;
  float scale_log2;  // scale * log2(e), computed in double and rounded once
};

// Rows of a packed tensor [rows, heads, d]; strides in elements.
struct Rows {
  void* data;
  long long row_stride, head_stride;
};

// Packed sequences after validation.
struct PackedProblem {
  Pack pk;
  int d, mask_kind;
  int deterministic = 0;
  float scale, scale_log2;
};

// Encode a 3-D tiled TMA map over a contiguous bf16 [BH, N, d] tensor:
// dims (d, N, BH), box (64, box_rows, 1), 128-byte swizzle, zero fill out of
// bounds.  Returns false on failure.
bool make_map_bf16(CUtensorMap* map, const void* base, int BH, int N, int d, int box_rows);
// The same [BH, N, d] view with a box of box_cols (32 or 64) x box_rows and the
// swizzle of the box's row width (64 or 128 bytes): for tiled stores.
bool make_map_bf16_box(CUtensorMap* map, const void* base, int BH, int N, int d, int box_cols, int box_rows);

// Rows [T, heads, d] as (d, T, heads), box box_cols x box_rows x 1: for tiled stores.
bool make_map_rows(CUtensorMap* map, const Rows& r, int T, int heads, int d, int box_cols, int box_rows);
// Rows [T, heads, d] as (d, row of the sequence, first row of the sequence,
// heads), box 64 x 128 x 1 x 1 (pack.cuh): for loads.
bool make_map_packed(CUtensorMap* map, const Rows& r, int T, int heads, int d);

// Same for a 2-D row-major bf16 matrix [rows, cols] (used by the self-test).
bool make_map_bf16_2d(CUtensorMap* map, const void* base, int rows, int cols, int box_rows);

// Sets a kernel's dynamic shared memory limit, once per device and kernel
// (`done` is the kernel's own, one bit per device).
bool allow_smem(std::atomic<uint64_t>& done, const void* kernel, int bytes);

template <typename... P, typename... A>
inline bool launch(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t s, A... args) {
  kernel<<<grid, threads, smem, s>>>(P(args)...);
  return cudaGetLastError() == cudaSuccess;
}

uint64_t wait_timeout_ns();
// Device address of the calling device's status word (nullptr on failure).
uint32_t* status_word();
int num_sms();

// Kernel launchers (defined next to their kernels).
fa_status launch_fwd(const Problem& p, const void* Q, const void* K, const void* V, void* O, float* LSE,
                     cudaStream_t s);
fa_status launch_fwd_packed(const PackedProblem& p, const Rows& Q, const Rows& K, const Rows& V, const Rows& O,
                            float* LSE, void* workspace, cudaStream_t s);
size_t fwd_packed_workspace_bytes(int B, int Tq, int Hq, int d);
// stage < 0: all three stages; otherwise only the given one (0, 1 or 2).
fa_status launch_bwd(const Problem& p, const void* Q, const void* K, const void* V, const void* O,
                     const void* dO, const float* LSE, void* dQ, void* dK, void* dV, void* workspace,
                     cudaStream_t s, int stage);
size_t bwd_workspace_bytes(int B, int H, int N, int d);
size_t bwd_packed_workspace_bytes(const Pack& k, int d);
fa_status launch_bwd_packed(const PackedProblem& p, const Rows& Q, const Rows& K, const Rows& V, const Rows& O,
                            const Rows& dO, const float* LSE, const Rows& dQ, const Rows& dK, const Rows& dV,
                            void* workspace, cudaStream_t s);
// Decode (few queries, long key history): workspace for the split-key
// partial results on the current device (0 on failure), and the launch.
size_t decode_workspace_bytes(int BH, int Nq, int Nk, int d);
fa_status launch_decode(const Problem& p, const void* Q, const void* K, const void* V, void* O, float* LSE,
                        void* workspace, size_t workspace_bytes, cudaStream_t s);
// Standard (materialising) attention, the baseline: workspace for S (fp32)
// and P (bf16), and the launch.
size_t standard_workspace_bytes(int BH, int N);
fa_status launch_standard_fwd(const Problem& p, const void* Q, const void* K, const void* V, void* O, float* LSE,
                              void* workspace, cudaStream_t s);
// A paged cache after validation (strides in elements; elem: bytes of one).
struct PagedCache {
  void* K;
  void* V;
  int elem, num_pages, page_size, Hkv, d;
  long long page_stride, head_stride, row_stride;
  const float* k_scale;
  const float* v_scale;
  const int* table;
  int B, max_pages;
  long long table_stride;
};

struct PagedDecode {
  Rows Q;
  int Hq;
  const int* lens;
  float scale_log2;
  float* W;  // accumulated weights, or nullptr
  long long w_batch, w_head;
  int accumulate;
  void* O;
  float* LSE;
  void* workspace;
};

struct Evict {
  const int* lens;
  const int* table_out;
  long long table_out_stride;
  int max_out;
  const float* W;
  long long w_batch, w_head;
  int budget, recent;
  float* Wout;
  long long wo_batch, wo_head;
  int wo_len;
  int* kept;
  int* lens_out;
};

fa_status launch_paged_append(const PagedCache& c, const Rows& K, const Rows& V, const int* cu, const int* lens, int T,
                              cudaStream_t s);
size_t paged_decode_workspace_bytes(int B, int Hq, int d, long long cap, bool weights);
fa_status launch_paged_decode(const PagedCache& c, const PagedDecode& a, cudaStream_t s);
fa_status launch_paged_evict(const PagedCache& c, const Evict& e, cudaStream_t s);
fa_status launch_selftest_wait(uint64_t timeout_ns, cudaStream_t s);
fa_status launch_selftest_mma(const void* A, const void* B, float* C, int n, int k, int mode, cudaStream_t s);

}  // namespace fa
