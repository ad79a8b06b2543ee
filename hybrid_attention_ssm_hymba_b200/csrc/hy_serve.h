// hy_serve.h -- host-side interface between the serving part of the C ABI (api_serve.cu) and its
// kernels: a paged K/V cache and a ragged batch as in include/hymba.h; every pointer is on the device.
#pragma once

#include "hy_kernels.h"

namespace hy {

enum CacheType : int { CACHE_F32 = 0, CACHE_BF16 = 1, CACHE_E4M3 = 2 };
struct PagedKv {
  void* pages;       // [2, n_pages, page_size, hkv * dh]
  float* scales;     // [2, n_pages, hkv, page_size] (CACHE_E4M3)
  const int* table;  // [batch, table_ld]
  int n_pages, page_size, table_ld, hkv, dh, type;
};
struct RaggedBatch {
  const int* q_start;  // [batch + 1]
  const int* kv_len;   // [batch]
  int batch, total_rows, max_rows;
};
cudaError_t launch_paged_append(const PagedKv& kv, const RaggedBatch& rb, const void* k, const void* v, long long ld,
                                bool bf16, unsigned* status, cudaStream_t st);
cudaError_t launch_paged_read(const PagedKv& kv, const RaggedBatch& rb, void* k, void* v, long long ld, bool bf16,
                              unsigned* status, cudaStream_t st);
struct PagedAttnDesc {
  PagedKv kv;
  RaggedBatch rb;
  const void* q; long long q_ld;
  void* out; long long out_ld;
  int n_q_heads, n_meta, window;
  bool bf16;
  unsigned* status;
  void* scratch;   // paged_attention_scratch() bytes, 256-byte aligned
};
size_t paged_attention_scratch(const PagedKv& kv, const RaggedBatch& rb, int n_q_heads, bool bf16);
cudaError_t launch_paged_attention(const PagedAttnDesc& a, cudaStream_t st);

cudaError_t launch_quantize_w4(const void* w, void* q4, float* scales, int N, int K, int group, bool bf16,
                               cudaStream_t st);
cudaError_t launch_dequantize_w4(const void* q4, const float* scales, void* w, int N, int K, int group, bool bf16,
                                 cudaStream_t st);
cudaError_t launch_gemm_w4(const void* a, const void* q4, const float* scales, void* c, int M, int N, int K, int group,
                           bool bf16, cudaStream_t st);

}  // namespace hy
