// api_serve.cu -- the serving part of the C ABI (include/hymba.h): argument checks of the
// paged K/V cache, its attention and the 4-bit weight products, and their launches.
#include "hy_serve.h"
#include "hymba.h"

namespace {

inline bool aligned_to(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned_to(p, 16); }
inline int esize(hymba_dtype_t t) { return t == HYMBA_BF16 ? 2 : 4; }
inline bool valid_dtype(hymba_dtype_t t) { return t == HYMBA_BF16 || t == HYMBA_F32; }

hymba_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? HYMBA_OK : HYMBA_ERR_CUDA; }

// A kernel reads its tensors where it is launched: the current device.  One pointer of the
// call stands for all of them.
hymba_status_t check_device(const void* p) {
  int dev = 0;
  cudaPointerAttributes at{};
  if (cudaGetDevice(&dev) != cudaSuccess || cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return HYMBA_ERR_CUDA;
  }
  if (at.type == cudaMemoryTypeManaged) return HYMBA_OK;
  return at.type == cudaMemoryTypeDevice && at.device == dev ? HYMBA_OK : HYMBA_ERR_INVALID_ARG;
}

hymba_status_t check_cache(const hymba_paged_kv_t* kv, hymba_dtype_t dtype) {
  if (!kv || !valid_dtype(dtype) || !kv->pages || !kv->page_table) return HYMBA_ERR_INVALID_ARG;
  if (kv->n_pages < 1 || kv->page_size < 1 || kv->table_ld < 1 || kv->n_kv_heads < 1 || kv->head_dim < 1 ||
      kv->cache_type < HYMBA_CACHE_F32 || kv->cache_type > HYMBA_CACHE_E4M3)
    return HYMBA_ERR_INVALID_ARG;
  if (kv->cache_type == HYMBA_CACHE_E4M3 && !kv->scales) return HYMBA_ERR_INVALID_ARG;
  if ((kv->cache_type == HYMBA_CACHE_F32 && dtype != HYMBA_F32) ||
      (kv->cache_type == HYMBA_CACHE_BF16 && dtype != HYMBA_BF16))
    return HYMBA_ERR_UNSUPPORTED;
  const int ps = kv->page_size;
  if (!(ps == 8 || ps == 16 || ps == 32 || ps == 64 || ps % 128 == 0)) return HYMBA_ERR_UNSUPPORTED;
  if (kv->head_dim % 16 || kv->head_dim > 256) return HYMBA_ERR_UNSUPPORTED;
  // row numbers, in the cache and in a sequence, and row widths are 32-bit, with room for the
  // difference of two places in a sequence and a window
  if (static_cast<long long>(kv->n_pages) * ps > (1ll << 31) - 1 ||
      static_cast<long long>(kv->table_ld) * ps > (1ll << 30) ||
      static_cast<long long>(kv->n_kv_heads) * kv->head_dim > (1 << 16))
    return HYMBA_ERR_UNSUPPORTED;
  if (!aligned16(kv->pages) || !aligned_to(kv->page_table, 4) || (kv->cache_type == HYMBA_CACHE_E4M3 && !aligned16(kv->scales)))
    return HYMBA_ERR_UNSUPPORTED;
  return HYMBA_OK;
}

hymba_status_t check_batch(int batch, const int* q_start, const int* kv_len, int total_rows) {
  if (batch < 1 || !q_start || !kv_len || total_rows < 0) return HYMBA_ERR_INVALID_ARG;
  return aligned_to(q_start, 4) && aligned_to(kv_len, 4) ? HYMBA_OK : HYMBA_ERR_UNSUPPORTED;
}

hymba_status_t check_workspace(const void* workspace, size_t ws_bytes, size_t need) {
  if (!workspace || ws_bytes < need) return HYMBA_ERR_WORKSPACE;
  return reinterpret_cast<uintptr_t>(workspace) & 255 ? HYMBA_ERR_INVALID_ARG : HYMBA_OK;
}

hy::PagedKv paged(const hymba_paged_kv_t& kv) {
  return {kv.pages, kv.scales, kv.page_table, kv.n_pages, kv.page_size, kv.table_ld, kv.n_kv_heads, kv.head_dim,
          kv.cache_type};
}

hymba_status_t check_copy(const hymba_paged_kv_t* kv, const void* k, const void* v, int ld, int batch,
                          const int* q_start, const int* kv_len, int total_rows, hymba_dtype_t dtype, void* workspace,
                          size_t ws_bytes) {
  hymba_status_t s = check_cache(kv, dtype);
  if (s != HYMBA_OK) return s;
  if ((s = check_batch(batch, q_start, kv_len, total_rows)) != HYMBA_OK) return s;
  if (!k || !v || ld < kv->n_kv_heads * kv->head_dim) return HYMBA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || (static_cast<long long>(ld) * esize(dtype)) % 16) return HYMBA_ERR_UNSUPPORTED;
  return check_workspace(workspace, ws_bytes, 256);
}

hymba_status_t check_attention(const hymba_paged_kv_t* kv, int batch, int total_rows, int max_rows, int n_q_heads,
                               hymba_dtype_t dtype) {
  const hymba_status_t s = check_cache(kv, dtype);
  if (s != HYMBA_OK) return s;
  if (batch < 1 || total_rows < 0 || max_rows < 1 || n_q_heads < 1 || n_q_heads % kv->n_kv_heads)
    return HYMBA_ERR_INVALID_ARG;
  if (dtype == HYMBA_BF16 ? (kv->head_dim != 128 || n_q_heads / kv->n_kv_heads > 128) : kv->head_dim > 128)
    return HYMBA_ERR_UNSUPPORTED;
  if (static_cast<long long>(n_q_heads) * kv->head_dim > (1 << 19) ||
      static_cast<long long>(total_rows) * n_q_heads > (1ll << 31) - 1)
    return HYMBA_ERR_UNSUPPORTED;
  return HYMBA_OK;
}

hymba_status_t check_w4(const void* w, const void* q4, const float* scales, int N, int K, int group,
                        hymba_dtype_t dtype) {
  if (!w || !q4 || !scales || N < 1 || K < 1 || group < 1 || !valid_dtype(dtype)) return HYMBA_ERR_INVALID_ARG;
  if ((group != 32 && group != 64 && group != 128) || K % group || N > (1 << 30) || K > (1 << 30) || !aligned16(w) || !aligned16(q4) ||
      !aligned_to(scales, 4))
    return HYMBA_ERR_UNSUPPORTED;
  return HYMBA_OK;
}

}  // namespace

extern "C" {

hymba_status_t hymba_paged_kv_append(const hymba_paged_kv_t* kv, const void* k, const void* v, int ld, int batch,
                                     const int* q_start, const int* kv_len, int total_rows, hymba_dtype_t dtype,
                                     void* workspace, size_t ws_bytes, void* stream) {
  hymba_status_t s = check_copy(kv, k, v, ld, batch, q_start, kv_len, total_rows, dtype, workspace, ws_bytes);
  if (s != HYMBA_OK || total_rows == 0) return s;
  if ((s = check_device(kv->pages)) != HYMBA_OK) return s;
  return cuda_status(hy::launch_paged_append(paged(*kv), {q_start, kv_len, batch, total_rows, total_rows}, k, v, ld,
                                             dtype == HYMBA_BF16, static_cast<unsigned*>(workspace),
                                             static_cast<cudaStream_t>(stream)));
}

hymba_status_t hymba_paged_kv_read(const hymba_paged_kv_t* kv, void* k, void* v, int ld, int batch,
                                   const int* q_start, const int* kv_len, int total_rows, hymba_dtype_t dtype,
                                   void* workspace, size_t ws_bytes, void* stream) {
  hymba_status_t s = check_copy(kv, k, v, ld, batch, q_start, kv_len, total_rows, dtype, workspace, ws_bytes);
  if (s != HYMBA_OK || total_rows == 0) return s;
  if ((s = check_device(kv->pages)) != HYMBA_OK) return s;
  return cuda_status(hy::launch_paged_read(paged(*kv), {q_start, kv_len, batch, total_rows, total_rows}, k, v, ld,
                                           dtype == HYMBA_BF16, static_cast<unsigned*>(workspace),
                                           static_cast<cudaStream_t>(stream)));
}

size_t hymba_paged_attention_workspace_size(const hymba_paged_kv_t* kv, int batch, int total_rows, int max_rows,
                                            int n_q_heads, hymba_dtype_t dtype) {
  if (check_attention(kv, batch, total_rows, max_rows, n_q_heads, dtype) != HYMBA_OK) return 0;
  return 256 + hy::paged_attention_scratch(paged(*kv), {nullptr, nullptr, batch, total_rows, max_rows}, n_q_heads,
                                           dtype == HYMBA_BF16);
}

hymba_status_t hymba_paged_attention(const void* q, int q_ld, const hymba_paged_kv_t* kv, void* out, int out_ld,
                                     int batch, const int* q_start, const int* kv_len, int total_rows, int max_rows,
                                     int n_q_heads, int n_meta, int window, hymba_dtype_t dtype, void* workspace,
                                     size_t ws_bytes, void* stream) {
  hymba_status_t s = check_attention(kv, batch, total_rows, max_rows, n_q_heads, dtype);
  if (s != HYMBA_OK) return s;
  if ((s = check_batch(batch, q_start, kv_len, total_rows)) != HYMBA_OK) return s;
  const int wq = n_q_heads * kv->head_dim;
  if (!q || !out || n_meta < 0 || window < -1 || q_ld < wq || out_ld < wq) return HYMBA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || (static_cast<long long>(q_ld) * esize(dtype)) % 16 ||
      (static_cast<long long>(out_ld) * esize(dtype)) % 16)
    return HYMBA_ERR_UNSUPPORTED;
  hy::PagedAttnDesc a;
  a.kv = paged(*kv);
  a.rb = {q_start, kv_len, batch, total_rows, max_rows};
  const size_t need = 256 + hy::paged_attention_scratch(a.kv, a.rb, n_q_heads, dtype == HYMBA_BF16);
  if ((s = check_workspace(workspace, ws_bytes, need)) != HYMBA_OK || total_rows == 0) return s;
  if ((s = check_device(kv->pages)) != HYMBA_OK) return s;
  a.q = q;
  a.q_ld = q_ld;
  a.out = out;
  a.out_ld = out_ld;
  a.n_q_heads = n_q_heads;
  a.n_meta = n_meta;
  // a window that no sequence can outgrow is none
  a.window = window >= static_cast<long long>(kv->table_ld) * kv->page_size ? -1 : window;
  a.bf16 = dtype == HYMBA_BF16;
  a.status = static_cast<unsigned*>(workspace);
  a.scratch = static_cast<uint8_t*>(workspace) + 256;
  return cuda_status(hy::launch_paged_attention(a, static_cast<cudaStream_t>(stream)));
}

hymba_status_t hymba_quantize_w4(const void* w, void* w_q4, float* scales, int N, int K, int group,
                                 hymba_dtype_t dtype, void* stream) {
  hymba_status_t s = check_w4(w, w_q4, scales, N, K, group, dtype);
  if (s != HYMBA_OK || (s = check_device(w)) != HYMBA_OK) return s;
  return cuda_status(hy::launch_quantize_w4(w, w_q4, scales, N, K, group, dtype == HYMBA_BF16,
                                            static_cast<cudaStream_t>(stream)));
}

hymba_status_t hymba_dequantize_w4(const void* w_q4, const float* scales, void* w, int N, int K, int group,
                                   hymba_dtype_t dtype, void* stream) {
  hymba_status_t s = check_w4(w, w_q4, scales, N, K, group, dtype);
  if (s != HYMBA_OK || (s = check_device(w_q4)) != HYMBA_OK) return s;
  return cuda_status(hy::launch_dequantize_w4(w_q4, scales, w, N, K, group, dtype == HYMBA_BF16,
                                              static_cast<cudaStream_t>(stream)));
}

hymba_status_t hymba_gemm_w4(const void* a, const void* w_q4, const float* scales, void* c, int M, int N, int K,
                             int group, hymba_dtype_t dtype, void* stream) {
  hymba_status_t s = check_w4(a, w_q4, scales, N, K, group, dtype);
  if (s != HYMBA_OK) return s;
  if (!c || M < 1) return HYMBA_ERR_INVALID_ARG;
  if (M > 16 || !aligned_to(c, esize(dtype))) return HYMBA_ERR_UNSUPPORTED;
  if ((s = check_device(w_q4)) != HYMBA_OK) return s;
  return cuda_status(hy::launch_gemm_w4(a, w_q4, scales, c, M, N, K, group, dtype == HYMBA_BF16,
                                        static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
