// paged.cuh -- device-side view of a paged K/V cache and of the ragged batch that goes with
// it (include/hymba.h): which rows of the batch are whose, where a cache row lies, and the
// conversions between the cache's element types and fp32.
#pragma once

#include <cuda_fp8.h>

#include "hy_common.cuh"
#include "hy_serve.h"

namespace hy {

constexpr unsigned kStatusInvalid = 1;  // == HYMBA_ERR_INVALID_ARG

HY_DEV void report_invalid(unsigned* status) {
  // a timeout recorded by another kernel is not overwritten
  atomicCAS(status, 0u, kStatusInvalid);
}

// Sequence b of the batch: its new rows are [q0, q0 + n) of the ragged tensors and cache
// rows [len - n, len).  False when its lengths do not fit together (the sequence is skipped).
struct Seq {
  int q0, n, len;
};
HY_DEV bool load_seq(const RaggedBatch& rb, const PagedKv& kv, int b, Seq* s) {
  const long long q0 = rb.q_start[b], q1 = rb.q_start[b + 1], len = rb.kv_len[b];
  s->q0 = static_cast<int>(q0);
  s->n = static_cast<int>(q1 - q0);
  s->len = static_cast<int>(len);
  return q0 >= 0 && q1 >= q0 && q1 <= rb.total_rows && q1 - q0 <= len && q1 - q0 <= rb.max_rows &&
         len <= static_cast<long long>(kv.table_ld) * kv.page_size;
}

// Records every sequence whose lengths do not fit together (one CTA of a launch calls this
// with all its threads; the kernels that visit a sequence only skip it).
HY_DEV void check_batch(const RaggedBatch& rb, const PagedKv& kv, unsigned* status) {
  Seq s;
  for (int b = threadIdx.x; b < rb.batch; b += blockDim.x)
    if (!load_seq(rb, kv, b, &s)) report_invalid(status);
}

// The sequence that row r of the ragged tensors belongs to, or -1 (empty sequences own no row).
HY_DEV int seq_of_row(const RaggedBatch& rb, int r) {
  int lo = 0, hi = rb.batch;  // first b in (0, batch] with q_start[b] > r is in (lo, hi]
  if (r < rb.q_start[0] || r >= rb.q_start[rb.batch]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (rb.q_start[mid] <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Page of cache row `row` of sequence b; -1 when the table holds no valid page number.
HY_DEV int page_of(const PagedKv& kv, int b, int row) {
  const int pg = kv.table[static_cast<long long>(b) * kv.table_ld + row / kv.page_size];
  return pg >= 0 && pg < kv.n_pages ? pg : -1;
}

// Element offset of (K: which = 0 / V: which = 1, page, row of the page, head), and of its scale.
HY_DEV long long page_elem(const PagedKv& kv, int which, int page, int row, int head) {
  return (((static_cast<long long>(which) * kv.n_pages + page) * kv.page_size + row) * kv.hkv + head) * kv.dh;
}
HY_DEV long long page_scale(const PagedKv& kv, int which, int page, int row, int head) {
  return ((static_cast<long long>(which) * kv.n_pages + page) * kv.hkv + head) * kv.page_size + row;
}

// Two e4m3 codes (the low or the high half of u) as fp16.
HY_DEV uint32_t f16_of_e4m3(uint32_t u, int half) {
  uint32_t v;
  if (half) asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, hi;}" : "=r"(v) : "r"(u));
  else asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo;}" : "=r"(v) : "r"(u));
  return v;
}

// ------------------------------------------------------------------ eight elements as fp32
template <typename T> struct Vec8;  // how a lane moves eight consecutive elements
template <> struct Vec8<float> {
  uint4 a, b;
  HY_DEV void load(const float* p) {
    a = reinterpret_cast<const uint4*>(p)[0];
    b = reinterpret_cast<const uint4*>(p)[1];
  }
  HY_DEV void store(float* p) const {
    reinterpret_cast<uint4*>(p)[0] = a;
    reinterpret_cast<uint4*>(p)[1] = b;
  }
  HY_DEV void to_f32(float (&f)[8]) const {
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
  }
  HY_DEV void from_f32(const float (&f)[8]) {
    a = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    b = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
  }
};
template <> struct Vec8<__nv_bfloat16> {
  uint4 a;
  HY_DEV void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  HY_DEV void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
  HY_DEV void to_f32(float (&f)[8]) const {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16lo(u[i]);
      f[2 * i + 1] = bf16hi(u[i]);
    }
  }
  HY_DEV void from_f32(const float (&f)[8]) {
    a = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  }
};
template <> struct Vec8<__nv_fp8_e4m3> {
  uint2 a;
  HY_DEV void load(const __nv_fp8_e4m3* p) { a = *reinterpret_cast<const uint2*>(p); }
  HY_DEV void store(__nv_fp8_e4m3* p) const { *reinterpret_cast<uint2*>(p) = a; }
  HY_DEV void to_f32(float (&f)[8]) const {
    const uint32_t u[2] = {a.x, a.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h(__nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>((u[i >> 1] >> (16 * (i & 1))) & 0xFFFFu), __NV_E4M3));
      const float2 v = __half22float2(h);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
  HY_DEV void from_f32(const float (&f)[8]) {
    uint32_t u[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u[i >> 1] |= static_cast<uint32_t>(
                       __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3))
                   << (16 * (i & 1));
    a = make_uint2(u[0], u[1]);
  }
};

}  // namespace hy
