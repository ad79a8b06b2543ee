// paged.cu -- the paged K/V cache of the attention heads (blog.outta.ai Hymba review,
// "Efficiency and KV cache optimization"): new rows written into the pages (quantised to
// e4m3 with one scale per row and head, or as they are), cache rows read back, and the
// attention of the new rows over the cache on the CUDA cores (fp32).
//
//   paged_copy_kernel   a CTA takes ROWS rows of the batch: one thread per row finds its
//                       sequence and page, then groups of lanes (eight elements each) move
//                       one (row, K or V, head) vector, with the maximum over the group by
//                       shuffles when it is quantised.
#include "paged.cuh"

namespace hy {
namespace {

constexpr int kCopyThreads = 256;

// n / d for n * d < 2^32 with d's multiplier ceil(2^32 / d) (0 for d = 1).
HY_DEV int div_by(int n, uint32_t mul) { return mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(n), mul)) : n; }
uint32_t multiplier(int d) { return d == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + d - 1) / d); }

// The largest magnitude among a vector's eight elements, as the bits of an fp32 value: a NaN is
// the largest of all.
HY_DEV uint32_t most_bits(const Vec8<float>& v) {
  const uint32_t u[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, u[i] & 0x7fffffffu);
  return m;
}
HY_DEV uint32_t most_bits(const Vec8<__nv_bfloat16>& v) {   // two 16-bit maxima at a time
  const uint32_t m = __vmaxu2(__vmaxu2(v.a.x & 0x7fff7fffu, v.a.y & 0x7fff7fffu), __vmaxu2(v.a.z & 0x7fff7fffu, v.a.w & 0x7fff7fffu));
  return max(m << 16, m & 0xffff0000u);
}
HY_DEV uint32_t most_bits(const Vec8<__nv_fp8_e4m3>&) { return 0; }   // (never quantised)

// WRITE: x (the batch's rows) -> cache; else cache -> x.  T: element type of x, C: of the cache.
// Bound by HBM when there are many rows; then the instructions of the address arithmetic and the
// conversions are what competes (a division per vector and a whole maximum per element: 41 us
// for 4 x 8320 rows of 4 heads where the bytes take 16).
template <typename T, typename C, bool WRITE, int ROWS>
__global__ void __launch_bounds__(kCopyThreads) paged_copy_kernel(const PagedKv kv, const RaggedBatch rb, T* xk, T* xv,
                                                                  long long ld, int lpu, uint32_t row_mul,
                                                                  unsigned* status) {
  constexpr bool kQuant = sizeof(C) == 1;
  constexpr int kAhead = 4;   // vectors in flight before any is used
  __shared__ int s_page[ROWS], s_row[ROWS];
  pdl_trigger();
  pdl_wait();
  const int r0 = blockIdx.x * ROWS;
  if (blockIdx.x == 0) check_batch(rb, kv, status);
  for (int i = threadIdx.x; i < ROWS; i += kCopyThreads) {
    int page = -1, row = 0;
    const int r = r0 + i;
    const int b = r < rb.total_rows ? seq_of_row(rb, r) : -1;
    if (b >= 0) {
      Seq s;
      if (load_seq(rb, kv, b, &s) && r >= s.q0 && r < s.q0 + s.n) {
        const int at = s.len - s.n + (r - s.q0);
        page = page_of(kv, b, at);
        row = at % kv.page_size;
        if (page < 0) report_invalid(status);
      }
    }
    s_page[i] = page;
    s_row[i] = row;
  }
  __syncthreads();
  const int e0 = (threadIdx.x & (lpu - 1)) * 8, per_row = 2 * kv.hkv;
  const int units = ROWS * per_row, step = kCopyThreads / lpu;
  const long long v_off = static_cast<long long>(kv.n_pages) * kv.page_size * kv.hkv;   // rows x heads of one half
  for (int u0 = threadIdx.x / lpu; u0 < units; u0 += kAhead * step) {
    Vec8<T> vx[kAhead];
    Vec8<C> vc[kAhead];
    T* px[kAhead];
    C* pc[kAhead];       // nullptr: nothing to do
    float* ps[kAhead];
    float sc[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int u = u0 + k * step, i = min(div_by(u, row_mul), ROWS - 1), slot = u - i * per_row;
      const int w = slot >= kv.hkv, h = slot - w * kv.hkv, page = s_page[i];
      pc[k] = nullptr;
      sc[k] = 0.f;
      if (u >= units || page < 0 || e0 >= kv.dh) continue;
      const long long at = static_cast<long long>(page) * kv.page_size + s_row[i];
      pc[k] = static_cast<C*>(kv.pages) + ((at * kv.hkv + h) + (w ? v_off : 0)) * kv.dh + e0;
      px[k] = (w ? xv : xk) + (r0 + i) * ld + h * kv.dh + e0;
      if (kQuant) ps[k] = kv.scales + (static_cast<long long>(page) * kv.hkv + h) * kv.page_size + s_row[i] + (w ? v_off : 0);
      if (WRITE) {
        vx[k].load(px[k]);
      } else {
        vc[k].load(pc[k]);
        if (kQuant) sc[k] = *ps[k];
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (sizeof(T) == sizeof(C)) {   // as it is
        if (!pc[k]) continue;
        if (WRITE) *reinterpret_cast<Vec8<T>*>(&vc[k]) = vx[k];
        else vx[k] = *reinterpret_cast<Vec8<T>*>(&vc[k]);
      } else if (WRITE) {
        uint32_t mb = pc[k] ? most_bits(vx[k]) : 0u;
        for (int o = lpu >> 1; o > 0; o >>= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
        if (!pc[k]) continue;
        // the floor keeps 1 / scale finite for rows of zeros and of subnormal values
        const float d = __fdiv_rn(__uint_as_float(mb), 448.f);
        sc[k] = d < 1.17549435e-38f ? 1.17549435e-38f : d;
        const float inv = __frcp_rn(sc[k]);
        float f[8];
        vx[k].to_f32(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= inv;
        vc[k].from_f32(f);
        if (e0 == 0) *ps[k] = sc[k];
      } else {
        if (!pc[k]) continue;
        float f[8];
        vc[k].to_f32(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= sc[k];
        vx[k].from_f32(f);
      }
      if (WRITE) vc[k].store(pc[k]);
      else vx[k].store(px[k]);
    }
  }
}

template <typename T, typename C, bool WRITE>
cudaError_t launch_copy_t(const PagedKv& kv, const RaggedBatch& rb, void* k, void* v, long long ld, unsigned* status,
                          cudaStream_t st) {
  int lpu = 2;
  while (lpu * 8 < kv.dh) lpu *= 2;
  // many rows: enough vectors a thread that finding the rows' pages does not show; few: many CTAs
  const uint32_t rm = multiplier(2 * kv.hkv);
  const auto go = [&](auto kernel, int rows) {
    return launch(kernel, dim3((rb.total_rows + rows - 1) / rows), dim3(kCopyThreads), 0, st, kv, rb, static_cast<T*>(k),
                  static_cast<T*>(v), ld, lpu, rm, status);
  };
  return rb.total_rows >= 16 * 4 * num_sms() ? go(paged_copy_kernel<T, C, WRITE, 16>, 16) : go(paged_copy_kernel<T, C, WRITE, 4>, 4);
}

template <bool WRITE>
cudaError_t launch_copy(const PagedKv& kv, const RaggedBatch& rb, void* k, void* v, long long ld, bool bf16,
                        unsigned* status, cudaStream_t st) {
  if (rb.total_rows <= 0) return cudaSuccess;
  if (kv.type == CACHE_E4M3)
    return bf16 ? launch_copy_t<__nv_bfloat16, __nv_fp8_e4m3, WRITE>(kv, rb, k, v, ld, status, st)
                : launch_copy_t<float, __nv_fp8_e4m3, WRITE>(kv, rb, k, v, ld, status, st);
  return bf16 ? launch_copy_t<__nv_bfloat16, __nv_bfloat16, WRITE>(kv, rb, k, v, ld, status, st)
              : launch_copy_t<float, float, WRITE>(kv, rb, k, v, ld, status, st);
}

// Attention, one warp per (new row, query head): online softmax in fp32 over the visible
// keys (meta rows below the window, then the window up to the row itself).
template <typename T, typename C>
__global__ void __launch_bounds__(128) paged_attn_simt(const PagedAttnDesc p, float scale) {
  pdl_trigger();
  pdl_wait();
  const PagedKv& kv = p.kv;
  const long long wid = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, dh = kv.dh;
  if (blockIdx.x == 0) check_batch(p.rb, kv, p.status);
  if (wid >= static_cast<long long>(p.rb.total_rows) * p.n_q_heads) return;
  const int r = static_cast<int>(wid / p.n_q_heads), h = static_cast<int>(wid % p.n_q_heads);
  const int kvh = h / (p.n_q_heads / kv.hkv);
  const int b = seq_of_row(p.rb, r);
  if (b < 0) return;
  Seq s;
  if (!load_seq(p.rb, kv, b, &s) || r < s.q0 || r >= s.q0 + s.n) return;
  const int i = s.len - s.n + (r - s.q0);
  float qv[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
  const T* q = static_cast<const T*>(p.q) + r * p.q_ld + h * dh;
#pragma unroll
  for (int e = 0; e < 4; ++e) qv[e] = lane + 32 * e < dh ? to_f<T>(q[lane + 32 * e]) : 0.f;
  const int w_lo = p.window < 0 ? 0 : max(0, i - p.window), m_cnt = min(p.n_meta, w_lo);
  const int n = m_cnt + (i - w_lo + 1);
  const C* pages = static_cast<const C*>(kv.pages);
  float m = -INFINITY, l = 0.f;
  for (int x = 0; x < n; ++x) {
    const int j = x < m_cnt ? x : w_lo + (x - m_cnt);
    const int page = page_of(kv, b, j), row = j % kv.page_size;
    if (page < 0) {
      if (lane == 0) report_invalid(p.status);
      continue;
    }
    const C* k = pages + page_elem(kv, 0, page, row, kvh);
    const C* v = pages + page_elem(kv, 1, page, row, kvh);
    float sk = 1.f, sv = 1.f;
    if (kv.type == CACHE_E4M3) {
      sk = kv.scales[page_scale(kv, 0, page, row, kvh)];
      sv = kv.scales[page_scale(kv, 1, page, row, kvh)];
    }
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (lane + 32 * e < dh) t = fmaf(qv[e], static_cast<float>(k[lane + 32 * e]), t);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    t *= scale * sk;
    const float mn = fmaxf(m, t);
    const float corr = expf(m - mn), pj = expf(t - mn);
    l = l * corr + pj;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (lane + 32 * e < dh) acc[e] = acc[e] * corr + pj * sv * static_cast<float>(v[lane + 32 * e]);
    m = mn;
  }
  T* out = static_cast<T*>(p.out) + r * p.out_ld + h * dh;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (lane + 32 * e < dh) out[lane + 32 * e] = from_f<T>(l != 0.f ? acc[e] / l : 0.f);
}

}  // namespace

cudaError_t launch_paged_append(const PagedKv& kv, const RaggedBatch& rb, const void* k, const void* v, long long ld,
                                bool bf16, unsigned* status, cudaStream_t st) {
  return launch_copy<true>(kv, rb, const_cast<void*>(k), const_cast<void*>(v), ld, bf16, status, st);
}

cudaError_t launch_paged_read(const PagedKv& kv, const RaggedBatch& rb, void* k, void* v, long long ld, bool bf16,
                              unsigned* status, cudaStream_t st) {
  return launch_copy<false>(kv, rb, k, v, ld, bf16, status, st);
}

// paged_decode.cu (at most 16 rows per K/V head) and paged_attn_tc.cu
bool paged_decode_takes(const PagedKv& kv, const RaggedBatch& rb, int n_q_heads);
size_t paged_decode_scratch(const PagedKv& kv, const RaggedBatch& rb, int n_q_heads);
cudaError_t launch_paged_decode(const PagedAttnDesc& a, cudaStream_t st);
size_t paged_attention_tc_scratch(const PagedKv& kv, const RaggedBatch& rb, int n_q_heads);
cudaError_t launch_paged_attention_tc(const PagedAttnDesc& a, cudaStream_t st);

size_t paged_attention_scratch(const PagedKv& kv, const RaggedBatch& rb, int n_q_heads, bool bf16) {
  if (!bf16) return 0;
  return paged_decode_takes(kv, rb, n_q_heads) ? paged_decode_scratch(kv, rb, n_q_heads) : paged_attention_tc_scratch(kv, rb, n_q_heads);
}

cudaError_t launch_paged_attention(const PagedAttnDesc& a, cudaStream_t st) {
  if (a.bf16) return paged_decode_takes(a.kv, a.rb, a.n_q_heads) ? launch_paged_decode(a, st) : launch_paged_attention_tc(a, st);
  const long long warps = static_cast<long long>(a.rb.total_rows) * a.n_q_heads;
  if (warps <= 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((warps + 3) / 4));
  const float scale = 1.f / sqrtf(static_cast<float>(a.kv.dh));
  return a.kv.type == CACHE_E4M3 ? launch(paged_attn_simt<float, __nv_fp8_e4m3>, grid, dim3(128), 0, st, a, scale)
                                 : launch(paged_attn_simt<float, float>, grid, dim3(128), 0, st, a, scale);
}

}  // namespace hy
