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

// m / 448 rounded to nearest: a quotient within an ulp, corrected once by its exact remainder
// (Markstein's theorem on correctly rounded division; a subnormal quotient is replaced by the
// caller's floor, and the remainder of an infinity or NaN gives NaN).
HY_DEV float div448(float m) {
  constexpr float y = 1.f / 448.f;
  const float q = m * y;
  return fmaf(fmaf(-q, 448.f, m), y, q);
}

// Quantising spends most on what a lane does once per vector (its part of the maximum, the
// scale, the addresses), so a lane then holds 16 elements instead of 8.
template <typename C, bool WRITE> HY_DEV constexpr int lane_vectors() { return WRITE && sizeof(C) == 1 ? 2 : 1; }

// WRITE: x (the batch's rows) -> cache; else cache -> x.  T: element type of x, C: of the cache.
// Bound by HBM when there are many rows; what competes are the instructions around each vector,
// so a thread keeps its place in a row (K or V, head, elements) and walks the rows.
template <typename T, typename C, bool WRITE, int ROWS>
__global__ void __launch_bounds__(kCopyThreads) paged_copy_kernel(const PagedKv kv, const RaggedBatch rb, T* xk, T* xv,
                                                                  long long ld, int lpu, unsigned* status) {
  constexpr bool kQuant = sizeof(C) == 1;
  constexpr int kVec = lane_vectors<C, WRITE>();   // eights of elements a lane holds
  constexpr int kAhead = 4 / kVec;                 // vectors in flight before any is used
  __shared__ long long s_elem[ROWS], s_scale[ROWS];   // the row's place in the pool (-1: none) and among the scales
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
    s_elem[i] = page < 0 ? -1 : (static_cast<long long>(page) * kv.page_size + row) * kv.hkv * kv.dh;
    s_scale[i] = static_cast<long long>(page) * kv.hkv * kv.page_size + row;
  }
  __syncthreads();
  // lpu lanes hold a vector; with fewer (K or V, head) places than groups
  // of lanes the groups share the rows
  const int grp = threadIdx.x / lpu, groups = kCopyThreads / lpu, places = 2 * kv.hkv;
  const int e0 = (threadIdx.x & (lpu - 1)) * 8 * kVec, share = places < groups ? groups / places : 1;
  const int first = places < groups ? grp / places : 0;
  const unsigned mask = (lpu == 32 ? 0xffffffffu : ((1u << lpu) - 1u) << ((threadIdx.x & 31) & ~(lpu - 1)));
  const long long half = static_cast<long long>(kv.n_pages) * kv.page_size * kv.hkv;   // rows x heads of K
  if (first >= share) return;
  for (int place = grp - first * places; place < places; place += groups) {
    const int w = place >= kv.hkv, h = place - w * kv.hkv;
    C* cache = static_cast<C*>(kv.pages) + (w ? half : 0) * kv.dh + h * kv.dh + e0;
    T* x = (w ? xv : xk) + r0 * ld + h * kv.dh + e0;
    float* scales = kQuant ? kv.scales + (w ? half : 0) + static_cast<long long>(h) * kv.page_size : nullptr;
    for (int i0 = first; i0 < ROWS; i0 += kAhead * share) {
      Vec8<T> vx[kAhead][kVec];
      Vec8<C> vc[kAhead][kVec];
      float sc[kAhead];
      long long at[kAhead];   // the row's place in the pool, -1: nothing to do
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k * share;
        at[k] = i < ROWS && e0 < kv.dh ? s_elem[i] : -1;
        sc[k] = 0.f;
        if (at[k] < 0) continue;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          if (WRITE) vx[k][v].load(x + i * ld + 8 * v);
          else vc[k][v].load(cache + at[k] + 8 * v);
        }
        if (!WRITE && kQuant) sc[k] = scales[s_scale[i]];
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k * share;
        float inv = 0.f, s = 0.f;
        if (WRITE && kQuant) {
          uint32_t mb = 0;
          if (at[k] >= 0) {
#pragma unroll
            for (int v = 0; v < kVec; ++v) mb = max(mb, most_bits(vx[k][v]));
          }
          for (int o = lpu >> 1; o > 0; o >>= 1) mb = max(mb, __shfl_xor_sync(mask, mb, o));
          // the floor keeps 1 / scale finite for rows of zeros and of subnormal values
          const float d = div448(__uint_as_float(mb));
          s = d < 1.17549435e-38f ? 1.17549435e-38f : d;
          inv = __frcp_rn(s);
        }
        if (at[k] < 0) continue;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          if constexpr (sizeof(T) == sizeof(C)) {   // as it is
            if (WRITE) vx[k][v].store(reinterpret_cast<T*>(cache + at[k] + 8 * v));
            else vc[k][v].store(reinterpret_cast<C*>(x + i * ld + 8 * v));
          } else {
            float f[8];
            if (WRITE) vx[k][v].to_f32(f);
            else vc[k][v].to_f32(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= WRITE ? inv : sc[k];
            if (WRITE) vc[k][v].from_f32(f);
            else vx[k][v].from_f32(f);
            if (!WRITE) vx[k][v].store(x + i * ld + 8 * v);
          }
        }
        if constexpr (WRITE && kQuant) {
          *reinterpret_cast<uint4*>(cache + at[k]) = make_uint4(vc[k][0].a.x, vc[k][0].a.y, vc[k][kVec - 1].a.x, vc[k][kVec - 1].a.y);
          if (e0 == 0) scales[s_scale[i]] = s;
        }
      }
    }
  }
}

template <typename T, typename C, bool WRITE>
cudaError_t launch_copy_t(const PagedKv& kv, const RaggedBatch& rb, void* k, void* v, long long ld, unsigned* status,
                          cudaStream_t st) {
  const int per_lane = WRITE && sizeof(C) == 1 ? 16 : 8;
  int lpu = 1;
  while (lpu * per_lane < kv.dh) lpu *= 2;
  // many rows: enough vectors a thread that finding the rows' pages does not show; few: many CTAs
  const auto go = [&](auto kernel, int rows) {
    return launch(kernel, dim3((rb.total_rows + rows - 1) / rows), dim3(kCopyThreads), 0, st, kv, rb, static_cast<T*>(k),
                  static_cast<T*>(v), ld, lpu, status);
  };
  return rb.total_rows >= 16 * 4 * num_sms() ? go(paged_copy_kernel<T, C, WRITE, 32>, 32) : go(paged_copy_kernel<T, C, WRITE, 4>, 4);
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
