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
// Many rows: HBM sets the floor; most stalls are waits for the loads, at 7 CTAs of work an SM of which
// five fit at a time, and the scheduler issues in 54 % (into e4m3) and 61 % (back) of its cycles.  A
// thread keeps its place in a row (K or V, head, elements) and walks the rows, to keep what it does
// around each vector small.  33280 rows of 4 x 128 from bf16 into e4m3: 24.1 us, 4.3 TB/s (65 % of
// the measured copy rate); back: 21.7 us, 4.7 TB/s (71 %); 21.8 and 17.8 one behind another.
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
  // many rows: enough vectors a thread that finding the rows' pages does not show; few: many CTAs.
  // (CTAs of 32 rows or of 4, from L2: 33280 rows of 4 x 128 into e4m3 21.7 us, 40.1; back 17.6, 33.6;
  // four rows 5.0, 3.3.  From 16 rows for each of four CTAs
  // per SM on, CTAs of 32 leave no SM without work.)
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

// Attention in fp32 on the CUDA cores: a CTA of four warps per (new row, K/V head, up to eight of
// its query heads).  A warp takes 32 of the visible keys (meta rows below the window, then the
// window up to the row itself) at a time: lane = key for the scores (its K row against the queries
// in shared memory), lane = dims for P V (whole V rows, eight in flight); online softmax, the warps
// joined at the end.  What bounds this kernel is the re-reading of K and V by every row (L2, where a
// lane's K row is not its neighbour's: L1 is busy in 65 % of the cycles, the scheduler in 34 %);
// 4 x 275 rows of 16 x 128 over 275 to 1000 keys each take 766 us.  (The products could run on the
// tensor cores with each fp32 operand in three bf16 parts, as in w4.cu; this kernel does not.)  With
// few rows the keys of a row are split over `splits` CTAs, each leaving its unnormalised output, m and sum per head
// in part[(row * Hq + head) * splits + split][dh + 2]; paged_join_simt joins them.
constexpr int kSimtWarps = 4, kSimtHeads = 8, kSimtDh = 128;

template <typename C>
__global__ void __launch_bounds__(32 * kSimtWarps) paged_attn_simt(const PagedAttnDesc p, float scale_log2, int splits) {
  constexpr bool kScaled = sizeof(C) == 1;
  __shared__ __align__(16) float sq[kSimtHeads][kSimtDh];
  __shared__ float s_m[kSimtWarps][kSimtHeads], s_l[kSimtWarps][kSimtHeads];
  __shared__ float s_o[kSimtWarps][kSimtHeads][kSimtDh];
  pdl_trigger();
  pdl_wait();
  const PagedKv& kv = p.kv;
  const int r = blockIdx.x, kvh = blockIdx.y, group = p.n_q_heads / kv.hkv, dh = kv.dh;
  const int hz = blockIdx.z / splits, split = blockIdx.z - hz * splits;
  const int h0 = kvh * group + hz * kSimtHeads, heads = min(kSimtHeads, group - hz * kSimtHeads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) check_batch(p.rb, kv, p.status);
  const int b = seq_of_row(p.rb, r);
  if (b < 0) return;
  Seq s;
  if (!load_seq(p.rb, kv, b, &s) || r < s.q0 || r >= s.q0 + s.n) return;
  const int i = s.len - s.n + (r - s.q0);
  const float* q = static_cast<const float*>(p.q) + r * p.q_ld + static_cast<long long>(h0) * dh;
  for (int x = threadIdx.x; x < heads * dh; x += 32 * kSimtWarps) sq[x / dh][x % dh] = q[x];
  __syncthreads();
  const int w_lo = p.window < 0 ? 0 : max(0, i - p.window), m_cnt = min(p.n_meta, w_lo);
  const int all = m_cnt + (i - w_lo + 1);
  // this CTA's keys: a multiple of 128 of them each
  const int per = ((all + splits - 1) / splits + 127) / 128 * 128, first = min(all, split * per), n = min(all, first + per);
  const C* pages = static_cast<const C*>(kv.pages);
  const long long half = static_cast<long long>(kv.n_pages) * kv.page_size * kv.hkv;   // rows x heads of K
  float m[kSimtHeads], l[kSimtHeads], o[kSimtHeads][4];
#pragma unroll
  for (int g = 0; g < kSimtHeads; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[g][e] = 0.f;
  }
  for (int c0 = first + warp * 32; c0 < n; c0 += 32 * kSimtWarps) {
    const int x = c0 + lane, j = x < m_cnt ? x : w_lo + (x - m_cnt);
    long long at = -1;   // the key's row x head of the pool, -1: none
    float sk = 1.f, sv = 1.f;
    if (x < n) {
      const int page = page_of(kv, b, j);
      if (page < 0) {
        report_invalid(p.status);
      } else {
        const int row = j % kv.page_size;
        at = (static_cast<long long>(page) * kv.page_size + row) * kv.hkv + kvh;
        if (kScaled) {
          sk = kv.scales[page_scale(kv, 0, page, row, kvh)];
          sv = kv.scales[page_scale(kv, 1, page, row, kvh)];
        }
      }
    }
    float t[kSimtHeads];
#pragma unroll
    for (int g = 0; g < kSimtHeads; ++g) t[g] = 0.f;
    if (at >= 0) {
      for (int d = 0; d < dh; d += 16) {
        Vec8<C> v[2];
        v[0].load(pages + at * dh + d);
        v[1].load(pages + at * dh + d + 8);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float f[8];
          v[u].to_f32(f);
#pragma unroll
          for (int g = 0; g < kSimtHeads; ++g) {
            if (g >= heads) break;
            const float4 a = *reinterpret_cast<const float4*>(&sq[g][d + 8 * u]), c = *reinterpret_cast<const float4*>(&sq[g][d + 8 * u + 4]);
            t[g] = fmaf(a.x, f[0], fmaf(a.y, f[1], fmaf(a.z, f[2], fmaf(a.w, f[3], t[g]))));
            t[g] = fmaf(c.x, f[4], fmaf(c.y, f[5], fmaf(c.z, f[6], fmaf(c.w, f[7], t[g]))));
          }
        }
      }
    }
    float pr[kSimtHeads];
#pragma unroll
    for (int g = 0; g < kSimtHeads; ++g) {
      pr[g] = 0.f;
      if (g >= heads) break;
      const float v = at >= 0 ? t[g] * sk * scale_log2 : -INFINITY;
      float mx = v;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      // no number yet: no key so far, or scores that are all NaN, which the maximum passes over and
      // the sum keeps
      const float mn = fmaxf(m[g], mx), mr = mn == -INFINITY ? 0.f : mn;
      const float corr = exp2f(m[g] - mr), e = exp2f(v - mr);
      float sum = e;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      l[g] = fmaf(l[g], corr, sum);
      m[g] = mn;
      pr[g] = at >= 0 ? e * sv : 0.f;
#pragma unroll
      for (int d = 0; d < 4; ++d) o[g][d] *= corr;
    }
    const int nk = min(32, n - c0);
    for (int k0 = 0; k0 < nk; k0 += 8) {
      float vf[8][4];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const long long row = __shfl_sync(0xffffffffu, at, k0 + u);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          vf[u][e] = row >= 0 && lane + 32 * e < dh ? static_cast<float>(pages[(half + row) * dh + lane + 32 * e]) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int g = 0; g < kSimtHeads; ++g) {
          if (g >= heads) break;
          const float w = __shfl_sync(0xffffffffu, pr[g], k0 + u);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[g][e] = fmaf(w, vf[u][e], o[g][e]);
        }
    }
  }
#pragma unroll
  for (int g = 0; g < kSimtHeads; ++g) {
    if (g >= heads) break;
    if (lane == 0) {
      s_m[warp][g] = m[g];
      s_l[warp][g] = l[g];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (lane + 32 * e < dh) s_o[warp][g][lane + 32 * e] = o[g][e];
  }
  __syncthreads();
  float* out = static_cast<float*>(p.out) + r * p.out_ld + static_cast<long long>(h0) * dh;
  for (int x = threadIdx.x; x < heads * dh; x += 32 * kSimtWarps) {
    const int g = x / dh, d = x - g * dh;
    float mm = -INFINITY, ll = 0.f, oo = 0.f;
#pragma unroll
    for (int w = 0; w < kSimtWarps; ++w) mm = fmaxf(mm, s_m[w][g]);
#pragma unroll
    for (int w = 0; w < kSimtWarps; ++w) {
      const float f = s_m[w][g] == -INFINITY ? 0.f : exp2f(s_m[w][g] - mm);
      ll = fmaf(s_l[w][g], f, ll);
      oo = fmaf(s_o[w][g][d], f, oo);
    }
    if (splits == 1) {
      out[x] = ll != 0.f ? oo / ll : 0.f;
    } else {
      float* part = static_cast<float*>(p.scratch) +
                    ((static_cast<long long>(r) * p.n_q_heads + h0 + g) * splits + split) * (dh + 2);
      part[d] = oo;
      if (d == 0) {
        part[dh] = mm;
        part[dh + 1] = ll;
      }
    }
  }
}

__global__ void __launch_bounds__(128) paged_join_simt(const PagedAttnDesc p, int splits) {
  pdl_trigger();
  pdl_wait();
  const int r = blockIdx.x, h = blockIdx.y, dh = p.kv.dh, b = seq_of_row(p.rb, r);
  Seq s;
  if (b < 0 || !load_seq(p.rb, p.kv, b, &s) || r < s.q0 || r >= s.q0 + s.n) return;   // (left as it was)
  const float* part = static_cast<const float*>(p.scratch) + (static_cast<long long>(r) * p.n_q_heads + h) * splits * (dh + 2);
  float mm = -INFINITY;
  for (int c = 0; c < splits; ++c) mm = fmaxf(mm, part[c * (dh + 2) + dh]);
  for (int d = threadIdx.x; d < dh; d += 128) {
    float ll = 0.f, oo = 0.f;
    for (int c = 0; c < splits; ++c) {
      const float* q = part + c * (dh + 2);
      const float f = q[dh] == -INFINITY ? 0.f : exp2f(q[dh] - mm);
      ll = fmaf(q[dh + 1], f, ll);
      oo = fmaf(q[d], f, oo);
    }
    static_cast<float*>(p.out)[r * p.out_ld + static_cast<long long>(h) * dh + d] = ll != 0.f ? oo / ll : 0.f;
  }
}

// CTAs over which the keys of a row are split: four CTAs per SM of the B200 in all, and no piece
// shorter than 128 keys of the longest sequence that the table holds (one token over 4000 rows: 27 us,
// unsplit 425).
constexpr long long kSimtCtas = 4 * 148;
long long simt_row_ctas(const PagedKv& kv, int n_q_heads) {   // without a split
  return static_cast<long long>(kv.hkv) * ((n_q_heads / kv.hkv + kSimtHeads - 1) / kSimtHeads);
}
long long simt_most_splits(const PagedKv& kv) {
  const long long most = (static_cast<long long>(kv.table_ld) * kv.page_size + 127) / 128;
  return most < 64 ? most : 64;
}
int simt_splits(const PagedKv& kv, const RaggedBatch& rb, int n_q_heads) {
  const long long ctas = rb.total_rows * simt_row_ctas(kv, n_q_heads), most = simt_most_splits(kv);
  const long long s = ctas > 0 ? kSimtCtas / ctas : 1;
  return s < 1 ? 1 : static_cast<int>(s < most ? s : most);
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
  if (!bf16) {
    // rows x splits: fewer rows are split further, so that what holds the most rows' parts holds any
    // smaller call's (a server's one workspace)
    const long long any = kSimtCtas / simt_row_ctas(kv, n_q_heads), most = simt_most_splits(kv), all = rb.total_rows * most;
    return any < 2 || most < 2 ? 0 : static_cast<size_t>(any < all ? any : all) * n_q_heads * (kv.dh + 2) * 4;
  }
  return paged_decode_takes(kv, rb, n_q_heads) ? paged_decode_scratch(kv, rb, n_q_heads) : paged_attention_tc_scratch(kv, rb, n_q_heads);
}

cudaError_t launch_paged_attention(const PagedAttnDesc& a, cudaStream_t st) {
  if (a.bf16) return paged_decode_takes(a.kv, a.rb, a.n_q_heads) ? launch_paged_decode(a, st) : launch_paged_attention_tc(a, st);
  const int group = a.n_q_heads / a.kv.hkv, splits = simt_splits(a.kv, a.rb, a.n_q_heads);
  const dim3 grid(a.rb.total_rows, a.kv.hkv, (group + kSimtHeads - 1) / kSimtHeads * splits);
  const float scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(a.kv.dh));
  const cudaError_t e =
      a.kv.type == CACHE_E4M3 ? launch(paged_attn_simt<__nv_fp8_e4m3>, grid, dim3(32 * kSimtWarps), 0, st, a, scale_log2, splits)
                              : launch(paged_attn_simt<float>, grid, dim3(32 * kSimtWarps), 0, st, a, scale_log2, splits);
  if (e != cudaSuccess || splits == 1) return e;
  return launch(paged_join_simt, dim3(a.rb.total_rows, a.n_q_heads), dim3(128), 0, st, a, splits);
}

}  // namespace hy
