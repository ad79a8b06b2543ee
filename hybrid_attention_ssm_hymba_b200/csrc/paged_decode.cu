// paged_decode.cu -- attention of a few new rows per sequence (a generation step: at most 16
// rows per K/V head, counting its query heads) over the paged K/V cache (blog.outta.ai Hymba
// review, "Efficiency and KV cache optimization").
//
//   out = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),  s_j = log2(e) q.k_j / sqrt(dh)
//
// Every K/V row is read once for all query heads that share it, and that reading bounds the
// call.  The products are mma.sync m16n8k16 with the keys (Q K^T) and the dims (P V) as the
// sixteen rows and the queries as the eight columns, one or two such tiles (a 128-row
// tensor-core tile would be mostly empty, and its K and V would have to pass through shared
// memory); K and V go from global memory straight to the registers that the products read: the
// order of the summed index and of the output's rows is free, so each lane loads 16 consecutive
// bytes of a row and the products are told apart by that order alone.
//   K Q^T  lane (g, t) holds, of keys g and g + 8 of sixteen, the dims of its 16-byte pieces
//          (the four lanes of a key read 64 consecutive bytes); Q is read in the same order.
//   V^T P^T  lane (g, t) holds keys 2t, 2t+1, 2t+8, 2t+9 of sixteen at the dims of piece g
//          (eight lanes read 128 consecutive bytes); the two keys of a register are put together
//          by one byte permutation, and P's 8 x 8 pieces are transposed between the lanes.
// A CTA of four warps takes 32 keys of each 128-key block per warp and walks its part of the
// line of blocks (paged_plan.cuh).  K of the next step is loaded as soon as K Q^T has read this
// one's, V as soon as V^T P^T has, page numbers two steps and scales one step earlier.  16 long e4m3
// histories (348 MB): 69 us, 5.0 TB/s, 77 % of the measured copy rate, three CTAs an SM with 27 million
// warp instructions in 40 % of the issue slots.  4 rows in a window of 1024: 11.8 us, of which the bytes
// are 1.4; the rest is two launches, the plan, a page number's, a row's and the join's way from memory.
//
// e4m3 codes are exact in fp16, one conversion for two of them, so the 8-bit products run in
// fp16 with their ranges kept by powers of two: a row of Q is scaled to at most 2^8 (its bf16
// values stay exact down to 2^-25 of the largest), and P V sums n_j = 2^(s_j + log2 sv_j - m' + 8)
// times the codes, with a running maximum m' of its own, while sum_j 2^(s_j - m) is kept apart.
#include "paged_plan.cuh"

namespace hy {
namespace {

constexpr int DH = 128, kWarps = 4, kRows = 16;
// Batches up to this are planned by every CTA itself (4 rows in a window of 1024: 11.8 us, with the
// plan kernel 18.8; 1000 of them 372 and 396).
constexpr int kPlanBatch = 1024;
constexpr float kLazy = 7.f;       // a maximum moves when it is exceeded by 2^7: n_j stays below 2^15
constexpr float kLazySum = 60.f;   // the same for a sum in fp32
constexpr float kUp = 8.f;         // the exponent added to n_j

template <bool F16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 ldg_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Two bf16 values times f as fp16.
__device__ __forceinline__ uint32_t f16_of_bf16(uint32_t u, float f) { return pack_f16(bf16lo(u) * f, bf16hi(u) * f); }
// The transpose of an 8 x 8 matrix of 16-bit values, row g's columns 2t, 2t + 1 in lane (g, t).
__device__ __forceinline__ uint32_t transpose8(uint32_t u) {
  uint32_t v;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(v) : "r"(u));
  return v;
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One key of a step, held by the lane of its number: its row of the pool (-1: not to be read)
// and its scales, V's as its logarithm.
struct Key {
  int row;
  float sk, sv;
};

struct Shared {
  float m[kWarps][kRows], l[kWarps][kRows];
  float o[kWarps][kRows][DH + 4];
  long long prefix[kPlanBatch + 1];
  long long warp_sum[kWarps];
};

// prefix of paged_plan_kernel by one CTA, one tile per sequence and head.
__device__ void plan_here(const PagedAttnParams& p, Shared& sm, bool report) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long carry = 0;
  for (int b0 = 0; b0 < p.rb.batch; b0 += 32 * kWarps) {
    const int b = b0 + threadIdx.x;
    long long own = 0;
    Seq s;
    if (b < p.rb.batch) {
      if (!load_seq(p.rb, p.kv, b, &s)) {
        if (report) report_invalid(p.status);
      } else if (s.n > 0) {
        own = static_cast<long long>(tile_span(p.g, s, 0).n) * p.kv.hkv;
      }
    }
    long long v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) sm.warp_sum[warp] = v;
    __syncthreads();
    long long all = 0, before = carry;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sm.warp_sum[w];
      all += sm.warp_sum[w];
    }
    if (b < p.rb.batch) sm.prefix[b] = before + v - own;
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) sm.prefix[p.rb.batch] = carry;
  __syncthreads();
}

// NT: tiles of eight queries.
template <bool FP8, int NT>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 ? 3 : 2) paged_decode_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int kStep = FP8 ? 32 : 16;       // keys of a warp's step: 4 KB of K and of V either way
  constexpr int kSub = 32 / kStep;           // steps per block and warp
  constexpr int kKt = kStep / 16;
  constexpr int es = FP8 ? 1 : 2;
  constexpr unsigned kAll = kStep == 32 ? 0xffffffffu : 0xffffu;
  __shared__ Shared sm;
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const long long* prefix = p.prefix;
  if (p.rb.batch <= kPlanBatch) {
    plan_here(p, sm, blockIdx.x == 0);
    prefix = sm.prefix;
  }
  const uint8_t* kbase = static_cast<const uint8_t*>(p.kv.pages);
  const uint8_t* vbase = kbase + static_cast<long long>(p.kv.n_pages) * p.kv.page_size * p.kv.hkv * DH * es;
  const long long row_bytes = static_cast<long long>(p.kv.hkv) * DH * es;

  PieceWalk walk(p, prefix, threadIdx.x == 0);
  Piece pc;
  while (walk.next(p, &pc, threadIdx.x == 0)) {
    const int rows = pc.ts.toks * p.g.G;
    // Q of queries 8 n + g in the dims' order; qs turns the products of queries 8 n + 2t + e into
    // log2 units; at: those queries' places in the sequence
    uint32_t qb[NT][8][2];
    float qs[NT][2];
    int at[NT][2];
    {
      const __nv_bfloat16* q0 = p.q + pc.row0 * p.q_ld + static_cast<long long>(pc.kvh) * p.g.G * DH;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = 8 * n + g;
        const uint4* q = reinterpret_cast<const uint4*>(q0 + (r / p.g.G) * p.q_ld + (r % p.g.G) * DH);
        uint4 v[4];
        uint32_t mx = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // bf16: piece t of 32 dims j; e4m3: dims 64 (j / 2) + 16 t + 8 (j % 2)
          v[j] = r < rows ? q[FP8 ? (j >> 1) * 8 + t * 2 + (j & 1) : j * 4 + t] : make_uint4(0, 0, 0, 0);
          if (FP8) {
#pragma unroll
            for (int w = 0; w < 4; ++w) mx = max(mx, max(word(v[j], w) & 0x7fffu, (word(v[j], w) >> 16) & 0x7fffu));
          }
        }
        float up = 1.f, down = p.scale_log2;
        if (FP8) {   // the row times 2^(f - 127), so that its largest value is in [2^7, 2^8)
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const int f = min(261 - static_cast<int>(mx >> 7), 253);
          up = __uint_as_float(static_cast<uint32_t>(f) << 23);
          down *= __uint_as_float(static_cast<uint32_t>(254 - f) << 23);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          qb[n][2 * j][0] = FP8 ? f16_of_bf16(v[j].x, up) : v[j].x;
          qb[n][2 * j][1] = FP8 ? f16_of_bf16(v[j].y, up) : v[j].y;
          qb[n][2 * j + 1][0] = FP8 ? f16_of_bf16(v[j].z, up) : v[j].z;
          qb[n][2 * j + 1][1] = FP8 ? f16_of_bf16(v[j].w, up) : v[j].w;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          qs[n][e] = __shfl_sync(0xffffffffu, down, (2 * t + e) * 4);
          at[n][e] = pc.ts.p0 + (8 * n + 2 * t + e) / p.g.G;
        }
      }
    }
    const int lo = p.g.window < 0 ? 0 : pc.ts.p0 - p.g.window;             // first key of any row's window
    const uint8_t* kh = kbase + pc.kvh * (DH * es) + t * 16;
    const uint8_t* vh = vbase + pc.kvh * (DH * es) + g * 16;
    const int* table = p.kv.table + static_cast<long long>(pc.b) * p.kv.table_ld;

    const int steps = (pc.blk1 - pc.blk0) * kSub;
    auto key0 = [&](int s) { return pc.ts.block(pc.blk0 + s / kSub) * kKeyBlock + warp * 32 + (s % kSub) * kStep; };
    // this lane's key of step s: its page number (kNoKey: nobody sees it), then its row and scales
    constexpr int kNoKey = -2147483647 - 1;
    auto lookup = [&](int s) {
      const int j = key0(s) + lane;
      if (s >= steps || lane >= kStep || j > pc.ts.p1 || (j < lo && j >= p.g.n_meta)) return kNoKey;
      const int page = table[p.page_shift >= 0 ? j >> p.page_shift : j / p.kv.page_size];
      return page == kNoKey ? -1 : page;
    };
    auto find = [&](int s, int page) -> Key {
      Key k{-1, 0.f, 0.f};
      if (page == kNoKey) return k;
      if (page < 0 || page >= p.kv.n_pages) {
        report_invalid(p.status);
        return k;
      }
      const int j = key0(s) + lane, at = p.page_shift >= 0 ? j & (p.kv.page_size - 1) : j % p.kv.page_size;
      k.row = page * p.kv.page_size + at;
      if (FP8) {
        k.sk = p.kv.scales[page_scale(p.kv, 0, page, at, pc.kvh)];
        k.sv = p.kv.scales[page_scale(p.kv, 1, page, at, pc.kvh)];
      }
      return k;
    };
    // a key that is not there loads the pool's first row (a predicated or branched load costs the
    // kernel a quarter of its time and more); its scores are hidden and its V is zeroed below
    constexpr int kLoadsK = FP8 ? 2 : 4, kLoadsV = FP8 ? 1 : 2;   // 16-byte pieces of a key per lane
    uint4 kr[kKt][2][kLoadsK], vr[kKt][4][kLoadsV];
    auto load_k = [&](const Key& k) {
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = __shfl_sync(0xffffffffu, k.row, kt * 16 + h * 8 + g);
          const uint8_t* a = kh + max(row, 0) * row_bytes;
#pragma unroll
          for (int j = 0; j < kLoadsK; ++j) kr[kt][h][j] = ldg_once(a + j * 64);
        }
    };
    auto load_v = [&](const Key& k) {
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int row = __shfl_sync(0xffffffffu, k.row, kt * 16 + 2 * t + (c & 1) + (c >> 1) * 8);
          const uint8_t* a = vh + max(row, 0) * row_bytes;
#pragma unroll
          for (int h = 0; h < kLoadsV; ++h) vr[kt][c][h] = ldg_once(a + h * 128);
        }
    };

    // of queries 8 n + 2t + e: m, l of the softmax; mp (e4m3) the running maximum of what P V sums
    float o[NT][8][4], m[NT][2], mp[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[n][e] = mp[n][e] = -INFINITY;
        l[n][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
    }
    const int pg1 = lookup(1);
    int pg2 = lookup(2);
    Key cur = find(0, lookup(0)), nxt = find(1, pg1);
    load_k(cur);
    load_v(cur);
    for (int s = 0; s < steps; ++s) {
      // sc[n][kt]: keys g (elements 0, 1) and g + 8 (2, 3) of sixteen, queries 2t (0, 2), 2t + 1 (1, 3)
      float sc[NT][kKt][4];
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][kt][e] = 0.f;
#pragma unroll
        for (int j = 0; j < kLoadsK; ++j) {
#pragma unroll
          for (int w = 0; w < (FP8 ? 4 : 2); ++w) {
            uint32_t a[4];
            if constexpr (FP8) {
              a[0] = f16_of_e4m3(word(kr[kt][0][j], w), 0);
              a[1] = f16_of_e4m3(word(kr[kt][1][j], w), 0);
              a[2] = f16_of_e4m3(word(kr[kt][0][j], w), 1);
              a[3] = f16_of_e4m3(word(kr[kt][1][j], w), 1);
            } else {
              a[0] = word(kr[kt][0][j], 2 * w);
              a[1] = word(kr[kt][1][j], 2 * w);
              a[2] = word(kr[kt][0][j], 2 * w + 1);
              a[3] = word(kr[kt][1][j], 2 * w + 1);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint32_t (&b)[2] = qb[n][(FP8 ? 4 : 2) * j + w];
              mma16<FP8>(sc[n][kt], a, b[0], b[1]);
            }
          }
        }
      }
      if (s + 1 < steps) load_k(nxt);
      // K's scales and log2 of V's, of keys g and g + 8
      float lv[kKt][2];
      const float own_lv = FP8 && cur.row >= 0 ? lg2_approx(cur.sv) : 0.f;
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          lv[kt][h] = 0.f;
          if (FP8) {
            const float sk = __shfl_sync(0xffffffffu, cur.sk, kt * 16 + h * 8 + g);
            lv[kt][h] = __shfl_sync(0xffffffffu, own_lv, kt * 16 + h * 8 + g);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              sc[n][kt][2 * h] *= sk;
              sc[n][kt][2 * h + 1] *= sk;
            }
          }
        }
      // hidden keys -inf (most steps have none)
      const int k0 = key0(s), k1 = k0 + kStep - 1;
      const unsigned there = __ballot_sync(0xffffffffu, cur.row >= 0);
      if (there != kAll || k1 > pc.ts.p0 || (p.g.window >= 0 && pc.ts.p1 - k0 > p.g.window && k1 >= p.g.n_meta)) {
#pragma unroll
        for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = kt * 16 + h * 8 + g;
            const bool in = (there >> c) & 1u;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (!in || !key_visible(p.g, at[n][e], k0 + c)) sc[n][kt][2 * h + e] = -INFINITY;
          }
      }
      // this lane's maxima of each query: of the scores and (e4m3) of the scores with log2 sv in
      // them.  The lanes meet only when one of them has to move a reference: sums of 2^(s - m)
      // stay finite far beyond m, P's 16 bits set the limit for what they hold
      bool move = false;
      float mx[NT][2], mxp[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = -INFINITY, y = -INFINITY;
#pragma unroll
          for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              x = fmaxf(x, sc[n][kt][2 * h + e]);
              if (FP8) y = fmaxf(y, fmaf(sc[n][kt][2 * h + e], qs[n][e], lv[kt][h]));
            }
          mx[n][e] = x * qs[n][e];
          mxp[n][e] = y;
          move |= mx[n][e] > m[n][e] + (FP8 ? kLazySum : kLazy) || (FP8 && y > mp[n][e] + kLazy);
        }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float nm = fmaxf(m[n][e], mx[n][e]), np = fmaxf(mp[n][e], mxp[n][e]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, d));
              if (FP8) np = fmaxf(np, __shfl_xor_sync(0xffffffffu, np, d));
            }
            const float al = nm == -INFINITY ? 1.f : ex2_approx(m[n][e] - nm);
            const float ao = FP8 ? (np == -INFINITY ? 1.f : ex2_approx(mp[n][e] - np)) : al;
            l[n][e] *= al;
            m[n][e] = nm;
            mp[n][e] = FP8 ? np : nm;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[n][i][e] *= ao;
              o[n][i][2 + e] *= ao;
            }
          }
      }
      uint32_t pb[NT][kKt][2];   // P, rounded once to the products' 16 bits, transposed
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float r[2], rp[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          r[e] = m[n][e] == -INFINITY ? 0.f : m[n][e];
          rp[e] = mp[n][e] == -INFINITY ? 0.f : mp[n][e] - kUp;
        }
#pragma unroll
        for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float s0 = sc[n][kt][2 * h], s1 = sc[n][kt][2 * h + 1];
            const float x0 = ex2_approx(fmaf(s0, qs[n][0], -r[0])), x1 = ex2_approx(fmaf(s1, qs[n][1], -r[1]));
            l[n][0] += x0;
            l[n][1] += x1;
            pb[n][kt][h] = transpose8(FP8 ? pack_f16(ex2_approx(fmaf(s0, qs[n][0], lv[kt][h] - rp[0])),
                                                     ex2_approx(fmaf(s1, qs[n][1], lv[kt][h] - rp[1])))
                                          : pack_bf16(x0, x1));
          }
      }
      // O += P V
      if (there != kAll) {
#pragma unroll
        for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int h = 0; h < kLoadsV; ++h)
              if (!((there >> (kt * 16 + 2 * t + (c & 1) + (c >> 1) * 8)) & 1u)) vr[kt][c][h] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // two neighbouring dims, of two keys each: the pieces' word i / 2 (e4m3), i (bf16)
          const int w = FP8 ? i >> 1 : i & 3, h = FP8 ? 0 : i >> 2;
          const uint32_t a0 = word(vr[kt][0][h], w), a1 = word(vr[kt][1][h], w), a2 = word(vr[kt][2][h], w), a3 = word(vr[kt][3][h], w);
          uint32_t a[4];
          if constexpr (FP8) {
            const uint32_t sel = i & 1 ? 0x7362 : 0x5140;
            const uint32_t x = __byte_perm(a0, a1, sel), y = __byte_perm(a2, a3, sel);
            a[0] = f16_of_e4m3(x, 0);
            a[1] = f16_of_e4m3(x, 1);
            a[2] = f16_of_e4m3(y, 0);
            a[3] = f16_of_e4m3(y, 1);
          } else {
            a[0] = __byte_perm(a0, a1, 0x5410);
            a[1] = __byte_perm(a0, a1, 0x7632);
            a[2] = __byte_perm(a2, a3, 0x5410);
            a[3] = __byte_perm(a2, a3, 0x7632);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16<FP8>(o[n][i], a, pb[n][kt][0], pb[n][kt][1]);
        }
      if (s + 1 < steps) load_v(nxt);
      cur = nxt;
      nxt = find(s + 2, pg2);
      pg2 = lookup(s + 3);
    }
    // the lanes of a query, then the four warps; O relative to m, like l
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * t + e;
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
        if (g == 0) {
          sm.m[warp][r] = m[n][e];
          sm.l[warp][r] = l[n][e];
        }
        const float f = !FP8 ? 1.f : m[n][e] == -INFINITY ? 0.f : ex2_approx(mp[n][e] - kUp - m[n][e]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int dim = FP8 ? 16 * g + 4 * q : 64 * (q >> 1) + 8 * g + 4 * (q & 1);
          *reinterpret_cast<float4*>(&sm.o[warp][r][dim]) =
              make_float4(o[n][2 * q][e] * f, o[n][2 * q][2 + e] * f, o[n][2 * q + 1][e] * f, o[n][2 * q + 1][2 + e] * f);
        }
      }
    __syncthreads();
    {
      const int r = threadIdx.x >> 3, d0 = (threadIdx.x & 7) * 4;
      if (r < rows) {
        float m = -INFINITY, l = 0.f, f[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.m[w][r]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          f[w] = sm.m[w][r] == -INFINITY ? 0.f : ex2_approx(sm.m[w][r] - m);
          l = fmaf(sm.l[w][r], f[w], l);
        }
        const float inv = pc.whole ? (l != 0.f ? 1.f / l : 0.f) : 1.f;
        const long long prow = (2LL * blockIdx.x + (pc.blk0 == 0 ? 1 : 0)) * p.part_rows + r;
        __nv_bfloat16* out = p.out + (pc.row0 + r / p.g.G) * p.out_ld + (static_cast<long long>(pc.kvh) * p.g.G + r % p.g.G) * DH;
        if (!pc.whole && d0 == 0) p.part_ml[prow] = make_float2(m, l);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int d = d0 + 32 * q;
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(&sm.o[w][r][d]);
            a = make_float4(fmaf(v.x, f[w], a.x), fmaf(v.y, f[w], a.y), fmaf(v.z, f[w], a.z), fmaf(v.w, f[w], a.w));
          }
          if (pc.whole)
            *reinterpret_cast<uint2*>(out + d) = make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
          else
            *reinterpret_cast<float4*>(p.part + prow * DH + d) = a;
        }
      }
    }
    __syncthreads();
  }
  // not at the start: the join's CTAs would take places next to this kernel's and keep the next
  // call's from theirs (16 long histories, called in a row: 125 us against 78)
  pdl_trigger();
}

// Joins the parts of the tile that CTA i of the attention began and others finished: a warp a
// row, eight rows a CTA.  A row's parts are weighted by 2^(m - max).
__global__ void __launch_bounds__(256) paged_join_rows(const __grid_constant__ PagedAttnParams p) {
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.x;
  const CutRecord cut = p.cut[i];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.y * 8 + warp, tok = row / p.g.G, rg = row % p.g.G;
  if (tok < cut.toks) {
    // part c of the row lies at first[(2 c + (c == i)) * part_rows]: the first one is CTA i's own
    float m = -INFINITY;
    for (int c = i + lane; c <= cut.last; c += 32)
      m = fmaxf(m, p.part_ml[(2LL * c + (c == i)) * p.part_rows + row].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int c = i; c <= cut.last; ++c) {
      const long long at = (2LL * c + (c == i)) * p.part_rows + row;
      const float2 ml = p.part_ml[at];
      const float4 v = reinterpret_cast<const float4*>(p.part + at * DH)[lane];
      const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
      l = fmaf(ml.y, f, l);
      if (ml.y != 0.f) acc = make_float4(fmaf(v.x, f, acc.x), fmaf(v.y, f, acc.y), fmaf(v.z, f, acc.z), fmaf(v.w, f, acc.w));
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    __nv_bfloat16* o = p.out + static_cast<long long>(cut.row0 + tok) * p.out_ld + (cut.kvh * p.g.G + rg) * DH;
    reinterpret_cast<uint2*>(o)[lane] = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  }
}

// CTAs per SM that the registers allow, with one and with two tiles of queries.  One where it holds
// the rows: 16 long e4m3 histories 69 us, with two tiles 88.
constexpr int kPerSm[2] = {3, 2};
constexpr int kMaxSms = 148;   // the scratch is sized for the B200
int query_tiles(const PagedKv& kv, const RaggedBatch& rb, int n_q_heads) { return rb.max_rows * (n_q_heads / kv.hkv) <= 8 ? 1 : 2; }

}  // namespace

// Whether this kernel takes the call: the rows of one K/V head fit two products' 16 columns (4 rows
// in a window of 1024: 11.8 us, on the tensor-core kernel 16.0; 16 long e4m3 histories 69 and 205).
bool paged_decode_takes(const PagedKv& kv, const RaggedBatch& rb, int n_q_heads) {
  return static_cast<long long>(rb.max_rows) * (n_q_heads / kv.hkv) <= kRows;
}

size_t paged_decode_scratch(const PagedKv& kv, const RaggedBatch& rb, int n_q_heads) {
  const int nt = query_tiles(kv, rb, n_q_heads);
  return paged_scratch_layout(rb.batch, kPerSm[nt - 1] * kMaxSms, 8 * nt, DH).total;
}

cudaError_t launch_paged_decode(const PagedAttnDesc& a, cudaStream_t st) {
  PagedAttnParams p{};
  p.kv = a.kv;
  p.rb = a.rb;
  p.g.G = a.n_q_heads / a.kv.hkv;
  p.g.TQ = p.g.tile_tok = a.rb.max_rows;
  p.g.n_meta = a.n_meta;
  p.g.window = a.window;
  const int nt = query_tiles(a.kv, a.rb, a.n_q_heads);
  p.part_rows = 8 * nt;
  p.page_shift = page_shift(a.kv.page_size);
  const PagedScratch L = paged_scratch_layout(a.rb.batch, kPerSm[nt - 1] * kMaxSms, p.part_rows, DH);
  uint8_t* sc = static_cast<uint8_t*>(a.scratch);
  p.prefix = reinterpret_cast<long long*>(sc + L.prefix);
  p.part = reinterpret_cast<float*>(sc + L.part);
  p.part_ml = reinterpret_cast<float2*>(sc + L.ml);
  p.cut = reinterpret_cast<CutRecord*>(sc + L.cut);
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_ld = a.q_ld;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.out_ld = a.out_ld;
  p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(DH));
  p.status = a.status;
  const int ctas = kPerSm[nt - 1] * (num_sms() < kMaxSms ? num_sms() : kMaxSms);
  if (a.rb.batch > kPlanBatch)
    if (cudaError_t e = launch(paged_plan_kernel, dim3(1), dim3(1024), 0, st, a.kv, a.rb, p.g, p.prefix, a.status)) return e;
  const auto kernel = a.kv.type == CACHE_E4M3 ? (nt == 1 ? paged_decode_kernel<true, 1> : paged_decode_kernel<true, 2>)
                                              : (nt == 1 ? paged_decode_kernel<false, 1> : paged_decode_kernel<false, 2>);
  if (cudaError_t e = launch(kernel, dim3(ctas), dim3(32 * kWarps), 0, st, p)) return e;
  return launch(paged_join_rows, dim3(ctas - 1, nt), dim3(256), 0, st, p);
}

}  // namespace hy
