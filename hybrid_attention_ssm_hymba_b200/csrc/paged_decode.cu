// paged_decode.cu -- attention of a few new rows per sequence (a generation step: at most 16
// rows per K/V head, counting its query heads) over the paged K/V cache (blog.outta.ai Hymba
// review, "Efficiency and KV cache optimization").
//
//   out = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),  s_j = log2(e) q.k_j / sqrt(dh)
//
// Every K/V row is read once for all query heads that share it, and that reading bounds the
// call.  The rows are the 16 rows of mma.sync m16n8k16 products (a 128-row tensor-core tile
// would be mostly empty, and its K and V would have to pass through shared memory); K and V go
// from global memory straight to the registers that the products read: the order of the
// summed index (dims for Q K^T, keys for P V) and of the output columns is free, so each lane
// loads 16 consecutive bytes of a row and the products are told apart by that order alone.
//   Q K^T  lane (g, t) holds, of key g of eight, the dims of its 16-byte pieces (the four
//          lanes of a key read 64 consecutive bytes); Q is read in the same order.
//   P V    lane (g, t) holds keys 2t, 2t+1, 2t+8, 2t+9 of sixteen (as Q K^T left their P) at
//          the dims of piece g (eight lanes read 128 consecutive bytes); the two keys of a
//          register are put together by one byte permutation.
// A CTA of four warps takes 32 keys of each 128-key block per warp and walks its part of the
// line of blocks (paged_plan.cuh); K of the next step is loaded before the softmax of this one.
#include "paged_plan.cuh"

namespace hy {
namespace {

constexpr int DH = 128, kWarps = 4, kRows = 16;
constexpr int kPlanBatch = 1024;   // batches up to this are planned by every CTA itself

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
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

// One key of a step, held by the lane of its number: its row of the pool (-1: not to be read)
// and its scales.
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
  if (report)   // the join reads it
    for (int b = threadIdx.x; b <= p.rb.batch; b += 32 * kWarps) p.prefix[b] = sm.prefix[b];
}

template <bool FP8>
__global__ void __launch_bounds__(32 * kWarps, 2) paged_decode_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int kStep = FP8 ? 32 : 16;       // keys of a warp's step: 4 KB of K and of V either way
  constexpr int kSub = 32 / kStep;           // steps per block and warp
  constexpr int kNt = kStep / 8, kKt = kStep / 16;
  constexpr int es = FP8 ? 1 : 2;
  __shared__ Shared sm;
  pdl_trigger();
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

  PieceWalk walk;
  Piece pc;
  walk.init(p, prefix);
  while (walk.next(p, &pc)) {
    const int rows = pc.ts.toks * p.g.G;
    // Q of rows g and g + 8 in the dims' order
    uint32_t qa[8][4];
    {
      const __nv_bfloat16* q0 = p.q + pc.row0 * p.q_ld + static_cast<long long>(pc.kvh) * p.g.G * DH;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = g + 8 * half;
        const uint4* q = reinterpret_cast<const uint4*>(q0 + (r / p.g.G) * p.q_ld + (r % p.g.G) * DH);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // bf16: piece t of 32 dims j; e4m3: dims 64 (j / 2) + 16 t + 8 (j % 2)
          const int at = FP8 ? (j >> 1) * 8 + t * 2 + (j & 1) : j * 4 + t;
          const uint4 v = r < rows ? q[at] : make_uint4(0, 0, 0, 0);
          qa[2 * j][half] = v.x;
          qa[2 * j][2 + half] = v.y;
          qa[2 * j + 1][half] = v.z;
          qa[2 * j + 1][2 + half] = v.w;
        }
      }
    }
    const int i0 = pc.ts.p0 + g / p.g.G, i1 = pc.ts.p0 + (g + 8) / p.g.G;   // places of the two rows
    const int lo = p.g.window < 0 ? 0 : pc.ts.p0 - p.g.window;             // first key of any row's window
    const uint8_t* kh = kbase + pc.kvh * (DH * es);
    const uint8_t* vh = vbase + pc.kvh * (DH * es);

    const int steps = (pc.blk1 - pc.blk0) * kSub;
    auto key0 = [&](int s) { return pc.ts.block(pc.blk0 + s / kSub) * kKeyBlock + warp * 32 + (s % kSub) * kStep; };
    auto lookup = [&](int s) -> Key {
      Key k{-1, 0.f, 0.f};
      if (s < steps && lane < kStep) {
        const int j = key0(s) + lane;
        if (j <= pc.ts.p1 && (j >= lo || j < p.g.n_meta)) {
          const int page = page_of(p.kv, pc.b, j);
          if (page < 0) {
            report_invalid(p.status);
          } else {
            const int at = j % p.kv.page_size;
            k.row = page * p.kv.page_size + at;
            if (FP8) {
              k.sk = p.kv.scales[page_scale(p.kv, 0, page, at, pc.kvh)];
              k.sv = p.kv.scales[page_scale(p.kv, 1, page, at, pc.kvh)];
            }
          }
        }
      }
      return k;
    };
    // rows that are not read count as zeros
    constexpr int kLoadsK = FP8 ? 2 : 4;   // 16-byte pieces of a key per lane
    uint4 kr[kNt][kLoadsK];
    auto load_k = [&](const Key& k) {
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) {
        const int row = __shfl_sync(0xffffffffu, k.row, nt * 8 + g);
        const uint8_t* a = kh + row * row_bytes + t * 16;
#pragma unroll
        for (int j = 0; j < kLoadsK; ++j) kr[nt][j] = row >= 0 ? ldg_once(a + j * 64) : make_uint4(0, 0, 0, 0);
      }
    };

    float o[16][4], m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    Key cur = lookup(0), nxt = lookup(1);
    load_k(cur);
    for (int s = 0; s < steps; ++s) {
      // V of this step
      uint4 vr[kKt][4][FP8 ? 1 : 2];
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int row = __shfl_sync(0xffffffffu, cur.row, kt * 16 + 2 * t + (c & 1) + (c >> 1) * 8);
          const uint8_t* a = vh + row * row_bytes + g * 16;
#pragma unroll
          for (int h = 0; h < (FP8 ? 1 : 2); ++h) vr[kt][c][h] = row >= 0 ? ldg_once(a + h * 128) : make_uint4(0, 0, 0, 0);
        }
      const Key aft = lookup(s + 2);
      // S = Q K^T
      float sc[kNt][4];
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
#pragma unroll
        for (int j = 0; j < kLoadsK; ++j) {
          if constexpr (FP8) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint2 b = bf16_of_e4m3(word(kr[nt][j], w));
              mma_bf16(sc[nt], qa[4 * j + w], b.x, b.y);
            }
          } else {
            mma_bf16(sc[nt], qa[2 * j], kr[nt][j].x, kr[nt][j].y);
            mma_bf16(sc[nt], qa[2 * j + 1], kr[nt][j].z, kr[nt][j].w);
          }
        }
      }
      if (s + 1 < steps) load_k(nxt);
      // scores in log2 units, hidden keys -inf
      const int k0 = key0(s);
      const unsigned there = __ballot_sync(0xffffffffu, cur.row >= 0);
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = nt * 8 + 2 * t + e, j = k0 + c;
          float f = p.scale_log2;
          if (FP8) f *= __shfl_sync(0xffffffffu, cur.sk, c);
          const bool in = (there >> c) & 1u;
          sc[nt][e] = in && key_visible(p.g, i0, j) ? sc[nt][e] * f : -INFINITY;
          sc[nt][2 + e] = in && key_visible(p.g, i1, j) ? sc[nt][2 + e] * f : -INFINITY;
          mx0 = fmaxf(mx0, sc[nt][e]);
          mx1 = fmaxf(mx1, sc[nt][2 + e]);
        }
      }
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
      }
      if (__any_sync(0xffffffffu, mx0 > m0 || mx1 > m1)) {
        const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
        const float a0 = n0 == -INFINITY ? 1.f : ex2_approx(m0 - n0), a1 = n1 == -INFINITY ? 1.f : ex2_approx(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          o[i][0] *= a0;
          o[i][1] *= a0;
          o[i][2] *= a1;
          o[i][3] *= a1;
        }
      }
      const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
      uint32_t pa[kKt][4];   // P, rounded to bf16 once, with V's scales in it
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float (&x)[4] = sc[2 * kt + h];
          x[0] = ex2_approx(x[0] - r0);
          x[1] = ex2_approx(x[1] - r0);
          x[2] = ex2_approx(x[2] - r1);
          x[3] = ex2_approx(x[3] - r1);
          l0 += x[0] + x[1];
          l1 += x[2] + x[3];
          if (FP8) {   // (a key that is not there has scale 0)
            const int c = (2 * kt + h) * 8 + 2 * t;
            const float s0 = __shfl_sync(0xffffffffu, cur.sv, c), s1 = __shfl_sync(0xffffffffu, cur.sv, c + 1);
            x[0] *= s0;
            x[1] *= s1;
            x[2] *= s0;
            x[3] *= s1;
          }
          pa[kt][2 * h] = pack_bf16(x[0], x[1]);
          pa[kt][2 * h + 1] = pack_bf16(x[2], x[3]);
        }
      // O += P V
#pragma unroll
      for (int kt = 0; kt < kKt; ++kt) {
        if constexpr (FP8) {
#pragma unroll
          for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const uint32_t sel = (b | (b << 4)) | ((4 + b) << 8) | ((4 + b) << 12);
              mma_bf16(o[4 * w + b], pa[kt], bf16_of_e4m3_high(__byte_perm(word(vr[kt][0][0], w), word(vr[kt][1][0], w), sel)),
                       bf16_of_e4m3_high(__byte_perm(word(vr[kt][2][0], w), word(vr[kt][3][0], w), sel)));
            }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t sel = e & 1 ? 0x7632 : 0x5410;
              mma_bf16(o[8 * h + e], pa[kt], __byte_perm(word(vr[kt][0][h], e >> 1), word(vr[kt][1][h], e >> 1), sel),
                       __byte_perm(word(vr[kt][2][h], e >> 1), word(vr[kt][3][h], e >> 1), sel));
            }
        }
      }
      cur = nxt;
      nxt = aft;
    }
    // the four lanes of a row, then the four warps
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if (t == 0) {
      sm.m[warp][g] = m0;
      sm.m[warp][g + 8] = m1;
      sm.l[warp][g] = l0;
      sm.l[warp][g + 8] = l1;
    }
    // output column n = 2t + e of product i is dim 16 n + i (e4m3) or 64 (i / 8) + 8 n + i % 8 (bf16)
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = 2 * t + e, dim = FP8 ? 16 * n + 4 * q : 64 * (q >> 1) + 8 * n + 4 * (q & 1);
          *reinterpret_cast<float4*>(&sm.o[warp][g + 8 * half][dim]) =
              make_float4(o[4 * q][2 * half + e], o[4 * q + 1][2 * half + e], o[4 * q + 2][2 * half + e],
                          o[4 * q + 3][2 * half + e]);
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
}

// Two CTAs per SM (their registers allow no third).
constexpr int kDecodeCtas = 2 * 148;

}  // namespace

// Whether this kernel takes the call: the rows of one K/V head fit one product's 16.
bool paged_decode_takes(const PagedKv& kv, const RaggedBatch& rb, int n_q_heads) {
  return static_cast<long long>(rb.max_rows) * (n_q_heads / kv.hkv) <= kRows;
}

size_t paged_decode_scratch(const RaggedBatch& rb) {
  return paged_scratch_layout(rb.batch, kDecodeCtas, kRows, DH).total;
}

cudaError_t launch_paged_decode(const PagedAttnDesc& a, cudaStream_t st) {
  PagedAttnParams p{};
  p.kv = a.kv;
  p.rb = a.rb;
  p.g.G = a.n_q_heads / a.kv.hkv;
  p.g.TQ = p.g.tile_tok = a.rb.max_rows;
  p.g.n_meta = a.n_meta;
  p.g.window = a.window;
  p.part_rows = kRows;
  p.min_blocks = 1;
  const PagedScratch L = paged_scratch_layout(a.rb.batch, kDecodeCtas, kRows, DH);
  uint8_t* sc = static_cast<uint8_t*>(a.scratch);
  p.prefix = reinterpret_cast<long long*>(sc + L.prefix);
  p.part = reinterpret_cast<float*>(sc + L.part);
  p.part_ml = reinterpret_cast<float2*>(sc + L.ml);
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_ld = a.q_ld;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.out_ld = a.out_ld;
  p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(DH));
  p.status = a.status;
  const int ctas = 2 * num_sms() < kDecodeCtas ? 2 * num_sms() : kDecodeCtas;
  if (a.rb.batch > kPlanBatch)
    if (cudaError_t e = launch(paged_plan_kernel, dim3(1), dim3(1024), 0, st, a.kv, a.rb, p.g, p.prefix, a.status)) return e;
  if (cudaError_t e = a.kv.type == CACHE_E4M3 ? launch(paged_decode_kernel<true>, dim3(ctas), dim3(32 * kWarps), 0, st, p)
                                              : launch(paged_decode_kernel<false>, dim3(ctas), dim3(32 * kWarps), 0, st, p))
    return e;
  return launch_paged_join(p, ctas, st);
}

}  // namespace hy
