// w4.cu -- weights in 4 bits with group scales, w[n, k] = q[n, k] * scales[n, k / group]:
// quantised, read back, and multiplied with a few rows (a generation step's products).
#include "paged.cuh"

namespace hy {
namespace {

// Eight weights per lane and two (fp32) or four (bf16) such vectors in flight; the group / 8 lanes of a group share
// its maximum by shuffles.  HBM sets the floor: 2 or 4 bytes in and half a byte out per weight; 11264 x
// 2048 from bf16 and back 25.9 us (4.0 TB/s, 61 % of the measured copy rate).  What bounds it: quantising
// from bf16, two thirds of that time, issues in 78 % of the cycles (the nearest-even quotients); going back
// waits for its loads and for L1 (71 % busy).  In flight, there and back:
// bf16 2, 4, 8 vectors 26.4, 25.6, 28.3 us; fp32 (2048 x 2048) 2, 4: 11.9, 17.7.
template <typename T> constexpr int kQuantAhead = sizeof(T) == 4 ? 2 : 4;

template <typename T>
__global__ void __launch_bounds__(256) quantize_w4_kernel(const T* __restrict__ w, uint32_t* __restrict__ q4,
                                                          float* __restrict__ scales, long long n8, int lshift) {
  pdl_trigger();
  pdl_wait();
  constexpr int kAhead = kQuantAhead<T>;
  const long long i0 = static_cast<long long>(blockIdx.x) * (256 * kAhead) + threadIdx.x;
  Vec8<T> v[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (i0 + k * 256 < n8) v[k].load(w + (i0 + k * 256) * 8);
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const long long i = i0 + k * 256;
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (i < n8) v[k].to_f32(f);
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
    for (int o = 1 << (lshift - 1); o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (i >= n8) continue;
    const float most = fmaxf(m, 1.17549435e-38f), y = __frcp_rn(most);
    // the quotient 7 w / most, within an ulp and then corrected by its remainder (Markstein's
    // theorem: rounded to nearest, so a half that is exact stays one), and 1.5 * 2^23 added, which
    // rounds it to the nearest even integer in the sum's low bits.  bf16: 7 w is exact.  fp32: it
    // is not, and next to a half 64 bits decide, as where the remainder is subnormal or 7 w of the
    // largest weight would leave fp32's range (FLT_MAX / 7 = 4.86e37).
    uint32_t u = 0;
    bool near = !(most >= 1e-30f && most <= 4.8e37f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float w7 = 7.f * f[e], t0 = w7 * y, t = fmaf(fmaf(-t0, most, w7), y, t0), s = t + 12582912.f;
      if (sizeof(T) == 4) near |= !(fabsf(t - (s - 12582912.f)) <= 0.49999f);
      u |= ((__float_as_uint(s) + 8u) & 15u) << (4 * e);
    }
    if (near) {
      u = 0;
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        u = (u >> 4) | static_cast<uint32_t>(static_cast<int>(rint(7.0 * f[0] / static_cast<double>(most))) + 8) << 28;
#pragma unroll
        for (int x = 0; x < 7; ++x) f[x] = f[x + 1];
      }
    }
    q4[i] = u;
    if ((i & ((1 << lshift) - 1)) == 0) scales[i >> lshift] = fmaxf(__fdiv_rn(m, 7.f), 1.17549435e-38f);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) dequantize_w4_kernel(const uint32_t* __restrict__ q4,
                                                            const float* __restrict__ scales, T* __restrict__ w,
                                                            long long n8, int lshift) {
  pdl_trigger();
  pdl_wait();
  constexpr int kAhead = kQuantAhead<T>;
  const long long i0 = static_cast<long long>(blockIdx.x) * (256 * kAhead) + threadIdx.x;
  uint32_t u[kAhead];
  float s[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (i0 + k * 256 < n8) {
      u[k] = q4[i0 + k * 256];
      s[k] = scales[(i0 + k * 256) >> lshift];
    }
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const long long i = i0 + k * 256;
    if (i >= n8) continue;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)   // 2^23 + code, less 2^23 + 8
      f[e] = (__uint_as_float(0x4b000000u | ((u[k] >> (4 * e)) & 15u)) - 8388616.f) * s[k];
    Vec8<T> v;
    v.from_f32(f);
    v.store(w + i * 8);
  }
}

// C = A W^T for a few rows of A on mma.sync m16n8k16: W's rows are the products' 16 rows, A's
// rows their 8 columns (NT tiles of them), so 16 x 16 weights meet all rows of A in one
// instruction and the stream over W stays what bounds the kernel (CUDA-core sums would take
// longer than the stream from three rows on).  q in [-8, 7] is exact in bf16: a group's
// products are summed in fp32 by the tensor core and scaled once per group.  fp32 rows of A are
// split into three bf16 columns (8 + 8 + 8 of the 24 bits), which are summed at the end.
//
// A CTA of 16 warps owns a range of 16-row tiles and takes K in slabs whose columns of A fit
// shared memory, already in the order of the products.  The chunks of 256 k (16 rows x 128 bytes) of
// all its tiles are shared out evenly: each warp streams its own through a ring of its own by cp.async,
// and the parts of a tile meet in shared memory at the slab's end, in the warps' order.  Eight rows
// against 16384 x 8192: 25.4 us (3.0 TB/s, 46 % of the measured copy rate); four against 11264 x 5632:
// 14.6.  One change at a time: each tile shared by a fixed number of warps, a CTA in whole rounds, 26.3 and
// 18.9; chunks in even shares 26.9 and 15.4 (uneven rounds cost the four rows most, and the eight nothing);
// the next slab's first chunks under way while the parts meet 25.4 and 14.6.  The stream alone
// takes 14 us, taking the nibbles apart and the products alone 20, at four warps an SM quarter
// that issue in half of the cycles.  One row against 2048 x 5632: 5.7 us, a launch and two slabs (A is
// laid out for eight columns whatever the rows, so that 4096 k fill shared memory).  Sixteen rows against
// 16384 x 8192: 36 us; fp32 rows, three columns each: eight 75, sixteen 194 (six tiles of columns leave
// slabs of 512 k and a ring of two, whose parts meet every two chunks).
//
// The 32 k of 16 bytes of a row are one or part of one group; lane (g, t) takes 4 of them
// (8 k) of rows g and g + 8.  A word's nibbles i and i + 4 make one bf16 pair: (word >> 4 i)
// & 0x000f000f over the bits of 128.0 is 128 + code, and 136 less is q.
constexpr int kWarps = 16, kChunk = 256, kRowPitch = kChunk / 2 + 16, kTileRowsMax = 128;

struct GemmW4Params {
  const void* a;
  const uint8_t* q4;
  const float* scales;
  void* c;
  int M, N, K, tiles, slab;   // slab: k of one pass
};

template <int NT> struct W4Shape {
  static constexpr int ring = NT <= 2 ? 3 : 2;
  static constexpr int slab = NT == 1 ? 4096 : NT == 2 ? 2048 : NT == 3 ? 1024 : 512;
  static constexpr int x_bytes = slab / 32 * NT * 8 * 64;
  static constexpr int part = 16 * 8 * NT;                       // a tile's sums
  static constexpr int chunk_bytes = 16 * kRowPitch + 16 * 8 * 4;   // codes, then scales [row][8]
  static constexpr int stage = chunk_bytes > part * 4 ? chunk_bytes : part * 4;
  static constexpr int red_bytes = kWarps * part * 4;
  static constexpr int acc_bytes = kTileRowsMax * 8 * NT * 4;
  static constexpr int smem = x_bytes + kWarps * ring * stage + red_bytes + acc_bytes;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// q of nibbles i and i + 4 of a word, times 2^-10, as a bf16 pair (exact).  The power of two,
// taken out again at the end, lets a group's unscaled sum of the largest fp32 values stay finite.
constexpr float kQUp = 1024.f;
__device__ __forceinline__ uint32_t q_pair(uint32_t u, int i) {
  uint32_t v;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(v) : "r"(u >> (4 * i)));   // (u & mask) | 128.0: 128 + code
  const __nv_bfloat162 q = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v), __float2bfloat162_rn(1.f / kQUp),
                                   __float2bfloat162_rn(-136.f / kQUp));
  return *reinterpret_cast<const uint32_t*>(&q);
}

// GS: log2 of the group.
template <typename T, int NT, int GS>
__global__ void __launch_bounds__(32 * kWarps, 1) gemm_w4_kernel(const __grid_constant__ GemmW4Params p) {
  using W = W4Shape<NT>;
  constexpr int kSplit = sizeof(T) == 4 ? 3 : 1;   // columns of a row of A
  extern __shared__ __align__(16) uint8_t smem[];
  uint4* sx = reinterpret_cast<uint4*>(smem);                       // [k / 32][column][t]
  uint8_t* ring = smem + W::x_bytes;
  float* red = reinterpret_cast<float*>(ring + kWarps * W::ring * W::stage);   // [warp][row][column]
  float* acc = red + kWarps * 16 * 8 * NT;                                     // [row of the CTA][column]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int tile0 = static_cast<int>(static_cast<long long>(blockIdx.x) * p.tiles / gridDim.x),
            tile1 = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * p.tiles / gridDim.x);
  const int tiles = tile1 - tile0;                                    // at most eight
  constexpr int per_chunk = kChunk >> GS, kLog = 8 - GS;              // scales of a row and chunk
  const long long row_bytes = p.K / 2, row_scales = p.K >> GS;
  const uint32_t my_ring = smem_u32(ring + warp * W::ring * W::stage);
  pdl_trigger();
  pdl_wait();
  // A slab of K.  The CTA's chunks, tile by tile, go to the warps in equal shares; a share is no longer than
  // a tile (eight tiles and sixteen warps), so it is the end of one tile and the beginning of the next at most.
  int k0, chunks, all, share, begin, end, chunk;   // chunk: the next one to compute, in its tile
  int fi, ft, fc, fs;   // the next chunk to fetch: its number, its tile, its number in the tile, its slot
  auto fetch = [&]() {
    if (fi < end) {
      const int kc = fc * kChunk + k0, n0 = (tile0 + ft) * 16;
      const uint32_t dst = my_ring + fs * W::stage, dq = dst + (lane >> 3) * kRowPitch + (lane & 7) * 16;
      const int k = kc + (lane & 7) * 32;
      if (n0 + 16 <= p.N && kc + kChunk <= p.K) {   // eight lanes: the 128 bytes of a row
        const uint8_t* src = p.q4 + (n0 + (lane >> 3)) * row_bytes + (k >> 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async16(dq + i * 4 * kRowPitch, src + i * 4 * row_bytes, true);
#pragma unroll
        for (int i = lane; i < 16 * per_chunk; i += 32)
          cp_async4(dst + 16 * kRowPitch + ((i >> kLog) * 8 + (i & (per_chunk - 1))) * 4,
                    p.scales + (n0 + (i >> kLog)) * row_scales + (kc >> GS) + (i & (per_chunk - 1)), true);
      } else {   // rows behind the last read it again, k behind the last count as zeros
        const bool ok = k < p.K;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          cp_async16(dq + i * 4 * kRowPitch, p.q4 + min(n0 + i * 4 + (lane >> 3), p.N - 1) * row_bytes + (ok ? k >> 1 : 0), ok);
        for (int i = lane; i < 16 * per_chunk; i += 32) {
          const int row = i >> kLog, q = i & (per_chunk - 1), gi = (kc >> GS) + q;
          const bool have = gi < row_scales;
          cp_async4(dst + 16 * kRowPitch + (row * 8 + q) * 4, p.scales + min(n0 + row, p.N - 1) * row_scales + (have ? gi : 0),
                    have);
        }
      }
      ++fi;
      if (++fc == chunks) {
        fc = 0;
        ++ft;
      }
      fs = fs + 1 == W::ring ? 0 : fs + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto enter = [&](int k) {
    k0 = k;
    chunks = (min(p.slab, p.K - k0) + kChunk - 1) / kChunk;
    all = tiles * chunks;
    share = (all + kWarps - 1) / kWarps;
    begin = min(warp * share, all);
    end = min(begin + share, all);
    fi = begin;
    ft = begin / chunks;
    chunk = fc = begin - ft * chunks;
    fs = 0;
#pragma unroll
    for (int i = 0; i + 1 < W::ring; ++i) fetch();
  };
  enter(0);
  for (bool last = false; !last;) {
    const int ks = min(p.slab, p.K - k0);
    // the slab's columns of A, in the products' order: x0 x4 x1 x5 x2 x6 x3 x7 of each eight
    __syncthreads();   // (the previous slab's, and its parts, are no longer read)
    constexpr int kColWarps = NT * 8 >= kWarps ? 1 : 2;   // warps that share a column
    for (int col = warp / kColWarps; col < NT * 8; col += kWarps / kColWarps) {
      const int m = col / kSplit, part = col - m * kSplit;
      const T* a = static_cast<const T*>(p.a) + static_cast<long long>(m) * p.K + k0;
      for (int b8 = (warp % kColWarps) * 32 + lane; b8 < chunks * (kChunk / 8); b8 += 4 * 32 * kColWarps) {
        Vec8<T> v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = (b8 + j * 32 * kColWarps) * 8;
          if (m < p.M && k < ks) v[j].load(a + k);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int q8 = b8 + j * 32 * kColWarps;
          float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          if (q8 >= chunks * (kChunk / 8)) break;
          if (m < p.M && q8 * 8 < ks) v[j].to_f32(f);
          if (kSplit == 3) {   // the leading 8 bits, the next 8, the rest
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const bool finite = fabsf(f[e]) < INFINITY;   // (an infinity or NaN is its leading part)
              const float hi = finite ? __uint_as_float(__float_as_uint(f[e]) & 0xffff0000u) : f[e], r = finite ? f[e] - hi : 0.f;
              const float mid = __uint_as_float(__float_as_uint(r) & 0xffff0000u);
              f[e] = part == 0 ? hi : part == 1 ? mid : r - mid;
            }
          }
          sx[((q8 >> 2) * NT * 8 + col) * 4 + (q8 & 3)] =
              make_uint4(pack_bf16(f[0], f[4]), pack_bf16(f[1], f[5]), pack_bf16(f[2], f[6]), pack_bf16(f[3], f[7]));
        }
      }
    }
    __syncthreads();
    constexpr int kPart = W::part;
    int slot = 0;
    float sum[NT][4], part[NT][4];
    auto clear = [&] {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[n][e] = 0.f;
    };
    auto put = [&](float* dst) {   // [row][column]
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(&dst[(g + 8 * h) * 8 * NT + n * 8 + 2 * t]) = make_float2(sum[n][2 * h], sum[n][2 * h + 1]);
    };
    clear();
    for (int i = begin; i < end; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(W::ring - 2) : "memory");
      __syncwarp();   // every lane's pieces of this chunk are there, and the next slot is free
      fetch();
      const uint32_t st = my_ring + slot * W::stage, codes = st + g * kRowPitch + t * 4;
      const uint32_t sc = st + 16 * kRowPitch + g * 32;
      slot = slot + 1 == W::ring ? 0 : slot + 1;
      const uint32_t xk = smem_u32(sx) + ((chunk * (kChunk / 32) * NT * 8 + g) * 4 + t) * 16;
#pragma unroll
      for (int q = 0; q < kChunk / 32; ++q) {
        const uint32_t u0 = lds_u32(codes + q * 16), u1 = lds_u32(codes + 8 * kRowPitch + q * 16);
        const uint32_t a0[4] = {q_pair(u0, 0), q_pair(u1, 0), q_pair(u0, 1), q_pair(u1, 1)};
        const uint32_t a1[4] = {q_pair(u0, 2), q_pair(u1, 2), q_pair(u0, 3), q_pair(u1, 3)};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float4 x = lds_f4(xk + (q * NT + n) * 512);
          if ((q * 32) % (1 << GS) == 0) {   // a group begins
#pragma unroll
            for (int e = 0; e < 4; ++e) part[n][e] = 0.f;
          }
          mma_bf16(part[n], a0, __float_as_uint(x.x), __float_as_uint(x.y));
          mma_bf16(part[n], a1, __float_as_uint(x.z), __float_as_uint(x.w));
        }
        if ((q * 32 + 32) % (1 << GS) == 0) {   // the group is complete
          const float s0 = lds_f32(sc + (q * 32 >> GS) * 4), s1 = lds_f32(sc + 8 * 32 + (q * 32 >> GS) * 4);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[n][e] = fmaf(part[n][e], e < 2 ? s0 : s1, sum[n][e]);
        }
      }
      if (++chunk == chunks && i + 1 < end) {   // on to the next tile
        put(red + warp * kPart);
        clear();
        chunk = 0;
      }
    }
    // the tiles' sums, over their warps in order; a warp's last part lies in the last stage of its ring, whose
    // chunks have been read; the next slab's begin to fill the other stages meanwhile
    auto last_part = [&](int w) { return reinterpret_cast<float*>(ring + ((w + 1) * W::ring - 1) * W::stage); };
    __syncwarp();
    if (end > begin) put(last_part(warp));
    const int n_chunks = chunks, n_all = all, n_share = share;
    const bool first = k0 == 0;
    last = k0 + p.slab >= p.K;
    if (!last) enter(k0 + p.slab);
    __syncthreads();
    for (int i = threadIdx.x; i < tiles * kPart; i += 32 * kWarps) {
      const int tl = i / kPart, e = i - tl * kPart, c0 = tl * n_chunks, c1 = c0 + n_chunks;
      const int w1 = (c1 - 1) / n_share;   // the only one that may go on to the next tile
      float v = first ? 0.f : acc[i];
#pragma unroll 4
      for (int w = c0 / n_share; w < w1; ++w) v += last_part(w)[e];
      v += min((w1 + 1) * n_share, n_all) <= c1 ? last_part(w1)[e] : red[w1 * kPart + e];
      if (!last || kSplit > 1) acc[i] = v;
      const int n = (tile0 + tl) * 16 + e / (8 * NT), m = e % (8 * NT);
      if (last && kSplit == 1 && n < p.N && m < p.M)
        static_cast<T*>(p.c)[static_cast<long long>(m) * p.N + n] = from_f<T>(v * kQUp);
    }
    if (last && kSplit > 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < tiles * 16 * p.M; i += 32 * kWarps) {
        const int r = i / p.M, m = i - r * p.M, n = tile0 * 16 + r;
        const float* v = &acc[r * 8 * NT + m * kSplit];
        if (n < p.N) static_cast<T*>(p.c)[static_cast<long long>(m) * p.N + n] = from_f<T>(((v[2] + v[1]) + v[0]) * kQUp);
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename T, int NT>
cudaError_t launch_gemm_w4_t(GemmW4Params p, int group, cudaStream_t st) {
  using W = W4Shape<NT>;
  static_assert(W::smem <= 227 * 1024, "shared memory of one CTA");
  static std::atomic<uint64_t> done[3];
  const int gs = group == 32 ? 0 : group == 64 ? 1 : 2;
  const auto kernel = gs == 0 ? gemm_w4_kernel<T, NT, 5> : gs == 1 ? gemm_w4_kernel<T, NT, 6> : gemm_w4_kernel<T, NT, 7>;
  if (cudaError_t e = smem_attr_once(kernel, W::smem, done[gs])) return e;
  p.slab = W::slab;
  p.tiles = (p.N + 15) / 16;
  // a CTA per SM, or more where eight tiles each are all that their sums have room for
  const int sms = num_sms(), least = (p.tiles + kTileRowsMax / 16 - 1) / (kTileRowsMax / 16);
  const int grid = least > sms ? least : p.tiles < sms ? p.tiles : sms;
  return launch(kernel, dim3(grid), dim3(32 * kWarps), W::smem, st, p);
}

unsigned blocks_for(long long items, int per) { return static_cast<unsigned>((items + per - 1) / per); }

}  // namespace

cudaError_t launch_quantize_w4(const void* w, void* q4, float* scales, int N, int K, int group, bool bf16,
                               cudaStream_t st) {
  const long long n8 = static_cast<long long>(N) * K / 8;
  const dim3 grid(blocks_for(n8, 256 * (bf16 ? kQuantAhead<__nv_bfloat16> : kQuantAhead<float>)));
  const int ls = group == 32 ? 2 : group == 64 ? 3 : 4;   // log2 of a group's lanes
  return bf16 ? launch(quantize_w4_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, static_cast<const __nv_bfloat16*>(w),
                       static_cast<uint32_t*>(q4), scales, n8, ls)
              : launch(quantize_w4_kernel<float>, grid, dim3(256), 0, st, static_cast<const float*>(w),
                       static_cast<uint32_t*>(q4), scales, n8, ls);
}

cudaError_t launch_dequantize_w4(const void* q4, const float* scales, void* w, int N, int K, int group, bool bf16,
                                 cudaStream_t st) {
  const long long n8 = static_cast<long long>(N) * K / 8;
  const dim3 grid(blocks_for(n8, 256 * (bf16 ? kQuantAhead<__nv_bfloat16> : kQuantAhead<float>)));
  const int ls = group == 32 ? 2 : group == 64 ? 3 : 4;
  return bf16 ? launch(dequantize_w4_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, static_cast<const uint32_t*>(q4),
                       scales, static_cast<__nv_bfloat16*>(w), n8, ls)
              : launch(dequantize_w4_kernel<float>, grid, dim3(256), 0, st, static_cast<const uint32_t*>(q4), scales,
                       static_cast<float*>(w), n8, ls);
}

cudaError_t launch_gemm_w4(const void* a, const void* q4, const float* scales, void* c, int M, int N, int K, int group,
                           bool bf16, cudaStream_t st) {
  GemmW4Params p{a, static_cast<const uint8_t*>(q4), scales, c, M, N, K, 0, 0};
  // the fewest tiles of eight columns that hold the rows (against 16384 x 8192 in L2: 8 bf16 rows in one tile
  // 23 us, in two 35; 5 fp32 rows in two 45, in three 73; 8 fp32 rows in three 74, in six 175)
  if (bf16) return M <= 8 ? launch_gemm_w4_t<__nv_bfloat16, 1>(p, group, st) : launch_gemm_w4_t<__nv_bfloat16, 2>(p, group, st);
  // three columns a row
  if (M <= 2) return launch_gemm_w4_t<float, 1>(p, group, st);
  if (M <= 5) return launch_gemm_w4_t<float, 2>(p, group, st);
  if (M <= 8) return launch_gemm_w4_t<float, 3>(p, group, st);
  return launch_gemm_w4_t<float, 6>(p, group, st);
}

}  // namespace hy
