// paged_attn_tc.cu -- attention of new rows over the paged K/V cache on the sm_100a tensor
// cores (the layer's attention heads, blog.outta.ai Hymba review, "Design formulation" and
// "Combine global and local attention"; meta rows always visible).
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = 2^(s_ij - m_i),   s_ij = log2(e) q_i.k_j / sqrt(dh)
//
// in one pass over the keys with a running m_i.  The G query heads that share a K/V head are
// packed into the rows of a tile, so every K/V row is read once for all of them; two row
// groups of up to 128 rows (TQ tokens x G heads) share each 128-key block.  The work is one
// line of key blocks, cut evenly over a persistent CTA per SM (paged_plan.cuh); parts of a cut
// tile leave their unnormalised output, m and sum in scratch, and paged_join_tc joins them.
//
//   warp 0      producer: Q of both groups by TMA; K and V block by block, one TMA per page
//               piece and 64-column half, through the page table (two 2-deep rings)
//   warp 1      UMMA issuer, per block: P_a V, S_a of the next block, P_b V, S_b of the next
//   warps 2..9  softmax of group a, warps 10..17 of group b (e4m3 cache: two later): two threads
//               per row, each over 64 of the block's keys and 64 of O's columns
//   warps 2, 3  (e4m3 cache only) turn the 8-bit K and V of a block into the fp16 tiles the
//               tensor core reads.  An e4m3 code is exact in fp16.  V: its scale and the code
//               times it are each rounded to fp16's 11 bits (2^-11 in all, where the output's own
//               rounding is 2^-8).  K: a score of hundreds would lose too much that way, so K is
//               the code alone and the softmax threads multiply S's columns by its scale in fp32:
//               rows of any magnitude stand side by side.  Powers of two keep fp16's range: V's
//               scales are held below 2^7 with the largest that the tile has met, a row of Q is
//               scaled to at most 2^8, and P to at most 2^15.  V's scales keep their 11 bits down
//               to 2^-21 of the largest.  From the first block with scales further apart
//               (kSpread) on, V is the code times its scale's mantissa, and the scale's power of
//               two goes into P, relative to the largest of the row's own keys: a large V row
//               costs no bits of the rows that do not see it.
// TMEM (512 columns): S_a | S_b | O_a | O_b; P in 16 bits over the consumed S columns.
//
// Bound by the round of a group: S (tensor core), softmax, P V, one after another, with the other
// group's round half a turn behind.  4096 rows of 16 heads over 32K bf16 rows: 970 us, 1066 TFLOP/s,
// 64 % of the measured bf16 rate; of a round's 4100 cycles the softmax takes 1900 and the tensor core
// 2050 for both groups.  e4m3 rows: 1290 us; reading K's scales and converting share the shared
// memory with the products.  Nine ragged sequences of up to 1604 e4m3 rows in a window of 1024 (16
// blocks a CTA): 94 us, of which 16 blocks take about 51; starting up, and per tile Q's conversion,
// the first S and the output take the rest.  A third group per CTA has no TMEM left, and one group with
// twice the keys would read every K/V row twice as often.
//
// Rows of V that no query of the tile sees (behind the sequence, between the meta rows and
// the window) may hold NaN, and 0 x NaN would reach every output: page pieces of such rows
// are loaded from beyond the tensor map (zeros), and in a partly visible piece the softmax
// threads zero them before P V.
#include "paged_plan.cuh"

namespace hy {
namespace {

constexpr int DH = 128, TILE_BYTES = 128 * DH * 2, HALF = 128 * 64 * 2;
// kind::f16 with bf16 or (FP8) fp16 operands
constexpr uint32_t kFmtBits = (1u << 7) | (1u << 10);
template <bool FP8> constexpr uint32_t IDESC_QK = idesc_bf16(128, 128, false, false) & ~(FP8 ? kFmtBits : 0u);
template <bool FP8> constexpr uint32_t IDESC_PV = idesc_bf16(128, DH, false, true) & ~(FP8 ? kFmtBits : 0u);
constexpr int kUp = 7;         // FP8: V's scales are held below 2^kUp, code times scale below 2^16
constexpr float kPUp = 11.f;   // FP8: P is 2^(s - m + kPUp)
// FP8: V's scales of a tile stand in V as they are while their exponents differ by at most this.  Beyond,
// a block takes a second exponential: scales of 2^+-15 in random order, 4096 rows over 32K keys 2110 us
// against 1290, ragged chunks 132 against 96.  (Always so, the usual scales would pay it too.)
constexpr int kSpread = 20;
constexpr int kApart = 1 << 20;   // BlockInfo::ev of such a block
// FP8: a row of Q is scaled up by at most 2^kMostUp, so that the factor from S to log2 units stays
// a normal number (0 times a hidden score's -inf would be no number).
constexpr int kMostUp = 120;

// What the producer tells the softmax threads of each tile (they give the slot back) and of
// each key block (it is at most four blocks ahead of them: a ring of 8 needs no giving back).
constexpr int kTileSlots = 4, kBlockSlots = 8;
struct TileInfo {
  int p0, p1, toks;   // places of the first and last token; their number (0: no more tiles)
  int n;              // key blocks to do
  int row0, kvh;
  int part;           // -1: the whole tile is done here; else 1 its first part, 0 a later one
  int groups;
};
struct BlockInfo {
  int k0;
  uint32_t flags;     // bit x: group x masks; bit 2: some rows of V are to be zeroed
  int ev;             // FP8: V's scales are held times 2^(kUp - ev); kApart: without their powers of two
  uint32_t valid[4];  // rows whose page number is valid, one bit each
};
constexpr uint32_t kZeroV = 4u;

// Batches up to this are planned by every CTA itself (4 sequences of 40 rows in a window of 1024: 24 us,
// with the plan kernel 32; 64 of 17 rows 61 and 70); the 8-bit path's tiles leave no room for many more.
constexpr int kPlanBatch = 64;
template <bool FP8> struct Smem;
template <> struct Smem<true>;   // with the scales and barriers of the 8-bit path, below
template <> struct Smem<false> {   // behind the six tiles
  uint64_t q_full, q_empty, k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], o_done[2];   // per group; o_done completes once per P V
  uint64_t tile_full[kTileSlots], tile_empty[kTileSlots], mma_done;
  uint32_t tmem_slot;
  int abort_flag;
  alignas(16) TileInfo tile[kTileSlots];
  alignas(16) BlockInfo block[kBlockSlots];
  float smax[2][2][2][128];   // [block parity][group][half][row]
  long long prefix[kPlanBatch + 1];
};
// 8-bit path: raw K and V come in half tiles of 64 rows through a ring of three, their scales
// through a ring of four blocks (the producer is at most three blocks ahead of the softmax).
constexpr int kRawStages = 3, kRawBytes = 64 * DH, kScaleSlots = 4;
template <> struct Smem<true> : Smem<false> {
  uint64_t raw_full[kRawStages], raw_empty[kRawStages], scale_full[kScaleSlots], scale_ready[kScaleSlots], q_ready[2];
  // As copied: K's and V's scales [slot][K, V][row].  As used: K's scale, and for V a word with the factor
  // of its codes in fp16 (low half) and (kApart) the scale's exponent in bf16 (high half).
  alignas(16) float scale[kScaleSlots][2][128];
};
template <bool FP8> constexpr int smem_bytes() {
  return 6 * TILE_BYTES + 1024 + (FP8 ? kRawStages * kRawBytes : 0) + static_cast<int>(sizeof(Smem<FP8>));
}
static_assert(smem_bytes<true>() <= 227 * 1024, "shared memory of one CTA");

// The n low bits of a word (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Maximum of 64 values in eight independent chains of three-input maxima.
__device__ __forceinline__ float row_max64(const uint32_t (&sv)[64]) {
  float m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = fmaxf(__uint_as_float(sv[i]), __uint_as_float(sv[i + 8]));
#pragma unroll
  for (int e = 16; e < 64; e += 16)
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = max3f(m[i], __uint_as_float(sv[e + i]), __uint_as_float(sv[e + 8 + i]));
  return max3f(max3f(m[0], m[1], m[2]), max3f(m[3], m[4], m[5]), fmaxf(m[6], m[7]));
}
// 64 values times a shared vector, the same for every row; eight loads ahead (one: 1385 us against
// 1328 for 4096 rows over 32K e4m3 keys), since shared memory is busy with the tensor core's operands.
__device__ __forceinline__ void scale64(uint32_t (&sv)[64], uint32_t vec) {
  float4 ring[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) ring[q] = lds_f4(vec + 16 * q);
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const float4 k = ring[q % 8];
    if (q + 8 < 16) ring[q % 8] = lds_f4(vec + 16 * (q + 8));
    const float2 a = __fmul2_rn(make_float2(__uint_as_float(sv[4 * q]), __uint_as_float(sv[4 * q + 1])), make_float2(k.x, k.y));
    const float2 b = __fmul2_rn(make_float2(__uint_as_float(sv[4 * q + 2]), __uint_as_float(sv[4 * q + 3])), make_float2(k.z, k.w));
    sv[4 * q] = __float_as_uint(a.x);
    sv[4 * q + 1] = __float_as_uint(a.y);
    sv[4 * q + 2] = __float_as_uint(b.x);
    sv[4 * q + 3] = __float_as_uint(b.y);
  }
}
// FP8, a kApart block: the exponent of V's scale from its word.
__device__ __forceinline__ float v_exponent(float word) { return __uint_as_float(__float_as_uint(word) & 0xffff0000u); }
// The largest of s sc + e, e the exponent of V's scale: what the terms of P V reach.
__device__ __forceinline__ float row_reach64(const uint32_t (&sv)[64], uint32_t vec, float sc) {
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const float4 w = lds_f4(vec + 16 * q);
    m = max3f(m, fmaf(__uint_as_float(sv[4 * q]), sc, v_exponent(w.x)), fmaf(__uint_as_float(sv[4 * q + 1]), sc, v_exponent(w.y)));
    m = max3f(m, fmaf(__uint_as_float(sv[4 * q + 2]), sc, v_exponent(w.z)), fmaf(__uint_as_float(sv[4 * q + 3]), sc, v_exponent(w.w)));
  }
  return m;
}
// P = 2^(s sc - m + e + up) in place as pairs of fp16; returns the sum of the 2^(s sc - m + kPUp).
__device__ __forceinline__ float row_exp64_apart(uint32_t (&sv)[64], uint32_t vec, float sc, float m, float up) {
  float sum = 0.f;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const float4 w = lds_f4(vec + 16 * q);
    const float e[4] = {v_exponent(w.x), v_exponent(w.y), v_exponent(w.z), v_exponent(w.w)};
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = fmaf(__uint_as_float(sv[4 * q + i]), sc, -m);
      sum += ex2_approx(x + kPUp);
      y[i] = ex2_approx(x + (e[i] + up));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2 r = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
      sv[2 * q + i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
  return sum;
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((min(max(e, -126), 127) + 127) << 23); }
// P = 2^(S scale - m_ref), packed in place as pairs of bf16 or fp16 (sv[q] <- p[2q], p[2q + 1]);
// returns the sum of the fp32 values.  P is rounded once, as the P V operand.
template <bool F16>
__device__ __forceinline__ float row_exp64(uint32_t (&sv)[64], float scale_log2, float m_ref) {
  const float2 sc = make_float2(scale_log2, scale_log2), nm = make_float2(-m_ref, -m_ref);
  float2 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll
  for (int q = 0; q < 32; ++q) {
    const float2 x = __ffma2_rn(make_float2(__uint_as_float(sv[2 * q]), __uint_as_float(sv[2 * q + 1])), sc, nm);
    const float2 pq = make_float2(ex2_approx(x.x), ex2_approx(x.y));
    acc[q & 3] = __fadd2_rn(acc[q & 3], pq);
    if (F16) {
      const __half2 r = __floats2half2_rn(pq.x, pq.y);
      sv[q] = *reinterpret_cast<const uint32_t*>(&r);
    } else {
      sv[q] = pack_bf16(pq.x, pq.y);
    }
  }
  const float2 t = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
  return t.x + t.y;
}

constexpr int kThreads = 576, kThreadsFp8 = 640;
// 8-bit path: registers of a thread at launch, of the softmax warpgroups and of the warpgroup of the
// other four warps.  (Ragged e4m3 chunks: 98 us, without the shift 105; the bf16 path, two idle
// warps added for it: 1010 us for 4096 rows over 32K, without 970.)
constexpr int kRegs = 96, kRegsSoft = 104, kRegsFew = 64;
static_assert(512 * kRegsSoft + 128 * kRegsFew <= kThreadsFp8 * kRegs, "more registers than the launch has");
template <int N> __device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

template <bool FP8>
__global__ void __launch_bounds__(FP8 ? kThreadsFp8 : kThreads, 1)
    paged_attn_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* sQ = smem_raw + pad;       // 2 groups
  uint8_t* sK = sQ + 2 * TILE_BYTES;  // 2 stages
  uint8_t* sV = sK + 2 * TILE_BYTES;  // 2 stages
  uint8_t* sRaw = sV + 2 * TILE_BYTES;   // FP8: kRawStages half tiles
  Smem<FP8>& sm = *reinterpret_cast<Smem<FP8>*>(sRaw + (FP8 ? kRawStages * kRawBytes : 0));
  volatile int* abort_flag = &sm.abort_flag;

  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.k_full[s], FP8 ? 128 : 1);
      mbar_init(&sm.k_empty[s], 1);
      mbar_init(&sm.v_full[s], FP8 ? 128 : 1);
      mbar_init(&sm.v_empty[s], 1);
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.p_full[s], 8);   // a lane of each warp
      mbar_init(&sm.o_done[s], 1);
    }
    for (int s = 0; s < kTileSlots; ++s) {
      mbar_init(&sm.tile_full[s], 1);
      mbar_init(&sm.tile_empty[s], 16);
    }
    mbar_init(&sm.mma_done, 1);
    if constexpr (FP8) {
      for (int s = 0; s < kRawStages; ++s) {
        mbar_init(&sm.raw_full[s], 1);
        mbar_init(&sm.raw_empty[s], 64);
      }
      for (int s = 0; s < kScaleSlots; ++s) {
        mbar_init(&sm.scale_full[s], 1);
        mbar_init(&sm.scale_ready[s], 1);
      }
      for (int s = 0; s < 2; ++s) mbar_init(&sm.q_ready[s], 8);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch(&tmQ);
    tma_prefetch(&tmK);
    tma_prefetch(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = sm.tmem_slot;
  pdl_wait();
  const long long* prefix = p.prefix;
  if (p.rb.batch <= kPlanBatch) {
    plan_by_warps(p, sm.prefix, blockIdx.x == 0);
    prefix = sm.prefix;
  }

  constexpr int kSoft = FP8 ? 4 : 2;   // first softmax warp
  if (warp < kSoft) {
    if constexpr (FP8) reg_dec<kRegsFew>();
    if (warp == 0) {
      // ---------------------------------------------------------------- producer (whole warp)
      PieceWalk walk(p, prefix, lane == 0);
      Piece pc;
      const int npc = 128 / p.piece;   // K/V loads per block and half: lane i < npc issues piece i's
      const int none = p.kv.n_pages * p.kv.page_size;   // a row beyond the map: zeros
      uint32_t jb = 0, seg = 0;        // blocks and tiles so far
      uint32_t k_iss = 0, v_iss = 0, k_par = 0, v_par = 0;
      uint32_t raw = 0, scales_issued = 0;   // FP8: half tiles, and blocks whose scales are under way
      bool ok = true;
      for (;;) {
        const bool more = walk.next(p, &pc, lane == 0);
        const int groups = pc.ts.toks > p.g.TQ ? 2 : 1;   // row groups with tokens
        ok = mbar_wait(&sm.q_empty, (seg & 1) ^ 1u, p.status, abort_flag) &&
             mbar_wait(&sm.tile_empty[seg & (kTileSlots - 1)], ((seg / kTileSlots) & 1) ^ 1u, p.status, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (lane == 0) {
          TileInfo& ti = sm.tile[seg & (kTileSlots - 1)];
          ti.toks = more && ok ? pc.ts.toks : 0;
          if (more) {
            ti.p0 = pc.ts.p0;
            ti.p1 = pc.ts.p1;
            ti.n = pc.blk1 - pc.blk0;
            ti.row0 = pc.row0;
            ti.kvh = pc.kvh;
            ti.part = pc.whole ? -1 : (pc.blk0 == 0 ? 1 : 0);
            ti.groups = groups;
          }
          mbar_arrive(&sm.tile_full[seg & (kTileSlots - 1)]);
        }
        if (!more || !ok) break;
        if (lane == 0) {
          const int bytes = p.g.TQ * p.g.G * 128;
          mbar_arrive_expect_tx(&sm.q_full, 2 * groups * bytes);
          for (int x = 0; x < groups; ++x) {
            tma_load_3d(sQ + x * TILE_BYTES, &tmQ, &sm.q_full, 0, pc.kvh * p.g.G, pc.row0 + x * p.g.TQ);
            tma_load_3d(sQ + x * TILE_BYTES + HALF, &tmQ, &sm.q_full, 64, pc.kvh * p.g.G, pc.row0 + x * p.g.TQ);
          }
        }
        ++seg;
        __syncwarp();
        const int lo = p.g.window < 0 ? 0 : pc.ts.p0 - p.g.window;   // first key of any query's window
        for (int x = pc.blk0; x < pc.blk1; ++x, ++jb) {
          const int k0 = pc.ts.block(x) * kKeyBlock, s = jb & 1;
          const uint32_t par = (jb >> 1) & 1;
          int row = none;
          bool bad = false;
          if (lane < npc) {
            const int r0 = k0 + lane * p.piece, r1 = r0 + p.piece - 1;
            if (r0 <= pc.ts.p1 && (r0 < p.g.n_meta || r1 >= lo)) {
              const int page = page_of(p.kv, pc.b, r0);
              bad = page < 0;
              if (!bad) row = page * p.kv.page_size + r0 % p.kv.page_size;
            }
          }
          const unsigned bads = __ballot_sync(0xffffffffu, bad);
          if (bads && lane == 0) report_invalid(p.status);
          BlockInfo& bi = sm.block[jb & (kBlockSlots - 1)];
          if (lane < 4) {   // 32 rows per word
            uint32_t m = 0xffffffffu;
            if (bads)
              for (int r = 0; r < 32; ++r)
                if ((bads >> ((lane * 32 + r) / p.piece)) & 1u) m &= ~(1u << r);
            bi.valid[lane] = m;
          }
          if (lane == 0) {
            uint32_t f = 0;
            const int k1 = k0 + kKeyBlock - 1;
            for (int gx = 0; gx < 2; ++gx) {   // places of the group's rows: pa .. pb
              const int pa = pc.ts.p0 + gx * p.g.TQ, pb = min(pc.ts.p1, pa + p.g.TQ - 1);
              if (bads || k1 > pa || (p.g.window >= 0 && pb - k0 > p.g.window && k1 >= p.g.n_meta)) f |= 1u << gx;
            }
            if (k1 > pc.ts.p1 || max(k0, p.g.n_meta) < min(k0 + kKeyBlock, lo)) f |= kZeroV;
            bi.k0 = k0;
            bi.flags = f;
          }
          __syncwarp();
          if constexpr (FP8) {
            // the scales of the pieces that are there, then K and V in half tiles
            const int page = row / p.kv.page_size, at = row - page * p.kv.page_size;
            const bool have = lane < npc && row != none;
            const unsigned haves = __ballot_sync(0xffffffffu, have);
            uint64_t* sf = &sm.scale_full[jb % kScaleSlots];
            if (lane == 0) mbar_arrive_expect_tx(sf, 2 * __popc(haves) * p.piece * 4);
            __syncwarp();
            if (have) {
#pragma unroll
              for (int w = 0; w < 2; ++w)
                bulk_load_1d(&sm.scale[jb % kScaleSlots][w][lane * p.piece], p.kv.scales + page_scale(p.kv, w, page, at, pc.kvh),
                             p.piece * 4, sf);
            }
            scales_issued = jb + 1;
#pragma unroll 1
            for (int u = 0; ok && u < 4; ++u, ++raw) {   // K rows 0.., K rows 64.., V rows 0.., V rows 64..
              const uint32_t rs = raw % kRawStages;
              ok = __all_sync(0xffffffffu, mbar_wait(&sm.raw_empty[rs], ((raw / kRawStages) & 1) ^ 1u, p.status, abort_flag));
              if (!ok) break;
              if (lane == 0) mbar_arrive_expect_tx(&sm.raw_full[rs], kRawBytes);
              __syncwarp();
              const int r0 = lane * p.piece;
              if (lane < npc && (r0 >> 6) == (u & 1))
                tma_load_2d(sRaw + rs * kRawBytes + (r0 & 63) * DH, u < 2 ? &tmK : &tmV, &sm.raw_full[rs], pc.kvh * DH, row);
            }
            if (!ok) break;
            continue;
          }
          ok = __all_sync(0xffffffffu, mbar_wait(&sm.k_empty[s], par ^ 1u, p.status, abort_flag));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&sm.k_full[s], TILE_BYTES);
          __syncwarp();
          if (lane < npc) {
            uint8_t* dst = sK + s * TILE_BYTES + lane * p.piece * 128;
            tma_load_2d(dst, &tmK, &sm.k_full[s], pc.kvh * DH, row);
            tma_load_2d(dst + HALF, &tmK, &sm.k_full[s], pc.kvh * DH + 64, row);
          }
          k_iss |= 1u << s;
          k_par = (k_par & ~(1u << s)) | (par << s);
          ok = __all_sync(0xffffffffu, mbar_wait(&sm.v_empty[s], par ^ 1u, p.status, abort_flag));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&sm.v_full[s], TILE_BYTES);
          __syncwarp();
          if (lane < npc) {
            uint8_t* dst = sV + s * TILE_BYTES + lane * p.piece * 128;
            tma_load_2d(dst, &tmV, &sm.v_full[s], pc.kvh * DH, row);
            tma_load_2d(dst + HALF, &tmV, &sm.v_full[s], pc.kvh * DH + 64, row);
          }
          v_iss |= 1u << s;
          v_par = (v_par & ~(1u << s)) | (par << s);
        }
        if (!ok) break;   // the others leave by the abort flag
      }
      // every issued copy lands before the CTA may exit
      int never = 0;
      for (int s = 0; s < 2; ++s) {
        if (k_iss & (1u << s)) mbar_wait(&sm.k_full[s], (k_par >> s) & 1u, nullptr, &never, 100000000ull);
        if (v_iss & (1u << s)) mbar_wait(&sm.v_full[s], (v_par >> s) & 1u, nullptr, &never, 100000000ull);
      }
      if constexpr (FP8) {
        for (uint32_t u = raw > kRawStages ? raw - kRawStages : 0; u < raw; ++u)
          mbar_wait(&sm.raw_full[u % kRawStages], (u / kRawStages) & 1, nullptr, &never, 100000000ull);
        for (uint32_t u = scales_issued > kScaleSlots ? scales_issued - kScaleSlots : 0; u < scales_issued; ++u)
          mbar_wait(&sm.scale_full[u % kScaleSlots], (u / kScaleSlots) & 1, nullptr, &never, 100000000ull);
      }
      if (seg) mbar_wait(&sm.q_full, (seg - 1) & 1u, nullptr, &never, 100000000ull);
    } else if (warp == 1) {
      // ---------------------------------------------------------------- UMMA issuer (lane 0)
      if (lane == 0) {
        const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024), dK = sdesc_sw128(smem_u32(sK), 16, 1024),
                       dV = sdesc_sw128(smem_u32(sV), HALF, 1024);
        auto issue_s = [&](int x, int s) {  // S_x = Q_x K^T into TMEM columns [128 x, 128 x + 128)
          const uint64_t qd = sdesc_add(dQ, x * TILE_BYTES), kd = sdesc_add(dK, s * TILE_BYTES);
#pragma unroll
          for (int k = 0; k < DH / 16; ++k) {
            const uint32_t off = (k >> 2) * HALF + (k & 3) * 32;
            umma_bf16_ss(tmem_base + x * 128, sdesc_add(qd, off), sdesc_add(kd, off), IDESC_QK<FP8>, k != 0 ? 1u : 0u);
          }
          umma_commit(&sm.s_full[x]);
        };
        auto issue_pv = [&](int x, int s, bool acc) {  // O_x (+)= P_x V, P_x from TMEM over S_x
          const uint64_t vd = sdesc_add(dV, s * TILE_BYTES);
#pragma unroll
          for (int k = 0; k < 128 / 16; ++k)
            umma_bf16_ts(tmem_base + 256 + x * 128, tmem_base + x * 128 + k * 8, sdesc_add(vd, k * 16 * 128), IDESC_PV<FP8>,
                         (acc || k != 0) ? 1u : 0u);
          umma_commit(&sm.o_done[x]);
        };
        uint32_t jb = 0, cnt[2] = {0, 0};   // blocks so far: all, and per group
        uint32_t tiles[2] = {0, 0};         // and tiles, per group
        bool ok = true;
        for (uint32_t seg = 0; ok; ++seg) {
          const TileInfo& ti = sm.tile[seg & (kTileSlots - 1)];
          ok = mbar_wait(&sm.tile_full[seg & (kTileSlots - 1)], (seg / kTileSlots) & 1, p.status, abort_flag);
          if (!ok || ti.toks == 0) break;
          const int n = ti.n, gr = ti.groups;
          ok = mbar_wait(&sm.q_full, seg & 1, p.status, abort_flag) &&
               mbar_wait(&sm.k_full[jb & 1], (jb >> 1) & 1, p.status, abort_flag);
          // one group after the other, so that the first begins while the second still has its last tile's
          // output to write: S_x needs Q_x (FP8: in fp16), and the last P V of the previous tile, which
          // reads the TMEM columns that S_x goes over, done
          for (int x = 0; ok && x < gr; ++x) {
            if constexpr (FP8) ok = mbar_wait(&sm.q_ready[x], tiles[x]++ & 1, p.status, abort_flag);
            if (ok && cnt[x] > 0) ok = mbar_wait(&sm.o_done[x], (cnt[x] - 1) & 1, p.status, abort_flag);
            if (!ok) break;
            tc_fence_after();
            issue_s(x, jb & 1);
          }
          if (!ok) break;
          umma_commit(&sm.k_empty[jb & 1]);
          if (n == 1) umma_commit(&sm.q_empty);
          for (int j = 0; ok && j < n; ++j, ++jb) {
            for (int x = 0; ok && x < gr; ++x) {
              const uint32_t par = cnt[x] & 1;
              if (!mbar_wait(&sm.p_full[x], par, p.status, abort_flag)) { ok = false; break; }
              if (x == 0 && !mbar_wait(&sm.v_full[jb & 1], (jb >> 1) & 1, p.status, abort_flag)) { ok = false; break; }
              tc_fence_after();
              issue_pv(x, jb & 1, j > 0);
              ++cnt[x];
              if (x == gr - 1) umma_commit(&sm.v_empty[jb & 1]);
              if (j + 1 < n) {
                // S_x of the next block overwrites the TMEM columns this P V reads: wait for it
                if (!mbar_wait(&sm.o_done[x], par, p.status, abort_flag)) { ok = false; break; }
                if (x == 0 && !mbar_wait(&sm.k_full[(jb + 1) & 1], ((jb + 1) >> 1) & 1, p.status, abort_flag)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
                issue_s(x, (jb + 1) & 1);
                if (x == gr - 1) {
                  umma_commit(&sm.k_empty[(jb + 1) & 1]);
                  if (j + 2 == n) umma_commit(&sm.q_empty);
                }
              }
            }
          }
        }
        umma_commit(&sm.mma_done);
        int never = 0;
        mbar_wait(&sm.mma_done, 0, nullptr, &never, 100000000ull);
      }
    } else {
      // ---------------------------------------------------------------- e4m3 -> fp16 (two warps)
      if constexpr (FP8) {
        const int t = threadIdx.x - 2 * 32;   // of 64
        uint32_t jb = 0, raw = 0;
        bool ok = true;
        for (uint32_t seg = 0; ok; ++seg) {
          const volatile TileInfo& ti = sm.tile[seg & (kTileSlots - 1)];
          ok = __all_sync(0xffffffffu, mbar_wait(&sm.tile_full[seg & (kTileSlots - 1)], (seg / kTileSlots) & 1, p.status,
                                                 abort_flag));
          if (!ok || ti.toks == 0) break;
          const int n = ti.n, p1 = ti.p1, lo = p.g.window < 0 ? 0 : ti.p0 - p.g.window;
          uint32_t most = 0, least = 0x7f7fffffu;   // the largest and the least of V's scales so far, as bits
          for (int j = 0; ok && j < n; ++j, ++jb) {
            const uint32_t s = jb & 1, par = (jb >> 1) & 1, slot = jb % kScaleSlots, slot_par = (jb / kScaleSlots) & 1;
            BlockInfo& bi = sm.block[jb & (kBlockSlots - 1)];
            if (warp == 2) {
              // the scales as the products use them (see Smem), 0 for rows that no query of the tile sees.
              // Done before k_full, so that S of the block implies it.
              ok = __all_sync(0xffffffffu, mbar_wait(&sm.scale_full[slot], slot_par, p.status, abort_flag));
              if (!ok) break;
              const uint32_t valid = bi.valid[lane >> 3] >> ((lane & 7) * 4);
              const int key0 = bi.k0 + lane * 4;
              uint32_t seen = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (((valid >> e) & 1u) && key0 + e <= p1 && (key0 + e >= lo || key0 + e < p.g.n_meta)) seen |= 1u << e;
              float4& k4 = *reinterpret_cast<float4*>(&sm.scale[slot][0][lane * 4]);
              float4& v4 = *reinterpret_cast<float4*>(&sm.scale[slot][1][lane * 4]);
              float k[4] = {k4.x, k4.y, k4.z, k4.w}, v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (!((seen >> e) & 1u)) k[e] = v[e] = 0.f;
                const uint32_t bits = __float_as_uint(v[e]) & 0x7fffffffu;   // (an infinity or NaN: kApart)
                most = max(most, bits);
                if ((seen >> e) & 1u) least = min(least, bits);
              }
              most = __reduce_max_sync(0xffffffffu, most);
              const int ex = max(static_cast<int>(most >> 23) - 126, kUp - 127);   // every scale is below 2^ex
              const bool apart = __any_sync(0xffffffffu, (most >> 23) > (least >> 23) + kSpread);
              if (lane == 0) bi.ev = apart ? kApart : ex;
              if (!apart) {
                const float up = pow2(kUp - ex);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const __half2 h = __floats2half2_rn(v[e] * up, 0.f);
                  v[e] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&h));
                }
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t bits = __float_as_uint(v[e]);
                  const int x = static_cast<int>(bits >> 23) & 0xff;
                  const float exponent = x == 255 ? 0.f : static_cast<float>(max(x, 1) - 127);
                  const __half2 h = __floats2half2_rn(
                      x == 255 ? v[e] : x == 0 ? v[e] * pow2(126) : __uint_as_float((bits & 0x807fffffu) | 0x3f800000u), 0.f);
                  v[e] = __uint_as_float((__float_as_uint(exponent) & 0xffff0000u) | *reinterpret_cast<const uint32_t*>(&h));
                }
              }
              k4 = make_float4(k[0], k[1], k[2], k[3]);
              v4 = make_float4(v[0], v[1], v[2], v[3]);
              __syncwarp();
              if (lane == 0) mbar_arrive(&sm.scale_ready[slot]);
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&sm.scale_ready[slot], slot_par, p.status, abort_flag));
#pragma unroll 1
            for (int u = 0; ok && u < 4; ++u, ++raw) {
              const uint32_t rs = raw % kRawStages;
              if ((u & 1) == 0)
                ok = __all_sync(0xffffffffu, mbar_wait(u ? &sm.v_empty[s] : &sm.k_empty[s], par ^ 1u, p.status, abort_flag));
              ok = ok && __all_sync(0xffffffffu, mbar_wait(&sm.raw_full[rs], (raw / kRawStages) & 1, p.status, abort_flag));
              if (!ok) break;
              // 16 codes (one of a row's eight chunks) at a time, to two 16-byte chunks of the swizzled
              // tile.  The lanes of a row's upper half take the neighbouring row, so that eight lanes
              // meet no bank twice in either tile.
              const int up = (t >> 2) & 1, row0 = (t >> 3) ^ up, c = (t & 3) * 2;
              const uint32_t src = smem_u32(sRaw + rs * kRawBytes) + row0 * DH + (t & 7) * 16;
              const uint32_t dst = smem_u32((u < 2 ? sK : sV) + s * TILE_BYTES + up * HALF + ((u & 1) * 64 + row0) * 128);
              const uint32_t fs = smem_u32(&sm.scale[slot][1][(u & 1) * 64 + row0]);
              const uint32_t at0 = dst + ((c ^ row0) << 4), at1 = dst + (((c + 1) ^ row0) << 4);   // row & 7 = row0
              const bool hide = u >= 2 && (bi.flags & kZeroV);
              const int key0 = bi.k0 + (u & 1) * 64 + row0;
#pragma unroll 1
              for (int i0 = 0; i0 < 8; i0 += 4) {   // (eight at a time: 98 us against 93, see kRegs)
                float4 r4[4];   // in flight before the first is used
                uint32_t f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) r4[i] = lds_f4(src + (i0 + i) * 1024);
#pragma unroll
                for (int i = 0; i < 4; ++i)   // K: times 1
                  f[i] = u < 2 ? 0x3c003c00u : __byte_perm(lds_u32(fs + (i0 + i) * 32), 0u, 0x1010);
                if (hide) {   // rows of V that no query of the tile sees (they may hold NaN codes)
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const int key = key0 + (i0 + i) * 8;
                    if (key > p1 || (key < lo && key >= p.g.n_meta)) r4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                  }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const uint32_t w[4] = {__float_as_uint(r4[i].x), __float_as_uint(r4[i].y), __float_as_uint(r4[i].z),
                                         __float_as_uint(r4[i].w)};
                  uint32_t h[8];
#pragma unroll
                  for (int e = 0; e < 8; ++e) {
                    const uint32_t x = f16_of_e4m3(w[e >> 1], e & 1);
                    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&f[i]));
                    h[e] = *reinterpret_cast<const uint32_t*>(&y);
                  }
                  sts_u32x4(at0 + (i0 + i) * 1024, h[0], h[1], h[2], h[3]);
                  sts_u32x4(at1 + (i0 + i) * 1024, h[4], h[5], h[6], h[7]);
                }
              }
              fence_proxy_async_smem();
              // only now: an arrival right behind the loads can overtake them, and the next copy would
              // land in what they still read
              mbar_arrive(&sm.raw_empty[rs]);
              mbar_arrive(u < 2 ? &sm.k_full[s] : &sm.v_full[s]);
            }
          }
        }
      }
    }
  } else {
    if constexpr (FP8) reg_inc<kRegsSoft>();
    // ------------------------------------------------------------------ softmax (two groups of 8 warps)
    const int x = (warp - kSoft) >> 3;         // row group
    const int kh = ((warp - kSoft) >> 2) & 1;  // half of the keys and of O's columns
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tSx = tmem_base + x * 128 + lane_off, tOx = tmem_base + 256 + x * 128 + lane_off + kh * 64;
    const int rtok = x * p.g.TQ + r / p.g.G;   // this row's token of the tile
    constexpr float kRescaleLog2 = FP8 ? 4.0f : 8.0f;
    uint32_t jb = 0, cnt = 0;
    bool ok = true;
    for (uint32_t seg = 0;; ++seg) {
      const volatile TileInfo& ti = sm.tile[seg & (kTileSlots - 1)];
      ok = ok && __all_sync(0xffffffffu, mbar_wait(&sm.tile_full[seg & (kTileSlots - 1)], (seg / kTileSlots) & 1,
                                                   p.status, abort_flag));
      // every thread of the group takes the same steps from here on, so the group barriers are
      // reached by all of them; the group leaves together when any of them gave up
      ok = !bar_red_or(1 + x, 256, !ok);
      if (!ok || ti.toks == 0) break;
      const int n = ti.n;
      if (x >= ti.groups) {
        jb += n;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.tile_empty[seg & (kTileSlots - 1)]);
        continue;
      }
      float m_used = -INFINITY, l = 0.f, to_log2 = p.scale_log2;
      // FP8: O is held times 2^(kPUp - m_used + kUp - e_used); e_used is ev, or the row's own (kApart)
      float e_used = 0.f;
      if constexpr (FP8) {
        // this half of the row of Q from bf16 to fp16, its largest value in [2^7, 2^8)
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&sm.q_full, seg & 1, p.status, abort_flag));
        const uint32_t row = smem_u32(sQ + x * TILE_BYTES + kh * HALF + r * 128);
        uint32_t q[32], mx = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float4 v = lds_f4(row + ((c ^ (r & 7)) << 4));
          q[4 * c] = __float_as_uint(v.x);
          q[4 * c + 1] = __float_as_uint(v.y);
          q[4 * c + 2] = __float_as_uint(v.z);
          q[4 * c + 3] = __float_as_uint(v.w);
#pragma unroll
          for (int e = 0; e < 4; ++e) mx = max(mx, max(q[4 * c + e] & 0x7fffu, (q[4 * c + e] >> 16) & 0x7fffu));
        }
        sm.smax[cnt & 1][x][kh][r] = __uint_as_float(mx);
        bar_sync_n(1 + x, 256);
        mx = max(mx, __float_as_uint(sm.smax[cnt & 1][x][kh ^ 1][r]));
        const int f = min(134 - static_cast<int>(mx >> 7), kMostUp);   // (a row of zeros: kMostUp)
        const float up = pow2(f);
        to_log2 *= pow2(-f);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2 h = __floats2half2_rn(bf16lo(q[4 * c + e]) * up, bf16hi(q[4 * c + e]) * up);
            q[4 * c + e] = *reinterpret_cast<const uint32_t*>(&h);
          }
          sts_u32x4(row + ((c ^ (r & 7)) << 4), q[4 * c], q[4 * c + 1], q[4 * c + 2], q[4 * c + 3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_ready[x]);
      }
      for (int j = 0; j < n; ++j, ++jb, ++cnt) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&sm.s_full[x], cnt & 1, p.status, abort_flag));
        uint32_t sv[64];
        float m_half = -INFINITY;
        const volatile BlockInfo& bi = sm.block[jb & (kBlockSlots - 1)];
        const uint32_t flags = bi.flags;
        const int ev = FP8 ? bi.ev : 0;
        if (ok) {
          tc_fence_after();
          tmem_ld32(tSx + kh * 64, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
          tmem_ld32(tSx + kh * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
          tmem_wait_ld();
          if constexpr (FP8) scale64(sv, smem_u32(&sm.scale[jb % kScaleSlots][0][kh * 64]));
          if (flags & (1u << x)) {
            // key e of this half is visible iff e <= hi and (e >= lo or e < me), on a valid page
            const int base = bi.k0 + kh * 64, hi = ti.p0 + rtok - base, me = p.g.n_meta - base;
            const int lo = p.g.window < 0 ? -base : hi - p.g.window;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint32_t see = low_bits(hi + 1 - 32 * w) & (~low_bits(lo - 32 * w) | low_bits(me - 32 * w)) & bi.valid[kh * 2 + w];
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(see & (1u << e))) sv[32 * w + e] = __float_as_uint(-INFINITY);
            }
          }
          m_half = row_max64(sv) * to_log2;
        }
        if constexpr (FP8) {   // (the other parity is free: S of this block came after the last block's reads of it)
          if (__builtin_expect(ev == kApart, 0))
            sm.smax[(cnt + 1) & 1][x][kh][r] = row_reach64(sv, smem_u32(&sm.scale[jb % kScaleSlots][1][kh * 64]), to_log2);
        }
        // the row maximum over both halves; the barrier also orders this half's reads of
        // S before the other half's P stores (P of keys 64..127 lands in S columns 32..63)
        sm.smax[cnt & 1][x][kh][r] = m_half;
        tc_fence_before();
        bar_sync_n(1 + x, 256);
        tc_fence_after();
        const float m_cand = fmaxf(m_half, sm.smax[cnt & 1][x][kh ^ 1][r]);
        if (ok) {
          const bool need = m_cand > m_used + kRescaleLog2;
          float alpha = 1.f, down = 0.f;
          if (need) {
            down = m_used - m_cand;
            alpha = ex2_approx(down);  // 0 when m_used is -inf
            m_used = m_cand;
          }
          const float m_ref = (m_used == -INFINITY) ? 0.f : (FP8 ? m_used - kPUp : m_used);
          float alpha_o = alpha, sum;
          bool moved = need;
          if constexpr (FP8) {
            if (__builtin_expect(ev == kApart, 0)) {
              // e_used for the maximum as it is now (-inf: O holds nothing yet), then what this block's
              // reach asks for.  The first such block may also lower it, by what O's range allows: the
              // rows' scales were within 2^kSpread so far, so it ends at or below the row's own reach.
              const bool first = sm.block[(jb - 1) & (kBlockSlots - 1)].ev != kApart;
              const float m0 = m_used == -INFINITY ? 0.f : m_used;
              const float e_was = j == 0 || m_used == -INFINITY || down == -INFINITY ? -INFINITY : e_used + down;
              const volatile float(&reach)[2][128] = sm.smax[(cnt + 1) & 1][x];
              const float cand = fmaxf(reach[0][r], reach[1][r]) - m0 + kUp;
              e_used = first ? fmaxf(cand, e_was - 40.f) : cand > e_was + kRescaleLog2 ? cand : e_was;
              if (e_used == -INFINITY) e_used = 0.f;
              alpha_o = ex2_approx(e_was - e_used);
              moved |= e_was != e_used;
              sum = row_exp64_apart(sv, smem_u32(&sm.scale[jb % kScaleSlots][1][kh * 64]), to_log2, m0, kPUp + kUp - e_used);
            } else {
              sum = row_exp64<FP8>(sv, to_log2, m_ref);
              moved |= ev != static_cast<int>(e_used);
              alpha_o *= ex2_approx(e_used - ev);
              e_used = ev;
            }
          } else {
            sum = row_exp64<FP8>(sv, to_log2, m_ref);
          }
          tmem_st32(tSx + kh * 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
          if (j > 0 && __any_sync(0xffffffffu, moved)) {
            // rescale this half of O (every earlier P V of this group has completed: S_x(j)
            // was issued after it, and P_x V_j cannot start before p_full below)
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[16];
              tmem_ld16(tOx + c * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha_o);
              tmem_st16(tOx + c * 16, o);
            }
          }
          if (!FP8 && (flags & kZeroV)) {
            // rows of V that no query of the tile sees: [a0, a1) between the meta rows and the
            // window, [b0, 128) behind the last query
            const int k0 = bi.k0, tid = (warp - kSoft - 8 * x) * 32 + lane;
            const int a0 = max(0, p.g.n_meta - k0);
            const int a1 = min(kKeyBlock, p.g.window < 0 ? 0 : ti.p0 - p.g.window - k0), b0 = max(0, ti.p1 + 1 - k0);
            ok = __all_sync(0xffffffffu, mbar_wait(&sm.v_full[jb & 1], (jb >> 1) & 1, p.status, abort_flag));
            if (ok) {
              uint8_t* v = sV + (jb & 1) * TILE_BYTES;
              const int na = max(0, a1 - a0), rows = na + max(0, kKeyBlock - b0);
              for (int c = tid; c < rows * 16; c += 256) {
                const int q = c >> 4, row = q < na ? a0 + q : b0 + (q - na);
                *reinterpret_cast<uint4*>(v + ((c >> 3) & 1) * HALF + row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
            }
          }
          tmem_wait_st();
          l = fmaf(l, alpha, sum);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[x]);
      }
      ok = ok && __all_sync(0xffffffffu, mbar_wait(&sm.o_done[x], (cnt - 1) & 1, p.status, abort_flag));
      // the row sum over both halves
      sm.smax[cnt & 1][x][kh][r] = l;
      bar_sync_n(1 + x, 256);
      const float lsum = l + sm.smax[cnt & 1][x][kh ^ 1][r];
      if (ok) {
        tc_fence_after();
        const bool mine = rtok < (x + 1) * p.g.TQ && rtok < ti.toks, whole = ti.part < 0;
        const float down = FP8 ? ex2_approx(e_used - kUp) : 1.f, inv = lsum != 0.f ? 1.f / lsum : 0.f;
        __nv_bfloat16* orow = p.out + static_cast<long long>(ti.row0 + rtok) * p.out_ld +
                              (ti.kvh * p.g.G + r % p.g.G) * DH + kh * 64;
        const long long prow = (static_cast<long long>(blockIdx.x) * 2 + ti.part) * p.part_rows + x * 128 + r;
        // parts: [eight rows][four columns][row], which a warp writes in whole lines
        uint4* part = reinterpret_cast<uint4*>(p.part) + (prow >> 3) * (2 * DH) + kh * 128 + (r & 7);
        if (!whole && kh == 0) p.part_ml[prow] = make_float2(FP8 ? m_used - kPUp : m_used, lsum);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[16];
          tmem_ld16(tOx + c * 16, o);
          tmem_wait_ld();
          if constexpr (FP8) {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * down);
          }
          if (!whole) {
#pragma unroll
            for (int q = 0; q < 4; ++q) part[(4 * c + q) * 8] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          } else if (mine) {
            uint4* dst = reinterpret_cast<uint4*>(orow + c * 16);
#pragma unroll
            for (int q = 0; q < 2; ++q)
              dst[q] = make_uint4(pack_bf16(__uint_as_float(o[8 * q]) * inv, __uint_as_float(o[8 * q + 1]) * inv),
                                  pack_bf16(__uint_as_float(o[8 * q + 2]) * inv, __uint_as_float(o[8 * q + 3]) * inv),
                                  pack_bf16(__uint_as_float(o[8 * q + 4]) * inv, __uint_as_float(o[8 * q + 5]) * inv),
                                  pack_bf16(__uint_as_float(o[8 * q + 6]) * inv, __uint_as_float(o[8 * q + 7]) * inv));
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.tile_empty[seg & (kTileSlots - 1)]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Joins the parts of the tile that CTA i of the attention began and others finished, weighted by
// 2^(m - max): eight rows a CTA at a time, a warp 16 of their columns.
__global__ void __launch_bounds__(256) paged_join_tc(const __grid_constant__ PagedAttnParams p) {
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.x;
  const CutRecord cut = p.cut[i];
  const int c4 = (threadIdx.x >> 5) * 4 + ((threadIdx.x & 31) >> 3);   // column / 4
  for (int row = blockIdx.y * 8 + (threadIdx.x & 7); row < p.part_rows; row += gridDim.y * 8) {
    const int x = row >> 7, r = row & 127, tok = x * p.g.TQ + r / p.g.G, rg = r % p.g.G;
    if (r >= p.g.TQ * p.g.G || tok >= cut.toks) continue;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = i; c0 <= cut.last; c0 += 4) {   // CTA i's part is its second, the others' their first
      float2 ml[4];
      float4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        ml[u] = make_float2(-INFINITY, 0.f);
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c0 + u > cut.last) continue;
        const long long at = (2LL * (c0 + u) + (c0 + u == i)) * p.part_rows + row;
        ml[u] = p.part_ml[at];
        v[u] = reinterpret_cast<const float4*>(p.part)[(at >> 3) * (2 * DH) + c4 * 8 + (row & 7)];
      }
      const float mn = fmaxf(fmaxf(m, fmaxf(ml[0].x, ml[1].x)), fmaxf(ml[2].x, ml[3].x)), mr = mn == -INFINITY ? 0.f : mn;
      const float f0 = ex2_approx(m - mr);
      m = mn;
      l *= f0;
      acc = make_float4(acc.x * f0, acc.y * f0, acc.z * f0, acc.w * f0);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        // a part that saw no key; one whose scores are all NaN has a NaN for its sum, and counts
        if (ml[u].y == 0.f) continue;
        const float f = ex2_approx(ml[u].x - mr);
        l = fmaf(ml[u].y, f, l);
        acc = make_float4(fmaf(v[u].x, f, acc.x), fmaf(v[u].y, f, acc.y), fmaf(v[u].z, f, acc.z), fmaf(v[u].w, f, acc.w));
      }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    __nv_bfloat16* o = p.out + static_cast<long long>(cut.row0 + tok) * p.out_ld + (cut.kvh * p.g.G + rg) * DH;
    reinterpret_cast<uint2*>(o)[c4] = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<EncodeTiledFn>(ptr)
               : nullptr;
  }();
  return fn;
}

// A map of bf16 (128-byte swizzled boxes of 64 columns) or of bytes (plain boxes of 128).
bool encode(CUtensorMap* m, bool bytes, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  const cuuint32_t es[3] = {1, 1, 1};
  const EncodeTiledFn fn = encode_fn();
  return fn && fn(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                  const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  bytes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// The scratch is sized for the B200's 148 SMs; a launch uses at most that many CTAs.
constexpr int kMaxCtas = 148;

namespace {
int tc_part_rows(const RaggedBatch& rb, int G) { return rb.max_rows > 128 / G ? 256 : 128; }
}  // namespace

size_t paged_attention_tc_scratch(const PagedKv& kv, const RaggedBatch& rb, int n_q_heads) {
  return paged_scratch_layout(rb.batch, kMaxCtas, tc_part_rows(rb, n_q_heads / kv.hkv), DH).total;
}

cudaError_t launch_paged_attention_tc(const PagedAttnDesc& a, cudaStream_t st) {
  static std::atomic<uint64_t> attr_done{0}, attr8_done{0};
  const bool fp8 = a.kv.type == CACHE_E4M3;
  if (cudaError_t e = fp8 ? smem_attr_once(paged_attn_tc<true>, smem_bytes<true>(), attr8_done)
                          : smem_attr_once(paged_attn_tc<false>, smem_bytes<false>(), attr_done))
    return e;
  if (fp8) {   // the registers that the softmax warps ask for have to be there: the others would wait for good
    static const bool have = [] {
      cudaFuncAttributes at;
      return cudaFuncGetAttributes(&at, paged_attn_tc<true>) == cudaSuccess && at.numRegs >= kRegs;
    }();
    if (!have) return cudaErrorInvalidConfiguration;
  }
  const int ctas = num_sms() < kMaxCtas ? num_sms() : kMaxCtas;
  PagedAttnParams p{};
  p.kv = a.kv;
  p.rb = a.rb;
  p.g.G = a.n_q_heads / a.kv.hkv;
  p.g.TQ = 128 / p.g.G;
  p.g.tile_tok = 2 * p.g.TQ;
  p.g.n_meta = a.n_meta;
  p.g.window = a.window;
  p.part_rows = tc_part_rows(a.rb, p.g.G);
  const PagedScratch L = paged_scratch_layout(a.rb.batch, kMaxCtas, p.part_rows, DH);
  uint8_t* sc = static_cast<uint8_t*>(a.scratch);
  p.prefix = reinterpret_cast<long long*>(sc + L.prefix);
  p.part = reinterpret_cast<float*>(sc + L.part);
  p.part_ml = reinterpret_cast<float2*>(sc + L.ml);
  p.cut = reinterpret_cast<CutRecord*>(sc + L.cut);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.out_ld = a.out_ld;
  const int most = fp8 ? 64 : 128;
  p.piece = a.kv.page_size < most ? a.kv.page_size : most;
  p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(DH));
  p.status = a.status;
  CUtensorMap tq, tk, tv;
  const cuuint64_t qd[3] = {DH, static_cast<cuuint64_t>(a.n_q_heads), static_cast<cuuint64_t>(a.rb.total_rows)};
  const cuuint64_t qs[2] = {DH * 2, static_cast<cuuint64_t>(a.q_ld) * 2};
  const cuuint32_t qb[3] = {64, static_cast<cuuint32_t>(p.g.G), static_cast<cuuint32_t>(p.g.TQ)};
  const cuuint64_t rows = static_cast<cuuint64_t>(a.kv.n_pages) * a.kv.page_size;
  const cuuint64_t row_bytes = static_cast<cuuint64_t>(a.kv.hkv) * DH * (fp8 ? 1 : 2);
  const cuuint64_t kd[2] = {static_cast<cuuint64_t>(a.kv.hkv) * DH, rows}, ks[1] = {row_bytes};
  const cuuint32_t kb[2] = {fp8 ? 128u : 64u, static_cast<cuuint32_t>(p.piece)};
  if (!encode(&tq, false, 3, a.q, qd, qs, qb) || !encode(&tk, fp8, 2, a.kv.pages, kd, ks, kb) ||
      !encode(&tv, fp8, 2, static_cast<const uint8_t*>(a.kv.pages) + rows * row_bytes, kd, ks, kb))
    return cudaErrorInvalidValue;
  if (a.rb.batch > kPlanBatch)
    if (cudaError_t e = launch(paged_plan_kernel, dim3(1), dim3(1024), 0, st, a.kv, a.rb, p.g, p.prefix, a.status)) return e;
  if (cudaError_t e = fp8 ? launch(paged_attn_tc<true>, dim3(ctas), dim3(kThreadsFp8), smem_bytes<true>(), st, tq, tk, tv, p)
                          : launch(paged_attn_tc<false>, dim3(ctas), dim3(kThreads), smem_bytes<false>(), st, tq, tk, tv, p))
    return e;
  return launch(paged_join_tc, dim3(ctas - 1, p.part_rows / 32), dim3(256), 0, st, p);
}

}  // namespace hy
