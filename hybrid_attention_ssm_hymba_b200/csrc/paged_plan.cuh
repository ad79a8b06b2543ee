// paged_plan.cuh -- how the attention over a paged cache is cut into equal pieces on the
// device (the host knows no length).  The queries of one sequence and K/V head are packed
// (token-major, the G query heads of a token next to one another) into row groups of TQ
// tokens (TQ * G <= 128 rows); a tile is `groups` row groups that share every K/V block, and
// visits 128-key blocks: those of the meta rows, then those of the window up to its last row.
// All blocks of all tiles, in the order (sequence, K/V head, tile, block), form one line of W
// blocks, of which each of n CTAs takes W / n or one more.  A tile cut by such a boundary is
// computed in parts; the CTA that begins it records who has the others, and a second kernel joins
// them in the order of the CTAs, so a call gives the same bits every time.  Few and many sequences,
// short and long, fill the SMs alike; what a cut costs is its part's 4 dh bytes a row, written and
// read once.
#pragma once

#include "paged.cuh"

namespace hy {

constexpr int kKeyBlock = 128;

struct PagedGeo {
  int G, TQ, tile_tok;   // query heads per K/V head; tokens per row group; tokens per tile
  int n_meta, window;
};

// A tile that CTA i begins and others finish: its rows, and the last CTA with a part of it.
// toks = 0: CTA i leaves no tile unfinished.
struct CutRecord {
  int row0, toks, kvh, last;
};

// What the attention kernels and the join share.
struct PagedAttnParams {
  PagedKv kv;
  RaggedBatch rb;
  PagedGeo g;
  long long* prefix;    // [batch + 1], see paged_plan_kernel
  const __nv_bfloat16* q;
  long long q_ld;
  __nv_bfloat16* out;
  long long out_ld;
  float* part;          // [CTA][2][part_rows][dh] (the rows' order is the kernel's own): 0 = the CTA's first
                        // tile continued, 1 = its last tile begun
  float2* part_ml;      // [CTA][2][part_rows] (m in log2 units, sum)
  CutRecord* cut;       // [CTA]
  int part_rows;
  int page_shift;       // log2(page_size) where that is a power of two, else -1
  int piece;            // tensor-core kernel: rows of one K/V load
  float scale_log2;     // log2(e) / sqrt(dh)
  unsigned* status;
};
inline int page_shift(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return (1 << s) == page_size ? s : -1;
}
struct PagedScratch {
  size_t prefix, part, ml, cut, total;
};
inline PagedScratch paged_scratch_layout(int batch, int ctas, int part_rows, int dh) {
  auto al = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  PagedScratch s;
  size_t o = 0;
  s.prefix = o; o = al(o + (static_cast<size_t>(batch) + 1) * 8);
  s.part = o; o = al(o + static_cast<size_t>(ctas) * 2 * part_rows * dh * 4);
  s.ml = o; o = al(o + static_cast<size_t>(ctas) * 2 * part_rows * 8);
  s.cut = o; o = al(o + static_cast<size_t>(ctas) * sizeof(CutRecord));
  s.total = o;
  return s;
}

// One tile's visit: block x of [0, n) starts at key 128 * block(x).
struct TileSpan {
  int tok0, toks;       // first token (of the sequence's new ones) and their number
  int p0, p1;           // cache rows of the first and last token
  int first, wlo, n;    // blocks [0, first), then [wlo, wlo + n - first)
  HY_DEV int block(int x) const { return x < first ? x : wlo + (x - first); }
};

HY_DEV TileSpan tile_span(const PagedGeo& g, const Seq& s, int t) {
  TileSpan r;
  r.tok0 = t * g.tile_tok;
  r.toks = min(g.tile_tok, s.n - r.tok0);
  r.p0 = s.len - s.n + r.tok0;
  r.p1 = r.p0 + r.toks - 1;
  r.first = r.wlo = 0;
  if (g.window >= 0) {
    r.wlo = max(0, r.p0 - g.window) / kKeyBlock;
    r.first = min((min(g.n_meta, r.p1 + 1) + kKeyBlock - 1) / kKeyBlock, r.wlo);
  }
  r.n = r.first + r.p1 / kKeyBlock - r.wlo + 1;
  return r;
}

HY_DEV bool key_visible(const PagedGeo& g, int i, int j) {
  return j <= i && (g.window < 0 || i - j <= g.window || j < g.n_meta);
}

// Blocks of all tiles of a sequence and one K/V head (every lane of the warp gets the sum).
HY_DEV long long seq_blocks(const PagedGeo& g, const Seq& s) {
  const int tiles = (s.n + g.tile_tok - 1) / g.tile_tok;
  long long sum = 0;
  for (int t = threadIdx.x & 31; t < tiles; t += 32) sum += tile_span(g, s, t).n;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Writes prefix[b] = blocks of all sequences before b (every K/V head), prefix[batch] = W; one
// CTA of 1024 threads.  Sequences whose lengths do not fit are recorded and have no blocks.
static __global__ void __launch_bounds__(1024) paged_plan_kernel(const PagedKv kv, const RaggedBatch rb, const PagedGeo g,
                                                                 long long* prefix, unsigned* status) {
  __shared__ long long cnt[1024], wsum[32];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long carry = 0;
  for (int b0 = 0; b0 < rb.batch; b0 += 1024) {
    for (int i = warp; i < 1024; i += 32) {
      Seq s;
      long long c = 0;
      if (b0 + i < rb.batch) {
        if (load_seq(rb, kv, b0 + i, &s)) c = seq_blocks(g, s) * kv.hkv;
        else if (lane == 0) report_invalid(status);
      }
      if (lane == 0) cnt[i] = c;
    }
    __syncthreads();
    long long v = cnt[threadIdx.x];
    const long long own = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) wsum[warp] = v;
    __syncthreads();
    long long before = carry;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    if (b0 + static_cast<int>(threadIdx.x) < rb.batch) prefix[b0 + threadIdx.x] = before + v - own;
    long long all = 0;
    for (int w = 0; w < 32; ++w) all += wsum[w];
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) prefix[rb.batch] = carry;
}

// a / b for non-negative a and positive b (32-bit where that does: a 64-bit division costs a
// kernel's first microsecond)
HY_DEV long long div_pos(long long a, long long b) {
  return (a | b) >> 32 ? a / b : static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// The pieces of a line of W blocks over at most `ctas` CTAs: the first `more` have one block more
// than the rest.  One block is worth a CTA: 64 rows on an empty cache, four tiles of a block, take
// 16.5 us, with two blocks at least 23.5 (four ragged prompts of up to 300 rows 28.1 and 27.2).
struct PieceLine {
  long long each, more;
  int n;
  HY_DEV PieceLine(long long w, int ctas) {
    n = static_cast<int>(w < ctas ? w : ctas);
    each = n ? div_pos(w, n) : 0;
    more = w - each * n;
  }
  HY_DEV long long start(int i) const { return i * each + (i < more ? i : more); }   // i <= n
  HY_DEV int owner(long long block) const {
    const long long wide = more * (each + 1);
    return static_cast<int>(block < wide ? div_pos(block, each + 1) : more + div_pos(block - wide, each));
  }
};

// A walk along the line from block `w`; every lane of a warp holds the same state.
struct Walk {
  int b, kvh, t, off;   // sequence, K/V head, tile, first block of the tile still to do
  int tiles;
  Seq s;

  HY_DEV void load(const RaggedBatch& rb, const PagedKv& kv, const PagedGeo& g) {
    tiles = load_seq(rb, kv, b, &s) ? (s.n + g.tile_tok - 1) / g.tile_tok : 0;
  }
  HY_DEV void seek(const RaggedBatch& rb, const PagedKv& kv, const PagedGeo& g, const long long* prefix, long long w) {
    int lo = 0, hi = rb.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= w) lo = mid;
      else hi = mid;
    }
    b = lo;
    load(rb, kv, g);
    long long rem = w - prefix[b];
    const long long per = div_pos(prefix[b + 1] - prefix[b], kv.hkv);
    kvh = static_cast<int>(div_pos(rem, per));
    rem -= kvh * per;
    const int lane = threadIdx.x & 31;
    for (int t0 = 0;; t0 += 32) {   // ends: rem < per = the sum over the tiles
      const long long c = t0 + lane < tiles ? tile_span(g, s, t0 + lane).n : 0;
      long long inc = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, inc > rem);
      if (hit || t0 + 32 >= tiles) {
        const int l = hit ? __ffs(hit) - 1 : 31;
        t = t0 + l;
        off = static_cast<int>(rem - __shfl_sync(0xffffffffu, inc - c, l));
        return;
      }
      rem -= __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  // To the next tile that has work (false: behind the last sequence).
  HY_DEV bool advance(const RaggedBatch& rb, const PagedKv& kv, const PagedGeo& g) {
    off = 0;
    if (++t < tiles) return true;
    t = 0;
    if (++kvh < kv.hkv) return true;
    kvh = 0;
    do {
      if (++b >= rb.batch) return false;
      load(rb, kv, g);
    } while (tiles == 0);
    return true;
  }
};

// A CTA's piece of the line, tile by tile (every lane of a warp holds the same state).
struct Piece {
  TileSpan ts;
  int b, kvh, row0;     // row0: ragged row of the tile's first token
  int blk0, blk1;       // blocks of the tile to do here
  bool whole;
};
struct PieceWalk {
  Walk w;
  long long left, at;    // blocks left of the piece, and the place on the line
  PieceLine line;
  bool first = true;
  // `writer`: the one thread of the CTA that records what it leaves unfinished (nothing, until
  // its walk comes to it: a CTA that gives up leaves no record of an earlier call)
  HY_DEV PieceWalk(const PagedAttnParams& p, const long long* prefix, bool writer)
      : line(prefix[p.rb.batch], gridDim.x) {
    const int cta = blockIdx.x;
    if (writer) p.cut[cta] = {0, 0, 0, 0};
    left = 0;
    if (cta >= line.n) return;
    at = line.start(cta);
    left = line.start(cta + 1) - at;
    w.seek(p.rb, p.kv, p.g, prefix, at);
  }
  HY_DEV bool next(const PagedAttnParams& p, Piece* o, bool writer) {
    if (left <= 0 || (!first && !w.advance(p.rb, p.kv, p.g))) return false;
    first = false;
    o->ts = tile_span(p.g, w.s, w.t);
    o->b = w.b;
    o->kvh = w.kvh;
    o->row0 = w.s.q0 + o->ts.tok0;
    o->blk0 = w.off;
    o->blk1 = static_cast<int>(min(static_cast<long long>(o->ts.n), w.off + left));
    o->whole = o->blk0 == 0 && o->blk1 == o->ts.n;
    left -= o->blk1 - o->blk0;
    at += o->blk1 - o->blk0;
    if (writer && left <= 0 && o->blk0 == 0 && !o->whole)
      p.cut[blockIdx.x] = {o->row0, o->ts.toks, o->kvh, line.owner(at + (o->ts.n - o->blk1) - 1)};
    return true;
  }
};

// The same prefix by a CTA itself, for a small batch: one warp a sequence.  cnt: shared,
// [batch + 1]; every thread of the CTA calls it.  `report`: what does not fit is recorded (one
// CTA of the launch).
HY_DEV void plan_by_warps(const PagedAttnParams& p, long long* cnt, bool report) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int b = warp; b < p.rb.batch; b += blockDim.x >> 5) {
    Seq s;
    long long c = 0;
    if (load_seq(p.rb, p.kv, b, &s)) c = seq_blocks(p.g, s) * p.kv.hkv;
    else if (report && lane == 0) report_invalid(p.status);
    if (lane == 0) cnt[b] = c;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    long long sum = 0;
    for (int b = 0; b < p.rb.batch; ++b) {
      const long long c = cnt[b];
      cnt[b] = sum;
      sum += c;
    }
    cnt[p.rb.batch] = sum;
  }
  __syncthreads();
}

}  // namespace hy
