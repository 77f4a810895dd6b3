// attend_tokens.cu -- attention of several query tokens a sequence, on the
// 5th-generation tensor cores: whole prompts (causal, packed or padded, behind rows
// that the sequence already has or none) and trees of drafted tokens over a cache.
//
// For one sequence and key head the query rows are those of one matrix Q [nq*N, D], N =
// G / H (of a part of the key head's, where they are more than 128), row t*N + j for token
// t and query head j:
//   S = Q K^T * scale,  P = e^(S - m),  O = P V,  l = sum P,
// over the sequence's own rows, which every token sees, and its tokens' keys, of which
// token t sees 0..t (a prompt) or itself and its ancestors (a tree). The arithmetic is
// that of attend_prefix.cu: 16-bit weights for the second product (the sum of two 16-bit
// parts with up to 128 query rows), the sum l of the unrounded ones in fp32 relative to
// m, which moves only when the maximum has grown by 2^8. Two parts at more rows, too, would
// give outputs whose error is their own rounding's; with one it is 1.2 to 1.5 times that (two
// half steps, independent), and the products are two instead of three: 8 x 4096 tokens 823
// us, 1265 with two parts, one prompt of 8192 390 and 585, of 512 13.6 and 16.6.
//
// Work: see TokensPlan. A half block is the rows of 128 / N tokens, which one TMA box
// brings. A block is PAIR: one half, its key tiles dealt alternately to two streams; else
// two halves, a stream for either, both on every tile. SPLIT, a PAIR of at most 64 query
// rows: they lie in Q twice, and of a tile's keys the first copy's weights are kept for the
// first 64 and the second's for the rest, so that all softmax threads have work. Key tiles
// past the last row's are not visited. A piece of a block that another CTA finishes
// leaves its unnormalised O, m and l in the workspace for the join kernel below.
//
// Roles in a 384-thread CTA, one an SM:
//   warp 0      walks the CTA's range and tells the others (Seg); one thread issues TMA
//               loads of key and value tiles (128 rows, 128-byte swizzle) into one ring,
//               in the order they are used;
//   warp 1      issues tcgen05.mma: S = Q K^T from shared memory, then O += P V with P
//               from TMEM and V as it lies in memory;
//   warps 2, 3  issue the TMA loads of the query rows, the next block's as soon as the
//               last logits of this one are done; mend tiles on their way: values that no
//               row of the block sees, or some rows do not and that are not finite, become
//               zeros (0 * NaN would spoil the sums); a cache's keys whose compaction is
//               pending are re-rotated;
//   warps 4..11 two softmax warpgroups, one per stream, a query row a thread. The next
//               block's first logits are computed while the outputs are written.
// A value that is not finite, in a tile that some rows see in part, is added to the
// output of the rows that see it at the end, from memory.
// Every mbarrier wait is bounded; on expiry the CTA leaves NaN in its rows.
//
// Measured on GB300 (D = 128, 32 query heads on 8 unless said): one prompt of 8192 tokens
// 385-400 us, 1.37-1.43 PFLOP/s (0.70-0.73 of the measured matrix rate; the tensor pipe 65%
// busy); 8 x 4096 tokens 815-830 us; 8 x 1024 101 us; 160 tokens 8.7 us, of which start and
// end are most; 32 sequences of 16 drafted tokens on 2048 rows 59 us, 4.7 TB/s of rows. A
// tile of 256 query rows, its rows in L2 and all to be seen, takes 1.55 (bf16) to 1.59 us
// (fp16) at 2.07 GHz, in which the products have 1.05 and the rest is the chain from logits to
// weights and back; D = 64 1.31; PAIR 1.24 and 1.0, SPLIT 1.12 and 0.91 (from the times of 152
// blocks on 1024 and on 8192 rows). A change of blocks costs 3.5 us beside their tiles, D = 64
// 3.1 (152 k blocks of three tiles, k 4 and 16). Tried and
// slower: the query rows by cp.async of the softmax or the helper warps (5 us a block; TMA
// below 1), every role walking its range itself (224 bytes of spills a thread, 1336 against
// 1032 us for 8 x 4096 tokens at the time), one loop over the two streams' products (450
// against 404 us for 8192 tokens), the code of a tile twice, with masks and without (D =
// 64 faster by 9%, 128 slower by 2 to 5).
#include "attend_tokens.cuh"
#include "tcgen05.cuh"

#include <algorithm>
#include <atomic>

namespace kvx {
namespace {

constexpr int kT = 128;                // query rows of a stream, keys of a tile
constexpr int kThreads = 384;
constexpr int kTmem = 512;
constexpr float kNegInf = -__builtin_huge_valf();
// As in attend_prefix.cu: how far (log2) a weight may exceed the first maximum's, and
// that maximum's own weight.
constexpr float kLazy = 8.f;
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 7.f : 0.f;
constexpr float kFar = 0x1p23f;        // base-2 logits from here on are whole numbers
// What the start of a block costs, in tiles of half a block: with 1, 2, 3 and 4 a prompt of
// 8192 tokens takes 392, 390, 395 and 399 us, unequal trees on up to 65521 rows 325, 297, 292 and
// 291, packed prompts 806, 777, 789 and 808.
constexpr int kStartTiles = 2;

// What a row tensor's TMA coordinates of heads and sequences are multiplied by: 0 where
// all share the rows.
struct Coords {
  int h, b;
};
struct MapArgs {
  Coords q, k, v, kn, vn;
};

struct Params {
  TokensArgs a;
  TokensPlan plan;
  MapArgs at;
  float* part_o;           // [slot][D/4][block_rows] float4
  float2* part_ml;         // [slot][block_rows]
  TokensAt* first;         // [ctas + 1]
  int* err;
  int stall;
  int out_box;             // omap describes the outputs, a half block's 32 columns a box
};

__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, const Coords& c, int d, int row, int h,
                                              int b, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(d), "r"(h * c.h), "r"(row), "r"(b * c.b), "r"(bar)
      : "memory");
}

// ---------------------------------------------------------------- the work
// Costs of one head group's half blocks (PAIR: blocks) of a sequence, in 1/128 tiles:
// half block j of causal tokens sees up to (j + 1) * half tokens' keys; a tree's see all.
struct Cost {
  int64_t base;
  int step, halves;        // of half block j: base + j * step
  __device__ __forceinline__ Cost(const TokensArgs& a, const TokensPlan& p, const Seq& s) {
    const int per = p.pair ? a.half : 2 * a.half;
    halves = (int)((unsigned)(s.nq + per - 1) / (unsigned)per) * (p.pair ? 1 : 2);
    base = p.even ? 1 : (int64_t)(1 + s.ta + kStartTiles) * kT;
    step = p.even || a.parents ? 0 : a.half;
  }
  __device__ __forceinline__ int64_t before(int j) const {   // of 0 .. j - 1
    return j * base + (int64_t)step * ((int64_t)j * (j - 1) / 2);
  }
  __device__ __forceinline__ int64_t head() const { return before(halves); }
  // The last j with before(j) <= y, 0 <= y < head().
  __device__ __forceinline__ int find(int64_t y) const {
    // (the root of step j^2 / 2 + b j = y, without a difference)
    const float b = (float)base - 0.5f * (float)step, f = (float)y;
    int j = (int)__fdividef(2.f * f, b + sqrtf(b * b + 2.f * (float)step * f));
    j = max(0, min(j, halves - 1));
    while (j > 0 && before(j) > y) --j;
    while (j < halves - 1 && before(j + 1) <= y) ++j;
    return j;
  }
};

// Tiles that the tokens before `tokens` of a sequence visit.
__device__ __forceinline__ int tiles_of(const TokensArgs& a, const Seq& s, int tokens) {
  return s.ta + ((a.parents ? s.nq : min(s.nq, tokens)) + kT - 1) / kT;
}
__device__ __forceinline__ int block_tokens(const TokensArgs& a, const TokensPlan& p) { return p.pair ? a.half : 2 * a.half; }
// (blocks are of at most 256 tokens, and there are fewer than 2^30)
__device__ __forceinline__ int block_tiles(const TokensArgs& a, const TokensPlan& p, const Seq& s, int i) {
  return tiles_of(a, s, (i + 1) * block_tokens(a, p));
}

// Start of the range that begins at cost y of sequence b, which is in it. Quotients are
// taken in floats: whatever they round to, both CTAs that meet here find the same.
__device__ __forceinline__ TokensAt locate(const TokensArgs& a, const TokensPlan& p, int b, int64_t y) {
  const Seq s = load_seq(a, b);
  const Cost c(a, p, s);
  const int64_t head = c.head();
  TokensAt at;
  at.b = b;
  at.h = max(0, min((int)__fdividef((float)y, (float)head), a.heads - 1));
  while (at.h > 0 && at.h * head > y) --at.h;
  while (at.h < a.heads - 1 && (at.h + 1) * head <= y) ++at.h;
  y -= at.h * head;
  const int per = p.pair ? 1 : 2;
  at.i = c.find(y) / per;
  at.k = 0;
  if (!p.whole) {
    const int64_t c0 = c.before(at.i * per), c1 = c.before((at.i + 1) * per);
    const int tiles = block_tiles(a, p, s, at.i);
    at.k = max(0, min((int)((float)tiles * __fdividef((float)(y - c0), (float)(c1 - c0))), tiles - 1));
  }
  return at;
}

// The range of this CTA, [ends_s[0], ends_s[1]), once the CTA has synchronised; all
// threads, with a barrier. Either end is found by a thread of its own.
__device__ __forceinline__ void find_range(const TokensArgs& a, const TokensPlan& p, int64_t* sums_s, TokensAt* ends_s) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool even = !a.starts && !a.new_lens && !a.lens;
  const int share = (int)((unsigned)(a.B + kThreads - 1) / (unsigned)kThreads);
  int64_t* const from_s = sums_s + kThreads / 32;    // where each thread's share begins in its warp's
  if (!even) {
    const int b0 = min(a.B, tid * share), b1 = min(a.B, b0 + share);
    int64_t own = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) own += a.heads * Cost(a, p, load_seq(a, b)).head();
    int64_t to = own;                                // of this and lower lanes
#pragma unroll 1
    for (int d = 1; d < 32; d *= 2) {
      const int64_t x = __shfl_up_sync(~0u, to, d);
      if (lane >= d) to += x;
    }
    from_s[tid] = to - own;
    if (lane == 31) sums_s[warp] = to;
    __syncthreads();
  }
  if (tid & ~32) return;                             // (threads 0 and 32 go on)
  if (even && p.even) {                              // a block a CTA
    const unsigned per = block_tokens(a, p), n = (a.S + per - 1) / per, u = blockIdx.x + (tid >> 5), hb = u / n;
    const int b = (int)(hb / (unsigned)a.heads);
    ends_s[tid >> 5] = TokensAt{b, (int)hb - b * a.heads, (int)(u - hb * n), 0};
    return;
  }
  int64_t seq = 0, total = 0;
  if (even) {
    seq = a.heads * Cost(a, p, load_seq(a, 0)).head();
    total = a.B * seq;
  } else {
#pragma unroll 1
    for (int w = 0; w < kThreads / 32; ++w) total += sums_s[w];
  }
  const int c = blockIdx.x + (tid >> 5);
  TokensAt at{a.B, 0, 0, 0};
  if (c < p.ctas && total > 0) {
    // c * total / ctas (or about that: any ascending function does)
    int64_t x = min((int64_t)(((double)total * c + 0.5) * p.per_cta), total - 1);
    int b;
    if (even) {
      b = max(0, min((int)__fdividef((float)x, (float)seq), a.B - 1));
      while (b > 0 && b * seq > x) --b;
      while (b < a.B - 1 && (b + 1) * seq <= x) ++b;
      x -= b * seq;
    } else {
      int w = 0;
      while (w < kThreads / 32 - 1 && x >= sums_s[w]) x -= sums_s[w++];
      int i = 31;                                    // the last share that begins at or before x
      while (i > 0 && from_s[w * 32 + i] > x) --i;
      x -= from_s[w * 32 + i];
#pragma unroll 1
      for (b = (w * 32 + i) * share; b < a.B - 1; ++b) {
        const int64_t of = a.heads * Cost(a, p, load_seq(a, b)).head();
        if (x < of) break;
        x -= of;
      }
    }
    at = locate(a, p, b, x);
  }
  ends_s[tid >> 5] = at;
}

// A block's tiles k0 .. k1 - 1, as the producer finds them and the other roles read them
// in shared memory (tiles counted from k0). Kept there, none of it stands in the softmax
// threads' registers.
struct Seg {
  int n[2];                // tiles that the first and the second half's rows visit (PAIR: all)
  int tiles;               // k1 - k0
  int own, first;          // the first of them: of own rows, from row `first` on
  int left;                // own rows from the first tile on
  int gap;                 // the evicted row still in place, so too; or -1
  int part, hole;          // the own tile that ends inside, and that with the evicted row; or -1
  int turn;                // the first own tile with keys that await their re-rotation
  int mask;                // the first tile of the tokens' that some rows see in part
  int kb;                  // what a tile's index is short of its place among the tokens'
  int b, h, kv, tok0, nq;  // sequence, head group, key head; its first token (packed) and number
  int tok;                 // the block's first token
  int whole, from_start;   // all of the block's tiles; its first
};
constexpr int kSegs = 8;                 // more than the ring can hold tiles of, at once
constexpr int kNever = 0x7FFFFFFF;

// The walk over a CTA's range (warp-collective).
struct Walk {
  TokensAt at, end;
  int loaded;
  Seq s;
  __device__ __forceinline__ Walk(const TokensAt* ends) : at(ends[0]), end(ends[1]), loaded(-1) {}
  __device__ __forceinline__ bool next(const TokensArgs& a, const TokensPlan& p, Seg& g) {
    while (true) {
      if (at.b > end.b || (at.b == end.b && (at.h > end.h || (at.h == end.h && (at.i > end.i || (at.i == end.i && at.k >= end.k))))))
        return false;
      if (at.b != loaded) {
        s = load_seq(a, at.b);
        loaded = at.b;
      }
      if (s.nq == 0) {                               // on to the next sequence that has tokens
        const int lane = threadIdx.x & 31;
        const bool some = at.b + 1 + lane >= a.B || load_seq(a, at.b + 1 + lane).nq > 0;
        const unsigned found = __ballot_sync(~0u, some);
        at = TokensAt{at.b + (found ? __ffs(found) : 32), 0, 0, 0};
        if (at.b >= a.B) return false;
        continue;
      }
      const int all = block_tiles(a, p, s, at.i), k0 = at.k;
      const int k1 = at.b == end.b && at.h == end.h && at.i == end.i ? end.k : all;
      g.b = at.b;
      g.h = at.h;
      g.kv = a.groups == 1 ? at.h : at.h / a.groups;
      const int e = a.pend ? a.pend[g.b * (a.groups == 1 ? a.heads : a.heads / a.groups) + g.kv] : -1, n = s.n + (e >= 0);
      g.tiles = k1 - k0;
      g.tok = at.i * block_tokens(a, p);
      for (int w = 0; w < 2; ++w) {
        const int lo = g.tok + w * a.half;
        g.n[w] = p.pair ? g.tiles : lo >= s.nq ? 0 : max(0, min(k1, tiles_of(a, s, lo + a.half)) - k0);
      }
      g.own = max(0, min(s.ta - k0, g.tiles));
      g.first = k0 * kT;
      g.left = n - k0 * kT;
      g.part = n < s.ta * kT && s.ta > k0 && s.ta <= k1 ? s.ta - 1 - k0 : -1;
      g.gap = e < 0 ? -1 : e - k0 * kT;
      g.hole = e >= 0 && g.gap >= 0 && g.gap < g.own * kT ? g.gap / kT : -1;
      g.turn = e < 0 ? kNever : max(0, g.gap + 1) / kT;
      g.kb = k0 - s.ta;
      g.mask = a.parents ? g.own : max(g.own, (g.tok + 1) / kT - g.kb);
      g.tok0 = s.tok0;
      g.nq = s.nq;
      g.whole = k0 == 0 && k1 == all;
      g.from_start = k0 == 0;
      at.k = k1;
      if (k1 == all) {
        at.k = 0;
        ++at.i;
        if (g.tok + block_tokens(a, p) >= s.nq) {
          at.i = 0;
          if (++at.h == a.heads) {
            at.h = 0;
            ++at.b;
          }
        }
      }
      return true;
    }
  }
};

template <int D, bool PAIR>
struct Geo {
  static constexpr int KH = D / 64;              // 128-byte halves of a row
  static constexpr int HALFB = kT * 128;         // one half tile, 16 KB
  static constexpr int TILEB = KH * HALFB;
  static constexpr int STAGES = 128 * 1024 / TILEB;
  static constexpr int CW = 32;                  // output columns staged at a time
  static constexpr int Q = 0, RING = 2 * TILEB, STAGE = RING + STAGES * TILEB;   // (PAIR: segments take turns with Q)
  static constexpr int BUFB = kT * CW * 2;       // a stream's staged outputs; two of them, but in PAIR
  static constexpr int ML = STAGE + 2 * (PAIR ? 1 : 2) * BUFB;   // PAIR: the streams' maxima and sums
  static constexpr int BARS = ML + (PAIR ? 2 * kT * 8 : 0);
  static constexpr int NBARS = 3 * STAGES + 13 + 2 * kSegs;
  static constexpr int SEGS = BARS + NBARS * 8 + 16 + kSegs * 4;
  static constexpr int ROWS = SEGS + kSegs * (int)sizeof(Seg);
  static constexpr int SMEM = ROWS + kT * 4 + 1024;   // slack to align to 1024 bytes
};

// The order in which a segment's key and value tiles are used, n of each: K0 V0 K1 V1 ..;
// PAIR, whose streams have a tile each under way, K0 K1 V0 K2 V1 ..
template <bool PAIR>
__device__ __forceinline__ int tile_at(int j, int n, bool& value) {
  if (!PAIR) {
    value = j & 1;
    return j >> 1;
  }
  value = j == 2 * n - 1 || (j && !(j & 1));
  return j == 2 * n - 1 ? n - 1 : value ? j / 2 - 1 : (j + 1) / 2;
}

// Whether the helper warps mend a tile before it is used: values that are not there, or
// that some rows do not see; keys that await their re-rotation.
__device__ __forceinline__ bool mends(const TokensArgs& a, const Seg& g, bool value, int i) {
  if (!value) return i >= g.turn && i < g.own;
  // (rows behind the tensor's last are zeros already)
  return i >= g.own ? i >= g.mask : i == g.hole || (i == g.part && (a.lens || a.pend));
}

// The low `left` of 32 bits.
__device__ __forceinline__ uint32_t low_bits(int left) { return left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1u; }

template <typename T, int D, bool PAIR, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tokens_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap omap, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                         const __grid_constant__ CUtensorMap knmap, const __grid_constant__ CUtensorMap vnmap,
                         const __grid_constant__ Params p) {
  using Gm = Geo<D, PAIR>;
  constexpr int NS = Gm::STAGES;
  constexpr int kRows = SPLIT ? kT / 2 : kT;         // query rows of a half block
  constexpr int KC = kRows;                          // keys of a tile that a softmax thread has
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Gm::BARS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Gm::BARS + Gm::NBARS * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* marks = reinterpret_cast<volatile int*>(tmem_slot + 4);   // segments with values that are not finite
  auto full = [&](int s) { return smem_addr(&bars[s]); };
  auto empty = [&](int s) { return smem_addr(&bars[NS + s]); };
  auto mended = [&](int s) { return smem_addr(&bars[2 * NS + s]); };
  auto s_full = [&](int w) { return smem_addr(&bars[3 * NS + w]); };
  auto o_done = [&](int w) { return smem_addr(&bars[3 * NS + 2 + w]); };
  // query blocks: of a stream; PAIR: of every other segment
  auto q_full = [&](int x) { return smem_addr(&bars[3 * NS + 4 + x]); };
  auto p_full = [&](int w, int c) { return smem_addr(&bars[3 * NS + 6 + 2 * w + c]); };   // halves of 64 keys
  auto q_free = [&](int x) { return smem_addr(&bars[3 * NS + 10 + x]); };
  const uint32_t drain = smem_addr(&bars[3 * NS + 12]);
  auto seg_full = [&](int i) { return smem_addr(&bars[3 * NS + 13 + i % kSegs]); };
  auto seg_empty = [&](int i) { return smem_addr(&bars[3 * NS + 13 + kSegs + i % kSegs]); };
  Seg* const segs = reinterpret_cast<Seg*>(smem + Gm::SEGS);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const TokensArgs& a = p.a;

  launch_dependents();
  if (tid == 0) {
#pragma unroll 1
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 3);          // the products, and either helper warp
      mbar_init(mended(s), 2);
    }
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {
      mbar_init(s_full(w), 1);
      mbar_init(o_done(w), 1);
      mbar_init(q_full(w), 1);
      mbar_init(q_free(w), 1);
      mbar_init(p_full(w, 0), 4);
      mbar_init(p_full(w, 1), 4);
    }
#pragma unroll 1
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(seg_full(i), 1);
      mbar_init(seg_empty(i), 11);     // all warps but the producer's
      marks[i] = -1;
    }
    mbar_init(drain, 1);               // abort path only
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == 1) tmem_alloc(smem_addr(tmem_slot), kTmem);
  // The query rows that no box brings are zeros: what lies there could send their warp the
  // way of logits that are not finite.
  for (int x = tid; x < 2 * Gm::KH * (kRows - a.N * a.half) * 8; x += kThreads) {
    const int c = x & 7, h = (x >> 3) % (2 * Gm::KH), r = a.N * a.half + (x >> 3) / (2 * Gm::KH);
    for (int s = 0; s < kT; s += kRows)
      *reinterpret_cast<uint4*>(smem + Gm::Q + h * Gm::HALFB + (s + r) * 128 + c * 16) = make_uint4(0, 0, 0, 0);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  // a half block's rows: token and query head
  uint32_t* const row_of = reinterpret_cast<uint32_t*>(smem + Gm::ROWS);
  if (warp >= 8) {
    const unsigned r = (tid - 256) % kRows, t = r / (unsigned)a.N;
    row_of[tid - 256] = t << 16 | (r - t * a.N);
  }
  // (where outputs are staged: the producer has its range before it tells of any block)
  int64_t* const sums_s = reinterpret_cast<int64_t*>(smem + Gm::STAGE);
  TokensAt* const ends_s = reinterpret_cast<TokensAt*>(sums_s + kThreads / 32 + kThreads);
  find_range(a, p.plan, sums_s, ends_s);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && !p.plan.whole) {
    p.first[blockIdx.x] = ends_s[0];
    if (blockIdx.x == gridDim.x - 1) p.first[gridDim.x] = ends_s[1];
  }
  const uint32_t tmem = *tmem_slot;
  // TMEM columns: O of stream w at 128 w, S (and P over it) at 256 + 128 w
  auto tm_o = [&](int w) { return tmem + (uint32_t)(kT * w); };
  auto tm_s = [&](int w) { return tmem + (uint32_t)(2 * kT + kT * w); };

  // The segments, in order: the producer finds one after the other; after the last comes
  // one of no tiles. After a wait that ran out (ok is false) the roles still go through
  // them, without work, so that the softmax warps come to every row.
  int seg = 0;
  bool ok = true;
  auto take = [&]() -> const Seg* {      // the next one, or null
    const uint32_t phase = (uint32_t)(seg / kSegs) & 1;
    if (ok) ok = wait_or_abort(seg_full(seg), phase, abort_flag, p.err);
    ok = __all_sync(~0u, ok);
    // (all lanes alike: the warp stays whole for the collective instructions behind this)
    if (!ok && !__all_sync(~0u, mbar_wait_bounded(seg_full(seg), phase))) return nullptr;
    __syncwarp();
    const Seg* g = &segs[seg % kSegs];
    return g->tiles ? g : nullptr;
  };
  auto give = [&] {                      // it is not needed any more
    __syncwarp();
    if (lane == 0) mbar_arrive(seg_empty(seg));
    ++seg;
  };
  // The launch's 384 x 168 registers, shared out anew: 4 warps of 120 and 8 of
  // 192 a thread, so that a softmax thread holds a row's 128 logits.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    if (warp == 0) {
      // ---------------------------------------------------------------- TMA producer
      int s = 0, held = 0;               // next stage, stages in flight (at most NS)
      uint32_t phase = 0;
      bool more = true, stall = p.stall && blockIdx.x == 0;   // test hook: CTA 0's first tile never comes
      Walk walk(ends_s);
      for (; more; ++seg) {
        Seg g;
        more = walk.next(a, p.plan, g);
        if (!more) g.tiles = 0;
        if (seg >= kSegs) {
          const uint32_t free = (uint32_t)(seg / kSegs - 1) & 1;
          if (ok) ok = wait_or_abort(seg_empty(seg), free, abort_flag, p.err);
          ok = __all_sync(~0u, ok);
          if (!ok && !__all_sync(~0u, mbar_wait_bounded(seg_empty(seg), free))) break;
        }
        if (lane == 0) {
          segs[seg % kSegs] = g;
          mbar_arrive(seg_full(seg));
        }
        if (lane == 0 && ok) {
          auto load = [&](bool value, int i) {
            if (held == NS && !wait_or_abort(empty(s), phase ^ 1, abort_flag, p.err)) return false;
            if (!stall) {
              mbar_expect_tx(full(s), Gm::TILEB);
              const bool own = i < g.own;
              const CUtensorMap* map = value ? (own ? &vmap : &vnmap) : (own ? &kmap : &knmap);
              const Coords& c = value ? (own ? p.at.v : p.at.vn) : (own ? p.at.k : p.at.kn);
              const int row = own ? g.first + i * kT : g.tok0 + (g.kb + i) * kT;
              for (int kh = 0; kh < Gm::KH; ++kh)
                tma_load_rows(base + Gm::RING + s * Gm::TILEB + kh * Gm::HALFB, map, c, kh * 64, row, g.kv, g.b, full(s));
            }
            stall = false;
            held = min(held + 1, NS);
            if (++s == NS) s = 0, phase ^= 1;
            return true;
          };
#pragma unroll 1
          for (int j = 0; j < 2 * g.tiles && ok; ++j) {
            bool value;
            const int i = tile_at<PAIR>(j, g.tiles, value);
            ok = load(value, i);
          }
        }
        ok = __shfl_sync(~0u, (int)ok, 0) != 0;
      }
      if (lane == 0 && *abort_flag)      // let copies in flight land before the CTA leaves
        for (int i = 0; i < held; ++i) {
          if (--s < 0) s = NS - 1, phase ^= 1;
          (void)mbar_wait_bounded(full(s), phase, 10000000ull);
        }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer
      constexpr uint32_t kIdS = f16_idesc<T>(kT, false), kIdO = f16_idesc<T>(D, true);
      // descriptors of the first query block and ring stage; an offset adds to the
      // address field, in 16-byte units
      const uint64_t qd = sw128_desc(base + Gm::Q), kd = sw128_desc(base + Gm::RING);
      const uint64_t vd = sw128_mn_desc(base + Gm::RING, Gm::HALFB);
      int next = 0;                      // ring stage and its phase
      uint32_t phase = 0, mend_phase = 0;   // (of each stage, a bit)
      uint32_t np = 0, nq = 0;           // phases of the weights, and (not PAIR) queries, of either stream: a bit each
      for (const Seg* sg; (sg = take()); give()) {
        if (!ok) continue;
        const Seg g = *sg;
        const int n = g.tiles;
        auto tile = [&](bool value, int i) -> int {   // the next ring stage, once its tile is there; -1 on abort
          const int s = next;
          bool here;
          if (__builtin_expect(mends(a, g, value, i), 0)) {
            here = wait_or_abort(mended(s), (mend_phase >> s) & 1, abort_flag, p.err);
            mend_phase ^= 1u << s;
          } else {
            here = wait_or_abort(full(s), phase, abort_flag, p.err);
          }
          if (++next == NS) next = 0, phase ^= 1;
          here = __all_sync(~0u, here);
          tc_fence_after();
          return here ? s : -1;
        };
        auto mma_s = [&](int w, int s) {
          if (elect_one()) {
            const uint64_t qa = qd + (uint64_t)((PAIR ? seg & 1 : w) * (Gm::TILEB >> 4)), kb = kd + (uint64_t)(s * (Gm::TILEB >> 4));
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = (uint64_t)(((kk >> 2) * Gm::HALFB + (kk & 3) * 32) >> 4);
              tc_mma_ss(tm_s(w), qa + off, kb + off, kIdS, kk > 0);
            }
            tc_commit(s_full(w));
          }
        };
        auto commit = [&](uint32_t bar) {
          if (elect_one()) tc_commit(bar);
        };
        // O_w += P_w V: P of keys 0..63 in S's columns 0..31, of keys 64..127 in
        // 64..95, the second parts (PAIR) 32 columns on
        auto mma_o = [&](int w, int s, bool first) {
          const uint64_t vb = vd + (uint64_t)(s * (Gm::TILEB >> 4));
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (!__all_sync(~0u, wait_or_abort(p_full(w, c), np >> w & 1, abort_flag, p.err))) return false;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int part = 0; part < (PAIR ? 2 : 1); ++part)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  tc_mma_ts(tm_o(w), tm_s(w) + (uint32_t)(c * 64 + kk * 8 + 32 * part),
                            vb + (uint64_t)((4 * c + kk) * (2048 >> 4)), kIdO, !(first && c + kk + part == 0));
            }
          }
          np ^= 1u << w;
          return true;
        };
        auto queries = [&](int x, uint32_t count) {
          const bool here = __all_sync(~0u, wait_or_abort(q_full(x), count & 1, abort_flag, p.err));
          tc_fence_after();
          return here;
        };
        // (one place for either product, in the code: instructions that are not in the
        // SM's cache cost more than the loops)
        if (PAIR) {
          if (!(ok = queries(seg & 1, (uint32_t)seg >> 1))) continue;
#pragma unroll 1
          for (int i = -2; i < n; ++i) {
            const int w = i & 1;
            if (i >= 0) {
              const int s = tile(true, i);
              if (!(ok = s >= 0) || !(ok = mma_o(w, s, i < 2))) break;
              commit(empty(s));
              if (i + 2 >= n) commit(o_done(w));
            }
            if (i + 2 < n) {
              const int s = tile(false, i + 2);
              if (!(ok = s >= 0)) break;
              mma_s(w, s);
              commit(empty(s));
              if (i + 3 == n) commit(q_free(seg & 1));
            }
          }
        } else {
          // (the softmax warps give the stages back)
#pragma unroll 1
          for (int i = -1; i < n && ok; ++i) {
            int s = 0, sk = 0;
            if (i >= 0 && !(ok = (s = tile(true, i)) >= 0)) break;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int nw = w ? g.n[1] : g.n[0];
              if (i >= 0 && i < nw && !(ok = mma_o(w, s, i == 0))) break;
              if (w == 0 && i + 1 < n && !(ok = (sk = tile(false, i + 1)) >= 0)) break;
              if (i + 1 < nw) {
                if (i < 0) {
                  if (!(ok = queries(w, nq >> w & 1))) break;
                  nq ^= 1u << w;
                }
                mma_s(w, sk);
                if (i + 2 == nw) commit(q_free(w));
              } else if (i + 1 == nw && i >= 0) {
                commit(o_done(w));
              }
            }
          }
        }
      }
    } else {
      // ---------------------------------------------------------------- queries, tile mending
      const int ht = (warp - 2) * 32 + lane;         // of 64 threads
      int next = 0;
      uint32_t phase = 0;
      int queries[2] = {0, 0};           // that either place has had
      // re-rotation: a thread has one 16-byte piece of a row's first half and its pair
      constexpr int PC = D / 16, PER = 64 / PC;      // pieces, rows at a time
      const int pc = ht % PC, pr = ht / PC;
      auto piece = [&](int s, int r, int c) {
        return reinterpret_cast<uint4*>(smem + Gm::RING + s * Gm::TILEB + (c >> 3) * Gm::HALFB + r * 128 + (((c ^ r) & 7) << 4));
      };
      for (const Seg* sg; (sg = take()); give()) {
        if (!ok) continue;
        const Seg g = *sg;
        // Queries set out when their place is free: when the last logits there are done,
        // while their softmax and the last products run.
#pragma unroll 1
        for (int w = 0; w < (PAIR ? 1 : 2); ++w) {
          if ((w ? g.n[1] : g.n[0]) == 0) continue;
          const int x = PAIR ? seg & 1 : w;
          const int had = x ? queries[1]++ : queries[0]++;
          if (had && !(ok = __all_sync(~0u, wait_or_abort(q_free(x), (had - 1) & 1, abort_flag, p.err)))) break;
          if (ht == 0) {
            mbar_expect_tx(q_full(x), (kT / kRows) * Gm::KH * 128 * a.N * a.half);
            for (int kh = 0; kh < Gm::KH; ++kh)
              for (int s = 0; s < kT; s += kRows)
                tma_load_rows(base + Gm::Q + x * Gm::TILEB + kh * Gm::HALFB + s * 128, &qmap, p.at.q, kh * 64,
                              g.tok0 + g.tok + w * a.half, g.h * a.N, g.b, q_full(x));
          }
        }
        auto visit = [&](bool value, int i) {
          const int s = next;
          const uint32_t ph = phase;
          if (++next == NS) next = 0, phase ^= 1;
          // (every tile is waited for, and given back: a phase's parity alone does not
          // tell a tile from the one two rounds of the ring before it)
          if (!__all_sync(~0u, wait_or_abort(full(s), ph, abort_flag, p.err))) return false;
          if (!mends(a, g, value, i)) {
            if (lane == 0) mbar_arrive(empty(s));
            return true;
          }
          const int left = max(0, min(kT, i < g.own ? g.left - i * kT : g.nq - (g.kb + i) * kT));
          if (!value) {
            if constexpr (std::is_same<T, __half>::value) {   // (a handle's rows)
              for (int r = max(0, g.gap + 1 - i * kT) + pr; r < left; r += PER)
                rotate_back(*piece(s, r, pc), *piece(s, r, pc + PC), a.rope_c + 8 * pc, a.rope_s + 8 * pc);
            }
          } else {
            for (int x = ht; x < (kT - left) * (D / 8); x += 64)
              *piece(s, left + x / (D / 8), x % (D / 8)) = make_uint4(0, 0, 0, 0);
            if (i == g.hole && ht < D / 8) *piece(s, g.gap - i * kT, ht) = make_uint4(0, 0, 0, 0);
            if (i >= g.own) {
              // (keys up to the block's first token all of its rows see)
              const int seen = a.parents ? 0 : max(0, g.tok + 1 - (g.kb + i) * kT) * (D / 8);
              uint32_t found = 0;
#pragma unroll 4
              for (int x = seen + ht; x < left * (D / 8); x += 64) {
                const uint4 v = *piece(s, x / (D / 8), x % (D / 8));
                found |= not_finite<T>(v.x) | not_finite<T>(v.y) | not_finite<T>(v.z) | not_finite<T>(v.w);
              }
              if (__any_sync(~0u, found != 0)) {
                for (int x = seen + ht; x < left * (D / 8); x += 64) {
                  uint4* at = piece(s, x / (D / 8), x % (D / 8));
                  const uint4 v = *at;
                  *at = make_uint4(drop_not_finite<T>(v.x), drop_not_finite<T>(v.y), drop_not_finite<T>(v.z),
                                   drop_not_finite<T>(v.w));
                }
                marks[seg % kSegs] = seg;
              }
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(mended(s));
            mbar_arrive(empty(s));
          }
          return true;
        };
#pragma unroll 1
        for (int j = 0; j < 2 * g.tiles && ok; ++j) {
          bool value;
          const int i = tile_at<PAIR>(j, g.tiles, value);
          ok = visit(value, i);
        }
      }
      if (ht == 0 && *abort_flag)        // let queries in flight land before the CTA leaves
        for (int x = 0; x < 2; ++x)
          if (queries[x]) (void)mbar_wait_bounded(q_full(x), (queries[x] - 1) & 1, 10000000ull);
    }
  } else {
    // ---------------------------------------------------------------- softmax warpgroups
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int w = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;          // query row of the stream = TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t ns = 0, no = 0;                         // logits tiles and finished outputs seen
    int ring = 0;                                    // stage of the segment's first tile
    // One stream (the second, where it has rows: it has every tile) gives the ring's stages
    // back. When it sees its logits of key tile i (the segment's tile 2 i), those keys have
    // been read, and the values of tile i - 1 (2 i - 1) by the products before. A commit by
    // the MMA warp for each would be one more stop in its stream of products; PAIR waits
    // for memory and wants its stages sooner.
    auto release = [&](int nth) {
      if (lane == 0 && (warp & 3) == 0) mbar_arrive(empty((ring + nth) % NS));
    };
    // this thread's row of a half block: a token's place in it and a query head
    const int share = row / kRows;                   // (SPLIT: 0 or 1, the keys that this thread has of the row's)
    const int row_t = (int)((unsigned)(row % kRows) / (unsigned)a.N), row_h = row % kRows - row_t * a.N;
    // a tree: the tokens that token t sees, as bits (warp-collective)
    auto seen_of = [&](const Seg& g, int t) {
      uint64_t anc[2];
      ancestors(a, g.b, g.nq, anc);
      const uint64_t m0 = __shfl_sync(~0u, anc[0], t & 31), m1 = __shfl_sync(~0u, anc[1], t & 31);
      return t < 32 ? m0 : m1;
    };
    for (const Seg* sg; (sg = take()); give()) {
      const Seg& g = *sg;
      const int n = g.n[w], part = g.part, hole = g.hole, mask = g.mask, tiles = g.tiles;
      const bool releases = !PAIR && (w == 1 ? n > 0 : g.n[1] == 0);
      const int tok = g.tok + (PAIR ? 0 : w * a.half), t = min(tok + row_t, g.nq - 1);
      const bool valid = row_t < a.half && tok + row_t < g.nq;
      float m = kNegInf, l = 0.f;
      bool begun = false;
      const uint32_t ts = tm_s(w) + lanes, to = tm_o(w) + lanes, tsv = ts + (SPLIT ? 64 * share : 0);
      for (int i = PAIR ? w : 0; i < n && ok; i += PAIR ? 2 : 1) {
        ok = __all_sync(~0u, wait_or_abort(s_full(w), ns & 1, abort_flag, p.err));
        if (!ok) break;
        ++ns;
        tc_fence_after();
        if (releases) {
          release(2 * i);
          if (i > 0) release(2 * i - 1);
        }
        // Which of the tile's keys the row sees: the first `left`, but for a cache's evicted
        // row, or an ancestor's bits.
        const bool ends = i == part || (i >= mask && !a.parents), bitwise = i == hole || (i >= mask && a.parents);
        int left = kT;
        if (ends) left = i == part ? g.left - i * kT : t + 1 - (g.kb + i) * kT;
        uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
        if constexpr (PAIR) {                        // masked in registers, below
          if (ends) {
#pragma unroll
            for (int x = 0; x < 4; ++x) see[x] = low_bits(left - 32 * x);
          }
          if (bitwise) {
            const uint64_t mm = i == hole ? 0 : seen_of(g, t);
            const int gap = g.gap - i * kT;
#pragma unroll
            for (int x = 0; x < 4; ++x)
              see[x] &= i == hole ? ~((gap >> 5) == x ? 1u << (gap & 31) : 0u) : x < 2 ? (uint32_t)(mm >> (32 * x)) : 0u;
          }
          if (SPLIT && share) {
            see[0] = see[2];
            see[1] = see[3];
          }
        } else {
          // Masked where the logits are, 16 TMEM columns at a time: selects over all of v, in
          // a row, are 6 KB of instructions that the SM's cache for them does not keep, nor
          // what is behind them (8 x 4096 tokens 855 us so, 815 thus; PAIR, which waits for
          // memory, is faster with the selects: 64 trees of 32 tokens on 1000 rows 73 | 83).
          if (ends) {
            const int lo = max(0, (int)__reduce_min_sync(~0u, left)), hi = __reduce_max_sync(~0u, left);   // of the warp's rows
#pragma unroll 1
            for (int c = lo / 16; c < KC / 16; ++c) {
              float x[16];
              uint32_t o[16];
              if (16 * c < hi) tmem_ld16(ts + 16 * c, x);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(16 * c + e < left ? x[e] : kNegInf);
              tmem_st16(ts + 16 * c, o);
            }
            tmem_st_wait();
          }
          if (bitwise) {
            const uint64_t mm = i == hole ? 0 : seen_of(g, t);
            const int gap = g.gap - i * kT;
#pragma unroll 1
            for (int c = 0; c < KC / 16; ++c) {
              const int c0 = 16 * c;
              const uint32_t bits = i == hole ? ~(gap >= c0 && gap < c0 + 16 ? 1u << (gap - c0) : 0u) : c0 < 64 ? (uint32_t)(mm >> c0) : 0u;
              if (__all_sync(~0u, (bits & 0xFFFFu) == 0xFFFFu)) continue;
              float x[16];
              uint32_t o[16];
              tmem_ld16(ts + c0, x);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint((bits >> e) & 1u ? x[e] : kNegInf);
              tmem_st16(ts + c0, o);
            }
            tmem_st_wait();
          }
        }
        float v[KC];
        auto load_logits = [&] {
          if constexpr (SPLIT) {
            tmem_ld64(tsv, v);
          } else {
            tmem_ld128(tsv, v);
          }
        };
        load_logits();
        if constexpr (PAIR) {
          if (ends || bitwise) {
#pragma unroll
            for (int e = 0; e < KC; ++e) v[e] = (see[e >> 5] >> (e & 31)) & 1u ? v[e] : kNegInf;
          }
        }
        // (a NaN stays in the maximum, so that one compare finds logits that are not finite)
        float m4[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) m4[x] = max_nan(v[x], v[4 + x], v[8 + x]);
#pragma unroll
        for (int e = 12; e < KC; e += 8)
#pragma unroll
          for (int x = 0; x < 4; ++x) m4[x] = e + 4 < KC ? max_nan(m4[x], v[e + x], v[e + 4 + x]) : max_nan(m4[x], v[e + x]);
        const float mx = max_nan(max_nan(m4[0], m4[1]), max_nan(m4[2], m4[3])) * a.scale2;
        // Rare: logits of NaN or +-inf, and a maximum so large that it is rounded by a half
        // or more, as its own logit need not be near it in the fused product and
        // difference below.
        const bool none = PAIR ? (see[0] | see[1] | (SPLIT ? 0u : see[2] | see[3])) == 0u : left <= 0;
        const bool odd = !none && !(fabsf(mx) < kFar), up = mx > m + (kLazy + kLift<T>);
        float nb = m == kNegInf ? 0.f : -m;          // masked: every weight 2^-inf = 0
        if (__any_sync(~0u, up || odd)) {
          const float nm = odd ? fmaxf(m, mx) : up ? mx - kLift<T> : m, f = nm == m ? 1.f : ex2(m - nm);
          m = nm;
          l *= f;
          if (begun) {
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              float x[16];
              uint32_t o[16];
              tmem_ld16(to + 16 * c, x);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(x[e] * f);
              tmem_st16(to + 16 * c, o);
            }
          }
          nb = m == kNegInf ? 0.f : -m;
          if (__builtin_expect(__any_sync(~0u, odd), 0)) {
            // the difference, of a product rounded as the maximum was, goes through the
            // fused product instead (in such rows alone: no row's bits depend on its neighbours)
            const float inv = 1.f / a.scale2;
#pragma unroll 1
            for (int c = 0; c < KC / 16; ++c) {
              float x[16];
              uint32_t o[16];
              const uint32_t bits = (c < 2 ? see[0] : c < 4 ? see[1] : c < 6 ? see[2] : see[3]) >> (16 * (c & 1));   // (TILES: all)
              tmem_ld16(tsv + 16 * c, x);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                o[e] = __float_as_uint(!((bits >> e) & 1u) ? kNegInf
                                       : odd ? __fadd_rn(__fmul_rn(x[e], a.scale2), nb) * inv : x[e]);
              tmem_st16(tsv + 16 * c, o);
            }
            tmem_st_wait();
            load_logits();
            if (odd) nb = 0.f;
          }
        }
        if (SPLIT) {
          // the other thread's keys: weights of 0 (O is as it is to be: their product reads and
          // writes it)
          uint32_t zero[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) zero[e] = 0u;
#pragma unroll
          for (int c = 0; c < 64; c += 16) tmem_st16(ts + 64 * (1 - share) + c, zero);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(w, 1 - share));
        }
        begun = true;
        const float2 sc2 = make_float2(a.scale2, a.scale2), nb2 = make_float2(nb, nb);
        float2 l4[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) l4[x] = make_float2(0.f, 0.f);
        // 64 keys at a time: the tensor cores start on the first half's weights
        // while the second half's are computed
#pragma unroll
        for (int c = 0; c < KC / 64; ++c) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const int k = 64 * c + 32 * h + e;
              const float2 x = ffma2(make_float2(v[k], v[k + 1]), sc2, nb2);
              const float2 pp = make_float2(ex2(x.x), ex2(x.y));
              l4[(e >> 1) & 3] = fadd2(l4[(e >> 1) & 3], pp);
              hi[e / 2] = pack16<T>(pp.x, pp.y);
              if (PAIR) {
                const float2 back = unpack16<T>(hi[e / 2]);
                lo[e / 2] = pack16<T>(pp.x - back.x, pp.y - back.y);
              }
            }
            tmem_st16(tsv + 64 * c + 16 * h, hi);
            if (PAIR) tmem_st16(tsv + 64 * c + 32 + 16 * h, lo);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(w, SPLIT ? share : c));
        }
        l4[0] = fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3]));
        l += l4[0].x + l4[0].y;
      }
      if (begun && ok) {
        ok = __all_sync(~0u, wait_or_abort(o_done(w), no & 1, abort_flag, p.err));
        ++no;
        tc_fence_after();
        if (releases) release(2 * n - 1);
      }
      ring = (ring + 2 * tiles) % NS;
      // (all lanes alike, as the accumulators' loads want it. The mark may be on its way for a tile
      // that only the second half of the block visits: either answer gives these rows the same sums.)
      const bool poisoned = __any_sync(~0u, marks[seg % kSegs] == seg);
      if (__builtin_expect(poisoned && begun, 0)) {
        // values that are not finite, dropped from the tiles that rows see in part
        const uint64_t seen = a.parents ? seen_of(g, t) : 0;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float x[16];
          tmem_ld16(to + c, x);
#pragma unroll 1
          for (int j = a.parents ? max(0, g.kb) * kT : max((g.kb + g.own) * kT, g.tok + 1); j < min((g.kb + g.tiles) * kT, t + 1); ++j) {
            // (PAIR: of this stream's tiles)
            if ((a.parents && !((seen >> j) & 1)) || (PAIR && ((j / kT - g.kb) & 1) != w)) continue;
            const T* src = static_cast<const T*>(a.v_new) + g.b * a.vn_stride[0] + (int64_t)(g.tok0 + j) * a.vn_stride[1] +
                           g.kv * a.vn_stride[2] + c;
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const uint32_t word = *reinterpret_cast<const uint32_t*>(src + e), f = not_finite<T>(word);
              const float2 y = unpack16<T>(word);
              if (f & 0x8000u) x[e] += y.x;
              if (f & 0x80000000u) x[e + 1] += y.y;
            }
          }
          uint32_t o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(x[e]);
          tmem_st16(to + c, o);
        }
        tmem_st_wait();
      }
      float f0 = 1.f, f1 = 0.f;
      if (!ok) l = __int_as_float(0x7FFFFFFF);       // NaN: this row's result is lost
      if (PAIR) {
        // the two streams' maxima and sums meet in shared memory, their O in the
        // registers of whichever warpgroup writes the columns: a warp of either
        // reaches the same TMEM lanes
        float2* ml = reinterpret_cast<float2*>(smem + Gm::ML);
        ml[w * kT + row] = make_float2(m, l);
        tc_fence_before();
        asm volatile("bar.sync 3, 256;" ::: "memory");
        tc_fence_after();
        const float2 x = ml[row], y = ml[kT + row];
        m = fmaxf(x.x, y.x);
        if (SPLIT) m = fmaxf(m, fmaxf(ml[row ^ 64].x, ml[kT + (row ^ 64)].x));
        f0 = x.x == m ? 1.f : ex2(x.x - m);
        f1 = y.x == m ? 1.f : ex2(y.x - m);
        l = x.y * f0 + y.y * f1;
        if (SPLIT) {
          const float2 z = ml[row ^ 64], u = ml[kT + (row ^ 64)];
          l += z.y * (z.x == m ? 1.f : ex2(z.x - m)) + u.y * (u.x == m ? 1.f : ex2(u.x - m));
        }
      }
      constexpr int CW = Gm::CW;
      auto columns = [&](int c, float (&v)[CW]) {    // O's columns c .. c + CW - 1 of this row
        const uint32_t at = tmem + lanes + c;
        if (n == 0) {
#pragma unroll
          for (int e = 0; e < CW; ++e) v[e] = 0.f;
        } else if constexpr (!PAIR) {
          tmem_ld32(at + kT * w, v);
        } else {
          tmem_ld32(at, v);
          if (n > 1) {
            float y[32];
            tmem_ld32(at + kT, y);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = fmaf(y[e], f1, v[e] * f0);
          } else if (SPLIT) {                        // (the other share's maximum may be larger)
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= f0;
          }
        }
      };
      // SPLIT: the second thread of a row hands its part of O to the first, 32 columns at a
      // time: [piece of 4 columns][row]
      float4* const halves = reinterpret_cast<float4*>(smem + Gm::STAGE + w * (64 * 32 * 4));
      auto join_shares = [&](float (&v)[CW]) {
        if (share) {
#pragma unroll
          for (int e = 0; e < CW; e += 4) halves[(e / 4) * 64 + row % kRows] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
        asm volatile("bar.sync %0, 128;" ::"r"(4 + w) : "memory");
        if (!share) {
#pragma unroll
          for (int e = 0; e < CW; e += 4) {
            const float4 y = halves[(e / 4) * 64 + row];
            v[e] += y.x;
            v[e + 1] += y.y;
            v[e + 2] += y.z;
            v[e + 3] += y.w;
          }
        }
        asm volatile("bar.sync %0, 128;" ::"r"(4 + w) : "memory");
      };
      constexpr int COLS = PAIR ? D / 2 : D;         // this warpgroup's columns, from `begin` on
      const int begin = PAIR ? w * COLS : 0;
      if (g.whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float2 inv2 = make_float2(inv, inv);
        constexpr int PR = CW / 8;                   // 16-byte pieces of a row
        unsigned char* stage = smem + Gm::STAGE + w * (PAIR ? 1 : 2) * Gm::BUFB;   // [row][64 bytes], as TMA swizzles them
        auto staged = [&](int r, int c) {
          return reinterpret_cast<uint4*>(stage + r * (CW * 2) + (((c ^ (r >> 1)) & (PR - 1)) << 4));
        };
        T* const out = static_cast<T*>(a.out) + g.b * a.out_stride[0] + (int64_t)(g.tok0 + tok) * a.out_stride[1] +
                       (int64_t)g.h * a.N * a.out_stride[2];
        const unsigned rows_on = __ballot_sync(~0u, valid);
        // Half blocks whose tokens are all there go out by TMA, 32 columns at a time from two
        // buffers in turn; others row by row.
        const bool box = !PAIR && p.out_box && tok + a.half <= g.nq, first = (warp & 3) == 0 && lane == 0;
        if (!PAIR && !box) {                         // the last box has been read
          if (first) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          asm volatile("bar.sync %0, 128;" ::"r"(1 + w) : "memory");
        }
#pragma unroll 1
        for (int c0 = begin; c0 < begin + COLS; c0 += CW) {
          float v[CW];
          columns(c0, v);
          if constexpr (SPLIT) {
            // few rows, straight from the registers
            join_shares(v);
            T* const dst = out + row_t * a.out_stride[1] + row_h * a.out_stride[2] + c0;
            if (valid && !share) {
#pragma unroll
              for (int e = 0; e < CW; e += 8)
                *reinterpret_cast<uint4*>(dst + e) =
                    make_uint4(pack16<T>(v[e] * inv, v[e + 1] * inv), pack16<T>(v[e + 2] * inv, v[e + 3] * inv),
                               pack16<T>(v[e + 4] * inv, v[e + 5] * inv), pack16<T>(v[e + 6] * inv, v[e + 7] * inv));
            }
            continue;
          }
          if (!PAIR && box && c0 != CW) {            // the buffer's last box has been read
            if (first) {
              if (c0 == 0)
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
              else
                asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            }
            asm volatile("bar.sync %0, 128;" ::"r"(1 + w) : "memory");
          }
#pragma unroll
          for (int e = 0; e < CW; e += 8) {
            uint32_t o[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float2 y = fmul2(make_float2(v[e + 2 * x], v[e + 2 * x + 1]), inv2);
              o[x] = pack16<T>(y.x, y.y);
            }
            *staged(row, e / 8) = make_uint4(o[0], o[1], o[2], o[3]);
          }
          if (box) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            asm volatile("bar.sync %0, 128;" ::"r"(1 + w) : "memory");
            if (first) {
              asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                               reinterpret_cast<uint64_t>(&omap)),
                           "r"(c0), "r"(g.h * a.N), "r"(g.tok0 + tok), "r"(a.starts ? 0 : g.b), "r"(smem_addr(stage))
                           : "memory");
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            stage = smem + Gm::STAGE + 2 * w * Gm::BUFB + (stage == smem + Gm::STAGE + 2 * w * Gm::BUFB ? Gm::BUFB : 0);
          } else {
            __syncwarp();
            uint4 y[PR];
#pragma unroll
            for (int x = 0; x < PR; ++x) y[x] = *staged((warp & 3) * 32 + x * (32 / PR) + lane / PR, lane % PR);
#pragma unroll
            for (int x = 0; x < PR; ++x) {
              const int r = x * (32 / PR) + lane / PR;
              const uint32_t th = row_of[(warp & 3) * 32 + r];
              if ((rows_on >> r) & 1u)
                *reinterpret_cast<uint4*>(out + (th >> 16) * a.out_stride[1] + (th & 0xFFFFu) * a.out_stride[2] + c0 + 8 * (lane % PR)) = y[x];
            }
            __syncwarp();
          }
        }
        if (valid && a.lse && !(PAIR && w) && !share)
          a.lse[((a.starts ? (int64_t)g.tok0 : (int64_t)g.b * a.S) + t) * a.G + g.h * a.N + row_h] =
              l == 0.f ? kNegInf : (m + log2f(l)) * 0.69314718055994531f;
      } else {
        const int64_t slot = 2 * blockIdx.x + g.from_start;
        const int R = p.plan.block_rows, rr = (PAIR ? 0 : w * kT) + row;
        float4* o = reinterpret_cast<float4*>(p.part_o) + slot * (R * (D / 4)) + rr;
#pragma unroll 1
        for (int c0 = begin; c0 < begin + COLS; c0 += CW) {
          float v[CW];
          columns(c0, v);
          if constexpr (SPLIT) join_shares(v);
#pragma unroll
          for (int e = 0; e < CW; e += 4)
            if (valid && !share) o[(int64_t)((c0 + e) / 4) * R] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
        if (!(PAIR && w) && !share) p.part_ml[slot * R + rr] = make_float2(m, l);
      }
      tc_fence_before();
      // (PAIR: either warpgroup reads both accumulators, and the maxima)
      if (PAIR) asm volatile("bar.sync 3, 256;" ::: "memory");
    }
  }

  if (!PAIR) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");   // outputs on their way
  // -------------------------------------------------------------------- teardown
  __syncthreads();
  if (*abort_flag && tid == 32) {
    // let any MMA still in flight finish before the accumulators are freed
    tc_commit(drain);
    (void)mbar_wait_bounded(drain, 0, 10000000ull);
  }
  __syncwarp();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
}

// Joins the parts of cut blocks: grid (boundary between CTAs, 32 rows of the block, 32
// columns), where the first boundary inside a block takes it. A lane is a row, a warp
// four columns, and a block's parts follow one another: few of them where there are many
// blocks; one block over all SMs has up to one an SM, 0.37 us each (16 tokens of 4 query heads on
// one key head of 16384 rows: 62 us in all, 8 key heads 30).
template <typename T, int D>
__global__ void __launch_bounds__(256) tokens_join_kernel(const __grid_constant__ Params p) {
  const TokensArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, R = p.plan.block_rows;
  const int rr = blockIdx.y * 32 + lane, d4 = blockIdx.z * 8 + warp, c0 = blockIdx.x;
  wait_for_primary();                        // in every block: this kernel ends after the one before it
  const TokensAt x = p.first[c0 + 1], y = p.first[c0];
  auto same = [&](const TokensAt& o) { return o.b == x.b && o.h == x.h && o.i == x.i; };
  if (x.b >= a.B || x.k == 0 || (same(y) && y.k > 0)) return;
  const Seq s = load_seq(a, x.b);
  const int r = rr & (kT - 1), rt = (int)((unsigned)r / (unsigned)a.N), head = x.h * a.N + r - rt * a.N;
  const int t = x.i * block_tokens(a, p.plan) + (rr / kT) * a.half + rt;
  if (rt >= a.half || t >= s.nq) return;
  // a range that begins where the next one does is empty and has left no part
  float m = kNegInf, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  TokensAt at = y, to = x;
  for (int c = c0;; ++c) {
    if (c > c0) {
      at = to;
      if (c == p.plan.ctas || !same(at)) break;
      to = p.first[c + 1];
    }
    if (same(to) && to.k <= at.k && c > c0) continue;
    const int64_t slot = 2 * c + (c == c0);
    const float2 ml = p.part_ml[slot * R + rr];
    const float4 v = reinterpret_cast<const float4*>(p.part_o)[slot * (R * (D / 4)) + (int64_t)d4 * R + rr];
    const float nm = fmaxf(m, ml.x), f = m == nm ? 1.f : ex2(m - nm), h = ml.x == nm ? 1.f : ex2(ml.x - nm);
    m = nm;
    l = l * f + ml.y * h;
    o = make_float4(o.x * f + v.x * h, o.y * f + v.y * h, o.z * f + v.z * h, o.w * f + v.w * h);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* dst = static_cast<T*>(a.out) + x.b * a.out_stride[0] + (int64_t)(s.tok0 + t) * a.out_stride[1] + head * a.out_stride[2] + 4 * d4;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack16<T>(o.x * inv, o.y * inv), pack16<T>(o.z * inv, o.w * inv));
  if (d4 == 0 && a.lse)
    a.lse[((a.starts ? (int64_t)s.tok0 : (int64_t)x.b * a.S) + t) * a.G + head] =
        l == 0.f ? kNegInf : (m + log2f(l)) * 0.69314718055994531f;
}

template <typename Elem, int Dim, bool Pair, bool Split>
struct Kind {
  using T = Elem;
  static constexpr int D = Dim, SMEM = Geo<Dim, Pair>::SMEM;
  static_assert(SMEM <= 227 * 1024, "shared memory of a block");
  static constexpr auto kernel = attend_tokens_kernel<Elem, Dim, Pair, Split>;
};
template <typename Elem, typename F>
auto pick_shape(int D, const TokensPlan& p, F&& f) {
  if (D == 64) return p.split ? f(Kind<Elem, 64, true, true>{}) : p.pair ? f(Kind<Elem, 64, true, false>{}) : f(Kind<Elem, 64, false, false>{});
  return p.split ? f(Kind<Elem, 128, true, true>{}) : p.pair ? f(Kind<Elem, 128, true, false>{}) : f(Kind<Elem, 128, false, false>{});
}
template <typename F>
auto pick(int D, int dtype, const TokensPlan& p, F&& f) {
  return dtype == kBf16 ? pick_shape<__nv_bfloat16>(D, p, f) : pick_shape<__half>(D, p, f);
}

std::atomic<bool> g_off{false};   // test hook

// Rows as a 4-D tensor [sequence, row, head, D], whatever the strides (a dimension of one
// entry, or that all share, with any); boxes of 64 elements (128 bytes), or 32, of so many
// heads and rows; rows past the last read as zeros.
bool encode_rows(CUtensorMap* map, const TokensRows& r, int heads, int rows, int D, int dtype, Coords* c, int cols = 64) {
  auto enc = encode_fn();
  if (!enc) return false;
  c->h = r.H > 1 && r.stride[1] != 0;
  c->b = r.B > 1 && r.stride[0] != 0;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)(c->h ? r.H : 1), (cuuint64_t)r.rows, (cuuint64_t)(c->b ? r.B : 1)};
  const cuuint64_t strides[3] = {(cuuint64_t)(c->h ? r.stride[1] : D) * 2, (cuuint64_t)(r.rows > 1 ? r.stride[2] : D) * 2,
                                 (cuuint64_t)(c->b ? r.stride[0] : D) * 2};
  const cuuint32_t box[4] = {(cuuint32_t)cols, (cuuint32_t)heads, (cuuint32_t)rows, 1}, estr[4] = {1, 1, 1, 1};
  return enc(map, dtype == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
             const_cast<void*>(r.base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

TokensPlan tokens_plan(bool pair, bool split, int64_t blocks, int heads, int64_t tiles, int64_t mean, int sms) {
  TokensPlan pl{};
  pl.pair = pair;
  pl.split = split;
  pl.block_rows = pl.pair ? kT : 2 * kT;
  const int64_t units = blocks * heads;
  // Cut blocks cost their parts' way through memory and the join, about nine tiles' time;
  // whole ones leave CTAs with less than others: 32 query heads on 8 of 1024 tokens 20.9 us
  // whole, 33.8 cut, of 2048 60.3 and 55.7; 2 x 40 drafted tokens on 1500 rows 28.3 and 21.5.
  const double even = (double)units * (double)mean / sms;
  pl.whole = tiles <= 6 || (units <= sms ? (double)tiles : even + 0.6 * (double)tiles) < even + 9;
  pl.even = pl.whole && units <= sms;
  // (a tile's time is that of 256 query rows at D = 64, between the others' 0.9 to 1.6 us; a cut
  // call's parts are charged as if there were few, too little for one block over all SMs)
  pl.us = 7 + 1.3 * (pl.even ? (double)tiles : pl.whole ? even + 0.6 * (double)tiles : even + 8);
  pl.ctas = (int)std::min<int64_t>(sms, pl.whole || units >= sms ? units : units * tiles);
  pl.per_cta = 1.0 / pl.ctas;
  return pl;
}

bool tokens_kernel_ready(int D, int dtype, const TokensPlan& plan, int device) {
  if (g_off.load(std::memory_order_relaxed) || !encode_fn()) return false;
  return pick(D, dtype, plan, [&](auto kind) {
    using K = decltype(kind);
    // The kernel's redistribution of registers needs the 168 a thread that its
    // launch bound gives it: checked, as it would wait forever with fewer.
    static std::atomic<uint64_t> ready{0};   // devices on which that, and its shared memory, are settled
    const uint64_t bit = 1ull << device;
    if (ready.load(std::memory_order_relaxed) & bit) return true;
    cudaFuncAttributes f;
    if (cudaFuncGetAttributes(&f, K::kernel) != cudaSuccess || f.numRegs != 168 ||
        cudaFuncSetAttribute(K::kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, K::SMEM) != cudaSuccess) {
      (void)cudaGetLastError();
      return false;
    }
    ready.fetch_or(bit, std::memory_order_relaxed);
    return true;
  });
}

void tokens_kernel_off(bool off) { g_off.store(off); }

cudaError_t launch_attend_tokens(const TokensLaunch& l, int D, int dtype, cudaStream_t s) {
  Params p{};
  p.a = l.a;
  p.plan = l.plan;
  p.err = l.err;
  p.stall = l.stall;
  if (!l.plan.whole) {
    char* space = static_cast<char*>(l.workspace);
    p.part_o = reinterpret_cast<float*>(space);
    p.part_ml = reinterpret_cast<float2*>(space + l.plan.o_bytes(D));
    p.first = reinterpret_cast<TokensAt*>(space + l.plan.o_bytes(D) + l.plan.ml_bytes());
  }
  CUtensorMap qmap{}, omap{}, kmap{}, vmap{}, knmap{}, vnmap{};
  if (!encode_rows(&qmap, l.q, l.a.N, l.a.half, D, dtype, &p.at.q) || !encode_rows(&knmap, l.k_new, 1, kT, D, dtype, &p.at.kn) ||
      !encode_rows(&vnmap, l.v_new, 1, kT, D, dtype, &p.at.vn))
    return cudaErrorInvalidValue;
  // (outputs have any strides: those that no map describes are stored row by row)
  Coords none;
  p.out_box = !l.plan.pair && l.out_fits && encode_rows(&omap, l.out, l.a.N, l.a.half, D, dtype, &none, 32);
  if (l.a.n + (l.a.pend ? 1 : 0) > 0 &&
      (!encode_rows(&kmap, l.k, 1, kT, D, dtype, &p.at.k) || !encode_rows(&vmap, l.v, 1, kT, D, dtype, &p.at.v)))
    return cudaErrorInvalidValue;
  return pick(D, dtype, l.plan, [&](auto kind) {
    using K = decltype(kind);
    K::kernel<<<l.plan.ctas, kThreads, K::SMEM, s>>>(qmap, omap, kmap, vmap, knmap, vnmap, p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || l.plan.whole || l.plan.ctas < 2) return e;
    const dim3 grid(l.plan.ctas - 1, l.plan.block_rows / 32, K::D / 32);
    return launch_after(tokens_join_kernel<typename K::T, K::D>, grid, 256, 0, 1, true, s, p);
  });
}

}  // namespace kvx
