// attend_rows.cu -- attention of one query token per sequence over key and
// value rows: the sequence's own (a cache layer's kept rows, or rows that the
// caller lays out), rows that all sequences share, and the token's own key and
// value.
//
//   s_j = q . k_j * scale;  out = sum_j e^(s_j) v_j / sum_j e^(s_j);
//   lse = log sum_j e^(s_j);  no rows at all: out = 0, lse = -inf
//
// Bound by memory: each key and value row is used for the N = G / H query
// heads of its key head only. So no shared-memory stage stands between HBM
// and the matrix instructions: every lane loads 16-byte pieces of the rows
// straight into the registers that mma.m16n8k16 wants them in.
//   logits: A = queries (rows: up to 16 heads), B = keys. The contraction may
//     run over the head dimension in any order, so a lane's 16-byte piece of a
//     key serves as two k-steps' B registers, with the queries loaded in the
//     same order.
//   output (transposed): A = values, B = weights. Two keys' values at one d
//     share a register, so the lane that holds both keys' pieces interleaves
//     them with one byte permute each; the weights are the logits' accumulator
//     registers as they are.
// A warp takes 16 rows at a time, 32 in a stream with up to 8 query heads. Its key
// registers are refilled as soon as the logits are out of them, its value registers
// as soon as the sums are, so one of the two is always in flight. Running maximum,
// sum and output stay in fp32 registers; the maximum is looked at again only when
// some lane exceeds it.
//
// The weights go into the second product as a sum of two 16-bit parts
// (p = hi + lo): the matrix pipe has room for the second instruction here, and the
// output keeps the accuracy of its own rounding. In bf16 that is 16 bits of every
// weight. fp16's smallest step is 2^-24, so its weights, at most 1, go in times 2^15
// (and out again, both exact): 22 bits down to 2^-17 of the largest weight, and steps
// of 2^-39 of it below, which leave a tail of a million rows its sum.
//
// Work: a unit is a sequence's key head with up to 16 of its query heads.
//   Few tiles (a latency, mostly): one cluster of CTAs a unit, its tiles dealt to
//     the cluster's warps, the sums joined through distributed shared memory; one
//     launch, no workspace.
//   Many (STREAM): all units' tiles in a row are cut into one contiguous range per
//     resident CTA, so that no SM waits for another whatever the lengths are. A
//     unit that is one CTA's alone is written out by it, a cut one leaves its
//     parts in the workspace for a second, small kernel, which joins them in a
//     fixed order, with the shared prefix's parts if there are any.
//
// Measured on GB300 (D = 128, 32 query heads on 8, fp16): 32 sequences of 2048 rows
// 44-46 us, 5.8-6.1 TB/s of rows (0.88 of the measured copy rate), 64 of them 80 us, 6.7
// TB/s; 7 unequal ones of up to 65521 rows 139-142 us, 6.0 TB/s; one of 512 rows 5-6 us,
// all latency. A cache's rows 46-47 us for the same 32 x 2048, 51 us with a compaction
// pending (its rows re-rotated on the way). Tried and slower: the tiles through shared memory by cp.async, two more in
// flight (63 against 50 us), 32-byte loads (53 against 50), more and smaller ranges
// (54-59), L2 prefetches throughout (150 against 139 on the unequal lengths). Bound by
// the loads that a warp's registers hold in flight, 16 KB, 8 warps an SM, with the
// latencies of start, join and unequal SMs on top (SMs are busy 84% of the time).
#include "attend_internal.cuh"

#include <cooperative_groups.h>

#include <type_traits>

namespace kvx {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kNegInf = -__builtin_huge_valf();
// A stream from this many tiles of 16 rows a warp on; beside a prefix from fewer,
// as a cluster that has its sums would wait for the prefix's parts.
constexpr int kStreamTiles = 8, kBesideTiles = 1;
// A stream too where a cluster's warps would have this many tiles each: few, long
// units that a cluster cannot spread over the GPU.
constexpr int kClusterTiles = 8;
// Parts of a head that one warp joins, with many heads (half as many with few): 32
// sequences of 1024 rows 24.8 us, 28.3 with eight warps a head; 2 of 4096, 40 parts,
// 10.0 with eight, 11.5 with one.
constexpr int kFewParts = 32;

// What the weights of the second product are multiplied by: the top of fp16's range
// (65504) is used, with a factor of two to spare.
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 32768.f : 1.f;

constexpr int stream_ctas_per_sm(int D) { return D == 64 ? 3 : 2; }
int rows_qt(int N) { return N <= 8 ? 1 : 2; }
// Rows a warp takes at a time: 32 where a stream's registers hold them.
constexpr int tile_rows(int qt, bool stream) { return stream && qt == 1 ? 32 : 16; }
// CTAs of a unit's cluster: its tiles are split while all CTAs are resident
// together (two an SM: a second wave costs the call's latency again, 8 sequences of
// 512 rows 7.9 us against 11) and a warp has more than one tile.
int cluster_ctas(int64_t units, int64_t tiles, int sms) {
  int C = 1;
  while (C < 8 && units * C <= sms && (int64_t)C * kWarps < tiles) C *= 2;
  return C;
}
int64_t rows_tiles(int rows, int n, int P, bool has_new, bool pend) {   // of a unit, at most
  return ((int64_t)P + rows - 1) / rows + ((int64_t)n + pend + rows - 1) / rows + has_new;
}

template <typename T>
__device__ __forceinline__ void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// 16 KG consecutive rows of one source; row r is there if bit r of `live` is set.
template <typename T>
struct Tile {
  const T* k;
  const T* v;
  int64_t ks, vs;
  uint32_t live;
  int moved;    // rows from here on await the re-rotation by -1 (32: none)
};

template <typename T, int D, int KG>
struct Rows {
  static constexpr int KC = D / 32;   // 16-byte pieces of a key row in one lane
  static constexpr int VH = D / 64;   // 64-wide column groups of a value row

  __device__ __forceinline__ static void load_k(uint4 (&kr)[2 * KG][KC], const Tile<T>& t, int g, int c) {
#pragma unroll
    for (int nt = 0; nt < 2 * KG; ++nt) {
      const int r = g + 8 * nt;
      const T* p = t.k + (int64_t)r * t.ks + 8 * c;
      const bool on = (t.live >> r) & 1u;
#pragma unroll
      for (int i = 0; i < KC; ++i) kr[nt][i] = on ? ld_stream16(p + 32 * i) : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ static void load_v(uint4 (&vr)[VH][4 * KG], const Tile<T>& t, int g, int c) {
#pragma unroll
    for (int j = 0; j < 4 * KG; ++j) {
      const int r = 2 * c + (j & 1) + 8 * (j >> 1);
      const T* p = t.v + (int64_t)r * t.vs + 8 * g;
      const bool on = (t.live >> r) & 1u;
#pragma unroll
      for (int h = 0; h < VH; ++h) vr[h][j] = on ? ld_stream16(p + 64 * h) : make_uint4(0, 0, 0, 0);
    }
  }
};

// Starts a tile towards L2 (rows that lie together only). Used for a range's
// second tile, whose loads the registers cannot yet take; for every tile it
// costs more than it hides (7 ragged sequences of up to 65521 rows: 138 us so,
// 150 us prefetching throughout, 139 us not at all).
template <typename T, int D>
__device__ __forceinline__ void prefetch_tile(const Tile<T>& t, int lane) {
  const int rows = 32 - __clz(t.live);           // up to the last one that is there
  if (t.ks == D && t.vs == D && lane < 2 && rows)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(lane ? t.v : t.k), "r"(rows * D * 2) : "memory");
}

// A cache key whose compaction is pending: rotated by -1 position, every
// product and sum rounded to fp32, then to fp16, as the step kernel and the
// flush do it, so the logits see the very key the cache will hold. lo and hi
// are the pieces with elements i and i + D/2.
__device__ __forceinline__ void rotate_back(uint4& lo, uint4& hi, const float* rc, const float* rs) {
  uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack16<__half>(a[i]), y = unpack16<__half>(b[i]);
    const float2 c = *reinterpret_cast<const float2*>(rc + 2 * i), s = *reinterpret_cast<const float2*>(rs + 2 * i);
    a[i] = pack16<__half>(__fsub_rn(__fmul_rn(x.x, c.x), __fmul_rn(y.x, s.x)),
                          __fsub_rn(__fmul_rn(x.y, c.y), __fmul_rn(y.y, s.y)));
    b[i] = pack16<__half>(__fadd_rn(__fmul_rn(x.x, s.x), __fmul_rn(y.x, c.x)),
                          __fadd_rn(__fmul_rn(x.y, s.y), __fmul_rn(y.y, c.y)));
  }
  lo = make_uint4(a[0], a[1], a[2], a[3]);
  hi = make_uint4(b[0], b[1], b[2], b[3]);
}

// Columns d .. d + 3 of query head gq from its sums, and the head's log sum.
template <typename T>
__device__ __forceinline__ void write_out(const AttendArgs& a, int b, int gq, int d, float m, float l, float4 o) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* dst = static_cast<T*>(a.out) + b * a.out_stride[0] + (int64_t)gq * a.out_stride[1] + d;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack16<T>(o.x * inv, o.y * inv), pack16<T>(o.z * inv, o.w * inv));
  if (d == 0 && a.lse) a.lse[(int64_t)b * a.G + gq] = l == 0.f ? kNegInf : (m + log2f(l)) * 0.69314718055994531f;
}

// Rows of sequence b: shared (np) and own (n), and the tiles of TR that they make.
template <int TR>
struct SeqRows {
  int np, n, tp, to;
  __device__ __forceinline__ SeqRows(const AttendArgs& a, int b) {
    np = a.plens ? max(0, min(a.plens[b], a.P)) : a.P;
    n = a.lens ? max(0, min(a.lens[b], a.n)) : a.n;
    tp = (np + TR - 1) / TR;
    to = (n + (a.pend ? 1 : 0) + TR - 1) / TR;   // an evicted row may still be in place
  }
  // of a unit; in a stream every unit has at least one
  __device__ __forceinline__ int tiles(const AttendArgs& a) const { return tp + to + (a.k_new ? 1 : 0); }
};
template <int TR>
__device__ __forceinline__ int stream_tiles(const AttendArgs& a, int b) {
  return max(1, SeqRows<TR>(a, b).tiles(a));
}

// Where sequences lie in the row of all units' tiles. With unequal lengths the
// stream kernel finds that out and leaves it in the workspace for the join: the
// first tile of every sequence, and the total after them.
struct Stream {
  int64_t total;
  int ctas;                                   // that have work: never more than there are tiles
  __device__ __forceinline__ Stream(int64_t tiles, const RowsPlan& plan)
      : total(tiles), ctas((int)min((int64_t)plan.ctas, tiles)) {}
  __device__ __forceinline__ int64_t start(int c) const { return c * total / ctas; }
  __device__ __forceinline__ int cta_of(int64_t x) const { return (int)(((x + 1) * ctas - 1) / total); }
};
__device__ __forceinline__ bool even_lengths(const AttendArgs& a) { return !a.lens && !a.plens; }

// For a CTA of the stream: the sequence that its first tile belongs to (b) and
// that sequence's first tile (base). All threads take a share of the sequences;
// sums_s: [kThreads].
template <int TR>
__device__ __forceinline__ Stream find_range(const AttendArgs& a, const RowsPlan& plan, int64_t* sums_s, int& b,
                                             int64_t& base) {
  const int upb = a.H * plan.qchunks;          // units of a sequence
  if (even_lengths(a)) {
    const int64_t per = (int64_t)upb * stream_tiles<TR>(a, 0);
    const Stream st(a.B * per, plan);
    b = (int)min((int64_t)a.B - 1, st.start(min((int)blockIdx.x, st.ctas - 1)) / per);
    base = b * per;
    return st;
  }
  const int tid = threadIdx.x, share = (a.B + kThreads - 1) / kThreads;
  int64_t own = 0;
  for (int i = tid * share; i < min(a.B, (tid + 1) * share); ++i) own += stream_tiles<TR>(a, i);
  sums_s[tid] = own;
  __syncthreads();
  int64_t sum = 0;
  for (int i = 0; i < kThreads; ++i) sum += sums_s[i];
  const Stream st(sum * upb, plan);
  const int64_t x = st.start(min((int)blockIdx.x, st.ctas - 1));
  base = 0;
  int i = 0;
  while (i < kThreads - 1 && (base + sums_s[i]) * upb <= x) base += sums_s[i++];
  for (b = i * share; b < a.B - 1; ++b) {
    const int t = stream_tiles<TR>(a, b);
    if ((base + t) * upb > x) break;
    base += t;
  }
  base *= upb;
  return st;
}

// QT: groups of 8 query heads (1 or 2). STREAM: two CTAs an SM at D = 128, three
// at 64 (the registers of a warp's tile, its sums and its queries).
template <typename T, int D, int QT, bool PEND, bool STREAM>
__global__ void __launch_bounds__(kThreads, STREAM ? stream_ctas_per_sm(D) : 1)
    attend_rows_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ PrefixParts parts,
                       const __grid_constant__ RowsPlan plan) {
  constexpr int TR = tile_rows(QT, STREAM), KG = TR / 16;
  using R = Rows<T, D, KG>;
  constexpr int KC = R::KC, VH = R::VH, QN = 8 * QT;
  __shared__ __align__(16) float part_o[kWarps][QN][D];
  __shared__ float part_ml[kWarps][QN][2];
  __shared__ __align__(16) float cta_o[STREAM ? 1 : QN][D];
  __shared__ float cta_ml[QN][2];

  cg::cluster_group cluster = cg::this_cluster();
  const int C = STREAM ? 1 : (int)cluster.num_blocks(), rank = STREAM ? 0 : (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int N = a.G / a.H, qchunks = plan.qchunks;

  launch_dependents();
  int b, ub;                                      // sequence, unit of it
  int64_t at = 0, end = 0, base = 0;              // STREAM: next tile, the range's end, the sequence's first tile
  int upb = 0;
  if (STREAM) {
    __shared__ int64_t sums_s[kThreads];
    const Stream st = find_range<TR>(a, plan, sums_s, b, base);
    if ((int)blockIdx.x >= st.ctas) {
      if ((int)blockIdx.x == plan.ctas - 1) wait_for_primary();
      return;
    }
    at = st.start(blockIdx.x);
    end = st.start(blockIdx.x + 1);
    upb = a.H * qchunks;
    if (blockIdx.x == 0 && tid == 0 && !even_lengths(a)) plan.first[a.B] = st.total;
    ub = 0;
  } else {
    const int unit = (int)(blockIdx.x / (unsigned)C);
    b = unit / (a.H * qchunks);
    ub = unit - b * a.H * qchunks;
  }

  while (true) {                                  // STREAM: the range's segments, each of one unit
    const SeqRows<TR> seq(a, b);
    int first = 0, total = seq.tiles(a);
    bool whole = true;
    int64_t slot = 0;
    int next_b = b;
    if (STREAM) {
      if (at >= end) break;
      total = max(1, total);
      const int tb = total;
      const int64_t rem = at - base;
      ub = (int)(rem / tb);
      first = (int)(rem - (int64_t)ub * tb);
      total = (int)min((int64_t)tb, first + (end - at));
      at += total - first;
      whole = plan.final && first == 0 && total == tb;
      slot = plan.slot((int64_t)b * upb + ub, blockIdx.x, first == 0);
      if (rem == 0 && tid == 0 && !even_lengths(a)) plan.first[b] = base;
      if (at == base + (int64_t)upb * tb) {
        base = at;
        next_b = b + 1;
      }
    }
    const int qc = ub % qchunks, h = ub / qchunks, bh = b * a.H + h;
    const int q0 = qc * QN, nq = min(QN, N - q0);   // query heads h*N + q0 .. + nq - 1
    const int np = seq.np, tp = seq.tp, to = seq.to;
    int n = seq.n;
    int e = -1;                                     // the evicted row still in place
    if (PEND) {
      e = a.pend[bh];
      if (e >= 0) n += 1;
    }
    auto tile_at = [&](int t) {
      Tile<T> x;
      x.moved = 32;
      if (t < tp) {
        x.ks = a.pk_stride[1];
        x.vs = a.pv_stride[1];
        x.k = static_cast<const T*>(a.pk) + h * a.pk_stride[0] + (int64_t)t * TR * x.ks;
        x.v = static_cast<const T*>(a.pv) + h * a.pv_stride[0] + (int64_t)t * TR * x.vs;
        const int left = np - t * TR;
        x.live = left >= TR ? ~0u >> (32 - TR) : (1u << left) - 1u;
      } else if (t < tp + to) {
        const int r0 = (t - tp) * TR;
        x.ks = a.k_stride[2];
        x.vs = a.v_stride[2];
        x.k = static_cast<const T*>(a.k) + b * a.k_stride[0] + h * a.k_stride[1] + (int64_t)r0 * x.ks;
        x.v = static_cast<const T*>(a.v) + b * a.v_stride[0] + h * a.v_stride[1] + (int64_t)r0 * x.vs;
        const int left = n - r0;
        x.live = left >= TR ? ~0u >> (32 - TR) : left > 0 ? (1u << left) - 1u : 0u;
        if (PEND && e >= 0) {
          if (e >= r0 && e < r0 + TR) x.live &= ~(1u << (e - r0));
          x.moved = max(0, min(32, e - r0 + 1));
        }
      } else {
        x.ks = x.vs = 0;
        x.k = static_cast<const T*>(a.k_new) + b * a.kn_stride[0] + h * a.kn_stride[1];
        x.v = static_cast<const T*>(a.v_new) + b * a.vn_stride[0] + h * a.vn_stride[1];
        x.live = a.k_new ? 1u : 0u;            // (a unit without any rows has one tile of none)
      }
      return x;
    };

    const int stride = C * kWarps;
    int t = first + rank * kWarps + warp;
    uint4 kr[2 * KG][KC], vr[VH][4 * KG];
    Tile<T> cur{};
    if (t < total) {
      cur = tile_at(t);
      R::load_k(kr, cur, g, c);
      R::load_v(vr, cur, g, c);
      if (t + stride < total) prefetch_tile<T, D>(tile_at(t + stride), lane);
    }
    // queries: row g of each group of 8, in the keys' order
    uint4 qr[QT][KC];
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      const int q = q0 + g + 8 * i;
      const T* p = static_cast<const T*>(a.q) + b * a.q_stride[0] + (int64_t)(h * N + q) * a.q_stride[1] + 8 * c;
#pragma unroll
      for (int j = 0; j < KC; ++j)
        qr[i][j] = q < N ? *reinterpret_cast<const uint4*>(p + 32 * j) : make_uint4(0, 0, 0, 0);
    }

    float m[QT], l[QT], acc[VH][4][QT][4];
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      m[i] = kNegInf;
      l[i] = 0.f;
    }
#pragma unroll
    for (int x = 0; x < VH * 4 * QT * 4; ++x) (&acc[0][0][0][0])[x] = 0.f;

    while (t < total) {
      if (PEND && cur.moved < TR) {
#pragma unroll
        for (int nt = 0; nt < 2 * KG; ++nt)
          if (g + 8 * nt >= cur.moved) {
#pragma unroll
            for (int i = 0; i < KC / 2; ++i)
              rotate_back(kr[nt][i], kr[nt][i + KC / 2], a.rope_c + 32 * i + 8 * c, a.rope_s + 32 * i + 8 * c);
          }
      }
      float s[2 * KG][4];
#pragma unroll
      for (int nt = 0; nt < 2 * KG; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[nt][x] = 0.f;
      // (the groups of eight keys are independent: one's sum hides the other's)
#pragma unroll
      for (int i = 0; i < KC; ++i)
#pragma unroll
        for (int w = 0; w < 4; w += 2)
#pragma unroll
          for (int nt = 0; nt < 2 * KG; ++nt)
            mma16816<T>(s[nt], word(qr[0][i], w), QT > 1 ? word(qr[QT - 1][i], w) : 0u, word(qr[0][i], w + 1),
                        QT > 1 ? word(qr[QT - 1][i], w + 1) : 0u, word(kr[nt][i], w), word(kr[nt][i], w + 1));
      const uint32_t live = cur.live;
      t += stride;
      const bool more = t < total;
      if (more) {
        cur = tile_at(t);
        R::load_k(kr, cur, g, c);
      }

      // weights of this lane's rows 2c, 2c + 1, 2c + 8, 2c + 9 for query g (and g + 8)
      uint32_t hi[QT][2 * KG], lo[QT][2 * KG];
      float grow[QT];
      bool up = false;
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        float tm = kNegInf;
#pragma unroll
        for (int nt = 0; nt < 2 * KG; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float& v = s[nt][2 * i + x];
            v = ((live >> (8 * nt + 2 * c + x)) & 1u) ? v * a.scale2 : kNegInf;
            tm = fmaxf(tm, v);
          }
        grow[i] = tm;
        up |= tm > m[i];
      }
      if (__any_sync(~0u, up)) {
#pragma unroll
        for (int i = 0; i < QT; ++i) {
          float tm = grow[i];
          tm = fmaxf(tm, __shfl_xor_sync(~0u, tm, 1));
          tm = fmaxf(tm, __shfl_xor_sync(~0u, tm, 2));
          const float nm = fmaxf(m[i], tm);
          const float f = nm == m[i] ? 1.f : ex2(m[i] - nm);   // first rows: 2^-inf = 0
          m[i] = nm;
          l[i] *= f;
          // the accumulators' columns are queries 2c and 2c + 1
          const float f0 = __shfl_sync(~0u, f, 8 * c), f1 = __shfl_sync(~0u, f, 8 * c + 4);
#pragma unroll
          for (int x = 0; x < VH; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[x][j][i][0] *= f0;
              acc[x][j][i][1] *= f1;
              acc[x][j][i][2] *= f0;
              acc[x][j][i][3] *= f1;
            }
        }
      }
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        const float base = m[i] == kNegInf ? 0.f : m[i];   // nothing so far: every weight 2^-inf = 0
#pragma unroll
        for (int nt = 0; nt < 2 * KG; ++nt) {
          const float p0 = ex2(s[nt][2 * i] - base), p1 = ex2(s[nt][2 * i + 1] - base);
          l[i] += p0 + p1;
          const float2 w = make_float2(p0 * kLift<T>, p1 * kLift<T>);
          hi[i][nt] = pack16<T>(w.x, w.y);
          const float2 back = unpack16<T>(hi[i][nt]);
          lo[i][nt] = pack16<T>(w.x - back.x, w.y - back.y);
        }
      }
#pragma unroll
      for (int k = 0; k < KG; ++k)
#pragma unroll
        for (int x = 0; x < VH; ++x)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w0 = word(vr[x][4 * k], j), w1 = word(vr[x][4 * k + 1], j);
            const uint32_t w2 = word(vr[x][4 * k + 2], j), w3 = word(vr[x][4 * k + 3], j);
            const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
            const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
            for (int i = 0; i < QT; ++i) {
              mma16816<T>(acc[x][j][i], a0, a1, a2, a3, hi[i][2 * k], hi[i][2 * k + 1]);
              mma16816<T>(acc[x][j][i], a0, a1, a2, a3, lo[i][2 * k], lo[i][2 * k + 1]);
            }
          }
      if (more) R::load_v(vr, cur, g, c);
    }
#pragma unroll
    for (int x = 0; x < VH * 4 * QT * 4; ++x) (&acc[0][0][0][0])[x] *= 1.f / kLift<T>;

    // ---------------------------------------------------------------- the prefix's parts
    // Each part (a range of shared rows that one CTA of attend_prefix.cu took) joins
    // one warp's sums as if it were another tile; the query rows b * N + q0 + q may
    // lie in two blocks.
    if (!STREAM && parts.plan.ctas) {
      wait_for_primary();
      const int RB = parts.plan.block_rows;
      const int64_t r0 = (int64_t)b * N + q0;
      for (int64_t blk = r0 / RB; blk <= (r0 + nq - 1) / RB; ++blk) {
        const int u = h * parts.plan.blocks + (int)blk, off = (int)(r0 - blk * RB);   // query q is row off + q
        const int c0 = parts.plan.cta_of((int64_t)u * parts.plan.nkt);
        const int c1 = parts.plan.cta_of((int64_t)(u + 1) * parts.plan.nkt - 1);
        auto inside = [&](int q) { return q < nq && off + q >= 0 && off + q < RB; };
        for (int pc = c0 + rank * kWarps + warp; pc <= c1; pc += stride) {
          const int64_t slot = parts.plan.slot(u, pc, pc == c0);
          const float2* ml = parts.ml + slot * RB;
          const float4* po = reinterpret_cast<const float4*>(parts.o) + slot * (RB * (D / 4));
#pragma unroll
          for (int i = 0; i < QT; ++i) {
            float4 v[2][VH][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int q = 2 * c + k + 8 * i;
              const bool in = inside(q);
#pragma unroll
              for (int x = 0; x < VH; ++x)
#pragma unroll
                for (int w = 0; w < 2; ++w)
                  v[k][x][w] = in ? po[(16 * x + 2 * g + w) * RB + off + q] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            const int q = g + 8 * i;
            float2 part = inside(q) ? ml[off + q] : make_float2(kNegInf, 0.f);
            const float nm = fmaxf(m[i], part.x);
            const float f = m[i] == nm ? 1.f : ex2(m[i] - nm);
            // a part without rows has left no O; a NaN sum (NaN logits, a wait that ran out)
            // passes on, however far its maximum is below the others
            const float fp = part.y == 0.f ? 0.f : part.y != part.y ? part.y : part.x == nm ? 1.f : ex2(part.x - nm);
            m[i] = nm;
            l[i] = l[i] * f + (c == 0 && fp != 0.f ? part.y * fp : 0.f);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float fa = __shfl_sync(~0u, f, 8 * c + 4 * k), fb = __shfl_sync(~0u, fp, 8 * c + 4 * k);
#pragma unroll
              for (int x = 0; x < VH; ++x)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                  const float4 y = fb != 0.f ? v[k][x][w] : make_float4(0.f, 0.f, 0.f, 0.f);
                  acc[x][2 * w][i][k] = acc[x][2 * w][i][k] * fa + y.x * fb;
                  acc[x][2 * w][i][k + 2] = acc[x][2 * w][i][k + 2] * fa + y.y * fb;
                  acc[x][2 * w + 1][i][k] = acc[x][2 * w + 1][i][k] * fa + y.z * fb;
                  acc[x][2 * w + 1][i][k + 2] = acc[x][2 * w + 1][i][k + 2] * fa + y.w * fb;
                }
            }
          }
        }
      }
    }

    // ---------------------------------------------------------------- join the warps
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      l[i] += __shfl_xor_sync(~0u, l[i], 1);
      l[i] += __shfl_xor_sync(~0u, l[i], 2);
      if (c == 0) {
        part_ml[warp][g + 8 * i][0] = m[i];
        part_ml[warp][g + 8 * i][1] = l[i];
      }
#pragma unroll
      for (int x = 0; x < VH; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int d = 64 * x + 8 * g + 2 * j;
          *reinterpret_cast<float2*>(&part_o[warp][8 * i + 2 * c][d]) = make_float2(acc[x][j][i][0], acc[x][j][i][2]);
          *reinterpret_cast<float2*>(&part_o[warp][8 * i + 2 * c + 1][d]) = make_float2(acc[x][j][i][1], acc[x][j][i][3]);
        }
    }
    __syncthreads();
    constexpr int D4 = D / 4;
    for (int x = tid; x < nq * D4; x += kThreads) {
      const int q = x / D4, d = (x - q * D4) * 4;
      float mm = kNegInf;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, part_ml[w][q][0]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = part_ml[w][q][0], f = mw == mm ? 1.f : ex2(mw - mm);
        const float4 v = *reinterpret_cast<const float4*>(&part_o[w][q][d]);
        o.x = fmaf(f, v.x, o.x);
        o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z);
        o.w = fmaf(f, v.w, o.w);
        ll = fmaf(f, part_ml[w][q][1], ll);
      }
      if (!STREAM) {
        *reinterpret_cast<float4*>(&cta_o[STREAM ? 0 : q][d]) = o;
        if (d == 0) {
          cta_ml[q][0] = mm;
          cta_ml[q][1] = ll;
        }
      } else if (whole) {
        write_out<T>(a, b, h * N + q0 + q, d, mm, ll, o);
      } else {
        reinterpret_cast<float4*>(plan.part_o)[(slot * QN + q) * D4 + d / 4] = o;
        if (d == 0) plan.part_ml[slot * QN + q] = make_float2(mm, ll);
      }
    }
    if (STREAM) {
      __syncthreads();                              // the next segment's sums go where these were
      b = next_b;
      if (b >= a.B) break;
      continue;
    }
    // ---------------------------------------------------------------- join the cluster
    cluster.sync();
    for (int x = rank * kThreads + tid; x < nq * D4; x += C * kThreads) {
      const int q = x / D4, d = (x - q * D4) * 4;
      float mm = kNegInf;
      for (int r = 0; r < C; ++r) mm = fmaxf(mm, *cluster.map_shared_rank(&cta_ml[q][0], r));
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float ll = 0.f;
      for (int r = 0; r < C; ++r) {
        const float mr = *cluster.map_shared_rank(&cta_ml[q][0], r), f = mr == mm ? 1.f : ex2(mr - mm);
        const float4 v = *reinterpret_cast<const float4*>(cluster.map_shared_rank(&cta_o[q][d], r));
        o.x = fmaf(f, v.x, o.x);
        o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z);
        o.w = fmaf(f, v.w, o.w);
        ll = fmaf(f, *cluster.map_shared_rank(&cta_ml[q][1], r), ll);
      }
      write_out<T>(a, b, h * N + q0 + q, d, mm, ll, o);
    }
    cluster.sync();   // no CTA leaves while another reads its shared memory
    break;
  }
  // The join that follows waits for this kernel alone, so its last CTA ends after
  // the prefix's kernel, beside which the others may have come and gone.
  if (STREAM && (int)blockIdx.x == plan.ctas - 1) wait_for_primary();
}

// Joins the parts of a stream's cut units, and the prefix's: JW warps a query
// head (one, in blocks of four heads, where a head has few parts), a lane for four
// columns, the parts dealt to the warps and eight loads under way at once.
template <typename T, int D, int QT, int JW>
__global__ void __launch_bounds__(JW == 1 ? 128 : 32 * JW)
    attend_rows_join_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ PrefixParts parts,
                            const __grid_constant__ RowsPlan plan) {
  constexpr int D4 = D / 4, QN = 8 * QT, TR = tile_rows(QT, true), LOADS = 8;
  __shared__ float2 ml_s[JW];
  __shared__ float4 o_s[JW][D4];
  const int warp = JW == 1 ? 0 : threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned head = JW == 1 ? blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  const bool there = head < (unsigned)a.B * (unsigned)a.G;
  const int b = there ? (int)(head / (unsigned)a.G) : 0, gq = there ? (int)(head - (unsigned)b * a.G) : 0;
  // where the head's parts are: all but unequal lengths' before the wait
  const int N = a.G / a.H, h = gq / N, j = gq - h * N, qc = j / QN, q = j - qc * QN;
  const int upb = a.H * plan.qchunks, ub = h * plan.qchunks + qc, tb = stream_tiles<TR>(a, b);
  const int64_t u = (int64_t)b * upb + ub;
  int c0 = 0, c1 = 0;
  auto range = [&](int64_t total, int64_t first) {
    const Stream st(total, plan);
    c0 = st.cta_of(first + (int64_t)ub * tb);
    c1 = st.cta_of(first + (int64_t)ub * tb + tb - 1);
  };
  const bool even = even_lengths(a);
  if (even) range((int64_t)a.B * upb * tb, (int64_t)b * upb * tb);
  int np = 0, p0 = 0, pu = 0, prow = 0;
  if (parts.plan.ctas) {
    const int64_t r = (int64_t)b * N + j;
    const int blk = (int)(r / parts.plan.block_rows);
    prow = (int)(r - (int64_t)blk * parts.plan.block_rows);
    pu = h * parts.plan.blocks + blk;
    p0 = parts.plan.cta_of((int64_t)pu * parts.plan.nkt);
    np = parts.plan.cta_of((int64_t)(pu + 1) * parts.plan.nkt - 1) - p0 + 1;
  }
  wait_for_primary();                             // in every block: this kernel ends after the one before it
  if (!there) return;
  if (!even) range(plan.first[a.B], plan.first[b]);
  if (plan.final && c0 == c1) return;             // written out by that CTA
  const int nr = c1 - c0 + 1;
  float m = kNegInf, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = warp; i0 < nr + np; i0 += LOADS * JW) {
    float2 ml[LOADS];
    float4 v[LOADS];
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
      const int i = i0 + JW * k;
      ml[k] = make_float2(kNegInf, 0.f);
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < nr) {
        const int64_t slot = plan.slot(u, c0 + i, i == 0) * QN + q;
        ml[k] = plan.part_ml[slot];
        if (lane < D4) v[k] = reinterpret_cast<const float4*>(plan.part_o)[slot * D4 + lane];
      } else if (i < nr + np) {
        const int64_t slot = parts.plan.slot(pu, p0 + i - nr, i == nr) * parts.plan.block_rows;
        ml[k] = parts.ml[slot + prow];
        if (lane < D4)
          v[k] = reinterpret_cast<const float4*>(parts.o)[slot * D4 + (int64_t)lane * parts.plan.block_rows + prow];
      }
    }
    float nm = m;
#pragma unroll
    for (int k = 0; k < LOADS; ++k) nm = fmaxf(nm, ml[k].x);
    const float f = m == nm ? 1.f : ex2(m - nm);
    m = nm;
    l *= f;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
      const float w = ml[k].x == nm ? 1.f : ex2(ml[k].x - nm);
      l = fmaf(ml[k].y, w, l);
      o = make_float4(fmaf(v[k].x, w, o.x), fmaf(v[k].y, w, o.y), fmaf(v[k].z, w, o.z), fmaf(v[k].w, w, o.w));
    }
  }
  if (JW > 1) {
    if (lane == 0) ml_s[warp] = make_float2(m, l);
    if (lane < D4) o_s[warp][lane] = o;
    __syncthreads();
    if (warp != 0) return;
    for (int w = 1; w < JW; ++w) {
      const float2 ml = ml_s[w];
      const float4 v = o_s[w][min(lane, D4 - 1)];
      const float nm = fmaxf(m, ml.x), f = m == nm ? 1.f : ex2(m - nm), y = ml.x == nm ? 1.f : ex2(ml.x - nm);
      m = nm;
      l = l * f + ml.y * y;
      o = make_float4(o.x * f + v.x * y, o.y * f + v.y * y, o.z * f + v.z * y, o.w * f + v.w * y);
    }
  }
  if (lane < D4) write_out<T>(a, b, gq, 4 * lane, m, l, o);
}

template <typename T, int D, int QT, bool PEND>
cudaError_t launch_one(const AttendArgs& a, const PrefixParts& parts, const RowsPlan& plan, int sms, cudaStream_t s) {
  if (plan.ctas) {
    // either may begin while the kernel before it ends (the first one only where
    // that is the prefix's of this call)
    const cudaError_t e = launch_after(attend_rows_kernel<T, D, QT, PEND, true>, plan.ctas, kThreads, 0, 1,
                                       parts.plan.ctas > 0, s, a, parts, plan);
    if (e != cudaSuccess) return e;
    // parts of a head, about: the prefix's and its unit's
    const int64_t heads = (int64_t)a.B * a.G;
    const int64_t count = parts.plan.ctas / std::max(1, parts.plan.units) + plan.ctas / plan.units + 2;
    if (count <= (heads >= 4 * sms ? kFewParts : kFewParts / 2))
      return launch_after(attend_rows_join_kernel<T, D, QT, 1>, dim3((unsigned)((heads + 3) / 4)), 128, 0, 1, true, s, a,
                          parts, plan);
    return launch_after(attend_rows_join_kernel<T, D, QT, 8>, dim3((unsigned)heads), 256, 0, 1, true, s, a, parts, plan);
  }
  const int64_t units = (int64_t)a.B * a.H * plan.qchunks;
  const int64_t tiles = rows_tiles(tile_rows(QT, false), a.n, a.P, a.k_new, a.pend) + parts.plan.ctas / a.H;
  const int C = cluster_ctas(units, tiles, sms);
  if (units * C > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return launch_after(attend_rows_kernel<T, D, QT, PEND, false>, dim3((unsigned)(units * C)), kThreads, 0, C,
                      parts.plan.ctas > 0, s, a, parts, plan);
}

template <typename T, int D, bool PEND>
cudaError_t launch_q(const AttendArgs& a, const PrefixParts& parts, const RowsPlan& plan, int sms, cudaStream_t s) {
  return rows_qt(a.G / a.H) == 1 ? launch_one<T, D, 1, PEND>(a, parts, plan, sms, s)
                                 : launch_one<T, D, 2, PEND>(a, parts, plan, sms, s);
}

}  // namespace

RowsPlan rows_plan(int B, int G, int H, int D, int n, int P, bool has_new, bool pend, bool prefix_parts, int sms) {
  RowsPlan pl{};
  const int qt = rows_qt(G / H);
  pl.qn = 8 * qt;
  pl.batch = B;
  pl.qchunks = (G / H + pl.qn - 1) / pl.qn;
  pl.units = (int64_t)B * H * pl.qchunks;
  pl.final = !prefix_parts;
  const int64_t ctas = (int64_t)sms * stream_ctas_per_sm(D), tiles = rows_tiles(16, n, P, has_new, pend);
  const int64_t total = pl.units * tiles;
  if ((int64_t)B * G <= 0x7FFFFFFF && (total >= ctas * kWarps * (prefix_parts ? kBesideTiles : kStreamTiles) ||
                                       tiles >= (int64_t)cluster_ctas(pl.units, tiles, sms) * kWarps * kClusterTiles))
    pl.ctas = (int)std::min<int64_t>(ctas, (total + kWarps - 1) / kWarps);
  pl.slots = pl.final ? 2 * (int64_t)pl.ctas : pl.units + ctas;
  return pl;
}

int stream_ctas(int D, int sms) { return sms * stream_ctas_per_sm(D); }

size_t RowsPlan::o_bytes(int D) const { return (size_t)slots * qn * D * 4; }
size_t RowsPlan::ml_bytes() const { return (size_t)slots * qn * 8; }
size_t RowsPlan::bytes(int D) const { return ctas ? o_bytes(D) + ml_bytes() + ((size_t)batch + 1) * 8 : 0; }

cudaError_t launch_attend_rows(const AttendArgs& a, const PrefixParts& parts, const RowsPlan& plan, int D, int dtype,
                               int sms, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  if (a.pend)   // a handle's rows are fp16
    return D == 64 ? launch_q<__half, 64, true>(a, parts, plan, sms, s) : launch_q<__half, 128, true>(a, parts, plan, sms, s);
  if (dtype == kBf16)
    return D == 64 ? launch_q<bf16, 64, false>(a, parts, plan, sms, s) : launch_q<bf16, 128, false>(a, parts, plan, sms, s);
  return D == 64 ? launch_q<__half, 64, false>(a, parts, plan, sms, s) : launch_q<__half, 128, false>(a, parts, plan, sms, s);
}

}  // namespace kvx
