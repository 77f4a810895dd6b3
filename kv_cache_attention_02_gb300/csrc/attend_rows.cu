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
// A warp takes 16 rows at a time. Its key registers are refilled as soon as the
// logits are out of them, its value registers as soon as the sums are, so one
// of the two is always in flight. Running maximum, sum and output stay in fp32
// registers; the maximum is looked at again only when some lane exceeds it.
//
// The weights go into the second product as a sum of two 16-bit parts
// (p = hi + lo), 22 bits in all for fp16 and 16 for bf16: the matrix pipe has
// room for the second instruction here, and the output keeps the accuracy of
// its own rounding.
//
// A (sequence, key head, up to 16 query heads) is split over a cluster of CTAs
// when there are too few of them to fill the GPU; the parts are joined through
// distributed shared memory, in a fixed order, with no second launch and no
// workspace.
#include "attend_internal.cuh"

#include <cooperative_groups.h>

namespace kvx {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kNegInf = -__builtin_huge_valf();

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

// 16 consecutive rows of one source; row r is there if bit r of `live` is set.
template <typename T>
struct Tile {
  const T* k;
  const T* v;
  int64_t ks, vs;
  uint32_t live;
  int moved;    // rows from here on await the re-rotation by -1 (16: none)
};

template <typename T, int D>
struct Rows {
  static constexpr int KC = D / 32;   // 16-byte pieces of a key row in one lane
  static constexpr int VH = D / 64;   // 64-wide column groups of a value row

  __device__ __forceinline__ static void load_k(uint4 (&kr)[2][KC], const Tile<T>& t, int g, int c) {
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const int r = g + 8 * nt;
      const T* p = t.k + (int64_t)r * t.ks + 8 * c;
      const bool on = (t.live >> r) & 1u;
#pragma unroll
      for (int i = 0; i < KC; ++i) kr[nt][i] = on ? ld_stream16(p + 32 * i) : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ static void load_v(uint4 (&vr)[VH][4], const Tile<T>& t, int g, int c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 2 * c + (j & 1) + 8 * (j >> 1);
      const T* p = t.v + (int64_t)r * t.vs + 8 * g;
      const bool on = (t.live >> r) & 1u;
#pragma unroll
      for (int h = 0; h < VH; ++h) vr[h][j] = on ? ld_stream16(p + 64 * h) : make_uint4(0, 0, 0, 0);
    }
  }
};

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

// QT: groups of 8 query heads (1 or 2).
template <typename T, int D, int QT, bool PEND>
__global__ void __launch_bounds__(kThreads) attend_rows_kernel(const __grid_constant__ AttendArgs a,
                                                                  const __grid_constant__ PrefixParts parts, const int qchunks) {
  using R = Rows<T, D>;
  constexpr int KC = R::KC, VH = R::VH, QN = 8 * QT;
  __shared__ __align__(16) float part_o[kWarps][QN][D];
  __shared__ float part_ml[kWarps][QN][2];
  __shared__ __align__(16) float cta_o[QN][D];
  __shared__ float cta_ml[QN][2];

  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int N = a.G / a.H;
  const int unit = (int)(blockIdx.x / (unsigned)C);
  const int qc = unit % qchunks, bh = unit / qchunks;
  const int b = bh / a.H, h = bh - b * a.H;
  const int q0 = qc * QN, nq = min(QN, N - q0);   // query heads h*N + q0 .. + nq - 1

  // rows of each source, in tiles of 16: shared, own, the token's own
  const int np = a.plens ? max(0, min(a.plens[b], a.P)) : a.P;
  int n = a.lens ? max(0, min(a.lens[b], a.n)) : a.n;
  int e = -1;                                     // the evicted row still in place
  if (PEND) {
    e = a.pend[bh];
    if (e >= 0) n += 1;
  }
  const int tp = (np + 15) >> 4, to = (n + 15) >> 4;
  const int total = tp + to + (a.k_new ? 1 : 0);
  auto tile_at = [&](int t) {
    Tile<T> x;
    x.moved = 16;
    if (t < tp) {
      x.ks = a.pk_stride[1];
      x.vs = a.pv_stride[1];
      x.k = static_cast<const T*>(a.pk) + h * a.pk_stride[0] + (int64_t)t * 16 * x.ks;
      x.v = static_cast<const T*>(a.pv) + h * a.pv_stride[0] + (int64_t)t * 16 * x.vs;
      const int left = np - t * 16;
      x.live = left >= 16 ? 0xFFFFu : (1u << left) - 1u;
    } else if (t < tp + to) {
      const int r0 = (t - tp) * 16;
      x.ks = a.k_stride[2];
      x.vs = a.v_stride[2];
      x.k = static_cast<const T*>(a.k) + b * a.k_stride[0] + h * a.k_stride[1] + (int64_t)r0 * x.ks;
      x.v = static_cast<const T*>(a.v) + b * a.v_stride[0] + h * a.v_stride[1] + (int64_t)r0 * x.vs;
      const int left = n - r0;
      x.live = left >= 16 ? 0xFFFFu : (1u << left) - 1u;
      if (PEND && e >= 0) {
        if (e >= r0 && e < r0 + 16) x.live &= ~(1u << (e - r0));
        x.moved = max(0, min(16, e - r0 + 1));
      }
    } else {
      x.ks = x.vs = 0;
      x.k = static_cast<const T*>(a.k_new) + b * a.kn_stride[0] + h * a.kn_stride[1];
      x.v = static_cast<const T*>(a.v_new) + b * a.vn_stride[0] + h * a.vn_stride[1];
      x.live = 1u;
    }
    return x;
  };

  const int stride = C * kWarps;
  int t = rank * kWarps + warp;
  uint4 kr[2][KC], vr[VH][4];
  Tile<T> cur{};
  if (t < total) {
    cur = tile_at(t);
    R::load_k(kr, cur, g, c);
    R::load_v(vr, cur, g, c);
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
    if (PEND && cur.moved < 16) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
        if (g + 8 * nt >= cur.moved) {
#pragma unroll
          for (int i = 0; i < KC / 2; ++i)
            rotate_back(kr[nt][i], kr[nt][i + KC / 2], a.rope_c + 32 * i + 8 * c, a.rope_s + 32 * i + 8 * c);
        }
    }
    float s[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
      for (int x = 0; x < 4; ++x) s[nt][x] = 0.f;
#pragma unroll
      for (int i = 0; i < KC; ++i)
#pragma unroll
        for (int w = 0; w < 4; w += 2)
          mma16816<T>(s[nt], word(qr[0][i], w), QT > 1 ? word(qr[QT - 1][i], w) : 0u, word(qr[0][i], w + 1),
                      QT > 1 ? word(qr[QT - 1][i], w + 1) : 0u, word(kr[nt][i], w), word(kr[nt][i], w + 1));
    }
    const uint32_t live = cur.live;
    t += stride;
    const bool more = t < total;
    if (more) {
      cur = tile_at(t);
      R::load_k(kr, cur, g, c);
    }

    // weights of this lane's rows 2c, 2c + 1, 2c + 8, 2c + 9 for query g (and g + 8)
    uint32_t hi[QT][2], lo[QT][2];
    float grow[QT];
    bool up = false;
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      float tm = kNegInf;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
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
        const float f = nm == m[i] ? 1.f : ex2_approx(m[i] - nm);   // first rows: 2^-inf = 0
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
      for (int nt = 0; nt < 2; ++nt) {
        const float p0 = ex2_approx(s[nt][2 * i] - base), p1 = ex2_approx(s[nt][2 * i + 1] - base);
        l[i] += p0 + p1;
        hi[i][nt] = pack16<T>(p0, p1);
        const float2 back = unpack16<T>(hi[i][nt]);
        lo[i][nt] = pack16<T>(p0 - back.x, p1 - back.y);
      }
    }
#pragma unroll
    for (int x = 0; x < VH; ++x)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w0 = word(vr[x][0], j), w1 = word(vr[x][1], j), w2 = word(vr[x][2], j), w3 = word(vr[x][3], j);
        const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
        const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
        for (int i = 0; i < QT; ++i) {
          mma16816<T>(acc[x][j][i], a0, a1, a2, a3, hi[i][0], hi[i][1]);
          mma16816<T>(acc[x][j][i], a0, a1, a2, a3, lo[i][0], lo[i][1]);
        }
      }
    if (more) R::load_v(vr, cur, g, c);
  }

  // ---------------------------------------------------------------- the prefix's parts
  // Each part (a range of shared rows that one CTA of attend_prefix.cu took) joins
  // one warp's sums as if it were another tile; the query rows b * N + q0 + q may
  // lie in two blocks.
  if (parts.plan.ctas) {
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
          const float f = m[i] == nm ? 1.f : ex2_approx(m[i] - nm);
          // a part without rows has left no O; a NaN sum passes on
          const float fp = part.y == 0.f ? 0.f : part.x == nm ? 1.f : ex2_approx(part.x - nm);
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
      const float mw = part_ml[w][q][0], f = mw == mm ? 1.f : ex2_approx(mw - mm);
      const float4 v = *reinterpret_cast<const float4*>(&part_o[w][q][d]);
      o.x = fmaf(f, v.x, o.x);
      o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z);
      o.w = fmaf(f, v.w, o.w);
      ll = fmaf(f, part_ml[w][q][1], ll);
    }
    *reinterpret_cast<float4*>(&cta_o[q][d]) = o;
    if (d == 0) {
      cta_ml[q][0] = mm;
      cta_ml[q][1] = ll;
    }
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
      const float mr = *cluster.map_shared_rank(&cta_ml[q][0], r), f = mr == mm ? 1.f : ex2_approx(mr - mm);
      const float4 v = *reinterpret_cast<const float4*>(cluster.map_shared_rank(&cta_o[q][d], r));
      o.x = fmaf(f, v.x, o.x);
      o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z);
      o.w = fmaf(f, v.w, o.w);
      ll = fmaf(f, *cluster.map_shared_rank(&cta_ml[q][1], r), ll);
    }
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    const int gq = h * N + q0 + q;
    T* dst = static_cast<T*>(a.out) + b * a.out_stride[0] + (int64_t)gq * a.out_stride[1] + d;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack16<T>(o.x * inv, o.y * inv), pack16<T>(o.z * inv, o.w * inv));
    if (d == 0 && a.lse) a.lse[(int64_t)b * a.G + gq] = ll == 0.f ? kNegInf : (mm + log2f(ll)) * 0.69314718055994531f;
  }
  cluster.sync();   // no CTA leaves while another reads its shared memory
}

template <typename T, int D, int QT, bool PEND>
cudaError_t launch_one(const AttendArgs& a, const PrefixParts& parts, int sms, cudaStream_t s) {
  const int N = a.G / a.H;
  const int qchunks = (N + 8 * QT - 1) / (8 * QT);
  const int64_t units = (int64_t)a.B * a.H * qchunks;
  const int64_t tiles = ((int64_t)a.P + 15) / 16 + ((int64_t)a.n + 15) / 16 + 1 + parts.plan.ctas / a.H;
  // Split a unit's rows over a cluster until the GPU has about 16 warps an SM
  // or a warp has one tile.
  int C = 1;
  while (C < 16 && units * C * kWarps < (int64_t)sms * 12 && (int64_t)C * kWarps < tiles) C *= 2;
  if (units * C > 0x7FFFFFFF) return cudaErrorInvalidValue;
  auto kernel = attend_rows_kernel<T, D, QT, PEND>;
  if (C > 8) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, parts, qchunks);
}

template <typename T, int D, bool PEND>
cudaError_t launch_q(const AttendArgs& a, const PrefixParts& parts, int sms, cudaStream_t s) {
  return a.G / a.H <= 8 ? launch_one<T, D, 1, PEND>(a, parts, sms, s) : launch_one<T, D, 2, PEND>(a, parts, sms, s);
}

}  // namespace

cudaError_t launch_attend_rows(const AttendArgs& a, const PrefixParts& parts, int D, int dtype, int sms, cudaStream_t s) {
  if (a.pend)   // a handle's rows are fp16
    return D == 64 ? launch_q<__half, 64, true>(a, parts, sms, s) : launch_q<__half, 128, true>(a, parts, sms, s);
  if (dtype == kBf16)
    return D == 64 ? launch_q<__nv_bfloat16, 64, false>(a, parts, sms, s) : launch_q<__nv_bfloat16, 128, false>(a, parts, sms, s);
  return D == 64 ? launch_q<__half, 64, false>(a, parts, sms, s) : launch_q<__half, 128, false>(a, parts, sms, s);
}

}  // namespace kvx
