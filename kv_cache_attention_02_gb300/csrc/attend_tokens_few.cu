// attend_tokens_few.cu -- attention of several query tokens a sequence (kvevict_attend_prompt,
// kvevict_attend_tree) where there is little of it: short prompts, small trees. The
// tensor-core kernel of attend_tokens.cu takes 7 to 8 us for its start, one tile and its end.
// Where that kernel cannot be launched, this one answers its calls, too.
//
// A unit is 16 query rows (tokens x the query heads of a key head) of a sequence's key
// head: one cluster of CTAs, the unit's tiles of 16 keys dealt to the cluster's warps, the
// sums joined through distributed shared memory; one launch, no workspace. The arithmetic
// is that of attend_rows.cu: rows from memory straight into the registers of
// mma.m16n8k16, weights as the sum of two 16-bit parts, everything else in fp32.
// Every 16 query rows read their keys again, from L2 after the first.
//
// Of the tokens' keys, token t sees 0..t, or itself and its ancestors. Values that are not
// finite, in tiles that the unit's rows see in part, are left out of the products (their
// weight of 0 would spoil the sums) and added at the end to the rows that see them.
//
// Bound by latency. Measured on GB300 (us, a call among others on the device): a prompt of 37
// tokens, 4 heads of 64, 3.6; 8 drafted tokens on 32 rows 3.7; 16 tokens x 24 query heads on 8
// of 512 rows 8.9, on 2048 (32 heads) 12.5. The cluster's sums one after the other instead
// of all at once: 0.4 to 0.8 more.
#include "attend_tokens.cuh"
#include "mma_rows.cuh"

#include <cooperative_groups.h>

namespace kvx {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4, kThreads = kWarps * 32, kRows = 16, kCluster = 8;   // (at most)
constexpr float kNegInf = -__builtin_huge_valf();

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2) tokens_few_kernel(const __grid_constant__ TokensArgs a,
                                                                 const __grid_constant__ FewArgs f) {
  using R = Rows<T, D, 1>;
  constexpr int KC = R::KC, VH = R::VH, D4 = D / 4;
  __shared__ __align__(16) float part_o[kWarps][kRows][D];
  __shared__ float part_ml[kWarps][kRows][2];
  __shared__ __align__(16) float cta_o[kRows][D];
  __shared__ __align__(8) float cta_ml[kRows][2];
  __shared__ int dropped, found_s[2], sums_s[kWarps];

  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int N = a.G / f.H;
  const unsigned unit = blockIdx.x / (unsigned)C, h = unit % (unsigned)f.H;
  int chunk = (int)(unit / (unsigned)f.H), b = 0;      // of the sequence's rows
  if (tid == 0) dropped = 0;
  if (!a.starts) {
    b = (int)((unsigned)chunk / (unsigned)f.chunks);
    chunk -= b * f.chunks;
  } else {
    // packed: the sequence whose chunks this one is among, a sequence a thread at a time. (Sums
    // end at a number above every chunk's: sequences that overlap could add up to anything.)
    constexpr int kEnd = 1 << 29;
    int before = 0;
    if (tid == 0) found_s[0] = -1;
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
      const Seq s = b0 + tid < a.B ? load_seq(a, b0 + tid) : Seq{0, 0, 0, 0};
      const int own = (int)((unsigned)(s.nq * N + kRows - 1) / (unsigned)kRows);
      int to = own;
      for (int d = 1; d < 32; d *= 2) {
        const int x = __shfl_up_sync(~0u, to, d);
        if (lane >= d) to = min(to + x, kEnd);
      }
      if (lane == 31) sums_s[warp] = to;
      __syncthreads();
      for (int w = 0; w < kWarps; ++w) {
        if (w == warp) {
          to = min(to + before, kEnd);
          if (chunk >= to - own && chunk < to) {
            found_s[0] = b0 + tid;
            found_s[1] = chunk - (to - own);
          }
        }
        before = min(before + sums_s[w], kEnd);
      }
      __syncthreads();
      if (found_s[0] >= 0) break;
    }
    b = found_s[0];
    chunk = found_s[1];
    if (b < 0) return;                                 // (the whole cluster)
  }
  const Seq s = load_seq(a, b);
  const int r0 = chunk * kRows, nr = min(kRows, s.nq * N - r0);
  if (nr <= 0) return;
  const int first = (int)((unsigned)r0 / (unsigned)N), last = (int)((unsigned)(r0 + nr - 1) / (unsigned)N);   // tokens
  int e = -1, n = s.n;                                 // the evicted row still in place; rows as they lie
  if (a.pend) {
    e = a.pend[b * f.H + h];
    n += e >= 0;
  }
  const int to = (n + 15) / 16, total = to + (a.parents ? s.nq + 15 : last + 16) / 16;

  // this lane's two query rows: their tokens, and what they see
  int t[2];
  const T* q[2];
  uint64_t seen[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + min(g + 8 * i, nr - 1);
    t[i] = (int)((unsigned)r / (unsigned)N);
    q[i] = static_cast<const T*>(f.q) + b * f.q_stride[0] + (int64_t)(s.tok0 + t[i]) * f.q_stride[1] +
           (int64_t)(h * N + r - t[i] * N) * f.q_stride[2] + 8 * c;
  }
  auto tile_at = [&](int x) {
    Tile<T> y;
    y.moved = 32;
    int left;
    if (x < to) {
      const int row = 16 * x;
      y.ks = f.k_stride[2];
      y.vs = f.v_stride[2];
      y.k = static_cast<const T*>(f.k) + b * f.k_stride[0] + h * f.k_stride[1] + row * y.ks;
      y.v = static_cast<const T*>(f.v) + b * f.v_stride[0] + h * f.v_stride[1] + row * y.vs;
      left = n - row;
      if (e >= 0) y.moved = max(0, min(32, e - row + 1));
    } else {
      const int row = 16 * (x - to);
      y.ks = f.kn_stride[1];
      y.vs = a.vn_stride[1];
      y.k = static_cast<const T*>(f.k_new) + b * f.kn_stride[0] + h * f.kn_stride[2] + (s.tok0 + row) * y.ks;
      y.v = static_cast<const T*>(a.v_new) + b * a.vn_stride[0] + h * a.vn_stride[2] + (s.tok0 + row) * y.vs;
      left = (a.parents ? s.nq : last + 1) - row;
    }
    y.live = left >= 16 ? 0xFFFFu : (1u << left) - 1u;
    if (e >= 0 && x < to && e >= 16 * x && e < 16 * x + 16) y.live &= ~(1u << (e & 15));
    return y;
  };

  const int stride = C * kWarps;
  int x = rank * kWarps + warp;
  uint4 kr[2][KC], vr[VH][4];
  Tile<T> cur{};
  if (x < total) {
    cur = tile_at(x);
    R::load_k(kr, cur, g, c);
    R::load_v(vr, cur, g, c);
  }
  uint4 qr[2][KC];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < KC; ++j) qr[i][j] = *reinterpret_cast<const uint4*>(q[i] + 32 * j);
  if (a.parents) {
    uint64_t anc[2];
    ancestors(a, b, s.nq, anc);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t m0 = __shfl_sync(~0u, anc[0], t[i] & 31), m1 = __shfl_sync(~0u, anc[1], t[i] & 31);
      seen[i] = t[i] < 32 ? m0 : m1;
    }
  }
  float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f}, acc[VH][4][2][4];
#pragma unroll
  for (int y = 0; y < VH * 32; ++y) (&acc[0][0][0][0])[y] = 0.f;
  __syncthreads();                                     // `dropped` is 0

#pragma unroll 1
  while (x < total) {
    if constexpr (std::is_same<T, __half>::value) {    // (a handle's rows)
      if (cur.moved < 16) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
          if (g + 8 * nt >= cur.moved) {
#pragma unroll
            for (int i = 0; i < KC / 2; ++i)
              rotate_back(kr[nt][i], kr[nt][i + KC / 2], a.rope_c + 32 * i + 8 * c, a.rope_s + 32 * i + 8 * c);
          }
      }
    }
    float z[2][4];
#pragma unroll
    for (int y = 0; y < 8; ++y) (&z[0][0])[y] = 0.f;
#pragma unroll
    for (int i = 0; i < KC; ++i)
#pragma unroll
      for (int w = 0; w < 4; w += 2)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
          mma16816<T>(z[nt], word(qr[0][i], w), word(qr[1][i], w), word(qr[0][i], w + 1), word(qr[1][i], w + 1),
                      word(kr[nt][i], w), word(kr[nt][i], w + 1));
    // what the rows see of the tile
    uint32_t sees[2] = {cur.live, cur.live};
    bool part = false;
    if (x >= to) {
      const int k0 = 16 * (x - to);
      part = a.parents || k0 + 15 > first;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int left = t[i] + 1 - k0;
        sees[i] &= a.parents ? (uint32_t)(seen[i] >> k0) : left >= 16 ? 0xFFFFu : left <= 0 ? 0u : (1u << left) - 1u;
      }
    }
    x += stride;
    const bool more = x < total;
    if (more) {
      cur = tile_at(x);
      R::load_k(kr, cur, g, c);
    }
    // weights of this lane's keys 2c, 2c + 1, 2c + 8, 2c + 9 for rows g and g + 8
    uint32_t hi[2][2], lo[2][2];
    float grow[2];
    bool up = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = kNegInf;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float& v = z[nt][2 * i + y];
          v = ((sees[i] >> (8 * nt + 2 * c + y)) & 1u) ? v * a.scale2 : kNegInf;
          top = fmaxf(top, v);
        }
      grow[i] = top;
      up |= top > m[i];
    }
    if (__any_sync(~0u, up)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float top = grow[i];
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        const float nm = fmaxf(m[i], top), k = nm == m[i] ? 1.f : ex2(m[i] - nm);   // first keys: 2^-inf = 0
        m[i] = nm;
        l[i] *= k;
        // the accumulators' columns are rows 2c and 2c + 1
        const float k0 = __shfl_sync(~0u, k, 8 * c), k1 = __shfl_sync(~0u, k, 8 * c + 4);
#pragma unroll
        for (int y = 0; y < VH; ++y)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[y][j][i][0] *= k0;
            acc[y][j][i][1] *= k1;
            acc[y][j][i][2] *= k0;
            acc[y][j][i][3] *= k1;
          }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float base = m[i] == kNegInf ? 0.f : m[i];   // nothing so far: every weight 2^-inf = 0
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const float p0 = ex2(z[nt][2 * i] - base), p1 = ex2(z[nt][2 * i + 1] - base);
        l[i] += p0 + p1;
        const float2 w = make_float2(p0 * kWeightLift<T>, p1 * kWeightLift<T>);
        hi[i][nt] = pack16<T>(w.x, w.y);
        const float2 back = unpack16<T>(hi[i][nt]);
        lo[i][nt] = pack16<T>(w.x - back.x, w.y - back.y);
      }
    }
    if (part) {
      uint32_t bad = 0;
#pragma unroll
      for (int y = 0; y < VH * 4; ++y) {
        const uint4 v = (&vr[0][0])[y];
        bad |= not_finite<T>(v.x) | not_finite<T>(v.y) | not_finite<T>(v.z) | not_finite<T>(v.w);
      }
      if (__builtin_expect(__any_sync(~0u, bad != 0), 0)) {
#pragma unroll
        for (int y = 0; y < VH * 4; ++y) {
          uint4& v = (&vr[0][0])[y];
          v = make_uint4(drop_not_finite<T>(v.x), drop_not_finite<T>(v.y), drop_not_finite<T>(v.z), drop_not_finite<T>(v.w));
        }
        dropped = 1;
      }
    }
#pragma unroll
    for (int y = 0; y < VH; ++y)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w0 = word(vr[y][0], j), w1 = word(vr[y][1], j), w2 = word(vr[y][2], j), w3 = word(vr[y][3], j);
        const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
        const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mma16816<T>(acc[y][j][i], a0, a1, a2, a3, hi[i][0], hi[i][1]);
          mma16816<T>(acc[y][j][i], a0, a1, a2, a3, lo[i][0], lo[i][1]);
        }
      }
    if (more) R::load_v(vr, cur, g, c);
  }

  // ---------------------------------------------------------------- join the warps
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(~0u, l[i], 1);
    l[i] += __shfl_xor_sync(~0u, l[i], 2);
    if (c == 0) {
      part_ml[warp][g + 8 * i][0] = m[i];
      part_ml[warp][g + 8 * i][1] = l[i];
    }
#pragma unroll
    for (int y = 0; y < VH; ++y)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = 64 * y + 8 * g + 2 * j;
        constexpr float k = 1.f / kWeightLift<T>;
        *reinterpret_cast<float2*>(&part_o[warp][8 * i + 2 * c][d]) = make_float2(acc[y][j][i][0] * k, acc[y][j][i][2] * k);
        *reinterpret_cast<float2*>(&part_o[warp][8 * i + 2 * c + 1][d]) = make_float2(acc[y][j][i][1] * k, acc[y][j][i][3] * k);
      }
  }
  __syncthreads();
#pragma unroll 1
  for (int y = tid; y < nr * D4; y += kThreads) {
    const int r = y / D4, d = (y - r * D4) * 4;
    float mm = kNegInf;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, part_ml[w][r][0]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float ll = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = part_ml[w][r][0], k = mw == mm ? 1.f : ex2(mw - mm);
      const float4 v = *reinterpret_cast<const float4*>(&part_o[w][r][d]);
      o = make_float4(fmaf(k, v.x, o.x), fmaf(k, v.y, o.y), fmaf(k, v.z, o.z), fmaf(k, v.w, o.w));
      ll = fmaf(k, part_ml[w][r][1], ll);
    }
    *reinterpret_cast<float4*>(&cta_o[r][d]) = o;
    if (d == 0) {
      cta_ml[r][0] = mm;
      cta_ml[r][1] = ll;
    }
  }
  // ---------------------------------------------------------------- join the cluster
  cluster.sync();
  bool poisoned = false;
#pragma unroll
  for (int k = 0; k < kCluster; ++k)
    if (k < C) poisoned |= *cluster.map_shared_rank(&dropped, k) != 0;
#pragma unroll 1
  for (int y = rank * kThreads + tid; y < nr * D4; y += C * kThreads) {
    const int r = y / D4, d = (y - r * D4) * 4;
    // (all of the other CTAs' sums on their way at once)
    float2 ml[kCluster];
    float4 v[kCluster];
#pragma unroll
    for (int k = 0; k < kCluster; ++k) {
      ml[k] = make_float2(kNegInf, 0.f);
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < C) {
        ml[k] = *reinterpret_cast<const float2*>(cluster.map_shared_rank(&cta_ml[r][0], k));
        v[k] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(&cta_o[r][d], k));
      }
    }
    float mm = kNegInf;
#pragma unroll
    for (int k = 0; k < kCluster; ++k) mm = fmaxf(mm, ml[k].x);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float ll = 0.f;
#pragma unroll
    for (int k = 0; k < kCluster; ++k) {
      const float w = ml[k].x == mm ? 1.f : ex2(ml[k].x - mm);
      o = make_float4(fmaf(w, v[k].x, o.x), fmaf(w, v[k].y, o.y), fmaf(w, v[k].z, o.z), fmaf(w, v[k].w, o.w));
      ll = fmaf(w, ml[k].y, ll);
    }
    const int tt = (int)((unsigned)(r0 + r) / (unsigned)N), head = h * N + r0 + r - tt * N;
    if (__builtin_expect(poisoned, 0)) {
      // the values left out, for the keys that the row sees
#pragma unroll 1
      for (int j = a.parents ? tt : first & ~15; j >= 0 && j <= tt;) {
        const T* v = static_cast<const T*>(a.v_new) + b * a.vn_stride[0] + (s.tok0 + j) * a.vn_stride[1] + h * a.vn_stride[2] + d;
        const uint2 w = *reinterpret_cast<const uint2*>(v);
        const uint32_t bx = not_finite<T>(w.x), by = not_finite<T>(w.y);
        const float2 lo = unpack16<T>(w.x), up = unpack16<T>(w.y);
        if (bx & 0x8000u) o.x += lo.x;
        if (bx & 0x80000000u) o.y += lo.y;
        if (by & 0x8000u) o.z += up.x;
        if (by & 0x80000000u) o.w += up.y;
        if (a.parents) {                                // on to the parent
          const int up_to = a.parents[b * a.parents_stride + j];
          if (up_to >= j) break;
          j = up_to;
        } else {
          ++j;
        }
      }
    }
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    T* dst = static_cast<T*>(a.out) + b * a.out_stride[0] + (s.tok0 + tt) * a.out_stride[1] + head * a.out_stride[2] + d;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack16<T>(o.x * inv, o.y * inv), pack16<T>(o.z * inv, o.w * inv));
    if (d == 0 && a.lse)
      a.lse[((a.starts ? (int64_t)s.tok0 : (int64_t)b * a.S) + tt) * a.G + head] =
          ll == 0.f ? kNegInf : (mm + log2f(ll)) * 0.69314718055994531f;
  }
  cluster.sync();   // no CTA leaves while another reads its shared memory
}

template <typename T, int D>
cudaError_t launch_one(const TokensArgs& a, const FewArgs& f, const FewPlan& p, cudaStream_t s) {
  if (p.units * p.cluster > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return launch_after(tokens_few_kernel<T, D>, dim3((unsigned)(p.units * p.cluster)), kThreads, 0, p.cluster, false, s, a, f);
}

}  // namespace

FewPlan few_plan(int64_t B, int64_t rows, bool packed, int H, int64_t n, int64_t tokens, int sms) {
  FewPlan p{};
  p.chunks = (rows + kRows - 1) / kRows;
  p.units = (packed ? rows / kRows + B : B * p.chunks) * H;
  const int64_t tiles = (n + 15) / 16 + (tokens + 15) / 16;
  p.us = 1e30;
  // CTAs of a unit's cluster: its tiles are split while all CTAs are resident together
  // and a warp has more than one tile.
  p.cluster = 1;
  while (p.cluster < kCluster && p.units * p.cluster <= sms && (int64_t)p.cluster * kWarps < tiles) p.cluster *= 2;
  // Taken where all CTAs run at once and this time, from the cases below, is shorter than
  // the tensor-core kernel's (this | that, us): 8 drafted tokens of 24 query heads on 8 on
  // 512 rows 8.7 | 12.2, on 8192 26.1 | 24.5; 8 x 8 tokens, 32 heads, on 2048 rows 29.9 |
  // 25.8, one sequence of 16 on 2048 12.5 | 19.7; 128 tokens of a prompt 9.0 | 8.5, 64 6.4 | 8.3.
  const double warp_tiles = (double)((tiles + p.cluster * kWarps - 1) / (p.cluster * kWarps));
  const int64_t ctas = p.units * p.cluster;
  if (ctas <= 2 * sms && !(packed && B > kThreads))   // (a sequence a thread, in one go)
    p.us = 4.5 + 0.9 * warp_tiles + (p.cluster > 1 ? 1.5 : 0) + (ctas > sms ? 1 + 0.5 * warp_tiles : 0);
  return p;
}

cudaError_t launch_attend_tokens_few(const TokensArgs& a, const FewArgs& f, const FewPlan& p, int D, int dtype, cudaStream_t s) {
  if (dtype == kBf16) return D == 64 ? launch_one<__nv_bfloat16, 64>(a, f, p, s) : launch_one<__nv_bfloat16, 128>(a, f, p, s);
  return D == 64 ? launch_one<__half, 64>(a, f, p, s) : launch_one<__half, 128>(a, f, p, s);
}

}  // namespace kvx
