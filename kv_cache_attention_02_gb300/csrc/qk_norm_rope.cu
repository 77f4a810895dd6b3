// qk_norm_rope.cu -- RMS norm of each query and key head and the rotation to
// the token's position, in one pass.
//
//   y = x * w / sqrt(mean(x^2) + eps)            (skipped without a weight)
//   (y_i, y_{i+D/2}) -> (y_i c - y_{i+D/2} s, y_i s + y_{i+D/2} c),
//   c, s = cos, sin(p * theta^(-2i/D)): the half-split convention the cache's
//   re-rotation uses (page "veloxquant_mlx.quantizers.keyformer module",
//   KeyformerState.rope_base).
//
// Bound by memory: each element is read once and written once, and the norm,
// the weight and the rotation stay in fp32 registers; the one rounding is the
// store's. D/16 lanes share a head, each with the two 8-element chunks that
// its rotation pairs need, so the sum of squares is three (D = 128) or two
// shuffles and no partner value crosses lanes.
//
// Angles: the turn count p * w / 2 pi is taken modulo 1 in 64-bit fixed point
// (one integer product; the fraction is exact up to p * 2^-65 plus the 2^-53
// of the frequency itself: within 2^-21 rad at the farthest positions, +-2^31), and
// no fp64 instruction runs. The lanes of a warp compute a token's D/2 angles once
// between them, then take the warp's heads of that token with them.
//
// Measured on GB300: 32 x 4096 tokens of 40 heads of 128, bf16, 414-418 us, 6.4-6.5
// TB/s (0.95 of the measured copy rate); 3 x 1021 fp32 tokens of 32 heads 17.1 us, 4.4
// TB/s, 4 us of it launch and first loads (13.5 us with its 75 MB in L2); one token of 8
// heads 4.3 us.
#include "kvevict_internal.cuh"
#include "attend_internal.cuh"

namespace kvx {
namespace {

constexpr int kQkThreads = 256;
constexpr int kQkCtas = 3;     // CTAs an SM

template <typename T>
struct Chunk8;   // 8 consecutive elements
template <>
struct Chunk8<__half> {
  uint4 r;
  __device__ __forceinline__ void load(const __half* p) { r = ld_stream16(p); }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack16<__half>(w[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
};
template <>
struct Chunk8<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = ld_stream16(p); }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack16<__nv_bfloat16>(w[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
};
template <>
struct Chunk8<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = ld_stream16(p);
    b = ld_stream16(p + 4);
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
    f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
    f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
  }
};

__device__ __forceinline__ float weight_at(const void* w, int dtype, int i) {
  if (dtype == kFp32) return static_cast<const float*>(w)[i];
  if (dtype == kBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
  return __half2float(static_cast<const __half*>(w)[i]);
}

// RUNS: several sequences a unit (a loop more; 3% of the call with 40 heads).
template <typename TI, typename TO, int D, bool RUNS>
__global__ void __launch_bounds__(kQkThreads, kQkCtas) qk_norm_rope_kernel(const QkArgs a) {
  constexpr int LPH = D / 16;            // lanes of a head
  constexpr int HPW = 32 / LPH;          // heads a warp takes at a time
  constexpr int APL = 8 / HPW;           // angles a lane computes
  constexpr int kAhead = sizeof(TI) == 4 ? 1 : 2;   // groups of heads whose loads are under way (32 bytes a lane each in fp32)
  __shared__ float w_s[2][D];
  __shared__ uint64_t turn_s[D / 2];
  const int tid = threadIdx.x, lane = tid & 31;
  const int c = lane % LPH, sub = lane / LPH;
  for (int i = tid; i < D; i += kQkThreads) {
    w_s[0][i] = a.q_weight ? weight_at(a.q_weight, a.w_dtype, i) : 1.f;
    w_s[1][i] = a.k_weight ? weight_at(a.k_weight, a.w_dtype, i) : 1.f;
  }
  for (int i = tid; i < D / 2; i += kQkThreads) turn_s[i] = a.turn[i];
  __syncthreads();

  const int heads = a.G + a.H;
  // a unit: `runs` sequences' tokens of one position (one token where the caller
  // gives positions), per_part of their heads
  const int64_t chunks = (a.B + a.runs - 1) / a.runs, units = a.S * chunks * a.parts;
  const int64_t step = (int64_t)gridDim.x * (kQkThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kQkThreads / 32) + (tid >> 5); u < units; u += step) {
    const int64_t rest = u / a.parts;
    const int part = (int)(u - rest * a.parts);
    const int64_t chunk = rest / a.S, s = rest - chunk * a.S;
    const int b0 = (int)chunk * (RUNS ? a.runs : 1), b_end = RUNS ? min(a.B, b0 + a.runs) : b0 + 1;
    const int h0 = part * a.per_part + sub, h_end = min(heads, (part + 1) * a.per_part);
    const TI* const qs = static_cast<const TI*>(a.q) + b0 * a.q_stride[0] + s * a.q_stride[1] + 8 * c;
    const TI* const ks = static_cast<const TI*>(a.k) + b0 * a.k_stride[0] + s * a.k_stride[1] + 8 * c;
    TO* const qd = static_cast<TO*>(a.q_out) + b0 * a.qo_stride[0] + s * a.qo_stride[1] + 8 * c;
    TO* const kd = static_cast<TO*>(a.k_out) + b0 * a.ko_stride[0] + s * a.ko_stride[1] + 8 * c;
    auto src = [&](int b, int h) {
      const TI* p = h < a.G ? qs + (int64_t)h * a.q_stride[2] : ks + (int64_t)(h - a.G) * a.k_stride[2];
      return RUNS ? p + (b - b0) * (h < a.G ? a.q_stride[0] : a.k_stride[0]) : p;
    };
    // kAhead groups of heads under way: the loads of one ahead of the others' arithmetic
    Chunk8<TI> lo[kAhead], hi[kAhead];
    int fb = b0, fh = h0;                // the next to load
    auto next = [&](int& b, int& h) {
      h += HPW;
      if (RUNS && h - sub >= h_end) {
        h = h0;
        ++b;
      }
    };
    auto fetch = [&](int k) {
      if ((!RUNS || fb < b_end) && fh < h_end) {
        const TI* p = src(fb, fh);
        lo[k].load(p);
        hi[k].load(p + D / 2);
      }
      next(fb, fh);
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      lo[k] = {};
      hi[k] = {};
      fetch(k);
    }
    // the position's angles: lane (c, sub) computes pairs 8c + sub*APL .. + APL - 1
    const int64_t pos = a.positions ? (int64_t)a.positions[(int64_t)b0 * a.S + s] : a.pos0 + s;
    float cs[8], sn[8];
    {
      float mc[APL], ms[APL];
#pragma unroll
      for (int j = 0; j < APL; ++j) {
        const uint64_t t = (uint64_t)pos * turn_s[8 * c + sub * APL + j];
        sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &ms[j], &mc[j]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cs[i] = __shfl_sync(~0u, mc[i % APL], (i / APL) * LPH + c);
        sn[i] = __shfl_sync(~0u, ms[i % APL], (i / APL) * LPH + c);
      }
    }
    int b = b0, h = h0;
    auto done = [&] { return RUNS ? b >= b_end : h - sub >= h_end; };
    while (!done()) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (done()) break;
        float x[8], y[8];
        lo[k].get(x);
        hi[k].get(y);
        const bool live = h < h_end;
        fetch(k);
        const int kind = h < a.G ? 0 : 1;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
        for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(~0u, ss, o);
        if (kind ? a.k_weight != nullptr : a.q_weight != nullptr) {
          const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = x[i] * r * w_s[kind][8 * c + i];
            y[i] = y[i] * r * w_s[kind][D / 2 + 8 * c + i];
          }
        }
        if (live) {
          uint32_t ol[4], oh[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = 2 * i;
            ol[i] = pack16<TO>(x[e] * cs[e] - y[e] * sn[e], x[e + 1] * cs[e + 1] - y[e + 1] * sn[e + 1]);
            oh[i] = pack16<TO>(x[e] * sn[e] + y[e] * cs[e], x[e + 1] * sn[e + 1] + y[e + 1] * cs[e + 1]);
          }
          TO* d = kind ? kd + (int64_t)(h - a.G) * a.ko_stride[2] : qd + (int64_t)h * a.qo_stride[2];
          if (RUNS) d += (b - b0) * (kind ? a.ko_stride[0] : a.qo_stride[0]);
          *reinterpret_cast<uint4*>(d) = make_uint4(ol[0], ol[1], ol[2], ol[3]);
          *reinterpret_cast<uint4*>(d + D / 2) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
        }
        next(b, h);
      }
    }
  }
}

template <typename TI, typename TO, bool RUNS>
cudaError_t launch_d(const QkArgs& a, int D, unsigned grid, cudaStream_t s) {
  if (D == 64)
    qk_norm_rope_kernel<TI, TO, 64, RUNS><<<grid, kQkThreads, 0, s>>>(a);
  else
    qk_norm_rope_kernel<TI, TO, 128, RUNS><<<grid, kQkThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename TI, typename TO>
cudaError_t launch_r(const QkArgs& a, int D, unsigned grid, cudaStream_t s) {
  return a.runs > 1 ? launch_d<TI, TO, true>(a, D, grid, s) : launch_d<TI, TO, false>(a, D, grid, s);
}

template <typename TI>
cudaError_t launch_o(const QkArgs& a, int D, int out_dtype, unsigned grid, cudaStream_t s) {
  return out_dtype == kBf16 ? launch_r<TI, __nv_bfloat16>(a, D, grid, s) : launch_r<TI, __half>(a, D, grid, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(QkArgs a, int D, int in_dtype, int out_dtype, int sms, cudaStream_t s) {
  const int hpw = 512 / D;   // heads a warp takes at a time
  const int64_t tokens = (int64_t)a.B * a.S;
  const int heads = a.G + a.H;
  // Units for every resident warp twice over: a token's heads are spread over
  // warps while there are fewer tokens. With few heads several sequences' tokens
  // of one position go to one warp, which computes their angles once (where
  // positions are pos0 + s): 64 x 4096 tokens of 4 + 4 heads, D = 64, 148 -> 102
  // us; with 40 heads the angles cost nothing, and this order of the rows 4%.
  const int groups = (heads + hpw - 1) / hpw;
  const int64_t goal = (int64_t)2 * sms * kQkCtas * (kQkThreads / 32);
  const int parts = (int)std::min<int64_t>((goal + tokens - 1) / tokens, groups);
  a.per_part = (groups + parts - 1) / parts * hpw;
  a.parts = (heads + a.per_part - 1) / a.per_part;
  a.runs = a.positions ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>({tokens / goal, 8 / groups, a.B}));
  const int64_t units = (int64_t)a.S * ((a.B + a.runs - 1) / a.runs) * a.parts;
  const int64_t blocks = (units + kQkThreads / 32 - 1) / (kQkThreads / 32);
  const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)sms * kQkCtas);
  if (in_dtype == kFp32) return launch_o<float>(a, D, out_dtype, grid, s);
  if (in_dtype == kBf16) return launch_o<__nv_bfloat16>(a, D, out_dtype, grid, s);
  return launch_o<__half>(a, D, out_dtype, grid, s);
}

}  // namespace kvx
