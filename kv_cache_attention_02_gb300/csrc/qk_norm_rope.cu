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
// of the frequency itself), so far positions lose nothing and no fp64
// instruction runs. The lanes of a warp compute a token's D/2 angles once
// between them, then take the warp's heads of that token with them.
#include "kvevict_internal.cuh"
#include "attend_internal.cuh"

namespace kvx {
namespace {

constexpr int kQkThreads = 256;

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

template <typename TI, typename TO, int D>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_kernel(const QkArgs a) {
  constexpr int LPH = D / 16;            // lanes of a head
  constexpr int HPW = 32 / LPH;          // heads a warp takes at a time
  constexpr int APL = 8 / HPW;           // angles a lane computes
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
  const int64_t units = (int64_t)a.B * a.S * a.parts;
  const int64_t step = (int64_t)gridDim.x * (kQkThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kQkThreads / 32) + (tid >> 5); u < units; u += step) {
    const int64_t token = u / a.parts;
    const int part = (int)(u - token * a.parts);
    const int64_t b = token / a.S, s = token - b * a.S;
    const int h_end = min(heads, (part + 1) * a.per_part);
    const TI* qb = static_cast<const TI*>(a.q) + b * a.q_stride[0] + s * a.q_stride[1];
    const TI* kb = static_cast<const TI*>(a.k) + b * a.k_stride[0] + s * a.k_stride[1];
    TO* qo = static_cast<TO*>(a.q_out) + b * a.qo_stride[0] + s * a.qo_stride[1];
    TO* ko = static_cast<TO*>(a.k_out) + b * a.ko_stride[0] + s * a.ko_stride[1];
    auto src = [&](int h) {
      return (h < a.G ? qb + (int64_t)h * a.q_stride[2] : kb + (int64_t)(h - a.G) * a.k_stride[2]) + 8 * c;
    };
    int h = part * a.per_part + sub;
    Chunk8<TI> lo{}, hi{};
    if (h < h_end) {
      const TI* p = src(h);
      lo.load(p);
      hi.load(p + D / 2);
    }
    // the token's angles: lane (c, sub) computes pairs 8c + sub*APL .. + APL - 1
    const int64_t pos = a.positions ? (int64_t)a.positions[token] : a.pos0 + s;
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
    for (int h0 = part * a.per_part; h0 < h_end; h0 += HPW) {
      float x[8], y[8];
      lo.get(x);
      hi.get(y);
      const bool live = h < h_end;
      const int hn = h + HPW;
      if (hn < h_end) {                    // the next heads' loads, ahead of this pass's arithmetic
        const TI* p = src(hn);
        lo.load(p);
        hi.load(p + D / 2);
      }
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
        TO* d = (kind ? ko + (int64_t)(h - a.G) * a.ko_stride[2] : qo + (int64_t)h * a.qo_stride[2]) + 8 * c;
        *reinterpret_cast<uint4*>(d) = make_uint4(ol[0], ol[1], ol[2], ol[3]);
        *reinterpret_cast<uint4*>(d + D / 2) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
      }
      h = hn;
    }
  }
}

template <typename TI, typename TO>
cudaError_t launch_d(const QkArgs& a, int D, unsigned grid, cudaStream_t s) {
  if (D == 64)
    qk_norm_rope_kernel<TI, TO, 64><<<grid, kQkThreads, 0, s>>>(a);
  else
    qk_norm_rope_kernel<TI, TO, 128><<<grid, kQkThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename TI>
cudaError_t launch_o(const QkArgs& a, int D, int out_dtype, unsigned grid, cudaStream_t s) {
  return out_dtype == kBf16 ? launch_d<TI, __nv_bfloat16>(a, D, grid, s) : launch_d<TI, __half>(a, D, grid, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(QkArgs a, int D, int in_dtype, int out_dtype, int sms, cudaStream_t s) {
  const int hpw = 512 / D;   // heads a warp takes at a time
  const int64_t tokens = (int64_t)a.B * a.S;
  const int heads = a.G + a.H;
  // With few tokens a token's heads are spread over warps (the call is one
  // latency); with many, one warp takes all of a token's heads and computes
  // its angles once.
  const bool spread = tokens < (int64_t)sms * 32;
  a.per_part = spread ? hpw : heads;
  a.parts = (heads + a.per_part - 1) / a.per_part;
  const int64_t units = tokens * a.parts;
  const int64_t blocks = (units + kQkThreads / 32 - 1) / (kQkThreads / 32);
  const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)sms * 8);
  if (in_dtype == kFp32) return launch_o<float>(a, D, out_dtype, grid, s);
  if (in_dtype == kBf16) return launch_o<__nv_bfloat16>(a, D, out_dtype, grid, s);
  return launch_o<__half>(a, D, out_dtype, grid, s);
}

}  // namespace kvx
