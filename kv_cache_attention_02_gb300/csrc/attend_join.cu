// attend_join.cu -- joins the parts of an attention over disjoint rows.
//
// A part p is the normalised output o_p of a query head over some rows and the log
// l_p of its sum of e^(s_j):
//   lse = log sum_p e^(l_p),   out = sum_p e^(l_p - lse) o_p.
// A part without rows has l_p = -inf and takes no part, whatever its o_p holds; a head
// with none at all gets out 0 and lse -inf. Weights and sums are fp32; out is rounded
// once (the parts' own roundings to 16 bits are in it, weighted: half a step of each).
//
// Bound by memory: every part is read once and out written once. A lane has 16 bytes
// of a head, of all its parts at once, so that D/8 neighbouring lanes make a head's
// weights out of the same few log sums. Measured on GB300: three parts of 16384 tokens x 32
// heads of 128, bf16, 96 us, 5.7 TB/s (0.84 of the measured copy rate); two of 32 x 32 heads
// 2.0 us, a launch.
#include "attend_tokens.cuh"

namespace kvx {
namespace {

constexpr int kJoinThreads = 256;

template <typename T, int D, int PARTS>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ JoinArgs a) {
  constexpr int L = D / 8;                          // lanes of a head
  const int64_t x = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x, head = x / L;
  const int c = (int)(x % L);
  const bool there = head < (int64_t)a.B * a.S * a.G;
  int64_t at[3];                                    // sequence, token, head
  if (there) {
    const int64_t token = head / a.G;
    at[2] = head - token * a.G;
    at[0] = token / a.S;
    at[1] = token - at[0] * a.S;
  }
  constexpr int MP = PARTS ? PARTS : kMaxJoin;
  float w[MP];
  uint4 v[MP];
  float top = -INFINITY;
  bool lost = false;                                // (fmaxf drops a NaN)
#pragma unroll
  for (int p = 0; p < MP; ++p) {
    const bool on = there && p < a.parts;
    w[p] = on ? a.part_lse[p][head] : -INFINITY;
    v[p] = on ? *reinterpret_cast<const uint4*>(static_cast<const T*>(a.part[p]) + at[0] * a.part_stride[p][0] +
                                                at[1] * a.part_stride[p][1] + at[2] * a.part_stride[p][2] + 8 * c)
              : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int p = 0; p < MP; ++p) {
    lost |= w[p] != w[p];
    top = fmaxf(top, w[p]);
  }
  __syncwarp();                                     // lse may be one of the parts'
  if (!there) return;
  float sum = 0.f, o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll
  for (int p = 0; p < MP; ++p) {
    if (w[p] == -INFINITY) continue;
    const float f = w[p] == top ? 1.f : ex2((w[p] - top) * 1.4426950408889634f);
    sum += f;
    const uint32_t words[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 y = unpack16<T>(words[e]);
      o[2 * e] = fmaf(f, y.x, o[2 * e]);
      o[2 * e + 1] = fmaf(f, y.y, o[2 * e + 1]);
    }
  }
  float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (lost || top == INFINITY) inv = __int_as_float(0x7FFFFFFF);
  T* out = static_cast<T*>(a.out) + at[0] * a.out_stride[0] + at[1] * a.out_stride[1] + at[2] * a.out_stride[2] + 8 * c;
  *reinterpret_cast<uint4*>(out) = make_uint4(pack16<T>(o[0] * inv, o[1] * inv), pack16<T>(o[2] * inv, o[3] * inv),
                                              pack16<T>(o[4] * inv, o[5] * inv), pack16<T>(o[6] * inv, o[7] * inv));
  if (c == 0 && a.lse) a.lse[head] = inv != inv ? inv : sum == 0.f ? -INFINITY : top + logf(sum);
}

template <typename T, int D>
cudaError_t launch_parts(const JoinArgs& a, cudaStream_t s) {
  const int64_t threads = (int64_t)a.B * a.S * a.G * (D / 8), blocks = (threads + kJoinThreads - 1) / kJoinThreads;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks);
  switch (a.parts) {
    case 1:
    case 2: return launch_after(join_kernel<T, D, 2>, grid, kJoinThreads, 0, 1, false, s, a);
    case 3: return launch_after(join_kernel<T, D, 3>, grid, kJoinThreads, 0, 1, false, s, a);
    case 4: return launch_after(join_kernel<T, D, 4>, grid, kJoinThreads, 0, 1, false, s, a);
    default: return launch_after(join_kernel<T, D, 0>, grid, kJoinThreads, 0, 1, false, s, a);
  }
}

}  // namespace

cudaError_t launch_attend_join(const JoinArgs& a, int D, int dtype, cudaStream_t s) {
  if (dtype == kBf16) return D == 64 ? launch_parts<__nv_bfloat16, 64>(a, s) : launch_parts<__nv_bfloat16, 128>(a, s);
  return D == 64 ? launch_parts<__half, 64>(a, s) : launch_parts<__half, 128>(a, s);
}

}  // namespace kvx
