// mma_rows.cuh -- rows of keys and values from memory straight into the registers that
// mma.m16n8k16 wants them in (attend_rows.cu says how), shared by the kernels that attend
// over rows with few query rows (attend_rows.cu, attend_tokens_few.cu).
#pragma once

#include "attend_internal.cuh"

#include <type_traits>

namespace kvx {

// What the weights of the second product are multiplied by: the top of fp16's range
// (65504) is used, with a factor of two to spare.
template <typename T>
constexpr float kWeightLift = std::is_same<T, __half>::value ? 32768.f : 1.f;

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

}  // namespace kvx
