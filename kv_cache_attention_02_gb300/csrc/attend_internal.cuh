// attend_internal.cuh -- structures and helpers shared by the query/key norm
// with rotation (qk_norm_rope.cu), the attention kernels (attend_rows.cu) and
// their entry points (attend.cu, runtime.cu).
#pragma once

#include "kvevict.h"
#include "kvevict_internal.cuh"

#include <cuda_bf16.h>

#include <string>

namespace kvx {

constexpr int kFp16 = KVEVICT_DTYPE_FP16;
constexpr int kBf16 = KVEVICT_DTYPE_BF16;
constexpr int kFp32 = KVEVICT_DTYPE_FP32;

struct QkArgs {
  const void* q;           // element strides between sequences, tokens and heads
  const void* k;
  void* q_out;
  void* k_out;
  int64_t q_stride[3], k_stride[3], qo_stride[3], ko_stride[3];
  const void* q_weight;    // [D] or null: no norm
  const void* k_weight;
  int w_dtype;
  float eps;
  const int32_t* positions;  // [B, S] or null: pos0 + s
  int64_t pos0;
  int B, S, G, H;          // G query heads, H key heads
  int parts, per_part;     // a token's heads go to `parts` warps, per_part heads each
  int runs;                // sequences whose tokens of one position go to one warp
  uint64_t turn[64];       // theta^(-2i/D) / 2 pi, as a 64-bit fraction of a turn
};

struct AttendArgs {
  const void* q;           // [B, G, D]: element strides between sequences and heads
  void* out;
  float* lse;              // [B, G] or null
  const void* k;           // own rows [B, H, n, D]
  const void* v;
  const int32_t* lens;     // [B] or null: n rows each
  const void* k_new;       // the token's own key and value [B, H, D], or null
  const void* v_new;
  const void* pk;          // shared rows [H, P, D]
  const void* pv;
  const int32_t* plens;    // [B] or null: P rows each
  int64_t q_stride[2], out_stride[2], k_stride[3], v_stride[3], kn_stride[2], vn_stride[2], pk_stride[2],
      pv_stride[2];
  const int32_t* pend;     // cache rows with a compaction pending: [B, H] the evicted slot or -1, else null
  const float* rope_c;     // [D/2], the shift by -1 (with pend)
  const float* rope_s;
  int B, G, H, n, P;
  float scale2;            // scale * log2(e): logits in base-2 units
};

// How the prefix kernel's work, the (key head, query block, 128-key tile)
// triples in that order, is cut into one contiguous range per CTA: evenly, or
// (split) each block alone into as many ranges, where that uses nearly as many
// CTAs: a range that begins a second block pays for its start twice. ctas = 0:
// not used.
struct PrefixPlan {
  int ctas, split, pair, blocks, block_rows, nkt, units, final;   // units = H * blocks; final: no own rows to join
  int64_t slots;                // parts that the workspace has room for
  __host__ __device__ int64_t total() const { return (int64_t)units * nkt; }
  __host__ __device__ int64_t start(int c) const {
    if (!split) return c * total() / ctas;
    const int u = c / split;
    return (int64_t)u * nkt + (int64_t)(c - u * split) * nkt / split;
  }
  __host__ __device__ int cta_of(int64_t x) const {
    if (!split) return (int)(((x + 1) * ctas - 1) / total());
    const int u = (int)(x / nkt);
    return u * split + (int)(((x - (int64_t)u * nkt + 1) * split - 1) / nkt);
  }
  // Workspace slot of the part of block u that CTA c computed. Where whole
  // blocks go straight to the output, a CTA leaves at most two parts: one that
  // begins inside a block and one that begins with it.
  __host__ __device__ int64_t slot(int u, int c, bool from_start) const { return final ? 2 * c + from_start : u + c; }
  size_t o_bytes(int D) const;
  size_t bytes(int D) const;
  bool shared_blocks() const;   // whether any block is cut
};
bool prefix_strides_fit(const int64_t* stride, int H, int P, int D);
// Whether the kernel can be launched as it was compiled, on a device below 64 (looked up once).
bool prefix_kernel_ready(int D, int dtype, bool pair, int device);
void prefix_kernel_off(bool off);   // test hook: never ready
// What the row kernel streams beside the prefix's.
struct Streamed {
  int64_t bytes, units;
};
// own: whether there are own rows to join; the workspace does not depend on `stream`.
PrefixPlan prefix_plan(int B, int G, int H, int D, int P, bool own, Streamed stream, int sms);

// The parts of the prefix's attention in the workspace: per slot O as
// [D/4][block_rows] float4 and (m, l) as [block_rows] float2, base-2 units.
struct PrefixParts {
  PrefixPlan plan;
  const float* o;
  const float2* ml;
};

struct PrefixArgs {
  AttendArgs a;
  PrefixPlan plan;
  float* part_o;
  float2* part_ml;
  int* err;                // error word for bounded waits, or null
  int stall;               // test hook: CTA 0's first tile is never issued
  bool k_row_first, v_row_first;
  __host__ __device__ PrefixParts parts() const { return PrefixParts{plan, part_o, part_ml}; }
};
cudaError_t launch_attend_prefix(const PrefixArgs& p, int D, int dtype, cudaStream_t s);

// What a launch needs to know of the current device, looked up once.
struct DeviceInfo {
  int sms = 0;
  int device = 0;
};
int device_info(DeviceInfo* out);   // KVEVICT_* code; sets the last error
void set_last_error(const std::string& msg);

cudaError_t launch_qk_norm_rope(QkArgs a, int D, int in_dtype, int out_dtype, int sms, cudaStream_t s);

// How the row kernel's work is cut: with ctas > 0 all units' tiles in a row, one
// contiguous range per CTA; otherwise a cluster per unit.
struct RowsPlan {
  int ctas, qchunks, qn, final;   // a unit: qn query heads of a key head, qchunks units; final: no prefix parts to join
  int batch;
  int64_t units;
  int64_t* first;                 // [B + 1], unequal lengths: the first tile of each sequence, their total
  float* part_o;                  // [slot][qn][D]
  float2* part_ml;                // [slot][qn] maximum (base 2) and sum
  __host__ __device__ int64_t slot(int64_t u, int c, bool from_start) const { return final ? 2 * c + from_start : u + c; }
  int64_t slots;                  // parts that the workspace has room for
  size_t o_bytes(int D) const;
  size_t ml_bytes() const;
  size_t bytes(int D) const;
};
// prefix_parts: the prefix's kernel runs beside it.
RowsPlan rows_plan(int B, int G, int H, int D, int n, int P, bool has_new, bool pend, bool prefix_parts, int sms);
int stream_ctas(int D, int sms);   // resident on so many SMs
// parts.plan.ctas > 0: joins the prefix's parts too (a.P is 0 then).
cudaError_t launch_attend_rows(const AttendArgs& a, const PrefixParts& parts, const RowsPlan& plan, int D, int dtype,
                               int sms, cudaStream_t s);

// Checks the caller's description and fills the kernel's; own rows come from
// `rows` (a handle's layer) where that is not null.
struct CacheRows {
  const void* k;
  const void* v;
  int64_t stride[3];
  int n;
  const int32_t* pend;
  const float* rope_c;
  const float* rope_s;
  int batch, n_kv_heads, head_dim;
  int* err;                // the handle's error word
};
int attend_run(const kvevict_attention* d, const CacheRows* rows, cudaStream_t s);

// A launch in clusters of `cluster` CTAs; overlap: it may begin before the kernel
// launched before it on the stream has ended (that one calls launch_dependents,
// this one wait_for_primary before it uses its results).
template <typename... K, typename... A>
cudaError_t launch_after(void (*kernel)(K...), dim3 grid, int threads, size_t smem, int cluster, bool overlap,
                         cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  cfg.attrs = at;
  if (cluster > 1) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs].val.clusterDim.x = cluster;
    at[cfg.numAttrs].val.clusterDim.y = 1;
    at[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  if (overlap) {
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---------------------------------------------------------------- device helpers
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// 16 bytes that no later access of this SM wants: past L1.
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

template <typename T>
__device__ __forceinline__ float2 unpack16(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack16<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack16<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace kvx
