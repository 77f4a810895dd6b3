// attend_tokens.cuh -- structures shared by the attention of several query tokens a
// sequence (attend_tokens.cu), its joins (attend_join.cu) and their entry points
// (attend_tokens_entry.cu, runtime.cu).
#pragma once

#include "attend_internal.cuh"

namespace kvx {

struct TokensArgs {
  void* out;               // element strides between sequences, tokens and heads
  float* lse;              // [B, S, G] (packed: [T, G]) or null
  const void* v_new;
  int64_t out_stride[3], vn_stride[3];
  const int32_t* starts;   // [B + 1] first token of each sequence, or null
  const int32_t* new_lens; // [B] tokens of each sequence, or null: S each
  const int32_t* parents;  // [B, S] tree, or null: causal
  int64_t parents_stride;
  const int32_t* lens;     // [B] own rows, or null: n each
  const int32_t* pend;     // [B, H] the evicted slot still in place, or -1; or null
  const float* rope_c;     // [D/2], the shift by -1 (with pend)
  const float* rope_s;
  int B, S, G, n;          // S: tokens of a sequence, or in all with starts
  // Query heads are dealt to `heads` groups of N <= 128, a key head's to `groups` of them
  // (one, but for more than 128 query heads a key head); half a block of query rows is
  // `half` = 128 / N (split: 64 / N) tokens of one.
  int N, heads, groups, half;
  float scale2;            // scale * log2(e): logits in base-2 units
};

// One CTA's start: a key tile of a block of query rows.
struct TokensAt {
  int b, h, i, k;
};

// How the work, the (sequence, head group, block of query rows, 128-key tile) in that
// order, is cut into one contiguous range per CTA, evenly by cost. Costs have a closed
// form, about half a block's tiles and a constant for its start, so that every CTA finds
// its range itself.
struct TokensPlan {
  int ctas, pair, split, block_rows;
  int whole;               // ranges begin and end with blocks: no parts to join
  int even;                // (with whole) every block costs the same
  double per_cta;          // 1 / ctas
  double us;               // the call's time, about
  size_t o_bytes(int D) const { return (size_t)2 * ctas * block_rows * D * 4; }
  size_t ml_bytes() const { return (size_t)2 * ctas * block_rows * 8; }
  size_t bytes(int D) const { return whole ? 0 : o_bytes(D) + ml_bytes() + (size_t)(ctas + 1) * sizeof(TokensAt); }
};
// pair: no sequence has more than half a block; split: of at most 64 query rows. blocks: of all sequences in one head group,
// at most; tiles, mean: of a block, at most and on average.
TokensPlan tokens_plan(bool pair, bool split, int64_t blocks, int heads, int64_t tiles, int64_t mean, int sms);

// Rows [batch, head, row] as TMA sees them.
struct TokensRows {
  const void* base;
  int64_t stride[3];       // between sequences, heads and rows
  int B, H;
  int64_t rows;
};

struct TokensLaunch {
  TokensArgs a;
  TokensPlan plan;
  TokensRows q, out, k, v, k_new, v_new;   // (q's and out's rows are tokens)
  bool out_fits;           // a tensor map can describe out
  void* workspace;
  int* err;                // error word for bounded waits, or null
  int stall;               // test hook: CTA 0's first tile is never issued
};
// Whether the kernel can be launched as it was compiled, on a device below 64 (looked up once).
bool tokens_kernel_ready(int D, int dtype, const TokensPlan& plan, int device);
void tokens_kernel_off(bool off);   // test hook: never ready
cudaError_t launch_attend_tokens(const TokensLaunch& l, int D, int dtype, cudaStream_t s);
int tokens_run(const kvevict_tokens* d, bool tree, const CacheRows* rows, cudaStream_t s);

// The kernel for few query rows (attend_tokens_few.cu). It answers any call, one of many
// rows slowly.
struct FewArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* k_new;
  int64_t q_stride[3], kn_stride[3];   // between sequences, tokens and heads
  int64_t k_stride[3], v_stride[3];    // between sequences, heads and rows
  int H, chunks;                       // chunks of 16 query rows of a sequence's key head
};
struct FewPlan {
  int64_t units, chunks;
  int cluster;
  double us;               // the call's time, about; infinite where its CTAs do not all run at once
};
FewPlan few_plan(int64_t B, int64_t rows, bool packed, int H, int64_t n, int64_t tokens, int sms);
cudaError_t launch_attend_tokens_few(const TokensArgs& a, const FewArgs& f, const FewPlan& p, int D, int dtype, cudaStream_t s);

constexpr int kMaxJoin = KVEVICT_MAX_JOIN;
struct JoinArgs {
  const void* part[kMaxJoin];
  const float* part_lse[kMaxJoin];
  int64_t part_stride[kMaxJoin][3];   // between sequences, tokens and heads
  void* out;
  float* lse;
  int64_t out_stride[3];
  int B, S, G, parts;
};
cudaError_t launch_attend_join(const JoinArgs& a, int D, int dtype, cudaStream_t s);

// ---------------------------------------------------------------- device helpers
struct Seq {
  int tok0, nq, n, ta;     // first token (packed), tokens, own rows, their tiles of 128
};
__device__ __forceinline__ Seq load_seq(const TokensArgs& a, int b) {
  Seq s;
  s.tok0 = 0;
  s.nq = a.S;
  if (a.starts) {
    s.tok0 = max(0, min(a.starts[b], a.S));
    s.nq = max(0, min(a.starts[b + 1], a.S) - s.tok0);
  } else if (a.new_lens) {
    s.nq = max(0, min(a.new_lens[b], a.S));
  }
  s.n = a.lens ? max(0, min(a.lens[b], a.n)) : a.n;
  s.ta = (s.n + (a.pend ? 1 : 0) + 127) / 128;     // an evicted row may still be in place
  return s;
}

// Bits of any 16-bit float in a word whose exponent is all ones: NaN or infinity.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return std::is_same<T, __half>::value ? ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u
                                        : ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
template <typename T>
__device__ __forceinline__ uint32_t drop_not_finite(uint32_t w) {
  const uint32_t f = not_finite<T>(w);
  return (f & 0x8000u ? 0u : w & 0xFFFFu) | (f & 0x80000000u ? 0u : w & 0xFFFF0000u);
}

// Ancestors of the tokens lane and lane + 32 of sequence b, themselves included, as
// bits (warp-collective): powers of two of the step to the parent.
__device__ __forceinline__ void ancestors(const TokensArgs& a, int b, int nq, uint64_t (&m)[2]) {
  const int lane = threadIdx.x & 31;
  const int32_t* parents = a.parents + b * a.parents_stride;
  int p[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int t = lane + 32 * x;
    p[x] = t < nq ? parents[t] : -1;
    if (p[x] >= t) p[x] = -1;                        // not before it: none
    m[x] = 1ull << t;
  }
#pragma unroll 1
  for (int step = 1; step < nq; step *= 2) {
    uint64_t um[2];
    int up[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint64_t m0 = __shfl_sync(~0u, m[0], p[x] & 31), m1 = __shfl_sync(~0u, m[1], p[x] & 31);
      const int p0 = __shfl_sync(~0u, p[0], p[x] & 31), p1 = __shfl_sync(~0u, p[1], p[x] & 31);
      um[x] = p[x] < 0 ? m[x] : m[x] | (p[x] < 32 ? m0 : m1);
      up[x] = p[x] < 0 ? -1 : p[x] < 32 ? p0 : p1;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      m[x] = um[x];
      p[x] = up[x];
    }
  }
}

}  // namespace kvx
