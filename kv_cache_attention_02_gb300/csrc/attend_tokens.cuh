// attend_tokens.cuh -- structures shared by the attention of several query tokens a
// sequence (attend_tokens.cu), its joins (attend_join.cu) and their entry points
// (attend_tokens_entry.cu, runtime.cu).
#pragma once

#include "attend_internal.cuh"

namespace kvx {

struct TokensArgs {
  const void* q;           // element strides between sequences, tokens and heads
  void* out;
  float* lse;              // [B, S, G] (packed: [T, G]) or null
  const void* v_new;
  int64_t q_stride[3], out_stride[3], vn_stride[3];
  const int32_t* starts;   // [B + 1] first token of each sequence, or null
  const int32_t* new_lens; // [B] tokens of each sequence, or null: S each
  const int32_t* parents;  // [B, S] tree, or null: causal
  int64_t parents_stride;
  const int32_t* lens;     // [B] own rows, or null: n each
  const int32_t* pend;     // [B, H] the evicted slot still in place, or -1; or null
  const float* rope_c;     // [D/2], the shift by -1 (with pend)
  const float* rope_s;
  int B, S, G, H, n;       // S: tokens of a sequence, or in all with starts
  float scale2;            // scale * log2(e): logits in base-2 units
};

// One CTA's start: a key tile of a block of query rows.
struct TokensAt {
  int b, h, i, k;
};

// How the work, the (sequence, key head, block of query rows, 128-key tile) in that
// order, is cut into one contiguous range per CTA, evenly by cost. Costs have a closed
// form (half a block's tiles and a constant for the start of a block), so that every CTA
// finds its range itself.
struct TokensPlan {
  int ctas, pair, block_rows;
  int whole;               // ranges begin and end with blocks: no parts to join
  int even;                // (with whole) every block costs the same
  size_t o_bytes(int D) const { return (size_t)2 * ctas * block_rows * D * 4; }
  size_t ml_bytes() const { return (size_t)2 * ctas * block_rows * 8; }
  size_t bytes(int D) const { return whole ? 0 : o_bytes(D) + ml_bytes() + (size_t)(ctas + 1) * sizeof(TokensAt); }
};
// rows: of a sequence's matrix of query rows (tokens x query heads of a key head), at most.
TokensPlan tokens_plan(int B, int64_t rows, int64_t blocks, int H, int64_t tiles, int sms);

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
  TokensRows k, v, k_new, v_new;
  void* workspace;
  int* err;                // error word for bounded waits, or null
  int stall;               // test hook: CTA 0's first tile is never issued
};
bool tokens_kernel_ready(int D, int dtype, bool pair, int device);
cudaError_t launch_attend_tokens(const TokensLaunch& l, int D, int dtype, cudaStream_t s);
int tokens_run(const kvevict_tokens* d, bool tree, const CacheRows* rows, cudaStream_t s);

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

}  // namespace kvx
