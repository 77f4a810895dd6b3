// attend_tokens_entry.cu -- the entry points kvevict_attend_prompt, kvevict_attend_tree,
// kvevict_attend_tokens_workspace and kvevict_attend_join of include/kvevict.h: argument
// checks and dispatch. Host code only; nothing on the device is touched before the checks
// pass.
#include "attend_tokens.cuh"
#include "entry.cuh"

#include <atomic>
#include <cmath>

namespace kvx {
namespace {

std::atomic<bool> g_without_few{false};   // test hook

int tokens_check(const kvevict_tokens* d, bool tree) {
  if (!d) return invalid("args must not be null");
  if (!is16(d->dtype)) return invalid("dtype must be KVEVICT_DTYPE_FP16 or _BF16");
  if (d->batch < 0 || d->seq < 0) return invalid("batch and seq must be >= 0");
  if (d->n_kv_heads < 1 || d->n_heads < 1 || d->n_heads % d->n_kv_heads != 0)
    return invalid("n_heads must be a positive multiple of n_kv_heads");
  if (d->head_dim != 64 && d->head_dim != 128) return invalid("head_dim must be 64 or 128");
  if (d->n < 0 || (int64_t)d->n + d->seq >= (1 << 30)) return invalid("n must be >= 0, and n and seq below 2^30 together");
  if ((int64_t)d->batch * d->n_heads > (1 << 26)) return invalid("batch * n_heads must be at most 2^26");
  if ((int64_t)d->seq * (d->n_heads / d->n_kv_heads) > (1 << 30))
    return invalid("seq * n_heads / n_kv_heads must be at most 2^30");
  // more than 2^127 could overflow with the factor log2(e)
  if (d->scale != 0.f && !(d->scale >= 0x1p-126f && d->scale <= 0x1p127f))
    return invalid("scale must be 0, or from 2^-126 to 2^127");
  if (d->reserved || d->reserved2) return invalid("reserved must be 0");
  if (d->starts && d->new_lens) return invalid("starts and new_lens must not be given together");
  if (tree && d->seq > KVEVICT_MAX_TREE) return invalid("a tree has at most 64 tokens");
  if (tree && d->starts) return invalid("starts must be null for trees");
  if (!tree && d->parents) return invalid("parents must be null for prompts");
  return KVEVICT_OK;
}

// What TMA can describe: rows apart, strides of 0 .. 2^40 bytes.
bool map_strides_fit(const int64_t (&s)[3], int B, int H, int64_t rows, int row, int D) {
  const int64_t top = (int64_t)1 << 39;
  const int head = row == 1 ? 2 : 1;
  return (B <= 1 || (s[0] >= 0 && s[0] < top)) && (H <= 1 || (s[head] >= 0 && s[head] < top)) &&
         (rows <= 1 || (s[row] >= D && s[row] < top));
}

// Query heads of a key head in groups of at most 128.
int head_groups(int N) {
  int c = 1;
  while (N % c || N / c > 128) ++c;
  return c;
}

TokensPlan plan_of(const kvevict_tokens* d, int64_t n, const DeviceInfo& dev) {
  const int all = d->n_heads / d->n_kv_heads, groups = head_groups(all), N = all / groups;
  const bool split = (int64_t)d->seq * N <= 64, pair = split || d->seq <= 128 / N;
  const int half = (split ? 64 : 128) / N;
  const int64_t per = pair ? half : 2 * half;
  const int64_t blocks = d->starts ? d->seq / per + d->batch : d->batch * ((d->seq + per - 1) / per);
  const int64_t own = (n + 127) / 128, top = (d->seq + 127) / 128;
  const int64_t tokens = d->starts ? d->seq / std::max(1, d->batch) : d->seq;   // of a sequence, about
  return tokens_plan(pair, split, blocks, d->n_kv_heads * groups, own + top, own + ((tokens + 127) / 128 + 1) / 2, dev.sms);
}

}  // namespace

int tokens_run(const kvevict_tokens* d, bool tree, const CacheRows* rows, cudaStream_t s) {
  if (int rc = tokens_check(d, tree)) return rc;
  if (rows) {
    if (d->dtype != kFp16) return invalid("a handle's rows are fp16: dtype must be KVEVICT_DTYPE_FP16");
    if (d->batch != rows->batch || d->n_kv_heads != rows->n_kv_heads || d->head_dim != rows->head_dim)
      return invalid("batch, n_kv_heads and head_dim must be the handle's");
    if (d->n != 0 || d->k || d->v || d->lens) return invalid("n, k, v and lens must be 0 and null with a handle's rows");
  }
  if (d->batch == 0 || d->seq == 0) return KVEVICT_OK;
  if (!d->q || !d->out || !d->k_new || !d->v_new) return invalid("q, out, k_new and v_new must not be null");
  if (d->n > 0 && (!d->k || !d->v)) return invalid("k and v must not be null with n > 0");
  const int D = d->head_dim, B = d->starts ? 1 : d->batch;          // sequences that strides are for
  const int32_t qx[3] = {B, d->seq, d->n_heads}, nx[3] = {B, d->seq, d->n_kv_heads}, kx[3] = {d->batch, d->n_kv_heads, d->n};
  if (!aligned(d->q) || !aligned(d->out) || !strides16(d->q_stride, qx, 2) || !strides16(d->out_stride, qx, 2))
    return invalid("q and out must be 16-byte aligned, with strides of multiples of 16 bytes");
  if (rows_overlap(d->out_stride, qx, D)) return invalid("the rows of out must not overlap: strides of at least head_dim");
  if (!aligned(d->k_new) || !aligned(d->v_new) || !strides16(d->k_new_stride, nx, 2) || !strides16(d->v_new_stride, nx, 2))
    return invalid("k_new and v_new must be 16-byte aligned, with strides of multiples of 16 bytes");
  if (d->n > 0 && (!aligned(d->k) || !aligned(d->v) || !strides16(d->k_stride, kx, 2) || !strides16(d->v_stride, kx, 2)))
    return invalid("k and v must be 16-byte aligned, with strides of multiples of 16 bytes");
  if (!map_strides_fit(d->k_new_stride, B, d->n_kv_heads, d->seq, 1, D) ||
      !map_strides_fit(d->v_new_stride, B, d->n_kv_heads, d->seq, 1, D) ||
      (d->n > 0 && (!map_strides_fit(d->k_stride, d->batch, d->n_kv_heads, d->n, 2, D) ||
                    !map_strides_fit(d->v_stride, d->batch, d->n_kv_heads, d->n, 2, D))))
    return invalid("strides of keys and values must be >= 0, between tokens and rows at least head_dim, and below 2^39");
  if (!map_strides_fit(d->q_stride, B, d->n_heads, d->seq, 1, D) || (d->n_heads > 1 && d->q_stride[2] < D))
    return invalid("strides of q must be >= 0, between tokens and heads at least head_dim, and below 2^39");
  if (!aligned(d->lse, 4) || !aligned(d->starts, 4) || !aligned(d->new_lens, 4) || !aligned(d->parents, 4) || !aligned(d->lens, 4))
    return invalid("lse, starts, new_lens, parents and lens must be 4-byte aligned");
  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  TokensLaunch l{};
  TokensArgs& a = l.a;
  a.out = d->out;
  a.lse = d->lse;
  a.v_new = d->v_new;
  a.starts = d->starts;
  a.new_lens = d->new_lens;
  a.parents = d->parents;
  a.parents_stride = d->parents_stride;
  a.B = d->batch;
  a.S = d->seq;
  a.G = d->n_heads;
  a.groups = head_groups(d->n_heads / d->n_kv_heads);
  a.heads = d->n_kv_heads * a.groups;
  a.N = a.G / a.heads;
  for (int i = 0; i < 3; ++i) {
    const bool on = i > 0 || !d->starts;                              // packed: no stride between sequences
    a.out_stride[i] = on ? d->out_stride[i] : 0;
    a.vn_stride[i] = on ? d->v_new_stride[i] : 0;
  }
  l.q = TokensRows{d->q, {d->q_stride[0], d->q_stride[2], d->q_stride[1]}, B, a.G, a.S};
  l.out = TokensRows{d->out, {d->out_stride[0], d->out_stride[2], d->out_stride[1]}, B, a.G, a.S};
  l.out_fits = map_strides_fit(d->out_stride, B, d->n_heads, d->seq, 1, D) && (d->n_heads == 1 || d->out_stride[2] >= D) &&
               (B == 1 || d->out_stride[0] >= D);
  l.k_new = TokensRows{d->k_new, {d->k_new_stride[0], d->k_new_stride[2], d->k_new_stride[1]}, B, d->n_kv_heads, a.S};
  l.v_new = TokensRows{d->v_new, {d->v_new_stride[0], d->v_new_stride[2], d->v_new_stride[1]}, B, d->n_kv_heads, a.S};
  if (rows) {
    a.n = rows->n;
    a.pend = rows->pend;
    a.rope_c = rows->rope_c;
    a.rope_s = rows->rope_s;
    l.k = TokensRows{rows->k, {rows->stride[0], rows->stride[1], rows->stride[2]}, a.B, d->n_kv_heads, (int64_t)a.n + 1};
    l.v = l.k;
    l.v.base = rows->v;
    l.err = rows->err;
  } else {
    a.n = d->n;
    a.lens = d->n > 0 ? d->lens : nullptr;
    l.k = TokensRows{d->k, {d->k_stride[0], d->k_stride[1], d->k_stride[2]}, a.B, d->n_kv_heads, a.n};
    l.v = TokensRows{d->v, {d->v_stride[0], d->v_stride[1], d->v_stride[2]}, a.B, d->n_kv_heads, a.n};
  }
  const double scale = d->scale > 0.f ? (double)d->scale : 1.0 / std::sqrt((double)D);
  a.scale2 = (float)(scale * 1.4426950408889634);
  const int64_t all = (int64_t)a.n + (a.pend ? 1 : 0);
  const FewPlan few = few_plan(d->batch, (int64_t)d->seq * (d->n_heads / d->n_kv_heads), d->starts != nullptr, d->n_kv_heads, all,
                               d->seq, dev.sms);
  l.plan = plan_of(d, all, dev);
  // (where the tensor-core kernel cannot be launched, the other one answers every call)
  if ((few.us < l.plan.us && !g_without_few.load(std::memory_order_relaxed)) ||
      !tokens_kernel_ready(D, d->dtype, l.plan, dev.device)) {
    FewArgs f{};
    f.q = d->q;
    f.k = l.k.base;
    f.v = l.v.base;
    f.k_new = d->k_new;
    for (int i = 0; i < 3; ++i) {
      const bool on = i > 0 || !d->starts;
      f.q_stride[i] = on ? d->q_stride[i] : 0;
      f.kn_stride[i] = on ? d->k_new_stride[i] : 0;
      f.k_stride[i] = l.k.stride[i];
      f.v_stride[i] = l.v.stride[i];
    }
    f.H = d->n_kv_heads;
    f.chunks = (int)few.chunks;
    return cuda_result(launch_attend_tokens_few(a, f, few, D, d->dtype, s), "launch");
  }
  a.half = (l.plan.split ? 64 : 128) / a.N;
  const size_t need = l.plan.bytes(D);
  if (need && (d->workspace_bytes < need || !d->workspace || !aligned(d->workspace))) {
    set_last_error("workspace must be 16-byte aligned and hold kvevict_attend_tokens_workspace bytes");
    return KVEVICT_ERR_WORKSPACE;
  }
  l.workspace = d->workspace;
  l.stall = take_scorer_stall() ? 1 : 0;
  return cuda_result(launch_attend_tokens(l, D, d->dtype, s), "launch");
}

namespace {

int join_run(const kvevict_join* d, cudaStream_t s) {
  if (!d) return invalid("args must not be null");
  if (!is16(d->dtype)) return invalid("dtype must be KVEVICT_DTYPE_FP16 or _BF16");
  if (d->batch < 0 || d->seq < 0 || d->n_heads < 0) return invalid("batch, seq and n_heads must be >= 0");
  if (d->head_dim != 64 && d->head_dim != 128) return invalid("head_dim must be 64 or 128");
  if (d->parts < 1 || d->parts > KVEVICT_MAX_JOIN) return invalid("parts must be 1 to 8");
  if (d->reserved[0] || d->reserved[1]) return invalid("reserved must be 0");
  if (d->batch == 0 || d->seq == 0 || d->n_heads == 0) return KVEVICT_OK;
  if ((double)d->batch * d->seq * d->n_heads > 0x1p34) return invalid("batch * seq * n_heads must be at most 2^34");
  if (!d->out) return invalid("out must not be null");
  const int32_t x[3] = {d->batch, d->seq, d->n_heads};
  if (!aligned(d->out) || !strides16(d->out_stride, x, 2))
    return invalid("out must be 16-byte aligned, with strides of multiples of 16 bytes");
  if (rows_overlap(d->out_stride, x, d->head_dim)) return invalid("the rows of out must not overlap: strides of at least head_dim");
  JoinArgs a{};
  for (int p = 0; p < d->parts; ++p) {
    if (!d->part[p] || !d->part_lse[p]) return invalid("part and part_lse must not be null");
    if (!aligned(d->part[p]) || !strides16(d->part_stride[p], x, 2))
      return invalid("part must be 16-byte aligned, with strides of multiples of 16 bytes");
    if (!aligned(d->part_lse[p], 4)) return invalid("part_lse and lse must be 4-byte aligned");
    a.part[p] = d->part[p];
    a.part_lse[p] = d->part_lse[p];
    for (int i = 0; i < 3; ++i) a.part_stride[p][i] = d->part_stride[p][i];
  }
  if (!aligned(d->lse, 4)) return invalid("part_lse and lse must be 4-byte aligned");
  a.out = d->out;
  a.lse = d->lse;
  for (int i = 0; i < 3; ++i) a.out_stride[i] = d->out_stride[i];
  a.B = d->batch;
  a.S = d->seq;
  a.G = d->n_heads;
  a.parts = d->parts;
  return cuda_result(launch_attend_join(a, d->head_dim, d->dtype, s), "launch");
}

}  // namespace
}  // namespace kvx

extern "C" int kvevict_attend_prompt(const kvevict_tokens* args, void* stream) {
  return kvx::entry(__func__, [&] { return kvx::tokens_run(args, false, nullptr, (cudaStream_t)stream); });
}

extern "C" int kvevict_attend_tree(const kvevict_tokens* args, void* stream) {
  return kvx::entry(__func__, [&] { return kvx::tokens_run(args, true, nullptr, (cudaStream_t)stream); });
}

extern "C" int kvevict_attend_tokens_workspace(const kvevict_tokens* args, int32_t with_cache, size_t* bytes) {
  return kvx::entry(__func__, [&] {
    if (!bytes) return kvx::invalid("bytes must not be null");
    if (int rc = kvx::tokens_check(args, args && args->parents)) return rc;
    *bytes = 0;
    if (args->batch == 0 || args->seq == 0) return KVEVICT_OK;
    kvx::DeviceInfo dev;
    if (int rc = kvx::device_info(&dev)) return rc;
    // a handle's rows are not in the description: as many as there can be
    *bytes = kvx::plan_of(args, with_cache ? 1 << 29 : args->n, dev).bytes(args->head_dim);
    return KVEVICT_OK;
  });
}

extern "C" int kvevict_test_without_few_kernel(int32_t without) {
  kvx::g_without_few.store(without != 0);
  return KVEVICT_OK;
}

extern "C" int kvevict_test_without_tokens_kernel(int32_t without) {
  kvx::tokens_kernel_off(without != 0);
  return KVEVICT_OK;
}

extern "C" int kvevict_attend_join(const kvevict_join* args, void* stream) {
  return kvx::entry(__func__, [&] { return kvx::join_run(args, (cudaStream_t)stream); });
}
