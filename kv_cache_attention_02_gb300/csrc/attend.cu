// attend.cu -- the entry points kvevict_qk_norm_rope, kvevict_attend and
// kvevict_attend_workspace of include/kvevict.h: argument checks and dispatch.
// Host code only; nothing on the device is touched before the checks pass.
#include "attend_internal.cuh"

#include <nvtx3/nvToolsExt.h>

#include <atomic>
#include <cmath>

namespace kvx {
namespace {

constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];   // multiprocessors of each device, 0: not looked up yet

int invalid(const char* msg) {
  set_last_error(msg);
  return KVEVICT_ERR_INVALID_ARG;
}

int cuda_result(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return KVEVICT_OK;
  set_last_error(std::string(what) + ": " + cudaGetErrorString(e));
  return e == cudaErrorMemoryAllocation ? KVEVICT_ERR_OOM : KVEVICT_ERR_CUDA;
}

bool aligned(const void* p, unsigned to = 16) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Whole 16-byte pieces between the entries of every dimension that has several.
template <int K>
bool strides16(const int64_t (&s)[K], const int32_t (&extent)[K], int elem) {
  for (int i = 0; i < K; ++i)
    if (extent[i] > 1 && ((s[i] * elem) & 15)) return false;
  return true;
}

// Rows of D elements that cannot lie apart (written by several threads at once).
template <int K>
bool rows_overlap(const int64_t (&s)[K], const int32_t (&extent)[K], int D) {
  for (int i = 0; i < K; ++i)
    if (extent[i] > 1 && s[i] < D && s[i] > -D) return true;
  return false;
}

bool is16(int dtype) { return dtype == kFp16 || dtype == kBf16; }

}  // namespace

int device_info(DeviceInfo* out) {
  int dev = 0;
  if (int rc = cuda_result(cudaGetDevice(&dev), "cudaGetDevice")) return rc;
  if (dev < 0 || dev >= kMaxDevices) return invalid("device ordinal beyond the supported 64");
  int sms = g_sms[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    if (int rc = cuda_result(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev),
                             "multiprocessor count"))
      return rc;
    g_sms[dev].store(sms, std::memory_order_relaxed);
  }
  out->sms = sms;
  out->device = dev;
  return KVEVICT_OK;
}

namespace {

int qk_run(const kvevict_qk* d, cudaStream_t s) {
  if (!d) return invalid("args must not be null");
  if (d->in_dtype != kFp32 && !is16(d->in_dtype)) return invalid("in_dtype must be KVEVICT_DTYPE_FP16, _BF16 or _FP32");
  if (!is16(d->out_dtype)) return invalid("out_dtype must be KVEVICT_DTYPE_FP16 or _BF16");
  if (d->weight_dtype != kFp32 && !is16(d->weight_dtype))
    return invalid("weight_dtype must be KVEVICT_DTYPE_FP16, _BF16 or _FP32");
  if (d->batch < 0 || d->seq < 0 || d->n_heads < 0 || d->n_kv_heads < 0)
    return invalid("batch, seq, n_heads and n_kv_heads must be >= 0");
  if ((int64_t)d->n_heads + d->n_kv_heads > 65536) return invalid("more than 65536 heads");
  if (d->head_dim != 64 && d->head_dim != 128) return invalid("head_dim must be 64 or 128");
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return invalid("eps must be >= 0 and finite");
  if (!(d->rope_theta > 0.0) || !std::isnormal(d->rope_theta))   // a subnormal's powers overflow
    return invalid("rope_theta must be > 0, normal and finite");
  // a frequency's 53 bits leave a position of 2^31 an angle within 2^-21, one of 2^50 none
  if (!d->positions && (d->pos0 < INT32_MIN || d->pos0 > (int64_t)INT32_MAX + 1 - std::max(d->seq, 1)))
    return invalid("pos0 and the positions after it must fit 32 bits");
  if (d->reserved) return invalid("reserved must be 0");
  if (d->batch == 0 || d->seq == 0 || d->n_heads + d->n_kv_heads == 0) return KVEVICT_OK;
  if (d->n_heads > 0 && (!d->q || !d->q_out)) return invalid("q and q_out must not be null");
  if (d->n_kv_heads > 0 && (!d->k || !d->k_out)) return invalid("k and k_out must not be null");
  const int ie = d->in_dtype == kFp32 ? 4 : 2;
  const int32_t qx[3] = {d->batch, d->seq, d->n_heads}, kx[3] = {d->batch, d->seq, d->n_kv_heads};
  if (d->n_heads > 0 && (!aligned(d->q) || !aligned(d->q_out) || !strides16(d->q_stride, qx, ie) ||
                         !strides16(d->q_out_stride, qx, 2)))
    return invalid("q and q_out must be 16-byte aligned, with strides of multiples of 16 bytes");
  if (d->n_kv_heads > 0 && (!aligned(d->k) || !aligned(d->k_out) || !strides16(d->k_stride, kx, ie) ||
                            !strides16(d->k_out_stride, kx, 2)))
    return invalid("k and k_out must be 16-byte aligned, with strides of multiples of 16 bytes");
  if ((d->n_heads > 0 && rows_overlap(d->q_out_stride, qx, d->head_dim)) ||
      (d->n_kv_heads > 0 && rows_overlap(d->k_out_stride, kx, d->head_dim)))
    return invalid("the rows of q_out and of k_out must not overlap: strides of at least head_dim");
  const unsigned we = d->weight_dtype == kFp32 ? 4 : 2;
  if (!aligned(d->q_weight, we) || !aligned(d->k_weight, we) || !aligned(d->positions, 4))
    return invalid("q_weight, k_weight and positions must be aligned to their elements");
  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  QkArgs a{};
  a.q = d->q;
  a.k = d->k;
  a.q_out = d->q_out;
  a.k_out = d->k_out;
  for (int i = 0; i < 3; ++i) {
    a.q_stride[i] = d->q_stride[i];
    a.k_stride[i] = d->k_stride[i];
    a.qo_stride[i] = d->q_out_stride[i];
    a.ko_stride[i] = d->k_out_stride[i];
  }
  a.q_weight = d->q_weight;
  a.k_weight = d->k_weight;
  a.w_dtype = d->weight_dtype;
  a.eps = d->eps;
  a.positions = d->positions;
  a.pos0 = d->pos0;
  a.B = d->batch;
  a.S = d->seq;
  a.G = d->n_heads;
  a.H = d->n_kv_heads;
  // The frequencies as 64-bit fractions of a turn. A table of (theta, D) that
  // the calling thread last used: 64 powers would cost more than the launch.
  struct Table {
    double theta = 0.0;
    int D = 0;
    uint64_t turn[64];
  };
  static thread_local Table table;
  if (table.theta != d->rope_theta || table.D != d->head_dim) {
    for (int i = 0; i < d->head_dim / 2; ++i) {
      const double w = std::pow(d->rope_theta, -2.0 * i / d->head_dim) / 6.283185307179586476925286766559;
      table.turn[i] = (uint64_t)std::ldexp(w - std::floor(w), 64);
    }
    table.theta = d->rope_theta;
    table.D = d->head_dim;
  }
  for (int i = 0; i < d->head_dim / 2; ++i) a.turn[i] = table.turn[i];
  return cuda_result(launch_qk_norm_rope(a, d->head_dim, d->in_dtype, d->out_dtype, dev.sms, s), "launch");
}

int attend_check(const kvevict_attention* d) {
  if (!d) return invalid("args must not be null");
  if (!is16(d->dtype)) return invalid("dtype must be KVEVICT_DTYPE_FP16 or _BF16");
  if (d->batch < 0) return invalid("batch must be >= 0");
  if (d->n_kv_heads < 1 || d->n_heads < 1 || d->n_heads % d->n_kv_heads != 0)
    return invalid("n_heads must be a positive multiple of n_kv_heads");
  if (d->head_dim != 64 && d->head_dim != 128) return invalid("head_dim must be 64 or 128");
  if (d->n < 0 || d->prefix < 0 || (int64_t)d->n + d->prefix >= (1 << 30))
    return invalid("n and prefix must be >= 0 and below 2^30 together");
  if ((int64_t)d->batch * d->n_heads > (1 << 26)) return invalid("batch * n_heads must be at most 2^26");
  // more than 2^127 could overflow with the factor log2(e)
  if (d->scale != 0.f && !(d->scale >= 0x1p-126f && d->scale <= 0x1p127f))
    return invalid("scale must be 0, or from 2^-126 to 2^127");
  if (d->reserved || d->reserved2) return invalid("reserved must be 0");
  return KVEVICT_OK;
}

// The prefix kernel's plan; not used (the row kernel reads the shared rows
// itself) where TMA cannot describe the rows, or the kernel cannot be launched.
PrefixPlan plan_prefix(const kvevict_attention* d, bool own, Streamed stream, const DeviceInfo& dev) {
  if (d->prefix == 0 || !prefix_strides_fit(d->prefix_k_stride, d->n_kv_heads, d->prefix, d->head_dim) ||
      !prefix_strides_fit(d->prefix_v_stride, d->n_kv_heads, d->prefix, d->head_dim))
    return PrefixPlan{};
  const PrefixPlan plan = prefix_plan(d->batch, d->n_heads, d->n_kv_heads, d->head_dim, d->prefix, own, stream, dev.sms);
  return plan.ctas && prefix_kernel_ready(d->head_dim, d->dtype, plan.pair, dev.device) ? plan : PrefixPlan{};
}

}  // namespace

int attend_run(const kvevict_attention* d, const CacheRows* rows, cudaStream_t s) {
  if (int rc = attend_check(d)) return rc;
  if (rows) {
    if (d->dtype != kFp16) return invalid("a handle's rows are fp16: dtype must be KVEVICT_DTYPE_FP16");
    if (d->batch != rows->batch || d->n_kv_heads != rows->n_kv_heads || d->head_dim != rows->head_dim)
      return invalid("batch, n_kv_heads and head_dim must be the handle's");
    if (d->n != 0 || d->k || d->v || d->lens) return invalid("n, k, v and lens must be 0 and null with a handle's rows");
  }
  if (d->batch == 0) return KVEVICT_OK;
  if (!d->q || !d->out) return invalid("q and out must not be null");
  if (d->n > 0 && (!d->k || !d->v)) return invalid("k and v must not be null with n > 0");
  if (d->prefix > 0 && (!d->prefix_k || !d->prefix_v)) return invalid("prefix_k and prefix_v must not be null with prefix > 0");
  if (!d->k_new != !d->v_new) return invalid("k_new and v_new must be given together");
  const int32_t qx[2] = {d->batch, d->n_heads}, kx[3] = {d->batch, d->n_kv_heads, d->n};
  const int32_t nx[2] = {d->batch, d->n_kv_heads}, px[2] = {d->n_kv_heads, d->prefix};
  if (!aligned(d->q) || !aligned(d->out) || !strides16(d->q_stride, qx, 2) || !strides16(d->out_stride, qx, 2))
    return invalid("q and out must be 16-byte aligned, with strides of multiples of 16 bytes");
  if (rows_overlap(d->out_stride, qx, d->head_dim))
    return invalid("the rows of out must not overlap: strides of at least head_dim");
  if (d->n > 0 && (!aligned(d->k) || !aligned(d->v) || !strides16(d->k_stride, kx, 2) || !strides16(d->v_stride, kx, 2)))
    return invalid("k and v must be 16-byte aligned, with strides of multiples of 16 bytes");
  if (d->k_new && (!aligned(d->k_new) || !aligned(d->v_new) || !strides16(d->k_new_stride, nx, 2) ||
                   !strides16(d->v_new_stride, nx, 2)))
    return invalid("k_new and v_new must be 16-byte aligned, with strides of multiples of 16 bytes");
  if (d->prefix > 0 && (!aligned(d->prefix_k) || !aligned(d->prefix_v) || !strides16(d->prefix_k_stride, px, 2) ||
                        !strides16(d->prefix_v_stride, px, 2)))
    return invalid("prefix_k and prefix_v must be 16-byte aligned, with strides of multiples of 16 bytes");
  if (!aligned(d->lse, 4) || !aligned(d->lens, 4) || !aligned(d->prefix_lens, 4))
    return invalid("lse, lens and prefix_lens must be 4-byte aligned");
  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  AttendArgs a{};
  a.q = d->q;
  a.out = d->out;
  a.lse = d->lse;
  for (int i = 0; i < 2; ++i) {
    a.q_stride[i] = d->q_stride[i];
    a.out_stride[i] = d->out_stride[i];
    a.kn_stride[i] = d->k_new_stride[i];
    a.vn_stride[i] = d->v_new_stride[i];
    a.pk_stride[i] = d->prefix_k_stride[i];
    a.pv_stride[i] = d->prefix_v_stride[i];
  }
  if (rows) {
    a.k = rows->k;
    a.v = rows->v;
    a.n = rows->n;
    a.pend = rows->pend;
    a.rope_c = rows->rope_c;
    a.rope_s = rows->rope_s;
    for (int i = 0; i < 3; ++i) a.k_stride[i] = a.v_stride[i] = rows->stride[i];
  } else {
    a.k = d->k;
    a.v = d->v;
    a.n = d->n;
    a.lens = d->n > 0 ? d->lens : nullptr;
    for (int i = 0; i < 3; ++i) {
      a.k_stride[i] = d->k_stride[i];
      a.v_stride[i] = d->v_stride[i];
    }
  }
  a.k_new = d->k_new;
  a.v_new = d->v_new;
  a.pk = d->prefix_k;
  a.pv = d->prefix_v;
  a.plens = d->prefix > 0 ? d->prefix_lens : nullptr;
  a.B = d->batch;
  a.G = d->n_heads;
  a.H = d->n_kv_heads;
  a.P = d->prefix;
  const double scale = d->scale > 0.f ? (double)d->scale : 1.0 / std::sqrt((double)d->head_dim);
  a.scale2 = (float)(scale * 1.4426950408889634);
  const int D = d->head_dim;
  PrefixArgs p{};
  const int own = a.n + (a.k_new ? 1 : 0);             // rows of a sequence, at most
  p.plan = plan_prefix(d, rows || own, Streamed{}, dev);
  const bool alone = p.plan.ctas && p.plan.final;      // the prefix is all there is
  RowsPlan rp{};
  if (!alone)
    rp = rows_plan(a.B, a.G, a.H, D, a.n, p.plan.ctas ? 0 : a.P, a.k_new, rows != nullptr, p.plan.ctas > 0, dev.sms);
  if (p.plan.ctas && rp.ctas) {                        // both at once, each on its SMs
    p.plan = plan_prefix(d, true, Streamed{(int64_t)a.B * a.H * own * D * 4, rp.units}, dev);
    rp.ctas = std::min(rp.ctas, stream_ctas(D, std::max(1, dev.sms - p.plan.ctas)));
  }
  const size_t need = p.plan.bytes(D) + rp.bytes(D);
  if (need && (d->workspace_bytes < need || !d->workspace || !aligned(d->workspace))) {
    set_last_error("workspace must be 16-byte aligned and hold kvevict_attend_workspace bytes");
    return KVEVICT_ERR_WORKSPACE;
  }
  char* space = static_cast<char*>(d->workspace);
  if (p.plan.ctas) {
    p.a = a;
    p.part_o = reinterpret_cast<float*>(space);
    p.part_ml = reinterpret_cast<float2*>(space + p.plan.o_bytes(D));
    p.err = rows ? rows->err : nullptr;
    p.stall = take_scorer_stall() ? 1 : 0;
    const cudaError_t e = launch_attend_prefix(p, D, d->dtype, s);
    if (e != cudaSuccess) return cuda_result(e, "launch");
    if (alone) return KVEVICT_OK;
    space += p.plan.bytes(D);
    a.P = 0;               // joined from its parts
    a.plens = nullptr;
  }
  rp.part_o = reinterpret_cast<float*>(space);
  rp.part_ml = reinterpret_cast<float2*>(space + rp.o_bytes(D));
  rp.first = reinterpret_cast<int64_t*>(space + rp.o_bytes(D) + rp.ml_bytes());
  return cuda_result(launch_attend_rows(a, p.parts(), rp, D, d->dtype, dev.sms, s), "launch");
}

}  // namespace kvx

namespace {
// An NVTX range named after the entry point, and no C++ exception past it (an
// error message is the only thing that allocates).
template <typename F>
int entry(const char* name, F&& body) {
  nvtxRangePushA(name);
  int rc;
  try {
    rc = body();
  } catch (...) {
    rc = KVEVICT_ERR_OOM;
  }
  nvtxRangePop();
  return rc;
}
}  // namespace

extern "C" int kvevict_qk_norm_rope(const kvevict_qk* args, void* stream) {
  return entry(__func__, [&] { return kvx::qk_run(args, (cudaStream_t)stream); });
}

extern "C" int kvevict_attend(const kvevict_attention* args, void* stream) {
  return entry(__func__, [&] { return kvx::attend_run(args, nullptr, (cudaStream_t)stream); });
}

extern "C" int kvevict_attend_workspace(const kvevict_attention* args, int32_t with_cache, size_t* bytes) {
  return entry(__func__, [&] {
    if (!bytes) return kvx::invalid("bytes must not be null");
    if (int rc = kvx::attend_check(args)) return rc;
    *bytes = 0;
    if (args->batch == 0) return KVEVICT_OK;
    kvx::DeviceInfo dev;
    if (int rc = kvx::device_info(&dev)) return rc;
    const int B = args->batch, G = args->n_heads, H = args->n_kv_heads, D = args->head_dim;
    const bool own = with_cache || args->n > 0 || args->k_new;
    const kvx::PrefixPlan pp = kvx::plan_prefix(args, own, kvx::Streamed{}, dev);
    *bytes = pp.bytes(D);
    if (pp.ctas && !own) return KVEVICT_OK;
    // a handle's rows are not in the description: as many as there can be
    const int n = with_cache ? 1 << 29 : args->n;
    *bytes += kvx::rows_plan(B, G, H, D, n, pp.ctas ? 0 : args->prefix, args->k_new != nullptr, with_cache != 0,
                             pp.ctas > 0, dev.sms).bytes(D);
    return KVEVICT_OK;
  });
}

extern "C" int kvevict_test_without_prefix_kernel(int32_t without) {
  kvx::prefix_kernel_off(without != 0);
  return KVEVICT_OK;
}
