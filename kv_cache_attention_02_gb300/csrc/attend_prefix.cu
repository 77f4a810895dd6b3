// attend_prefix.cu -- attention of many query rows over rows that all
// sequences share, on the 5th-generation tensor cores: the prefix's part of
// kvevict_attend, its keys and values read once for the whole batch.
//
// For one key head the queries of all sequences and of its N = G / H query
// heads are the rows of one matrix Q [B*N, D], row b*N + j:
//   S = Q K^T * scale,  P = e^(S - m),  O = P V,  l = sum P,
// with the running sum l of each row in fp32, relative to m: the running maximum, or
// less. P is rounded to the inputs' 16-bit type for the second product and l is summed
// before that rounding, so the roundings average out; with few rows (see PAIR) it goes
// in as the sum of two 16-bit parts, as in attend_rows.cu. m moves only when the true
// maximum is more than 2^8 above the one it was set by, which P and l carry without
// loss: most tiles then need no rescaling of O. In fp16 m is set 2^7 below that maximum,
// so that P uses the type's upper range and only weights below 2^-32 of the largest
// vanish (2^16 rows of them are 2^-16 of the sum).
//
// Work: the (key head, block of query rows, 128-key tile) triples, in that
// order, are cut into one contiguous range per CTA (one CTA an SM, which holds
// all of the tensor memory), whatever the sizes: a block's tiles may end in one
// CTA and begin in another. A range's piece of a block leaves its unnormalised
// O, m and l in the workspace, where the join (attend_rows.cu or the kernel
// below) finds them in a fixed order; a block that is one CTA's alone is written
// out directly where nothing else has to join it.
//
// Two streams of 128 query rows share a CTA, each with its own accumulators S
// and O (four times 128 TMEM columns), so that one stream's softmax runs while
// the tensor cores work for the other:
//   TILES  (more than 128 query rows a key head) the streams are two row blocks
//          and both use every key and value tile;
//   PAIR   (at most 128 rows, bound by memory) both are the same rows, and the
//          streams take even and odd tiles.
// Roles in a 384-thread CTA:
//   warp 0      one thread issues TMA loads of key and value tiles (128 rows,
//               128-byte swizzle) into one ring, in the order they are used;
//   warp 1      issues tcgen05.mma: S = Q K^T from shared memory, then O += P V
//               with P from TMEM and V as it lies in memory (its rows are the
//               contraction: an MN-major operand);
//   warps 4..11 two softmax warpgroups, one per stream, a query row a thread:
//               tcgen05.ld S, mask, maximum, exp2, sum, P back into S's columns.
// A stream's tcgen05.commit after S also covers the P V before it, so a thread
// that has seen S may rescale O without another wait.
// Every mbarrier wait is bounded; on expiry the CTA leaves NaN in its rows.
//
// Measured on GB300: 4096 x 32 query rows on 8192 keys, D = 128, bf16, 365-408 us by
// the GPU's clocks, 1.35-1.51 PFLOP/s (0.72-0.81 of the measured matrix rate); its MMAs
// with no softmax between them take 327 us, without waits 309. 32 sequences on 65536
// rows 50 us for the kernel, 5.4 TB/s, and 6 us for the join. A call's start, one tile and
// its end are 8 us (setup 0.9, queries 2, first tile and its softmax 2, end 2), which
// is most of a short prefix's time. Tried and slower: three logits buffers at D = 64
// with one general issue loop (53 against 47 us), a suspended or a longer plain poll
// of the barriers (524, 542 against 505), the operands' low words added apart (no change).
#include "attend_internal.cuh"
#include "tcgen05.cuh"

#include <algorithm>
#include <atomic>

namespace kvx {
namespace {

constexpr int kT = 128;                // query rows of a stream, keys of a tile
constexpr int kPxThreads = 384;
constexpr int kPxTmem = 512;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLazy = 8.f;           // log2 of how far a weight may exceed the first maximum's
// log2 of the first maximum's weight: with kLazy on top, half of fp16's range. bf16 has fp32's exponents.
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 7.f : 0.f;
constexpr float kFar = 0x1p23f;        // base-2 logits from here on are whole numbers

template <int D>
struct PxGeo {
  static constexpr int KH = D / 64;              // 128-byte halves of a row
  static constexpr int HALFB = kT * 128;         // one half tile, 16 KB
  static constexpr int TILEB = KH * HALFB;
  static constexpr int STAGES = 160 * 1024 / TILEB;
  static constexpr int Q = 0, RING = 2 * TILEB, BARS = RING + STAGES * TILEB;
  static constexpr int ML = TILEB;   // PAIR: the streams' maxima and sums, where TILES has its second query block
  static constexpr int SMEM = BARS + (2 * STAGES + 12) * 8 + 16 + 1024;   // slack to align to 1024 bytes
};

// Instruction descriptors, kind::f16, f32 accumulator, M = 128: bits 7 and 10
// the inputs' type (1: bf16), 16 B is MN-major, 17.. N / 8, 24.. M / 16.
template <typename T>
__host__ __device__ constexpr uint32_t px_idesc(int n, bool b_mn_major) {
  return (1u << 4) | (std::is_same<T, __half>::value ? 0u : (1u << 7) | (1u << 10)) | (b_mn_major ? 1u << 16 : 0u) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kT >> 4) << 24);
}

// MN-major operand, 128-byte swizzle: 64 consecutive columns are 128 bytes,
// 8 rows of the contraction 1024 bytes apart (stride byte offset), the next 64
// columns one half tile on (leading byte offset).
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr, uint32_t half_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(half_bytes >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// All 128 columns of this thread's lane, waited for.
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float* v) {
  uint32_t r[128];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]), "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]), "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]), "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]), "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]), "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]), "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]), "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]), "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int e = 0; e < 128; ++e) v[e] = __uint_as_float(r[e]);
}

// 16 consecutive columns of this thread's lane, waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(r[e]);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
      ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// One thread of the warp, always the same, chosen in a way that tells the
// compiler that the warp stays uniform: descriptors then live in uniform
// registers. With `lane == 0` instead, moving them there bound the rate at which
// MMAs were issued (388 against 322 us for the MMAs of 4096 x 32 query rows on
// 8192 keys alone).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// One CTA's walk over its range of (block, tile) pairs, the same in every role.
struct Walk {
  int64_t x, end;
  int nkt;
  __device__ __forceinline__ Walk(const PrefixArgs& p, int cta)
      : x(p.plan.start(cta)), end(p.plan.start(cta + 1)), nkt(p.plan.nkt) {}
  // Next segment: tiles k0 .. k1 - 1 of block u; false at the end.
  __device__ __forceinline__ bool next(int& u, int& k0, int& k1) {
    if (x >= end) return false;
    u = (int)(x / nkt);
    k0 = (int)(x - (int64_t)u * nkt);
    k1 = (int)min((int64_t)nkt, k0 + (end - x));
    x += k1 - k0;
    return true;
  }
};

// Rows of the prefix that some query row of block u has (warp-collective).
__device__ __forceinline__ int block_limit(const PrefixArgs& p, int u) {
  if (!p.a.plens) return p.a.P;
  const int N = p.a.G / p.a.H;
  const int64_t r0 = (int64_t)(u % p.plan.blocks) * p.plan.block_rows;
  const int b0 = (int)(r0 / N);
  const int b1 = (int)min((int64_t)p.a.B - 1, (r0 + p.plan.block_rows - 1) / N);
  int lim = 0;
  for (int b = b0 + (int)(threadIdx.x & 31); b <= b1; b += 32) lim = max(lim, p.a.plens[b]);
  return min((int)__reduce_max_sync(~0u, lim), p.a.P);
}

template <typename T, int D, bool PAIR>
__global__ void __launch_bounds__(kPxThreads, 1)
    attend_prefix_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                         const __grid_constant__ PrefixArgs p) {
  using Gm = PxGeo<D>;
  constexpr int NS = Gm::STAGES;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Gm::BARS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Gm::BARS + (2 * NS + 12) * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto full = [&](int s) { return smem_addr(&bars[s]); };
  auto empty = [&](int s) { return smem_addr(&bars[NS + s]); };
  auto s_full = [&](int w) { return smem_addr(&bars[2 * NS + w]); };
  auto p_full = [&](int w, int c) { return smem_addr(&bars[2 * NS + 8 + 2 * w + c]); };   // halves of 64 keys
  auto o_done = [&](int w) { return smem_addr(&bars[2 * NS + 4 + w]); };
  const uint32_t q_full = smem_addr(&bars[2 * NS + 6]);
  const uint32_t drain = smem_addr(&bars[2 * NS + 7]);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const AttendArgs& a = p.a;
  const int N = a.G / a.H;

  launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(s_full(w), 1);
      mbar_init(p_full(w, 0), 4);
      mbar_init(p_full(w, 1), 4);
      mbar_init(o_done(w), 1);
    }
    mbar_init(q_full, 8);
    mbar_init(drain, 1);               // abort path only
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == 1) tmem_alloc(smem_addr(tmem_slot), kPxTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // TMEM columns: O of stream w at 128 w, S (and P over it) at 256 + 128 w
  auto tm_o = [&](int w) { return tmem + (uint32_t)(kT * w); };
  auto tm_s = [&](int w) { return tmem + (uint32_t)(2 * kT + kT * w); };

  Walk walk(p, blockIdx.x);
  int u, k0, k1;
  // The launch's 384 x 168 registers, shared out anew: 4 warps of 120 and 8 of
  // 192 a thread, so that a softmax thread holds a row's 128 logits.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    if (warp == 0) {
      // ---------------------------------------------------------------- TMA producer
      if (lane < 2)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane ? &vmap : &kmap)) : "memory");
      int s = 0, held = 0;               // next stage, stages in flight (at most NS)
      uint32_t phase = 0;
      bool ok = true, stall = p.stall && blockIdx.x == 0;   // test hook: CTA 0's first tile never comes
      while (ok && walk.next(u, k0, k1)) {
        const int n = min(k1, (block_limit(p, u) + kT - 1) / kT) - k0;
        const int h = u / p.plan.blocks;
        if (lane == 0) {
          auto load = [&](const CUtensorMap* map, bool row_first, int kt) {
            if (held == NS && !wait_or_abort(empty(s), phase ^ 1, abort_flag, p.err)) return false;
            if (!stall) {
              mbar_expect_tx(full(s), Gm::TILEB);
              const int row = (k0 + kt) * kT;
              for (int kh = 0; kh < Gm::KH; ++kh)
                tma_load_3d(base + Gm::RING + s * Gm::TILEB + kh * Gm::HALFB, map, kh * 64, row_first ? row : h,
                            row_first ? h : row, full(s));
            }
            stall = false;
            held = min(held + 1, NS);
            if (++s == NS) s = 0, phase ^= 1;
            return true;
          };
          for (int i = 0; i < n && ok; ++i) {
            if (i == 0) {
              ok = load(&kmap, p.k_row_first, 0);
              if (PAIR && ok && n > 1) ok = load(&kmap, p.k_row_first, 1);
            }
            ok = ok && load(&vmap, p.v_row_first, i);
            const int nk = PAIR ? i + 2 : i + 1;
            if (ok && nk < n) ok = load(&kmap, p.k_row_first, nk);
          }
        }
        ok = __shfl_sync(~0u, (int)ok, 0) != 0;
      }
      if (lane == 0 && *abort_flag)      // let copies in flight land before the CTA leaves
        for (int i = 0; i < held; ++i) {
          if (--s < 0) s = NS - 1, phase ^= 1;
          (void)mbar_wait_bounded(full(s), phase, 10000000ull);
        }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer
      constexpr uint32_t kIdS = px_idesc<T>(kT, false), kIdO = px_idesc<T>(D, true);
      // descriptors of the first query block and ring stage; an offset adds to the
      // address field, in 16-byte units
      const uint64_t qd = sw128_desc(base + Gm::Q), kd = sw128_desc(base + Gm::RING);
      const uint64_t vd = sw128_mn_desc(base + Gm::RING, Gm::HALFB);
      int next = 0;                      // ring stage and its phase
      uint32_t phase = 0;
      uint32_t np[2] = {0, 0};           // weights tiles consumed, per stream
      int seg = 0;                       // segments that have tiles
      bool ok = true;
      while (ok && walk.next(u, k0, k1)) {
        const int limit = block_limit(p, u);
        const int n = min(k1, (limit + kT - 1) / kT) - k0;
        if (n <= 0) continue;
        ok = __all_sync(~0u, wait_or_abort(q_full, (uint32_t)(seg & 1), abort_flag, p.err));
        ++seg;
        if (!ok) break;
        tc_fence_after();
        auto tile = [&]() -> int {       // the next ring stage, once its tile is there; -1 on abort
          const int s = next;
          const bool here = wait_or_abort(full(s), phase, abort_flag, p.err);
          if (++next == NS) next = 0, phase ^= 1;
          return __all_sync(~0u, here) ? s : -1;
        };
        auto mma_s = [&](int w, int s) {
          if (elect_one()) {
            const uint64_t qa = qd + (uint64_t)((PAIR ? 0 : w) * (Gm::TILEB >> 4)), kb = kd + (uint64_t)(s * (Gm::TILEB >> 4));
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = (uint64_t)(((kk >> 2) * Gm::HALFB + (kk & 3) * 32) >> 4);
              tc_mma_ss(tm_s(w), qa + off, kb + off, kIdS, kk > 0);
            }
            tc_commit(s_full(w));
          }
        };
        // (TILES: the softmax warps give the stages back)
        auto release = [&](int s) {
          if (elect_one()) tc_commit(empty(s));
        };
        // O_w += P_w V: P of keys 0..63 in S's columns 0..31, of keys 64..127 in
        // 64..95, the second parts (PAIR) 32 columns on
        auto mma_o = [&](int w, int s, bool first) {
          const uint64_t vb = vd + (uint64_t)(s * (Gm::TILEB >> 4));
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (!__all_sync(~0u, wait_or_abort(p_full(w, c), np[w] & 1, abort_flag, p.err))) return false;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int part = 0; part < (PAIR ? 2 : 1); ++part)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  tc_mma_ts(tm_o(w), tm_s(w) + (uint32_t)(c * 64 + kk * 8 + 32 * part),
                            vb + (uint64_t)((4 * c + kk) * (2048 >> 4)), kIdO, !(first && c + kk + part == 0));
            }
          }
          ++np[w];
          return true;
        };
        // A value tile that reaches past the block's rows: what lies there may be
        // anything, and 0 * NaN would spoil the sums, so it becomes zeros.
        auto clean = [&](int s, int kt) {
          const int from = limit - kt * kT;
          if (from >= kT || limit == a.P) return;      // TMA has filled rows past P with zeros
          for (int x = lane; x < (kT - from) * (D / 8); x += 32) {
            const int row = from + x / (D / 8), c = x % (D / 8);
            *reinterpret_cast<uint4*>(smem + Gm::RING + s * Gm::TILEB + (c >> 3) * Gm::HALFB + row * 128 + (c & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        };
        int s;
        if (PAIR) {
          for (int i = 0; i < min(n, 2) && ok; ++i) {
            ok = (s = tile()) >= 0;
            if (ok) mma_s(i, s), release(s);
          }
          for (int i = 0; i < n && ok; ++i) {
            const int w = i & 1;
            if (!(ok = (s = tile()) >= 0)) break;
            clean(s, k0 + i);
            if (!(ok = mma_o(w, s, i < 2))) break;
            release(s);
            if (i + 2 >= n && elect_one()) tc_commit(o_done(w));
            if (i + 2 < n) {
              if (!(ok = (s = tile()) >= 0)) break;
              mma_s(w, s);
              release(s);
            }
          }
        } else {
          ok = (s = tile()) >= 0;
          if (ok) mma_s(0, s), mma_s(1, s);
          for (int i = 0; i < n && ok; ++i) {
            const bool more = i + 1 < n;
            int sk = 0;
            if (!(ok = (s = tile()) >= 0)) break;
            clean(s, k0 + i);
            if (!(ok = mma_o(0, s, i == 0))) break;
            if (more) {
              if (!(ok = (sk = tile()) >= 0)) break;
              mma_s(0, sk);
            } else if (elect_one()) {
              tc_commit(o_done(0));
            }
            if (!(ok = mma_o(1, s, i == 0))) break;
            if (more) {
              mma_s(1, sk);
            } else if (elect_one()) {
              tc_commit(o_done(1));
            }
          }
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax warpgroups
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int w = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;          // query row of the stream = TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t ns = 0, no = 0;                         // logits tiles and finished outputs seen
    int ring = 0;                                    // stage of the segment's first tile
    // TILES: the second stream gives the ring's stages back. When it sees its logits
    // of key tile i (the segment's tile 2 i), those keys have been read, and the values
    // of tile i - 1 (2 i - 1) by the products before. A commit by the MMA warp for
    // each would be one more stop in its stream of products (368 against 383 us for 16 x
    // 256-token chunks on 8192 keys); PAIR waits for memory and wants its stages
    // sooner.
    auto release = [&](int nth) {
      if (lane == 0 && (warp & 3) == 0) mbar_arrive(empty((ring + nth) % NS));
    };
    while (walk.next(u, k0, k1)) {
      const int limit = block_limit(p, u);
      const int n = max(0, min(k1, (limit + kT - 1) / kT) - k0);
      const int h = u / p.plan.blocks;
      const int r = (u - h * p.plan.blocks) * p.plan.block_rows + (PAIR ? 0 : w * kT) + row;   // below 2^26 + 256
      const bool valid = r < a.B * N;
      const int b = valid ? r / N : 0, head = h * N + (valid ? r - b * N : 0);
      const int rows = valid && a.plens ? max(0, min(a.plens[b], a.P)) : a.P;
      // The warp's 32 rows of the query block, as TMA would swizzle them; PAIR: each
      // warpgroup has half of every row's pieces. Between global and shared memory
      // neighbouring lanes move neighbouring pieces of a row (a lane a row would
      // touch 32 lines an instruction, 2 to 4 us a block).
      constexpr int CPR = PAIR ? D / 16 : D / 8;     // 16-byte pieces of a row
      unsigned char* const mine = smem + Gm::Q + (PAIR ? 0 : w) * Gm::TILEB;
      auto piece_of = [&](int r_, int c) { return mine + r_ * 128 + (c >> 3) * Gm::HALFB + (((c ^ r_) & 7) << 4); };
      auto each_piece = [&](int64_t offset, auto&& move) {   // offset: of this lane's row
#pragma unroll
        for (int i = 0; i < CPR; ++i) {
          const int from = i * (32 / CPR) + lane / CPR, c = (PAIR ? w * CPR : 0) + lane % CPR;
          const int64_t at = __shfl_sync(~0u, offset, from);
          const bool on = __shfl_sync(~0u, (int)valid, from);
          move(i, on, at + 8 * c, piece_of((warp & 3) * 32 + from, c));
        }
      };
      if (n > 0) {
        uint4 v[CPR];                                // all on their way before the first is stored
        const T* const q = static_cast<const T*>(a.q);
        const int64_t at = b * a.q_stride[0] + (int64_t)head * a.q_stride[1];
        each_piece(at, [&](int i, bool on, int64_t from, unsigned char*) {
          v[i] = on ? *reinterpret_cast<const uint4*>(q + from) : make_uint4(0, 0, 0, 0);
        });
        each_piece(at, [&](int i, bool, int64_t, unsigned char* to) { *reinterpret_cast<uint4*>(to) = v[i]; });
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      float m = kNegInf, l = 0.f;
      bool ok = true, begun = false;
      const uint32_t ts = tm_s(w) + lanes, to = tm_o(w) + lanes;
      for (int i = PAIR ? w : 0; i < n; i += PAIR ? 2 : 1) {
        ok = __all_sync(~0u, wait_or_abort(s_full(w), ns & 1, abort_flag, p.err));
        if (!ok) break;
        ++ns;
        tc_fence_after();
        if (!PAIR && w == 1) {
          release(2 * i);
          if (i > 0) release(2 * i - 1);
        }
        const int left = rows - (k0 + i) * kT;       // columns from here on are masked
        const bool none = left <= 0;
        // a length ends inside this tile, or rows that no sequence has begin in it
        const bool partial = __any_sync(~0u, !none && left < kT) || limit - (k0 + i) * kT < kT;
        float v[kT];
        tmem_ld128(ts, v);
        if (partial) {
#pragma unroll
          for (int e = 0; e < kT; ++e) v[e] = e < left ? v[e] : kNegInf;
        }
        // (a NaN stays in the maximum, so that one compare finds logits that are not finite)
        float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int e = 4; e < kT; e += 8)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            m4[x] = e + 4 < kT ? max_nan(m4[x], max_nan(v[e + x], v[e + 4 + x])) : max_nan(m4[x], v[e + x]);
        const float top = max_nan(max_nan(m4[0], m4[1]), max_nan(m4[2], m4[3]));
        const float mx = none ? kNegInf : top * a.scale2;
        // Rare: logits of NaN or +inf in a row past its length (keys that other rows have),
        // which the addend -inf below would leave NaN; and a maximum so large that it is
        // rounded by a half or more, as its own logit need not be near it in the fused
        // product and difference below. (One vote with the common case, as each one stands
        // in the way of everything after it: 51.3 us for the unequal lengths so, 52.5 with two.)
        const bool odd = none ? !(top < -kNegInf) : !(fabsf(mx) < kFar), up = mx > m + (kLazy + kLift<T>);
        // a row past its length: every weight 2^-inf = 0 (and so are masked ones, with a
        // row that has had nothing so far)
        float nb = none ? kNegInf : m == kNegInf ? 0.f : -m;
        if (__any_sync(~0u, up || odd)) {
          const float nm = odd ? fmaxf(m, mx) : up ? mx - kLift<T> : m, f = nm == m ? 1.f : ex2(m - nm);
          m = nm;
          l *= f;
          if (begun) {
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              float x[16];
              uint32_t o[16];
              tmem_ld16(to + 16 * c, x);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(x[e] * f);
              tmem_st16(to + 16 * c, o);
            }
          }
          nb = none ? kNegInf : m == kNegInf ? 0.f : -m;
          if (__builtin_expect(__any_sync(~0u, odd), 0)) {
            // the difference, of a product rounded as the maximum was, goes through the
            // fused product instead (in such rows alone: no row's bits depend on its neighbours)
            const float inv = 1.f / a.scale2;
#pragma unroll 1
            for (int c = 0; c < kT / 16; ++c) {
              float x[16];
              uint32_t o[16];
              tmem_ld16(ts + 16 * c, x);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                o[e] = __float_as_uint(16 * c + e >= left ? kNegInf
                                       : odd ? __fadd_rn(__fmul_rn(x[e], a.scale2), nb) * inv : x[e]);
              tmem_st16(ts + 16 * c, o);
            }
            tmem_st_wait();
            tmem_ld128(ts, v);
            if (odd) nb = 0.f;
          }
        }
        begun = true;
        const float2 sc2 = make_float2(a.scale2, a.scale2), nb2 = make_float2(nb, nb);
        float2 l4[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) l4[x] = make_float2(0.f, 0.f);
        // 64 keys at a time: the tensor cores start on the first half's weights
        // while the second half's are computed
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const int k = 64 * c + 32 * g + e;
              const float2 t = ffma2(make_float2(v[k], v[k + 1]), sc2, nb2);
              const float2 pp = make_float2(ex2(t.x), ex2(t.y));
              l4[(e >> 1) & 3] = fadd2(l4[(e >> 1) & 3], pp);
              hi[e / 2] = pack16<T>(pp.x, pp.y);
              if (PAIR) {
                const float2 back = unpack16<T>(hi[e / 2]);
                lo[e / 2] = pack16<T>(pp.x - back.x, pp.y - back.y);
              }
            }
            tmem_st16(ts + 64 * c + 16 * g, hi);
            if (PAIR) tmem_st16(ts + 64 * c + 32 + 16 * g, lo);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(w, c));
        }
        l4[0] = fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3]));
        l += l4[0].x + l4[0].y;
      }
      if (begun && ok) {
        ok = __all_sync(~0u, wait_or_abort(o_done(w), no & 1, abort_flag, p.err));
        ++no;
        tc_fence_after();
        if (!PAIR && w == 1) release(2 * n - 1);
      }
      ring = (ring + 2 * n) % NS;
      if (!ok) l = __int_as_float(0x7FFFFFFF);       // NaN: this row's result is lost
      float f0 = 1.f, f1 = 0.f;
      if (PAIR) {
        // the two streams' maxima and sums meet in shared memory, their O in the
        // registers of whichever warpgroup writes the columns: a warp of either
        // reaches the same TMEM lanes
        float2* ml = reinterpret_cast<float2*>(smem + Gm::ML);
        ml[w * kT + row] = make_float2(m, l);
        tc_fence_before();
        asm volatile("bar.sync 3, 256;" ::: "memory");
        tc_fence_after();
        const float2 x = ml[row], y = ml[kT + row];
        m = fmaxf(x.x, y.x);
        f0 = x.x == m ? 1.f : ex2(x.x - m);
        f1 = y.x == m ? 1.f : ex2(y.x - m);
        l = x.y * f0 + y.y * f1;
      }
      auto columns = [&](int c, float* v) {          // O's columns 32 c .. + 31 of this row
        const uint32_t at = tmem + lanes + 32 * c;
        if (n == 0) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0.f;
        } else if (!PAIR) {
          tmem_ld32(at + kT * w, v);
        } else {
          tmem_ld32(at, v);
          if (n > 1) {
            float y[32];
            tmem_ld32(at + kT, y);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = fmaf(y[e], f1, v[e] * f0);
          }
        }
      };
      constexpr int CC = PAIR ? D / 64 : D / 32;
      // a block of this CTA alone goes to the output, any other to the workspace
      if (p.plan.final && k0 == 0 && k1 == p.plan.nkt) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
        for (int i = 0; i < CC; ++i) {
          const int c = (PAIR ? w * CC : 0) + i;
          float v[32];
          columns(c, v);
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t o[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) o[x] = pack16<T>(v[e + 2 * x] * inv, v[e + 2 * x + 1] * inv);
            *reinterpret_cast<uint4*>(piece_of(row, 4 * c + e / 8)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        __syncwarp();                                // the queries' place serves: their products are done
        T* const out = static_cast<T*>(a.out);
        each_piece(b * a.out_stride[0] + (int64_t)head * a.out_stride[1], [&](int, bool on, int64_t to, unsigned char* from) {
          if (on) *reinterpret_cast<uint4*>(out + to) = *reinterpret_cast<const uint4*>(from);
        });
        if (valid && a.lse && !(PAIR && w))
          a.lse[(int64_t)b * a.G + head] = l == 0.f ? kNegInf : (m + log2f(l)) * 0.69314718055994531f;
      } else {
        const int64_t slot = p.plan.slot(u, blockIdx.x, k0 == 0);
        const int R = p.plan.block_rows, rr = (PAIR ? 0 : w * kT) + row;
        float4* o = reinterpret_cast<float4*>(p.part_o) + slot * (R * (D / 4)) + rr;
#pragma unroll 1
        for (int i = 0; i < CC; ++i) {
          const int c = (PAIR ? w * CC : 0) + i;
          float v[32];
          columns(c, v);
#pragma unroll
          for (int e = 0; e < 32; e += 4) o[(int64_t)(8 * c + e / 4) * R] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
        if (!(PAIR && w)) p.part_ml[slot * R + rr] = make_float2(m, l);
      }
      tc_fence_before();
      // both warpgroups are through with this block's queries and accumulators
      uint32_t stop;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\t"
          "setp.ne.u32 p, %1, 0;\n\t"
          "bar.red.or.pred q, 3, 256, p;\n\t"
          "selp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(stop)
          : "r"((uint32_t)(!ok || *abort_flag))
          : "memory");
      if (stop) {
        // the blocks this CTA will not come to: NaN as well
        while (walk.next(u, k0, k1)) {
          const int rr = (PAIR ? 0 : w * kT) + row;
          const int64_t r2 = (int64_t)(u % p.plan.blocks) * p.plan.block_rows + rr;
          if (!(p.plan.final && k0 == 0 && k1 == p.plan.nkt)) {
            p.part_ml[p.plan.slot(u, blockIdx.x, k0 == 0) * p.plan.block_rows + rr] =
                make_float2(0.f, __int_as_float(0x7FFFFFFF));
          } else if (r2 < (int64_t)a.B * N) {
            const int b2 = (int)(r2 / N), h2 = (u / p.plan.blocks) * N + (int)(r2 - (int64_t)b2 * N);
            T* dst = static_cast<T*>(a.out) + b2 * a.out_stride[0] + (int64_t)h2 * a.out_stride[1];
            for (int c = 0; c < D / 8; ++c)
              *reinterpret_cast<uint4*>(dst + 8 * c) = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
            if (a.lse) a.lse[(int64_t)b2 * a.G + h2] = __int_as_float(0x7FFFFFFF);
          }
        }
        break;
      }
    }
  }

  // -------------------------------------------------------------------- teardown
  __syncthreads();
  if (*abort_flag && tid == 32) {
    // let any MMA still in flight finish before the accumulators are freed
    tc_commit(drain);
    (void)mbar_wait_bounded(drain, 0, 10000000ull);
  }
  __syncwarp();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kPxTmem);
  }
}

// Joins the parts of blocks that several CTAs share, where the prefix is all
// there is: grid (block, 32 rows of it, 32 columns), or, with more blocks than
// CTAs, (boundary between CTAs, ..), where the first boundary inside a block
// takes it. A lane is a row, and the eight warps
// take every eighth part, so that all of a block's loads are under way at once.
template <typename T, int D>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ PrefixArgs p) {
  const PrefixPlan& pl = p.plan;
  const AttendArgs& a = p.a;
  int u = blockIdx.x;
  bool mine = true;
  if (pl.units >= pl.ctas) {
    const int64_t x = pl.start(blockIdx.x + 1);
    u = (int)(x / pl.nkt);
    mine = x != (int64_t)u * pl.nkt && pl.start(blockIdx.x) <= (int64_t)u * pl.nkt;
  }
  const int64_t u0 = (int64_t)u * pl.nkt;
  __shared__ float2 ml_s[8][32];
  __shared__ float4 o_s[8][8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int N = a.G / a.H, R = pl.block_rows, h = u / pl.blocks;
  const int rr = blockIdx.y * 32 + lane, d4 = blockIdx.z * 8;
  const int c0 = pl.cta_of(u0), c1 = pl.cta_of(u0 + pl.nkt - 1);
  wait_for_primary();                        // in every block: this kernel ends after the one before it
  if (!mine || c0 == c1) return;             // one CTA's alone: written out by it
  float m = kNegInf, l = 0.f;
  float4 o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int c = c0 + warp; c <= c1; c += 8) {
    const int64_t slot = pl.slot(u, c, c == c0);
    const float2 ml = p.part_ml[slot * R + rr];
    const float4* src = reinterpret_cast<const float4*>(p.part_o) + slot * (R * (D / 4)) + (int64_t)d4 * R + rr;
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = src[i * R];
    const float nm = fmaxf(m, ml.x), f = m == nm ? 1.f : ex2(m - nm), g = ml.x == nm ? 1.f : ex2(ml.x - nm);
    m = nm;
    l = l * f + ml.y * g;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      o[i].x = o[i].x * f + v[i].x * g;
      o[i].y = o[i].y * f + v[i].y * g;
      o[i].z = o[i].z * f + v[i].z * g;
      o[i].w = o[i].w * f + v[i].w * g;
    }
  }
  ml_s[warp][lane] = make_float2(m, l);
#pragma unroll
  for (int i = 0; i < 8; ++i) o_s[warp][i][lane] = o[i];
  __syncthreads();
  const int64_t r = (int64_t)(u % pl.blocks) * R + rr;
  if (r >= (int64_t)a.B * N) return;
  m = kNegInf;
  l = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, ml_s[w][lane].x);
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const float2 ml = ml_s[w][lane];
    const float g = ml.x == m ? 1.f : ex2(ml.x - m);
    const float4 v = o_s[w][warp][lane];
    l = fmaf(ml.y, g, l);
    y.x = fmaf(v.x, g, y.x);
    y.y = fmaf(v.y, g, y.y);
    y.z = fmaf(v.z, g, y.z);
    y.w = fmaf(v.w, g, y.w);
  }
  const int b = (int)(r / N), head = h * N + (int)(r - (int64_t)b * N);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* dst = static_cast<T*>(a.out) + b * a.out_stride[0] + (int64_t)head * a.out_stride[1] + 4 * (d4 + warp);
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack16<T>(y.x * inv, y.y * inv), pack16<T>(y.z * inv, y.w * inv));
  if (d4 + warp == 0 && a.lse) a.lse[(int64_t)b * a.G + head] = l == 0.f ? kNegInf : (m + log2f(l)) * 0.69314718055994531f;
}

// One instantiation of the kernel.
template <typename Elem, int Dim, bool Pair>
struct PxKind {
  using T = Elem;
  static constexpr int D = Dim;
  static constexpr auto kernel = attend_prefix_kernel<Elem, Dim, Pair>;
};
template <typename F>
auto px_pick(int D, int dtype, bool pair, F&& f) {
  if (dtype == kBf16) {
    if (D == 64) return pair ? f(PxKind<__nv_bfloat16, 64, true>{}) : f(PxKind<__nv_bfloat16, 64, false>{});
    return pair ? f(PxKind<__nv_bfloat16, 128, true>{}) : f(PxKind<__nv_bfloat16, 128, false>{});
  }
  if (D == 64) return pair ? f(PxKind<__half, 64, true>{}) : f(PxKind<__half, 64, false>{});
  return pair ? f(PxKind<__half, 128, true>{}) : f(PxKind<__half, 128, false>{});
}

std::atomic<bool> g_off{false};   // test hook

// Strides between heads and rows, where a dimension of one has none of its own.
void row_strides(const int64_t* stride, int H, int P, int D, int64_t* hs, int64_t* rs) {
  *rs = P == 1 ? D : stride[1];
  *hs = H == 1 ? (int64_t)P * *rs : stride[0];
}

// Shared rows [H, P, D] as a 3-D tensor, the dimension of the smaller stride
// first; boxes of 64 elements (128 bytes) x 128 rows; rows past P read as zeros.
bool encode_rows(CUtensorMap* map, const void* base, const int64_t* stride, int H, int P, int D, int dtype,
                 bool* row_first) {
  auto enc = encode_fn();
  if (!enc) return false;
  int64_t hs, rs;
  row_strides(stride, H, P, D, &hs, &rs);
  *row_first = rs <= hs;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)(*row_first ? P : H), (cuuint64_t)(*row_first ? H : P)};
  const cuuint64_t strides[2] = {(cuuint64_t)(*row_first ? rs : hs) * 2, (cuuint64_t)(*row_first ? hs : rs) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)(*row_first ? kT : 1), (cuuint32_t)(*row_first ? 1 : kT)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, dtype == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// What TMA can describe: rows that are apart, strides below 2^40 bytes.
bool prefix_strides_fit(const int64_t* stride, int H, int P, int D) {
  int64_t hs, rs;
  row_strides(stride, H, P, D, &hs, &rs);
  return hs >= D && rs >= D && hs < ((int64_t)1 << 39) && rs < ((int64_t)1 << 39);
}

PrefixPlan prefix_plan(int B, int G, int H, int D, int P, bool own, Streamed stream, int sms) {
  PrefixPlan pl{};
  const int64_t rows = (int64_t)B * (G / H);
  // The row kernel reads the prefix once for every sequence (and 16 query heads),
  // from L2 after the first: faster while that is little, as this kernel and its
  // join take 11 us at least. 32 query heads on 8 of 128, no own rows, this | that:
  // 8 x 2048 shared rows (67 MB) 12 | 13 us, 16 x 2048 12 | 21, 4 x 2048 12 | 10; beside
  // 256 own rows 16 x 2048 (134 MB) 16 | 22, 8 x 2048 16 | 14.
  const int64_t visits = (int64_t)B * ((G / H + 15) / 16);
  if (visits < 2 || (double)visits * H * P * D * 4 < (own ? 96e6 : 64e6)) return pl;   // ctas = 0
  pl.pair = rows <= kT;
  pl.block_rows = pl.pair ? kT : 2 * kT;
  pl.blocks = (int)((rows + pl.block_rows - 1) / pl.block_rows);
  pl.nkt = (P + kT - 1) / kT;
  pl.units = H * pl.blocks;
  pl.final = !own;
  const int64_t total = pl.total();
  int64_t most = std::min<int64_t>(sms, pl.pair ? (total + 1) / 2 : total);
  if (stream.bytes > 0) {
    // The row kernel streams its rows on the other SMs meanwhile. Both times by SM
    // count, in us: this kernel's start and end and its longest range of tiles; the
    // stream's, 1.8 a unit of its CTAs and its bytes at 50 GB/s a SM. The split whose longer one is
    // shortest (32 sequences on 16384 shared + 512 own rows: 33 us against 44
    // one after the other; 8192 + 2048: 51 against 84 with the SMs shared by rows read).
    const double tile = pl.pair ? (D == 128 ? 1.4 : 0.9) : (D == 128 ? 1.9 : 1.5);
    double best = 1e30;
    int64_t at = most;
    for (int64_t p = 1; p <= std::min<int64_t>(most, sms - 4); ++p) {
      const double mine = 8.0 + tile * (double)((total + p - 1) / p);
      const double rows = 3.0 + 1.8 * (double)stream.units / stream_ctas(D, (int)(sms - p)) +
                          (double)stream.bytes / (50e3 * (double)(sms - p));
      if (std::max(mine, rows) < best) {
        best = std::max(mine, rows);
        at = p;
      }
    }
    most = at;
  }
  pl.ctas = (int)most;
  if (pl.units <= most) {
    const int split = (int)std::min<int64_t>(most / pl.units, pl.nkt);
    if ((int64_t)split * pl.units * 20 >= most * 17) {
      pl.split = split;
      pl.ctas = split * pl.units;
    }
  }
  pl.slots = own ? pl.units + sms : 2 * (int64_t)pl.ctas;
  return pl;
}

size_t PrefixPlan::o_bytes(int D) const { return (size_t)slots * block_rows * D * 4; }
size_t PrefixPlan::bytes(int D) const { return ctas ? o_bytes(D) + (size_t)slots * block_rows * 8 : 0; }
bool PrefixPlan::shared_blocks() const {
  for (int c = 1; c < ctas; ++c)
    if (start(c) % nkt) return true;
  return false;
}

bool prefix_kernel_ready(int D, int dtype, bool pair, int device) {
  if (g_off.load(std::memory_order_relaxed) || !encode_fn()) return false;
  return px_pick(D, dtype, pair, [&](auto kind) {
    using K = decltype(kind);
    // The kernel's redistribution of registers needs the 168 a thread that its
    // launch bound gives it: checked, as it would wait forever with fewer.
    static std::atomic<uint64_t> ready{0};   // devices on which that, and its shared memory, are settled
    const uint64_t bit = 1ull << device;
    if (ready.load(std::memory_order_relaxed) & bit) return true;
    cudaFuncAttributes f;
    if (cudaFuncGetAttributes(&f, K::kernel) != cudaSuccess || f.numRegs != 168 ||
        cudaFuncSetAttribute(K::kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PxGeo<K::D>::SMEM) != cudaSuccess) {
      (void)cudaGetLastError();
      return false;
    }
    ready.fetch_or(bit, std::memory_order_relaxed);
    return true;
  });
}

void prefix_kernel_off(bool off) { g_off.store(off); }

cudaError_t launch_attend_prefix(const PrefixArgs& args, int D, int dtype, cudaStream_t s) {
  PrefixArgs p = args;
  CUtensorMap kmap, vmap;
  if (!encode_rows(&kmap, p.a.pk, p.a.pk_stride, p.a.H, p.a.P, D, dtype, &p.k_row_first) ||
      !encode_rows(&vmap, p.a.pv, p.a.pv_stride, p.a.H, p.a.P, D, dtype, &p.v_row_first))
    return cudaErrorInvalidValue;
  return px_pick(D, dtype, p.plan.pair, [&](auto kind) {
    using K = decltype(kind);
    K::kernel<<<p.plan.ctas, kPxThreads, PxGeo<K::D>::SMEM, s>>>(kmap, vmap, p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.plan.final || !p.plan.shared_blocks()) return e;
    const dim3 grid(std::min(p.plan.units, p.plan.ctas - 1), p.plan.block_rows / 32, K::D / 32);
    return launch_after(attend_join_kernel<typename K::T, K::D>, grid, 256, 0, 1, true, s, p);
  });
}

}  // namespace kvx
