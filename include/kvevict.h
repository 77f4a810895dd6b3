/*
 * kvevict.h -- C ABI of the GB300 (sm_103a) cumulative proxy-attention
 * KV-cache eviction library: H2O-adapted, Keyformer-adapted (Gumbel
 * regulariser with an annealed temperature) and PyramidKV-adapted (per-layer
 * budget taper), all one decode step.
 *
 * What one step computes, for every (batch, layer, KV head) row of the cache
 * (page "veloxquant_mlx.quantizers.keyformer module", keyformer_update steps
 * 1-3; page "PyramidKV -- Layer-Adaptive Budget Attention-Mass Eviction",
 * "How it works"):
 *   1. append the new fp16 key k with score 0, its absolute position p and a
 *      frozen Gumbel value g(seed, layer, head, p);
 *   2. attn = softmax(K k / sqrt(D)) over every stored row, the new one
 *      included; scores += attn;
 *   3. if the layer's budget is exceeded, evict the lowest
 *      score + tau(p) * g over rows n_sink <= j < n+1-recent (lowest slot on
 *      ties); the
 *      rows after it move down one slot in order, each key re-rotated by -1
 *      RoPE position in fp32 and stored as fp16.
 *
 * Conventions shared by every entry point:
 *  - fp16 values cross the boundary as uint16_t bit patterns (IEEE binary16).
 *  - Device pointers are CUDA global-memory pointers on the device that was
 *    current at kvevict_create (mapped page-locked host memory counts as
 *    one); device key and value buffers must start on a 16-byte boundary
 *    (INVALID_ARG otherwise). Host pointers are plain host memory; the
 *    host-buffer entry point moves page-locked buffers with its own kernels
 *    (see kvevict_run_host).
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream). All work
 *    is enqueued on it; calls return before the GPU finishes unless stated.
 *  - The caller owns every buffer it passes and keeps it alive until the
 *    stream has passed the call. The library owns its state arena.
 *  - Return codes: 0 on success, else one of KVEVICT_ERR_*; the message of the
 *    last failure on the calling thread is kvevict_last_error().
 *  - One handle is not thread-safe; use one handle per thread or lock.
 */
#ifndef KVEVICT_H
#define KVEVICT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KVEVICT_OK 0
#define KVEVICT_ERR_INVALID_ARG (-1)  /* bad config, pointer or size */
#define KVEVICT_ERR_BAD_STATE (-2)    /* call out of order (e.g. prefill after a step) */
#define KVEVICT_ERR_CUDA (-3)         /* a CUDA runtime call failed */
#define KVEVICT_ERR_OOM (-4)          /* device allocation failed */
#define KVEVICT_ERR_DEVICE_CHECK (-5) /* a kernel raised its error word (bounded wait ran out) */
#define KVEVICT_ERR_WORKSPACE (-6)    /* kvevict_attend*: the workspace is missing, too small or not aligned */

#define KVEVICT_MAX_LAYERS 256
#define KVEVICT_MAX_PREFILL 16384

/* Cache configuration (page "veloxquant_mlx.quantizers.keyformer module",
 * KeyformerState and init_keyformer_state; page "PyramidKV ...", Parameters). */
typedef struct kvevict_config {
  int32_t batch;          /* B >= 1 */
  int32_t n_layers;       /* L, 1 .. KVEVICT_MAX_LAYERS */
  int32_t n_kv_heads;     /* H >= 1 */
  int32_t head_dim;       /* D, 64 or 128 */
  int32_t avg_budget;     /* average kept rows per layer, sinks included */
  double pyramid_beta;    /* >= 1; 1 = the same budget in every layer (plain H2O) */
  const int32_t* layer_budgets; /* optional host array [n_layers]; overrides avg/beta */
  int32_t n_sink;         /* leading rows never evicted, >= 0; every budget >= n_sink + 1 */
  float tau_init;         /* Gumbel temperature at position 0, >= 0 */
  float tau_end;          /* temperature once position >= anneal_steps, >= 0 */
  int32_t anneal_steps;   /* >= 0; 0 = constant tau_init */
  double rope_theta;      /* RoPE base of the model's attention, > 0 */
  uint64_t seed;          /* base seed of the frozen Gumbel values */
  int32_t max_prefill;    /* longest prompt kvevict_prefill will take, 0 .. KVEVICT_MAX_PREFILL */
  int32_t recent;         /* trailing protected window, >= 0; 0 = off (keyformer page,
                             KeyformerState.recent); every budget >= n_sink + recent + 1 */
  int32_t score_mode;     /* KVEVICT_SCORE_CUMULATIVE (H2O rule) or KVEVICT_SCORE_CURRENT */
  int32_t prefill_mode;   /* KVEVICT_PREFILL_BULK or KVEVICT_PREFILL_SEQUENTIAL */
  int32_t with_values;    /* 1: the cache also holds value rows (fp16 [.., D]); they move with
                             their keys and are never rotated (keyformer page,
                             KeyformerState.values); 0: keys only */
  int32_t decode_kernel;  /* KVEVICT_DECODE_AUTO (0), KVEVICT_DECODE_STREAM or
                             KVEVICT_DECODE_RESIDENT: which kernel runs the decode steps */
} kvevict_config;

/* Decode kernels; both compute the same steps and give the same results bit
 * for bit. STREAM: every step streams each row's keys from device memory
 * through shared memory, any row length. RESIDENT: a call of several steps
 * keeps each row in one CTA's shared memory for all of them (key-only handles
 * whose rows fit: about 780 keys at head_dim 128, 1023 at 64; the rows of a
 * large cache run in waves). AUTO takes RESIDENT for calls of at least 4
 * steps on key-only handles whose rows fit in one wave of CTAs, or in two at
 * two CTAs an SM, and STREAM otherwise (kvevict_decode_kernel_for reports the
 * choice); asking for RESIDENT on a handle whose rows do not fit, or that
 * carries values, is INVALID_ARG at create. */
#define KVEVICT_DECODE_AUTO 0
#define KVEVICT_DECODE_STREAM 1
#define KVEVICT_DECODE_RESIDENT 2

/* Prompt modes. BULK: score the whole prompt, then a row over budget evicts its
 * lowest (score + tau(S-1) * g, slot) rows at once. SEQUENTIAL: every prompt
 * token is absorbed as one step (page "veloxquant_mlx.quantizers.keyformer
 * module", keyformer_update: "For each of the S incoming tokens", steps 1-3),
 * so evictions happen inside the prompt, each with tau at its own position. */
#define KVEVICT_PREFILL_BULK 0
#define KVEVICT_PREFILL_SEQUENTIAL 1

/* Score modes (page "PyramidKV ...", method table): cumulative attention mass
 * (H2O-adapted, Keyformer-adapted, PyramidKV-adapted) or the current step's
 * attention weight (TOVA-adapted; a prompt then scores each token by the
 * prompt's last token's attention). */
#define KVEVICT_SCORE_CUMULATIVE 0
#define KVEVICT_SCORE_CURRENT 1

typedef struct kvevict kvevict_t;

/* Per-layer budget taper, host only (page "PyramidKV ...", "The budget
 * schedule"): linear from its maximum at layer 0 to its minimum at the last
 * layer, mean avg_budget, each >= n_sink + 1; beta = 1 is flat. Half-spread
 * h = min((beta-1)*avg, avg-(n_sink+1)); layer l gets
 * avg + round(h*(1 - 2l/(L-1))), the offset rounded half away from zero.
 * out: host int32[n_layers]. Errors: INVALID_ARG if beta < 1, n_layers < 0,
 * n_sink < 0 or avg_budget < n_sink + 1. */
int kvevict_budgets(int32_t n_layers, int32_t avg_budget, int32_t n_sink, double beta,
                    int32_t* out);

/* Validate cfg, compute the budgets and allocate the device state on the
 * current device: per row of the cache, (budget_l + 1) x D fp16 keys plus
 * float scores, float Gumbel values and int32 positions, and prefill scratch
 * for max_prefill tokens. The state starts empty (position 0).
 * Errors: INVALID_ARG (tau < 0, beta < 1, a budget <= n_sink, D not 64/128,
 * null pointers, sizes out of range), OOM, CUDA. *out is set only on success. */
int kvevict_create(const kvevict_config* cfg, void* stream, kvevict_t** out);

/* Free the handle and its device memory (synchronises the device first).
 * The pages keep a cache's state in a KeyformerState object that lives as long
 * as its owner holds it (page "veloxquant_mlx.quantizers.keyformer module",
 * KeyformerState); this ends the life of the device arena holding it here.
 * Errors: none (a null handle is ignored). */
int kvevict_destroy(kvevict_t* h);

/* Return the handle to the empty state at position 0 (the arena is reused). */
int kvevict_reset(kvevict_t* h, void* stream);

/* Absorb a prompt of S tokens at positions 0..S-1 (the state must be empty).
 * keys: device fp16 [B, L, H, S, D], each key already RoPE-rotated at its
 * position. Scores are the column sums of the causal softmax(K K^T/sqrt(D))
 * (the diagonal included), i.e. what S decode steps without eviction would
 * accumulate. A row whose layer budget b is below S then bulk-evicts the
 * S - b non-sink rows with the lowest (score + tau(S-1) * g, slot); survivors
 * keep their order and each is re-rotated by (new slot - old slot).
 * Errors: INVALID_ARG (null keys, S < 0 or S > max_prefill), BAD_STATE (state
 * not empty), CUDA. */
int kvevict_prefill(kvevict_t* h, const uint16_t* keys, int32_t S, void* stream);

/* kvevict_prefill with an optional log of the prompt's evictions: evicted is
 * device int32 [S, B, L, H] or NULL; in SEQUENTIAL mode entry [t] is the slot
 * the token at position t evicted (index into the rows after its append) or
 * -1; in BULK mode every entry is -1 (the bulk choice shows in the kept
 * positions). SEQUENTIAL mode runs the first min(S, smallest budget) tokens
 * through the prompt scorer (no row can evict yet, so this equals as many
 * single steps) and each further token as one decode step read straight from
 * the prompt buffer. Errors: as kvevict_prefill. */
int kvevict_prefill_ex(kvevict_t* h, const uint16_t* keys, int32_t S, int32_t* evicted,
                       void* stream);

/* The value-carrying forms (handles created with with_values = 1; the
 * key-only calls above return INVALID_ARG on such a handle). values /
 * v_new have the layouts of keys / k_new: device fp16 [B, L, H, S, D],
 * [B, L, H, D] and [T, B, L, H, D]. A value row is stored, moved and evicted
 * with its key; it is never rotated. Errors: as the key-only forms. */
int kvevict_prefill_kv(kvevict_t* h, const uint16_t* keys, const uint16_t* values, int32_t S,
                       int32_t* evicted, void* stream);
int kvevict_step_kv(kvevict_t* h, const uint16_t* k_new, const uint16_t* v_new, int32_t* evicted,
                    void* stream);
int kvevict_decode_kv(kvevict_t* h, const uint16_t* keys, const uint16_t* values, int32_t T,
                      int32_t* evicted, void* stream);

/* Copy one row's value rows to host memory (synchronises the stream):
 * values [n, D] fp16 bits in slot order, n = *n_kept. Errors: INVALID_ARG
 * (indices out of range, or a key-only handle), CUDA, DEVICE_CHECK. */
int kvevict_read_values(kvevict_t* h, int32_t b, int32_t l, int32_t head, uint16_t* values,
                        int32_t* n_kept, void* stream);

/* One decode step for every row at position p = kvevict_next_pos(): the
 * three steps of keyformer_update for one incoming token (page
 * "veloxquant_mlx.quantizers.keyformer module"), applied to every (batch,
 * layer, KV head) row at once as keyformer_update_batched applies them to
 * every (batch, head) row of a layer, with each layer's own budget (page
 * "PyramidKV ...", "How it works").
 * k_new: device fp16 [B, L, H, D], RoPE-rotated at p. evicted: device int32
 * [B, L, H] or NULL; receives the evicted slot (index into the rows after the
 * append, 0..n) or -1 when the row was within budget. One fused kernel launch.
 * Errors: INVALID_ARG (null k_new), CUDA. */
int kvevict_step(kvevict_t* h, const uint16_t* k_new, int32_t* evicted, void* stream);

/* T consecutive decode steps at positions p .. p + T - 1 in one kernel launch:
 * the same result as T kvevict_step calls. Rows are independent, so a row's
 * step t + 1 starts as soon as its own step t is done, with no wait for the
 * rest of the cache between steps.
 * keys: device fp16 [T, B, L, H, D]; evicted: device int32 [T, B, L, H] or NULL.
 * Errors: as kvevict_step; T < 0 is INVALID_ARG, T = 0 does nothing,
 * BAD_STATE once more than 2^31 - 1 decode steps follow a reset. */
int kvevict_decode(kvevict_t* h, const uint16_t* keys, int32_t T, int32_t* evicted,
                   void* stream);

/* End to end from host memory: prefill S prompt keys (host fp16
 * [B, L, H, S, D]; S may be 0) then T decode steps (host fp16 [T, B, L, H, D]),
 * with the evicted slots written back to host int32 [T, B, L, H] (or NULL).
 * The state must be empty. Returns after the stream has finished.
 * Each buffer must be one allocation. A page-locked buffer (cudaHostAlloc,
 * cudaMallocHost or cudaHostRegister; both its ends are checked) is accessed
 * by the library's kernels through its device mapping: the prompt is staged
 * to the device by a copy kernel, the decode keys are read in place by the
 * decode step, and the evicted slots are written back by a copy kernel.
 * Pageable memory goes through cudaMemcpyAsync in chunks on a second stream
 * that overlap with compute. Device staging (up to 2 x 256 MiB, or one batch's
 * prompt) is allocated on first use and kept with the handle.
 * Errors: INVALID_ARG, BAD_STATE, OOM, CUDA, DEVICE_CHECK. */
int kvevict_run_host(kvevict_t* h, const uint16_t* prefill_keys, int32_t S,
                     const uint16_t* decode_keys, int32_t T, int32_t* evicted, void* stream);
/* (key-only handles; a with_values handle returns INVALID_ARG) */

/* Apply the compaction the last decode step decided: the second half of
 * keyformer_update step 3 (page "veloxquant_mlx.quantizers.keyformer module":
 * survivors after the evicted token shift down by one and are re-rotated),
 * which this library defers (the step kernel leaves
 * the evicted row in place and the next step or this call removes it while
 * re-rotating the rows that move). kvevict_read_state calls it itself; a
 * caller that reads the device arena by other means, or that wants a step's
 * work finished in full inside a timed region, calls it explicitly. One
 * kernel launch; a no-op for rows with nothing pending. Errors: CUDA. */
int kvevict_flush(kvevict_t* h, void* stream);

/* Copy one row's state to host memory (synchronises the stream): the keys
 * keyformer_get_kv returns and the KeyformerState fields scores, gumbel and
 * positions (page "veloxquant_mlx.quantizers.keyformer module"; values:
 * kvevict_read_values). Rows
 * are given in slot order: keys [n, D] fp16 bits, scores [n], gumbel [n],
 * positions [n] (the original absolute position of each kept key), n =
 * *n_kept = min(next_pos, budget of layer l). Buffers need room for
 * budget_l + 1 rows; any of the four may be NULL. Errors: INVALID_ARG
 * (indices out of range), CUDA, DEVICE_CHECK. */
int kvevict_read_state(kvevict_t* h, int32_t b, int32_t l, int32_t head, uint16_t* keys,
                       float* scores, float* gumbel, int32_t* positions, int32_t* n_kept,
                       void* stream);

/* Synchronise the stream and report a kernel error word (DEVICE_CHECK) if set.
 * After DEVICE_CHECK the state is not valid; kvevict_reset clears the error
 * word and the state, after which the handle works as a new one. */
int kvevict_check(kvevict_t* h, void* stream);

/* Test hook for the failure path, with no counterpart on the pages. With a
 * handle: in its next decode launch, the first CTA's copy of its first key
 * tile (the resident step: of its row) is never issued, so a wait on it runs
 * out (4 s) and the kernel sets the handle's error word (wait timeout) and
 * returns. With h = NULL: the next
 * launch of the tensor-core prompt scorer in this process (kvevict_prefill of
 * any handle in a cumulative score mode, or kvevict_prefill_scores_noalloc)
 * never issues the query-tile copy of its first work item, with the same
 * outcome: a
 * handle then reports DEVICE_CHECK, the allocation-free call writes NaN
 * scores. A launch of kvevict_attend's prefix kernel that comes first takes the
 * hook instead (its first key tile), and writes NaN; so does one of
 * the tensor-core kernel of kvevict_attend_prompt and kvevict_attend_tree. Nothing faults or hangs. One-shot. Errors: none. */
int kvevict_test_stall_next_step(kvevict_t* h);

/* Position the next decode key will occupy (= tokens absorbed so far): the
 * KeyformerState.next_pos counter, one value shared by every row (page
 * "veloxquant_mlx.quantizers.keyformer module", KeyformerState and
 * keyformer_update_batched). *p: host int64. Errors: INVALID_ARG (null). */
int kvevict_next_pos(const kvevict_t* h, int64_t* p);

/* Which decode kernel a call of T steps runs on this handle (the choice
 * kvevict_decode / kvevict_step make, see KVEVICT_DECODE_*): *kernel is
 * KVEVICT_DECODE_STREAM or KVEVICT_DECODE_RESIDENT. Host only. Errors:
 * INVALID_ARG (null pointers, T < 0). */
int kvevict_decode_kernel_for(const kvevict_t* h, int32_t T, int32_t* kernel);

/* Budget of layer l as resolved at create time. */
int kvevict_layer_budget(const kvevict_t* h, int32_t l, int32_t* budget);

/* Per-layer cache statistics, host arithmetic only (page "PyramidKV ...":
 * each layer's cache exposes layer_budget, compression_ratio and
 * tokens_kept; page "veloxquant_mlx.quantizers.keyformer module":
 * keyformer_fp16_bytes, full_keyformer_fp16_bytes). For layer l, with p the
 * tokens seen (kvevict_next_pos):
 *   tokens_kept  = min(p, budget_l), the rows each (batch, KV head) row holds;
 *   stored_bytes = B * H * tokens_kept * D * 2 bytes of fp16 keys, doubled
 *                  on a value-carrying handle (scores, Gumbel values and
 *                  positions are bookkeeping, not counted, as on the
 *                  keyformer page);
 *   full_bytes   = the same with p tokens: what keeping every token takes;
 *   compression_ratio = full_bytes / stored_bytes (1 while p = 0).
 * Any output pointer may be NULL. Errors: INVALID_ARG (null handle, layer
 * out of range). */
int kvevict_layer_stats(const kvevict_t* h, int32_t l, int32_t* tokens_kept, uint64_t* stored_bytes,
                        uint64_t* full_bytes, double* compression_ratio);

/* Device bytes held by the handle (arena + scratch + staging). */
int kvevict_device_bytes(const kvevict_t* h, size_t* bytes);

/* Checkpoint and resume. The pages keep the state in an immutable object
 * returned by each call (page "veloxquant_mlx.quantizers.keyformer module",
 * KeyformerState); here it lives in the handle's device arena, and these calls
 * copy it to and from host memory. A snapshot holds every row's keys (and
 * values), scores, Gumbel values and positions, the next position and whether
 * a decode step has run, plus the handle's shape, layer budgets and method
 * parameters (n_sink, recent, score mode, tau schedule, RoPE base, seed); the
 * frozen Gumbel values depend only on (seed, layer, head, position), so a
 * resumed handle continues exactly as the saved one would have.
 *
 * kvevict_state_bytes: size of a snapshot of this handle.
 * kvevict_save_state: applies any pending compaction (as kvevict_flush), then
 *   copies the state into buf (host memory, at least kvevict_state_bytes
 *   bytes, caller-owned); returns after the stream has finished. Errors:
 *   INVALID_ARG (null, buffer too small), CUDA, DEVICE_CHECK (the handle's
 *   error word is set; buf's contents are then unspecified).
 * kvevict_load_state: replaces this handle's state with the snapshot in buf
 *   (host memory, bytes long); returns after the stream has finished, so buf
 *   may be freed. The handle must have the snapshot's batch, layers, KV heads,
 *   head_dim, value rows, layer budgets and method parameters; max_prefill and
 *   prefill_mode may differ. Errors: INVALID_ARG (not a snapshot, a size or
 *   configuration mismatch; the handle is unchanged), CUDA. */
int kvevict_state_bytes(const kvevict_t* h, size_t* bytes);
int kvevict_save_state(kvevict_t* h, void* buf, size_t bytes, void* stream);
int kvevict_load_state(kvevict_t* h, const void* buf, size_t bytes, void* stream);

/* Prompt scoring that allocates nothing. The paper has no counterpart: this is
 * for callers that cannot call cudaMalloc -- an inference engine that reserves
 * the whole device heap for its own memory pool at start-up (a further
 * cudaMalloc then fails or fragments that pool), or a latency-bound serving
 * loop that cannot take cudaMalloc's implicit device-wide synchronisation.
 * It runs the same two tensor-core passes as kvevict_prefill's scorer and
 * writes each row's causal softmax column sums (diagonal included): the
 * scores kvevict_prefill gives a prompt before any eviction.
 *   keys:   device fp16 [heads, S, D], each key RoPE-rotated at its position.
 *   colsum: device float [heads, S], written in full by the call.
 * Working memory is a fixed 16 MiB device array inside the library, present on
 * every GPU that loads the library until the process exits. It limits a call
 * to 2 * heads * round_up(S, 128) <= 4,194,304 floats (for example 512 rows of
 * 4096 tokens); a larger call returns INVALID_ARG without launching anything.
 * Every call shares that array and leaves its contents behind; nothing in it
 * needs to start at zero, since a call reads only entries it wrote itself
 * (padding entries it reads are masked out). Calls whose work overlaps on the
 * GPU (other streams, other threads) race on the array: serialise them.
 * A failure on the GPU cannot reach the return code, which comes back before
 * the GPU runs the call: if one of the scorer's bounded waits runs out (4 s),
 * the call writes NaN to every entry of colsum instead of scores, so a caller
 * that must know checks colsum for NaN after the stream has passed the call.
 * (A device error word beside the array records it. It and the scorer's two
 * work-item counters, also beside the array, are cleared by each call first
 * with cudaMemsetAsync, which allocates nothing.)
 * The first call on each device (and head_dim) looks up the device addresses
 * of the array and the error word, the device's multiprocessor count, and sets
 * the kernels' shared-memory attribute, with that device current; make that
 * first call before any stream capture. The addresses are kept for the life of
 * the process: do not reset the device (cudaDeviceReset) after the first call.
 * With lazy module loading the driver places the array when the library's
 * kernels first load, which can be during that first call. Errors:
 * INVALID_ARG (null pointers, keys not 16-byte aligned, head_dim not 64/128,
 * negative or over-limit sizes), CUDA. */
int kvevict_prefill_scores_noalloc(const uint16_t* keys, int32_t heads, int32_t S,
                                   int32_t head_dim, float* colsum, void* stream);

/* ------------------------------------------------------------------------
 * Around the step: what makes a token's keys, and what reads the cache.
 * The pages leave both to the model that owns the cache (page
 * "veloxquant_mlx.quantizers.keyformer module", keyformer_get_kv hands keys and
 * values to its attention); these are that model's two operators on this
 * library's layouts. A decoding layer l calls, per token,
 *     kvevict_qk_norm_rope   queries and keys of the token
 *     kvevict_attend_cache   its attention over layer l's rows and itself
 * and, once every layer has run, kvevict_step_kv inserts the token's keys and
 * values and evicts.
 *
 * Both hold no state and allocate nothing on the device. They run on the
 * device that is current, which must be the one the pointers belong to. Their
 * descriptions are read before the call returns. Strides count elements; the
 * last dimension is contiguous, pointers start on a 16-byte boundary and the
 * stride of every dimension of more than one entry is a multiple of 16 bytes;
 * inputs may broadcast (strides of 0), the rows of outputs lie apart. Calls may
 * overlap on any streams and threads as long as none writes what another uses. */
#define KVEVICT_DTYPE_FP16 0
#define KVEVICT_DTYPE_BF16 1
#define KVEVICT_DTYPE_FP32 2   /* inputs and weights of kvevict_qk_norm_rope only */

typedef struct kvevict_qk {
  int32_t in_dtype;       /* of q and k: FP16, BF16 or FP32 */
  int32_t out_dtype;      /* of q_out and k_out: FP16 (the cache's) or BF16 */
  int32_t weight_dtype;   /* of q_weight and k_weight: FP16, BF16 or FP32 */
  int32_t batch, seq;     /* >= 0 */
  int32_t n_heads;        /* query heads, >= 0 */
  int32_t n_kv_heads;     /* key heads, >= 0 */
  int32_t head_dim;       /* D, 64 or 128 */
  float eps;              /* of the norm, >= 0 */
  int32_t reserved;       /* 0 */
  double rope_theta;      /* RoPE base, > 0 and normal; the cache's kvevict_config.rope_theta */
  int64_t pos0;           /* position of token 0 where positions is null */
  const void* q;          /* device [batch, seq, n_heads, D]; null if n_heads = 0 */
  const void* k;          /* device [batch, seq, n_kv_heads, D]; null if n_kv_heads = 0 */
  void* q_out;            /* device, the shapes of q and k */
  void* k_out;
  const void* q_weight;   /* device [D], or null: queries are rotated without a norm */
  const void* k_weight;   /* device [D], or null */
  const int32_t* positions; /* device int32 [batch, seq], contiguous, or null: pos0 + s */
  int64_t q_stride[3];    /* between sequences, tokens and heads */
  int64_t k_stride[3];
  int64_t q_out_stride[3];
  int64_t k_out_stride[3]; /* any order: [B, H, S, D] is what kvevict_prefill takes */
} kvevict_qk;

/* RMS norm of every query and key head, y = x * w / sqrt(mean(x^2) + eps), and
 * the rotation of the pairs (i, i + D/2) by p * theta^(-2i/D), in fp32 with one
 * rounding to out_dtype. (Squares are summed in fp32, too: a head of elements
 * beyond 1e18 overflows to 0.) q_out may be q itself, and k_out k, with the same type
 * and strides; outputs overlap nothing else. Positions are any int32 (pos0 + s
 * too); angles are within 2^-21 of exact for rope_theta >= 1. One kernel launch. Errors: INVALID_ARG, CUDA. */
int kvevict_qk_norm_rope(const kvevict_qk* args, void* stream);

typedef struct kvevict_attention {
  int32_t dtype;          /* FP16 or BF16: q, out and every key and value */
  int32_t batch;          /* B, sequences with one query token each, >= 0 */
  int32_t n_heads;        /* G query heads, a multiple of n_kv_heads */
  int32_t n_kv_heads;     /* H >= 1 */
  int32_t head_dim;       /* D, 64 or 128 */
  int32_t n;              /* own rows a sequence has room for, >= 0 */
  int32_t prefix;         /* shared rows P, >= 0; n + prefix < 2^30 */
  int32_t reserved;       /* 0 */
  float scale;            /* of the logits, 2^-126 to 2^127; 0 = 1/sqrt(D) */
  int32_t reserved2;      /* 0 */
  const void* q;          /* device [B, G, D] */
  void* out;              /* device [B, G, D] */
  float* lse;             /* device float [B, G], contiguous, or null */
  const void* k;          /* device [B, H, n, D]; null if n = 0 */
  const void* v;
  const int32_t* lens;    /* device int32 [B]: sequence b has min(max(lens[b], 0), n) rows; null: n */
  const void* k_new;      /* device [B, H, D], the token's own key and value, or both null */
  const void* v_new;
  const void* prefix_k;   /* device [H, P, D], the rows all sequences share; null if P = 0 */
  const void* prefix_v;
  const int32_t* prefix_lens; /* device int32 [B]: sequence b shares the first min(max(.., 0), P); null: P */
  void* workspace;        /* device, kvevict_attend_workspace bytes, 16-byte aligned; null if that is 0 */
  int64_t q_stride[2];    /* between sequences and heads */
  int64_t out_stride[2];
  int64_t k_stride[3];    /* between sequences, heads and rows */
  int64_t v_stride[3];
  int64_t k_new_stride[2];
  int64_t v_new_stride[2];
  int64_t prefix_k_stride[2]; /* between heads and rows */
  int64_t prefix_v_stride[2];
  uint64_t workspace_bytes;
} kvevict_attention;

/* Attention of one query token a sequence: with s_j = q . k_j * scale over the
 * sequence's own rows, the token's own key (k_new) and the shared rows,
 *   out = sum_j e^(s_j) v_j / sum_j e^(s_j),   lse = log sum_j e^(s_j).
 * Query head i reads key head i / (G / H). A sequence with no rows at all gets
 * out = 0 and lse = -inf. Rows past a length are not read, whatever they hold.
 * The shared rows are read once for all sequences, not once for each; without
 * own rows the call is the prefix's part of a longer attention (a prompt
 * chunk's tokens given as sequences), and lse joins it with the rest. Logits,
 * softmax and sums are fp32; out is rounded once, and where many query rows share a prefix
 * every weight of its rows, too, before its product with v_j. out and lse overlap no input.
 * A key whose logit is NaN or +inf makes its sequences' out and lse NaN; one of
 * -inf takes no weight. A value that is NaN or infinite shows in its column of
 * out as NaN or infinite (which of the two depends on the sizes: a weight is
 * split in two, and 0 times infinity is NaN), whatever its row's weight. Where
 * prefix_lens differ, such a value may show in sequences that do not share
 * its row (their weight of it is 0), such a key does not; rows past the longest
 * length are not looked at. Waits in the prefix's kernel are bounded
 * (4 s); one that runs out leaves NaN in out and lse, and on a handle sets its
 * error word (kvevict_check).
 * The workspace holds nothing between calls and needs no initial value; calls
 * that may run at the same time (captured graphs too) need one each.
 * Errors: INVALID_ARG, CUDA, WORKSPACE (nothing has been launched: ask
 * kvevict_attend_workspace for the size and call again). */
int kvevict_attend(const kvevict_attention* args, void* stream);

/* Test hook: while `without` is not 0, calls of this process are planned as if
 * the prefix's tensor-core kernel could not be launched (a driver without tensor maps, a
 * compiler that gave the kernel other registers): the row kernel then reads the shared rows
 * itself, with the same results. Not while a call is under way. Errors: none. */
int kvevict_test_without_prefix_kernel(int32_t without);

/* Device bytes that a call of this description needs as workspace, on the
 * current device; of the pointers only k_new counts (whether it is null).
 * with_cache: 1 for
 * kvevict_attend_cache, 0 for kvevict_attend. *bytes: host. Errors:
 * INVALID_ARG, CUDA. */
int kvevict_attend_workspace(const kvevict_attention* args, int32_t with_cache, size_t* bytes);

/* kvevict_attend with layer l's kept rows of a value-carrying handle as the own
 * rows: keys and values as kvevict_read_state and kvevict_read_values give
 * them, a compaction still pending included, without changing the handle. batch,
 * n_kv_heads and head_dim are the handle's, dtype is FP16, and n, k, v and lens
 * must be 0 and null (the row count is min(next_pos, budget_l) when the call is
 * made: a captured call keeps it). q and k_new are rotated at position
 * kvevict_next_pos, or at `prefix` + kvevict_next_pos behind a prefix, whose rows
 * have the positions from 0 on: the prompt's keys were then rotated from `prefix`
 * on, too (the cache's own positions start at 0 all the same; only differences
 * count). Errors: as kvevict_attend; INVALID_ARG (a key-only handle,
 * another device current than the handle's, layer out of range). */
int kvevict_attend_cache(const kvevict_t* h, int32_t l, const kvevict_attention* args, void* stream);

/* ------------------------------------------------------------------------
 * Several tokens a sequence: the attention of whole prompts, before
 * kvevict_prefill takes their keys, and of trees of drafted tokens, before those
 * that are accepted go into the cache as steps (kvevict_decode_kv takes several).
 * The rules of the block above hold: no state, nothing allocated, the current
 * device, strides in elements. Queries, keys and values are read through tensor maps:
 * their strides are >= 0 and below 2^39, and tokens (rows), and heads of q, lie at least
 * D apart. */
#define KVEVICT_MAX_TREE 64   /* tokens of a tree */
#define KVEVICT_MAX_JOIN 8    /* parts that one join takes */

typedef struct kvevict_tokens {
  int32_t dtype;          /* FP16 or BF16: q, out and every key and value */
  int32_t batch;          /* B sequences, >= 0 */
  int32_t seq;            /* tokens a sequence has room for, S; with starts: of all sequences together, T */
  int32_t n_heads;        /* G query heads, a multiple of n_kv_heads */
  int32_t n_kv_heads;     /* H >= 1 */
  int32_t head_dim;       /* D, 64 or 128 */
  int32_t n;              /* own rows a sequence has room for, >= 0; n + seq < 2^30 */
  int32_t reserved;       /* 0 */
  float scale;            /* of the logits, 2^-126 to 2^127; 0 = 1/sqrt(D) */
  int32_t reserved2;      /* 0 */
  const void* q;          /* device [B, S, G, D]; with starts [T, G, D] */
  void* out;              /* device, the shape of q */
  float* lse;             /* device float [B, S, G] or [T, G], contiguous, or null */
  const void* k_new;      /* device [B, S, H, D] or [T, H, D]: the tokens' own keys and values */
  const void* v_new;
  const int32_t* starts;  /* device int32 [B + 1], ascending, or null: sequence b has the tokens
                             starts[b] .. starts[b + 1] - 1 of T (clamped to it) */
  const int32_t* new_lens; /* device int32 [B]: sequence b has min(max(new_lens[b], 0), S) tokens; null: S */
  const int32_t* parents; /* trees: device int32 [B, S], the token that each one continues, -1 where it
                             continues the sequence itself; null: the one before it */
  const void* k;          /* device [B, H, n, D]; null if n = 0: rows before the tokens */
  const void* v;
  const int32_t* lens;    /* device int32 [B]: sequence b has min(max(lens[b], 0), n) rows; null: n */
  void* workspace;        /* device, kvevict_attend_tokens_workspace bytes, 16-byte aligned; null if that is 0 */
  int64_t q_stride[3];    /* between sequences (with starts: not used), tokens and heads */
  int64_t out_stride[3];
  int64_t k_new_stride[3]; /* any order: [B, H, S, D] is what kvevict_prefill takes */
  int64_t v_new_stride[3];
  int64_t k_stride[3];    /* between sequences, heads and rows */
  int64_t v_stride[3];
  int64_t parents_stride; /* between sequences; 0: the same tree for all */
  uint64_t workspace_bytes;
} kvevict_tokens;

/* Causal attention of prompts: token i of a sequence sees the sequence's own rows
 * (k, v: an earlier chunk's) and its tokens 0 .. i; with s_j = q . k_j * scale over
 * those,
 *   out = sum_j e^(s_j) v_j / sum_j e^(s_j),   lse = log sum_j e^(s_j).
 * Query head i reads key head i / (G / H). Tokens behind a sequence's last are neither
 * read nor written: their out and lse stay as they are. Logits, softmax and sums are
 * fp32; out is rounded once, and in calls of many query rows every weight e^(s_j), too, before
 * its product with v_j (to dtype: half a step of each, at random). out and lse overlap no input.
 * A key whose logit is NaN or +inf makes out and lse of the query heads that see it
 * NaN; one of -inf takes no weight. A value that is NaN or infinite shows in its
 * column of out, as NaN or infinite, wherever it is seen and nowhere else. Rows and
 * tokens past a length may hold anything. Waits in the kernel are bounded (4 s); one
 * that runs out leaves NaN in out and lse, and on a handle sets its error word.
 * The workspace holds nothing between calls and needs no initial value; calls that
 * may run at the same time (captured graphs too) need one each.
 * Errors: INVALID_ARG (parents not null), CUDA, WORKSPACE (nothing has been launched:
 * ask kvevict_attend_tokens_workspace for the size and call again). */
int kvevict_attend_prompt(const kvevict_tokens* args, void* stream);

/* The same for drafted tokens that form a tree: token i sees the sequence's own rows,
 * itself, its parent, the parent's parent and so on. seq is at most KVEVICT_MAX_TREE
 * and starts null; a parent that is not before its token (or negative) counts as -1.
 * Errors: as kvevict_attend_prompt. */
int kvevict_attend_tree(const kvevict_tokens* args, void* stream);

/* kvevict_attend_tree with layer l's kept rows of a value-carrying handle as the own
 * rows, as kvevict_attend_cache has them (a compaction still pending included, the
 * handle unchanged). batch, n_kv_heads and head_dim are the handle's, dtype is FP16,
 * and n, k, v and lens must be 0 and null. A token at depth d of its tree (0: it
 * continues the sequence) is rotated at kvevict_next_pos + d. Errors: as
 * kvevict_attend_tree and kvevict_attend_cache. */
int kvevict_attend_tree_cache(const kvevict_t* h, int32_t l, const kvevict_tokens* args, void* stream);

/* Test hook: while `without` is not 0, calls of this process never take the kernel for
 * few query rows, but the tensor cores' whatever their size. Errors: none. */
int kvevict_test_without_few_kernel(int32_t without);

/* Test hook: while `without` is not 0, calls of this process are planned as if the tensor-core
 * kernel of kvevict_attend_prompt and kvevict_attend_tree could not be launched (a driver without
 * tensor maps, a compiler that gave the kernel other registers): the kernel for few query rows then
 * answers all of them, with the same results, large calls slowly. Errors: none. */
int kvevict_test_without_tokens_kernel(int32_t without);

/* Device bytes that a call of this description needs as workspace, on the current
 * device (at most); of the pointers only starts and parents count (whether they are null:
 * packed tokens; a tree's limits). with_cache: 1 for
 * kvevict_attend_tree_cache, else 0. *bytes: host. Errors: INVALID_ARG, CUDA. */
int kvevict_attend_tokens_workspace(const kvevict_tokens* args, int32_t with_cache, size_t* bytes);

typedef struct kvevict_join {
  int32_t dtype;          /* FP16 or BF16: of the parts and of out */
  int32_t batch, seq;     /* >= 0 */
  int32_t n_heads;        /* G >= 0 */
  int32_t head_dim;       /* D, 64 or 128 */
  int32_t parts;          /* 1 .. KVEVICT_MAX_JOIN */
  int32_t reserved[2];    /* 0 */
  const void* part[8];    /* device [batch, seq, G, D] each: outputs of attention over disjoint rows */
  const float* part_lse[8]; /* device float [batch, seq, G] each, contiguous: their lse */
  void* out;              /* device [batch, seq, G, D] */
  float* lse;             /* device float [batch, seq, G], contiguous, or null */
  int64_t part_stride[8][3]; /* between sequences, tokens and heads */
  int64_t out_stride[3];
} kvevict_join;

/* Joins parts of an attention over disjoint rows: lse = log sum_p e^(lse_p) and
 * out = sum_p e^(lse_p - lse) part_p, in fp32, rounded once. A part whose lse is -inf
 * takes no weight, whatever it holds; a head with no other gets out 0 and lse -inf. A
 * lse that is NaN or +inf makes out and lse NaN. out may be one of the parts, with the
 * same strides, and lse its lse; otherwise they overlap no input. One kernel launch.
 * Errors: INVALID_ARG, CUDA. */
int kvevict_attend_join(const kvevict_join* args, void* stream);

/* Message of the last failure on the calling thread ("" if none). */
const char* kvevict_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* KVEVICT_H */
