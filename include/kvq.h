/*
 * kvq.h -- C ABI of the certified quantized-KV decode-attention library (GB300, sm_103a).
 *
 * The method is "Runtime-Certified Bounded-Error Quantized Attention" (gist.science
 * technical summary).  Section names used below:
 *   Method §1  tiered storage: tier 1 in VRAM holds per-channel INT8 keys, per-group INT4
 *              values, their scale/offset metadata and a per-block error annotation;
 *              tier 2 keeps the unquantised FP16 keys and values in pinned system RAM as
 *              the ground truth for fallback.
 *   Method §2  two-term error decomposition: E_key bounds the total-variation distortion
 *              of the softmax caused by key quantisation through the per-token score
 *              perturbation Delta; E_val bounds the INT4 value reconstruction error as the
 *              attention-mass-weighted sum of the per-block errors eta_b.  Both come from
 *              quantities already tracked (scales, query norms, value ranges).
 *   Method §3  a light INT8 scoring pass estimates per-block attention mass; the top-K*
 *              blocks covering tau_cov of it get FP16 keys from tier 2; a ranking check
 *              compares INT8 and FP16 block orderings; a four-rung fallback ladder (more
 *              coverage, FP16 values, per-head dense, per-layer dense) follows.
 *   Contributions, "deterministic recovery": when the certified bound cannot be met the
 *              returned output is the dense FP16 attention O_dense.
 *
 * Conventions for every call
 *   - Shapes: B = batch, Hq = query heads, Hkv = KV heads, D = head_dim = 128, blocks of
 *     64 tokens, value groups of 32 channels.  Query head h uses KV head h / (Hq / Hkv).
 *   - FP16 data is IEEE binary16, passed as void*.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Work is enqueued on
 *     it in stream order; a call returns once its work is enqueued, unless it says
 *     otherwise.  One cache must not be used from two streams at once: every call
 *     reuses the cache's scratch memory.
 *   - Errors: every call returns a kvq_status; kvq_last_error() gives the text of the
 *     calling thread's last failure.  A failed call leaves the cache as it was, except
 *     after KVQ_ERR_CUDA, which reports an error of the CUDA runtime (the context may be
 *     unusable).
 *   - Inputs must be finite.
 */
#ifndef KVQ_H_
#define KVQ_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kvq_status {
  KVQ_OK = 0,
  KVQ_ERR_INVALID = 1,   /* bad argument, NULL pointer, unsupported shape, empty cache */
  KVQ_ERR_OOM = 2,       /* device memory allocation failed */
  KVQ_ERR_HOST_OOM = 3,  /* pinned host (tier-2) allocation failed */
  KVQ_ERR_CAPACITY = 4,  /* append beyond max_ctx tokens */
  KVQ_ERR_CUDA = 5,      /* a CUDA runtime call failed */
  KVQ_ERR_TIMEOUT = 6    /* reserved for bounded device waits */
} kvq_status;

/* Cache shape and the method's open parameters.  head_dim must be 128, block_tokens 64
 * and value_group 32; n_q_heads / n_kv_heads must be 1, 2, 3 or 4. */
typedef struct kvq_config {
  int n_layers;
  int batch;
  int n_q_heads;
  int n_kv_heads;
  int head_dim;
  int block_tokens;
  int value_group;
  int max_ctx;             /* tokens per sequence and layer, at most 2097152 */
  int rank_positions;      /* ranking check compares the top-R blocks (R >= 1; default 1) */
  float l4_head_fraction;  /* rung 4 when >= this fraction of a sequence's heads are at
                              rung 3 (in (0, 1]; default 0.5) */
  int value_bits;          /* 4 (or 0): INT4 values in VRAM, FP16 values in tier 2 (the
                              paper's configuration).  16: the paper's FP16-values ablation
                              (Results, structured reasoning): values stay FP16 in VRAM,
                              tier 2 holds keys only, E_val = 0 and rung 2 pages nothing
                              in; VRAM per token and KV head 388 B instead of 212 B (dense
                              FP16: 512 B) */
  float v_tol;             /* value tolerance: a head is certified only if also E_val <=
                              v_tol, and rung 2 pages in values until it holds (the paper's
                              v_tol, Results: structured reasoning).  0 (or +inf): no budget
                              beyond eps.  Must not be negative or NaN. */
  int resident_blocks;     /* cross-step residency (not part of the paper: an option of
                              this library).  Each layer may keep up to this many FP16
                              tier-2 blocks (keys or values, 16 KiB each) in device memory
                              across decode calls, so that a block paged in again by a
                              later call is read from HBM instead of over the host link.
                              A block read from tier 2 takes a free slot if one is left;
                              after each certified call the slots its layer did not use in
                              that call are freed.  Outputs and certificates are unchanged
                              (the copies are bit-identical).  Costs resident_blocks x
                              16 KiB of device memory per layer.  0 (the default): none. */
} kvq_config;

/* Per-head certificate of one decode call (Method §2, §3). */
typedef struct kvq_certificate {
  float e_key;             /* bound on the key-quantisation error of the output (max-abs) */
  float e_val;             /* bound on the value-reconstruction error (max-abs) */
  int32_t rank_ok;         /* 1 if the INT8 and FP16 rankings of the selected blocks agree */
  int32_t level;           /* ladder rung reached: 0 certified as is, 1 coverage expanded,
                              2 values promoted, 3 per-head dense, 4 per-layer dense */
  int32_t k_star;          /* blocks selected for this head by the top-K* pass */
  int32_t n_val_promoted;  /* value blocks paged in for the head's certified result */
  int64_t promoted_bytes;  /* FP16 tier-2 bytes paged in for this head's KV group during
                              the call (same for all heads of the group).  With
                              resident_blocks > 0 part of them may come from the resident
                              copies in HBM (kvq_residency_stats) */
} kvq_certificate;

typedef struct kvq_cache kvq_cache;

/* Debug flags for kvq_set_debug. */
#define KVQ_DEBUG_FORCE_RANK_FAIL 0x1  /* every ranking check reports inconsistency */
#define KVQ_DEBUG_FORCE_DENSE     0x2  /* every head takes rung 4 */
#define KVQ_DEBUG_SYNC            0x4  /* synchronise and check after every kernel */
#define KVQ_DEBUG_PROFILE         0x8  /* time every kernel with CUDA events */
#define KVQ_DEBUG_BOUNDS          0x10 /* kernels check the indices they address tier 1, tier 2
                                          and scratch with; the first one out of range is
                                          recorded (the access skipped, nothing traps) and
                                          the call synchronises and returns KVQ_ERR_INVALID
                                          naming the kernel */
#define KVQ_DEBUG_FAIL_MIRROR     0x20 /* test aid: kvq_append's tier-2 mirror copy reports a
                                          CUDA error without being issued; the call returns
                                          KVQ_ERR_CUDA and the cache keeps its length */

/* kvq_cache_create -- allocate tier 1 (device), tier 2 (pinned, mapped host memory) and
 * scratch for `n_layers` layers of `batch` sequences of up to `max_ctx` tokens (Method §1).
 * The library owns all of it until kvq_cache_destroy.  Uses the current CUDA device.
 * Errors: KVQ_ERR_INVALID (cfg NULL or unsupported), KVQ_ERR_OOM, KVQ_ERR_HOST_OOM,
 * KVQ_ERR_CUDA (no usable CUDA device, or initialising tier 1 failed). */
kvq_status kvq_cache_create(const kvq_config* cfg, kvq_cache** out);

/* kvq_cache_destroy -- synchronise the device and free everything.  NULL is a no-op. */
kvq_status kvq_cache_destroy(kvq_cache* cache);

/* kvq_append -- quantise-and-append `n_tokens` new tokens to every sequence of `layer`
 * (Method §1).  k and v are caller-owned device buffers [B, Hkv, n_tokens, D] of FP16,
 * 16-byte aligned.
 * Full 64-token blocks are quantised into tier 1 (INT8 keys with one fp16 scale per
 * block and channel; INT4 values with fp16 scale and offset per token and 32-channel
 * group; eta_b = max |v - v_hat| over the block); the partial last block stays FP16 in
 * VRAM until it fills.  Every token is also mirrored to tier 2 by a copy on an internal
 * side stream that `stream` waits for before any later work, so k and v may be reused
 * by later work on `stream`.  n_tokens = 0 is a no-op.
 * Errors: KVQ_ERR_INVALID (layer out of range, NULL, host or unaligned buffers,
 * n_tokens < 0), KVQ_ERR_CAPACITY (length would exceed max_ctx), KVQ_ERR_CUDA. */
kvq_status kvq_append(kvq_cache* cache, int layer, const void* k, const void* v,
                      int n_tokens, void* stream);

/* kvq_decode_attention -- certified decode attention of one query token per sequence
 * against the cached `layer` (Method §2, §3; deterministic recovery).
 *   q            [B, Hq, D] FP16, device or host memory
 *   tau_cov      coverage target in (0, 1]; tau_cov == 1 takes rung 4 for every head
 *   eps          certificate budget on E_key + E_val (max-abs over the head's output),
 *                eps >= 0; +inf accepts every head whose ranking check passes
 *   out          [B, Hq, D] FP16, device or host memory
 *   cert         [B * Hq] certificates (may be NULL), device or host memory
 *   ladder_level [B] highest rung reached per sequence (may be NULL), device or host
 * Host memory for any of q, out, cert or ladder_level is staged through the cache's own
 * device buffers.  Page-locked host buffers (cudaHostAlloc, cudaHostRegister) are copied
 * in stream order, like cudaMemcpyAsync: q is read when the stream reaches the call, and
 * out, cert and ladder_level hold the results once the stream has completed it.  If any
 * host buffer is pageable, the call synchronises `stream` before returning, so every
 * result is in place on return.  Device buffers are used in
 * place and must be aligned: q and out to 16 bytes, cert to 8, ladder_level to 4.  Tier-2 blocks are read
 * directly by the kernels through the host link (NVLink-C2C); no host round trip
 * happens inside the call.
 * Errors: KVQ_ERR_INVALID (layer out of range, empty layer, tau_cov outside (0, 1],
 * eps < 0 or NaN, NULL q/out, unaligned device buffers), KVQ_ERR_CUDA. */
kvq_status kvq_decode_attention(kvq_cache* cache, int layer, const void* q, float tau_cov,
                                float eps, void* out, kvq_certificate* cert,
                                int32_t* ladder_level, void* stream);

/* kvq_decode_attention_uncertified -- plain quantized decode attention: INT8 key scores
 * and INT4 values on every full block, exact FP16 on the partial block.  No block is
 * paged in from tier 2, no ranking check runs and no rung of the fallback ladder is
 * taken.  This is the uncertified INT8/INT4 baseline that the paper sets against the
 * certified path (Experiments, retrieval), and the speed ceiling of the tier-1 data.
 *   q, out, stream  as kvq_decode_attention
 *   cert            [B * Hq] (may be NULL): e_key and e_val are the bounds of this output,
 *                   computed as in kvq_decode_attention but not enforced; rank_ok 1,
 *                   level 0, k_star 0, n_val_promoted 0, promoted_bytes 0.
 * Debug flags that force rungs are ignored.  The selection state it leaves (nothing
 * selected) is what kvq_export_decode_state reports afterwards.
 * Errors: KVQ_ERR_INVALID (layer out of range, empty layer, NULL q/out, unaligned
 * device buffers), KVQ_ERR_CUDA. */
kvq_status kvq_decode_attention_uncertified(kvq_cache* cache, int layer, const void* q,
                                            void* out, kvq_certificate* cert, void* stream);

/* kvq_last_error -- text of the calling thread's last error ("" if none).  The pointer
 * stays valid until the thread's next failing call. */
const char* kvq_last_error(void);

/* kvq_set_debug -- set KVQ_DEBUG_* flags on the cache (0 clears them). */
kvq_status kvq_set_debug(kvq_cache* cache, int flags);

/* kvq_cache_length -- tokens currently cached for `layer`. */
kvq_status kvq_cache_length(const kvq_cache* cache, int layer, int* n_tokens);

/* kvq_export_tier1 -- copy the tier-1 contents of `layer` into caller device buffers in
 * canonical layout (nb = full blocks of the layer); any pointer may be NULL to skip it:
 *   kc int8 [B, Hkv, nb, 64, D]        ks fp16 [B, Hkv, nb, D]
 *   vc uint8 [B, Hkv, nb, 64, D] (one code 0..15 per byte)
 *   vs fp16 [B, Hkv, nb, 64, D/32]     vo fp16 [B, Hkv, nb, 64, D/32]
 *   eta float [B, Hkv, nb]             vmin, vmax float [B, Hkv, D]
 * Stream-ordered.  Errors: KVQ_ERR_INVALID, KVQ_ERR_CUDA. */
kvq_status kvq_export_tier1(kvq_cache* cache, int layer, void* kc, void* ks, void* vc,
                            void* vs, void* vo, float* eta, float* vmin, float* vmax,
                            void* stream);

/* kvq_export_decode_state -- copy the selection state of the last decode call into caller
 * device buffers (any may be NULL).  nb = full blocks of that call's layer.
 *   sel    uint8 [B, Hq, nb]   1 if the block is in the head's top-K* set S_h
 *   kprom0 uint8 [B, Hkv, nb]  FP16-key blocks of the first pass (union of S_h)
 *   kprom1 uint8 [B, Hkv, nb]  FP16-key blocks after rung 1 (== kprom0 if not run)
 *   vprom1 uint8 [B, Hkv, nb]  FP16-value blocks after rung 2
 *   lse8   float [B, Hq, nb]   INT8 block log-mass;  delta float [B, Hq, nb]  Delta_b
 * Stream-ordered.  Errors: KVQ_ERR_INVALID (no decode yet), KVQ_ERR_CUDA. */
kvq_status kvq_export_decode_state(kvq_cache* cache, uint8_t* sel, uint8_t* kprom0,
                                   uint8_t* kprom1, uint8_t* vprom1, float* lse8,
                                   float* delta, void* stream);

/* Per-kernel timing collected while KVQ_DEBUG_PROFILE is set. */
typedef struct kvq_kernel_stat {
  char name[32];
  int64_t launches;
  double total_ms;
} kvq_kernel_stat;

/* kvq_profile_read -- synchronise the cache's streams and return up to `max` kernel
 * statistics accumulated since the last reset (n = entries written).  reset != 0 clears
 * them afterwards.  Errors: KVQ_ERR_INVALID, KVQ_ERR_CUDA. */
kvq_status kvq_profile_read(kvq_cache* cache, kvq_kernel_stat* stats, int max, int* n,
                            int reset);

/* kvq_residency_stats -- FP16 block traffic of `layer`'s certified decode calls since the
 * last reset (cross-step residency, see kvq_config.resident_blocks): bytes of tier-2
 * blocks served from resident copies in device memory, bytes read over the host link,
 * and the slots currently holding a block.  Any output pointer may be NULL; reset != 0
 * clears the two byte counters.  Synchronises the device.
 * Errors: KVQ_ERR_INVALID (NULL cache, layer out of range), KVQ_ERR_CUDA. */
kvq_status kvq_residency_stats(kvq_cache* cache, int layer, int64_t* resident_bytes,
                               int64_t* host_bytes, int32_t* slots_in_use, int reset);

/* kvq_debug_fill_tier2 -- a test aid, not part of the paper: waits for the device, then
 * overwrites every FP16 element of `layer`'s tier 2 (the keys, and the values when they
 * live there) with the binary16 bit pattern `bits`.  Calls that page blocks in from
 * tier 2 afterwards see the pattern, so a test can show which passes never read it.
 * Errors: KVQ_ERR_INVALID (NULL cache, layer out of range), KVQ_ERR_CUDA. */
kvq_status kvq_debug_fill_tier2(kvq_cache* cache, int layer, uint16_t bits);

/* kvq_dense_attention_workspace -- device workspace bytes that kvq_dense_attention needs
 * for this shape on the current device (it depends on the device's SM count).
 * Errors: KVQ_ERR_INVALID (NULL bytes, bad shape), KVQ_ERR_CUDA. */
kvq_status kvq_dense_attention_workspace(int batch, int n_q_heads, int n_kv_heads, int n_tokens,
                                         size_t* bytes);

/* kvq_dense_attention -- exact dense FP16 decode attention, softmax(q K^T / sqrt(D)) V,
 * over keys and values held in device memory.  This is the dense FP16 attention that
 * Method §1 names as the ground truth and that Results (performance overhead) sets the
 * certified step against; the library uses it as that baseline on the same GPU.
 *   q         [B, Hq, D] FP16, device;  k, v [B, Hkv, n_tokens, D] FP16, device
 *   out       [B, Hq, D] FP16, device (caller-owned)
 *   workspace device buffer of at least kvq_dense_attention_workspace(...) bytes,
 *             caller-owned; its contents need no initialisation and are overwritten
 *   Hq / Hkv in 1..4, n_tokens >= 1; q, k, v, out and workspace 16-byte aligned and on
 *   the current device.
 * Two kernels on `stream`: a split pass that streams every key and value once from HBM
 * and a fixed-order combine.  Every device-side wait of the split pass is bounded (2 s);
 * a wait that runs out, which does not happen in correct operation, makes the affected
 * heads' outputs NaN.  Calls that share a workspace must not overlap on the GPU.
 * Stream-ordered.  Errors: KVQ_ERR_INVALID (NULL, host, unaligned or other-device
 * pointers, bad shape, workspace too small), KVQ_ERR_CUDA. */
kvq_status kvq_dense_attention(const void* q, const void* k, const void* v, int batch, int n_q_heads,
                               int n_kv_heads, int n_tokens, void* out, void* workspace,
                               size_t workspace_bytes, void* stream);

/* kvq_dense_decode_noalloc -- exact dense FP16 decode attention that allocates no memory.
 * The paper has no counterpart to this call.  It is for callers that cannot allocate
 * device memory when they call: a process whose device memory is fully held by another
 * framework's pool, an embedding that owns only fixed buffers, or a step that must not
 * fail on allocation.  It computes softmax(q K^T / sqrt(D)) V -- the same dense attention
 * as the ladder's rungs 3-4 -- over caller-owned FP16 keys and values, keeping its
 * split-K partials and counters in one static 8 MiB device array instead of calling
 * cudaMalloc, cudaFree or any allocating routine.
 *   q   [B, Hq, D] FP16, device;  k, v [B, Hkv, n_tokens, D] FP16, device
 *   out [B, Hq, D] FP16, device (caller-owned);  Hq / Hkv in 1..4, n_tokens >= 1
 *   q, k, v and out 16-byte aligned
 * Size limit: B * Hkv * ceil(n_tokens / 1024) * 2112 bytes of partials (plus a few
 * counters) must fit in the 8 MiB array, e.g. B * Hkv = 8 with up to 507904 tokens.
 * The array exists once per device that loads the library and is held until the
 * process exits.  Every call, with the device current, looks up the array's device
 * address (no allocation); make the first call on a device before any stream capture.
 * With the CUDA driver's lazy loading that first call is also when the library's device
 * code, and with it the 8 MiB array, is loaded onto the device: make it while 8 MiB of
 * device memory are still free (before another pool takes the rest), or it fails with
 * KVQ_ERR_CUDA.  After a cudaDeviceReset the next call loads the array again.
 * Every call shares the array and clears the counters it needs itself; calls whose work
 * overlaps on the GPU (other streams, other host threads) race on it and must be
 * serialised.  The kernel runs on the current device, on `stream`.
 * Stream-ordered.  Errors: KVQ_ERR_INVALID (NULL, host, unaligned or other-device
 * pointers, bad shape), KVQ_ERR_CAPACITY (beyond the size limit), KVQ_ERR_CUDA. */
kvq_status kvq_dense_decode_noalloc(const void* q, const void* k, const void* v, int batch,
                                    int n_q_heads, int n_kv_heads, int n_tokens, void* out,
                                    void* stream);

/* ------------------------------------------------------------------------------------
 * Paged 4-bit cache and rotary positions (not part of the paper: operators of this
 * library for serving loops that keep a whole cache in device memory).
 *
 * A page holds 64 consecutive tokens of every KV head; a pool of pages is one caller-owned
 * device buffer [n_pages][Hkv][kvq_paged_page_bytes(D)], 16-byte aligned, whose initial
 * contents do not matter.  Keys and values are held in 4 bits per element with a binary16
 * scale s and offset o per (token, 32-channel group), x^ = o + s * code, code in 0..15:
 * o = fp16 of the group's minimum, s = fp16 rounded up of (max - o) / 15 and code =
 * rint((x - o) / s), ties to even, clamped, for the x - o that fp32 holds.  Values of odd
 * slots count down from the maximum instead (o = fp16 of the maximum, s the negative of
 * (o - min) / 15 rounded up), so that sums of codes over tokens change sign from one token to
 * the next and do not lose precision to a common offset.
 * Elements beyond the binary16 range are held as +-65504; a NaN makes its group's offset NaN,
 * so that the 32 channels read as NaN.  Slot p * 64 + i is token i of
 * page p.
 *
 * Element types of q, k, v and outputs: kvq_dtype.  Strided operands [tokens, heads, D]
 * are given by a base pointer (16-byte aligned) and the strides of tokens and heads in
 * elements (multiples of 8); the D elements of a row are contiguous.  Rows of an input may
 * overlap (a stride of 0 repeats one), those of an output are refused when they do.  Every
 * buffer is device memory of the current device.  All calls are stream-ordered, allocate nothing
 * and may be captured into a CUDA graph.
 * ---------------------------------------------------------------------------------- */
typedef enum kvq_dtype { KVQ_F16 = 0, KVQ_BF16 = 1 } kvq_dtype;

/* How rotary frequencies are scaled for contexts beyond the trained one (factor f,
 * trained context n).  w_i = base^(-2i / rotary_dim) is pair i's angle per position and
 * u_i = n w_i / (2 pi) its turns within the trained context. */
typedef enum kvq_rope_scaling {
  KVQ_ROPE_NONE = 0,
  KVQ_ROPE_LINEAR = 1, /* w_i / f */
  KVQ_ROPE_NTK = 2,    /* base * f^(rotary_dim / (rotary_dim - 2)) in place of base */
  KVQ_ROPE_PARTS = 3,  /* k w_i + (1 - k) w_i / f, k = (u_i - low) / (high - low) clamped to
                          [0, 1] */
  KVQ_ROPE_YARN = 4    /* the same blend with k falling from 1 to 0 over the pair index,
                          between floor(d(high)) and ceil(d(low)), d(u) = rotary_dim
                          ln(n / (2 pi u)) / (2 ln base) (clamped to 0 and rotary_dim - 1);
                          cos and sin times `magnitude` */
} kvq_rope_scaling;

typedef struct kvq_rope_config {
  int head_dim;      /* even, 2..256 */
  int rotary_dim;    /* even, 2..head_dim: elements 0..rotary_dim-1 of a head are rotated */
  int interleaved;   /* 0: pairs (i, i + rotary_dim / 2); 1: pairs (2i, 2i + 1) */
  int scaling;       /* kvq_rope_scaling */
  double base;       /* > 1 */
  double factor;     /* >= 1; used by every scaling but NONE */
  int original_ctx;  /* n >= 1; used by PARTS and YARN */
  double low, high;  /* 0 < low < high, turns; used by PARTS and YARN */
  double magnitude;  /* factor on cos and sin, finite in fp32; 0: 1, and 0.1 ln(f) + 1 with YARN */
} kvq_rope_config;

/* What the kernels take: plain data, initialised on the host by kvq_rope_plan_init and
 * copied by value into every launch (no device memory, nothing to destroy). */
typedef struct kvq_rope_plan {
  int32_t head_dim, rotary_dim, interleaved;
  float magnitude;
  uint64_t step[128];   /* angle per position of each pair, in 2^-64 turns */
} kvq_rope_plan;

/* kvq_rope_plan_init -- fill `plan` from `cfg` (host only; no CUDA call).
 * Errors: KVQ_ERR_INVALID (NULL, or a field outside the ranges above). */
kvq_status kvq_rope_plan_init(const kvq_rope_config* cfg, kvq_rope_plan* plan);

/* kvq_rope -- rotary positions: out[t, h] = x[t, h] with pair i turned by positions[t] w_i
 * (times the plan's magnitude); elements from rotary_dim on are copied.
 *   x, out     [n_tokens, n_heads, plan->head_dim] strided; out may be x with the same
 *              strides (in place), and must not overlap it otherwise
 *   positions  [n_tokens] int32, device; any value.  A negative position turns back: with
 *              -p the call is the transpose of the call with p (its gradient), and undoes
 *              it where the magnitude is 1.
 * head_dim must be a multiple of 8.  Angles are right to 2^-33 turn, for positions of any
 * size, beside what the position makes of the frequency's own error (2^-63 turn, and its
 * rounding to double).  Arithmetic in fp32, one rounding to the element type.  n_tokens or
 * n_heads = 0 is a no-op.
 * Errors: KVQ_ERR_INVALID, KVQ_ERR_CUDA. */
kvq_status kvq_rope(const kvq_rope_plan* plan, int dtype, const void* x, int64_t x_token_stride,
                    int64_t x_head_stride, const int32_t* positions, int n_tokens, int n_heads, void* out,
                    int64_t out_token_stride, int64_t out_head_stride, void* stream);

/* kvq_paged_page_bytes -- bytes of one page of one KV head (head_dim 64 or 128).
 * Errors: KVQ_ERR_INVALID. */
kvq_status kvq_paged_page_bytes(int head_dim, size_t* bytes);

/* kvq_paged_append -- write tokens into pages: keys are turned by their positions in fp32
 * (plan != NULL), keys and values quantised from fp32 and stored in their slots.
 *   plan       NULL: keys are stored as they are (positions and q are then NULL)
 *   k, v       [n_tokens, n_kv_heads, head_dim] strided
 *   slots      [n_tokens] int32, device: where each token goes.  Slots outside the pool
 *              (negative ones: padding) are skipped.  The slots of one call must be
 *              distinct: a slot given twice ends up holding a mixture of its tokens.
 *   positions  [n_tokens] int32, device
 *   pages      the pool; only the bytes of the given slots change
 *   q, q_out   optional (NULL): [n_tokens, n_q_heads, head_dim] strided, turned by the same
 *              positions in the same launch (as kvq_rope), for every token, skipped or not;
 *              q_out may be q with the same strides, and must not overlap q, k or v otherwise
 * head_dim 64 or 128, n_kv_heads 1..4096.  One kernel.  n_tokens = 0 is a no-op.
 * Errors: KVQ_ERR_INVALID, KVQ_ERR_CUDA. */
kvq_status kvq_paged_append(const kvq_rope_plan* plan, int dtype, const void* k, int64_t k_token_stride,
                            int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
                            const int32_t* slots, const int32_t* positions, int n_tokens, int n_kv_heads,
                            int head_dim, void* pages, int n_pages, const void* q, int64_t q_token_stride,
                            int64_t q_head_stride, int n_q_heads, void* q_out, int64_t q_out_token_stride,
                            int64_t q_out_head_stride, void* stream);

/* kvq_paged_gather -- read tokens back from pages: k, v [n_tokens, n_kv_heads, head_dim]
 * strided receive o + s * code of the slots (keys as turned by the append), computed in
 * fp32 and rounded to the element type; rows of slots outside the pool become 0.  k and v
 * must not overlap.
 * Errors: KVQ_ERR_INVALID, KVQ_ERR_CUDA. */
kvq_status kvq_paged_gather(const void* pages, int n_pages, const int32_t* slots, int n_tokens, int n_kv_heads,
                            int head_dim, int dtype, void* k, int64_t k_token_stride, int64_t k_head_stride, void* v,
                            int64_t v_token_stride, int64_t v_head_stride, void* stream);

/* kvq_paged_attention_workspace -- device workspace bytes that kvq_paged_attention needs
 * for this shape on the current device, whatever the lengths.
 * Errors: KVQ_ERR_INVALID (NULL bytes, bad shape), KVQ_ERR_CUDA. */
kvq_status kvq_paged_attention_workspace(int batch, int n_q_tokens, int n_q_heads, int n_kv_heads, int head_dim,
                                         size_t* bytes);

/* kvq_paged_attention -- decode attention over the paged 4-bit cache:
 * out = softmax(scale q k^T) v over the tokens each query sees.
 *   q           [batch * n_q_tokens, Hq, head_dim] strided: the last n_q_tokens tokens of
 *               each sequence (1 for plain decoding, more when drafted tokens are verified)
 *   page_table  [batch, max_pages] int32, device, row stride table_stride elements: page j
 *               of a sequence holds its tokens 64j..64j+63.  Entries past the sequence's
 *               length are never read; tokens of an entry outside the pool are not seen.
 *   seq_lens    [batch] int32, device: tokens of each sequence in the cache, the
 *               n_q_tokens new ones included; clamped to 0..64 max_pages.  0: a padding
 *               sequence.
 *   window      0: query i of a sequence of n tokens sees tokens 0..n - n_q_tokens + i;
 *               w > 0: only the last w of them
 *   scale       0: 1 / sqrt(head_dim); else any number whose product with log2(e) is finite
 *   out         [batch, n_q_tokens, Hq, head_dim], contiguous, of q's type; must not overlap q
 *   lse         optional (NULL): [batch, n_q_tokens, Hq] float, natural log of the sum of
 *               exp(scale q k), for merging with attention over other keys
 * A query that sees no token gets out = 0 and lse = -inf.  What pages hold behind a
 * sequence's length (NaN included) does not matter.  A key or value that is NaN reaches the
 * outputs of the queries that see its token, and no others: those of the value's 32 channels,
 * or all of the row.
 *   workspace   at least kvq_paged_attention_workspace(...) bytes, 16-byte aligned, its
 *               first 4096 bytes set to zero once, before the first call that uses it: every
 *               call leaves them zero (they count the arrivals of a row's pieces), whatever
 *               its shape.  Calls that share it must not overlap on the GPU.
 * One kernel.  Hq / Hkv an integer in 1..64, Hkv <= 4096, n_q_tokens 1..64, batch <= 2048,
 * head_dim 64 or 128, batch * max_pages < 2^30.  Scores and sums in fp32; weights below
 * 2^-35 of a row's largest count as 0 (2^-(35 - j) where value scales reach 2^j).  batch = 0
 * is a no-op.  Every device-side wait is bounded (2 s); one that runs out, which does not
 * happen in correct operation, makes the affected outputs NaN.  Host threads may call at once,
 * each with its own workspace.
 * Errors: KVQ_ERR_INVALID, KVQ_ERR_CUDA. */
kvq_status kvq_paged_attention(int dtype, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                               const void* pages, int n_pages, const int32_t* page_table, int64_t table_stride,
                               int max_pages, const int32_t* seq_lens, int batch, int n_q_tokens, int n_q_heads,
                               int n_kv_heads, int head_dim, int window, float scale, void* out, float* lse,
                               void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_H_ */
