// kvq_paged_prefill.cu -- attention of prompts and chunks over the paged 4-bit cache:
//   out = softmax(scale q k^T) v over the tokens that each query sees,
// for chunks of any length, packed one behind the other, on the 5th-generation tensor cores.
//
// The rows of a (sequence, KV head) are its chunk's tokens times the query heads of that KV head: the heads of a group share
// every key and value that was unpacked.  A unit is 256 of these rows, two tiles of 128; it goes over its tokens 128 (two
// pages) at a time.  One CTA per SM, whose warps have roles:
//   warps 0-3, 4-7   softmax of tile 0 and of tile 1, a row per thread: scores out of TMEM, weights back into it
//   warps 8-11       keys and values: a token per thread, 4-bit codes to binary16 in shared memory, ahead of their use
//   warp 12          issues the MMAs: S = Q K^T (operands in shared memory), O += P V (P in TMEM, over half of S's columns)
//   warp 13          the next unit's queries into shared memory, as soon as the last scores of this one are there
// The two tiles take turns: while one's scores are turned into weights, the tensor cores work on the other.
//
// Unpacking: x^ = o + s code.  Two nibbles at a time are masked into binary16 numbers 1024 + n (or 64 + n), less 1024
// (exact), then one binary16 multiply-add, so each key and value is the held number rounded once (2^-11).  Nibbles four
// channels apart come out of one word side by side; keys stay in that order, and so do the queries (a dot product does not mind); values
// come out with channels of two groups in turn, so their scales and offsets enter in pairs, and the output is put in
// order when it is written.  Weights are rounded once to binary16 (2^-11) before their product with the values.  The three
// roundings weigh the same: on fp16 rows outputs are 4.3e-4 of their norm off, 2.1e-4 of it their own rounding (bf16: 1.7e-3, all
// but their own).  The decode attention keeps all exact, at four times the work per score.  Here, keys and values in two
// binary16 parts each (high parts exact, weights still rounded) brought that to 2.7e-4 for twice the MMAs and a shared memory that
// then holds one step instead of two: 2048 fp16 rows over 32768 tokens 874 -> 1493 us, at head_dim 64 over 16384 262 -> 344.
// What 4 bits lose is a hundred times as much, so the rows are not made to wait for it.
//
// Queries are brought to binary16, in the order that the MMAs take, by a kernel of their own before (a unit's 256 rows
// would keep a CTA's warps for 10 us), so that one bulk copy per 64 channels moves a tile of them.
//
// The softmax reference of a row moves only when a weight would pass 2^15, and is then set so that the largest is
// 2^10: accumulators in TMEM are rarely rescaled, and small weights stay normal binary16 numbers.
//
// The units' steps (128 tokens) are numbered, sequence by sequence, and cut into equal contiguous ranges, one per CTA,
// whatever the lengths; a unit counts PP_LEAD more than its steps, for what starting and finishing it takes.
// A unit within one range is written out directly; the pieces of one that is cut go to the workspace, and a second kernel
// merges them in a fixed order, so that results do not depend on timing.
//
// Measured (32 query heads on 8 KV heads of 128, bf16; 1925 TFLOP/s measured for a product of 8192^3): 2048 tokens over 32768
// 905 us = 1176 TFLOP/s (0.61; 899 to 937 on different GPUs), a prompt of 8192 tokens 524 us = 1049 (0.54); 64 tokens over 4096
// 29 us, of which the rows' kernel takes 3, the merge 8.  A step of 256 rows and 128 tokens takes about 3700 cycles, 2048 of them the MMAs': each
// tile's chain is its softmax (2700 cycles beside the other tile's and the unpacking, whose instructions fill 0.61 of the
// issue slots) and its two products (1070).  Every role's loop is as short as it is because straight code was slower: the
// same softmax with its four loads of scores unrolled took 968 us where this takes 879, unpacking unrolled 944 against 894.
#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "kvq.h"
#include "kvq_launch.h"
#include "kvq_paged.cuh"
#include "kvq_tc.cuh"

namespace kvq {

namespace {

struct PpArgs {
  const void* q;
  const unsigned char* pages;
  const int32_t *starts, *table, *lens;
  void* out;
  float* lse;
  int4* cut;      // [CTAs] the unit that a CTA begins and leaves: sequence, tile, KV head, pieces (0: none)
  unsigned char* rows;   // [Hkv][HD / 64][T n_rep] rows of 64 elements in binary16, swizzled
  float* scales;  // [Hkv][T n_rep] of a row's scores in base 2
  float* part;    // [CTAs][2] pieces of a unit begun in an earlier CTA, and of one that leaves the CTA: [HD + 2][256] floats
  long long qt, qh, table_stride;
  int n_pages, max_pages, T, B, Hq, Hkv, n_rep, window;
  float scale_log2;
  bool bf16, causal;
};

constexpr int PP_ROWS = 256, PP_TOK = 128, PP_STAGES = 2, PP_MAX_BATCH = 2048;
constexpr int PP_WARPS = 14, PP_THREADS = 32 * PP_WARPS, PP_MMA_WARP = 12;
// (a prompt of 8192 tokens: 598 us with one, 527 with two, 538 with four; without any the first CTA has 80 short units)
constexpr int PP_LEAD = 2;
constexpr float PP_TOP = 15.f, PP_SET = 10.f;             // weights are 2^15 at most, 2^10 when their reference is set

// A chunk and one of its units.
struct PpUnit {
  int b, qt, first, m, len;   // sequence, unit, first row of q, new tokens, cached tokens
  int tiles;                  // units of the sequence (of one KV head)
  int r0, rn, j0, np;         // rows, and first step and steps
};

__device__ __forceinline__ int pp_hi(const PpArgs& a, const PpUnit& u, int i) { return a.causal ? max(0, u.len - u.m + 1 + i) : u.len; }
__device__ __forceinline__ int pp_lo(const PpArgs& a, int hi) { return a.window ? max(0, hi - a.window) : 0; }

__device__ __forceinline__ void pp_sequence(const PpArgs& a, int b, PpUnit& u) {
  u.b = b;
  u.first = min(max(a.starts[b], 0), a.T);
  u.m = max(min(max(a.starts[b + 1], 0), a.T) - u.first, 0);   // (both ends clamped: the difference of any two fits)
  u.len = min(max(a.lens[b], 0), a.max_pages * PG);
  u.tiles = (u.m * a.n_rep + PP_ROWS - 1) / PP_ROWS;
}
// (every unit has a step, also one whose rows see nothing: its outputs are written all the same)
__device__ __forceinline__ void pp_unit(const PpArgs& a, int qt, PpUnit& u) {
  u.qt = qt, u.r0 = qt * PP_ROWS, u.rn = min(PP_ROWS, u.m * a.n_rep - u.r0);
  const int hi = pp_hi(a, u, (u.r0 + u.rn - 1) / a.n_rep), lo = pp_lo(a, pp_hi(a, u, u.r0 / a.n_rep));
  u.j0 = lo / PP_TOK;
  u.np = max(1, (hi + PP_TOK - 1) / PP_TOK - u.j0);
}

__device__ __forceinline__ float pp_max3(float x, float y, float z) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
  return m;
}
// ---- 4 bits to binary16 ----
// Nibbles k and k + 4 of a word as a pair of binary16 numbers 0..15: 1024 + n from the lowest bits of the halves, 64 + n from
// the next four (whose steps are 1 there), less 1024 or 64
template <int K>
__device__ __forceinline__ __half2 pp_nibbles(uint32_t w) {
  const uint32_t x = K < 2 ? w : w >> 8;
  if (K % 2 == 0) return __hsub2(u32_as_h2((x & 0x000F000Fu) | 0x64006400u), u32_as_h2(0x64006400u));
  return __hsub2(u32_as_h2((x & 0x00F000F0u) | 0x54005400u), u32_as_h2(0x54005400u));
}
// o + s n of a word's four pairs; CLAMP: no larger than binary16's largest (the held number may be, by a step's rounding)
template <bool CLAMP>
__device__ __forceinline__ uint4 pp_unpack(uint32_t w, __half2 s, __half2 o) {
  __half2 h[4] = {__hfma2(pp_nibbles<0>(w), s, o), __hfma2(pp_nibbles<1>(w), s, o), __hfma2(pp_nibbles<2>(w), s, o),
                  __hfma2(pp_nibbles<3>(w), s, o)};
  if (CLAMP) {
    const __half2 top = u32_as_h2(0x7BFF7BFFu), low = u32_as_h2(0xFBFFFBFFu);
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = __hmin2_nan(__hmax2_nan(h[k], low), top);
  }
  return make_uint4(h2_as_u32(h[0]), h2_as_u32(h[1]), h2_as_u32(h[2]), h2_as_u32(h[3]));
}
// Whether |o| + 15 |s| rounds beyond binary16
__device__ __forceinline__ bool pp_large(__half2 s, __half2 o) {
  const uint32_t x = h2_as_u32(__hfma2(__habs2(s), u32_as_h2(0x4B804B80u), __habs2(o))) & 0x7FFF7FFFu;
  return (x & 0xffffu) >= 0x7C00u || (x >> 16) >= 0x7C00u;
}
template <int HD>
struct PpSmem {
  static constexpr int Q = PP_ROWS * HD * 2, KV = PP_TOK * HD * 2;
  static constexpr int K0 = Q, V0 = K0 + PP_STAGES * KV, PRE = V0 + PP_STAGES * KV;
  static constexpr int bytes(int batch) { return PRE + 8 * (batch + 1) + 1024; }   // (1024: to the swizzle's boundary)
};

// A (token, query head)'s row: the lanes of HD / 8 hold 16 bytes each.  8192 tokens of 32 heads of 128, 134 MB: 29 us (issue:
// the rows' places and powers of two; at a copy's rate 20).
constexpr int PP_ROW_THREADS = 256;
template <int HD>
__global__ void __launch_bounds__(PP_ROW_THREADS) prefill_rows_kernel(PpArgs a) {
  constexpr int CH = HD / 8, PER = PP_ROW_THREADS / CH, RUN = 4;   // 16-byte pieces of a row; rows at once, and on their way
  const int c = threadIdx.x % CH;
  const long long rows = (long long)a.T * a.n_rep, all = rows * a.Hkv;
  pdl_trigger();
  pdl_wait();
  for (long long first = blockIdx.x * (long long)PER * RUN; first < all; first += (long long)gridDim.x * PER * RUN) {
    const long long x0 = first + threadIdx.x / CH;
    uint4 v[RUN];
    int place[RUN];       // a row's number in its chunk, modulo 8 (that of its place in shared memory)
    long long to[RUN];    // its number among all KV heads' rows (-1: none)
    int head[RUN];
#pragma unroll
    for (int k = 0; k < RUN; ++k) {
      // in the order of memory: tokens, then query heads
      const long long x = x0 + k * PER;
      v[k] = make_uint4(0, 0, 0, 0), place[k] = head[k] = 0, to[k] = -1;
      if (x >= all) continue;
      const int tok = (int)quotient(x, a.Hq), h = (int)(x - (long long)tok * a.Hq);
      v[k] = *reinterpret_cast<const uint4*>(static_cast<const unsigned short*>(a.q) + tok * a.qt + h * a.qh + 8 * c);
      int b = 0, b1 = a.B;
      while (b1 - b > 1) {   // the last chunk that starts at tok or before
        const int m = (b + b1) / 2;
        if (a.starts[m] <= tok) b = m; else b1 = m;
      }
      const int g = head[k] = h / a.n_rep, r = h - g * a.n_rep;
      place[k] = ((tok - min(max(a.starts[b], 0), a.T)) * a.n_rep + r) & 7;
      to[k] = g * rows + (long long)tok * a.n_rep + r;
    }
#pragma unroll
    for (int k = 0; k < RUN; ++k) {
      // the largest bits of an element but its sign: from INF on an infinity or a NaN, with which all of the row's outputs are NaN if it sees a token
      const uint32_t INF = a.bf16 ? 0x7F80u : 0x7C00u;
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = __vmaxu2(mx, word_of(v[k], i) & 0x7FFF7FFFu);
#pragma unroll
      for (int o = 1; o < CH; o <<= 1) mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mx = max(mx & 0xffffu, mx >> 16);
      float sc = fabsf(a.scale_log2);
      uint32_t w[4];
      // channels 0, 4, 1, 5, ...: as the keys' nibbles come
      if (a.bf16) {
        // the row times 2^e with a largest element in [2^9, 2^10), which binary16 holds down to 2^-34 of it; both powers are
        // normal fp32 numbers
        const int e = max(-126, min(126, 136 - (int)(mx >> 7)));
        const float up = __uint_as_float((uint32_t)(127 + e) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
        // never 0 or infinite, so that -inf stays -inf and 0 stays 0
        sc = fminf(fmaxf(sc * down, 1.17549435e-38f), 3.402823466e38f);
        const float f = a.scale_log2 < 0.f ? -up : up;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t p = word_of(v[k], i / 2), q = word_of(v[k], 2 + i / 2);
          const float y = __uint_as_float(i & 1 ? p & 0xffff0000u : p << 16), z = __uint_as_float(i & 1 ? q & 0xffff0000u : q << 16);
          w[i] = h2_as_u32(__floats2half2_rn(y * f, z * f));
        }
      } else {
        const uint32_t sign = a.scale_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __byte_perm(word_of(v[k], i / 2), word_of(v[k], 2 + i / 2), i & 1 ? 0x7632 : 0x5410) ^ sign;
      }
      if (to[k] < 0) continue;
      if (c == 0) a.scales[to[k]] = mx < INF ? sc : __int_as_float(0x7fc00000);
      // (KV head g's rows lie in HD / 64 blocks of `rows`)
      const long long at = HD == 64 ? to[k] : to[k] + (head[k] + c / 8) * rows;
      *reinterpret_cast<uint4*>(a.rows + at * 128 + (((c & 7) ^ place[k]) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// CTAs among which the steps are cut, and the first step of one of them
__device__ __forceinline__ int pp_ctas(long long total) { return (int)min((long long)gridDim.x, max(1ll, total)); }
__device__ __forceinline__ long long pp_cta0(long long total, int c) {
  const int ctas = pp_ctas(total);
  return total * min(c, ctas) / ctas;
}

template <int HD>
__global__ void __launch_bounds__(PP_THREADS, 1) paged_prefill_kernel(PpArgs a) {
  using L = Page<HD>;
  using S = PpSmem<HD>;
  constexpr int G = L::G, CH = HD / 8;                        // 16-byte pieces of a row
  constexpr uint32_t SCORES = 0, OUT = 256, TMEM = 512;       // columns: scores (and weights) of tiles 0 and 1, then outputs
  extern __shared__ unsigned char raw_smem[];
  unsigned char* sm = raw_smem + (1024 - (tc_smem(raw_smem) & 1023)) % 1024;
  long long* pre = reinterpret_cast<long long*>(sm + S::PRE);   // [B + 1] steps before each sequence, of one KV head
  __shared__ __align__(8) unsigned long long bars[23];
  __shared__ uint32_t tmem_at;
  __shared__ int failed_at;
  __shared__ int4 start_at;   // sequence, unit, KV head, step of this CTA's first position
  __shared__ int nan_at;      // whether a value that is NaN came by
  volatile int *failed = &failed_at, *nan_came = &nan_at;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t bar0 = __shfl_sync(0xffffffffu, tc_smem(bars), 0);
  const uint32_t k_full = bar0, k_empty = bar0 + 16, v_full = bar0 + 32, v_empty = bar0 + 48;            // [stage]
  const uint32_t q_full = bar0 + 64, s_full = bar0 + 80, p_full = bar0 + 96, o_full = bar0 + 112;        // [tile]
  const uint32_t o_empty = bar0 + 128, q_empty = bar0 + 144, done = bar0 + 160, p_half = bar0 + 168;
  if (threadIdx.x == 0) {
    auto init = [&](uint32_t bar, int count) { asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory"); };
    for (int k = 0; k < 2; ++k) {
      init(k_full + 8 * k, 128), init(k_empty + 8 * k, 1), init(v_full + 8 * k, 128), init(v_empty + 8 * k, 1);
      init(q_full + 8 * k, 1), init(o_empty + 8 * k, 128), init(s_full + 8 * k, 1), init(p_full + 8 * k, 128), init(o_full + 8 * k, 1);
      init(q_empty + 8 * k, 1), init(p_half + 8 * k, 128);
    }
    init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    failed_at = nan_at = 0;
    pre[0] = 0;
  }
  if (warp == PP_MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(tc_smem(&tmem_at)), "r"(TMEM) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_trigger();
  pdl_wait();

  // ---- this CTA's range of steps ----
  for (int b = warp; b < a.B; b += PP_WARPS) {
    PpUnit u;
    pp_sequence(a, b, u);
    long long sum = 0;
    for (int t = lane; t < u.tiles; t += 32) pp_unit(a, t, u), sum += u.np + PP_LEAD;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) pre[b + 1] = sum;
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = tmem_at;
  long long n_pos;   // of this CTA
  if (warp == 0) {
    long long run = 0;
    for (int base = 1; base <= a.B; base += 32) {
      long long inc = base + lane <= a.B ? pre[base + lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (base + lane <= a.B) pre[base + lane] = run + inc;
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
    __syncwarp();
    const long long total = run * a.Hkv, x0 = pp_cta0(total, blockIdx.x);
    int b = 0, b1 = a.B;
    while (b1 - b > 1) {   // the last sequence that starts at x0 or before
      const int m = (b + b1) / 2;
      if (pre[m] * a.Hkv <= x0) b = m; else b1 = m;
    }
    PpUnit u;
    pp_sequence(a, b, u);
    long long in = x0 - pre[b] * a.Hkv;   // position within the sequence: units, then KV heads, then steps
    int t0 = 0;
    for (; t0 < u.tiles; t0 += 32) {
      if (t0 + lane < u.tiles) pp_unit(a, t0 + lane, u);
      long long inc = t0 + lane < u.tiles ? (long long)(u.np + PP_LEAD) * a.Hkv : 0;
      const long long mine = inc;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const uint32_t here = __ballot_sync(0xffffffffu, mine > 0 && in >= inc - mine && in < inc);
      if (here) {
        const int src = __ffs(here) - 1;
        if (lane == src) {
          const long long at = in - (inc - mine);
          start_at = make_int4(b, t0 + lane, (int)(at / (u.np + PP_LEAD)), (int)(at % (u.np + PP_LEAD)));
        }
        break;
      }
      in -= __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  __syncthreads();
  {
    const long long total = pre[a.B] * a.Hkv;
    n_pos = pp_cta0(total, blockIdx.x + 1) - pp_cta0(total, blockIdx.x);
  }

  // ---- the walk over this CTA's pieces of units, the same in every role ----
  int g = start_at.z, p0 = start_at.w;   // KV head, position within the unit: PP_LEAD, then its steps
  PpUnit u;
  int s0 = 0, steps = 0, taken = 0;      // first step and steps of the piece (0: no more), its positions
  auto settle = [&]() {
    for (steps = 0; n_pos > 0;) {
      taken = (int)min((long long)(u.np + PP_LEAD - p0), n_pos);
      s0 = max(0, p0 - PP_LEAD), steps = max(0, p0 + taken - PP_LEAD) - s0;
      if (steps) return;
      n_pos = 0;   // (a range that ends within a unit's lead)
    }
  };
  auto begin = [&]() {
    if (n_pos == 0) return;
    pp_sequence(a, start_at.x, u);
    pp_unit(a, start_at.y, u);
    settle();
  };
  auto next = [&]() {
    n_pos -= taken;
    p0 = 0;
    if (n_pos > 0 && ++g == a.Hkv) {
      g = 0;
      if (u.qt + 1 < u.tiles) {
        pp_unit(a, u.qt + 1, u);
      } else {
        int b = u.b + 1;
        while (b + 1 < a.B && pre[b + 1] == pre[b]) ++b;
        pp_sequence(a, b, u);
        pp_unit(a, 0, u);
      }
    }
    settle();
  };

  if (warp < 8) {
    // ---- softmax ----
    const int rt = warp >> 2, tid = threadIdx.x & 127;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);   // this warp's lanes
    const uint32_t sp = lanes + SCORES + 128 * rt, op = lanes + OUT + HD * rt;
    uint32_t s_par = 0, o_par = 0;
    bool cut = false;
    for (begin(); steps > 0; next()) {
      if (128 * rt < u.rn) {
        const int r = u.r0 + 128 * rt + tid;   // this thread's row
        const bool live = 128 * rt + tid < u.rn;
        const int i = live ? r / a.n_rep : 0, h = g * a.n_rep + (live ? r - i * a.n_rep : 0);
        const float held = live ? a.scales[(long long)g * a.T * a.n_rep + (long long)u.first * a.n_rep + r] : 0.f;
        // a row with a NaN or an infinity is NaN if it sees a token; by a finite scale what it does not see has weight 0 here too
        const bool bad = held != held;
        const float sc = bad ? 1.f : held;
        bool saw = false;
        const int hi = live ? pp_hi(a, u, i) : 0, lo = live ? pp_lo(a, hi) : 0;
        const int hi_all = pp_hi(a, u, (u.r0 + 128 * rt) / a.n_rep);                                       // what every row of the tile sees
        const int lo_all = pp_lo(a, pp_hi(a, u, (u.r0 + min(u.rn, 128 * rt + 128) - 1) / a.n_rep));
        const int32_t* table = a.table + u.b * a.table_stride;
        float ref = -3.402823466e38f, lim = -INFINITY, l = 0.f;   // reference and limit of the scores, sum of weights
        for (int j = 0; j < steps; ++j) {
          const int t0 = (u.j0 + s0 + j) * PP_TOK;
          // pages outside of the pool are not seen
          uint32_t there = 0;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int page = t0 + k * PG < u.len ? table[t0 / PG + k] : -1;
            there |= (page >= 0 && page < a.n_pages) << k;
          }
          const bool edge = there != 3u || t0 < lo_all || t0 + PP_TOK > hi_all;
          uint32_t mask[4] = {};   // the tokens that this row sees
          if (edge) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int x = max(0, min(32, lo - t0 - 32 * c)), y = max(0, min(32, hi - t0 - 32 * c));
              const uint32_t low = x >= 32 ? 0u : 0xffffffffu << x, high = y >= 32 ? 0xffffffffu : (1u << y) - 1u;
              mask[c] = ((there >> (c >> 1)) & 1u) ? low & high : 0u;
            }
          }
          saw |= !edge || (mask[0] | mask[1] | mask[2] | mask[3]) != 0u;
          tc_wait(s_full + 8 * rt, s_par, failed);
          s_par ^= 1;
          tc_after();
          // The scores 32 tokens at a time, twice (in registers they would be 128): for the row's maximum, then for the
          // weights, which take the place of scores that were read.
          auto hide = [&](uint32_t (&v)[32], uint32_t seen) {
            if (edge) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!((seen >> k) & 1u)) v[k] = 0xff800000u;
            }
          };
          float m = -INFINITY;
          auto most = [&](uint32_t (&v)[32], uint32_t seen) {
            hide(v, seen);
#pragma unroll
            for (int k = 0; k < 32; k += 2) m = pp_max3(m, __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
          };
          // (rolled up, here and where the codes are unpacked: with each of the roles' loops straight, warps spent half of
          // their time on instructions that were not there yet)
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tc_ld32(v, sp + 32 * c);
            tc_wait_ld(v), most(v, c & 2 ? (c & 1 ? mask[3] : mask[2]) : (c & 1 ? mask[1] : mask[0]));
          }
          if (__any_sync(0xffffffffu, m > lim)) {
            const float now = m > lim ? m * sc - PP_SET : ref, al = exp2_approx(ref - now);
            if (m > lim) lim = (now + PP_TOP) / sc;
            ref = now;
            l *= al;
            if (j > 0) {   // (the products with the weights before are complete: the scores came behind them)
#pragma unroll 1
              for (int c = 0; c < HD; c += 16) {
                uint32_t x[16];
                tc_ld16(x, op + c);
              tc_wait_ld(x);
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * al);
                tc_st16(op + c, x);
              }
            }
          }
          float2 sum = make_float2(0.f, 0.f);
          auto weigh = [&](uint32_t (&v)[32], int c, uint32_t seen) {
            hide(v, seen);
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 x = fma2(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), make_float2(sc, sc), make_float2(-ref, -ref));
              const float2 p = make_float2(exp2_approx(x.x), exp2_approx(x.y));
              sum = add2(sum, p);
              w[k] = h2_as_u32(__floats2half2_rn(p.x, p.y));
            }
            tc_st16(sp + 16 * c, w);
          };
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tc_ld32(v, sp + 32 * c);
            tc_wait_ld(v), weigh(v, c, c & 2 ? (c & 1 ? mask[3] : mask[2]) : (c & 1 ? mask[1] : mask[0]));
            if (c == 1) {   // the product with the first half of the values can begin
              tc_wait_st();
              tc_before();
              tc_arrive(p_half + 8 * rt);
            }
          }
          l += sum.x + sum.y;
          tc_wait_st();
          tc_before();
          tc_arrive(p_full + 8 * rt);
        }

        // ---- the piece's end: to the output, or to the workspace ----
        tc_wait(o_full + 8 * rt, o_par, failed);
        o_par ^= 1;
        tc_after();
        const bool whole = steps == u.np, lost = *failed != 0;
        if (lost || (bad && saw)) l = __int_as_float(0x7fc00000);
        float* part = a.part + ((size_t)blockIdx.x * 2 + (s0 == 0)) * (HD + 2) * PP_ROWS + 128 * rt + tid;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const size_t at = (size_t)(u.first + i) * a.Hq + h;
        // Values that are NaN were 0 in the product (weights of 0 would not hide them from rows that do not see them): the row's
        // outputs of a group in which it sees one become NaN here.  32 tokens at a time, a token per lane.
        if (__any_sync(0xffffffffu, *nan_came)) {
          uint32_t nans = 0;   // bit gr: in group gr
          const int end = min((u.j0 + s0 + steps) * PP_TOK, u.len);
#pragma unroll 1
          for (int t0 = (u.j0 + s0) * PP_TOK; t0 < end; t0 += 32) {
            const int page = table[t0 / PG];
            if (page < 0 || page >= a.n_pages) continue;
            const unsigned short* vo = reinterpret_cast<const unsigned short*>(a.pages + ((size_t)page * a.Hkv + g) * L::BYTES + L::VO) +
                                       vscale_at((t0 & (PG - 1)) + lane);
            const int x = max(0, min(32, lo - t0)), y = max(0, min(32, hi - t0));
            const uint32_t sees = (x >= 32 ? 0u : 0xffffffffu << x) & (y >= 32 ? 0xffffffffu : (1u << y) - 1u);
#pragma unroll 1
            for (int gr = 0; gr < G; ++gr)
              nans |= (uint32_t)((__ballot_sync(0xffffffffu, t0 + lane < end && __hisnan(__ushort_as_half(vo[gr * PG]))) & sees) != 0u) << gr;
          }
          if (__any_sync(0xffffffffu, nans)) {
#pragma unroll 1
            for (int c = 0; c < HD; c += 16) {
              uint32_t x[16];
              tc_ld16(x, op + c);
              tc_wait_ld(x);
#pragma unroll
              for (int k = 0; k < 16; ++k)   // (columns: as below)
                if ((nans >> (2 * ((c / 8 + k / 8) % (G / 2)) + (k & 1))) & 1u) x[k] = 0x7fc00000u;
              tc_st16(op + c, x);
            }
            tc_wait_st();
          }
        }
        if (whole) {
          if (live && a.lse) a.lse[at] = l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.69314718055994531f;
        } else {
          part[HD * PP_ROWS] = l == 0.f ? -INFINITY : ref, part[(HD + 1) * PP_ROWS] = l;
        }
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t v[32];
          tc_ld32(v, op + 32 * c);
          tc_wait_ld(v);
          if (whole) {
            // column 8w + 2k + (g & 1): channel 32g + 4a + k, w = a G / 2 + g / 2; 32 columns are 32 / G channels of each group
            constexpr int RUN = 32 / G;
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
              uint32_t y[RUN / 2];
#pragma unroll
              for (int k = 0; k < RUN; k += 2) {
                const int col = 8 * ((k / 4) * (G / 2) + gr / 2) + 2 * (k % 4) + (gr & 1);
                y[k / 2] = f2_to_pair(__uint_as_float(v[col]) * inv, __uint_as_float(v[col + 2]) * inv, a.bf16);
              }
              uint4* o = reinterpret_cast<uint4*>(static_cast<unsigned short*>(a.out) + at * HD + 32 * gr + RUN * c);
              if (live) {
#pragma unroll
                for (int k = 0; k < RUN / 8; ++k) o[k] = make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
              }
            }
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) part[(32 * c + k) * PP_ROWS] = __uint_as_float(v[k]);
          }
        }
        tc_before();
        tc_arrive(o_empty + 8 * rt);
      }
      if (steps < u.np && s0 == 0 && threadIdx.x == 0) {
        // pieces: this CTA's and those of the CTAs that its other steps lie in
        const long long total = pre[a.B] * a.Hkv, end = pp_cta0(total, blockIdx.x + 1) + (u.np - steps) - 1;
        const int last = (int)(((end + 1) * pp_ctas(total) - 1) / total);
        a.cut[blockIdx.x] = make_int4(u.b, u.qt, g, last - (int)blockIdx.x + 1);
        cut = true;
      }
    }
    if (threadIdx.x == 0 && !cut) a.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
  } else if (warp < 12) {
    // ---- keys and values: a token per thread ----
    const int t = threadIdx.x & 127, pt = t & 63;
    constexpr int W4 = HD / 32;   // 16-byte pieces of a token's codes
    struct Held {                 // a key and a value as they are held
      uint4 code[2][W4];
      uint32_t s[2][G / 2], o[2][G / 2];   // scales and offsets, of two groups each
    };
    // Three steps are on their way: the page number of the one after the next, the next one's codes, and this one's into
    // shared memory.
    int left = 0, page = -1, head = 0;
    auto look = [&]() {   // the page of this thread's token in the walk's step, and on; false: there is none
      if (steps == 0) return false;
      const int tok = (u.j0 + s0 + steps - left) * PP_TOK + t;
      page = tok < u.len ? a.table[u.b * a.table_stride + tok / PG] : -1;
      head = g;
      if (--left == 0) next(), left = steps;
      return true;
    };
    auto fetch = [&](Held& x) {
      const bool in = page >= 0 && page < a.n_pages;
      const unsigned char* pg = a.pages + ((size_t)(in ? page : 0) * a.Hkv + head) * L::BYTES;
#pragma unroll
      for (int k = 0; k < W4; ++k) {
        x.code[0][k] = x.code[1][k] = make_uint4(0, 0, 0, 0);
        if (!in) continue;
        x.code[0][k] = *reinterpret_cast<const uint4*>(pg + pt * L::ROW + 16 * k);
        x.code[1][k] = *reinterpret_cast<const uint4*>(pg + L::VC + vcode_at<HD>(pt, 16 * k));
      }
#pragma unroll
      for (int k = 0; k < G / 2; ++k) {
        x.s[0][k] = x.o[0][k] = x.s[1][k] = x.o[1][k] = 0;
        if (!in) continue;
        x.s[0][k] = *reinterpret_cast<const uint32_t*>(pg + L::KS + pt * 2 * G + 4 * k);
        x.o[0][k] = *reinterpret_cast<const uint32_t*>(pg + L::KO + pt * 2 * G + 4 * k);
        const unsigned short* vs = reinterpret_cast<const unsigned short*>(pg + L::VS) + 2 * k * PG + vscale_at(pt);
        x.s[1][k] = vs[0] | (uint32_t)vs[PG] << 16;
        x.o[1][k] = vs[L::SCALES / 2] | (uint32_t)vs[L::SCALES / 2 + PG] << 16;
      }
    };
    // one operand's row of what is in hand
    auto unpack = [&](auto kind, Held& x, unsigned char* to) {
      constexpr bool values = decltype(kind)::value;
      __half2 sh[G], oh[G];   // keys: of each group, twice; values: of two groups, twice the same
      bool large = false;
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const __half2 s = u32_as_h2(x.s[values][k / 2]), o = u32_as_h2(x.o[values][k / 2]);
        sh[k] = values ? s : k & 1 ? __high2half2(s) : __low2half2(s);
        oh[k] = values ? o : k & 1 ? __high2half2(o) : __low2half2(o);
        large |= pp_large(sh[k], oh[k]);
      }
      auto words = [&](auto clamp) {
        constexpr bool CLAMP = decltype(clamp)::value;
#pragma unroll 1
        for (int k = 0; k < W4; ++k) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // word w = 4k + i of the row.  Keys: word G a + g is channels 32g + 8a .. + 7, piece 4g + a of the row; values:
            // word G / 2 a + g / 2
            const int gr = values ? 2 * (i % (G / 2)) : i % G, c = values ? 4 * k + i : 4 * (i % G) + 4 / G * k + i / G;
            *reinterpret_cast<uint4*>(to + tc_place(PP_TOK, t, c)) = pp_unpack<CLAMP>(word_of(x.code[values][0], i), sh[gr], oh[gr]);
          }
#pragma unroll
          for (int i = 0; i + 1 < W4; ++i) x.code[values][i] = x.code[values][i + 1];
        }
      };
      if (__any_sync(0xffffffffu, large)) words(std::true_type{}); else words(std::false_type{});
      tc_proxy();
    };
    uint32_t stage = 0, par = 1;
    auto put = [&](Held& x) {
      // a value that is NaN: 0 in the product, and known to the rows before their piece is complete
      bool nan = false;
#pragma unroll
      for (int k = 0; k < G / 2; ++k) {
        const __half2 o = u32_as_h2(x.o[1][k]);
        const bool lo = __hisnan(__low2half(o)), hi = __hisnan(__high2half(o));
        nan |= lo | hi;
        if (lo) x.o[1][k] &= 0xffff0000u, x.s[1][k] &= 0xffff0000u;
        if (hi) x.o[1][k] &= 0x0000ffffu, x.s[1][k] &= 0x0000ffffu;
      }
      if (nan) *nan_came = 1;
      tc_wait(k_empty + 8 * stage, par, failed);
      unpack(std::false_type{}, x, sm + S::K0 + stage * S::KV);
      tc_arrive(k_full + 8 * stage);
      tc_wait(v_empty + 8 * stage, par, failed);
      unpack(std::true_type{}, x, sm + S::V0 + stage * S::KV);
      tc_arrive(v_full + 8 * stage);
      if (++stage == PP_STAGES) stage = 0, par ^= 1;
    };
    begin();
    left = steps;
    Held x, y;
    bool has = look(), more = false;
    if (has) fetch(y), more = look();
#pragma unroll 1
    while (has) {
      x = y;
      has = more;
      if (more) fetch(y), more = look();
      put(x);
    }
  } else if (warp > PP_MMA_WARP) {
    // ---- queries ----
    if (lane == 0) {
      const long long rows = (long long)a.T * a.n_rep;
      uint32_t par = 0, used = 0;   // bit rt: parity of the tile's copies, whether there was one
      for (begin(); steps > 0; next())
        for (int rt = 0; rt < (u.rn > 128 ? 2 : 1); ++rt) {
          // the last unit's scores are there, so that its queries are not needed any more
          tc_wait(q_empty + 8 * rt, ((par >> rt) & 1u) ^ 1u, failed);
          const uint32_t bytes = 128u * min(128, u.rn - 128 * rt);
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(q_full + 8 * rt), "r"(bytes * (HD / 64)) : "memory");
#pragma unroll
          for (int k = 0; k < HD / 64; ++k)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                         :: "r"(tc_smem(sm) + rt * (S::Q / 2) + k * 128 * 128),
                            "l"(a.rows + ((g * (HD / 64) + k) * rows + (long long)u.first * a.n_rep + u.r0 + 128 * rt) * 128), "r"(bytes), "r"(q_full + 8 * rt)
                         : "memory");
          par ^= 1u << rt, used |= 1u << rt;
        }
      // (nothing is on its way when the CTA ends, also behind a wait that ran out)
      for (int rt = 0; rt < 2; ++rt)
        if ((used >> rt) & 1u)
          for (const unsigned long long t = tc_ns(); !tc_try(q_full + 8 * rt, ((par >> rt) & 1u) ^ 1u) && tc_ns() - t < TC_WAIT_NS;) {}
    }
  } else {
    // ---- MMAs ----
    constexpr uint32_t IQK = tc_idesc(PP_TOK, false), IPV = tc_idesc(HD, true);
    auto uniform = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
    const uint32_t tm = uniform(tmem), base = uniform(tc_smem(sm));
    const uint32_t q_at = tc_desc(base, 16), k_at = tc_desc(base + S::K0, 16), v_at = tc_desc(base + S::V0, PP_TOK * 128);
    const bool leader = tc_elect();
    uint32_t kn = 0, vn = 0;                     // steps of keys and values begun
    uint32_t q_par = 0, p_par = 0, o_par = 3;    // bit rt: parities
    auto scores = [&](int rt, uint32_t stage, bool last) {
#pragma unroll
      for (int k = 0; k < HD / 16; ++k) {
        const uint32_t at = ((k / 4) * 128 * 128 + (k % 4) * 32) >> 4;
        tc_mma_ss<IQK>(tm + SCORES + 128 * rt, q_at + rt * (S::Q / 32) + at, k_at + stage * (S::KV / 16) + at, k > 0, leader);
      }
      tc_commit(s_full + 8 * rt, leader);
      if (last) tc_commit(q_empty + 8 * rt, leader);   // the piece's queries have served
    };
    auto tiles = [&]() { return uniform(steps == 0 ? 0 : u.rn > 128 ? 2 : 1); };
    auto first_scores = [&](int rt, bool only) {   // of a piece
      tc_wait(q_full + 8 * rt, (q_par >> rt) & 1u, failed);
      q_par ^= 1u << rt;
      if (rt == 0) tc_wait(k_full + 8 * (kn % PP_STAGES), (kn / PP_STAGES) & 1u, failed);
      tc_after();
      scores(rt, kn % PP_STAGES, only);
    };
    begin();
    uint32_t now = uniform(steps), nt = tiles();
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
      if (rt < nt) first_scores(rt, now == 1);
    if (nt) tc_commit(k_empty, leader), ++kn;
    while (nt) {
      uint32_t then = 0, more = nt;
      for (uint32_t j = 0; j < now; ++j) {
        const uint32_t vs = vn % PP_STAGES, ks = kn % PP_STAGES;
        const bool last = j + 1 == now;
        if (last) {   // the next piece
          next();
          more = tiles();
          then = uniform(steps);
        }
        tc_wait(v_full + 8 * vs, (vn / PP_STAGES) & 1u, failed);
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
          if (rt < nt) {
            const uint32_t par = (p_par >> rt) & 1u;
            p_par ^= 1u << rt;
            if (j == 0) tc_wait(o_empty + 8 * rt, (o_par >> rt) & 1u, failed), o_par ^= 1u << rt;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              tc_wait((half ? p_full : p_half) + 8 * rt, par, failed);
              tc_after();
#pragma unroll
              for (int k = 4 * half; k < 4 * half + 4; ++k)
                tc_mma_ts<IPV>(tm + OUT + HD * rt, tm + SCORES + 128 * rt + 8 * k, v_at + vs * (S::KV / 16) + k * (2048 / 16), j > 0 || k > 0, leader);
            }
            if (last) tc_commit(o_full + 8 * rt, leader);
          }
          if (rt < more) {
            if (last) {
              first_scores(rt, then == 1);
            } else {
              if (rt == 0) tc_wait(k_full + 8 * ks, (kn / PP_STAGES) & 1u, failed), tc_after();
              scores(rt, ks, j + 2 == now);
            }
          }
        }
        tc_commit(v_empty + 8 * vs, leader);
        ++vn;
        if (more) tc_commit(k_empty + 8 * ks, leader), ++kn;
      }
      now = then, nt = more;
    }
    // nothing of this CTA's is in flight any more when it gives its TMEM back, also behind a wait that ran out
    tc_commit(done, leader);
    for (const unsigned long long t = tc_ns(); !tc_try(done, 0) && tc_ns() - t < TC_WAIT_NS;) {}
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == PP_MMA_WARP)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(TMEM) : "memory");
}

// The pieces of the unit that CTA blockIdx.x begins and leaves, merged in their order: 32 rows and 32 channels per block, a
// row per lane and eight output channels per warp.  Bound by the latency of its loads: pieces are read four at a time (64
// tokens over 4096, 19 pieces to a unit: the call took 40 us with 128 channels per block, one piece after the other, 30 so).
constexpr int PP_MERGE_THREADS = 128;
template <int HD>
__global__ void __launch_bounds__(PP_MERGE_THREADS) prefill_merge_kernel(PpArgs a) {
  constexpr int G = HD / 32, PART = (HD + 2) * PP_ROWS, RUN = 4;
  pdl_trigger();
  pdl_wait();
  const int4 cut = a.cut[blockIdx.x];
  const int n = cut.w;
  if (n == 0) return;
  PpUnit u;
  pp_sequence(a, cut.x, u);
  pp_unit(a, cut.y, u);
  const int lane = threadIdx.x & 31, x = threadIdx.x >> 5, gr = blockIdx.z, row = blockIdx.y * 32 + lane;
  if ((int)blockIdx.y * 32 >= u.rn) return;
  const float* part = a.part + (size_t)blockIdx.x * 2 * PART + row;
  // piece 0 is the CTA's second one, the others their CTAs' first
  auto at = [&](int k) { return part + (size_t)(k == 0 ? 1 : 2 * k) * PART; };
  float top = -INFINITY;
#pragma unroll 8
  for (int k = 0; k < n; ++k) top = fmaxf(top, at(k)[HD * PP_ROWS]);
  const float ref = top == -INFINITY ? 0.f : top;
  float l = 0.f, y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] = 0.f;
  const int col0 = 8 * (2 * x * (G / 2) + gr / 2) + (gr & 1);   // of channel 32 gr + 8 x
  for (int p0 = 0; p0 < n; p0 += RUN) {
    float v[RUN][8], w[RUN], sum[RUN];
#pragma unroll
    for (int p = 0; p < RUN; ++p) {
      const float* from = at(min(p0 + p, n - 1));
      w[p] = from[HD * PP_ROWS], sum[p] = from[(HD + 1) * PP_ROWS];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[p][k] = from[(col0 + 4 * G * (k / 4) + 2 * (k % 4)) * PP_ROWS];
    }
#pragma unroll
    for (int p = 0; p < RUN; ++p) {
      if (p0 + p >= n) break;
      const float f = exp2_approx(w[p] - ref);
      l = fmaf(sum[p], f, l);
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = fmaf(v[p][k], f, y[k]);
    }
  }
  if (row >= u.rn) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int r = u.r0 + row, i = r / a.n_rep, h = cut.z * a.n_rep + (r - i * a.n_rep);
  const size_t to = (size_t)(u.first + i) * a.Hq + h;
  if (x == 0 && gr == 0 && a.lse) a.lse[to] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
  uint32_t v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = f2_to_pair(y[2 * k] * inv, y[2 * k + 1] * inv, a.bf16);
  *reinterpret_cast<uint4*>(static_cast<unsigned short*>(a.out) + to * HD + 32 * gr + 8 * x) = make_uint4(v[0], v[1], v[2], v[3]);
}

const char* pp_shape_error(int T, int B, int Hq, int Hkv, int hd) {
  if (T < 0 || T > (1 << 24)) return "n_tokens must be in 0..16777216";
  if (B < 0 || B > PP_MAX_BATCH) return "batch must be in 0..2048";
  if (Hkv < 1 || Hkv > MAX_KV_HEADS) return "n_kv_heads must be in 1..4096";
  if (Hq < 1 || Hq % Hkv != 0 || Hq / Hkv > 64) return "n_q_heads / n_kv_heads must be an integer in 1..64";
  if (hd != 64 && hd != 128) return "head_dim must be 64 or 128";
  return nullptr;
}

size_t pp_cut_bytes(int sms) { return ((size_t)sms * sizeof(int4) + 255) / 256 * 256; }
size_t pp_part_bytes(int sms, int hd) { return (size_t)sms * 2 * (hd + 2) * PP_ROWS * sizeof(float); }   // (a multiple of 1024)
size_t pp_rows_bytes(int T, int Hq, int hd) { return (size_t)T * Hq * hd * 2; }
size_t pp_bytes(int sms, int T, int Hq, int hd) {
  return pp_cut_bytes(sms) + pp_part_bytes(sms, hd) + pp_rows_bytes(T, Hq, hd) + (size_t)T * Hq * sizeof(float);
}

template <int HD>
cudaError_t pp_launch(const PpArgs& a, int sms, cudaStream_t st) {
  auto* k = paged_prefill_kernel<HD>;
  // the limit belongs to the function and is every host thread's: always the one of the largest batch
  if (cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, PpSmem<HD>::bytes(PP_MAX_BATCH))) return e;
  const long long all = ((long long)a.T * a.Hq + PP_ROW_THREADS * 8 / HD * 4 - 1) / (PP_ROW_THREADS * 8 / HD * 4);
  if (cudaError_t e = launch_dependent(prefill_rows_kernel<HD>, dim3((unsigned)std::min<long long>(all, sms * 32)), dim3(PP_ROW_THREADS), 0, st, a))
    return e;
  if (cudaError_t e = launch_dependent(k, dim3(sms), dim3(PP_THREADS), PpSmem<HD>::bytes(a.B), st, a)) return e;
  return launch_dependent(prefill_merge_kernel<HD>, dim3(sms, PP_ROWS / 32, HD / 32), dim3(PP_MERGE_THREADS), 0, st, a);
}

kvq_status prefill_impl(int dtype, const void* q, int64_t qt, int64_t qh, const int32_t* starts, int T, const void* pages, int n_pages,
                        const int32_t* table, int64_t table_stride, int max_pages, const int32_t* lens, int B, int Hq, int Hkv,
                        int hd, int causal, int window, float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                        void* stream) {
  const char* fn = "kvq_paged_prefill";
  auto bad = [&](const char* what) { return paged_fail(KVQ_ERR_INVALID, fn, what); };
  if (dtype != KVQ_F16 && dtype != KVQ_BF16) return bad("dtype must be KVQ_F16 or KVQ_BF16");
  if (const char* msg = pp_shape_error(T, B, Hq, Hkv, hd)) return bad(msg);
  if (n_pages < 1 || n_pages > (1 << 25)) return bad("n_pages must be in 1..33554432");
  if (max_pages < 1 || max_pages > (1 << 24) || (long long)B * max_pages >= (1ll << 30))
    return bad("max_pages must be in 1..16777216 and batch * max_pages below 2^30");
  if (table_stride < 0) return bad("table_stride must be >= 0");
  if (causal != 0 && causal != 1) return bad("causal must be 0 or 1");
  if (window < 0 || (window && !causal)) return bad("window must be >= 0, and 0 unless causal");
  const float scale_log2 = (scale != 0.f ? scale : 1.f / std::sqrt((float)hd)) * LOG2E_F;
  if (!std::isfinite(scale_log2)) return bad("scale * log2(e) must be finite");
  // the steps of all units, times the CTAs, are counted in 64 bits, also where starts that do not ascend make every chunk the whole
  // of q (what fits a GPU's memory stays below 2^62 all the same)
  const double most = ((double)T * (Hq / Hkv) / PP_ROWS + 1) * B * (max_pages / 2 + 1 + PP_LEAD) * Hkv * 1024;
  if (most >= 9e18) return bad("n_tokens * max_pages * n_q_heads is too large for one call");
  if (B == 0 || T == 0) return KVQ_OK;
  if (q == out) return bad("out must not be q");
  if (kvq_status s = check_strides(qt, qh, fn, "q")) return s;
  int dev = 0, sms = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return paged_cuda_fail(e, fn, "no current CUDA device");
  if (cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) return paged_cuda_fail(e, fn, "device attributes");
  if (kvq_status s = check_buffer(q, dev, 16, fn, "q")) return s;
  if (kvq_status s = check_buffer(starts, dev, 4, fn, "q_starts")) return s;
  if (kvq_status s = check_buffer(pages, dev, 16, fn, "pages")) return s;
  if (kvq_status s = check_buffer(table, dev, 4, fn, "page_table")) return s;
  if (kvq_status s = check_buffer(lens, dev, 4, fn, "seq_lens")) return s;
  if (kvq_status s = check_buffer(out, dev, 16, fn, "out")) return s;
  if (lse)
    if (kvq_status s = check_buffer(lse, dev, 4, fn, "lse")) return s;
  if (kvq_status s = check_buffer(workspace, dev, 16, fn, "workspace")) return s;
  if (workspace_bytes < pp_bytes(sms, T, Hq, hd)) return bad("workspace smaller than kvq_paged_prefill_workspace reports");
  PpArgs a = {};
  a.q = q, a.pages = static_cast<const unsigned char*>(pages), a.starts = starts, a.table = table, a.lens = lens, a.out = out;
  a.lse = lse, a.qt = qt, a.qh = qh, a.table_stride = table_stride, a.n_pages = n_pages, a.max_pages = max_pages, a.T = T, a.B = B;
  a.Hq = Hq, a.Hkv = Hkv, a.n_rep = Hq / Hkv, a.window = std::min(window, 1 << 30), a.scale_log2 = scale_log2;
  a.bf16 = dtype == KVQ_BF16, a.causal = causal != 0;
  a.cut = static_cast<int4*>(workspace);
  unsigned char* ws = static_cast<unsigned char*>(workspace) + pp_cut_bytes(sms);
  a.part = reinterpret_cast<float*>(ws);
  a.rows = ws + pp_part_bytes(sms, hd);
  a.scales = reinterpret_cast<float*>(a.rows + pp_rows_bytes(T, Hq, hd));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = hd == 128 ? pp_launch<128>(a, sms, st) : pp_launch<64>(a, sms, st);
  if (e != cudaSuccess) return paged_cuda_fail(e, fn, "launch");
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

extern "C" kvq_status kvq_paged_prefill_workspace(int n_tokens, int batch, int n_q_heads, int n_kv_heads, int head_dim,
                                                  size_t* bytes) try {
  const char* fn = "kvq_paged_prefill_workspace";
  if (!bytes) return kvq::paged_fail(KVQ_ERR_INVALID, fn, "NULL output");
  if (const char* msg = kvq::pp_shape_error(n_tokens, batch, n_q_heads, n_kv_heads, head_dim))
    return kvq::paged_fail(KVQ_ERR_INVALID, fn, msg);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return kvq::paged_cuda_fail(e, fn, "no current CUDA device");
  }
  *bytes = kvq::pp_bytes(sms, n_tokens, n_q_heads, head_dim);
  return KVQ_OK;
} catch (...) {
  return KVQ_ERR_HOST_OOM;
}

extern "C" kvq_status kvq_paged_prefill(int dtype, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                        const int32_t* q_starts, int n_tokens, const void* pages, int n_pages,
                                        const int32_t* page_table, int64_t table_stride, int max_pages, const int32_t* seq_lens,
                                        int batch, int n_q_heads, int n_kv_heads, int head_dim, int causal, int window, float scale,
                                        void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) try {
  return kvq::prefill_impl(dtype, q, q_token_stride, q_head_stride, q_starts, n_tokens, pages, n_pages, page_table, table_stride,
                           max_pages, seq_lens, batch, n_q_heads, n_kv_heads, head_dim, causal, window, scale, out, lse, workspace,
                           workspace_bytes, stream);
} catch (...) {
  return KVQ_ERR_HOST_OOM;
}
