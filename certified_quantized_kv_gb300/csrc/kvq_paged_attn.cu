// kvq_paged_attn.cu -- decode attention over the paged 4-bit cache.
//
// With k^ = o + s code per group g of 32 channels (and v^ likewise),
//   score_t = scale (sum_g s_tg (q_g . code_tg) + sum_g o_tg sum(q_g))
//   out_c   = (sum_t (p_t s_tg) code_tc + sum_t p_t o_tg) / sum_t p_t,   p_t = exp(score_t - m)
// over the tokens that a query sees.  A token of one KV head is 160 bytes at head_dim 128 and
// is read once, so HBM is the floor; the work per byte is what the design is about.
//
//  - Nibbles are never converted: masked out of their words they are binary16 subnormals
//    n 2^-24 (low nibble of a byte) or 16 n 2^-24 (high nibble), exact MMA operands.
//    Scales and offsets enter outside the code products: the key scales multiply the group's
//    fp32 sums, the value scales the softmax weights, the offsets are MMAs of their own (8 of
//    the 72 per page at head_dim 128 and four rows).  Channels in high nibbles carry 1/16 in q.
//  - Scores: tokens are MMA rows, up to 8 query rows are columns: one m16n8k16 covers 16
//    tokens x 16 channels.  A score fragment turned by movmatrix is the B fragment (k = tokens)
//    of the value product, whose rows are channels.  With tiles of 16 rows the queries are MMA
//    rows instead, and nothing is turned.
//  - Weights go into the value product as binary16 halves hi + lo of p s (together 2^-21),
//    formed by exact products.  With at most four query rows they fill one tile's eight
//    columns (four hi, four lo); with more, hi and lo are two MMAs into the same sums.  One half
//    alone (2^-12) would cost 2.5 times the output's own rounding error: codes 0..15 are not
//    centred, so the errors of all weights add up in them.
//  - The softmax reference of a row moves only when a weight would pass 2^top, and is then set so
//    that the largest is 2^(top - 4): most pages rescale nothing.  top is 14 unless a value
//    scale of 2 or more appears (then smaller, so that p s stays finite in binary16): small
//    weights of long caches stay normal numbers.  Weights below 2^-25 count as 0: 2^-35 of the row's
//    largest one or less, 2^-(35 - j) where value scales reach 2^j (values that span 15 2^j).
//  - The (sequence, KV head, row tile, page) units are numbered in that order and cut into
//    equal contiguous ranges, one per warp, whatever the lengths; every warp works alone on
//    whole pages, fed by bulk copies into its own shared-memory ring.  A group (sequence, KV
//    head, row tile) that lies within one warp's range is written out directly.  The pieces
//    of one that is cut are merged within the CTA, and across CTAs by the last of them to
//    arrive, each time in a fixed order, so the result does not depend on timing.
//
// Measured (GB300, 32 query heads on 8 KV heads of 128, device time): 8 sequences of 65536 tokens,
// 671 MB: 109 us = 6.2 TB/s, 0.91 of a copy's 6.8; one of 131072: 35.4 us = 4.7 TB/s; one of 4096: 10.6 us.
// What long calls take beside their bytes is about 10 us; a short one: launch 1.2 us, lengths 0.6, ranges 0.5,
// page numbers and first pages (with the queries meanwhile) 1.5, one page's arithmetic 1.5, writing its piece
// 0.6, merging within the CTA 0.9, arrival 1.1, merging across CTAs 1.9, and 0.5 between the first and last warp.
#include <algorithm>
#include <cmath>
#include <string>

#include "kvq.h"
#include "kvq_launch.h"
#include "kvq_paged.cuh"
#include "kvq_paged_merge.cuh"

namespace kvq {

namespace {

constexpr int PA_STAGES = 2;   // pages on their way per warp (PA_WARPS)
// Positions that a group takes besides its pages, for what starting and finishing it costs in pages' time:
// two at head_dim 128 (64 ragged sequences up to 16384 tokens: 82 us; 89 with one, 101 with none, 82 with
// three; 8 with four query tokens: 32 us; 34, 41, 31), three at 64, whose pages take less (48 ragged with a
// window of 4096: 19.4 us; 20.0 with two, 27.3 with none).
constexpr int PA_MAX_LEAD = 3;
template <int HD>
constexpr int PA_LEAD = HD == 64 ? PA_MAX_LEAD : 2;
constexpr float PA_TOP = 14.f;                              // weights are 2^14 at most,
constexpr float PA_SLACK = 4.f;                             // 2^10 when their reference is set
constexpr unsigned long long PA_WAIT_NS = 2000000000ull;    // bounded waits: 2 s
constexpr int PA_MAX_BATCH = 2048;                          // positions and lengths lie in shared memory

struct PaArgs {
  const void* q;
  const unsigned char* pages;
  const int32_t *table, *lens;
  void* out;
  float* lse;
  int* arrived;  // [CTAs] arrivals at the group that starts in a CTA and leaves it; 0 between calls
  float* part;   // pieces of R (HD + 2) floats: [warps] the end of a group begun in an earlier
                 // warp, then [CTAs][2] (0: of a group begun in an earlier CTA, 1: of one that
                 // leaves the CTA)
  long long qt, qh, table_stride;
  int n_pages, max_pages, B, Q, Hq, Hkv, n_rep, rows, RT, window, grid;
  float scale_log2;   // scale * log2(e)
  bool bf16;
};

// Tokens, first page and page count of a sequence.
__device__ __forceinline__ int pa_len(const PaArgs& a, int b) { return min(max(a.lens[b], 0), a.max_pages * PG); }
__device__ __forceinline__ int pa_first(const PaArgs& a, int len) {
  return a.window ? max(0, len - a.Q + 1 - a.window) / PG : 0;
}

// Equal contiguous ranges of T unit positions for `ge` CTAs, none empty.  A group takes PA_LEAD
// positions besides one per page when the ranges are long enough.
struct PaSplit {
  long long T;
  int ge;
  __device__ __forceinline__ long long cta0(int c) const { return quotient(c * T, ge); }
  __device__ __forceinline__ int cta_of(long long x) const { return (int)quotient((x + 1) * ge - 1, T); }
};

__device__ __forceinline__ unsigned long long pa_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ bool pa_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __noinline__ bool pa_wait_slow(uint32_t bar, uint32_t parity) {
  const unsigned long long t0 = pa_ns();
  while (!pa_try(bar, parity))
    if (pa_ns() - t0 > PA_WAIT_NS) return false;
  return true;
}
__device__ __forceinline__ bool pa_wait(uint32_t bar, uint32_t parity) {
  return pa_try(bar, parity) || pa_wait_slow(bar, parity);
}

// Behind a wait that ran out, when nothing more is issued: for the copies still in flight (not inlined, to stay
// out of the page loop: 8 sequences of 65536 tokens take 0.9 us more with it inside)
__device__ __noinline__ void pa_drain(uint32_t bar0, int issued) {
  ring_drain<PA_STAGES>(issued, [&](int k, uint32_t parity) { pa_wait_slow(bar0 + 8 * k, parity); });
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// ... with a zero C
__device__ __forceinline__ void mma_z(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// ... of half the depth, with a zero C
__device__ __forceinline__ void mma_k8_z(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// N 32-bit words of shared memory in one load
template <int N>
__device__ __forceinline__ void lds(uint32_t (&w)[N], const unsigned char* p) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

template <int HD>
struct PaStage {
  static constexpr int FLOATS = 8 * (HD + 4) + 8 * (HD / 32) + 16;   // a multiple of 4
};

// R query rows per tile: 4 (hi and lo weights share the eight columns: 35.4 us for 131072 tokens, 39.1
// in a tile of 8), 8 (a row each), or 16, where
// queries are MMA rows instead of columns (WIDE): a score fragment then is an A fragment of
// the value product as it stands, and hi and lo weights multiply the same code fragments.
template <int HD, int R>
__global__ void __launch_bounds__(PA_THREADS, 1) paged_attention_kernel(PaArgs a) {
  using L = Page<HD>;
  constexpr bool PACK = R == 4, WIDE = R == 16;
  constexpr int G = L::G, MT = WIDE ? HD / 8 : HD / 16, PART = R * (HD + 2);   // MT: accumulator tiles
  // tiles of 16 tokens at once: a whole page, if registers allow (131072 tokens 35.4 us, 37.3 with two;
  // tiles of 16 rows: two 31.6 us, one 32.1)
  constexpr int STEP = WIDE ? 2 : 4;
  constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u, BYTE = 0x00FF00FFu;
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ __align__(8) unsigned long long bars[PA_WARPS][PA_STAGES];
  // groups of each warp that are cut (sequence, group; -1: none): the one it ends, and the
  // one it leaves open (started in this warp or before)
  __shared__ int2 ended[PA_WARPS], open_at[PA_WARPS];
  __shared__ bool open_new[PA_WARPS];
  __shared__ int wsum[PA_WARPS];
  __shared__ int final_n[2];
  __shared__ const float* piece_at[PA_WARPS][2];   // where a warp's ended and open pieces lie
  int* pre = reinterpret_cast<int*>(sm + PA_WARPS * (PA_STAGES * L::BYTES + PaStage<HD>::FLOATS * 4));   // [B + 1] positions before each sequence
  int* slen = pre + a.B + 1;                                                 // [B]

  // broadcast, so that the compiler knows it (and all that follows from it) as warp-uniform
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  unsigned char* ring = sm + warp * PA_STAGES * L::BYTES;
  // per warp: eight columns of a finished tile (rows padded to distinct banks), then their
  // offsets per group, weight sums and references
  constexpr int SROW = HD + 4;
  float* stage = reinterpret_cast<float*>(sm + PA_WARPS * PA_STAGES * L::BYTES) + warp * PaStage<HD>::FLOATS;
  float* stage_o = stage + 8 * SROW;   // [8][G]
  float* stage_l = stage_o + 8 * G;    // [8]
  float* stage_r = stage_l + 8;        // [8]
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
  const uint32_t bar_s = (uint32_t)__cvta_generic_to_shared(&bars[warp][0]);
  if (lane == 0) {
    for (int s = 0; s < PA_STAGES; ++s) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" :: "r"(bar_s + 8 * s) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    ended[warp].x = open_at[warp].x = -1;
  }

  pdl_trigger();
  pdl_wait();   // the launch and what lies above overlap the end of the previous kernel

  // Pages of every sequence and their sum, then the positions before each sequence.  A group takes
  // lead positions from one page per warp on (8 sequences of 1..4096 tokens, 1.6 pages per warp:
  // 14.6 us, 16.3 without; 48 of 512, less than a page per warp, took 12.4 us, 11.5 without).
  const int U = a.Hkv * a.RT;
  auto pages_of = [&](int len) { return len > 0 ? (len + PG - 1) / PG - pa_first(a, len) : 0; };
  auto lead_of = [&](int pages) { return (long long)pages * U >= (long long)a.grid * PA_WARPS ? PA_LEAD<HD> : 0; };
  auto sum_before = [&](int& inc) {   // inclusive sums over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
  };
  int lead;
  // (up to 32 sequences every warp by itself, all writing the same: one of 4096 tokens took 11.3 us, 11.7
  // through the other way's barriers)
  if (a.B <= 32) {
    const int len = lane < a.B ? pa_len(a, lane) : 0, np = pages_of(len);
    lead = lead_of(__reduce_add_sync(0xffffffffu, np));
    int inc = np ? np + lead : 0;
    sum_before(inc);
    if (lane < a.B) slen[lane] = len, pre[lane + 1] = inc;
    if (lane == 0) pre[0] = 0;
    __syncwarp();
  } else {
    int pages = 0;
    for (int b = threadIdx.x; b < a.B; b += PA_THREADS) {
      const int len = pa_len(a, b);
      slen[b] = len;
      pages += pages_of(len);
    }
    pages = __reduce_add_sync(0xffffffffu, pages);
    if (lane == 0) wsum[warp] = pages;
    __syncthreads();
    pages = 0;
#pragma unroll
    for (int w = 0; w < PA_WARPS; ++w) pages += wsum[w];
    lead = lead_of(pages);
    if (threadIdx.x == 0) pre[0] = 0;
    for (int base = 0, run = 0; base < a.B; base += PA_THREADS) {
      const int b = base + threadIdx.x;
      const int np = b < a.B ? pages_of(slen[b]) : 0;
      int inc = np ? np + lead : 0;
      sum_before(inc);
      __syncthreads();
      if (lane == 31) wsum[warp] = inc;
      __syncthreads();
      int before = run;
#pragma unroll
      for (int w = 0; w < PA_WARPS; ++w) {
        before += w < warp ? wsum[w] : 0;
        run += wsum[w];
      }
      if (b < a.B) pre[b + 1] = before + inc;
    }
    __syncthreads();
  }
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {   // rows of empty sequences
    if (slen[b] > 0) continue;
    const size_t row0 = (size_t)b * a.Q * a.Hq;
    for (size_t i = threadIdx.x; i < (size_t)a.Q * a.Hq * (HD / 8); i += PA_THREADS)
      reinterpret_cast<uint4*>(a.out)[row0 * (HD / 8) + i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int i = threadIdx.x; i < a.Q * a.Hq; i += PA_THREADS) a.lse[row0 + i] = -INFINITY;
  }

  const PaOut po = {a.out, a.lse, a.Q, a.Hq, a.n_rep, a.bf16};
  PaSplit sp;
  sp.T = (long long)pre[a.B] * U;
  sp.ge = (int)min((long long)a.grid, sp.T);
  if ((int)blockIdx.x >= sp.ge) return;
  const int gw = blockIdx.x * PA_WARPS + warp;
  long long x0 = 0;
  int n_pos = 0;   // positions of this warp
  {
    const long long c0 = sp.cta0(blockIdx.x);
    // as equal as they get; the first n warps, if there are fewer positions than warps
    const int n = (int)(sp.cta0(blockIdx.x + 1) - c0);
    auto warp0 = [&](int w) { return n < PA_WARPS ? min(w, n) : (int)((long long)w * n / PA_WARPS); };
    const int w0 = warp0(warp);
    x0 = c0 + w0;
    n_pos = warp0(warp + 1) - w0;
  }

  // a walk through the units: sequence b, group gr = KV head * RT + row tile, page p of np, at
  // position x of the warp's n_pos
  struct Walk {
    int b, gr, p, np, first, x;
  };
  const long long page_step = (long long)a.Hkv * L::BYTES;
  auto enter = [&](Walk& w) {   // a sequence's page range
    while (pre[w.b + 1] == pre[w.b]) ++w.b;
    w.np = pre[w.b + 1] - pre[w.b] - lead;
    w.first = pa_first(a, slen[w.b]);
  };
  auto advance = [&](Walk& w) {   // to the next page of the range, if there is one
    ++w.x;
    if (++w.p < w.np) return;
    w.x += lead;
    w.p = 0;
    if (++w.gr < U) return;
    w.gr = 0;
    ++w.b;
    if (w.x < n_pos) enter(w);
  };
  Walk cw = {0, 0, 0, 0, 0, 0};
  if (n_pos) {
    int lo = 0, hi = a.B - 1;   // the last sequence that starts at x0 or before
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((long long)pre[mid] * U <= x0) lo = mid;
      else hi = mid - 1;
    }
    cw.b = lo;
    enter(cw);
    const long long rem = x0 - (long long)pre[cw.b] * U;
    cw.gr = (int)quotient(rem, cw.np + lead);
    cw.p = (int)(rem - (long long)cw.gr * (cw.np + lead)) - lead;
    if (cw.p < 0) cw.x = -cw.p, cw.p = 0;
  }
  Walk pw = cw;             // the copies run PA_STAGES units ahead of the computation, the
                            // page numbers one further
  int next_id = pw.x < n_pos ? a.table[pw.b * a.table_stride + pw.first + pw.p] : 0;
  uint32_t valid = 0;       // bit s: stage s holds a page
  int issued = 0;           // copies so far
  const unsigned char* head = a.pages + (pw.gr / a.RT) * L::BYTES;   // the KV head's part of page 0
  // pages are read once, unless several row tiles take them
  unsigned long long pol = evict_first_policy();
  if (a.RT > 1) asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  auto issue = [&](int s) {
    const bool ok = next_id >= 0 && next_id < a.n_pages;
    valid = (valid & ~(1u << s)) | ((uint32_t)ok << s);
    if (lane == 0) {
      const uint32_t bar = bar_s + 8 * s;
      if (ok) {
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(L::BYTES) : "memory");
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
            :: "r"(ring_s + s * L::BYTES), "l"(head + next_id * page_step), "r"(L::BYTES), "r"(bar), "l"(pol) : "memory");
      } else {
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
      }
    }
    ++issued;
    const int gr = pw.gr;
    advance(pw);
    if (pw.gr != gr) head = a.pages + (pw.gr / a.RT) * L::BYTES;
    if (pw.x < n_pos) next_id = a.table[pw.b * a.table_stride + pw.first + pw.p];
  };
  // ---- state of the group at hand ----
  // q as MMA operands: group, low and high nibbles, columns (B) or rows gid and gid + 8 (A)
  uint32_t qf[G][2][WIDE ? 4 : 2];
  uint32_t qo[WIDE ? 2 : 1];  // the group sums of q (hi and lo halves), for the offsets
  // of this lane's two rows of the tile (its columns 2tig, 2tig + 1; WIDE: gid, gid + 8):
  float cs[2];                // score factor
  int c_lo[2], c_hi[2];       // tokens seen
  int t_lo = 0, t_hi = 0, t_all = 0, t_end = 0;   // seen by every row: [t_lo, t_hi); by any: [t_all, t_end)
  // softmax reference (base 2), and the largest score / cs that needs no new one
  float ref[2], lim[2];
  // Sums over the codes.  Accumulator rows are channels, gid the low nibble's and gid + 8 the
  // byte's (16 times the high nibble's plus the low one's), and columns are queries; WIDE: rows
  // are queries and tiles 4g + n the channels 4 gid + n of group g, odd n the bytes'.  off: the sums
  // of weights times offsets per group, then (group G) the weights' own.
  float acc[MT][4], off[4];
  float top = PA_TOP;         // weights stay below 2^top
  bool started = false, failed = false;

  // a group's rows of q, as they lie in memory: of row gid (and gid + 8) channels 32k + 8tig, +7
  struct Rows {
    uint4 v[WIDE ? 2 : 1][G];
  };
  auto fetch_q = [&](const Walk& w, Rows& rows) {
    const int g = w.gr / a.RT, r0 = (w.gr - g * a.RT) * R, rn = min(R, a.rows - r0);
#pragma unroll
    for (int rj = 0; rj < (WIDE ? 2 : 1); ++rj) {
      const int r = WIDE ? gid + 8 * rj : PACK ? gid & 3 : gid;   // this lane's row of q
      const int rr = r0 + (r < rn ? r : 0), i = rr / a.n_rep, h = g * a.n_rep + rr - i * a.n_rep;
      const unsigned short* src = static_cast<const unsigned short*>(a.q) +
                                  (size_t)(((long long)w.b * a.Q + i) * a.qt + h * a.qh) + 8 * tig;
#pragma unroll
      for (int k = 0; k < G; ++k) rows.v[rj][k] = r < rn ? *reinterpret_cast<const uint4*>(src + 32 * k) : make_uint4(0, 0, 0, 0);
    }
  };
  auto load_group = [&](const Walk& w, const Rows& rows) {
    const int len = slen[w.b], g = w.gr / a.RT, r0 = (w.gr - g * a.RT) * R;
    const int rn = min(R, a.rows - r0);
    const int i0 = r0 / a.n_rep, i1 = (r0 + rn - 1) / a.n_rep;   // first and last query token of the tile
    auto hi_of = [&](int i) { return max(0, len - a.Q + 1 + i); };
    auto lo_of = [&](int i) { return a.window ? max(0, hi_of(i) - a.window) : 0; };
    t_hi = hi_of(i0), t_lo = lo_of(i1), t_all = lo_of(i0), t_end = len;
#pragma unroll
    for (int rj = 0; rj < (WIDE ? 2 : 1); ++rj) {
      const int r = WIDE ? gid + 8 * rj : PACK ? gid & 3 : gid;   // this lane's row of q
      float f[G][8], mx = 0.f;
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const uint4 v = rows.v[rj][k];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 p = pair_to_f2(word_of(v, j), a.bf16);
          f[k][2 * j] = p.x, f[k][2 * j + 1] = p.y;
          mx = fmaxf(mx, fmaxf(fabsf(p.x), fabsf(p.y)));
        }
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // the row times 2^e with a largest element in [2^9, 2^10), whatever its size down to 2^-117.  Binary16 then
      // keeps all of a binary16 or bfloat16 element down to 2^-24 of 2^10, in odd channels, which carry another
      // 1/16, down to 2^-20 (elements below lose bits that are 2^-34 of the row's largest, 2^-30 in odd
      // channels), and the sums of 32 stay finite
      int e = 0;
      if (mx > 0.f) frexpf(mx, &e);
      e = max(-126, min(126, 10 - e));
      const float up = a.scale_log2 < 0.f ? -ldexpf(1.f, e) : ldexpf(1.f, e), upl = up * 0.0625f;
      float gs[G];
#pragma unroll
      for (int k = 0; k < G; ++k) {
        float t = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) t = fmaf(f[k][j], up, t);
        t += __shfl_xor_sync(0xffffffffu, t, 1);
        t += __shfl_xor_sync(0xffffffffu, t, 2);
        gs[k] = t;
        // A operands: rows gid, gid + 8 in registers 0 and 1, the upper half of k in 2 and 3
        constexpr int U = WIDE ? 2 : 1;
        qf[k][0][rj] = h2_as_u32(__floats2half2_rn(f[k][0] * up, f[k][4] * up));
        qf[k][0][U + rj] = h2_as_u32(__floats2half2_rn(f[k][2] * up, f[k][6] * up));
        qf[k][1][rj] = h2_as_u32(__floats2half2_rn(f[k][1] * upl, f[k][5] * upl));
        qf[k][1][U + rj] = h2_as_u32(__floats2half2_rn(f[k][3] * upl, f[k][7] * upl));
      }
      // k 2tig, 2tig+1: the sums of two groups, hi halves first, then lo halves
      const int pr = tig % (G / 2), piece = tig / (G / 2);
      const float u = pr ? gs[G - 2] : gs[0], v = pr ? gs[G - 1] : gs[1];
      const __half2 h2 = __floats2half2_rn(u, v);
      const float2 hf = __half22float2(h2);
      qo[rj] = piece == 0 ? h2_as_u32(h2) : piece == 1 ? h2_as_u32(__floats2half2_rn(u - hf.x, v - hf.y)) : 0u;
      // never 0 or infinite, so that -inf stays -inf and 0 stays 0; the scale's sign is in q
      const float mine = fminf(fmaxf(ldexpf(fabsf(a.scale_log2), -e), 1.17549435e-38f), 3.402823466e38f);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (WIDE && j != rj) continue;
        cs[j] = WIDE ? mine : __shfl_sync(0xffffffffu, mine, (2 * tig + j) * 4);
        const int c = WIDE ? r : PACK ? (2 * tig + j) & 3 : 2 * tig + j;
        const int ci = (r0 + min(c, rn - 1)) / a.n_rep;
        c_lo[j] = lo_of(ci), c_hi[j] = hi_of(ci);
        ref[j] = -3.402823466e38f, lim[j] = -INFINITY;
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[mt][j] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) off[j] = 0.f;
    top = PA_TOP;
  };

  const int pr_k = tig % (G / 2);
  const bool lo_col = gid >= 4;
  // A rows of the offset product: groups, then a row of ones, then nothing
  const uint32_t o_mask = gid < G ? 0xffffffffu : 0u, o_one = gid == G ? 0x3C003C00u : 0u;
  const int o_at = L::VO + (gid % G) * 2 * PG + tig * 32;
  // byte of this lane's value pieces of tokens 2tig and 2tig + 1
  const int vrow0 = (HD == 128 ? (2 * tig + (tig & 1)) : (2 * tig + (tig >> 1))) * L::ROW;
  const int vrow1 = (HD == 128 ? (2 * tig + 1 - (tig & 1)) : (2 * tig + 1 - (tig >> 1))) * L::ROW;
  const int vx = HD == 128 ? (gid * 8) ^ (32 * (tig >> 1)) : gid * 4;

  auto page = [&](unsigned char* pg, int tok0) {
    const bool edge = tok0 < t_lo || tok0 + PG > t_hi;
    if (edge) {
      if (tok0 + PG <= t_all || tok0 >= t_end) return;
      // what lies outside of every row's tokens may be anything, NaN included: the value
      // scales and offsets there become 0 (the scores are masked below)
      for (int i = lane; i < G * PG; i += 32) {
        const int t = i % PG, at = (i / PG) * PG + vscale_at(t);
        if (tok0 + t < t_all || tok0 + t >= t_end) {
          reinterpret_cast<__half*>(pg + L::VS)[at] = __ushort_as_half(0);
          reinterpret_cast<__half*>(pg + L::VO)[at] = __ushort_as_half(0);
        } else if (__hisnan(reinterpret_cast<const __half*>(pg + L::VO)[at])) {
          // a value that is NaN: into the token's score, which the rows that do not see it mask
          // (a weight of 0 would not)
          reinterpret_cast<__half*>(pg + L::VO)[at] = __ushort_as_half(0);
          reinterpret_cast<unsigned short*>(pg + L::KO)[t * G] = 0x7fff;
        }
      }
      // ordered before the bulk copy that will overwrite the stage
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    }
    // value scales of 2 or more (exponent field above 15) lower the weights' limit
    {
      uint32_t w[G];
      lds(w, pg + L::VS + lane * 4 * G);
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < G; ++i) any |= w[i];
      if (__any_sync(0xffffffffu, (any & 0x40004000u) != 0u)) {
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < G; ++i) mx = max(mx, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
        mx = __reduce_max_sync(0xffffffffu, mx);
        const float now = fminf(top, PA_TOP - (float)((int)(mx >> 10) - 15));
        if (now != top) {
          top = now;
#pragma unroll
          for (int j = 0; j < 2; ++j) lim[j] = ref[j] < -3e38f ? -INFINITY : (ref[j] + top) / cs[j];
        }
      }
    }

#pragma unroll 1
    for (int i0 = 0; i0 < 4; i0 += STEP) {
      // ---- scores: S cs is the score in base 2 ----
      // S[.][j]: tokens gid, gid + 8 (j / 2) of a tile and column j % 2; WIDE: S[.][h][j], tokens
      // 8h + 2tig + j % 2 and row j / 2
      float S[STEP][WIDE ? 8 : 4];
#pragma unroll
      for (int ii = 0; ii < STEP; ++ii) {
        const int ta = 16 * (i0 + ii) + gid, tb = ta + 8;
        uint32_t wa[G], wb[G];
        lds(wa, pg + ta * L::ROW + tig * 4 * G);
        lds(wb, pg + tb * L::ROW + tig * 4 * G);
        const uint32_t oa = *reinterpret_cast<const uint32_t*>(pg + L::KO + ta * 2 * G + 4 * pr_k);
        const uint32_t ob = *reinterpret_cast<const uint32_t*>(pg + L::KO + tb * 2 * G + 4 * pr_k);
        if constexpr (WIDE) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t sc[G];   // scales of tokens 2tig, 2tig + 1 of the eight: G / 2 words each
            lds(sc, pg + L::KS + (16 * (i0 + ii) + 8 * h + 2 * tig) * 2 * G);
            const uint32_t* w = h ? wb : wa;
            float2 r[2];
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const uint32_t x = w[g] >> 8;
              const float2 s0 = __half22float2(u32_as_h2(sc[g >> 1])), s1 = __half22float2(u32_as_h2(sc[G / 2 + (g >> 1)]));
              const float f0 = (g & 1) ? s0.y : s0.x, f1 = (g & 1) ? s1.y : s1.x;
              float X[4];
              mma_z(X, qf[g][0][0], qf[g][0][1], qf[g][0][2], qf[g][0][3], w[g] & LO, x & LO);
              mma(X, qf[g][1][0], qf[g][1][1], qf[g][1][2], qf[g][1][3], w[g] & HI, x & HI);
#pragma unroll
              for (int j = 0; j < 2; ++j) {   // (tokens 2tig, 2tig + 1) of a row at once
                const float2 x2 = make_float2(X[2 * j], X[2 * j + 1]), f = make_float2(f0, f1);
                r[j] = g == 0 ? mul2(x2, f) : fma2(x2, f, r[j]);
              }
            }
            float O[4];
            mma_k8_z(O, qo[0], qo[1], h ? ob : oa);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float2 v = fma2(r[j], make_float2(NIB_ROW_SCALE_LO, NIB_ROW_SCALE_LO), make_float2(O[2 * j], O[2 * j + 1]));
              S[ii][4 * h + 2 * j] = v.x, S[ii][4 * h + 2 * j + 1] = v.y;
            }
          }
        } else {
          uint32_t sa[G / 2], sb[G / 2];
          lds(sa, pg + L::KS + ta * 2 * G);
          lds(sb, pg + L::KS + tb * 2 * G);
          float r[4];
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const uint32_t xa = wa[g] >> 8, xb = wb[g] >> 8;
            const float2 s2a = __half22float2(u32_as_h2(sa[g >> 1])), s2b = __half22float2(u32_as_h2(sb[g >> 1]));
            const float fa = (g & 1) ? s2a.y : s2a.x, fb = (g & 1) ? s2b.y : s2b.x;
            float X[4];
            mma_z(X, wa[g] & LO, wb[g] & LO, xa & LO, xb & LO, qf[g][0][0], qf[g][0][1]);
            mma(X, wa[g] & HI, wb[g] & HI, xa & HI, xb & HI, qf[g][1][0], qf[g][1][1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = g == 0 ? X[j] * (j < 2 ? fa : fb) : fmaf(X[j], j < 2 ? fa : fb, r[j]);
          }
          float O[4];
          mma_k8_z(O, oa, ob, qo[0]);
#pragma unroll
          for (int j = 0; j < 4; ++j) S[ii][j] = fmaf(r[j], NIB_ROW_SCALE_LO, O[j]);
        }
      }
      constexpr int NS = WIDE ? 8 : 4;
      auto row_of = [](int j) { return WIDE ? (j >> 1) & 1 : j & 1; };   // which of the lane's two rows
      if (edge) {
#pragma unroll
        for (int ii = 0; ii < STEP; ++ii)
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            const int t = tok0 + 16 * (i0 + ii) + (WIDE ? 8 * (j >> 2) + 2 * tig + (j & 1) : gid + 8 * (j >> 1));
            if (t < c_lo[row_of(j)] || t >= c_hi[row_of(j)]) S[ii][j] = -INFINITY;
          }
      }

      // ---- softmax weights 2^(S cs - ref): the reference moves only when one would pass 2^top ----
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int ii = 0; ii < STEP; ++ii)
#pragma unroll
        for (int j = 0; j < NS; ++j) mx[row_of(j)] = fmaxf(mx[row_of(j)], S[ii][j]);
      if (__any_sync(0xffffffffu, mx[0] > lim[0] || mx[1] > lim[1])) {
        float al[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {   // over the lanes that hold a row's other tokens
          float t = mx[j];
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, WIDE ? 1 : 4));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, WIDE ? 2 : 8));
          if (!WIDE) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
          const float now = t > lim[j] ? t * cs[j] - (top - PA_SLACK) : ref[j];
          al[j] = exp2_approx(ref[j] - now);
          if (t > lim[j]) lim[j] = (now + top) / cs[j];
          ref[j] = now;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[mt][j] *= al[row_of(j)];
#pragma unroll
        for (int j = 0; j < 4; ++j) off[j] *= al[row_of(j)];
      }

      // ---- values ----
#pragma unroll
      for (int ii = 0; ii < STEP; ++ii) {
        const int i = i0 + ii;
        // Weights in hi and lo halves, tokens 2tig, +1 and 8 more.  B fragments (k = tokens,
        // column gid), turned; WIDE: A fragments as they are (rows gid, gid + 8, then 8 tokens on).
        constexpr int NP = WIDE ? 4 : 2;
        uint32_t ph[NP], pl[NP];
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          float2 p;   // (packed arithmetic where it pays: tiles of 16 rows 59.4 us, 60.5 without; of 8 40.9, 40.0)
          if constexpr (WIDE) {
            const float2 e = fma2(make_float2(S[ii][2 * k], S[ii][2 * k + 1]), make_float2(cs[k & 1], cs[k & 1]),
                                  make_float2(-ref[k & 1], -ref[k & 1]));
            p = make_float2(exp2_approx(e.x), exp2_approx(e.y));
          } else {
            p.x = exp2_approx(fmaf(S[ii][2 * k], cs[0], -ref[0]));
            p.y = exp2_approx(fmaf(S[ii][2 * k + 1], cs[1], -ref[1]));
          }
          const __half2 hi = __floats2half2_rn(p.x, p.y);
          const float2 hf = __half22float2(hi);
          const float2 d = WIDE ? sub2(p, hf) : make_float2(p.x - hf.x, p.y - hf.y);
          const __half2 lo = __floats2half2_rn(d.x, d.y);
          ph[k] = WIDE ? h2_as_u32(hi) : movmatrix_t(h2_as_u32(hi));
          pl[k] = WIDE ? h2_as_u32(lo) : movmatrix_t(h2_as_u32(lo));
        }
        // codes of token pairs: word g of x[h] holds four channels of group g of two tokens
        uint32_t x[2][G];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t t0[G / 2], t1[G / 2];
          lds(t0, pg + L::VC + (16 * i + 8 * h) * L::ROW + vrow0 + vx);
          lds(t1, pg + L::VC + (16 * i + 8 * h) * L::ROW + vrow1 + vx);
#pragma unroll
          for (int g = 0; g < G; ++g) x[h][g] = __byte_perm(t0[g >> 1], t1[g >> 1], (g & 1) ? 0x7632 : 0x5410);
        }
        uint32_t o[2];
        lds(o, pg + o_at + i * 8);
        o[0] = (o[0] & o_mask) | o_one, o[1] = (o[1] & o_mask) | o_one;
        uint32_t pm[2], pz[2];
        if constexpr (PACK) {
          // columns 4..7 take the lo halves: there p_hi s is formed again for its remainder
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            pm[h] = lo_col ? pl[h] : ph[h];
            pz[h] = lo_col ? ph[h] : 0u;
          }
          mma(off, o[0], 0u, o[1], 0u, pm[0], pm[1]);
        } else if constexpr (WIDE) {
          mma(off, ph[0], ph[1], ph[2], ph[3], o[0], o[1]);
          mma(off, pl[0], pl[1], pl[2], pl[3], o[0], o[1]);
        } else {
          mma(off, o[0], 0u, o[1], 0u, ph[0], ph[1]);
          mma(off, o[0], 0u, o[1], 0u, pl[0], pl[1]);
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          uint32_t sc[2];
          lds(sc, pg + L::VS + g * 2 * PG + tig * 32 + i * 8);
          const uint32_t y0 = __byte_perm(x[0][g], 0u, 0x4341), y1 = __byte_perm(x[1][g], 0u, 0x4341);
          if constexpr (PACK) {
            uint32_t b[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const __half2 sv = u32_as_h2(sc[h]), z = u32_as_h2(pz[h]);
              b[h] = h2_as_u32(__hfma2(u32_as_h2(pm[h]), sv, __hfma2(z, sv, __hneg2(__hmul2_rn(z, sv)))));
            }
            mma(acc[2 * g], x[0][g] & LO, x[0][g] & BYTE, x[1][g] & LO, x[1][g] & BYTE, b[0], b[1]);
            mma(acc[2 * g + 1], y0 & LO, y0, y1 & LO, y1, b[0], b[1]);
          } else {
            uint32_t hi[NP], lo[NP];
#pragma unroll
            for (int k = 0; k < NP; ++k) {
              const __half2 sv = u32_as_h2(sc[WIDE ? k >> 1 : k]), p = u32_as_h2(ph[k]);
              const __half2 w = __hmul2_rn(p, sv);
              hi[k] = h2_as_u32(w);
              lo[k] = h2_as_u32(__hfma2(u32_as_h2(pl[k]), sv, __hfma2(p, sv, __hneg2(w))));   // the remainder is exact
            }
            const uint32_t x0l = x[0][g] & LO, x0b = x[0][g] & BYTE, x1l = x[1][g] & LO, x1b = x[1][g] & BYTE;
            const uint32_t y0l = y0 & LO, y1l = y1 & LO;
            if constexpr (WIDE) {
              mma(acc[4 * g], hi[0], hi[1], hi[2], hi[3], x0l, x1l);
              mma(acc[4 * g + 1], hi[0], hi[1], hi[2], hi[3], x0b, x1b);
              mma(acc[4 * g + 2], hi[0], hi[1], hi[2], hi[3], y0l, y1l);
              mma(acc[4 * g + 3], hi[0], hi[1], hi[2], hi[3], y0, y1);
              mma(acc[4 * g], lo[0], lo[1], lo[2], lo[3], x0l, x1l);
              mma(acc[4 * g + 1], lo[0], lo[1], lo[2], lo[3], x0b, x1b);
              mma(acc[4 * g + 2], lo[0], lo[1], lo[2], lo[3], y0l, y1l);
              mma(acc[4 * g + 3], lo[0], lo[1], lo[2], lo[3], y0, y1);
            } else {
              mma(acc[2 * g], x0l, x0b, x1l, x1b, hi[0], hi[1]);
              mma(acc[2 * g + 1], y0l, y0, y1l, y1, hi[0], hi[1]);
              mma(acc[2 * g], x0l, x0b, x1l, x1b, lo[0], lo[1]);
              mma(acc[2 * g + 1], y0l, y0, y1l, y1, lo[0], lo[1]);
            }
          }
        }
      }
    }
  };

  // Writes the group's rows through the warp's stage: the finished output (dst == nullptr) or
  // a piece: sums [R][HD], then reference and weight sum [R][2].
  auto emit = [&](const Walk& w, float* dst) {
    const int g = w.gr / a.RT, r0 = (w.gr - g * a.RT) * R, rn = min(R, a.rows - r0);
#pragma unroll
    for (int ct = 0; ct < (WIDE ? 2 : 1); ++ct) {   // eight rows (columns) at a time
      __syncwarp();
      if constexpr (WIDE) {
#pragma unroll
        for (int gg = 0; gg < G; ++gg)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = 2 * ct + e;
            *reinterpret_cast<float4*>(stage + gid * SROW + 32 * gg + 8 * tig + 4 * e) =
                make_float4(acc[4 * gg][k] * NIB_ROW_SCALE_LO, (acc[4 * gg + 1][k] - acc[4 * gg][k]) * NIB_ROW_SCALE_HI,
                            acc[4 * gg + 2][k] * NIB_ROW_SCALE_LO, (acc[4 * gg + 3][k] - acc[4 * gg + 2][k]) * NIB_ROW_SCALE_HI);
          }
        if (tig < G / 2) stage_o[gid * G + 2 * tig] = off[2 * ct], stage_o[gid * G + 2 * tig + 1] = off[2 * ct + 1];
        if (tig == G / 2) stage_l[gid] = failed ? __int_as_float(0x7fc00000) : off[2 * ct];
        if (tig == 0) stage_r[gid] = ref[ct];
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float* row = stage + (2 * tig + j) * SROW + 4 * gid;
#pragma unroll
          for (int gg = 0; gg < G; ++gg) {
            const float e0 = acc[2 * gg][j], e1 = acc[2 * gg][j + 2], e2 = acc[2 * gg + 1][j], e3 = acc[2 * gg + 1][j + 2];
            *reinterpret_cast<float4*>(row + 32 * gg) =
                make_float4(e0 * NIB_ROW_SCALE_LO, (e1 - e0) * NIB_ROW_SCALE_HI, e2 * NIB_ROW_SCALE_LO, (e3 - e2) * NIB_ROW_SCALE_HI);
          }
          if (gid < G) stage_o[(2 * tig + j) * G + gid] = off[j];
          if (gid == G) stage_l[2 * tig + j] = failed ? __int_as_float(0x7fc00000) : off[j];
          if (gid == 0) stage_r[2 * tig + j] = ref[j];
        }
      }
      __syncwarp();
      constexpr int TR = PACK ? 4 : 8, F4 = HD / 4;   // rows of the tile, float4s of a row
      // lane c prepares row c: where it goes and 1 / its weight sum
      const int mine = lane % TR, rt0 = 8 * ct;
      float lt = stage_l[mine];
      if (PACK) lt += stage_l[mine + 4];   // columns 4..7 hold the lo halves' sums
      const float rf = stage_r[mine];
      float inv = 0.f;
      size_t row = 0;
      if (dst) {
        if (lane < TR) reinterpret_cast<float2*>(dst + R * HD)[rt0 + lane] = make_float2(lt == 0.f ? -INFINITY : rf, lt);
      } else {
        const bool live = rt0 + mine < rn;
        if (lt != 0.f) inv = 1.f / lt;
        if (live) row = po.row(w.b, g, r0 + rt0 + mine);
        if (lane < TR && live && a.lse) a.lse[row] = lt == 0.f ? -INFINITY : (rf + log2f(lt)) * 0.69314718055994531f;
      }
#pragma unroll
      for (int k = 0; k < TR * F4 / 32; ++k) {
        const int e = lane + 32 * k, c = e / F4, x = e % F4;
        auto at = [&](int col) {
          const float4 v = *reinterpret_cast<const float4*>(stage + col * SROW + 4 * x);
          const float o = stage_o[col * G + x / 8];
          return make_float4(v.x + o, v.y + o, v.z + o, v.w + o);
        };
        float4 v = at(c);
        if (PACK) {
          const float4 u = at(c + 4);
          v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
        }
        const float f = __shfl_sync(0xffffffffu, inv, c);
        const size_t to = __shfl_sync(0xffffffffu, (unsigned long long)row, c);
        if (dst)
          reinterpret_cast<float4*>(dst)[(rt0 + c) * F4 + x] = v;
        else if (rt0 + c < rn)
          reinterpret_cast<uint2*>(a.out)[to * F4 + x] = make_uint2(f2_to_pair(v.x * f, v.y * f, a.bf16), f2_to_pair(v.z * f, v.w * f, a.bf16));
      }
    }
  };

  bool open = n_pos > 0;
  int it = 0;
  if (open) {   // the first group's rows are on their way while the first pages are asked for
    Rows rows;
    fetch_q(cw, rows);
#pragma unroll 1
    for (int s = 0; s < PA_STAGES; ++s)
      if (pw.x < n_pos) issue(s);
    load_group(cw, rows);
    started = cw.p == 0;
  }
  while (cw.x < n_pos) {
    if (!open) {
      Rows rows;
      fetch_q(cw, rows);
      load_group(cw, rows);
      open = true;
      started = cw.p == 0;
    }
    const int s = ring_stage<PA_STAGES>(it);
    if (!failed && !pa_wait(bar_s + 8 * s, ring_parity<PA_STAGES>(it))) failed = true;
    failed = __any_sync(0xffffffffu, failed);
    if (!failed && ((valid >> s) & 1u)) page(ring + s * L::BYTES, (cw.first + cw.p) * PG);
    __syncwarp();
    if (!failed && pw.x < n_pos) issue(s);
    ++it;
    const Walk at = cw;
    advance(cw);
    const bool end = at.p + 1 == at.np;
    if (end || cw.x >= n_pos) {
      // an open group's piece goes to the ring, which no copy uses any more
      if (failed) pa_drain(bar_s, issued), issued = 0;
      float* dst = !end ? reinterpret_cast<float*>(ring) : started ? nullptr : a.part + (size_t)gw * PART;
      emit(at, dst);
      if (lane == 0) {
        if (dst) piece_at[warp][!end] = dst;
        if (end) {
          if (!started) ended[warp] = make_int2(at.b, at.gr);
        } else {
          open_at[warp] = make_int2(at.b, at.gr);
          open_new[warp] = started;
        }
      }
      open = false;
    }
  }
  const bool lost = __syncthreads_or(failed);   // a copy that never lands may still write over a piece in a ring

  // ---- groups that were cut ----
  float* cpart = a.part + (size_t)a.grid * PA_WARPS * PART;
  // Runs of pieces of one group within this CTA: that of a group begun in an earlier CTA (w =
  // -1), then those of the groups that a warp starts and leaves open.  Warps hold consecutive
  // ranges, so an open piece that its warp did not start, and an ended one, belong to the group
  // that the warp before left open: bit masks over the warps tell where each run ends.
  int2 away[2] = {make_int2(-1, 0), make_int2(-1, 0)};   // groups with pieces in other CTAs
  const bool is_end = lane < PA_WARPS && ended[lane].x >= 0, is_open = lane < PA_WARPS && open_at[lane].x >= 0;
  const bool is_new = is_open && open_new[lane];
  const uint32_t ends = __ballot_sync(0xffffffffu, is_end), news = __ballot_sync(0xffffffffu, is_new);
  const uint32_t goes_on = __ballot_sync(0xffffffffu, is_open && !is_new);
  // bit w + 1: a run starts in warp w
  for (uint32_t left = (news << 1) | ((ends | goes_on) & 1u); left; left &= left - 1) {
    const int w = __ffs(left) - 2;
    const int f = w + __ffs(~(goes_on >> (w + 1))) - 1;   // the last warp with an open piece of it
    const bool closed = (ends >> (f + 1)) & 1u;
    const int first = max(w, 0), n = f + closed - first + 1;
    const int2 grp = w < 0 && !(goes_on & 1u) ? ended[0] : open_at[first];
    const int slot = w >= 0;
    const bool all = closed && w >= 0;
    if (!all) away[slot] = grp;
    const int g = grp.y / a.RT, r0 = (grp.y - g * a.RT) * R;
    pa_merge<HD, R, false>(po, &piece_at[first][0], n, closed, lost, grp.x, g, r0, min(R, a.rows - r0),
                           all ? nullptr : cpart + ((size_t)blockIdx.x * 2 + slot) * PART);
  }
  if (away[0].x < 0 && away[1].x < 0) return;
  __syncthreads();
  int first_cta[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (away[k].x < 0) continue;
    const long long size = pre[away[k].x + 1] - pre[away[k].x];
    const long long at = (long long)pre[away[k].x] * U + away[k].y * size;
    // the CTAs that hold its first page and its last one
    first_cta[k] = k ? (int)blockIdx.x : sp.cta_of(at + lead);
    if (threadIdx.x == 32 * k) {
      const int n = sp.cta_of(at + size - 1) - first_cta[k] + 1;
      // releases this CTA's pieces (written before the barrier) and acquires the others'
      int before;
      asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(a.arrived + first_cta[k]) : "memory");
      final_n[k] = before == n - 1 ? n : 0;
      if (before == n - 1) a.arrived[first_cta[k]] = 0;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    if (away[k].x < 0 || final_n[k] == 0) continue;
    const float* at = cpart + (size_t)first_cta[k] * 2 * PART;
    const int g = away[k].y / a.RT, r0 = (away[k].y - g * a.RT) * R;
    pa_merge<HD, R, true>(po, &at, final_n[k], false, false, away[k].x, g, r0, min(R, a.rows - r0), nullptr);
  }
}

const char* shape_error(int B, int Q, int Hq, int Hkv, int hd) {
  if (B < 0 || B > PA_MAX_BATCH) return "batch must be in 0..2048";
  if (Q < 1 || Q > 64) return "n_q_tokens must be in 1..64";
  if (Hkv > MAX_KV_HEADS) return "n_kv_heads must be in 1..4096";
  if (Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || Hq / Hkv > 64) return "n_q_heads / n_kv_heads must be an integer in 1..64";
  if (hd != 64 && hd != 128) return "head_dim must be 64 or 128";
  return nullptr;
}

// Query rows per tile: 4 or 8 if those hold a KV head's rows, else 16 or, of 8, twice as many tiles,
// each of which reads the pages again (from L2).  Tiles of 16 take less time per page and row (16 rows, 8
// sequences of 16384 tokens: 60 us, 69 with tiles of 8; of 8192: 38 and 41), tiles of 8 start and
// finish faster (of 4096: 27 us, 28 with tiles of 16; of 1024: 15 and 18), and 17 to 24 rows fill
// three of them (20 rows, 8 sequences of 8192: 56 us, 61 with two tiles of 16).  The lengths are
// not known on the host, the most pages are.
constexpr int PA_FEW = 4;   // pages per warp, if all were in use
int tile_rows(int rows, long long most_pages, int sms) {
  if (rows <= 8) return rows <= 4 ? 4 : 8;
  if (rows > 16 && rows <= 24) return 8;
  return most_pages * ((rows + 15) / 16) < (long long)sms * PA_WARPS * PA_FEW ? 8 : 16;
}

cudaError_t sm_count(int* sms) {
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

// arrival counters, then pieces: one per warp and two per CTA
constexpr size_t PA_COUNTERS = 4096;
size_t ws_bytes(int sms, int Q, int Hq, int Hkv, int hd) {
  const int rows = Q * (Hq / Hkv);
  return PA_COUNTERS + (size_t)sms * (PA_WARPS + 2) * (rows <= 4 ? 4 : rows <= 8 ? 8 : 16) * (hd + 2) * sizeof(float);
}

template <int HD, int R>
cudaError_t launch(const PaArgs& a, cudaStream_t st) {
  auto bytes = [](int batch) {
    return (size_t)PA_WARPS * (PA_STAGES * Page<HD>::BYTES + PaStage<HD>::FLOATS * sizeof(float)) + (2 * (size_t)batch + 1) * sizeof(int);
  };
  auto* k = paged_attention_kernel<HD, R>;
  // the limit belongs to the function and is every host thread's: always the one of the largest batch, so that
  // no call lowers another's
  if (cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes(PA_MAX_BATCH))) return e;
  return launch_dependent(k, dim3(a.grid), dim3(PA_THREADS), bytes(a.B), st, a);
}

kvq_status attention_impl(int dtype, const void* q, int64_t qt, int64_t qh, const void* pages, int n_pages,
                          const int32_t* table, int64_t table_stride, int max_pages, const int32_t* lens, int B, int Q,
                          int Hq, int Hkv, int hd, int window, float scale, void* out, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const char* fn = "kvq_paged_attention";
  if (dtype != KVQ_F16 && dtype != KVQ_BF16) return paged_fail(KVQ_ERR_INVALID, fn, "dtype must be KVQ_F16 or KVQ_BF16");
  if (const char* msg = shape_error(B, Q, Hq, Hkv, hd)) return paged_fail(KVQ_ERR_INVALID, fn, msg);
  if (n_pages < 1 || n_pages > (1 << 25)) return paged_fail(KVQ_ERR_INVALID, fn, "n_pages must be in 1..33554432");
  if (max_pages < 1 || max_pages > (1 << 24) || (long long)B * max_pages >= (1ll << 30))
    return paged_fail(KVQ_ERR_INVALID, fn, "max_pages must be in 1..16777216 and batch * max_pages below 2^30");
  if (table_stride < 0) return paged_fail(KVQ_ERR_INVALID, fn, "table_stride must be >= 0");
  if (window < 0) return paged_fail(KVQ_ERR_INVALID, fn, "window must be >= 0");
  const float scale_log2 = (scale != 0.f ? scale : 1.f / std::sqrt((float)hd)) * LOG2E_F;
  if (!std::isfinite(scale_log2)) return paged_fail(KVQ_ERR_INVALID, fn, "scale * log2(e) must be finite");
  if (B == 0) return KVQ_OK;
  if (q == out) return paged_fail(KVQ_ERR_INVALID, fn, "out must not be q");
  if (kvq_status s = check_strides(qt, qh, fn, "q")) return s;
  int dev = 0, sms = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return paged_cuda_fail(e, fn, "no current CUDA device");
  if (cudaError_t e = sm_count(&sms)) return paged_cuda_fail(e, fn, "device attributes");
  if (kvq_status s = check_buffer(q, dev, 16, fn, "q")) return s;
  if (kvq_status s = check_buffer(pages, dev, 16, fn, "pages")) return s;
  if (kvq_status s = check_buffer(table, dev, 4, fn, "page_table")) return s;
  if (kvq_status s = check_buffer(lens, dev, 4, fn, "seq_lens")) return s;
  if (kvq_status s = check_buffer(out, dev, 16, fn, "out")) return s;
  if (lse)
    if (kvq_status s = check_buffer(lse, dev, 4, fn, "lse")) return s;
  if (kvq_status s = check_buffer(workspace, dev, 16, fn, "workspace")) return s;
  if (workspace_bytes < ws_bytes(sms, Q, Hq, Hkv, hd))
    return paged_fail(KVQ_ERR_INVALID, fn, "workspace smaller than kvq_paged_attention_workspace reports");
  PaArgs a = {};
  a.q = q, a.pages = static_cast<const unsigned char*>(pages), a.table = table, a.lens = lens, a.out = out, a.lse = lse;
  a.qt = qt, a.qh = qh, a.table_stride = table_stride, a.n_pages = n_pages, a.max_pages = max_pages;
  a.B = B, a.Q = Q, a.Hq = Hq, a.Hkv = Hkv, a.n_rep = Hq / Hkv, a.rows = Q * a.n_rep;
  a.window = std::min(window, 1 << 30);   // lengths stay below 2^30
  a.scale_log2 = scale_log2;
  a.bf16 = dtype == KVQ_BF16;
  const int R = tile_rows(a.rows, (long long)B * max_pages * Hkv, sms);
  a.RT = (a.rows + R - 1) / R;
  // one CTA per SM (the counters hold 1024), fewer when the table cannot hold that many units
  a.grid = (int)std::min<long long>(std::min(sms, 1024), (long long)B * max_pages * Hkv * a.RT);
  if ((long long)B * (max_pages + PA_MAX_LEAD) * Hkv * a.RT / a.grid >= (1ll << 30))   // a CTA's positions are ints
    return paged_fail(KVQ_ERR_INVALID, fn, "batch * max_pages * n_kv_heads is too large for one call");
  a.arrived = static_cast<int*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + PA_COUNTERS);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (hd == 128) e = R == 4 ? launch<128, 4>(a, st) : R == 8 ? launch<128, 8>(a, st) : launch<128, 16>(a, st);
  else e = R == 4 ? launch<64, 4>(a, st) : R == 8 ? launch<64, 8>(a, st) : launch<64, 16>(a, st);
  if (e != cudaSuccess) return paged_cuda_fail(e, fn, "launch");
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

extern "C" kvq_status kvq_paged_attention_workspace(int batch, int n_q_tokens, int n_q_heads, int n_kv_heads,
                                                    int head_dim, size_t* bytes) try {
  const char* fn = "kvq_paged_attention_workspace";
  if (!bytes) return kvq::paged_fail(KVQ_ERR_INVALID, fn, "NULL output");
  if (const char* msg = kvq::shape_error(batch, n_q_tokens, n_q_heads, n_kv_heads, head_dim))
    return kvq::paged_fail(KVQ_ERR_INVALID, fn, msg);
  int sms = 0;
  if (cudaError_t e = kvq::sm_count(&sms)) {
    cudaGetLastError();
    return kvq::paged_cuda_fail(e, fn, "no current CUDA device");
  }
  *bytes = kvq::ws_bytes(sms, n_q_tokens, n_q_heads, n_kv_heads, head_dim);
  return KVQ_OK;
} catch (...) {
  return KVQ_ERR_HOST_OOM;
}

extern "C" kvq_status kvq_paged_attention(int dtype, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                          const void* pages, int n_pages, const int32_t* page_table,
                                          int64_t table_stride, int max_pages, const int32_t* seq_lens, int batch,
                                          int n_q_tokens, int n_q_heads, int n_kv_heads, int head_dim, int window,
                                          float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                          void* stream) try {
  return kvq::attention_impl(dtype, q, q_token_stride, q_head_stride, pages, n_pages, page_table, table_stride, max_pages,
                             seq_lens, batch, n_q_tokens, n_q_heads, n_kv_heads, head_dim, window, scale, out, lse,
                             workspace, workspace_bytes, stream);
} catch (...) {
  return KVQ_ERR_HOST_OOM;
}
