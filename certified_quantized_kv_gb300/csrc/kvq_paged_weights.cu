// kvq_paged_weights.cu -- attention weights summed per cached token of the paged 4-bit cache:
//   w[b, g, t] = decay w[b, g, t] + sum over query tokens i and heads r of group g of exp(scale q_ir k^_t - lse_ir)
// over the rows that see token t.  Only the keys' halves of the pages are read (80 bytes of a token's 160 at
// head_dim 128).
//
// As in the attention over these pages, nibbles are never converted: masked out of their words they are binary16
// subnormals n 2^-24 (low nibble of a byte) or 16 n 2^-24 (high nibble, whose channels carry 1/16 in q), exact MMA
// operands; the key scales multiply each group's fp32 sums and the offsets are a product of their own,
//   score = sum_g s_tg (q_g . code_tg) + sum_g o_tg sum(q_g),
// so that scores are fp32 sums of exact products.  Tokens are MMA rows and query rows its columns: a lane holds two
// tokens of each 16, and their sums over all query rows stay in its registers.
//
// The (sequence, KV head, page) units are numbered in that order and cut into equal contiguous ranges, one per CTA and
// SM, whatever the lengths (each head counts PW_LEAD pages more, for its start).  For each (sequence, KV head) of its range,
// several at once, a CTA brings the query rows (WT_FROM - 1 at most) to binary16 in shared memory, in the order in which lanes
// take them (times a power of two per row, as in the attention); each warp then takes whole pages, which bulk copies bring into
// a ring of its own two ahead, across the heads' borders too: a quarter of a page's codes is masked into MMA operands once,
// and the rows' tiles pass by.  More rows go to the kernel further below.  Every sum has one owner and a fixed order.
// Bound by issue: 0.59 per cycle, some 800 instructions per page, with half of the MMA columns empty at four query heads to a
// KV head.  64 ragged sequences up to 16384 tokens, one query each, 8 KV heads of 128: 63.5 us, 3.9 TB/s.
#include <algorithm>
#include <cmath>
#include <string>

#include "kvq.h"
#include "kvq_launch.h"
#include "kvq_paged.cuh"
#include "kvq_tc.cuh"

namespace kvq {

namespace {

constexpr int PW_ROWS = 8;            // query rows of a tile (MMA columns)
constexpr int PW_TILES = 16;          // tiles in shared memory at once
constexpr int PW_THREADS = 512, PW_WARPS = PW_THREADS / 32, PW_MAX_BATCH = 2048;
// Positions that a (sequence, KV head) takes in the ranges besides its pages, for what starting it costs in pages' time
constexpr int PW_LEAD = 3;
constexpr int PW_STAGES = 2;          // pages on their way per warp
constexpr unsigned long long PW_WAIT_NS = 2000000000ull;   // bounded waits: 2 s

// Query rows of a KV head from which on the second kernel takes them, tokens as lanes.  us with tiles of 8 / with blocks of 32:
//   sequences x tokens, KV heads, head_dim    32 rows        56             64             80              128
//   1 x 131072, 8, 128                        38.5 / 41.4    57.3 / 61.9    63.6 / 61.9    76.3 / 82.2     114 / 103
//   1 x 4096, 8, 128                          7.2 / 7.5      9.4 / 9.1      10.1 / 9.1     11.6 / 10.7     15.9 / 12.4
//   64 x 2048, 8, 128                         46.4 / 56.3    70.2 / 82.8    77.5 / 83.0    96.1 / 107      142 / 132
//   256 x 256, 8, 128                         48.4 / 77.6    72.5 / 106     78.5 / 108     145 / 135       210 / 174
//   1 x 131072, 8, 64                         28.4 / 28.6    41.2 / 44.7    45.5 / 44.7    54.0 / 59.9     79.7 / 74.5
//   64 x 2048, 8, 64                          35.6 / 38.5    52.6 / 56.5    57.7 / 56.4    71.4 / 74.2     104 / 90.8
//   8 x 1000, 1, 64                           6.9 / 5.8      8.8 / 6.9      9.4 / 6.9      10.7 / 8.4      14.4 / 9.5
// The crossing moves with the number of sequences, which blocks of 32 pay for at each start, and with what a block leaves
// empty (65 to 96 rows); lengths are on the device, so the rule goes by rows alone.
constexpr int WT_FROM = 57;
static_assert(WT_FROM - 1 <= PW_ROWS * PW_TILES, "the first kernel holds all of its rows at once");

// A page's keys in a stage: the codes, then scales and offsets
template <int HD>
struct PwStage {
  static constexpr int KS = Page<HD>::CODES, KO = KS + Page<HD>::SCALES, BYTES = KO + Page<HD>::SCALES;
};

// One tile of query rows as the main kernel takes it.
template <int HD>
struct alignas(16) PwTile {
  uint4 q[HD / 32][32];       // per group and lane: B fragments of the low nibbles' and of the high nibbles' product
  uint32_t o[32];             // per lane: B fragment of the offsets' product (sums of two groups, hi and lo halves)
  float scale[PW_ROWS];       // of a score in base 2; 0 and
  float lse[PW_ROWS];         // +inf for rows that count nothing: 2^(0 - inf) = 0
  int lo[PW_ROWS], hi[PW_ROWS];   // tokens that a row sees
};

struct PwArgs {
  const void* q;
  const float* lse;
  const unsigned char* pages;
  const int32_t *table, *lens;
  float* weights;
  long long qt, qh, table_stride, ws, wh;
  int n_pages, max_pages, columns, B, Q, Hq, Hkv, n_rep, rows, RT, window;
  float scale_log2, decay;
  bool bf16;
};

__device__ __forceinline__ int pw_len(const PwArgs& a, int b) { return min(max(a.lens[b], 0), a.max_pages * PG); }

__device__ __forceinline__ void pw_mma(float (&c)[4], const uint32_t (&x)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void pw_mma_z(float (&c)[4], const uint32_t (&x)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void pw_mma_k8_z(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}

// Tile `rt` of a (sequence, KV head), by one warp: lane (gid, tig) holds the channels 32k + 8 tig .. + 7 of row gid.  True in
// lanes whose row counts nothing: what it holds may be NaN, so that its tile is masked by lo and hi.
template <int HD>
__device__ __forceinline__ bool pw_rows(const PwArgs& a, int b, int g, int rt, int n, PwTile<HD>& out) {
  constexpr int G = HD / 32;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int r = rt * PW_ROWS + gid;
  const bool live = r < a.rows;
  const int i = live ? r / a.n_rep : 0, h = g * a.n_rep + (live ? r - i * a.n_rep : 0);
  const unsigned short* src = static_cast<const unsigned short*>(a.q) + ((long long)b * a.Q + i) * a.qt + h * a.qh + 8 * tig;
  float f[G][8], mx = 0.f;
#pragma unroll
  for (int k = 0; k < G; ++k) {
    const uint4 v = live ? *reinterpret_cast<const uint4*>(src + 32 * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = pair_to_f2(word_of(v, j), a.bf16);
      f[k][2 * j] = p.x, f[k][2 * j + 1] = p.y;
      mx = fmaxf(mx, fmaxf(fabsf(p.x), fabsf(p.y)));
    }
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  // the row times 2^e with a largest element in [2^9, 2^10) (as in the attention: what binary16 then loses lies
  // 2^-30 below the row's largest element)
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
    out.q[k][lane] = make_uint4(h2_as_u32(__floats2half2_rn(f[k][0] * up, f[k][4] * up)), h2_as_u32(__floats2half2_rn(f[k][2] * up, f[k][6] * up)),
                                h2_as_u32(__floats2half2_rn(f[k][1] * upl, f[k][5] * upl)), h2_as_u32(__floats2half2_rn(f[k][3] * upl, f[k][7] * upl)));
  }
  const int pr = tig % (G / 2), piece = tig / (G / 2);
  const float x = pr ? gs[G - 2] : gs[0], y = pr ? gs[G - 1] : gs[1];
  const __half2 h2 = __floats2half2_rn(x, y);
  const float2 hf = __half22float2(h2);
  out.o[lane] = piece == 0 ? h2_as_u32(h2) : piece == 1 ? h2_as_u32(__floats2half2_rn(x - hf.x, y - hf.y)) : 0u;
  const float lse = live ? a.lse[((long long)b * a.Q + i) * a.Hq + h] : 0.f;
  // a row that sees nothing (lse -inf) counts nothing
  const bool counts = live && (lse > -INFINITY || lse != lse);
  if (tig == 0) {
    const int hi = max(0, n - a.Q + 1 + i), lo = a.window ? max(0, hi - a.window) : 0;
    out.scale[gid] = counts ? fminf(fmaxf(ldexpf(fabsf(a.scale_log2), -e), 1.17549435e-38f), 3.402823466e38f) : 0.f;
    out.lse[gid] = counts ? lse * LOG2E_F : INFINITY;
    out.lo[gid] = counts ? lo : 0, out.hi[gid] = counts ? hi : 0;
  }
  return live && !counts;
}

__device__ __forceinline__ bool pw_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __noinline__ bool pw_wait_slow(uint32_t bar, uint32_t parity) {
  unsigned long long t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  while (!pw_try(bar, parity)) {
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (t - t0 > PW_WAIT_NS) return false;
  }
  return true;
}

template <int HD>
__global__ void __launch_bounds__(PW_THREADS, 1) paged_weights_kernel(PwArgs a) {
  using L = Page<HD>;
  using St = PwStage<HD>;
  constexpr int G = L::G;
  constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u;
  extern __shared__ __align__(128) unsigned char sm[];
  PwTile<HD>* tiles = reinterpret_cast<PwTile<HD>*>(sm + PW_WARPS * PW_STAGES * St::BYTES);
  int* pre = reinterpret_cast<int*>(tiles + PW_TILES);   // [B + 1] positions before each sequence, of one KV head
  int* lens = pre + a.B + 1;                             // [B]
  __shared__ __align__(8) unsigned long long bars[PW_WARPS][PW_STAGES];
  __shared__ int wsum[PW_WARPS];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  unsigned char* ring = sm + warp * PW_STAGES * St::BYTES;
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring), bar_s = (uint32_t)__cvta_generic_to_shared(&bars[warp][0]);
  if (lane == 0) {
    for (int k = 0; k < PW_STAGES; ++k) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" :: "r"(bar_s + 8 * k) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_trigger();
  pdl_wait();
  if (threadIdx.x == 0) pre[0] = 0;
  for (int base = 0, run = 0; base < a.B; base += PW_THREADS) {
    const int b = base + threadIdx.x;
    const int len = b < a.B ? pw_len(a, b) : 0, np = (min(len, a.columns) + PG - 1) / PG;   // (tokens without a column count nothing)
    if (b < a.B) lens[b] = len;
    int inc = np ? np + PW_LEAD : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int all = run;
    for (int k = 0; k < PW_WARPS; ++k) {
      if (k < warp) inc += wsum[k];
      all += wsum[k];
    }
    if (b < a.B) pre[b + 1] = run + inc;
    run = all;
    __syncthreads();
  }
  const long long total = (long long)pre[a.B] * a.Hkv;
  const long long x0 = quotient(blockIdx.x * total, gridDim.x), x1 = quotient((blockIdx.x + 1) * total, gridDim.x);
  if (x0 == x1) return;

  // The part of this CTA's range that lies in one (sequence, KV head)
  struct Part {
    long long x, end;        // positions
    int b, g, page0, pages, n;
    int warp0;   // the first of its pages that this warp takes (every PW_WARPS-th unit of the CTA's range)
  };
  auto part_at = [&](long long x, int b) {   // b: a sequence at or before x's
    Part p;
    while ((long long)pre[b + 1] * a.Hkv <= x) ++b;
    const int np = pre[b + 1] - pre[b];
    const long long in = x - (long long)pre[b] * a.Hkv;
    p.x = x, p.b = b, p.g = (int)quotient(in, np);
    const int at = (int)(in - (long long)p.g * np), taken = (int)min((long long)(np - at), x1 - x);
    p.end = x + taken;
    p.page0 = max(0, at - PW_LEAD), p.pages = max(0, at + taken - PW_LEAD) - p.page0;
    p.n = lens[b];
    p.warp0 = (warp + PW_WARPS - (int)((x - x0) % PW_WARPS)) % PW_WARPS;
    return p;
  };
  auto first_of = [&](int n) { return a.window ? max(0, n - a.Q + 1 - a.window) : 0; };   // tokens before it no query sees
  int b0 = 0;
  for (int b1 = a.B; b1 - b0 > 1;) {   // the last sequence that starts at x0 or before
    const int m = (b0 + b1) / 2;
    if ((long long)pre[m] * a.Hkv <= x0) b0 = m; else b1 = m;
  }

  // ---- copies, two pages ahead of their use: parts, then this warp's pages ----
  Part ahead = part_at(x0, b0);
  int at_page = ahead.warp0, issued = 0, found = -1;
  bool failed = false, more = true;
  uint32_t valid = 0;   // bit k: stage k holds a page that is seen
  auto look = [&]() {   // the number of the walk's page (-1: none that is seen)
    while (at_page >= ahead.pages) {
      if (ahead.end >= x1) {
        more = false;
        return;
      }
      ahead = part_at(ahead.end, ahead.b);
      at_page = ahead.warp0;
    }
    const int page = ahead.page0 + at_page;
    found = a.table[ahead.b * a.table_stride + page];
    if (found < 0 || found >= a.n_pages || (page + 1) * PG <= first_of(ahead.n)) found = -1;
  };
  look();
  auto issue = [&]() {   // into the next stage, and look up the page after
    const int k = ring_stage<PW_STAGES>(issued);
    ++issued;
    valid = found >= 0 ? valid | 1u << k : valid & ~(1u << k);
    if (lane == 0) {
      const uint32_t bar = bar_s + 8 * k, to = ring_s + k * St::BYTES;
      if (found >= 0) {
        const unsigned char* pg = a.pages + ((size_t)found * a.Hkv + ahead.g) * L::BYTES;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(St::BYTES) : "memory");
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                     :: "r"(to), "l"(pg), "r"(L::CODES), "r"(bar) : "memory");
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                     :: "r"(to + St::KS), "l"(pg + L::KS), "r"(2 * L::SCALES), "r"(bar) : "memory");
      } else {
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
      }
    }
    at_page += PW_WARPS;
    look();
  };
  for (int k = 0; k < PW_STAGES; ++k)
    if (more) issue();

  // Rows of several parts at once where there is room for their tiles, so that warps meet once for all of them.
  const int nt = a.RT, batch = PW_TILES / nt;
  int used = 0;
  for (Part p = part_at(x0, b0);; p = part_at(p.end, p.b)) {
    int parts = 0;
    bool silent = false;
    __syncthreads();   // the tiles' last readers are done
    for (Part r = p;; r = part_at(r.end, r.b)) {
      // tile k of part y is number y nt + k, one warp's each
      for (int k = (warp + PW_WARPS - parts * nt % PW_WARPS) % PW_WARPS; k < nt; k += PW_WARPS)
        silent |= pw_rows<HD>(a, r.b, r.g, k, r.n, tiles[parts * nt + k]);
      if (++parts == batch || r.end >= x1) break;
    }
    silent = __syncthreads_or(silent);
    for (int y = 0; y < parts; ++y) {
      if (y) p = part_at(p.end, p.b);
      const int n = p.n, cols = min(n, a.columns);
      for (int page = p.warp0; page < p.pages; page += PW_WARPS) {
        const int tok0 = (p.page0 + page) * PG;
        float* w = a.weights + p.b * a.ws + p.g * a.wh + tok0;
        // what is there of this lane's tokens (decay 0 does not read it)
        float old[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) old[k] = a.decay != 0.f && tok0 + 32 * k + 8 * tig + gid < cols ? w[32 * k + 8 * tig + gid] : 0.f;
        const int stage = ring_stage<PW_STAGES>(used);
        const unsigned char* pg = ring + stage * St::BYTES;
        const uint32_t parity = ring_parity<PW_STAGES>(used);
        ++used;
        if (!failed && !pw_try(bar_s + 8 * stage, parity)) failed = !pw_wait_slow(bar_s + 8 * stage, parity);
        failed = __any_sync(0xffffffffu, failed);
        const bool seen = (valid >> stage) & 1u;
        // whether some row does not see all of the page, or counts nothing
        const bool edge = silent || tok0 + PG > n - a.Q + 1 || (a.window && tok0 < n - a.window);
        float mine[8];   // sums of tokens 8k + gid
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};   // tokens gid and gid + 8 of a tile; the even and the odd columns
          if (seen) {
            uint32_t low[G][4], high[G][4], off[2];
            float sc[2][G];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int t = 16 * i + 8 * k + gid;
              uint32_t c[G], h[G / 2];
              if constexpr (G == 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(pg + t * L::ROW + tig * 4 * G);
                c[0] = v.x, c[1] = v.y, c[2] = v.z, c[3] = v.w;
                const uint2 y = *reinterpret_cast<const uint2*>(pg + St::KS + t * 2 * G);
                h[0] = y.x, h[1] = y.y;
              } else {
                const uint2 v = *reinterpret_cast<const uint2*>(pg + t * L::ROW + tig * 4 * G);
                c[0] = v.x, c[1] = v.y;
                h[0] = *reinterpret_cast<const uint32_t*>(pg + St::KS + t * 2 * G);
              }
              off[k] = *reinterpret_cast<const uint32_t*>(pg + St::KO + t * 2 * G + 4 * (tig % (G / 2)));
#pragma unroll
              for (int g = 0; g < G; ++g) {
                low[g][k] = c[g] & LO, low[g][2 + k] = (c[g] >> 8) & LO;
                high[g][k] = c[g] & HI, high[g][2 + k] = (c[g] >> 8) & HI;
                const float2 f = __half22float2(u32_as_h2(h[g / 2]));
                sc[k][g] = g & 1 ? f.y : f.x;
              }
            }
#pragma unroll 1
            for (int rt = 0; rt < nt; ++rt) {
              const PwTile<HD>& T = tiles[y * nt + rt];
              uint4 q[G];
#pragma unroll
              for (int k = 0; k < G; ++k) q[k] = T.q[k][lane];
              const uint32_t qo = T.o[lane];
              const float2 scale = *reinterpret_cast<const float2*>(T.scale + 2 * tig), lse = *reinterpret_cast<const float2*>(T.lse + 2 * tig);
              const float2 minus = make_float2(-lse.x, -lse.y);
              float2 r[2];   // of the tile's two tokens, two columns each
#pragma unroll
              for (int g = 0; g < G; ++g) {
                float X[4];
                pw_mma_z(X, low[g], q[g].x, q[g].y);
                pw_mma(X, high[g], q[g].z, q[g].w);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const float2 x = make_float2(X[2 * k], X[2 * k + 1]), f = make_float2(sc[k][g], sc[k][g]);
                  r[k] = g == 0 ? mul2(x, f) : fma2(x, f, r[k]);
                }
              }
              float O[4];
              pw_mma_k8_z(O, off[0], off[1], qo);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float2 s = fma2(r[k], make_float2(NIB_ROW_SCALE_LO, NIB_ROW_SCALE_LO), make_float2(O[2 * k], O[2 * k + 1]));
                const float2 e = fma2(s, scale, minus);
                float2 pr = make_float2(exp2_approx(e.x), exp2_approx(e.y));
                if (edge) {
                  const int t = tok0 + 16 * i + 8 * k + gid;
                  const int2 lo = *reinterpret_cast<const int2*>(T.lo + 2 * tig), hi = *reinterpret_cast<const int2*>(T.hi + 2 * tig);
                  pr = make_float2(t >= lo.x && t < hi.x ? pr.x : 0.f, t >= lo.y && t < hi.y ? pr.y : 0.f);
                }
                sum[k] = add2(sum[k], pr);
              }
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) mine[2 * i + k] = sum[k].x + sum[k].y;
        }
        // over the four lanes with the other columns, each of which ends up with two tokens: 32k + 8 tig + gid
        float half[4], own[2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float keep = tig & 1 ? mine[2 * k + 1] : mine[2 * k], give = tig & 1 ? mine[2 * k] : mine[2 * k + 1];
          half[k] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float keep = tig & 2 ? half[2 * k + 1] : half[2 * k], give = tig & 2 ? half[2 * k] : half[2 * k + 1];
          own[k] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int t = 32 * k + 8 * tig + gid;
          const float x = failed ? __int_as_float(0x7fc00000) : own[k];
          if (tok0 + t < cols) w[t] = a.decay == 0.f ? x : fmaf(old[k], a.decay, x);
        }
        __syncwarp();   // the stage's last readers are done
        if (!failed && more) issue();
      }
    }
    if (p.end >= x1) break;
  }
  if (failed) ring_drain<PW_STAGES>(issued, [&](int k, uint32_t parity) { pw_wait_slow(bar_s + 8 * k, parity); });
}

// ---- many query rows: on the 5th-generation tensor cores ----
// The same sums with tokens as the rows of M = 128 tiles and up to 128 query rows as columns, 32 at a time: an accumulator
// of its own for each group of 32 channels, since the groups' scales come behind them.  A thread owns a token (a lane of
// TMEM), so its scales, offsets and sum stay in its registers and nothing is reduced across lanes; what a row brings (the
// sums of its groups for the offsets, scale, log-sum-exp) is read from shared memory, the same for all lanes.
// Bound by the reads of what rows bring: three 16-byte loads of shared memory per two rows and warp take two thirds of the
// load unit's cycles, and the issue slots are 0.63 busy (128 rows, 131072 tokens, 8 KV heads of 128).
//   warps 0-15    sums, four warps to a tile, each four with a quarter of TMEM (two tiles at once left them waiting for their
//                 own instructions)
//   warps 16-19   codes to MMA operands, a token per thread, ahead of their use
//   warp 20       issues the MMAs
constexpr int WT_TOK = 128, WT_ROWS = 32, WT_MOST = 128, WT_STAGES = 5, WT_SETS = 4;
constexpr int WT_SUM_WARPS = 4 * WT_SETS, WT_MMA_WARP = WT_SUM_WARPS + 4, WT_THREADS = 32 * (WT_MMA_WARP + 1);
constexpr int WT_MEET = 32 * (WT_SUM_WARPS + 1);   // threads that meet when the rows change
constexpr int WT_LEAD = 2;            // tiles that a head counts more, for its start

template <int HD>
struct WtSmem {
  static constexpr int TILE = WT_TOK * HD * 2, G = HD / 32;
  static constexpr int Q0 = WT_STAGES * TILE, SUMS = Q0 + WT_MOST * HD * 2;   // (sums of pairs of rows: [row / 2][G] float2)
  static constexpr int SCALE = SUMS + WT_MOST * G * 4, SPAN = SCALE + WT_MOST * 8, PRE = SPAN + WT_MOST * 8;
  static constexpr int bytes(int batch) { return PRE + 4 * (2 * batch + 1) + 1024; }   // (1024: to the swizzle's boundary)
};

// Rows r0.. (rn of them, WT_MOST at most; further ones are added to what the first ones left) of a (sequence, KV head) into shared
// memory, two (HD 64: four) per warp at a time: HD / 8 lanes hold a row
template <int HD>
__device__ __forceinline__ void wt_rows(const PwArgs& a, int b, int g, int r0, int rn, int n, unsigned char* sm) {
  using S = WtSmem<HD>;
  constexpr int CH = HD / 8, PER = 32 / CH;
  const int lane = threadIdx.x & 31, c = lane % CH;
  for (int x = (threadIdx.x >> 5) * PER + lane / CH; x < WT_MOST; x += WT_SUM_WARPS * PER) {
    const int r = r0 + x, i = x < rn ? r / a.n_rep : 0, h = g * a.n_rep + (x < rn ? r - i * a.n_rep : 0);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (x < rn) v = *reinterpret_cast<const uint4*>(static_cast<const unsigned short*>(a.q) + ((long long)b * a.Q + i) * a.qt + h * a.qh + 8 * c);
    float f[8], mx = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 p = pair_to_f2(word_of(v, k), a.bf16);
      f[2 * k] = p.x, f[2 * k + 1] = p.y;
      mx = fmaxf(mx, fmaxf(fabsf(p.x), fabsf(p.y)));
    }
#pragma unroll
    for (int o = 1; o < CH; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    int e = 0;   // as in pw_rows
    if (mx > 0.f) frexpf(mx, &e);
    e = max(-126, min(126, 10 - e));
    const float up = a.scale_log2 < 0.f ? -ldexpf(1.f, e) : ldexpf(1.f, e), upl = up * 0.0625f;
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = fmaf(f[k], up, sum);
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    // channels 0, 4, 1, 5, ...: as the codes come; odd ones meet 16 times their codes
    *reinterpret_cast<uint4*>(sm + S::Q0 + tc_place(WT_MOST, x, c)) =
        make_uint4(h2_as_u32(__floats2half2_rn(f[0] * up, f[4] * up)), h2_as_u32(__floats2half2_rn(f[1] * upl, f[5] * upl)),
                   h2_as_u32(__floats2half2_rn(f[2] * up, f[6] * up)), h2_as_u32(__floats2half2_rn(f[3] * upl, f[7] * upl)));
    if (c % 4 == 0) reinterpret_cast<float*>(sm + S::SUMS)[((x / 2) * S::G + c / 4) * 2 + x % 2] = sum;
    if (c == 0) {
      const int hi = max(0, n - a.Q + 1 + i), lo = a.window ? max(0, hi - a.window) : 0;
      const float lse = x < rn ? a.lse[((long long)b * a.Q + i) * a.Hq + h] : 0.f;
      const bool counts = x < rn && (lse > -INFINITY || lse != lse);
      // [row / 2]: scales of two rows, then their log-sum-exps in base 2, negated
      float* sl = reinterpret_cast<float*>(sm + S::SCALE) + (x / 2) * 4 + x % 2;
      sl[0] = counts ? fminf(fmaxf(ldexpf(fabsf(a.scale_log2), -e), 1.17549435e-38f), 3.402823466e38f) : 0.f;
      sl[2] = counts ? -lse * LOG2E_F : -INFINITY;
      int* span = reinterpret_cast<int*>(sm + S::SPAN) + (x / 2) * 4 + x % 2;
      span[0] = counts ? lo : 0, span[2] = counts ? hi : 0;
    }
  }
}

template <int HD>
__global__ void __launch_bounds__(WT_THREADS, 1) paged_weights_rows_kernel(PwArgs a) {
  using L = Page<HD>;
  using S = WtSmem<HD>;
  constexpr int G = L::G;
  constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u, TMEM = WT_SETS * WT_ROWS * G;
  extern __shared__ unsigned char raw_smem[];
  unsigned char* sm = raw_smem + (1024 - (tc_smem(raw_smem) & 1023)) % 1024;
  int* pre = reinterpret_cast<int*>(sm + S::PRE);   // [B + 1] positions before each sequence, of one KV head
  int* lens = pre + a.B + 1;                        // [B]
  __shared__ __align__(8) unsigned long long bars[2 * WT_STAGES + 2 * WT_SETS + 1];
  __shared__ uint32_t tmem_at;
  __shared__ int failed_at;
  volatile int* failed = &failed_at;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t bar0 = __shfl_sync(0xffffffffu, tc_smem(bars), 0);
  const uint32_t full = bar0, empty = bar0 + 8 * WT_STAGES, d_full = empty + 8 * WT_STAGES, d_empty = d_full + 8 * WT_SETS, done = d_empty + 8 * WT_SETS;
  if (threadIdx.x == 0) {
    auto init = [&](uint32_t bar, int count) { asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory"); };
    for (int k = 0; k < WT_STAGES; ++k) init(full + 8 * k, 128), init(empty + 8 * k, 1);
    for (int k = 0; k < WT_SETS; ++k) init(d_full + 8 * k, 1), init(d_empty + 8 * k, 128);
    init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    failed_at = 0;
  }
  if (warp == WT_MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(tc_smem(&tmem_at)), "r"(TMEM) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_trigger();
  pdl_wait();
  if (warp == 0) {
    int run = 0;
    if (lane == 0) pre[0] = 0;
    for (int base = 0; base < a.B; base += 32) {
      const int b = base + lane, len = b < a.B ? pw_len(a, b) : 0, cols = min(len, a.columns);
      int inc = cols ? (cols + WT_TOK - 1) / WT_TOK + WT_LEAD : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (b < a.B) lens[b] = len, pre[b + 1] = run + inc;
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_at, 0);
  const long long total = (long long)pre[a.B] * a.Hkv;
  const long long x1 = quotient((blockIdx.x + 1) * total, gridDim.x);
  // ---- the walk over this CTA's parts of (sequence, KV head)s and their chunks of rows, the same in every role ----
  long long x = quotient(blockIdx.x * total, gridDim.x);
  int b = 0, g = 0, tile0 = 0, tiles = 0, n = 0, r0 = 0, rn = 0;
  for (int b1 = a.B; b1 - b > 1;) {   // the last sequence that starts at x or before
    const int m = (b + b1) / 2;
    if ((long long)pre[m] * a.Hkv <= x) b = m; else b1 = m;
  }
  r0 = a.rows;   // (as behind the last chunk)
  auto next = [&]() {   // the next chunk of rows, or the first of the next part; false: there is none
    r0 += WT_MOST;
    while (r0 >= a.rows) {
      if (x >= x1) return false;
      while ((long long)pre[b + 1] * a.Hkv <= x) ++b;
      const int np = pre[b + 1] - pre[b];
      const long long in = x - (long long)pre[b] * a.Hkv;
      g = (int)quotient(in, np);
      const int at = (int)(in - (long long)g * np), taken = (int)min((long long)(np - at), x1 - x);
      tile0 = max(0, at - WT_LEAD), tiles = max(0, at + taken - WT_LEAD) - tile0;
      n = lens[b], x += taken;
      if (tiles) r0 = 0;
    }
    rn = min(WT_MOST, a.rows - r0);
    return true;
  };
  // the page of token `tok` (-1: not seen by any query, or in no page of the pool)
  const int q_first = a.window ? a.Q - 1 + a.window : 0;   // tokens before n - q_first no query sees
  auto page_of = [&](int tok) {
    if (tok >= n || (a.window && (tok / PG + 1) * PG <= n - q_first)) return -1;
    const int page = a.table[b * a.table_stride + tok / PG];
    return page >= 0 && page < a.n_pages ? page : -1;
  };

  if (warp < WT_SUM_WARPS) {
    // ---- sums ----
    const int w = warp >> 2, t = threadIdx.x & 127;
    const uint32_t dp = tmem + ((uint32_t)(warp & 3) << 21) + WT_ROWS * G * w;
    uint32_t par = 0;
    while (next()) {
      asm volatile("bar.sync 1, %0;" :: "n"(WT_MEET) : "memory");   // everybody is done with the last rows
      wt_rows<HD>(a, b, g, r0, rn, n, sm);
      tc_proxy();
      asm volatile("bar.sync 1, %0;" :: "n"(WT_MEET) : "memory");
      const int blocks = (rn + WT_ROWS - 1) / WT_ROWS;
      // whether some row counts nothing: what it holds may be NaN, so that all tiles are masked by the rows' spans
      bool silent = false;
      for (int x = lane; x < rn; x += 32) silent |= reinterpret_cast<const float*>(sm + S::SCALE)[(x / 2) * 4 + x % 2] == 0.f;
      silent = __any_sync(0xffffffffu, silent);
      // what a tile's token brings, on its way while the tile before is summed up, its page's number one tile earlier
      struct Held {
        uint32_t s[G / 2], o[G / 2];
        float old;
      };
      auto fetch = [&](int tok, int page) {
        Held x;
        x.old = (r0 || a.decay != 0.f) && tok < min(n, a.columns) ? a.weights[b * a.ws + g * a.wh + tok] : 0.f;   // (decay 0 does not read it)
        const unsigned char* pg = a.pages + ((size_t)max(page, 0) * a.Hkv + g) * L::BYTES + (tok % PG) * 2 * G;
#pragma unroll
        for (int k = 0; k < G / 2; ++k) {
          x.s[k] = page >= 0 ? *reinterpret_cast<const uint32_t*>(pg + L::KS + 4 * k) : 0u;
          x.o[k] = page >= 0 ? *reinterpret_cast<const uint32_t*>(pg + L::KO + 4 * k) : 0u;
        }
        return x;
      };
      int tok = (tile0 + w) * WT_TOK + t, page = page_of(tok), page1 = page_of(tok + WT_SETS * WT_TOK);
      Held held = fetch(tok, page);
      for (int k = w; k < tiles; k += WT_SETS) {
        const int tok0 = tok - t;
        float s[G], o[G];
#pragma unroll
        for (int k = 0; k < G; k += 2) {
          const float2 x = __half22float2(u32_as_h2(held.s[k / 2])), y = __half22float2(u32_as_h2(held.o[k / 2]));
          s[k] = x.x * NIB_ROW_SCALE_LO, s[k + 1] = x.y * NIB_ROW_SCALE_LO, o[k] = y.x, o[k + 1] = y.y;
        }
        const float old = held.old;
        held = fetch(tok + WT_SETS * WT_TOK, page1);
        const int page2 = page_of(tok + 2 * WT_SETS * WT_TOK);
        const bool edge = silent || tok0 + WT_TOK > n - a.Q + 1 || (a.window && tok0 < n - a.window);   // some row does not see all of it
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        for (int block = 0; block < blocks; ++block) {
          tc_wait(d_full + 8 * w, par, failed);
          par ^= 1;
          tc_after();
          // eight rows at a time
#pragma unroll 1
          for (int c = 0; c < WT_ROWS / 8; ++c) {
            uint32_t v[G][8];
#pragma unroll
            for (int j = 0; j < G; ++j) tc_ld8(v[j], dp + WT_ROWS * j + 8 * c);
#pragma unroll
            for (int j = 0; j < G; ++j) tc_wait_ld(v[j]);
            if (c + 1 == WT_ROWS / 8) {
              tc_before();
              tc_arrive(d_empty + 8 * w);
            }
            const int pair0 = (block * WT_ROWS + 8 * c) / 2;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float2 r = make_float2(0.f, 0.f), y = r;   // offsets' part, codes' part
#pragma unroll
              for (int j = 0; j < G; j += 2) {
                const float4 q = *reinterpret_cast<const float4*>(sm + S::SUMS + ((pair0 + k) * G + j) * 8);
                r = fma2(make_float2(q.x, q.y), make_float2(o[j], o[j]), r);
                r = fma2(make_float2(q.z, q.w), make_float2(o[j + 1], o[j + 1]), r);
              }
#pragma unroll
              for (int j = 0; j < G; ++j)
                y = fma2(make_float2(__uint_as_float(v[j][2 * k]), __uint_as_float(v[j][2 * k + 1])), make_float2(s[j], s[j]), y);
              const float4 sl = reinterpret_cast<const float4*>(sm + S::SCALE)[pair0 + k];
              const float2 e = fma2(add2(r, y), make_float2(sl.x, sl.y), make_float2(sl.z, sl.w));
              float2 p = make_float2(exp2_approx(e.x), exp2_approx(e.y));
              if (edge) {
                const int4 span = reinterpret_cast<const int4*>(sm + S::SPAN)[pair0 + k];   // lo, lo, hi, hi
                p = make_float2(tok >= span.x && tok < span.z ? p.x : 0.f, tok >= span.y && tok < span.w ? p.y : 0.f);
              }
              sum[k % 2] = add2(sum[k % 2], p);
            }
          }
        }
        const float all = *failed ? __int_as_float(0x7fc00000) : page >= 0 ? (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y) : 0.f;
        if (tok < min(n, a.columns)) a.weights[b * a.ws + g * a.wh + tok] = r0 ? old + all : a.decay == 0.f ? all : fmaf(old, a.decay, all);
        tok += WT_SETS * WT_TOK, page = page1, page1 = page2;
      }
    }
  } else if (warp < WT_MMA_WARP) {
    // ---- codes ----
    constexpr int W4 = HD / 32;   // 16-byte pieces of a token's codes
    const int t = threadIdx.x & 127;
    uint32_t stage = 0, par = 1;
    struct Held {
      uint4 code[W4];
    };
    auto fetch = [&](int tok, int page) {
      Held x;
      const unsigned char* pg = a.pages + ((size_t)max(page, 0) * a.Hkv + g) * L::BYTES + (tok % PG) * L::ROW;
#pragma unroll
      for (int i = 0; i < W4; ++i) x.code[i] = page >= 0 ? *reinterpret_cast<const uint4*>(pg + 16 * i) : make_uint4(0, 0, 0, 0);
      return x;
    };
    while (next()) {
      // the next tile's codes on their way while this one's are masked, its page's number one tile earlier
      int tok = tile0 * WT_TOK + t, page = page_of(tok + WT_TOK);
      Held held = fetch(tok, page_of(tok));
      for (int k = 0; k < tiles; ++k, tok += WT_TOK) {
        const Held x = held;
        held = fetch(tok + WT_TOK, page);
        page = page_of(tok + 2 * WT_TOK);
        tc_wait(empty + 8 * stage, par, failed);
        unsigned char* to = sm + stage * S::TILE;
#pragma unroll
        for (int i = 0; i < W4; ++i)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t c = word_of(x.code[i], y);   // word G a + g: channels 32g + 8a .. + 7, piece 4g + a
            const int word = 4 * i + y;
            *reinterpret_cast<uint4*>(to + tc_place(WT_TOK, t, 4 * (word % G) + word / G)) = make_uint4(c & LO, c & HI, (c >> 8) & LO, (c >> 8) & HI);
          }
        tc_proxy();
        tc_arrive(full + 8 * stage);
        if (++stage == WT_STAGES) stage = 0, par ^= 1;
      }
    }
  } else {
    // ---- MMAs ----
    const uint32_t base = __shfl_sync(0xffffffffu, tc_smem(sm), 0);
    const bool leader = tc_elect();
    uint32_t used = 0, d_par = (1u << WT_SETS) - 1;   // tiles; bit w: parity of the wait for a set's accumulators
    while (next()) {
      asm volatile("bar.sync 1, %0;" :: "n"(WT_MEET) : "memory");
      asm volatile("bar.sync 1, %0;" :: "n"(WT_MEET) : "memory");
      tc_after();
      const uint32_t blocks = __shfl_sync(0xffffffffu, (rn + WT_ROWS - 1) / WT_ROWS, 0), count = __shfl_sync(0xffffffffu, tiles, 0);
      for (uint32_t k0 = 0; k0 < count; k0 += WT_SETS) {   // the sets' tiles in turn
        const uint32_t sets = min((uint32_t)WT_SETS, count - k0);
        for (uint32_t block = 0; block < blocks; ++block)
#pragma unroll 1
          for (uint32_t w = 0; w < sets; ++w) {
            const uint32_t stage = (used + w) % WT_STAGES;
            if (block == 0) tc_wait(full + 8 * stage, ((used + w) / WT_STAGES) & 1u, failed);
            tc_wait(d_empty + 8 * w, (d_par >> w) & 1u, failed);
            d_par ^= 1u << w;
            tc_after();
#pragma unroll
            for (int k = 0; k < 2 * G; ++k) {   // 16 channels each
              const uint32_t at = (k / 4) * WT_TOK * 128 + (k % 4) * 32, qt = (k / 4) * WT_MOST * 128 + (k % 4) * 32;
              tc_mma_ss<tc_idesc(WT_ROWS, false)>(tmem + WT_ROWS * (G * w + k / 2), tc_desc(base + stage * S::TILE + at, 16),
                                                  tc_desc(base + S::Q0 + block * WT_ROWS * 128 + qt, 16), k % 2 > 0, leader);
            }
            tc_commit(d_full + 8 * w, leader);
            if (block + 1 == blocks) tc_commit(empty + 8 * stage, leader);
          }
        used += sets;
      }
    }
    // nothing of this CTA's is in flight any more when it gives its TMEM back, also behind a wait that ran out
    tc_commit(done, leader);
    for (const unsigned long long t = tc_ns(); !tc_try(done, 0) && tc_ns() - t < TC_WAIT_NS;) {}
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == WT_MMA_WARP)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(TMEM) : "memory");
}

template <int HD>
cudaError_t pw_launch(const PwArgs& a, int sms, cudaStream_t st) {
  auto bytes = [](int batch) {
    return PW_WARPS * PW_STAGES * PwStage<HD>::BYTES + PW_TILES * (int)sizeof(PwTile<HD>) + 4 * (2 * batch + 1);
  };
  auto* k = paged_weights_kernel<HD>;
  // the limit belongs to the function and is every host thread's: always the one of the largest batch
  if (cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(PW_MAX_BATCH))) return e;
  // one CTA per SM, fewer when the table cannot hold a page for each
  return launch_dependent(k, dim3((unsigned)std::min<long long>(sms, (long long)a.B * a.max_pages * a.Hkv)), dim3(PW_THREADS), bytes(a.B), st, a);
}

template <int HD>
cudaError_t wt_launch(const PwArgs& a, int sms, cudaStream_t st) {
  auto* k = paged_weights_rows_kernel<HD>;
  if (cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, WtSmem<HD>::bytes(PW_MAX_BATCH))) return e;
  return launch_dependent(k, dim3((unsigned)std::min<long long>(sms, (long long)a.B * a.max_pages * a.Hkv)), dim3(WT_THREADS), WtSmem<HD>::bytes(a.B), st, a);
}

const char* pw_shape_error(int B, int Q, int Hq, int Hkv, int hd) {
  if (B < 0 || B > 2048) return "batch must be in 0..2048";
  if (Q < 1 || Q > 64) return "n_q_tokens must be in 1..64";
  if (Hkv < 1 || Hkv > MAX_KV_HEADS) return "n_kv_heads must be in 1..4096";
  if (Hq < 1 || Hq % Hkv != 0 || Hq / Hkv > 64) return "n_q_heads / n_kv_heads must be an integer in 1..64";
  if (hd != 64 && hd != 128) return "head_dim must be 64 or 128";
  return nullptr;
}

kvq_status weights_impl(int dtype, const void* q, int64_t qt, int64_t qh, const float* lse, const void* pages, int n_pages,
                        const int32_t* table, int64_t table_stride, int max_pages, const int32_t* lens, int B, int Q, int Hq, int Hkv,
                        int hd, int window, float scale, float decay, float* weights, int64_t ws, int64_t wh, int columns,
                        void* stream) {
  const char* fn = "kvq_paged_weights";
  auto bad = [&](const char* what) { return paged_fail(KVQ_ERR_INVALID, fn, what); };
  if (dtype != KVQ_F16 && dtype != KVQ_BF16) return bad("dtype must be KVQ_F16 or KVQ_BF16");
  if (const char* msg = pw_shape_error(B, Q, Hq, Hkv, hd)) return bad(msg);
  if (n_pages < 1 || n_pages > (1 << 25)) return bad("n_pages must be in 1..33554432");
  if (max_pages < 1 || max_pages > (1 << 24) || (long long)B * max_pages >= (1ll << 30))
    return bad("max_pages must be in 1..16777216 and batch * max_pages below 2^30");
  if (table_stride < 0) return bad("table_stride must be >= 0");
  if (window < 0) return bad("window must be >= 0");
  if (columns < 1) return bad("weights need a column at least");
  const float scale_log2 = (scale != 0.f ? scale : 1.f / std::sqrt((float)hd)) * LOG2E_F;
  if (!std::isfinite(scale_log2)) return bad("scale * log2(e) must be finite");
  if (!std::isfinite(decay)) return bad("decay must be finite");
  if (B == 0) return KVQ_OK;
  if (kvq_status s = check_strides(qt, qh, fn, "q")) return s;
  if (ws < 0 || wh < 0 || rows_overlap(B, Hkv, ws, wh, columns)) return bad("weights: rows must not overlap");
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return paged_cuda_fail(e, fn, "no current CUDA device");
  if (kvq_status s = check_buffer(q, dev, 16, fn, "q")) return s;
  if (kvq_status s = check_buffer(lse, dev, 4, fn, "lse")) return s;
  if (kvq_status s = check_buffer(pages, dev, 16, fn, "pages")) return s;
  if (kvq_status s = check_buffer(table, dev, 4, fn, "page_table")) return s;
  if (kvq_status s = check_buffer(lens, dev, 4, fn, "seq_lens")) return s;
  if (kvq_status s = check_buffer(weights, dev, 4, fn, "weights")) return s;
  PwArgs a = {};
  a.q = q, a.lse = lse, a.pages = static_cast<const unsigned char*>(pages), a.table = table, a.lens = lens, a.weights = weights;
  a.qt = qt, a.qh = qh, a.table_stride = table_stride, a.ws = ws, a.wh = wh;
  a.n_pages = n_pages, a.max_pages = max_pages, a.columns = columns;
  a.B = B, a.Q = Q, a.Hq = Hq, a.Hkv = Hkv, a.n_rep = Hq / Hkv, a.rows = Q * a.n_rep, a.RT = (a.rows + PW_ROWS - 1) / PW_ROWS;
  a.window = std::min(window, 1 << 30);
  a.scale_log2 = scale_log2, a.decay = decay, a.bf16 = dtype == KVQ_BF16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int sms = 0;
  if (cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) return paged_cuda_fail(e, fn, "device attributes");
  const cudaError_t e = a.rows >= WT_FROM ? (hd == 128 ? wt_launch<128>(a, sms, st) : wt_launch<64>(a, sms, st))
                                          : (hd == 128 ? pw_launch<128>(a, sms, st) : pw_launch<64>(a, sms, st));
  if (e != cudaSuccess) return paged_cuda_fail(e, fn, "launch");
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

extern "C" kvq_status kvq_paged_weights(int dtype, const void* q, int64_t q_token_stride, int64_t q_head_stride, const float* lse,
                                        const void* pages, int n_pages, const int32_t* page_table, int64_t table_stride,
                                        int max_pages, const int32_t* seq_lens, int batch, int n_q_tokens, int n_q_heads,
                                        int n_kv_heads, int head_dim, int window, float scale, float decay, float* weights,
                                        int64_t weights_seq_stride, int64_t weights_head_stride, int n_columns, void* stream) try {
  return kvq::weights_impl(dtype, q, q_token_stride, q_head_stride, lse, pages, n_pages, page_table, table_stride, max_pages,
                           seq_lens, batch, n_q_tokens, n_q_heads, n_kv_heads, head_dim, window, scale, decay, weights,
                           weights_seq_stride, weights_head_stride, n_columns, stream);
} catch (...) {
  return KVQ_ERR_HOST_OOM;
}
