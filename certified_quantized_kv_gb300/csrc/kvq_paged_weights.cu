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
// SM, whatever the lengths (each head counts PW_LEAD pages more, for its start).  For each (sequence, KV head) of its range a CTA brings up to 128 query rows to binary16 in
// shared memory, in the order in which lanes take them (times a power of two per row, as in the attention); each warp
// then takes whole pages, which bulk copies bring into a ring of its own two ahead, across the heads' borders too: half
// a page's codes are masked into MMA operands once, and the rows' tiles pass by.  Further rows are added to what the
// first ones left.  Every sum has one owner and a fixed order.
#include <algorithm>
#include <cmath>
#include <string>

#include "kvq.h"
#include "kvq_launch.h"
#include "kvq_paged.cuh"

namespace kvq {

namespace {

constexpr int PW_ROWS = 8;            // query rows of a tile (MMA columns)
constexpr int PW_TILES = 16;          // tiles in shared memory at once
constexpr int PW_THREADS = 512, PW_WARPS = PW_THREADS / 32, PW_MAX_BATCH = 2048;
// Positions that a (sequence, KV head) takes in the ranges besides its pages, for what starting it costs in pages' time
constexpr int PW_LEAD = 3;
constexpr int PW_STAGES = 2;          // pages on their way per warp
constexpr unsigned long long PW_WAIT_NS = 2000000000ull;   // bounded waits: 2 s

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

// Tile `rt` of a (sequence, KV head), by one warp: lane (gid, tig) holds the channels 32k + 8 tig .. + 7 of row gid.
template <int HD>
__device__ __forceinline__ void pw_rows(const PwArgs& a, int b, int g, int rt, int n, PwTile<HD>& out) {
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
  if (tig == 0) {
    const int hi = max(0, n - a.Q + 1 + i), lo = a.window ? max(0, hi - a.window) : 0;
    const float lse = live ? a.lse[((long long)b * a.Q + i) * a.Hq + h] : 0.f;
    // a row that sees nothing (lse -inf) counts nothing
    const bool counts = live && lse > -INFINITY || lse != lse;
    out.scale[gid] = counts ? fminf(fmaxf(ldexpf(fabsf(a.scale_log2), -e), 1.17549435e-38f), 3.402823466e38f) : 0.f;
    out.lse[gid] = counts ? lse * LOG2E_F : INFINITY;
    out.lo[gid] = counts ? lo : 0, out.hi[gid] = counts ? hi : 0;
  }
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
  constexpr int STEP = 1;   // tiles of 16 tokens at once
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
  const int chunks = (a.RT + PW_TILES - 1) / PW_TILES;

  // ---- copies, two pages ahead of their use: parts, then chunks of rows, then this warp's pages ----
  Part ahead = part_at(x0, b0);
  int at_chunk = 0, at_page = ahead.warp0, issued = 0, found = -1;
  bool failed = false, more = true;
  uint32_t valid = 0;   // bit k: stage k holds a page that is seen
  auto look = [&]() {   // the number of the walk's page (-1: none that is seen)
    while (at_page >= ahead.pages) {
      at_page = ahead.warp0;
      if (++at_chunk < chunks) continue;
      at_chunk = 0;
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
  const int batch = max(1, PW_TILES / a.RT);
  int used = 0;
  for (Part first = part_at(x0, b0);;) {
    Part behind = first;   // the part behind the batch
    int parts = 0;
    bool end = false;
    for (int rt0 = 0; rt0 < a.RT; rt0 += PW_TILES) {
      const int nt = min(PW_TILES, a.RT - rt0);
      __syncthreads();   // the tiles' last readers are done
      behind = first;
      for (parts = 0; parts < batch; ++parts) {
        // tile k of part y is number y nt + k, one warp's each
        for (int k = (warp + PW_WARPS - parts * nt % PW_WARPS) % PW_WARPS; k < nt; k += PW_WARPS)
          pw_rows<HD>(a, behind.b, behind.g, rt0 + k, behind.n, tiles[parts * nt + k]);
        if (behind.end >= x1) {
          ++parts, end = true;
          break;
        }
        behind = part_at(behind.end, behind.b);
      }
      __syncthreads();
      Part p = first;
      for (int y = 0; y < parts; ++y) {
        if (y) p = part_at(p.end, p.b);
        const int n = p.n, cols = min(n, a.columns);
        for (int page = p.warp0; page < p.pages; page += PW_WARPS) {
          const int tok0 = (p.page0 + page) * PG;
          float* w = a.weights + p.b * a.ws + p.g * a.wh + tok0;
          // what is there of this lane's tokens (decay 0 does not read it)
          float old[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) old[k] = (rt0 || a.decay != 0.f) && tok0 + 32 * k + 8 * tig + gid < cols ? w[32 * k + 8 * tig + gid] : 0.f;
          const int stage = ring_stage<PW_STAGES>(used);
          const unsigned char* pg = ring + stage * St::BYTES;
          const uint32_t parity = ring_parity<PW_STAGES>(used);
          ++used;
          if (!failed && !pw_try(bar_s + 8 * stage, parity)) failed = !pw_wait_slow(bar_s + 8 * stage, parity);
          failed = __any_sync(0xffffffffu, failed);
          const bool seen = (valid >> stage) & 1u;
          // whether some row does not see all of the page
          const bool edge = tok0 + PG > n - a.Q + 1 || (a.window && tok0 < n - a.window);
          float mine[8];   // sums of tokens 8k + gid
#pragma unroll
          for (int i0 = 0; i0 < 4; i0 += STEP) {
            float2 sum[STEP][2];   // tokens gid and gid + 8 of a tile; the even and the odd columns
#pragma unroll
            for (int i = 0; i < STEP; ++i) sum[i][0] = sum[i][1] = make_float2(0.f, 0.f);
            if (seen) {
              uint32_t low[STEP][G][4], high[STEP][G][4], off[STEP][2];
              float sc[STEP][2][G];
#pragma unroll
              for (int i = 0; i < STEP; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int t = 16 * (i0 + i) + 8 * k + gid;
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
                  off[i][k] = *reinterpret_cast<const uint32_t*>(pg + St::KO + t * 2 * G + 4 * (tig % (G / 2)));
#pragma unroll
                  for (int g = 0; g < G; ++g) {
                    low[i][g][k] = c[g] & LO, low[i][g][2 + k] = (c[g] >> 8) & LO;
                    high[i][g][k] = c[g] & HI, high[i][g][2 + k] = (c[g] >> 8) & HI;
                    const float2 f = __half22float2(u32_as_h2(h[g / 2]));
                    sc[i][k][g] = g & 1 ? f.y : f.x;
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
#pragma unroll
                for (int i = 0; i < STEP; ++i) {
                  float2 r[2];   // of the tile's two tokens, two columns each
#pragma unroll
                  for (int g = 0; g < G; ++g) {
                    float X[4];
                    pw_mma_z(X, low[i][g], q[g].x, q[g].y);
                    pw_mma(X, high[i][g], q[g].z, q[g].w);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                      const float2 x = make_float2(X[2 * k], X[2 * k + 1]), f = make_float2(sc[i][k][g], sc[i][k][g]);
                      r[k] = g == 0 ? mul2(x, f) : fma2(x, f, r[k]);
                    }
                  }
                  float O[4];
                  pw_mma_k8_z(O, off[i][0], off[i][1], qo);
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    const float2 s = fma2(r[k], make_float2(NIB_ROW_SCALE_LO, NIB_ROW_SCALE_LO), make_float2(O[2 * k], O[2 * k + 1]));
                    const float2 e = fma2(s, scale, minus);
                    float2 pr = make_float2(exp2_approx(e.x), exp2_approx(e.y));
                    if (edge) {
                      const int t = tok0 + 16 * (i0 + i) + 8 * k + gid;
                      const int2 lo = *reinterpret_cast<const int2*>(T.lo + 2 * tig), hi = *reinterpret_cast<const int2*>(T.hi + 2 * tig);
                      pr = make_float2(t >= lo.x && t < hi.x ? pr.x : 0.f, t >= lo.y && t < hi.y ? pr.y : 0.f);
                    }
                    sum[i][k] = add2(sum[i][k], pr);
                  }
                }
              }
            }
#pragma unroll
            for (int i = 0; i < STEP; ++i)
#pragma unroll
              for (int k = 0; k < 2; ++k) mine[2 * (i0 + i) + k] = sum[i][k].x + sum[i][k].y;
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
            if (tok0 + t < cols) w[t] = rt0 ? old[k] + x : a.decay == 0.f ? x : fmaf(old[k], a.decay, x);
          }
          __syncwarp();   // the stage's last readers are done
          if (!failed && more) issue();
        }
      }
    }
    if (end) break;
    first = behind;
  }
  if (failed) ring_drain<PW_STAGES>(issued, [&](int k, uint32_t parity) { pw_wait_slow(bar_s + 8 * k, parity); });
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
  const cudaError_t e = hd == 128 ? pw_launch<128>(a, sms, st) : pw_launch<64>(a, sms, st);
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
