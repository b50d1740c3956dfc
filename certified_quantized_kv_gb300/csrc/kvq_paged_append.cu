// kvq_paged_append.cu -- tokens into the pages of the 4-bit cache (with the rotation of
// keys and queries on the way), and back out of them.
//
// Per token, KV head and group of 32 channels (x the rotated key or the value, in fp32):
//   s = fp16 rounded up of (max - min) / 15, o = fp16(min), code = clamp(rint((x - o) / s), 0, 15)
// and for the values of odd slots, counted down from the maximum,
//   s = -(fp16 rounded up of (max - min) / 15), o = fp16(max), code = clamp(rint((o - x) / |s|), 0, 15)
// so x^ = o + s code in both.  The scale is rounded up so that 15 steps span the group.
#include <algorithm>
#include <string>

#include "kvq.h"
#include "kvq_launch.h"
#include "kvq_paged.cuh"
#include "kvq_rope.cuh"

namespace kvq {

namespace {

struct AppendPagedArgs {
  const void *k, *v;
  const int32_t *slots, *pos;
  unsigned char* pages;
  long long kt, kh, vt, vh;   // strides in elements
  int T, Hkv, n_pages, per;   // per: KV heads of one item
  int kv_blocks;              // the other blocks turn q
  RopeArgs q;
};

constexpr int E = 4;   // neighbouring elements of a row that a lane holds
struct Quad {
  uint32_t w[2];
  __device__ __forceinline__ void load(const unsigned short* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
};

// Rotation of rows spread over HD / 4 lanes at one token's position.  The other element of a
// pair is in the same lane (INTERLEAVED), or a whole number of lanes away (LANES), or, when half of
// rotary_dim is no multiple of 4, anywhere (ELEMENTS).
enum class Turn { NONE, INTERLEAVED, LANES, ELEMENTS };
template <int HD, Turn TURN, bool BF16>
struct Rotation {
  int from[E], el[E];
  float c[E], s[E];  // y = x c + other s (s carries the sign; elements not rotated: 1, 0)
  __device__ __forceinline__ void set(const kvq_rope_plan& P, const uint64_t* steps, const int32_t* pos, int lane) {
    if (TURN == Turn::NONE) return;
    const int half = P.rotary_dim / 2, at = *pos, sub = lane % (HD / E);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int ch = E * sub + e;
      const bool in = ch < P.rotary_dim, second = TURN == Turn::INTERLEAVED ? (e & 1) : ch >= half;
      const int i = TURN == Turn::INTERLEAVED ? ch >> 1 : second ? ch - half : ch;
      const int other = !in ? ch : second ? ch - half : ch + half;
      from[e] = lane - sub + other / E, el[e] = other % E;
      float2 cs = make_float2(1.f, 0.f);
      if (TURN == Turn::INTERLEAVED && (e & 1)) cs = make_float2(c[e ^ 1], -s[e ^ 1]);
      else if (in) cs = rope_cos_sin(at, steps[i], P.magnitude);
      c[e] = cs.x;
      s[e] = second ? cs.y : -cs.y;
    }
  }
  __device__ __forceinline__ void apply(const Quad& r, float (&y)[E]) const {
    float x[E], o[E];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 p = pair_to_f2(r.w[k], BF16);
      x[2 * k] = p.x, x[2 * k + 1] = p.y;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = TURN == Turn::INTERLEAVED ? x[e ^ 1] : 0.f;
    if (TURN == Turn::LANES) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 p = pair_to_f2(__shfl_sync(0xffffffffu, r.w[k], from[0]), BF16);
        o[2 * k] = p.x, o[2 * k + 1] = p.y;
      }
    }
    if (TURN == Turn::ELEMENTS) {
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int k = 0; k < E; ++k) {
          const float v = __shfl_sync(0xffffffffu, x[k], from[e]);
          if (el[e] == k) o[e] = v;
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = TURN == Turn::NONE ? x[e] : fmaf(x[e], c[e], o[e] * s[e]);
  }
};

// minimum and maximum that are NaN when an operand is
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Extremes of a group (eight lanes) of fp32 elements, both NaN when an element is.
__device__ __forceinline__ float2 extremes(const float (&x)[E]) {
  float lo = min_nan(min_nan(x[0], x[1]), min_nan(x[2], x[3])), hi = max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3]));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  return make_float2(lo, hi);
}
// ... of 16-bit elements as they are: pairs (maximum, negated minimum), one shuffle a round
template <bool BF16>
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  if (BF16) {
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  return h2_as_u32(__hmax2_nan(u32_as_h2(a), u32_as_h2(b)));
}
template <bool BF16>
__device__ __forceinline__ float2 extremes(const Quad& r) {
  const uint32_t n0 = r.w[0] ^ 0x80008000u, n1 = r.w[1] ^ 0x80008000u;
  const uint32_t hi = max_pair<BF16>(r.w[0], r.w[1]), lo = max_pair<BF16>(n0, n1);
  uint32_t m = max_pair<BF16>(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = max_pair<BF16>(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float2 p = pair_to_f2(m, BF16);
  return make_float2(-p.y, p.x);
}

// Scale, offset and packed codes (4 bits each, from bit 0) of this lane's four elements of a
// group with extremes lo and hi.  The scale is the smallest binary16 h with 15 h >= the span (15 h
// is exact in fp32), which is the span / 15 rounded up.  Codes are rint(d / |s|) for the exact
// quotient: they come from a product with the reciprocal, and the remainder d - code s, exact
// near a half, tells where a neighbour is nearer, or as near and even (values on the binary16
// grid meet exact halves in about one element of a hundred).  The slow path also clamps the codes,
// which only elements beyond the rounded offset or the binary16 range need.  Extremes that are NaN
// make the offset NaN and the scale 0: the group then reads as NaN, whatever its codes.
__device__ __forceinline__ uint32_t quantize(const float (&x)[E], float2 ext, bool down, __half& sh, __half& oh) {
  constexpr float RND = 12582912.f;   // 1.5 2^23: adding it rounds to an integer, ties to even
  const float lo = min_nan(max_nan(ext.x, -65504.f), 65504.f), hi = min_nan(max_nan(ext.y, -65504.f), 65504.f);
  oh = __float2half_rn(down ? hi : lo);
  const float of = __half2float(oh), span = fmaxf(down ? of - lo : hi - of, 0.f);
  const float before = down ? ext.y - of : of - ext.x;   // how far the extreme lies before the offset,
  const float behind = (down ? of - ext.x : ext.y - of) - span;   // and the other one behind the span
  const unsigned short h = __half_as_ushort(__float2half_ru(span * 0.06666667f));
  const float sh1 = __half2float(__ushort_as_half(h)), sh0 = __half2float(__ushort_as_half((unsigned short)(h - 1)));
  const int step = 15.f * sh0 >= span ? -1 : 15.f * sh1 < span ? 1 : 0;   // (h = 0: sh0 is a NaN)
  sh = __ushort_as_half((unsigned short)(h + step));
  const float sa = __half2float(sh), s = down ? -sa : sa, half = 0.5f * sa;
  const float inv = sa > 0.f ? __fdividef(1.f, s) : 0.f;   // |s| lies in [2^-24, 2^14]
  const float2 rnd = make_float2(RND, RND);
  float2 t[2], r[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float2 d = sub2(make_float2(x[2 * k], x[2 * k + 1]), make_float2(of, of));
    t[k] = fma2(d, make_float2(inv, inv), rnd);   // bits: RND's plus the code
    r[k] = fma2(sub2(rnd, t[k]), make_float2(s, s), d);
  }
  const float worst = fmaxf(fmaxf(fabsf(r[0].x), fabsf(r[0].y)), fmaxf(fabsf(r[1].x), fabsf(r[1].y)));
  if (fmaxf(fmaxf(worst, before), behind) >= half) {
    auto fix = [&](float xe, float& te, float re) {
      const bool off = fabsf(re) > half || (fabsf(re) == half && (__float_as_uint(te) & 1u));
      const float to = off ? te + ((re < 0.f) == down ? 1.f : -1.f) : te;
      // beyond what the sum with RND holds as an integer, te is far from every code
      te = sa > 0.f ? fminf(fmaxf(to, RND), RND + 15.f) : RND;
    };
    fix(x[0], t[0].x, r[0].x), fix(x[1], t[0].y, r[0].y), fix(x[2], t[1].x, r[1].x), fix(x[3], t[1].y, r[1].y);
  }
  if (down) sh = __hneg(sh);
  // RND's bits lie above the codes' 16
  return __float_as_uint(t[0].x) + (__float_as_uint(t[0].y) << 4) + (__float_as_uint(t[1].x) << 8) + (__float_as_uint(t[1].y) << 12);
}

// One warp per item: a token's KV heads [h, h + a.per), one at a time at head_dim 128 and two at 64,
// with cos and sin formed once per item and the rows of two steps on their way at once.  The
// other blocks turn q, a thread per V pairs; the two kinds are spread over the grid in turn, since
// the first are bound by their arithmetic and the second by HBM.
constexpr int APPEND_THREADS = 128;
template <int HD, Turn TURN, int V, bool BF16>
__global__ void __launch_bounds__(APPEND_THREADS, 8) paged_append_kernel(const __grid_constant__ kvq_rope_plan P, AppendPagedArgs a) {
  using L = Page<HD>;
  constexpr int LANES = HD / E, HEADS = 32 / LANES, KU = 2;   // lanes of a row, heads of a step, steps at once
  constexpr int WARPS = APPEND_THREADS / 32;
  __shared__ __align__(16) uint64_t steps[128];
  pdl_trigger();
  if (TURN != Turn::NONE) load_steps(P, steps);
  pdl_wait();
  // block b is KV block number floor(b kv / all) when that number changes behind it
  const int k0 = (int)((long long)blockIdx.x * a.kv_blocks / gridDim.x), k1 = (int)((blockIdx.x + 1ll) * a.kv_blocks / gridDim.x);
  if (V > 0 && k0 == k1) {
    rope_part<V ? V : 1, TURN == Turn::INTERLEAVED, BF16, APPEND_THREADS, false>(P, steps, nullptr, a.q, (long long)(blockIdx.x - k0) * APPEND_THREADS,
                                                                          (long long)(gridDim.x - a.kv_blocks) * APPEND_THREADS);
    return;
  }
  const int lane = threadIdx.x & 31, sub = lane % LANES, hh = lane / LANES, g = sub / 8, j = sub % 8;
  const int items = (a.Hkv + a.per - 1) / a.per;
  const long long n = (long long)a.T * items;
  for (long long base = (long long)k0 * WARPS; base < n; base += (long long)a.kv_blocks * WARPS) {
    const long long u = base + (threadIdx.x >> 5), t = u / items;
    const int slot = u < n ? a.slots[t] : -1;
    if (slot < 0 || slot / PG >= a.n_pages) continue;
    const int at = slot % PG, h0 = (int)(u - t * items) * a.per, h1 = min(a.Hkv, h0 + a.per);
    const bool down = at & 1;
    const unsigned short* kp = static_cast<const unsigned short*>(a.k) + t * a.kt + (h0 + hh) * a.kh + E * sub;
    const unsigned short* vp = static_cast<const unsigned short*>(a.v) + t * a.vt + (h0 + hh) * a.vh + E * sub;
    // this lane's bytes of the codes, and its group's scale and offset (lane j = 0 writes)
    unsigned char* pg = a.pages + ((size_t)(slot / PG) * a.Hkv + h0 + hh) * L::BYTES;
    unsigned char* kc = pg + at * L::ROW + (j >> 1) * 4 * L::G + 4 * g + 2 * (j & 1);
    unsigned char* vc = pg + L::VC + vcode_at<HD>(at, j * 2 * L::G + 2 * g);
    __half* ks = reinterpret_cast<__half*>(pg + L::KS) + at * L::G + g;
    __half* vs = reinterpret_cast<__half*>(pg + L::VS) + g * PG + vscale_at(at);
    Rotation<HD, TURN, BF16> rot;
    for (int h = h0; h < h1; h += KU * HEADS) {   // (the same for the whole warp)
      Quad rk[KU], rv[KU];
#pragma unroll
      for (int k = 0; k < KU; ++k) {
        rk[k].w[0] = rk[k].w[1] = rv[k].w[0] = rv[k].w[1] = 0u;
        if (h + k * HEADS + hh < h1) {
          rk[k].load(kp);
          rv[k].load(vp);
          kp += HEADS * a.kh, vp += HEADS * a.vh;
        }
      }
      if (h == h0) rot.set(P, steps, a.pos + t, lane);
#pragma unroll
      for (int k = 0; k < KU; ++k) {
        if (h + k * HEADS >= h1) continue;
        const bool live = HEADS == 1 || h + k * HEADS + hh < h1;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          float x[E];
          float2 ext;
          if (kv || TURN == Turn::NONE) {
            const Quad& r = kv ? rv[k] : rk[k];
            ext = extremes<BF16>(r);
            const float2 p = pair_to_f2(r.w[0], BF16), q = pair_to_f2(r.w[1], BF16);
            x[0] = p.x, x[1] = p.y, x[2] = q.x, x[3] = q.y;
          } else {
            rot.apply(rk[k], x);
            ext = extremes(x);
          }
          __half s, o;
          const uint32_t code = quantize(x, ext, kv && down, s, o);
          if (live) {
            *reinterpret_cast<unsigned short*>((kv ? vc : kc) + k * HEADS * L::BYTES) = (unsigned short)code;
            if (j == 0) {
              __half* so = (kv ? vs : ks) + k * HEADS * (L::BYTES / 2);
              so[0] = s;
              so[L::SCALES / 2] = o;
            }
          }
        }
      }
      kc += KU * HEADS * L::BYTES, vc += KU * HEADS * L::BYTES, ks += KU * HEADS * L::BYTES / 2, vs += KU * HEADS * L::BYTES / 2;
    }
  }
}

template <int HD, bool BF16>
auto append_kernel_of(const kvq_rope_plan* plan, bool q) {
  using K = void (*)(kvq_rope_plan, AppendPagedArgs);
  if (!plan) return (K)paged_append_kernel<HD, Turn::NONE, 0, BF16>;
  const bool wide = q && rope_pairs(*plan) == 8;
  if (plan->interleaved)
    return wide ? (K)paged_append_kernel<HD, Turn::INTERLEAVED, 8, BF16> : (K)paged_append_kernel<HD, Turn::INTERLEAVED, 1, BF16>;
  if (plan->rotary_dim / 2 % E == 0)
    return wide ? (K)paged_append_kernel<HD, Turn::LANES, 8, BF16> : (K)paged_append_kernel<HD, Turn::LANES, 4, BF16>;
  return (K)paged_append_kernel<HD, Turn::ELEMENTS, 1, BF16>;
}

// Pairs per thread with which that kernel turns q.
int append_pairs(const kvq_rope_plan& plan) {
  const int V = rope_pairs(plan);
  return V == 8 || (V == 4 && !plan.interleaved) ? V : 1;
}

struct GatherArgs {
  const unsigned char* pages;
  const int32_t* slots;
  void *k, *v;
  long long kt, kh, vt, vh;
  int T, Hkv, n_pages, per;   // per: heads of one item
};

// One warp per item of a token's heads [h, h + a.per): half of the lanes read keys, half values, eight
// channels each (one 16-byte store); at head_dim 64 a warp takes two heads at once.  HBM bound.
constexpr int GATHER_THREADS = 128;
template <int HD, bool BF16>
__global__ void __launch_bounds__(GATHER_THREADS) paged_gather_kernel(GatherArgs a) {
  using L = Page<HD>;
  constexpr int LANES = HD / 8, HEADS = 32 / (2 * LANES), U = 4;   // lanes of a row, heads at once, steps on their way
  const int lane = threadIdx.x & 31, sub = lane % LANES, kv = (lane / LANES) & 1, hh = lane / (2 * LANES);
  const int g = sub / 4, piece = sub % 4;   // channels 32g + 8 piece
  const int items = (a.Hkv + a.per - 1) / a.per;
  const long long n = (long long)a.T * items;
  pdl_trigger();
  pdl_wait();
  for (long long u = blockIdx.x * (GATHER_THREADS / 32ll) + (threadIdx.x >> 5); u < n; u += gridDim.x * (GATHER_THREADS / 32ll)) {
    const long long t = u / items;
    const int h0 = (int)(u - t * items) * a.per, h1 = min(a.Hkv, h0 + a.per);
    const int slot = a.slots[t];
    const bool held = slot >= 0 && slot / PG < a.n_pages;
    const int at = held ? slot % PG : 0;
    const int h_ = h0 + hh;
    const unsigned char* pg = a.pages + ((held ? (size_t)(slot / PG) * a.Hkv : 0) + h_) * L::BYTES;
    const unsigned char* c0 = pg + (kv ? L::VC + vcode_at<HD>(at, 2 * piece * 2 * L::G + 2 * g) : at * L::ROW + piece * 4 * L::G + 4 * g);
    const unsigned char* c1 = kv ? pg + L::VC + vcode_at<HD>(at, (2 * piece + 1) * 2 * L::G + 2 * g) : c0 + 2;
    const __half* sc = reinterpret_cast<const __half*>(pg + (kv ? L::VS + 2 * (g * PG + vscale_at(at)) : L::KS + 2 * (at * L::G + g)));
    const long long step = HEADS * (kv ? a.vh : a.kh);
    unsigned short* out = static_cast<unsigned short*>(kv ? a.v : a.k) + t * (kv ? a.vt : a.kt) + h_ * (kv ? a.vh : a.kh) + 8 * sub;
    for (int h = h_; h < h1; h += U * HEADS) {
      uint32_t code[U];
      __half s[U], o[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        code[k] = 0u, s[k] = o[k] = __ushort_as_half(0);
        if (held && h + k * HEADS < h1) {
          constexpr int NEXT = HEADS * L::BYTES;
          code[k] = __byte_perm(*reinterpret_cast<const unsigned short*>(c0 + k * NEXT),
                                *reinterpret_cast<const unsigned short*>(c1 + k * NEXT), 0x5410);
          s[k] = sc[k * (NEXT / 2)];
          o[k] = sc[k * (NEXT / 2) + L::SCALES / 2];
        }
      }
      c0 += U * HEADS * L::BYTES, c1 += U * HEADS * L::BYTES, sc += U * HEADS * L::BYTES / 2;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (h + k * HEADS >= h1) continue;
        const float sf = __half2float(s[k]), of = __half2float(o[k]);
        uint32_t w[4];
        // 2^23 + code as a float's bits, less 2^23
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float n0 = __uint_as_float(((code[k] >> (8 * i)) & 15u) | 0x4B000000u) - 8388608.f;
          const float n1 = __uint_as_float(((code[k] >> (8 * i + 4)) & 15u) | 0x4B000000u) - 8388608.f;
          w[i] = f2_to_pair(fmaf(n0, sf, of), fmaf(n1, sf, of), BF16);
        }
        *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
        out += step;
      }
    }
  }
}

// Heads per item: few while the call does not fill the GPU, eight when it does.
int heads_per_item(long long T, int H) {
  return (int)std::min<long long>(8, std::max<long long>(1, T * H / (152 * 32)));   // 32 warps per SM
}

// checks shared by append and gather
kvq_status check_common(const char* fn, int dtype, int T, int Hkv, int hd, int n_pages) {
  if (dtype != KVQ_F16 && dtype != KVQ_BF16) return paged_fail(KVQ_ERR_INVALID, fn, "dtype must be KVQ_F16 or KVQ_BF16");
  if (hd != 64 && hd != 128) return paged_fail(KVQ_ERR_INVALID, fn, "head_dim must be 64 or 128");
  if (T < 0) return paged_fail(KVQ_ERR_INVALID, fn, "n_tokens must be >= 0");
  if (Hkv < 1 || Hkv > MAX_KV_HEADS) return paged_fail(KVQ_ERR_INVALID, fn, "n_kv_heads must be in 1..4096");
  if (n_pages < 1 || n_pages > (1 << 25))   // slots are int32
    return paged_fail(KVQ_ERR_INVALID, fn, "n_pages must be in 1..33554432");
  return KVQ_OK;
}

kvq_status append_impl(const kvq_rope_plan* plan, int dtype, const void* k, int64_t kt, int64_t kh, const void* v,
                       int64_t vt, int64_t vh, const int32_t* slots, const int32_t* positions, int T, int Hkv, int hd,
                       void* pages, int n_pages, const void* q, int64_t qt, int64_t qh, int Hq, void* q_out,
                       int64_t ot, int64_t oh, void* stream) {
  const char* fn = "kvq_paged_append";
  if (kvq_status s = check_common(fn, dtype, T, Hkv, hd, n_pages)) return s;
  if (plan) {
    if (kvq_status s = check_plan(plan, hd, fn)) return s;
    if (!positions) return paged_fail(KVQ_ERR_INVALID, fn, "positions is NULL with a plan");
  } else if (positions || q || q_out) {
    return paged_fail(KVQ_ERR_INVALID, fn, "positions, q and q_out need a plan");
  }
  if ((q == nullptr) != (q_out == nullptr)) return paged_fail(KVQ_ERR_INVALID, fn, "q and q_out go together");
  if (Hq < 0 || (q && Hq < 1)) return paged_fail(KVQ_ERR_INVALID, fn, "n_q_heads must be >= 1 with q");
  if (T == 0) return KVQ_OK;
  if (kvq_status s = check_strides(kt, kh, fn, "k")) return s;
  if (kvq_status s = check_strides(vt, vh, fn, "v")) return s;
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return paged_cuda_fail(e, fn, "no current CUDA device");
  if (kvq_status s = check_buffer(k, dev, 16, fn, "k")) return s;
  if (kvq_status s = check_buffer(v, dev, 16, fn, "v")) return s;
  if (kvq_status s = check_buffer(slots, dev, 4, fn, "slots")) return s;
  if (kvq_status s = check_buffer(pages, dev, 16, fn, "pages")) return s;
  if (plan)
    if (kvq_status s = check_buffer(positions, dev, 4, fn, "positions")) return s;
  if (q) {
    if (kvq_status s = check_strides(qt, qh, fn, "q")) return s;
    if (kvq_status s = check_strides(ot, oh, fn, "q_out")) return s;
    if ((T > 1 && ot == 0) || (Hq > 1 && oh == 0)) return paged_fail(KVQ_ERR_INVALID, fn, "q_out: rows must not overlap");
    if (q == q_out && ((T > 1 && qt != ot) || (Hq > 1 && qh != oh)))
      return paged_fail(KVQ_ERR_INVALID, fn, "q_out = q needs the same strides");
    if (kvq_status s = check_buffer(q, dev, 16, fn, "q")) return s;
    if (kvq_status s = check_buffer(q_out, dev, 16, fn, "q_out")) return s;
  }
  AppendPagedArgs a{k, v, slots, positions, static_cast<unsigned char*>(pages), kt, kh, vt, vh, T, Hkv, n_pages, heads_per_item(T, Hkv), 0, {}};
  const long long items = (long long)T * ((Hkv + a.per - 1) / a.per);
  long long blocks = std::min<long long>((items + APPEND_THREADS / 32 - 1) / (APPEND_THREADS / 32), 152 * 32);
  a.kv_blocks = (int)blocks;
  if (q) {
    const bool copy = q != q_out && plan->rotary_dim < hd;
    const int units = rope_units(*plan, append_pairs(*plan), copy);
    a.q = RopeArgs{q, q_out, positions, qt, qh, ot, oh, T, Hq, rope_lanes(T, Hq, units), copy};
    blocks += std::min<long long>(((long long)T * a.q.lanes * units + APPEND_THREADS - 1) / APPEND_THREADS, 152 * 32);
  }
  const bool bf16 = dtype == KVQ_BF16;
  auto* kern = hd == 128 ? (bf16 ? append_kernel_of<128, true>(plan, q) : append_kernel_of<128, false>(plan, q))
                         : (bf16 ? append_kernel_of<64, true>(plan, q) : append_kernel_of<64, false>(plan, q));
  kvq_rope_plan none = {};
  cudaError_t e = launch_dependent(kern, dim3((unsigned)blocks), dim3(APPEND_THREADS), 0, static_cast<cudaStream_t>(stream),
                                   plan ? *plan : none, a);
  if (e != cudaSuccess) return paged_cuda_fail(e, fn, "launch");
  return KVQ_OK;
}

kvq_status gather_impl(const void* pages, int n_pages, const int32_t* slots, int T, int Hkv, int hd, int dtype, void* k,
                       int64_t kt, int64_t kh, void* v, int64_t vt, int64_t vh, void* stream) {
  const char* fn = "kvq_paged_gather";
  if (kvq_status s = check_common(fn, dtype, T, Hkv, hd, n_pages)) return s;
  if (T == 0) return KVQ_OK;
  if (kvq_status s = check_strides(kt, kh, fn, "k")) return s;
  if (kvq_status s = check_strides(vt, vh, fn, "v")) return s;
  if ((T > 1 && (kt == 0 || vt == 0)) || (Hkv > 1 && (kh == 0 || vh == 0)))
    return paged_fail(KVQ_ERR_INVALID, fn, "k and v: rows must not overlap");
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return paged_cuda_fail(e, fn, "no current CUDA device");
  if (kvq_status s = check_buffer(pages, dev, 16, fn, "pages")) return s;
  if (kvq_status s = check_buffer(slots, dev, 4, fn, "slots")) return s;
  if (kvq_status s = check_buffer(k, dev, 16, fn, "k")) return s;
  if (kvq_status s = check_buffer(v, dev, 16, fn, "v")) return s;
  GatherArgs a{static_cast<const unsigned char*>(pages), slots, k, v, kt, kh, vt, vh, T, Hkv, n_pages, heads_per_item(T, Hkv)};
  const long long items = (long long)T * ((Hkv + a.per - 1) / a.per);
  const dim3 grid((unsigned)std::min<long long>((items + 3) / 4, 1 << 30));
  auto* kern = hd == 128 ? (dtype == KVQ_BF16 ? paged_gather_kernel<128, true> : paged_gather_kernel<128, false>)
                         : (dtype == KVQ_BF16 ? paged_gather_kernel<64, true> : paged_gather_kernel<64, false>);
  cudaError_t e = launch_dependent(kern, grid, dim3(GATHER_THREADS), 0, static_cast<cudaStream_t>(stream), a);
  if (e != cudaSuccess) return paged_cuda_fail(e, fn, "launch");
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

extern "C" kvq_status kvq_paged_page_bytes(int head_dim, size_t* bytes) try {
  if (!bytes) return kvq::paged_fail(KVQ_ERR_INVALID, "kvq_paged_page_bytes", "NULL output");
  if (head_dim != 64 && head_dim != 128)
    return kvq::paged_fail(KVQ_ERR_INVALID, "kvq_paged_page_bytes", "head_dim must be 64 or 128");
  *bytes = (size_t)kvq::page_bytes(head_dim);
  return KVQ_OK;
} catch (...) {
  return KVQ_ERR_HOST_OOM;
}

extern "C" kvq_status kvq_paged_append(const kvq_rope_plan* plan, int dtype, const void* k, int64_t k_token_stride,
                                       int64_t k_head_stride, const void* v, int64_t v_token_stride,
                                       int64_t v_head_stride, const int32_t* slots, const int32_t* positions,
                                       int n_tokens, int n_kv_heads, int head_dim, void* pages, int n_pages,
                                       const void* q, int64_t q_token_stride, int64_t q_head_stride, int n_q_heads,
                                       void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                                       void* stream) try {
  return kvq::append_impl(plan, dtype, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, slots,
                          positions, n_tokens, n_kv_heads, head_dim, pages, n_pages, q, q_token_stride, q_head_stride,
                          n_q_heads, q_out, q_out_token_stride, q_out_head_stride, stream);
} catch (...) {
  return KVQ_ERR_HOST_OOM;
}

extern "C" kvq_status kvq_paged_gather(const void* pages, int n_pages, const int32_t* slots, int n_tokens,
                                       int n_kv_heads, int head_dim, int dtype, void* k, int64_t k_token_stride,
                                       int64_t k_head_stride, void* v, int64_t v_token_stride, int64_t v_head_stride,
                                       void* stream) try {
  return kvq::gather_impl(pages, n_pages, slots, n_tokens, n_kv_heads, head_dim, dtype, k, k_token_stride,
                          k_head_stride, v, v_token_stride, v_head_stride, stream);
} catch (...) {
  return KVQ_ERR_HOST_OOM;
}
