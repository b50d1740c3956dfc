// kvq_paged_append.cu -- tokens into the pages of the 4-bit cache (with the rotation of
// keys and queries on the way), and back out of them.
//
// Per token, KV head and group of 32 channels (x the rotated key or the value, in fp32):
//   o = fp16(min), s = fp16 rounded up of (max - o) / 15, code = clamp(rint((x - o) / s), 0, 15)
// and for the values of odd slots, counted down from the maximum,
//   o = fp16(max), s = -(fp16 rounded up of (o - min) / 15), code = clamp(rint((o - x) / |s|), 0, 15)
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

constexpr int E = 8;   // neighbouring elements of a row that a lane holds
struct Octet {
  uint32_t w[4];
  __device__ __forceinline__ void load(const unsigned short* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
  __device__ __forceinline__ void unpack(float (&x)[E], bool bf16) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 p = pair_to_f2(w[k], bf16);
      x[2 * k] = p.x, x[2 * k + 1] = p.y;
    }
  }
};

// Rotation of rows spread over HD / 8 lanes at one token's position.  The other element of a
// pair is in the same lane (INTERLEAVED), or a whole number of lanes away (LANES), or, when half of
// rotary_dim is no multiple of 8, anywhere (ELEMENTS: through shared memory).
enum class Turn { NONE, INTERLEAVED, LANES, ELEMENTS };
template <int HD, Turn TURN, bool BF16, bool AXES>
struct Rotation {
  float c[E], s[E];  // y = x c + other s (s carries the sign; elements not rotated: 1, 0)
  int half, ch, from;   // this lane's first channel, the lane with the others (LANES)
  __device__ __forceinline__ bool in(int e) const { return ch + e < 2 * half; }
  __device__ __forceinline__ void set(const kvq_rope_plan& P, const uint64_t* steps, const Place<AXES>& at, int lane) {
    if (TURN == Turn::NONE) return;
    half = P.rotary_dim / 2;
    ch = E * (lane % (HD / E));
    auto turn = [&](int i) { return at.turn(steps[i], P.magnitude); };
    if (TURN == Turn::INTERLEAVED) {
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 cs = in(e) ? turn((ch + e) / 2) : make_float2(1.f, 0.f);
        c[e] = c[e + 1] = cs.x, s[e] = -cs.y, s[e + 1] = cs.y;
      }
    } else if (TURN == Turn::LANES) {
      // both lanes of a pair of lanes need the same eight turns: each forms four of them
      const bool second = ch >= half;
      from = in(0) ? lane + (second ? -half : half) / E : lane;
      const int i0 = second ? ch - half + 4 : ch;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 cs = in(0) ? turn(i0 + e) : make_float2(1.f, 0.f);
        const float x = __shfl_sync(0xffffffffu, cs.x, from), y = __shfl_sync(0xffffffffu, cs.y, from);
        c[e] = second ? x : cs.x, s[e] = second ? y : -cs.y;
        c[4 + e] = second ? cs.x : x, s[4 + e] = second ? cs.y : -y;
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool second = ch + e >= half;
        const float2 cs = in(e) ? turn(second ? ch + e - half : ch + e) : make_float2(1.f, 0.f);
        c[e] = cs.x, s[e] = second ? cs.y : -cs.y;
      }
    }
  }
  // room: 16 bytes per lane (ELEMENTS)
  __device__ __forceinline__ void apply(const Octet& r, float (&y)[E], uint4* room, int lane) const {
    float x[E], o[E];
    r.unpack(x, BF16);
    if (TURN == Turn::INTERLEAVED) {
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = in(e) ? x[e ^ 1] : 0.f;
    } else if (TURN == Turn::LANES) {
      Octet p;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w = __shfl_sync(0xffffffffu, r.w[k], from);
        p.w[k] = in(0) ? w : 0u;
      }
      p.unpack(o, BF16);
    } else if (TURN == Turn::ELEMENTS) {
      room[lane] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
      __syncwarp();
      const int row = (lane - lane % (HD / E)) * E;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = in(e) ? elem_to_f(room, row + (ch + e >= half ? ch + e - half : ch + e + half), BF16) : 0.f;
      __syncwarp();
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

// Extremes of a group (four lanes) of fp32 elements, both NaN when an element is.
__device__ __forceinline__ float2 extremes(const float (&x)[E]) {
  float lo = min_nan(min_nan(min_nan(x[0], x[1]), min_nan(x[2], x[3])), min_nan(min_nan(x[4], x[5]), min_nan(x[6], x[7])));
  float hi = max_nan(max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3])), max_nan(max_nan(x[4], x[5]), max_nan(x[6], x[7])));
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
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
__device__ __forceinline__ float2 extremes(const Octet& r) {
  constexpr uint32_t NEG = 0x80008000u;
  const uint32_t hi = max_pair<BF16>(max_pair<BF16>(r.w[0], r.w[1]), max_pair<BF16>(r.w[2], r.w[3]));
  const uint32_t lo = max_pair<BF16>(max_pair<BF16>(r.w[0] ^ NEG, r.w[1] ^ NEG), max_pair<BF16>(r.w[2] ^ NEG, r.w[3] ^ NEG));
  uint32_t m = max_pair<BF16>(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) m = max_pair<BF16>(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float2 p = pair_to_f2(m, BF16);
  return make_float2(-p.y, p.x);
}

// Scale, offset and packed codes (4 bits each, from bit 0) of this lane's elements of a
// group with extremes lo and hi.  The scale is the smallest binary16 h with 15 h >= the span,
// which is the span / 15 rounded up; 15 h is exact in fp32, so that it is at least the exact span
// where it is at least the span rounded up to fp32.  Codes are rint(d / |s|) for d = x - o in fp32 and
// the exact quotient: they come from a product with the reciprocal, and the remainder d - code s, exact
// near a half, tells where a neighbour is nearer, or as near and even (values on the binary16
// grid meet exact halves in about one element of a hundred).  The slow path also clamps the codes,
// which only elements beyond the rounded offset or the binary16 range need.  Extremes that are NaN
// make the offset NaN and the scale 0: the group then reads as NaN, whatever its codes.
__device__ __forceinline__ uint32_t quantize(const float (&x)[E], float2 ext, bool down, __half& sh, __half& oh) {
  constexpr float RND = 12582912.f;   // 1.5 2^23: adding it rounds to an integer, ties to even
  const float lo = min_nan(max_nan(ext.x, -65504.f), 65504.f), hi = min_nan(max_nan(ext.y, -65504.f), 65504.f);
  oh = __float2half_rn(down ? hi : lo);
  const float of = __half2float(oh), span = fmaxf(__fsub_ru(down ? of : hi, down ? lo : of), 0.f);
  const float before = down ? ext.y - of : of - ext.x;   // how far the extreme lies before the offset,
  const float behind = (down ? of - ext.x : ext.y - of) - span;   // and the other one behind the span
  const unsigned short h = __half_as_ushort(__float2half_ru(span * 0.06666667f));
  const float sh1 = __half2float(__ushort_as_half(h)), sh0 = __half2float(__ushort_as_half((unsigned short)(h - 1)));
  const int step = 15.f * sh0 >= span ? -1 : 15.f * sh1 < span ? 1 : 0;   // (h = 0: sh0 is a NaN)
  sh = __ushort_as_half((unsigned short)(h + step));
  const float sa = __half2float(sh), s = down ? -sa : sa, half = 0.5f * sa;
  const float inv = sa > 0.f ? __fdividef(1.f, s) : 0.f;   // |s| lies in [2^-24, 2^14]
  const float2 rnd = make_float2(RND, RND);
  float2 t[E / 2], r[E / 2];
  float worst = fmaxf(before, behind);
#pragma unroll
  for (int k = 0; k < E / 2; ++k) {
    const float2 d = sub2(make_float2(x[2 * k], x[2 * k + 1]), make_float2(of, of));
    t[k] = fma2(d, make_float2(inv, inv), rnd);   // bits: RND's plus the code
    r[k] = fma2(sub2(rnd, t[k]), make_float2(s, s), d);
    worst = fmaxf(worst, fmaxf(fabsf(r[k].x), fabsf(r[k].y)));
  }
  if (worst >= half) {
    auto fix = [&](float xe, float& te, float re) {
      const bool off = fabsf(re) > half || (fabsf(re) == half && (__float_as_uint(te) & 1u));
      const float to = off ? te + ((re < 0.f) == down ? 1.f : -1.f) : te;
      // beyond what the sum with RND holds as an integer, te is far from every code
      te = sa > 0.f ? fminf(fmaxf(to, RND), RND + 15.f) : RND;
    };
#pragma unroll
    for (int k = 0; k < E / 2; ++k) fix(x[2 * k], t[k].x, r[k].x), fix(x[2 * k + 1], t[k].y, r[k].y);
  }
  if (down) sh = __hneg(sh);
  // codes side by side, less the bits of RND (modulo 2^32)
  constexpr uint32_t BITS = 0x4B400000u;
  uint32_t code = 0u - (BITS + (BITS << 4) + (BITS << 8));   // (22 zeros at the end: nothing is left from << 12 on)
#pragma unroll
  for (int k = 0; k < E / 2; ++k) code += (__float_as_uint(t[k].x) << (8 * k)) + (__float_as_uint(t[k].y) << (8 * k + 4));
  return code;
}

// One warp per item: two tokens at head_dim 128, four at 64 (eight elements per lane: what is done once
// per group and lane, the extremes and the scale, costs half of what it does with four: 32768
// tokens without q 60 us, 79 with four), and of each the KV heads [h, h + a.per), one after the other
// with cos and sin formed once; the next head's rows are on their way while one is coded (55 us,
// 60 without).  The other blocks turn q, a thread per V pairs.
//
// The KV blocks are bound by the issue of their instructions (unpacking, rotation, the shuffles of
// the extremes, the verified scale and codes), the q blocks by HBM; so the two kinds are spread
// over the grid in turn.  32768 tokens of 32 + 8 heads of 128: 713 MB in 122 us (5.8 TB/s, a copy's
// 6.8); 158 with the read-back behind it (registers for 8 blocks per SM gave 160 where these gave 159,
// for 6 162).
constexpr int APPEND_THREADS = 128;
template <int HD, Turn TURN, int V, bool BF16, bool AXES>
__global__ void __launch_bounds__(APPEND_THREADS, 7) paged_append_kernel(const __grid_constant__ kvq_rope_plan P, AppendPagedArgs a) {
  using L = Page<HD>;
  constexpr int LANES = HD / E, TOKENS = 32 / LANES;   // lanes of a row, tokens of an item
  constexpr int WARPS = APPEND_THREADS / 32;
  __shared__ __align__(16) uint64_t steps[128];
  __shared__ uint4 rooms[TURN == Turn::ELEMENTS ? APPEND_THREADS : 1];
  pdl_trigger();
  if (TURN != Turn::NONE) load_steps(P, steps);
  pdl_wait();
  // block b is KV block number floor(b kv / all) when that number changes behind it
  const unsigned k0 = blockIdx.x * a.kv_blocks / gridDim.x, k1 = (blockIdx.x + 1) * a.kv_blocks / gridDim.x;   // (products below 2^26)
  if constexpr (TURN != Turn::NONE) {
    if (k0 == k1) {
      const long long mine = blockIdx.x - k0, all = gridDim.x - a.kv_blocks;
      if constexpr (V == 0) {
        __shared__ float2 turns[WARPS][128];
        const int warp = threadIdx.x >> 5;
        rope_rows<BF16, AXES>(P, steps, rooms + 32 * warp, turns[warp], a.q, mine * WARPS + warp, all * WARPS);
      } else {
        rope_part<V, TURN == Turn::INTERLEAVED, BF16, APPEND_THREADS, false, AXES>(P, steps, nullptr, a.q, mine * APPEND_THREADS,
                                                                             all * APPEND_THREADS);
      }
      return;
    }
  }
  const int lane = threadIdx.x & 31, sub = lane % LANES, hh = lane / LANES, g = sub / 4, j = sub % 4;
  uint4* room = rooms + (TURN == Turn::ELEMENTS ? threadIdx.x - lane : 0);
  const int items = (a.Hkv + a.per - 1) / a.per;
  const long long n = ((long long)a.T + TOKENS - 1) / TOKENS * items;
  for (long long u = (long long)k0 * WARPS + (threadIdx.x >> 5); u < n; u += (long long)a.kv_blocks * WARPS) {
    const long long tp = quotient(u, items), t = tp * TOKENS + hh;
    const int h0 = (int)(u - tp * items) * a.per, h1 = min(a.Hkv, h0 + a.per);
    const bool in = t < a.T;
    const unsigned short* kp = static_cast<const unsigned short*>(a.k) + t * a.kt + h0 * a.kh + E * sub;
    const unsigned short* vp = static_cast<const unsigned short*>(a.v) + t * a.vt + h0 * a.vh + E * sub;
    // the token's slot and position and its first rows in one go, whether it turns out to be skipped or not
    const int slot = in ? a.slots[t] : -1;
    Place<AXES> pos;
    if (TURN != Turn::NONE && in) pos.load(a.pos, a.q.ps, a.q.n_axes, t);
    else pos.none();
    Octet next_k = {}, next_v = {};
    if (in) next_k.load(kp), next_v.load(vp);
    const bool live = slot >= 0 && slot / PG < a.n_pages;
    if (!__any_sync(0xffffffffu, live)) continue;
    const int at = live ? slot % PG : 0;
    const bool down = at & 1;
    // this lane's bytes of the codes, and its group's scale and offset (lane j = 0 writes)
    unsigned char* pg = a.pages + ((size_t)(live ? slot / PG : 0) * a.Hkv + h0) * L::BYTES;
    unsigned char* kc = pg + at * L::ROW + j * 4 * L::G + 4 * g;
    unsigned char* vc = pg + L::VC + vcode_at<HD>(at, 2 * j * 2 * L::G + 2 * g);   // and 2G bytes on
    __half* ks = reinterpret_cast<__half*>(pg + L::KS) + at * L::G + g;
    __half* vs = reinterpret_cast<__half*>(pg + L::VS) + g * PG + vscale_at(at);
    Rotation<HD, TURN, BF16, AXES> rot;
    for (int h = h0; h < h1; ++h) {
      const Octet rk = next_k, rv = next_v;
      kp += a.kh, vp += a.vh;
      if (live && h + 1 < h1) next_k.load(kp), next_v.load(vp);   // on their way while this head is coded
      if (TURN != Turn::NONE && h == h0) rot.set(P, steps, pos, lane);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        float x[E];
        float2 ext;
        if (kv || TURN == Turn::NONE) {
          const Octet& r = kv ? rv : rk;
          ext = extremes<BF16>(r);
          r.unpack(x, BF16);
        } else {
          rot.apply(rk, x, room, lane);
          ext = extremes(x);
        }
        __half s, o;
        const uint32_t code = quantize(x, ext, kv && down, s, o);
        if (live) {
          if (kv) {
            *reinterpret_cast<unsigned short*>(vc) = (unsigned short)code;
            *reinterpret_cast<unsigned short*>(vc + 2 * L::G) = (unsigned short)(code >> 16);
          } else {
            *reinterpret_cast<uint32_t*>(kc) = code;
          }
          if (j == 0) {
            __half* so = kv ? vs : ks;
            so[0] = s;
            so[L::SCALES / 2] = o;
          }
        }
      }
      kc += L::BYTES, vc += L::BYTES, ks += L::BYTES / 2, vs += L::BYTES / 2;
    }
  }
}

using AppendKernel = void (*)(kvq_rope_plan, AppendPagedArgs);
template <int HD, bool BF16, bool AXES>
AppendKernel append_kernel_of(const kvq_rope_plan& plan) {
  const int V = rope_pairs(plan);   // per thread that turns q (0: rope_rows)
  if (plan.interleaved)
    return V == 8 ? paged_append_kernel<HD, Turn::INTERLEAVED, 8, BF16, AXES> : paged_append_kernel<HD, Turn::INTERLEAVED, 4, BF16, AXES>;
  return V == 8   ? paged_append_kernel<HD, Turn::LANES, 8, BF16, AXES>
         : V == 4 ? paged_append_kernel<HD, Turn::ELEMENTS, 4, BF16, AXES>
                  : paged_append_kernel<HD, Turn::ELEMENTS, 0, BF16, AXES>;
}
template <int HD, bool BF16>
AppendKernel append_kernel_of(const kvq_rope_plan* plan, bool axes) {
  if (!plan) return paged_append_kernel<HD, Turn::NONE, 0, BF16, false>;
  return axes ? append_kernel_of<HD, BF16, true>(*plan) : append_kernel_of<HD, BF16, false>(*plan);
}

struct GatherArgs {
  const unsigned char* pages;
  const int32_t* slots;
  void *k, *v;
  long long kt, kh, vt, vh;
  int T, Hkv, n_pages, per;   // per: heads of one item
};

// One warp per item of a token's heads [h, h + a.per): half of the lanes read keys, half values, eight
// channels each (one 16-byte store); at head_dim 64 a warp takes two heads at once.  HBM bound at
// large sizes (4-bit codes and scales in, two bytes per element out: 32768 tokens of 8 heads of 128,
// 176 MB, 35 us), by latency at small ones: four steps' loads are on their way at once (two:
// 38 us, eight: 39).
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
    const long long t = quotient(u, items);
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

// axes: NULL for plans of one axis
kvq_status append_impl(const char* fn, const kvq_rope_plan* plan, const kvq_rope_axes_plan* axes, int dtype, const void* k, int64_t kt,
                       int64_t kh, const void* v, int64_t vt, int64_t vh, const int32_t* slots, const int32_t* positions,
                       int64_t axis_stride, int T, int Hkv, int hd, void* pages, int n_pages, const void* q, int64_t qt, int64_t qh,
                       int Hq, void* q_out, int64_t ot, int64_t oh, void* stream) {
  if (kvq_status s = check_common(fn, dtype, T, Hkv, hd, n_pages)) return s;
  if (plan) {
    if (kvq_status s = check_plan(plan, hd, fn)) return s;
    if (axes)
      if (kvq_status s = check_axes(*axes, axis_stride, fn)) return s;
    if (!positions && T > 0) return paged_fail(KVQ_ERR_INVALID, fn, "positions is NULL with a plan");
  } else if (positions || q || q_out) {
    return paged_fail(KVQ_ERR_INVALID, fn, "positions, q and q_out need a plan");
  }
  if ((q == nullptr) != (q_out == nullptr)) return paged_fail(KVQ_ERR_INVALID, fn, "q and q_out go together");
  if (Hq < 0 || (q && Hq < 1)) return paged_fail(KVQ_ERR_INVALID, fn, "n_q_heads must be >= 1 with q");
  if (T == 0) return KVQ_OK;
  if (kvq_status s = check_strides(kt, kh, fn, "k")) return s;
  if (kvq_status s = check_strides(vt, vh, fn, "v")) return s;
  if (q) {
    if (kvq_status s = check_strides(qt, qh, fn, "q")) return s;
    if (kvq_status s = check_strides(ot, oh, fn, "q_out")) return s;
    if (q == q_out && ((T > 1 && qt != ot) || (Hq > 1 && qh != oh)))
      return paged_fail(KVQ_ERR_INVALID, fn, "q_out = q needs the same strides");
    if (rows_overlap(T, Hq, ot, oh, hd)) return paged_fail(KVQ_ERR_INVALID, fn, "q_out: rows must not overlap");
    if (q_out == k || q_out == v) return paged_fail(KVQ_ERR_INVALID, fn, "q_out must not be k or v");
  }
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return paged_cuda_fail(e, fn, "no current CUDA device");
  if (kvq_status s = check_buffer(k, dev, 16, fn, "k")) return s;
  if (kvq_status s = check_buffer(v, dev, 16, fn, "v")) return s;
  if (kvq_status s = check_buffer(slots, dev, 4, fn, "slots")) return s;
  if (kvq_status s = check_buffer(pages, dev, 16, fn, "pages")) return s;
  if (plan)
    if (kvq_status s = check_buffer(positions, dev, 4, fn, "positions")) return s;
  if (q) {
    if (kvq_status s = check_buffer(q, dev, 16, fn, "q")) return s;
    if (kvq_status s = check_buffer(q_out, dev, 16, fn, "q_out")) return s;
  }
  AppendPagedArgs a{k, v, slots, positions, static_cast<unsigned char*>(pages), kt, kh, vt, vh, T, Hkv, n_pages, 0, 0, {}};
  a.q.ps = axis_stride, a.q.n_axes = axes ? axes->n_axes : 1;
  const int tokens = 32 * E / hd;   // of one item
  const long long rows = ((long long)T + tokens - 1) / tokens;
  // 7 blocks of 4 warps per SM, half of them for q (heads_each)
  constexpr long long ROOM = 152 * 7 * (APPEND_THREADS / 32);
  a.per = heads_each(rows, Hkv, 1, q ? ROOM / 2 : ROOM);
  const long long items = rows * ((Hkv + a.per - 1) / a.per);
  long long blocks = std::min<long long>((items + APPEND_THREADS / 32 - 1) / (APPEND_THREADS / 32), 152 * 32);
  a.kv_blocks = (int)blocks;
  if (q) {
    const bool copy = q != q_out && plan->rotary_dim < hd;
    const int V = rope_pairs(*plan);
    a.q = RopeArgs{q, q_out, positions, qt, qh, ot, oh, T, Hq, 0, copy, 0, a.q.ps, a.q.n_axes};
    long long q_blocks;
    if (V) {
      const int units = rope_units(*plan, V, copy);
      a.q.lanes = rope_lanes(T, Hq, units, ROOM / 2 * 32);
      q_blocks = ((long long)T * a.q.lanes * units + APPEND_THREADS - 1) / APPEND_THREADS;
    } else {
      a.q.per = rope_rows_heads(*plan, copy, T, Hq, ROOM / 2);
      q_blocks = ((long long)T * ((Hq + a.q.per - 1) / a.q.per) + APPEND_THREADS / 32 - 1) / (APPEND_THREADS / 32);
    }
    blocks += std::min<long long>(q_blocks, 152 * 32);
  }
  const bool bf16 = dtype == KVQ_BF16;
  const AppendKernel kern = hd == 128 ? (bf16 ? append_kernel_of<128, true>(plan, axes) : append_kernel_of<128, false>(plan, axes))
                                      : (bf16 ? append_kernel_of<64, true>(plan, axes) : append_kernel_of<64, false>(plan, axes));
  kvq_rope_plan none = {};
  cudaError_t e = launch_dependent(kern, dim3((unsigned)blocks), dim3(APPEND_THREADS), 0, static_cast<cudaStream_t>(stream),
                                   axes ? with_axes(*axes) : plan ? *plan : none, a);
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
  if (k == v || rows_overlap(T, Hkv, kt, kh, hd) || rows_overlap(T, Hkv, vt, vh, hd))
    return paged_fail(KVQ_ERR_INVALID, fn, "k and v: rows must not overlap");
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return paged_cuda_fail(e, fn, "no current CUDA device");
  if (kvq_status s = check_buffer(pages, dev, 16, fn, "pages")) return s;
  if (kvq_status s = check_buffer(slots, dev, 4, fn, "slots")) return s;
  if (kvq_status s = check_buffer(k, dev, 16, fn, "k")) return s;
  if (kvq_status s = check_buffer(v, dev, 16, fn, "v")) return s;
  GatherArgs a{static_cast<const unsigned char*>(pages), slots, k, v, kt, kh, vt, vh, T, Hkv, n_pages, 0};
  a.per = heads_each(T, Hkv, 1, 152 * 48);   // warps that run at once
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
  return kvq::append_impl("kvq_paged_append", plan, nullptr, dtype, k, k_token_stride, k_head_stride, v, v_token_stride,
                          v_head_stride, slots, positions, 0, n_tokens, n_kv_heads, head_dim, pages, n_pages, q,
                          q_token_stride, q_head_stride, n_q_heads, q_out, q_out_token_stride, q_out_head_stride, stream);
} catch (...) {
  return KVQ_ERR_HOST_OOM;
}

extern "C" kvq_status kvq_paged_append_axes(const kvq_rope_axes_plan* plan, int dtype, const void* k, int64_t k_token_stride,
                                            int64_t k_head_stride, const void* v, int64_t v_token_stride,
                                            int64_t v_head_stride, const int32_t* slots, const int32_t* positions,
                                            int64_t axis_stride, int n_tokens, int n_kv_heads, int head_dim, void* pages,
                                            int n_pages, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                            int n_q_heads, void* q_out, int64_t q_out_token_stride,
                                            int64_t q_out_head_stride, void* stream) try {
  const char* fn = "kvq_paged_append_axes";
  if (!plan) return kvq::paged_fail(KVQ_ERR_INVALID, fn, "plan is NULL");
  return kvq::append_impl(fn, &plan->plan, plan, dtype, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride,
                          slots, positions, axis_stride, n_tokens, n_kv_heads, head_dim, pages, n_pages, q, q_token_stride,
                          q_head_stride, n_q_heads, q_out, q_out_token_stride, q_out_head_stride, stream);
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
