// kvq_paged.cuh -- layout of the paged 4-bit cache, rotary phases and the element types
// of the calls that use them.
//
// A page holds 64 consecutive tokens of one KV head in one contiguous piece, so that one
// bulk copy moves it (10240 bytes at head_dim 128, 5120 at 64).  With NG = head_dim / 32
// groups:
//   key codes      64 rows (tokens) of head_dim / 2 bytes; channel c = 32g + 8a + j sits in
//                  byte a * 4NG + 4g + (j >> 1), low nibble for even j.  Lane (gid, tig) of
//                  an mma.m16n8k16 reads the piece a = tig of row gid in one load: one 32-bit
//                  word (eight channels) per group.
//   value codes    64 rows of head_dim / 2 bytes; channel c = 32g + 4a + j sits in byte
//                  a * 2NG + 2g + (j >> 1): lane gid reads piece a = gid of the four tokens
//                  of its k columns.  Token t sits in row t ^ ((t >> 1) & 1), bytes XOR
//                  32 ((t >> 2) & 1), at head_dim 128 and in row t ^ ((t >> 2) & 1) at 64, so
//                  that the lanes of one load (two tokens apart) hit distinct banks.
//   key scales     binary16 [64][NG], then key offsets, the same
//   value scales   binary16 [NG][64], token t at 16((t >> 1) & 3) + 4(t >> 4) + 2((t >> 3) & 1)
//                  + (t & 1): the token pairs that lane tig multiplies are contiguous; then
//                  value offsets, the same
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

#include "kvq.h"
#include "kvq_common.cuh"

namespace kvq {

constexpr int PG = 64;   // tokens per page
constexpr int MAX_KV_HEADS = 4096;

template <int HD>
struct Page {
  static constexpr int G = HD / 32;              // 32-channel groups
  static constexpr int ROW = HD / 2;             // code bytes per token
  static constexpr int CODES = PG * ROW;         // code bytes of the keys (and of the values)
  static constexpr int SCALES = PG * G * 2;      // bytes of one scale or offset array
  static constexpr int VC = CODES, KS = 2 * CODES, KO = KS + SCALES, VS = KO + SCALES, VO = VS + SCALES;
  static constexpr int BYTES = VO + SCALES;
};

__host__ __device__ constexpr int page_bytes(int head_dim) { return head_dim == 128 ? Page<128>::BYTES : Page<64>::BYTES; }

// element of token t within one group's 64 value scales (or offsets)
__host__ __device__ __forceinline__ constexpr int vscale_at(int t) {
  return ((t >> 1) & 3) * 16 + (t >> 4) * 4 + ((t >> 3) & 1) * 2 + (t & 1);
}
// byte of (token t, piece byte x) within the value codes
template <int HD>
__host__ __device__ __forceinline__ constexpr int vcode_at(int t, int x) {
  return HD == 128 ? (t ^ ((t >> 1) & 1)) * Page<HD>::ROW + (x ^ (32 * ((t >> 2) & 1)))
                   : (t ^ ((t >> 2) & 1)) * Page<HD>::ROW + x;
}

// a / b for non-negative a and positive b: the 32-bit division (a quarter of the time) where it serves
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// ---- a ring of stages filled by bulk copies ----
// Copy number i goes to stage i % STAGES and completes phase i / STAGES of that stage's barrier.
template <int STAGES>
__host__ __device__ __forceinline__ constexpr int ring_stage(int i) { return i % STAGES; }
template <int STAGES>
__host__ __device__ __forceinline__ constexpr uint32_t ring_parity(int i) { return (uint32_t)(i / STAGES) & 1u; }
// Waits for what may be in flight once `issued` copies were issued: the last one of each stage.
template <int STAGES, typename Wait>
__host__ __device__ __forceinline__ void ring_drain(int issued, const Wait& wait) {   // wait(stage, parity)
  for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i) wait(ring_stage<STAGES>(i), ring_parity<STAGES>(i));
}

// ---- element types of q, k, v and outputs (kvq_dtype) ----
__device__ __forceinline__ float2 pair_to_f2(uint32_t u, bool bf16) {
  if (bf16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  return __half22float2(u32_as_h2(u));
}
__device__ __forceinline__ uint32_t f2_to_pair(float x, float y, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  return h2_as_u32(__floats2half2_rn(x, y));
}
__device__ __forceinline__ float elem_to_f(const void* p, size_t i, bool bf16) {
  const unsigned short u = static_cast<const unsigned short*>(p)[i];
  return bf16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
}

// ---- rotary phases ----
// The angle of position p and pair i is p * step_i in units of 2^-64 turn, an exact
// integer product modulo one turn whatever the position's size and sign.  Its top 32 bits,
// rounded, less the nearest quarter turn are an angle pi (x + l) with |x| <= 1/4, l what
// fp32 loses of it, where the Taylor series of sine and cosine to x^9 and x^10 end below 2^-29
// and 2^-33.  The leading terms are carried with their rounding errors, so that both results
// lie within 2^-24.2 (sincospif of an angle rounded to fp32: 2^-22.5, and no faster: the
// 32K-token append with its read-back 159 us, 158 with the series): keys are coded from them, and
// each error moves some quotient across a half.
__device__ __forceinline__ float2 rope_cos_sin(int pos, uint64_t step, float magnitude) {
  constexpr double PI = 3.14159265358979323846, P2 = PI * PI;
  constexpr float S1 = (float)PI, S1L = (float)(PI - (double)S1);
  constexpr float S3 = (float)(-PI * P2 / 6), S5 = (float)(PI * P2 * P2 / 120);
  constexpr float S7 = (float)(-PI * P2 * P2 * P2 / 5040), S9 = (float)(PI * P2 * P2 * P2 * P2 / 362880);
  constexpr float C2 = (float)(-P2 / 2), C2L = (float)(-P2 / 2 - (double)C2), C4 = (float)(P2 * P2 / 24);
  constexpr float C6 = (float)(-P2 * P2 * P2 / 720), C8 = (float)(P2 * P2 * P2 * P2 / 40320);
  constexpr float C10 = (float)(-P2 * P2 * P2 * P2 * P2 / 3628800), UNIT = 4.656612873077393e-10f /* 2^-31 */;
  const uint32_t a = (uint32_t)(((uint64_t)(int64_t)pos * step + 0x80000000ull) >> 32);   // 2^-32 turns
  const uint32_t quarter = (a + 0x20000000u) >> 30;
  const int32_t f = (int32_t)(a - (quarter << 30));
  const float xf = (float)f, x = xf * UNIT, l = (float)(f - (int32_t)xf) * UNIT;
  const float z = x * x, zl = fmaf(x + x, l, fmaf(x, x, -z));   // z + zl = (x + l)^2
  const float p = fmaf(fmaf(fmaf(fmaf(S9, z, S7), z, S5), z, S3), z, S1L);
  const float sn = fmaf(x, S1, fmaf(x, p, S1 * l));
  const float q = fmaf(fmaf(fmaf(fmaf(C10, z, C8), z, C6), z, C4), z, C2L);
  const float m = C2 * z, t = 1.f + m;   // their errors: fma(C2, z, -m), (1 - t) + m
  const float cn = t + (fmaf(q, z, fmaf(C2, zl, fmaf(C2, z, -m))) + ((1.f - t) + m));
  // cos and sin of the angle and quarter turns more: (c, s), (-s, c), (-c, -s), (s, -c)
  const float c = (quarter & 1u) ? sn : cn, s = (quarter & 1u) ? cn : sn;
  return make_float2(__uint_as_float(__float_as_uint(c * magnitude) ^ ((quarter + 1u) >> 1 << 31)),
                     __uint_as_float(__float_as_uint(s * magnitude) ^ (quarter >> 1 << 31)));
}

// Whether rows of n elements at t ts + h hs, t < T and h < H, share an element (strides >= 0).
inline bool rows_overlap(int64_t T, int64_t H, int64_t ts, int64_t hs, int64_t n) {
  if ((T > 1 && ts < n) || (H > 1 && hs < n)) return true;
  if (T <= 1 || H <= 1) return false;
  if ((ts - n) / (H - 1) >= hs || (hs - n) / (T - 1) >= ts) return false;   // a token's heads lie within its stride, or a head's tokens
  if (H > T) std::swap(T, H), std::swap(ts, hs);
  for (int64_t dh = 1; dh < H; ++dh) {   // rows (t, h + dh) and (t + dt, h): the tokens next to dh heads' distance
    const __int128 x = (__int128)dh * hs, dt = x / ts;
    if (dt < T && x - dt * ts < n) return true;
    if (dt + 1 < T && (dt + 1) * ts - x < n) return true;
  }
  return false;
}

// ---- checks shared by the calls of this file's users (kvq_rope.cu) ----
// Each returns KVQ_OK or reports `fn`'s failure through kvq_last_error().
kvq_status paged_fail(kvq_status s, const char* fn, const char* what);
kvq_status paged_cuda_fail(cudaError_t e, const char* fn, const char* what);
// device memory of `dev`, aligned to `align` bytes
kvq_status check_buffer(const void* p, int dev, size_t align, const char* fn, const char* name);
// rows of a strided [tokens, heads, head_dim] operand: non-negative strides, multiples of 8
kvq_status check_strides(int64_t token, int64_t head, const char* fn, const char* name);
kvq_status check_plan(const kvq_rope_plan* plan, int head_dim, const char* fn);
kvq_status check_axes(const kvq_rope_axes_plan& plan, int64_t axis_stride, const char* fn);

}  // namespace kvq
