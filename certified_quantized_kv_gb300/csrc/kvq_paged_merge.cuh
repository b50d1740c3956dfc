// kvq_paged_merge.cuh -- the paged attention's pieces: rows of a group that a warp or CTA has seen part of
// the tokens of, added up.
#pragma once

#include "kvq_paged.cuh"

namespace kvq {

// Eight warps with two pages each: 160 KB at head_dim 128, two warps per scheduler.  At head_dim 64 more
// would fit: 48 sequences of 4096 tokens took 23.3 us, with 12 warps 25.2, with 16 27.6 (8 sequences of
// 32768: 27.5, 27.7 and 30.7), since each warp's first and last page cost more than waiting does.
constexpr int PA_WARPS = 8;
constexpr int PA_THREADS = 32 * PA_WARPS;

// Where rows of the output go.
struct PaOut {
  void* out;
  float* lse;
  int Q, Hq, n_rep;
  bool bf16;
  // row of the output of row r of (sequence b, KV head g)
  __device__ __forceinline__ size_t row(int b, int g, int r) const {
    const int qi = n_rep == 1 ? r : r / n_rep;
    return ((size_t)b * Q + qi) * Hq + g * n_rep + (r - qi * n_rep);
  }
  // four channels of a row: v / lt, and its lse
  template <int HD>
  __device__ __forceinline__ void store(size_t row, int x, float4 v, float ref, float lt) const {
    const float inv = lt == 0.f ? 0.f : 1.f / lt;
    reinterpret_cast<uint2*>(out)[row * (HD / 4) + x] = make_uint2(f2_to_pair(v.x * inv, v.y * inv, bf16), f2_to_pair(v.z * inv, v.w * inv, bf16));
    if (x == 0 && lse) lse[row] = lt == 0.f ? -INFINITY : (ref + log2f(lt)) * 0.69314718055994531f;
  }
};

// Pieces added up: reference M, weight sum L and four channels' sums o.
struct PaSum {
  float M = -INFINITY, L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  template <int N>
  __device__ __forceinline__ void add(const float2 (&ml)[N], const float4 (&v)[N]) {   // (reference, weight sum), sums
    float to = M;
#pragma unroll
    for (int i = 0; i < N; ++i) to = fmaxf(to, ml[i].x);
    const float f = M == to ? 1.f : exp2_approx(M - to);   // (both -inf: nothing seen yet)
    M = to;
    L *= f;
    o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float w = ml[i].x == -INFINITY ? 0.f : exp2_approx(ml[i].x - to);
      L = fmaf(ml[i].y, w, L);
      o.x = fmaf(v[i].x, w, o.x), o.y = fmaf(v[i].y, w, o.y), o.z = fmaf(v[i].z, w, o.z), o.w = fmaf(v[i].w, w, o.w);
    }
  }
};

// The sum of n pieces of group grp in order, by the whole CTA (KS threads share a sum): into
// dst, or as output rows.  ACROSS: the pieces of the CTAs from *at on, the first one's second
// slot and the others' first; else those of warps, at their pointers from `at` on, the last
// one an ended piece when `closed`.  `lost`: a piece may be anything, the rows become NaN.  Not
// inlined: its registers and its schedule stay out of the page loop's.  Loads are not
// predicated (the last piece is read again in place of those behind it), so that a batch of
// them is on its way at once.
template <int HD, int R, bool ACROSS>
__device__ __noinline__ void pa_merge(PaOut po, const float* const* at, int n, bool closed, bool lost, int b, int g, int r0, int rn, float* dst) {
  constexpr int PART = R * (HD + 2), VEC = R * HD / 4, KS = PA_THREADS / VEC > 1 ? PA_THREADS / VEC : 1;
  constexpr int BATCH = KS > 1 ? 5 : ACROSS ? 10 : PA_WARPS;
  __shared__ float4 red[KS > 1 ? PA_THREADS : 1];
  __shared__ float2 redm[KS > 1 ? PA_THREADS : 1];
  const float* const base = ACROSS ? *at : nullptr;
  for (int e0 = 0; e0 < VEC; e0 += PA_THREADS) {
    const int e = (e0 + threadIdx.x) % VEC, ks = threadIdx.x / VEC, c = e / (HD / 4);
    const size_t row = dst || c >= rn ? 0 : po.row(b, g, r0 + c);   // before the loads, whose time covers it
    PaSum sum;
    for (int k0 = KS > 1 ? ks : 0; k0 < n; k0 += BATCH * KS) {
      float2 ml[BATCH];
      float4 v[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int k = min(k0 + i * KS, n - 1);
        if (ACROSS) {
          const float* src = base + (size_t)(2 * k + (k == 0)) * PART;
          v[i] = __ldcg(reinterpret_cast<const float4*>(src) + e);
          ml[i] = __ldcg(reinterpret_cast<const float2*>(src + R * HD) + c);
        } else {
          const float* src = at[2 * k + !(closed && k == n - 1)];
          v[i] = reinterpret_cast<const float4*>(src)[e];
          ml[i] = reinterpret_cast<const float2*>(src + R * HD)[c];
        }
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i)
        if (k0 + i * KS >= n) ml[i] = make_float2(-INFINITY, 0.f);
      sum.add(ml, v);
    }
    if (KS > 1) {
      red[threadIdx.x] = sum.o;
      redm[threadIdx.x] = make_float2(sum.M, sum.L);
      __syncthreads();
      if (ks == 0)
        for (int k = 1; k < KS; ++k) {
          float2 ml[1] = {redm[k * VEC + e]};
          float4 v[1] = {red[k * VEC + e]};
          sum.add(ml, v);
        }
      __syncthreads();
      if (ks != 0) continue;
    }
    if (lost) sum.L = __int_as_float(0x7fc00000);
    if (dst) {
      reinterpret_cast<float4*>(dst)[e] = sum.o;
      if (e % (HD / 4) == 0) reinterpret_cast<float2*>(dst + R * HD)[c] = make_float2(sum.M, sum.L);
    } else {
      if (c < rn) po.store<HD>(row, e % (HD / 4), sum.o, sum.M, sum.L);
    }
  }
}

}  // namespace kvq
