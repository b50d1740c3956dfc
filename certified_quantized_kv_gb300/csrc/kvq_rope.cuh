// kvq_rope.cuh -- rotation of strided rows by threads that each own some pairs of a token:
// the rotary operator, and the queries of the paged append.
#pragma once

#include <algorithm>

#include "kvq_paged.cuh"

namespace kvq {

struct RopeArgs {
  const void* x;
  void* out;
  const int32_t* pos;
  long long xt, xh, ot, oh;   // strides in elements
  int T, H, lanes;   // lanes: heads in step, each with a thread of its own per chunk of pairs
  bool copy;         // the elements behind the rotated ones as well
};

// One thread per V pairs of a token, for every `lanes`-th head: cos and sin are formed once and
// used for H / lanes heads, the loads of up to ROPE_UNROLL heads are on their way at once.
// HBM bound (4 bytes per element, 32K tokens of 40 heads of 128: 671 MB); at V = 8, which
// every even layout with rotary_dim a multiple of 16 takes, all accesses are 16 bytes.
// Smaller V serve the other rotary_dims (pairs that start or end between vectors).
constexpr int ROPE_UNROLL = 4;

template <int N>
struct Words {   // N elements in one or two loads of at most 16 bytes
  static constexpr int W = N > 2 ? N / 2 : 1;
  uint32_t w[W];
  __device__ __forceinline__ void load(const unsigned short* p) {
    if constexpr (N == 16) {
      const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else if constexpr (N == 8) {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    } else if constexpr (N == 4) {
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      w[0] = a.x, w[1] = a.y;
    } else if constexpr (N == 2) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *p;
    }
  }
  __device__ __forceinline__ void store(unsigned short* p) const {
    if constexpr (N == 16) {
      reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else if constexpr (N == 8) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (N == 4) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (N == 2) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
      *p = (unsigned short)w[0];
    }
  }
};

// The part of thread `first` of `threads`.
template <int V, bool INTERLEAVED, bool BF16>
__device__ __forceinline__ void rope_part(const kvq_rope_plan& P, const RopeArgs& a, long long first, long long threads) {
  constexpr int N0 = INTERLEAVED ? 2 * V : V;   // elements of one load (and of the other, half a head on)
  constexpr int NT = 2 * V < 8 ? 2 * V : 8;     // elements of one copied piece behind the rotated ones
  const int half = P.rotary_dim / 2, chunks = half / V;
  const long long n = (long long)a.T * a.lanes * chunks;
  for (long long u = first; u < n; u += threads) {
    const long long r = u / chunks, t = r / a.lanes;
    const int c = (int)(u - r * chunks), i0 = c * V, h0 = (int)(r - t * a.lanes);
    const int pos = a.pos[t];
    const int e0 = INTERLEAVED ? 2 * i0 : i0, e1 = i0 + half;
    const unsigned short* x = static_cast<const unsigned short*>(a.x) + t * a.xt;
    unsigned short* out = static_cast<unsigned short*>(a.out) + t * a.ot;
    Words<N0> A[ROPE_UNROLL], B[ROPE_UNROLL];
    auto fetch = [&](int h) {
#pragma unroll
      for (int k = 0; k < ROPE_UNROLL; ++k)
        if (h + k * a.lanes < a.H) {
          A[k].load(x + (h + k * a.lanes) * a.xh + e0);
          if (!INTERLEAVED) B[k].load(x + (h + k * a.lanes) * a.xh + e1);
        }
    };
    fetch(h0);   // on their way while cos and sin are formed
    float2 cs[V];
#pragma unroll
    for (int i = 0; i < V; ++i) cs[i] = rope_cos_sin(pos, P.step[i0 + i], P.magnitude);
    for (int h = h0; h < a.H; h += ROPE_UNROLL * a.lanes) {
      if (h != h0) fetch(h);
#pragma unroll
      for (int k = 0; k < ROPE_UNROLL; ++k) {
        if (h + k * a.lanes >= a.H) continue;
        if (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float2 p = pair_to_f2(A[k].w[i], BF16);
            A[k].w[i] = f2_to_pair(fmaf(p.x, cs[i].x, -p.y * cs[i].y), fmaf(p.y, cs[i].x, p.x * cs[i].y), BF16);
          }
        } else {
#pragma unroll
          for (int i = 0; i < Words<N0>::W; ++i) {
            const float2 p = pair_to_f2(A[k].w[i], BF16), q = pair_to_f2(B[k].w[i], BF16);
            const float2 c0 = cs[2 * i], c1 = cs[V > 1 ? 2 * i + 1 : 0];
            A[k].w[i] = f2_to_pair(fmaf(p.x, c0.x, -q.x * c0.y), fmaf(p.y, c1.x, -q.y * c1.y), BF16);
            B[k].w[i] = f2_to_pair(fmaf(q.x, c0.x, p.x * c0.y), fmaf(q.y, c1.x, p.y * c1.y), BF16);
          }
        }
        unsigned short* o = out + (h + k * a.lanes) * a.oh;
        A[k].store(o + e0);
        if (!INTERLEAVED) B[k].store(o + e1);
      }
    }
    if (a.copy)   // what follows the rotated elements
      for (int e = P.rotary_dim + NT * c; e < P.head_dim; e += NT * chunks)
        for (int h = h0; h < a.H; h += a.lanes) {
          Words<NT> w;
          w.load(x + h * a.xh + e);
          w.store(out + h * a.oh + e);
        }
  }
}

// Pairs per thread: the widest vectors that divide the rotated half.
inline int rope_pairs(const kvq_rope_plan& plan) {
  const int half = plan.rotary_dim / 2;
  return half % 8 == 0 ? 8 : half % 4 == 0 ? 4 : half % 2 == 0 ? 2 : 1;
}

// Heads in step (RopeArgs::lanes): a thread takes one head while the call does not fill the GPU (64
// tokens of 40 heads), and up to eight when it does, so that the angles, which cost as much as
// the rotation of four heads, are shared.
inline int rope_lanes(long long T, int H, int chunks) {
  const long long per = std::min<long long>(8, std::max<long long>(1, T * H * chunks / (152 * 1024)));
  return (int)((H + per - 1) / per);
}

}  // namespace kvq
