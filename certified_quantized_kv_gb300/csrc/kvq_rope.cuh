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
  int per;           // heads of one item (rope_rows)
};

// One thread per V pairs of a token, for every `lanes`-th head; the loads of several heads are on
// their way at once.  HBM bound (4 bytes per element, 32K tokens of 40 heads of 128: 671 MB);
// at V = 8, which every layout with rotary_dim a multiple of 16 takes, all accesses are 16
// bytes.  V = 4 serves halves that are odd multiples of 4, and interleaved pairs of every other
// rotary_dim; rope_rows (below) what is left.
// A cosine and sine cost about 40 instructions.  With TABLE a block forms those of its tokens once, in
// shared memory (64 tokens of 40 heads: 2.44 us, 2.65 without; 4099 tokens of 13: 9.1 and 9.7);
// without, each thread those of its pairs (in the append, whose blocks live on many warps in
// different phases, the table's barriers cost more than they saved: 179 us against 167 when measured).

template <int N>
struct Words {   // N = 4, 8 or 16 elements in one or two loads of at most 16 bytes
  static constexpr int W = N / 2;
  uint32_t w[W];
  __device__ __forceinline__ void load(const unsigned short* p) {
    if constexpr (N == 16) {
      const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else if constexpr (N == 8) {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      w[0] = a.x, w[1] = a.y;
    }
  }
  __device__ __forceinline__ void store(unsigned short* p) const {
    if constexpr (N == 16) {
      reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else if constexpr (N == 8) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
  }
};

// The plan's steps in shared memory: lanes read different ones at once, which constant memory
// would serve one at a time.
__device__ __forceinline__ void load_steps(const kvq_rope_plan& P, uint64_t (&step)[128]) {
  for (int i = threadIdx.x; i < P.rotary_dim / 2; i += blockDim.x) step[i] = P.step[i];
  __syncthreads();
}

// (cos, sin) of all pairs of tokens t0..t0 + n - 1, by the whole block.  With V = 8 two pairs of each
// chunk of eight lie side by side, then the next two of each: lanes with a chunk each read
// neighbouring 16 bytes.
template <int V>
__device__ __forceinline__ int turn_at(int i, int half) {
  return V == 8 ? ((i % 8) / 2 * (half / 8) + i / 8) * 2 + i % 2 : i;
}
template <int V>
__device__ __forceinline__ void fill_turns(const kvq_rope_plan& P, const uint64_t* step, const int32_t* pos, long long t0, int n,
                                           float2* turns) {
  const int half = P.rotary_dim / 2;
  for (int e = threadIdx.x; e < n * half; e += blockDim.x) {
    const int t = e / half, i = e - t * half;
    turns[t * half + turn_at<V>(i, half)] = rope_cos_sin(pos[t0 + t], step[i], P.magnitude);
  }
}

// The units of a block that starts with unit `base` and takes every `stride`-th run of THREADS units;
// turns (TABLE): room for THREADS * V + 2 * 128 elements.
template <int V, bool INTERLEAVED, bool BF16, int THREADS, bool TABLE>
__device__ __forceinline__ void rope_part(const kvq_rope_plan& P, const uint64_t* step, float2* turns, const RopeArgs& a, long long base,
                                          long long stride) {
  constexpr int ROPE_UNROLL = 4;
  constexpr int N0 = INTERLEAVED ? 2 * V : V;   // elements of one load (and of the other, half a head on)
  const int half = P.rotary_dim / 2, chunks = (half + V - 1) / V;
  const int copies = a.copy ? P.head_dim / 8 - (P.rotary_dim + 7) / 8 : 0;   // vectors behind the rotated elements
  const int units = chunks + copies;
  const long long n = (long long)a.T * a.lanes * units;
  const int per_token = a.lanes * units;
  for (; base < n; base += stride) {
    const long long u = base + threadIdx.x, t0 = base / per_token, t1 = min(n - 1, base + THREADS - 1) / per_token;
    const long long r = u / units, t = r / a.lanes;
    const int c = (int)(u - r * units), i0 = c * V, h0 = (int)(r - t * a.lanes);
    const bool live = u < n;
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
    const bool turned = live && c < chunks;
    if (turned) fetch(h0);   // on their way while cos and sin are formed
    if (TABLE) {
      __syncthreads();   // its previous readers are done
      fill_turns<V>(P, step, a.pos, t0, (int)(t1 - t0) + 1, turns);
      __syncthreads();
    }
    if (!live) continue;
    if (!turned) {
      const int e = (P.rotary_dim + 7) / 8 * 8 + 8 * (c - chunks);
#pragma unroll 4
      for (int h = h0; h < a.H; h += a.lanes)
        *reinterpret_cast<uint4*>(out + h * a.oh + e) = *reinterpret_cast<const uint4*>(x + h * a.xh + e);
      continue;
    }
    constexpr bool whole = !INTERLEAVED || V == 8;   // all pairs of every chunk are rotated
    auto pair = [&](int i) { return whole ? i0 + i : min(i0 + i, half - 1); };
    float2 cs[V];
    const float2* mine = turns + (t - t0) * half;
    if constexpr (!TABLE) {
      const int pos = a.pos[t];
#pragma unroll
      for (int i = 0; i < V; ++i) cs[i] = rope_cos_sin(pos, step[pair(i)], P.magnitude);
    } else if constexpr (V == 8) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 v = reinterpret_cast<const float4*>(mine)[k * chunks + c];
        cs[2 * k] = make_float2(v.x, v.y), cs[2 * k + 1] = make_float2(v.z, v.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) cs[i] = mine[pair(i)];
    }
    for (int h = h0; h < a.H; h += ROPE_UNROLL * a.lanes) {
      if (h != h0) fetch(h);
#pragma unroll
      for (int k = 0; k < ROPE_UNROLL; ++k) {
        if (h + k * a.lanes >= a.H) continue;
        if (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float2 p = pair_to_f2(A[k].w[i], BF16);
            const uint32_t y = f2_to_pair(fmaf(p.x, cs[i].x, -p.y * cs[i].y), fmaf(p.y, cs[i].x, p.x * cs[i].y), BF16);
            A[k].w[i] = whole || i0 + i < half ? y : A[k].w[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < Words<N0>::W; ++i) {
            const float2 p = pair_to_f2(A[k].w[i], BF16), q = pair_to_f2(B[k].w[i], BF16);
            const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
            A[k].w[i] = f2_to_pair(fmaf(p.x, c0.x, -q.x * c0.y), fmaf(p.y, c1.x, -q.y * c1.y), BF16);
            B[k].w[i] = f2_to_pair(fmaf(q.x, c0.x, p.x * c0.y), fmaf(q.y, c1.x, p.y * c1.y), BF16);
          }
        }
        unsigned short* o = out + (h + k * a.lanes) * a.oh;
        A[k].store(o + e0);
        if (!INTERLEAVED) B[k].store(o + e1);
      }
    }
  }
}

// Vectors of a row that are rotated, or all of them with the copied ones.
__host__ __device__ __forceinline__ int row_vectors(const kvq_rope_plan& P, bool copy) {
  return (copy ? P.head_dim : P.rotary_dim + 7) / 8;
}

// rope_rows (below): the first channel of a lane's vector.  Lanes left over behind the warp's last whole row
// count on from there, behind every rotated channel, so that their elements are their own partners.
__host__ __device__ __forceinline__ int row_channel(int lane, int vecs) {
  const int r = lane / vecs;
  return 8 * (r < 32 / vecs ? lane - r * vecs : lane);
}
// Where in a warp's room, eight elements per lane, the other element of the pair of channel ch lies, for a
// lane whose vector starts with channel c0; the channel's own place when it is not rotated.
__host__ __device__ __forceinline__ int row_partner(int lane, int c0, int ch, int half) {
  return (lane * 8 - c0) + (ch >= 2 * half ? ch : ch >= half ? ch - half : ch + half);
}

// The same for halves that are no multiple of 4, whose pairs start anywhere in their vectors: a warp
// takes whole rows of one token, as many at once as its lanes hold vectors of, and a lane reads the
// other elements of its vector's pairs out of shared memory (room: 32 vectors; turns: 128 (cos, sin)).
// 4000 tokens of 32 heads of 128 from buffer to buffer, 52 elements rotated: 13.6 us; pairs by threads of
// their own, as above with V = 2: 23.2.  With half = 52, V = 4: 14.3 us, rows 17.3.
// Item: a token's heads [h, h + a.per); warp w0 takes every `warps`-th one.
template <bool BF16>
__device__ __forceinline__ void rope_rows(const kvq_rope_plan& P, const uint64_t* step, uint4* room, float2* turns, const RopeArgs& a,
                                          long long w0, long long warps) {
  constexpr int U = 4;   // rows of a lane on their way at once
  const int lane = threadIdx.x & 31, half = P.rotary_dim / 2;
  const int vecs = row_vectors(P, a.copy), rows = 32 / vecs;   // vectors of a row, rows at once
  const int r = lane / vecs, c0 = row_channel(lane, vecs);     // this lane's row and first channel
  const bool even = half % 2 == 0;
  const int items = (a.H + a.per - 1) / a.per;
  const long long n = (long long)a.T * items;
  for (long long u = w0; u < n; u += warps) {
    const long long t = quotient(u, items);
    const int h0 = (int)(u - t * items) * a.per, h1 = min(a.H, h0 + a.per);
    const unsigned short* x = static_cast<const unsigned short*>(a.x) + t * a.xt;
    unsigned short* out = static_cast<unsigned short*>(a.out) + t * a.ot;
    uint4 v[U] = {};   // (lanes without a row take part in the exchange)
    auto fetch = [&](int h) {
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (r < rows && h + k * rows + r < h1) v[k] = *reinterpret_cast<const uint4*>(x + (h + k * rows + r) * a.xh + c0);
    };
    fetch(h0);   // on their way while cos and sin are formed
    const int pos = a.pos[t];
    __syncwarp();   // the last item's readers are done
    for (int i = lane; i < half; i += 32) turns[i] = rope_cos_sin(pos, step[i], P.magnitude);
    __syncwarp();
    float c[8], s[8];
    int from[8];   // the other element of the pair
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int ch = c0 + e;
      const bool in = ch < 2 * half, second = ch >= half;
      const float2 cs = in ? turns[second ? ch - half : ch] : make_float2(1.f, 0.f);
      c[e] = cs.x, s[e] = second ? cs.y : -cs.y;
      from[e] = row_partner(lane, c0, ch, half);
    }
    for (int h = h0; h < h1; h += U * rows) {
      if (h != h0) fetch(h);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (h + k * rows >= h1) continue;
        room[lane] = v[k];
        __syncwarp();
        uint32_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // (pairs of an even half lie in whole words)
          const uint32_t other = even ? reinterpret_cast<const uint32_t*>(room)[from[2 * i] / 2]
                                      : (uint32_t) reinterpret_cast<const unsigned short*>(room)[from[2 * i]] |
                                            ((uint32_t) reinterpret_cast<const unsigned short*>(room)[from[2 * i + 1]] << 16);
          const float2 p = pair_to_f2(word_of(v[k], i), BF16), o = pair_to_f2(other, BF16);
          const uint32_t w = f2_to_pair(fmaf(p.x, c[2 * i], o.x * s[2 * i]), fmaf(p.y, c[2 * i + 1], o.y * s[2 * i + 1]), BF16);
          y[i] = c0 + 2 * i < 2 * half ? w : word_of(v[k], i);   // (rotary_dim is even)
        }
        if (r < rows && h + k * rows + r < h1) *reinterpret_cast<uint4*>(out + (h + k * rows + r) * a.oh + c0) = make_uint4(y[0], y[1], y[2], y[3]);
        __syncwarp();
      }
    }
  }
}

// Pairs per thread: the widest vectors that divide the rotated half, and interleaved whole vectors of
// four pairs at least, of which the last may lie partly behind the rotated elements.  0: rope_rows.
inline int rope_pairs(const kvq_rope_plan& plan) {
  const int half = plan.rotary_dim / 2;
  return half % 8 == 0 ? 8 : half % 4 == 0 || plan.interleaved ? 4 : 0;
}

// Pieces of a row: chunks of V pairs, and the vectors that are only copied.
inline int rope_units(const kvq_rope_plan& plan, int V, bool copy) {
  return (plan.rotary_dim / 2 + V - 1) / V + (copy ? plan.head_dim / 8 - (plan.rotary_dim + 7) / 8 : 0);
}

// Heads per thread or warp: the fewest, 16 at most, with which all of a call's threads (or warps), `each`
// per token and share of the heads, have room on the GPU at once.  A second wave of blocks costs as
// much as more heads in one (1024 tokens of 32 heads of 128: 3.8 us with three heads per thread, 4.7 with
// two, 6.7 with one; 2048 tokens: 5.3 with five, 5.9 with three; the append of 4096 with 8 KV heads: 15.3
// us with 16 query heads per thread, 18.2 with eight, both with phases of lower accuracy; 16.4 as it
// is).  Else eight: enough to share the angles, which cost as much as the rotation of two heads
// (32768 tokens: 122 us, 126 with 16).
inline int heads_each(long long T, int H, int each, long long room) {
  for (int per = 1; per <= 16; ++per)
    if (T * ((H + per - 1) / per) * each <= room) return per;
  return 8;
}

// Heads per item of rope_rows when `room` warps run at once.
inline int rope_rows_heads(const kvq_rope_plan& plan, bool copy, long long T, int H, long long room) {
  const int rows = 32 / row_vectors(plan, copy);
  return heads_each(T, (H + rows - 1) / rows, 1, room) * rows;
}

// Heads in step (RopeArgs::lanes) when `room` threads run at once.
inline int rope_lanes(long long T, int H, int units, long long room) {
  const int per = heads_each(T, H, units, room);
  return (H + per - 1) / per;
}

}  // namespace kvq
