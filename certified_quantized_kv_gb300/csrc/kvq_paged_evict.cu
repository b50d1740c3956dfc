// kvq_paged_evict.cu -- a paged cache cut back to its heaviest tokens.
//
// Per (sequence of n tokens, KV head): the first `first` tokens and the last `recent` are kept, and of the others
// those with the largest weights, the lowest index first among equal ones, `keep` in all.  They move, in their order,
// into the pages of another table; codes, scales and offsets move as they are, so that nothing is rounded again (a
// token from an odd slot keeps its values' negative scales in an even one, which stand for the same values).
//
// Two kernels.  The first finds the keep-th largest weight of a row by radix selection (three passes of 9, 12
// and 11 bits over keys whose unsigned order is the weights') and writes the kept indices in order: a cluster of CTAs
// per row, each with a contiguous slice of it, whose histograms are added up in the first CTA's shared
// memory.  The second moves tokens, a block per destination page.
//
// Measured: one sequence of 131072 tokens and 8 KV heads of 128 cut to 16384: selection 24 us, of which the keys' way into
// shared memory takes 3, the first histogram 4, the others with their cluster barriers 10 and the indices' writing 6; the move
// of 42 MB 14.  Four sequences of 1100 tokens back to 1000: 7 and 7 us, chains of dependent loads and barriers.
#include <cooperative_groups.h>

#include <algorithm>
#include <cstddef>
#include <string>

#include "kvq.h"
#include "kvq_launch.h"
#include "kvq_paged.cuh"

namespace kvq {

namespace {

namespace cg = cooperative_groups;

struct EvictArgs {
  const unsigned char* pages;
  unsigned char* to;
  const int32_t *table, *lens, *new_table;
  int32_t *new_lens, *origin;
  const float* weights;
  float* new_weights;   // may be NULL
  long long table_stride, new_stride, ws, wh, nws, nwh;
  int n_pages, to_pages, max_pages, columns, B, Hkv, keep, first, recent;
};

__device__ __forceinline__ int ev_len(const EvictArgs& a, int b) {
  return min(max(a.lens[b], 0), (int)min((long long)a.max_pages * PG, (long long)a.columns));
}

// Unsigned keys in the order of the weights: both zeros equal, a NaN above everything.
__device__ __forceinline__ uint32_t ev_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);   // (-0 + 0 = 0)
  return w != w ? 0xffffffffu : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr int EV_THREADS = 1024, EV_WARPS = EV_THREADS / 32, EV_CLUSTER = 8;
constexpr int EV_COPIES = 8;   // of the first pass' 512 bins, of which a row's weights share a few: lanes meet less often
constexpr int EV_SLICE = 32768;   // keys of a slice that are kept in shared memory (128 KB); longer ones are read again

struct EvShared {
  alignas(16) uint32_t copies[512 * EV_COPIES];
  alignas(16) uint32_t bins[512 + 4096 + 2048];   // of the three passes
  uint32_t warp_sum[EV_WARPS];
  uint32_t prefix, need;     // the selected key's leading bits, how many of the keys with them are still wanted
  uint32_t settled;          // as many as there are of them
  uint32_t above[EV_WARPS], equal[EV_WARPS];   // kept for sure and undecided, of each warp's part
  uint32_t all_above, all_equal;
};

__global__ void __launch_bounds__(EV_THREADS, 1) evict_select_kernel(EvictArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ EvShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const long long row = blockIdx.x / C;
  const int b = (int)(row / a.Hkv), h = (int)(row - (long long)b * a.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  const int n = ev_len(a, b);
  int32_t* origin = a.origin + row * a.keep;
  if (n <= a.keep) {   // (the same for the whole cluster)
    for (int j = rank * EV_THREADS + threadIdx.x; j < a.keep; j += C * EV_THREADS) origin[j] = j < n ? j : -1;
    return;
  }
  const float* w = a.weights + b * a.ws + h * a.wh;
  const int lo = a.first, hi = n - a.recent;   // tokens that compete
  const int per = ((hi - lo + C - 1) / C + 31) / 32 * 32;
  const int s0 = min(hi, lo + rank * per), s1 = min(hi, s0 + per), sn = s1 - s0;   // this CTA's slice
  const bool held = per <= EV_SLICE;
  const int want = a.keep - a.first - a.recent;
  if (held) {
#pragma unroll 8
    for (int i = threadIdx.x; i < sn; i += EV_THREADS) keys[i] = ev_key(w[s0 + i]);
  }
  for (int j = rank * EV_THREADS + threadIdx.x; j < a.first; j += C * EV_THREADS) origin[j] = j;
  for (int j = rank * EV_THREADS + threadIdx.x; j < a.recent; j += C * EV_THREADS) origin[a.keep - a.recent + j] = hi + j;
  if (want == 0) return;
  auto key_at = [&](int i) { return held ? keys[i] : ev_key(w[s0 + i]); };
  {
    uint4* zero = reinterpret_cast<uint4*>(sh.copies);   // and the bins behind them
    static_assert(offsetof(EvShared, bins) == sizeof(sh.copies), "");
    for (int i = threadIdx.x; i < (int)((sizeof(sh.copies) + sizeof(sh.bins)) / 16); i += EV_THREADS) zero[i] = make_uint4(0, 0, 0, 0);
  }
  if (threadIdx.x == 0) sh.prefix = 0, sh.need = want, sh.settled = 0;
  int shift = 32;   // bits of a key that are not looked at yet
  cluster.sync();
  constexpr int SHIFT[4] = {32, 23, 11, 0}, FIRST[3] = {0, 512, 512 + 4096};
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = SHIFT[pass] - SHIFT[pass + 1], bins = 1 << bits;
    uint32_t* hist = sh.bins + FIRST[pass];
    uint32_t* sums = cluster.map_shared_rank(hist, 0);   // the first CTA's
    const uint32_t prefix = sh.prefix;
#pragma unroll 4
    for (int i = threadIdx.x; i < sn; i += EV_THREADS) {
      const uint32_t k = key_at(i);
      if (pass == 0) atomicAdd(&sh.copies[EV_COPIES * (k >> SHIFT[1]) + lane % EV_COPIES], 1u);
      else if ((k >> (SHIFT[pass] & 31)) == prefix) atomicAdd(&hist[(k >> SHIFT[pass + 1]) & (bins - 1)], 1u);
    }
    // what is not 0 to the first CTA (that every CTA read the others' took 5 us a pass)
    if (pass == 0) {
      __syncthreads();
      if (threadIdx.x < bins) {
        const uint4 x = reinterpret_cast<const uint4*>(sh.copies)[2 * threadIdx.x], y = reinterpret_cast<const uint4*>(sh.copies)[2 * threadIdx.x + 1];
        const uint32_t sum = x.x + x.y + x.z + x.w + y.x + y.y + y.z + y.w;
        if (sum) atomicAdd(sums + threadIdx.x, sum);
      }
    } else if (rank != 0) {
      __syncthreads();
      for (int i = threadIdx.x; i < bins; i += EV_THREADS)
        if (hist[i]) atomicAdd(sums + i, hist[i]);
    }
    cluster.sync();
    if (rank == 0) {   // the bin with the wanted key, from the largest keys down: four bins per thread
      uint32_t c[4] = {0, 0, 0, 0};
      if (4 * threadIdx.x < bins) {
        const uint4 x = reinterpret_cast<const uint4*>(hist)[bins / 4 - 1 - threadIdx.x];
        c[0] = x.w, c[1] = x.z, c[2] = x.y, c[3] = x.x;
      }
      uint32_t inc = c[0] + c[1] + c[2] + c[3];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) sh.warp_sum[warp] = inc;
      const uint32_t need = sh.need;
      __syncthreads();   // (need has been read)
      uint32_t before = inc - c[0] - c[1] - c[2] - c[3] + __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_sum[lane] : 0u);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (before < need && need <= before + c[k]) {
          for (int r = 0; r < C; ++r) {
            EvShared* to = cluster.map_shared_rank(&sh, r);
            to->prefix = (prefix << bits) | (uint32_t)(bins - 1 - (4 * (int)threadIdx.x + k));
            to->need = need - before;
            to->settled = need == before + c[k];
          }
        }
        before += c[k];
      }
    }
    cluster.sync();
    shift = SHIFT[pass + 1];
    if (sh.settled) break;   // (all of the keys with these bits are kept)
  }
  // keys whose leading bits lie above the selected ones are kept, and the first `need` of those with the same
  const uint32_t sel = sh.prefix, need = sh.need;
  const int part = ((sn + EV_WARPS - 1) / EV_WARPS + 31) / 32 * 32, p0 = min(sn, warp * part), p1 = min(sn, p0 + part);
  uint32_t above = 0, equal = 0;
#pragma unroll 4
  for (int i = p0; i < p1; i += 32) {
    const bool in = i + lane < p1;
    const uint32_t k = in ? key_at(i + lane) >> shift : 0u;
    above += __popc(__ballot_sync(0xffffffffu, in && k > sel));
    equal += __popc(__ballot_sync(0xffffffffu, in && k == sel));
  }
  if (lane == 0) sh.above[warp] = above, sh.equal[warp] = equal;
  __syncthreads();
  if (warp == 0) {
    const uint32_t x = __reduce_add_sync(0xffffffffu, sh.above[lane]), y = __reduce_add_sync(0xffffffffu, sh.equal[lane]);
    if (lane == 0) sh.all_above = x, sh.all_equal = y;
  }
  cluster.sync();
  // above and equal before this warp's part: in the CTAs before (a lane each) and in the warps before
  const EvShared* other = cluster.map_shared_rank(&sh, min(lane, C - 1));
  uint32_t x = lane < rank ? other->all_above : 0u, y = lane < rank ? other->all_equal : 0u;
  if (lane < warp) x += sh.above[lane], y += sh.equal[lane];
  x = __reduce_add_sync(0xffffffffu, x), y = __reduce_add_sync(0xffffffffu, y);
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
  for (int i = p0; i < p1; i += 32) {
    const bool in = i + lane < p1;
    const uint32_t k = in ? key_at(i + lane) >> shift : 0u;
    const uint32_t gt = __ballot_sync(0xffffffffu, in && k > sel), eq = __ballot_sync(0xffffffffu, in && k == sel);
    const uint32_t eq_before = y + __popc(eq & below);
    if (in && (k > sel || (k == sel && eq_before < need)))
      origin[a.first + x + __popc(gt & below) + min(eq_before, need)] = s0 + i + lane;
    x += __popc(gt), y += __popc(eq);
  }
  cluster.sync();   // no CTA leaves while its shared memory may be read
}

// Token at place p of one group's value scales (the inverse of vscale_at).
__device__ __forceinline__ int vscale_token(int p) { return ((p >> 4) & 3) << 1 | ((p >> 2) & 3) << 4 | ((p >> 1) & 1) << 3 | (p & 1); }

constexpr int MV_THREADS = 128;
template <int HD>
__global__ void __launch_bounds__(MV_THREADS) evict_move_kernel(EvictArgs a, long long units) {
  using L = Page<HD>;
  constexpr int G = L::G, CHUNKS = L::ROW / 16;   // 16-byte pieces of a row of codes
  __shared__ const unsigned char* from[PG];       // page of each token, NULL: none
  __shared__ unsigned char at[PG];                // its token there
  const int per = (a.keep + PG - 1) / PG;
  pdl_trigger();
  pdl_wait();
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    // the heads of a page, then the next page: neighbouring blocks write neighbouring memory
    const int b = (int)(u / ((long long)per * a.Hkv));
    const int r = (int)(u - (long long)b * per * a.Hkv), j = r / a.Hkv, h = r - j * a.Hkv;
    const int n = ev_len(a, b), m = min(n, a.keep), t0 = j * PG;
    const int32_t* origin = a.origin + ((long long)b * a.Hkv + h) * a.keep;
    if (j == 0 && h == 0 && threadIdx.x == 0) a.new_lens[b] = m;
    __syncthreads();
    if (threadIdx.x < PG && t0 + threadIdx.x < a.keep) {
      const int t = t0 + threadIdx.x, o = t < m ? origin[t] : -1;
      const int page = o >= 0 ? a.table[b * a.table_stride + o / PG] : -1;
      from[threadIdx.x] = page >= 0 && page < a.n_pages ? a.pages + ((size_t)page * a.Hkv + h) * L::BYTES : nullptr;
      at[threadIdx.x] = (unsigned char)(o & (PG - 1));
      if (a.new_weights) a.new_weights[b * a.nws + h * a.nwh + t] = o >= 0 ? a.weights[b * a.ws + h * a.wh + o] : 0.f;
    }
    __syncthreads();
    const int live = min(PG, m - t0), dest = live > 0 ? a.new_table[b * a.new_stride + j] : -1;
    if (dest < 0 || dest >= a.to_pages) continue;
    unsigned char* to = a.to + ((size_t)dest * a.Hkv + h) * L::BYTES;
    // codes of keys and values
    for (int e = threadIdx.x; e < live * CHUNKS; e += MV_THREADS) {
      const int t = e / CHUNKS, c = 16 * (e % CHUNKS), i = at[t];
      const unsigned char* p = from[t];
      uint4 k = make_uint4(0, 0, 0, 0), v = k;
      if (p) k = *reinterpret_cast<const uint4*>(p + i * L::ROW + c), v = *reinterpret_cast<const uint4*>(p + L::VC + vcode_at<HD>(i, c));
      *reinterpret_cast<uint4*>(to + t * L::ROW + c) = k;
      *reinterpret_cast<uint4*>(to + L::VC + vcode_at<HD>(t, c)) = v;
    }
    // scales and offsets: of a key's groups side by side, of values by group
    for (int e = threadIdx.x; e < 2 * live; e += MV_THREADS) {
      const int t = e >> 1, o = (e & 1) ? L::KO : L::KS, i = at[t];
      const unsigned char* p = from[t];
      if constexpr (G == 4) *reinterpret_cast<uint2*>(to + o + t * 2 * G) = p ? *reinterpret_cast<const uint2*>(p + o + i * 2 * G) : make_uint2(0, 0);
      else *reinterpret_cast<uint32_t*>(to + o + t * 2 * G) = p ? *reinterpret_cast<const uint32_t*>(p + o + i * 2 * G) : 0u;
    }
    for (int e = threadIdx.x; e < G * PG; e += MV_THREADS) {
      const int g = e / PG, t = vscale_token(e % PG);
      if (t >= live) continue;
      const unsigned char* p = from[t];
      const int i = 2 * (g * PG + vscale_at(at[t]));
      unsigned short s = 0, o = 0;
      if (p) s = *reinterpret_cast<const unsigned short*>(p + L::VS + i), o = *reinterpret_cast<const unsigned short*>(p + L::VO + i);
      *reinterpret_cast<unsigned short*>(to + L::VS + 2 * e) = s;
      *reinterpret_cast<unsigned short*>(to + L::VO + 2 * e) = o;
    }
  }
}

// CTAs per row: more for rows that can be longer, eight (the portable most) at most.  By the room for columns, as lengths are on the
// device: four sequences of 1100 tokens 10.9 us with 1152 columns and 25.4 with 131072; one of 16384 15.8 and 16.2.
int ev_cluster(int columns) { return columns <= 4096 ? 1 : columns <= 16384 ? 4 : EV_CLUSTER; }

kvq_status evict_impl(const void* pages, int n_pages, const int32_t* table, int64_t table_stride, int max_pages, const int32_t* lens,
                      int B, int Hkv, int hd, const float* weights, int64_t ws, int64_t wh, int columns, int keep, int first,
                      int recent, void* to, int to_pages, const int32_t* new_table, int64_t new_stride, int new_pages,
                      int32_t* new_lens, int32_t* origin, float* new_weights, int64_t nws, int64_t nwh, void* stream) {
  const char* fn = "kvq_paged_evict";
  auto bad = [&](const char* what) { return paged_fail(KVQ_ERR_INVALID, fn, what); };
  if (hd != 64 && hd != 128) return bad("head_dim must be 64 or 128");
  if (B < 0 || B > 2048) return bad("batch must be in 0..2048");
  if (Hkv < 1 || Hkv > MAX_KV_HEADS) return bad("n_kv_heads must be in 1..4096");
  if (n_pages < 1 || n_pages > (1 << 25) || to_pages < 1 || to_pages > (1 << 25)) return bad("n_pages and new_n_pages must be in 1..33554432");
  if (max_pages < 1 || max_pages > (1 << 24) || (long long)B * max_pages >= (1ll << 30))
    return bad("max_pages must be in 1..16777216 and batch * max_pages below 2^30");
  if (table_stride < 0 || new_stride < 0 || ws < 0 || wh < 0) return bad("strides must be >= 0");
  if (columns < 1) return bad("weights need a column at least");
  if (new_pages < 1 || keep < 1 || (keep + PG - 1) / PG > new_pages) return bad("keep must be in 1..64 new_max_pages");
  if (first < 0 || recent < 0 || (long long)first + recent > keep) return bad("first and recent must be >= 0, and keep at most together");
  if (B == 0) return KVQ_OK;
  if (B > 1 && new_stride < (keep + PG - 1) / PG) return bad("new_table: rows must not overlap");
  if (new_table == table) return bad("new_table must not be page_table");
  if (new_lens == lens) return bad("new_lens must not be seq_lens");
  if (new_weights) {
    if (nws < 0 || nwh < 0 || rows_overlap(B, Hkv, nws, nwh, keep)) return bad("new_weights: rows must not overlap");
    if (new_weights == weights) return bad("new_weights must not be weights");
  }
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return paged_cuda_fail(e, fn, "no current CUDA device");
  if (kvq_status s = check_buffer(pages, dev, 16, fn, "pages")) return s;
  if (kvq_status s = check_buffer(table, dev, 4, fn, "page_table")) return s;
  if (kvq_status s = check_buffer(lens, dev, 4, fn, "seq_lens")) return s;
  if (kvq_status s = check_buffer(weights, dev, 4, fn, "weights")) return s;
  if (kvq_status s = check_buffer(to, dev, 16, fn, "new_pages")) return s;
  if (kvq_status s = check_buffer(new_table, dev, 4, fn, "new_table")) return s;
  if (kvq_status s = check_buffer(new_lens, dev, 4, fn, "new_lens")) return s;
  if (kvq_status s = check_buffer(origin, dev, 4, fn, "origin")) return s;
  if (new_weights)
    if (kvq_status s = check_buffer(new_weights, dev, 4, fn, "new_weights")) return s;
  EvictArgs a{static_cast<const unsigned char*>(pages), static_cast<unsigned char*>(to), table, lens, new_table, new_lens, origin,
              weights, new_weights, table_stride, new_stride, ws, wh, nws, nwh, n_pages, to_pages, max_pages, columns, B, Hkv,
              keep, first, recent};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int most = (int)std::min<long long>((long long)max_pages * PG, columns), C = ev_cluster(most);
  // (always the largest: the limit belongs to the function and is every host thread's)
  if (cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, EV_SLICE * 4))
    return paged_cuda_fail(e, fn, "shared memory");
  const int per = ((most + C - 1) / C + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)B * Hkv * C));
  cfg.blockDim = dim3(EV_THREADS);
  cfg.dynamicSmemBytes = 4 * (size_t)std::min(per, EV_SLICE);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a)) return paged_cuda_fail(e, fn, "launch");
  const long long units = (long long)B * Hkv * ((keep + PG - 1) / PG);
  const dim3 grid((unsigned)std::min<long long>(units, 1 << 20));
  cudaError_t e = launch_dependent(hd == 128 ? evict_move_kernel<128> : evict_move_kernel<64>, grid, dim3(MV_THREADS), 0, st, a, units);
  if (e != cudaSuccess) return paged_cuda_fail(e, fn, "launch");
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

extern "C" kvq_status kvq_paged_evict(const void* pages, int n_pages, const int32_t* page_table, int64_t table_stride, int max_pages,
                                      const int32_t* seq_lens, int batch, int n_kv_heads, int head_dim, const float* weights,
                                      int64_t weights_seq_stride, int64_t weights_head_stride, int n_columns, int keep,
                                      int first, int recent, void* new_pages, int new_n_pages, const int32_t* new_table,
                                      int64_t new_table_stride, int new_max_pages, int32_t* new_lens, int32_t* origin,
                                      float* new_weights, int64_t new_weights_seq_stride, int64_t new_weights_head_stride,
                                      void* stream) try {
  return kvq::evict_impl(pages, n_pages, page_table, table_stride, max_pages, seq_lens, batch, n_kv_heads, head_dim, weights,
                         weights_seq_stride, weights_head_stride, n_columns, keep, first, recent, new_pages, new_n_pages,
                         new_table, new_table_stride, new_max_pages, new_lens, origin, new_weights, new_weights_seq_stride,
                         new_weights_head_stride, stream);
} catch (...) {
  return KVQ_ERR_HOST_OOM;
}
