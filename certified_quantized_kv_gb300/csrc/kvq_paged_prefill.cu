// kvq_paged_prefill.cu -- attention of prompts and chunks over the paged 4-bit cache:
//   out = softmax(scale q k^T) v over the tokens that each query sees,
// for chunks of any length, packed one behind the other.  The rows of a (sequence, KV head) are its chunk's tokens times
// the query heads of that KV head; a block takes 16 of them and goes over the pages once with a running maximum and sum.
#include <algorithm>
#include <cmath>
#include <string>

#include "kvq.h"
#include "kvq_launch.h"
#include "kvq_paged.cuh"

namespace kvq {

namespace {

struct PpArgs {
  const void* q;
  const unsigned char* pages;
  const int32_t *starts, *table, *lens;
  void* out;
  float* lse;
  long long qt, qh, table_stride;
  int n_pages, max_pages, T, B, Hq, Hkv, n_rep, window;
  float scale_log2;
  bool bf16, causal;
};

constexpr int PP_THREADS = 128, PP_ROWS = 16;

template <int HD>
__global__ void __launch_bounds__(PP_THREADS) paged_prefill_kernel(PpArgs a) {
  using L = Page<HD>;
  constexpr int G = L::G, PER = PP_ROWS * HD / PP_THREADS, LANES = HD / PER;   // channels of a thread, threads of a row
  __shared__ float q[PP_ROWS][HD];
  __shared__ float x[PG][HD + 1];
  __shared__ float s[PP_ROWS][PG];
  __shared__ float alpha[PP_ROWS], total[PP_ROWS], top[PP_ROWS];
  pdl_trigger();
  pdl_wait();
  const int g = blockIdx.y;
  // this block's sequence and tile
  int b = 0, first = 0, rows = 0;
  long long tile = blockIdx.x;
  for (; b < a.B; ++b) {
    first = min(max(a.starts[b], 0), a.T);
    rows = (min(max(a.starts[b + 1], first), a.T) - first) * a.n_rep;
    const int tiles = (rows + PP_ROWS - 1) / PP_ROWS;
    if (tile < tiles) break;
    tile -= tiles;
  }
  if (b == a.B) return;
  const int new_tokens = rows / a.n_rep, len = min(max(a.lens[b], 0), a.max_pages * PG);
  const int r0 = (int)tile * PP_ROWS, rn = min(PP_ROWS, rows - r0);
  auto hi_of = [&](int i) { return a.causal ? max(0, len - new_tokens + 1 + i) : len; };
  auto lo_of = [&](int i) { return a.window ? max(0, hi_of(i) - a.window) : 0; };
  auto row_at = [&](int r, long long ts, long long hs) {
    const int i = (r0 + r) / a.n_rep, h = g * a.n_rep + (r0 + r) % a.n_rep;
    return (first + i) * ts + h * hs;
  };
  for (int e = threadIdx.x; e < PP_ROWS * HD; e += PP_THREADS) {
    const int r = e / HD, c = e % HD;
    q[r][c] = r < rn ? elem_to_f(a.q, row_at(r, a.qt, a.qh) + c, a.bf16) : 0.f;
  }
  if (threadIdx.x < PP_ROWS) top[threadIdx.x] = -INFINITY, total[threadIdx.x] = 0.f;
  const int row = threadIdx.x / LANES, c0 = threadIdx.x % LANES;   // this thread's row and channels c0 + LANES k
  float acc[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) acc[k] = 0.f;
  const int t_lo = lo_of(r0 / a.n_rep), t_hi = hi_of((r0 + rn - 1) / a.n_rep);
  for (int tok0 = t_lo / PG * PG; tok0 < t_hi; tok0 += PG) {
    const int page = a.table[b * a.table_stride + tok0 / PG];
    if (page < 0 || page >= a.n_pages) continue;
    const unsigned char* pg = a.pages + ((size_t)page * a.Hkv + g) * L::BYTES;
    const int live = min(PG, t_hi - tok0);   // what lies behind is not read
    __syncthreads();
    for (int e = threadIdx.x; e < live * HD; e += PP_THREADS) {
      const int t = e / HD, c = e % HD, gr = c / 32, j = c % 32;
      const int code = pg[t * L::ROW + (j / 8) * 4 * G + 4 * gr + (j % 8) / 2] >> (4 * (j & 1)) & 15;
      const __half* sc = reinterpret_cast<const __half*>(pg + L::KS) + t * G + gr;
      x[t][c] = fmaf((float)code, __half2float(sc[0]), __half2float(sc[L::SCALES / 2]));
    }
    __syncthreads();
    for (int e = threadIdx.x; e < PP_ROWS * PG; e += PP_THREADS) {
      const int r = e / PG, t = e % PG, i = (r0 + r) / a.n_rep;
      float d = -INFINITY;
      if (r < rn && tok0 + t >= lo_of(i) && tok0 + t < hi_of(i)) {
        d = 0.f;
        for (int c = 0; c < HD; ++c) d = fmaf(q[r][c], x[t][c], d);
        d *= a.scale_log2;
      }
      s[r][t] = d;
    }
    __syncthreads();
    if (threadIdx.x < PP_ROWS) {
      float m = top[threadIdx.x];
      for (int t = 0; t < PG; ++t) m = fmaxf(m, s[threadIdx.x][t]);
      const float ref = m == -INFINITY ? 0.f : m;
      alpha[threadIdx.x] = exp2f(top[threadIdx.x] - ref);
      float sum = 0.f;
      for (int t = 0; t < PG; ++t) {
        const float p = exp2f(s[threadIdx.x][t] - ref);
        s[threadIdx.x][t] = p;
        sum += p;
      }
      total[threadIdx.x] = fmaf(total[threadIdx.x], alpha[threadIdx.x], sum);
      top[threadIdx.x] = m;
    }
    for (int e = threadIdx.x; e < live * HD; e += PP_THREADS) {
      const int t = e / HD, c = e % HD, gr = c / 32, j = c % 32;
      const int code = pg[L::VC + vcode_at<HD>(t, (j / 4) * 2 * G + 2 * gr + (j % 4) / 2)] >> (4 * (j & 1)) & 15;
      const __half* sc = reinterpret_cast<const __half*>(pg + L::VS) + gr * PG + vscale_at(t);
      x[t][c] = fmaf((float)code, __half2float(sc[0]), __half2float(sc[L::SCALES / 2]));
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PER; ++k) acc[k] *= alpha[row];
    for (int t = 0; t < live; ++t) {
      const int i = (r0 + row) / a.n_rep;
      // (a token that the row does not see may hold anything)
      if (tok0 + t < lo_of(i) || tok0 + t >= hi_of(i)) continue;
      const float p = s[row][t];
#pragma unroll
      for (int k = 0; k < PER; ++k) acc[k] = fmaf(p, x[t][c0 + LANES * k], acc[k]);
    }
  }
  __syncthreads();
  if (row >= rn) return;
  const float l = total[row], inv = l == 0.f ? 0.f : 1.f / l;
  const long long at = row_at(row, a.Hq, 1);
  for (int k = 0; k < PER; ++k) {
    const float y = acc[k] * inv;
    unsigned short* o = static_cast<unsigned short*>(a.out) + at * HD + c0 + LANES * k;
    *o = (unsigned short)(f2_to_pair(y, 0.f, a.bf16) & 0xffffu);
  }
  if (a.lse && c0 == 0) a.lse[at] = l == 0.f ? -INFINITY : (top[row] + log2f(l)) * 0.69314718055994531f;
}

const char* pp_shape_error(int T, int B, int Hq, int Hkv, int hd) {
  if (T < 0 || T > (1 << 24)) return "n_tokens must be in 0..16777216";
  if (B < 0 || B > 2048) return "batch must be in 0..2048";
  if (Hkv < 1 || Hkv > MAX_KV_HEADS) return "n_kv_heads must be in 1..4096";
  if (Hq < 1 || Hq % Hkv != 0 || Hq / Hkv > 64) return "n_q_heads / n_kv_heads must be an integer in 1..64";
  if (hd != 64 && hd != 128) return "head_dim must be 64 or 128";
  return nullptr;
}

size_t pp_bytes(int T, int B, int Hq, int Hkv, int hd) { return 16; }

kvq_status prefill_impl(int dtype, const void* q, int64_t qt, int64_t qh, const int32_t* starts, int T, const void* pages, int n_pages,
                        const int32_t* table, int64_t table_stride, int max_pages, const int32_t* lens, int B, int Hq, int Hkv,
                        int hd, int causal, int window, float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                        void* stream) {
  const char* fn = "kvq_paged_prefill";
  auto bad = [&](const char* what) { return paged_fail(KVQ_ERR_INVALID, fn, what); };
  if (dtype != KVQ_F16 && dtype != KVQ_BF16) return bad("dtype must be KVQ_F16 or KVQ_BF16");
  if (const char* msg = pp_shape_error(T, B, Hq, Hkv, hd)) return bad(msg);
  if (n_pages < 1 || n_pages > (1 << 25)) return bad("n_pages must be in 1..33554432");
  if (max_pages < 1 || max_pages > (1 << 24) || (long long)B * max_pages >= (1ll << 30))
    return bad("max_pages must be in 1..16777216 and batch * max_pages below 2^30");
  if (table_stride < 0) return bad("table_stride must be >= 0");
  if (causal != 0 && causal != 1) return bad("causal must be 0 or 1");
  if (window < 0 || (window && !causal)) return bad("window must be >= 0, and 0 unless causal");
  const float scale_log2 = (scale != 0.f ? scale : 1.f / std::sqrt((float)hd)) * LOG2E_F;
  if (!std::isfinite(scale_log2)) return bad("scale * log2(e) must be finite");
  if (B == 0 || T == 0) return KVQ_OK;
  if (q == out) return bad("out must not be q");
  if (kvq_status s = check_strides(qt, qh, fn, "q")) return s;
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return paged_cuda_fail(e, fn, "no current CUDA device");
  if (kvq_status s = check_buffer(q, dev, 16, fn, "q")) return s;
  if (kvq_status s = check_buffer(starts, dev, 4, fn, "q_starts")) return s;
  if (kvq_status s = check_buffer(pages, dev, 16, fn, "pages")) return s;
  if (kvq_status s = check_buffer(table, dev, 4, fn, "page_table")) return s;
  if (kvq_status s = check_buffer(lens, dev, 4, fn, "seq_lens")) return s;
  if (kvq_status s = check_buffer(out, dev, 16, fn, "out")) return s;
  if (lse)
    if (kvq_status s = check_buffer(lse, dev, 4, fn, "lse")) return s;
  if (kvq_status s = check_buffer(workspace, dev, 16, fn, "workspace")) return s;
  if (workspace_bytes < pp_bytes(T, B, Hq, Hkv, hd)) return bad("workspace smaller than kvq_paged_prefill_workspace reports");
  PpArgs a = {};
  a.q = q, a.pages = static_cast<const unsigned char*>(pages), a.starts = starts, a.table = table, a.lens = lens, a.out = out;
  a.lse = lse, a.qt = qt, a.qh = qh, a.table_stride = table_stride, a.n_pages = n_pages, a.max_pages = max_pages, a.T = T, a.B = B;
  a.Hq = Hq, a.Hkv = Hkv, a.n_rep = Hq / Hkv, a.window = std::min(window, 1 << 30), a.scale_log2 = scale_log2;
  a.bf16 = dtype == KVQ_BF16, a.causal = causal != 0;
  const dim3 grid((unsigned)(((long long)T * a.n_rep + PP_ROWS - 1) / PP_ROWS + B), (unsigned)Hkv);
  const cudaError_t e = launch_dependent(hd == 128 ? paged_prefill_kernel<128> : paged_prefill_kernel<64>, grid, dim3(PP_THREADS), 0,
                                         static_cast<cudaStream_t>(stream), a);
  if (e != cudaSuccess) return paged_cuda_fail(e, fn, "launch");
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

extern "C" kvq_status kvq_paged_prefill_workspace(int n_tokens, int batch, int n_q_heads, int n_kv_heads, int head_dim,
                                                  size_t* bytes) try {
  const char* fn = "kvq_paged_prefill_workspace";
  if (!bytes) return kvq::paged_fail(KVQ_ERR_INVALID, fn, "NULL output");
  if (const char* msg = kvq::pp_shape_error(n_tokens, batch, n_q_heads, n_kv_heads, head_dim))
    return kvq::paged_fail(KVQ_ERR_INVALID, fn, msg);
  *bytes = kvq::pp_bytes(n_tokens, batch, n_q_heads, n_kv_heads, head_dim);
  return KVQ_OK;
} catch (...) {
  return KVQ_ERR_HOST_OOM;
}

extern "C" kvq_status kvq_paged_prefill(int dtype, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                        const int32_t* q_starts, int n_tokens, const void* pages, int n_pages,
                                        const int32_t* page_table, int64_t table_stride, int max_pages, const int32_t* seq_lens,
                                        int batch, int n_q_heads, int n_kv_heads, int head_dim, int causal, int window, float scale,
                                        void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) try {
  return kvq::prefill_impl(dtype, q, q_token_stride, q_head_stride, q_starts, n_tokens, pages, n_pages, page_table, table_stride,
                           max_pages, seq_lens, batch, n_q_heads, n_kv_heads, head_dim, causal, window, scale, out, lse, workspace,
                           workspace_bytes, stream);
} catch (...) {
  return KVQ_ERR_HOST_OOM;
}
