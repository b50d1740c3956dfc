// kvq_paged_attn.cu -- decode attention over the paged 4-bit cache.
//
// With k^ = o + s code per group g of 32 channels,
//   score_t = sum_g s_tg (q_g . code_tg) + o_tg sum(q_g),   out = sum_t p_t (o_tg + s_tg code_tc) / sum_t p_t
// over the tokens that a query sees, p_t = exp(score_t - m).
#include <algorithm>
#include <cmath>
#include <string>

#include "kvq.h"
#include "kvq_launch.h"
#include "kvq_paged.cuh"

namespace kvq {

namespace {

struct PaArgs {
  const void* q;
  const unsigned char* pages;
  const int32_t *table, *lens;
  void* out;
  float* lse;
  long long qt, qh, table_stride;
  int n_pages, max_pages, B, Q, Hq, Hkv, n_rep, window;
  float scale;
  bool bf16;
};

// One warp per (sequence, query token, query head): lanes split the tokens of a page for
// the scores and the channels for the sums.
template <int HD>
__global__ void __launch_bounds__(128) paged_attention_kernel(PaArgs a) {
  using L = Page<HD>;
  __shared__ float qs[4][HD], ps[4][PG];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long n = (long long)a.B * a.Q * a.Hq;
  for (long long u = blockIdx.x * 4ll + warp; u < n; u += gridDim.x * 4ll) {
    const int h = (int)(u % a.Hq);
    const long long tok = u / a.Hq;
    const int b = (int)(tok / a.Q), i = (int)(tok % a.Q), g = h / a.n_rep;
    const int len = min(max(a.lens[b], 0), a.max_pages * PG);
    const int end = max(0, len - a.Q + 1 + i), begin = a.window ? max(0, end - a.window) : 0;
    __syncwarp();
    for (int c = lane; c < HD; c += 32) qs[warp][c] = elem_to_f(a.q, (size_t)(tok * a.qt + h * a.qh) + c, a.bf16);
    __syncwarp();
    float m = -INFINITY, l = 0.f, acc[L::G];
    for (int j = 0; j < L::G; ++j) acc[j] = 0.f;
    for (int pg = begin / PG; pg * PG < end; ++pg) {
      const int id = a.table[b * a.table_stride + pg];
      if (id < 0 || id >= a.n_pages) continue;
      const unsigned char* page = a.pages + ((size_t)id * a.Hkv + g) * L::BYTES;
      auto h16 = [&](int off, int e) { return __half2float(reinterpret_cast<const __half*>(page + off)[e]); };
      float s[2];
      for (int r = 0; r < 2; ++r) {
        const int t = lane + 32 * r;
        s[r] = -INFINITY;
        if (pg * PG + t < begin || pg * PG + t >= end) continue;
        float x = 0.f;
        for (int c = 0; c < HD; ++c) {
          const int j = c % 32, kb = page[t * L::ROW + (j >> 3) * 4 * L::G + 4 * (c / 32) + ((j & 7) >> 1)];
          x = fmaf(qs[warp][c], fmaf((float)((kb >> (4 * (c & 1))) & 15), h16(L::KS, t * L::G + c / 32), h16(L::KO, t * L::G + c / 32)), x);
        }
        s[r] = x * a.scale;
      }
      const float mn = fmaxf(m, warp_max(fmaxf(s[0], s[1])));
      if (mn == -INFINITY) continue;
      const float alpha = expf(m - mn), p0 = expf(s[0] - mn), p1 = expf(s[1] - mn);
      m = mn;
      l = l * alpha + warp_sum(p0 + p1);
      __syncwarp();
      ps[warp][lane] = p0;
      ps[warp][lane + 32] = p1;
      __syncwarp();
      for (int j = 0; j < L::G; ++j) {
        float x = 0.f;
        for (int t = 0; t < PG; ++t) {
          if (pg * PG + t < begin || pg * PG + t >= end) continue;
          const int e = j * PG + vscale_at(t);
          const int vb = page[L::VC + vcode_at<HD>(t, (lane >> 2) * 2 * L::G + 2 * j + ((lane & 3) >> 1))];
          x = fmaf(ps[warp][t], fmaf((float)((vb >> (4 * (lane & 1))) & 15), h16(L::VS, e), h16(L::VO, e)), x);
        }
        acc[j] = acc[j] * alpha + x;
      }
      __syncwarp();
    }
    for (int j = 0; j < L::G; ++j) f_to_elem(a.out, (size_t)u * HD + 32 * j + lane, l > 0.f ? acc[j] / l : 0.f, a.bf16);
    if (a.lse && lane == 0) a.lse[u] = l > 0.f ? m + logf(l) : -INFINITY;
  }
}

const char* shape_error(int B, int Q, int Hq, int Hkv, int hd) {
  if (B < 0 || B > 4096) return "batch must be in 0..4096";
  if (Q < 1 || Q > 64) return "n_q_tokens must be in 1..64";
  if (Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || Hq / Hkv > 64) return "n_q_heads / n_kv_heads must be an integer in 1..64";
  if (hd != 64 && hd != 128) return "head_dim must be 64 or 128";
  return nullptr;
}

size_t workspace_bytes_of(int, int, int, int, int) { return 16; }

kvq_status attention_impl(int dtype, const void* q, int64_t qt, int64_t qh, const void* pages, int n_pages,
                          const int32_t* table, int64_t table_stride, int max_pages, const int32_t* lens, int B, int Q,
                          int Hq, int Hkv, int hd, int window, float scale, void* out, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const char* fn = "kvq_paged_attention";
  if (dtype != KVQ_F16 && dtype != KVQ_BF16) return paged_fail(KVQ_ERR_INVALID, fn, "dtype must be KVQ_F16 or KVQ_BF16");
  if (const char* msg = shape_error(B, Q, Hq, Hkv, hd)) return paged_fail(KVQ_ERR_INVALID, fn, msg);
  if (n_pages < 1 || n_pages > (1 << 25)) return paged_fail(KVQ_ERR_INVALID, fn, "n_pages must be in 1..33554432");
  if (max_pages < 1 || max_pages > (1 << 25) || (long long)B * max_pages >= (1ll << 31))
    return paged_fail(KVQ_ERR_INVALID, fn, "max_pages must be in 1..33554432 and batch * max_pages below 2^31");
  if (table_stride < 0) return paged_fail(KVQ_ERR_INVALID, fn, "table_stride must be >= 0");
  if (window < 0) return paged_fail(KVQ_ERR_INVALID, fn, "window must be >= 0");
  if (!std::isfinite(scale)) return paged_fail(KVQ_ERR_INVALID, fn, "scale must be finite");
  if (B == 0) return KVQ_OK;
  if (kvq_status s = check_strides(qt, qh, fn, "q")) return s;
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return paged_cuda_fail(e, fn, "no current CUDA device");
  if (kvq_status s = check_buffer(q, dev, 16, fn, "q")) return s;
  if (kvq_status s = check_buffer(pages, dev, 16, fn, "pages")) return s;
  if (kvq_status s = check_buffer(table, dev, 4, fn, "page_table")) return s;
  if (kvq_status s = check_buffer(lens, dev, 4, fn, "seq_lens")) return s;
  if (kvq_status s = check_buffer(out, dev, 16, fn, "out")) return s;
  if (lse)
    if (kvq_status s = check_buffer(lse, dev, 4, fn, "lse")) return s;
  if (kvq_status s = check_buffer(workspace, dev, 16, fn, "workspace")) return s;
  if (workspace_bytes < workspace_bytes_of(B, Q, Hq, Hkv, hd))
    return paged_fail(KVQ_ERR_INVALID, fn, "workspace smaller than kvq_paged_attention_workspace reports");
  PaArgs a{q, static_cast<const unsigned char*>(pages), table, lens, out, lse, qt, qh, table_stride, n_pages, max_pages,
           B, Q, Hq, Hkv, Hq / Hkv, window, scale != 0.f ? scale : 1.f / std::sqrt((float)hd), dtype == KVQ_BF16};
  const long long blocks = ((long long)B * Q * Hq + 3) / 4;
  const int grid = (int)std::min<long long>(blocks, 152 * 64);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (hd == 128) paged_attention_kernel<128><<<grid, 128, 0, st>>>(a);
  else paged_attention_kernel<64><<<grid, 128, 0, st>>>(a);
  if (cudaError_t e = cudaGetLastError()) return paged_cuda_fail(e, fn, "launch");
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

extern "C" kvq_status kvq_paged_attention_workspace(int batch, int n_q_tokens, int n_q_heads, int n_kv_heads,
                                                    int head_dim, size_t* bytes) try {
  const char* fn = "kvq_paged_attention_workspace";
  if (!bytes) return kvq::paged_fail(KVQ_ERR_INVALID, fn, "NULL output");
  if (const char* msg = kvq::shape_error(batch, n_q_tokens, n_q_heads, n_kv_heads, head_dim))
    return kvq::paged_fail(KVQ_ERR_INVALID, fn, msg);
  *bytes = kvq::workspace_bytes_of(batch, n_q_tokens, n_q_heads, n_kv_heads, head_dim);
  return KVQ_OK;
} catch (...) {
  return KVQ_ERR_HOST_OOM;
}

extern "C" kvq_status kvq_paged_attention(int dtype, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                          const void* pages, int n_pages, const int32_t* page_table,
                                          int64_t table_stride, int max_pages, const int32_t* seq_lens, int batch,
                                          int n_q_tokens, int n_q_heads, int n_kv_heads, int head_dim, int window,
                                          float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                          void* stream) try {
  return kvq::attention_impl(dtype, q, q_token_stride, q_head_stride, pages, n_pages, page_table, table_stride, max_pages,
                             seq_lens, batch, n_q_tokens, n_q_heads, n_kv_heads, head_dim, window, scale, out, lse,
                             workspace, workspace_bytes, stream);
} catch (...) {
  return KVQ_ERR_HOST_OOM;
}
