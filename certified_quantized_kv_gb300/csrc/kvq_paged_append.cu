// kvq_paged_append.cu -- tokens into the pages of the 4-bit cache (with the rotation of
// keys and queries on the way), and back out of them.
//
// Per token, KV head and group of 32 channels (x the rotated key or the value, in fp32):
//   s = fp16 rounded up of (max - min) / 15, o = fp16(min), code = clamp(rint((x - o) / s), 0, 15)
// and for the values of odd slots, counted down from the maximum,
//   s = -(fp16 rounded up of (max - min) / 15), o = fp16(max), code = clamp(rint((o - x) / |s|), 0, 15)
// so x^ = o + s code in both.  The scale is rounded up so that 15 steps span the group.
#include <string>

#include "kvq.h"
#include "kvq_launch.h"
#include "kvq_paged.cuh"

namespace kvq {

namespace {

struct AppendPagedArgs {
  const void *k, *v, *q;
  void* q_out;
  const int32_t *slots, *pos;
  unsigned char* pages;
  long long kt, kh, vt, vh, qt, qh, ot, oh;   // strides in elements
  int T, Hkv, Hq, n_pages;
  bool bf16, rotate;
};

// rotated element c of the row at element offset `row`
__device__ float rotated(const kvq_rope_plan& P, const void* x, size_t row, int c, int pos, bool bf16) {
  const float own = elem_to_f(x, row + c, bf16);
  if (c >= P.rotary_dim) return own;
  const int half = P.rotary_dim / 2;
  const int i = P.interleaved ? c >> 1 : (c < half ? c : c - half);
  const bool first = P.interleaved ? (c & 1) == 0 : c < half;
  const int other = P.interleaved ? c ^ 1 : (first ? c + half : c - half);
  const float2 cs = rope_cos_sin(pos, P.step[i], P.magnitude);
  const float o = elem_to_f(x, row + other, bf16);
  return first ? fmaf(own, cs.x, -o * cs.y) : fmaf(own, cs.x, o * cs.y);
}

// One warp per (token, head): KV heads first, then query heads; lane = channel of a group.
template <int HD>
__global__ void __launch_bounds__(128) paged_append_kernel(const __grid_constant__ kvq_rope_plan P, AppendPagedArgs a) {
  using L = Page<HD>;
  const int lane = threadIdx.x & 31;
  const long long n = (long long)a.T * (a.Hkv + a.Hq);
  for (long long u = blockIdx.x * 4ll + (threadIdx.x >> 5); u < n; u += gridDim.x * 4ll) {
    const long long t = u / (a.Hkv + a.Hq);
    const int h = (int)(u - t * (a.Hkv + a.Hq));
    const int pos = a.rotate ? a.pos[t] : 0;
    if (h >= a.Hkv) {
      const size_t in = (size_t)(t * a.qt + (h - a.Hkv) * a.qh), out = (size_t)(t * a.ot + (h - a.Hkv) * a.oh);
      float y[L::G];
      for (int g = 0; g < L::G; ++g) y[g] = rotated(P, a.q, in, 32 * g + lane, pos, a.bf16);
      __syncwarp();   // q_out may be q: every lane has read before any writes
      for (int g = 0; g < L::G; ++g) f_to_elem(a.q_out, out + 32 * g + lane, y[g], a.bf16);
      continue;
    }
    const int slot = a.slots[t];
    if (slot < 0 || slot / PG >= a.n_pages) continue;
    unsigned char* page = a.pages + ((size_t)(slot / PG) * a.Hkv + h) * L::BYTES;
    const int at = slot % PG;
    for (int kv = 0; kv < 2; ++kv)
      for (int g = 0; g < L::G; ++g) {
        const int c = 32 * g + lane;
        const size_t row = kv ? (size_t)(t * a.vt + h * a.vh) : (size_t)(t * a.kt + h * a.kh);
        float x = kv || !a.rotate ? elem_to_f(kv ? a.v : a.k, row + c, a.bf16) : rotated(P, a.k, row, c, pos, a.bf16);
        x = fminf(fmaxf(x, -65504.f), 65504.f);
        const float hi = warp_max(x), lo = -warp_max(-x);
        const bool down = kv && (at & 1);
        const __half o = __float2half_rn(down ? hi : lo);
        const float of = __half2float(o);
        const __half s = __float2half_ru(__fdiv_rn(fmaxf(down ? of - lo : hi - of, 0.f), 15.f));
        const float sf = __half2float(s), d = down ? of - x : x - of;
        const int code = sf > 0.f ? (int)fminf(fmaxf(rintf(__fdiv_rn(d, sf)), 0.f), 15.f) : 0;
        const int next = __shfl_down_sync(0xffffffffu, code, 1);
        if ((lane & 1) == 0) {
          if (kv) page[L::VC + vcode_at<HD>(at, (lane >> 2) * 2 * L::G + 2 * g + ((lane & 3) >> 1))] = code | (next << 4);
          else page[at * L::ROW + (lane >> 3) * 4 * L::G + 4 * g + ((lane & 7) >> 1)] = code | (next << 4);
        }
        if (lane == 0) {
          const int e = kv ? g * PG + vscale_at(at) : at * L::G + g;
          reinterpret_cast<__half*>(page + (kv ? L::VS : L::KS))[e] = down ? __hneg(s) : s;
          reinterpret_cast<__half*>(page + (kv ? L::VO : L::KO))[e] = o;
        }
      }
  }
}

struct GatherArgs {
  const unsigned char* pages;
  const int32_t* slots;
  void *k, *v;
  long long kt, kh, vt, vh;
  int T, Hkv, n_pages;
  bool bf16;
};

// One thread per element.
template <int HD>
__global__ void __launch_bounds__(256) paged_gather_kernel(GatherArgs a) {
  using L = Page<HD>;
  const long long n = (long long)a.T * a.Hkv * HD;
  for (long long u = blockIdx.x * 256ll + threadIdx.x; u < n; u += gridDim.x * 256ll) {
    const int c = (int)(u % HD), g = c / 32, j = c % 32;
    const long long row = u / HD, t = row / a.Hkv, h = row - t * a.Hkv;
    const int slot = a.slots[t];
    float k = 0.f, v = 0.f;
    if (slot >= 0 && slot / PG < a.n_pages) {
      const unsigned char* page = a.pages + ((size_t)(slot / PG) * a.Hkv + h) * L::BYTES;
      const int at = slot % PG;
      const int kb = page[at * L::ROW + (j >> 3) * 4 * L::G + 4 * g + ((j & 7) >> 1)];
      const int vb = page[L::VC + vcode_at<HD>(at, (j >> 2) * 2 * L::G + 2 * g + ((j & 3) >> 1))];
      const int ke = at * L::G + g, ve = g * PG + vscale_at(at), sh = 4 * (c & 1);
      auto h16 = [&](int off, int e) { return __half2float(reinterpret_cast<const __half*>(page + off)[e]); };
      k = fmaf((float)((kb >> sh) & 15), h16(L::KS, ke), h16(L::KO, ke));
      v = fmaf((float)((vb >> sh) & 15), h16(L::VS, ve), h16(L::VO, ve));
    }
    f_to_elem(a.k, (size_t)(t * a.kt + h * a.kh) + c, k, a.bf16);
    f_to_elem(a.v, (size_t)(t * a.vt + h * a.vh) + c, v, a.bf16);
  }
}

constexpr int MAX_GRID = 152 * 64;

int grid_of(long long blocks) { return (int)(blocks < MAX_GRID ? blocks : MAX_GRID); }

// checks shared by append and gather
kvq_status check_common(const char* fn, int dtype, int T, int Hkv, int hd, int n_pages) {
  if (dtype != KVQ_F16 && dtype != KVQ_BF16) return paged_fail(KVQ_ERR_INVALID, fn, "dtype must be KVQ_F16 or KVQ_BF16");
  if (hd != 64 && hd != 128) return paged_fail(KVQ_ERR_INVALID, fn, "head_dim must be 64 or 128");
  if (T < 0) return paged_fail(KVQ_ERR_INVALID, fn, "n_tokens must be >= 0");
  if (Hkv < 1) return paged_fail(KVQ_ERR_INVALID, fn, "n_kv_heads must be >= 1");
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
    if (kvq_status s = check_buffer(q, dev, 16, fn, "q")) return s;
    if (kvq_status s = check_buffer(q_out, dev, 16, fn, "q_out")) return s;
  }
  AppendPagedArgs a{k,  v,  q,  q_out, slots, positions, static_cast<unsigned char*>(pages),
                    kt, kh, vt, vh,    qt,    qh,        ot, oh, T, Hkv, q ? Hq : 0, n_pages,
                    dtype == KVQ_BF16, plan != nullptr};
  kvq_rope_plan none = {};
  const int grid = grid_of(((long long)T * (Hkv + a.Hq) + 3) / 4);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (hd == 128) paged_append_kernel<128><<<grid, 128, 0, st>>>(plan ? *plan : none, a);
  else paged_append_kernel<64><<<grid, 128, 0, st>>>(plan ? *plan : none, a);
  if (cudaError_t e = cudaGetLastError()) return paged_cuda_fail(e, fn, "launch");
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
  GatherArgs a{static_cast<const unsigned char*>(pages), slots, k, v, kt, kh, vt, vh, T, Hkv, n_pages, dtype == KVQ_BF16};
  const int grid = grid_of(((long long)T * Hkv * hd + 255) / 256);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (hd == 128) paged_gather_kernel<128><<<grid, 256, 0, st>>>(a);
  else paged_gather_kernel<64><<<grid, 256, 0, st>>>(a);
  if (cudaError_t e = cudaGetLastError()) return paged_cuda_fail(e, fn, "launch");
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
