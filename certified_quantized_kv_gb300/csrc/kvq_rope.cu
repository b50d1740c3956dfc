// kvq_rope.cu -- rotary positions, and the argument checks of the paged-cache calls.
//
// Pair i of a head at position p is turned by p w_i: (a, b) -> (a cos - b sin, b cos + a sin).
// The plan holds w_i / (2 pi) as a 64-bit fraction of a turn, so p w_i modulo one turn is an
// integer product without rounding (rope_cos_sin): a position of 2 million costs no
// accuracy, which an fp32 product of position and frequency would.
#include <algorithm>
#include <cmath>
#include <limits>
#include <string>

#include "kvq.h"
#include "kvq_launch.h"
#include "kvq_paged.cuh"
#include "kvq_rope.cuh"

namespace kvq {

void set_last_error(const std::string& msg);

kvq_status paged_fail(kvq_status s, const char* fn, const char* what) {
  set_last_error(std::string(fn) + ": " + what);
  return s;
}

kvq_status paged_cuda_fail(cudaError_t e, const char* fn, const char* what) {
  set_last_error(std::string(fn) + ": " + what + ": " + cudaGetErrorString(e));
  return KVQ_ERR_CUDA;
}

kvq_status check_buffer(const void* p, int dev, size_t align, const char* fn, const char* name) {
  const std::string n(name);
  if (!p) return paged_fail(KVQ_ERR_INVALID, fn, (n + " is NULL").c_str());
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    at.type = cudaMemoryTypeUnregistered;
  }
  const bool ok = at.type == cudaMemoryTypeManaged || (at.type == cudaMemoryTypeDevice && at.device == dev);
  if (!ok) return paged_fail(KVQ_ERR_INVALID, fn, (n + " must be device memory of the current device").c_str());
  if (reinterpret_cast<uintptr_t>(p) % align != 0)
    return paged_fail(KVQ_ERR_INVALID, fn, (n + " must be " + std::to_string(align) + "-byte aligned").c_str());
  return KVQ_OK;
}

kvq_status check_strides(int64_t token, int64_t head, const char* fn, const char* name) {
  if (token < 0 || head < 0 || token % 8 != 0 || head % 8 != 0)
    return paged_fail(KVQ_ERR_INVALID, fn,
                      (std::string(name) + ": strides must be non-negative multiples of 8 elements").c_str());
  return KVQ_OK;
}

kvq_status check_plan(const kvq_rope_plan* plan, int head_dim, const char* fn) {
  if (plan->head_dim != head_dim) return paged_fail(KVQ_ERR_INVALID, fn, "the plan is for another head_dim");
  if (plan->rotary_dim < 2 || plan->rotary_dim > plan->head_dim || plan->rotary_dim % 2 != 0 || plan->head_dim > 256)
    return paged_fail(KVQ_ERR_INVALID, fn, "the plan was not initialised by kvq_rope_plan_init");
  return KVQ_OK;
}

namespace {

constexpr int ROPE_THREADS = 256;

// 32768 tokens of 40 heads of 128: 671 MB in 97.8 us, 6.86 TB/s (a copy: 6.79); 64 tokens: 2.4 us, most of
// it the launch and two dependent reads; 4099 tokens of 13 heads, 96 of 128 elements, interleaved:
// 7.7 us for 27 MB (positions in order; 8.6 at random), of which the elements that are only copied cost the
// most: all 128 rotated 6.7, 96 in place 6.0.
template <int V, bool INTERLEAVED, bool BF16>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const __grid_constant__ kvq_rope_plan P, RopeArgs a) {
  __shared__ __align__(16) uint64_t step[128];
  __shared__ __align__(16) float2 turns[ROPE_THREADS * V + 256];
  pdl_trigger();
  load_steps(P, step);
  pdl_wait();
  rope_part<V, INTERLEAVED, BF16, ROPE_THREADS, true>(P, step, turns, a, blockIdx.x * (long long)ROPE_THREADS, (long long)gridDim.x * ROPE_THREADS);
}

template <bool BF16>
__global__ void __launch_bounds__(ROPE_THREADS) rope_rows_kernel(const __grid_constant__ kvq_rope_plan P, RopeArgs a) {
  constexpr int WARPS = ROPE_THREADS / 32;
  __shared__ __align__(16) uint64_t step[128];
  __shared__ uint4 rooms[ROPE_THREADS];
  __shared__ float2 turns[WARPS][128];
  pdl_trigger();
  load_steps(P, step);
  pdl_wait();
  const int warp = threadIdx.x >> 5;
  rope_rows<BF16>(P, step, rooms + 32 * warp, turns[warp], a, (long long)blockIdx.x * WARPS + warp, (long long)gridDim.x * WARPS);
}

template <bool INTERLEAVED, bool BF16>
auto rope_kernel_of(int V) {
  if constexpr (INTERLEAVED) return V == 8 ? rope_kernel<8, true, BF16> : rope_kernel<4, true, BF16>;
  else return V == 8 ? rope_kernel<8, false, BF16> : V == 4 ? rope_kernel<4, false, BF16> : rope_rows_kernel<BF16>;
}

kvq_status rope_impl(const kvq_rope_plan* plan, int dtype, const void* x, int64_t xt, int64_t xh,
                     const int32_t* positions, int T, int H, void* out, int64_t ot, int64_t oh, void* stream) {
  const char* fn = "kvq_rope";
  if (!plan) return paged_fail(KVQ_ERR_INVALID, fn, "plan is NULL");
  if (kvq_status s = check_plan(plan, plan->head_dim, fn)) return s;
  if (plan->head_dim % 8 != 0) return paged_fail(KVQ_ERR_INVALID, fn, "head_dim must be a multiple of 8");
  if (dtype != KVQ_F16 && dtype != KVQ_BF16) return paged_fail(KVQ_ERR_INVALID, fn, "dtype must be KVQ_F16 or KVQ_BF16");
  if (T < 0 || H < 0) return paged_fail(KVQ_ERR_INVALID, fn, "n_tokens and n_heads must be >= 0");
  if (T == 0 || H == 0) return KVQ_OK;
  if (kvq_status s = check_strides(xt, xh, fn, "x")) return s;
  if (kvq_status s = check_strides(ot, oh, fn, "out")) return s;
  if (x == out && ((T > 1 && xt != ot) || (H > 1 && xh != oh)))
    return paged_fail(KVQ_ERR_INVALID, fn, "out = x needs the same strides");
  if (rows_overlap(T, H, ot, oh, plan->head_dim)) return paged_fail(KVQ_ERR_INVALID, fn, "out: rows must not overlap");
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return paged_cuda_fail(e, fn, "no current CUDA device");
  if (kvq_status s = check_buffer(x, dev, 16, fn, "x")) return s;
  if (kvq_status s = check_buffer(out, dev, 16, fn, "out")) return s;
  if (kvq_status s = check_buffer(positions, dev, 4, fn, "positions")) return s;
  const int V = rope_pairs(*plan);
  const bool copy = x != out && plan->rotary_dim < plan->head_dim;
  RopeArgs a{x, out, positions, xt, xh, ot, oh, T, H, 0, copy, 0};
  long long blocks;
  if (V) {
    const int units = rope_units(*plan, V, copy), resident = V == 8 ? 3 : 5;   // blocks per SM, by their registers
    a.lanes = rope_lanes(T, H, units, 152ll * ROPE_THREADS * resident);
    blocks = ((long long)T * a.lanes * units + ROPE_THREADS - 1) / ROPE_THREADS;
  } else {
    constexpr int WARPS = ROPE_THREADS / 32;
    a.per = rope_rows_heads(*plan, copy, T, H, 152 * WARPS * 3);
    blocks = ((long long)T * ((H + a.per - 1) / a.per) + WARPS - 1) / WARPS;
  }
  const bool bf16 = dtype == KVQ_BF16;
  auto* k = plan->interleaved ? (bf16 ? rope_kernel_of<true, true>(V) : rope_kernel_of<true, false>(V))
                              : (bf16 ? rope_kernel_of<false, true>(V) : rope_kernel_of<false, false>(V));
  const dim3 grid((unsigned)std::min<long long>(blocks, 152 * 32));
  const cudaError_t e = launch_dependent(k, grid, dim3(ROPE_THREADS), 0, static_cast<cudaStream_t>(stream), *plan, a);
  if (e != cudaSuccess) return paged_cuda_fail(e, fn, "launch");
  return KVQ_OK;
}

kvq_status plan_impl(const kvq_rope_config* c, kvq_rope_plan* p) {
  const char* fn = "kvq_rope_plan_init";
  auto bad = [&](const char* what) { return paged_fail(KVQ_ERR_INVALID, fn, what); };
  if (!c || !p) return bad("NULL argument");
  if (c->head_dim < 2 || c->head_dim > 256 || c->head_dim % 2) return bad("head_dim must be even and in 2..256");
  if (c->rotary_dim < 2 || c->rotary_dim > c->head_dim || c->rotary_dim % 2)
    return bad("rotary_dim must be even and in 2..head_dim");
  if (c->interleaved != 0 && c->interleaved != 1) return bad("interleaved must be 0 or 1");
  if (c->scaling < KVQ_ROPE_NONE || c->scaling > KVQ_ROPE_YARN) return bad("unknown scaling");
  if (!(c->base > 1.0) || !std::isfinite(c->base)) return bad("base must be finite and > 1");
  const bool scaled = c->scaling != KVQ_ROPE_NONE;
  const bool blend = c->scaling == KVQ_ROPE_PARTS || c->scaling == KVQ_ROPE_YARN;
  if (scaled && (!(c->factor >= 1.0) || !std::isfinite(c->factor))) return bad("factor must be finite and >= 1");
  if (blend && c->original_ctx < 1) return bad("original_ctx must be >= 1");
  if (blend && !(c->low > 0.0 && c->low < c->high && std::isfinite(c->high))) return bad("0 < low < high is needed");
  if (!(c->magnitude >= 0.0 && c->magnitude <= std::numeric_limits<float>::max())) return bad("magnitude must be finite in fp32 and >= 0");
  const int rd = c->rotary_dim;
  double base = c->base;
  if (c->scaling == KVQ_ROPE_NTK) {
    if (rd < 4) return bad("NTK scaling needs rotary_dim >= 4");
    base *= std::pow(c->factor, (double)rd / (rd - 2));
    if (!std::isfinite(base)) return bad("base * factor^(rotary_dim / (rotary_dim - 2)) overflows");
  }
  const double two_pi = 6.283185307179586476925286766559;
  double d_lo = 0, d_hi = 1;   // YARN: pair indices where the blend falls from 1 to 0
  if (c->scaling == KVQ_ROPE_YARN) {
    auto d = [&](double turns) { return rd * std::log(c->original_ctx / (two_pi * turns)) / (2.0 * std::log(base)); };
    d_lo = std::fmax(std::floor(d(c->high)), 0.0);
    d_hi = std::fmin(std::ceil(d(c->low)), rd - 1.0);
  }
  p->head_dim = c->head_dim;
  p->rotary_dim = rd;
  p->interleaved = c->interleaved;
  p->magnitude = (float)(c->magnitude > 0 ? c->magnitude
                                          : c->scaling == KVQ_ROPE_YARN ? 0.1 * std::log(c->factor) + 1.0 : 1.0);
  for (int i = 0; i < 128; ++i) {
    p->step[i] = 0;
    if (i >= rd / 2) continue;
    double w = std::pow(base, -2.0 * i / rd), k = 1.0;
    if (c->scaling == KVQ_ROPE_LINEAR) k = 0.0;
    if (c->scaling == KVQ_ROPE_PARTS) k = (c->original_ctx * w / two_pi - c->low) / (c->high - c->low);
    if (c->scaling == KVQ_ROPE_YARN) k = 1.0 - (i - d_lo) / std::fmax(d_hi - d_lo, 1e-3);
    k = std::fmin(std::fmax(k, 0.0), 1.0);
    if (scaled) w = c->scaling == KVQ_ROPE_NTK ? w : w * k + w / c->factor * (1.0 - k);
    p->step[i] = (uint64_t)std::llrint(std::ldexp(w / two_pi, 62)) << 2;   // w <= 1: below a sixth of a turn
  }
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

extern "C" kvq_status kvq_rope_plan_init(const kvq_rope_config* cfg, kvq_rope_plan* plan) try {
  return kvq::plan_impl(cfg, plan);
} catch (...) {   // no exception leaves the C ABI (only a failing string allocation can throw)
  return KVQ_ERR_HOST_OOM;
}

extern "C" kvq_status kvq_rope(const kvq_rope_plan* plan, int dtype, const void* x, int64_t x_token_stride,
                               int64_t x_head_stride, const int32_t* positions, int n_tokens, int n_heads, void* out,
                               int64_t out_token_stride, int64_t out_head_stride, void* stream) try {
  return kvq::rope_impl(plan, dtype, x, x_token_stride, x_head_stride, positions, n_tokens, n_heads, out,
                        out_token_stride, out_head_stride, stream);
} catch (...) {
  return KVQ_ERR_HOST_OOM;
}
