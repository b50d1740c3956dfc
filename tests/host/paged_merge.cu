// The merge of the paged attention's pieces, run by itself on the GPU: against sums in 64 bits, and with a piece
// that holds anything because a copy of its warp never arrived (the rows have to be NaN).
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#include "kvq_paged_merge.cuh"

using namespace kvq;

namespace {

int wrong = 0;

// pieces of a CTA's warps into slot 1 of `slots` or as rows; then, with `slots`, that one and the next CTA's
template <int HD, int R>
__global__ void __launch_bounds__(PA_THREADS) merge(PaOut po, const float* pieces, int n, bool closed, bool lost, int rn, float* slots) {
  constexpr int PART = R * (HD + 2);
  __shared__ const float* at[PA_WARPS][2];
  if (threadIdx.x < n) {
    const float* p = pieces + threadIdx.x * PART;
    const bool last = closed && threadIdx.x == n - 1;
    at[threadIdx.x][!last] = p, at[threadIdx.x][last] = p;
  }
  __syncthreads();
  pa_merge<HD, R, false>(po, &at[0][0], n, closed, lost, 0, 0, 0, rn, slots ? slots + PART : nullptr);
  if (!slots) return;
  __threadfence();
  __syncthreads();
  const float* base = slots;
  pa_merge<HD, R, true>(po, &base, 2, false, false, 0, 0, 0, rn, nullptr);
}

void CUDA(cudaError_t e) {
  if (e != cudaSuccess) std::printf("%s\n", cudaGetErrorString(e)), std::exit(2);
}

template <int HD, int R>
void check(int n, bool closed, bool lost, bool across, int rn) {
  constexpr int PART = R * (HD + 2);
  std::mt19937 rng(n + 7 * R + HD);
  std::normal_distribution<float> normal;
  const int all = n + (across ? 4 : 0);   // behind the pieces: slots 0..3 of two CTAs
  std::vector<float> p((size_t)all * PART);
  for (int k = 0; k < all; ++k)
    for (int i = 0; i < PART; ++i) {
      float& x = p[(size_t)k * PART + i];
      if (i < R * HD) x = normal(rng);
      else x = (i - R * HD) % 2 == 0 ? 6 * normal(rng) : 1 + std::fabs(normal(rng));
    }
  if (lost)   // bytes of a page over one of them
    for (int i = 0; i < PART; ++i) {
      const uint32_t u = rng();
      std::memcpy(&p[(size_t)(n / 2) * PART + i], &u, 4);
    }
  float *dp, *lse;
  unsigned short* out;
  CUDA(cudaMalloc(&dp, p.size() * 4));
  CUDA(cudaMalloc(&out, (size_t)R * HD * 2));
  CUDA(cudaMalloc(&lse, R * 4));
  CUDA(cudaMemcpy(dp, p.data(), p.size() * 4, cudaMemcpyHostToDevice));
  CUDA(cudaMemset(out, 0x11, (size_t)R * HD * 2));
  merge<HD, R><<<1, PA_THREADS>>>(PaOut{out, lse, 1, R, R, false}, dp, n, closed, lost, rn, across ? dp + (size_t)n * PART : nullptr);
  CUDA(cudaGetLastError());
  std::vector<__half> got((size_t)R * HD);
  std::vector<float> gl(R);
  CUDA(cudaMemcpy(got.data(), out, got.size() * 2, cudaMemcpyDeviceToHost));
  CUDA(cudaMemcpy(gl.data(), lse, R * 4, cudaMemcpyDeviceToHost));
  CUDA(cudaFree(dp));
  CUDA(cudaFree(out));
  CUDA(cudaFree(lse));
  int bad = 0;
  for (int r = 0; r < R; ++r) {
    double M = -INFINITY, L = 0;
    std::vector<int> from;
    for (int k = 0; k < n; ++k) from.push_back(k);
    if (across) from.push_back(n + 2);   // the next CTA's first slot
    for (int k : from) M = std::fmax(M, p[(size_t)k * PART + R * HD + 2 * r]);
    for (int k : from) L += p[(size_t)k * PART + R * HD + 2 * r + 1] * std::exp2(p[(size_t)k * PART + R * HD + 2 * r] - M);
    for (int c = 0; c < HD; ++c) {
      double o = 0, size = 0;
      for (int k : from) {
        const double w = std::exp2(p[(size_t)k * PART + R * HD + 2 * r] - M), x = p[(size_t)k * PART + r * HD + c];
        o += w * x, size += std::fabs(w * x);
      }
      const double y = __half2float(got[(size_t)r * HD + c]);
      if (r >= rn) bad += __half_as_ushort(got[(size_t)r * HD + c]) != 0x1111;
      else if (lost) bad += !std::isnan(y);
      // one rounding to binary16; exponents up to 40 in fp32 (40 2^-24) and exp2 (2^-22), twice when across, and sums
      else bad += !(std::fabs(y - o / L) <= std::fabs(o / L) * std::ldexp(1.0, -11) + std::ldexp(1.0, -24) + size / L * std::ldexp(1.0, -16));
    }
    if (r < rn) bad += lost ? !std::isnan(gl[r]) : !(std::fabs(gl[r] - (M + std::log2(L)) * std::log(2.0)) <= std::ldexp(1.0, -14));
  }
  if (bad) std::printf("head_dim %d, %d rows (%d), %d pieces, closed %d, lost %d, across %d: %d wrong\n", HD, R, rn, n, closed, lost, across, bad), ++wrong;
}

template <int HD, int R>
void sizes() {
  for (int n = 1; n <= PA_WARPS; n += n < 3 ? 1 : 5)
    for (int bits = 0; bits < 8; ++bits) check<HD, R>(n, bits & 1, bits & 2, bits & 4, bits & 1 ? R : R - 1);
}

}  // namespace

int main() {
  sizes<64, 4>(), sizes<64, 8>(), sizes<64, 16>(), sizes<128, 4>(), sizes<128, 8>(), sizes<128, 16>();
  if (!wrong) std::puts("ok");
  return wrong != 0;
}
