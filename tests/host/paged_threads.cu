// Host threads that call kvq_paged_attention at once, each on its own stream and with its own workspace, with
// batches of one and of many sequences (all of them padding: the calls, not the kernels, are what runs).
#include <cstdio>
#include <cstdlib>
#include <string>
#include <thread>
#include <vector>

#include <cuda_runtime.h>

#include "kvq.h"

namespace {

constexpr int HQ = 8, HKV = 2, D = 128, CALLS = 20000;

void cuda(cudaError_t e) {
  if (e != cudaSuccess) std::printf("%s\n", cudaGetErrorString(e)), std::exit(2);
}
template <typename T>
T* device(size_t n) {
  T* p = nullptr;
  cuda(cudaMalloc(&p, n * sizeof(T)));
  cuda(cudaMemset(p, 0, n * sizeof(T)));
  return p;
}

void calls(int batch, const void* pages, std::string* why) {
  cudaStream_t s;
  cuda(cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking));
  size_t bytes = 0;
  if (kvq_paged_attention_workspace(batch, 1, HQ, HKV, D, &bytes) != KVQ_OK) return void(*why = kvq_last_error());
  unsigned short *q = device<unsigned short>((size_t)batch * HQ * D), *out = device<unsigned short>((size_t)batch * HQ * D);
  int32_t *table = device<int32_t>(batch), *lens = device<int32_t>(batch);
  unsigned char* ws = device<unsigned char>(bytes);
  cuda(cudaDeviceSynchronize());
  for (int i = 0; i < CALLS && why->empty(); ++i)
    if (kvq_paged_attention(KVQ_F16, q, HQ * D, D, pages, 1, table, 1, 1, lens, batch, 1, HQ, HKV, D, 0, 0.f, out, nullptr, ws, bytes, s) != KVQ_OK)
      *why = "batch " + std::to_string(batch) + ", call " + std::to_string(i) + ": " + kvq_last_error();
  cuda(cudaStreamSynchronize(s));
}

}  // namespace

int main() {
  size_t page = 0;
  if (kvq_paged_page_bytes(D, &page) != KVQ_OK) return 2;
  const void* pages = device<unsigned char>(page * HKV);
  const int batches[] = {1, 2048, 1, 1500, 2, 2048};
  std::vector<std::string> why(6);
  std::vector<std::thread> threads;
  for (int i = 0; i < 6; ++i) threads.emplace_back(calls, batches[i], pages, &why[i]);
  for (auto& t : threads) t.join();
  int wrong = 0;
  for (const auto& w : why)
    if (!w.empty()) std::printf("%s\n", w.c_str()), ++wrong;
  if (!wrong) std::puts("ok");
  return wrong != 0;
}
