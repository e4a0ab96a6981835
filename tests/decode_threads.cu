// Two host threads that call stem_decode_select of libstem.so, each with a cache, a stream and buffers of
// its own; one table is narrow, one as wide as it may be (built and run by
// tests/test_gpu_decode_edges.py; in Python the threads would wait for one another too often).
#include <cuda_runtime.h>

#include <atomic>
#include <cstdio>
#include <thread>
#include <vector>

#include "stem.h"

static void* device(size_t bytes, const void* from = nullptr) {
  void* p = nullptr;
  if (cudaMalloc(&p, bytes) != cudaSuccess) return nullptr;
  if (from)
    cudaMemcpy(p, from, bytes, cudaMemcpyHostToDevice);
  else
    cudaMemset(p, 0, bytes);
  return p;
}

int main() {
  constexpr int kBlocks = 40, kCap = 12, kHeads = 2, kD = 64, kCalls = 20000;
  std::atomic<int> failed{0}, ready{0};
  auto work = [&](int wide) {
    std::vector<int32_t> table(wide, -1), budget(wide, kCap);
    for (int i = 0; i < kBlocks; ++i) table[i] = i;
    for (int i = 0; i < kCap; ++i) budget[i] = i + 1;
    const int32_t len = kBlocks * 64 - 5;
    stem_cache_t c{};
    c.pages = device(stem_cache_page_bytes(kD, 64, STEM_KV_Q4) * kBlocks);
    c.kbar = static_cast<float*>(device(sizeof(float) * kBlocks * kD));
    c.vnorm = static_cast<float*>(device(sizeof(float) * kBlocks));
    c.table = static_cast<int32_t*>(device(sizeof(int32_t) * wide, table.data()));
    c.num_pages = kBlocks, c.Hkv = 1, c.D = kD, c.block = 64, c.format = STEM_KV_Q4;
    c.nseq = 1, c.max_blocks = wide;
    stem_method_t m{};
    stem_decode_args_t a{};
    a.cache = &c, a.method = &m;
    a.q = device(2 * kHeads * kD);
    a.lens = static_cast<int32_t*>(device(sizeof(len), &len));
    a.budget = static_cast<int32_t*>(device(sizeof(int32_t) * wide, budget.data()));
    a.R = 1, a.Hq = kHeads, a.kcap = kCap;
    a.sel_idx = static_cast<int32_t*>(device(sizeof(int32_t) * kHeads * kCap));
    a.sel_cnt = static_cast<int32_t*>(device(sizeof(int32_t) * kHeads));
    cudaStream_t st = nullptr;
    int bad = cudaStreamCreate(&st) != cudaSuccess || stem_decode_select(&a, st) != STEM_OK ||
              cudaStreamSynchronize(st) != cudaSuccess;
    ++ready;
    while (ready < 2) std::this_thread::yield();
    for (int n = 0; n < kCalls && bad == 0; ++n) {
      bad = stem_decode_select(&a, st) != STEM_OK;
      if (n % 200 == 0) cudaStreamSynchronize(st);
    }
    if (cudaStreamSynchronize(st) != cudaSuccess) bad = 1;
    failed += bad;
  };
  std::thread narrow(work, kBlocks), wide(work, STEM_MAX_NB);
  narrow.join();
  wide.join();
  std::printf(failed ? "failed\n" : "ok\n");
  return failed != 0;
}
