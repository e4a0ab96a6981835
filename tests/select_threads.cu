// Two host threads that call stem_select_m of libstem.so with group-shared lists, one over few blocks and
// one over as many as it takes, each with a stream and buffers of its own (built and run by
// tests/test_gpu_select_threads.py).
#include <cuda_runtime.h>

#include <atomic>
#include <cstdio>
#include <thread>

#include "stem.h"

static void* device(size_t bytes) {
  void* p = nullptr;
  if (cudaMalloc(&p, bytes) != cudaSuccess) return nullptr;
  cudaMemset(p, 0, bytes);
  return p;
}

int main() {
  constexpr int kHq = 2, kD = 64, kCalls = 4000;
  std::atomic<int> failed{0}, ready{0};
  auto work = [&](int nb) {
    stem_method_t m{};
    m.schedule = STEM_SCHED_EXP, m.rho_min = 0.1f, m.tau = 8.f, m.k_min = 2;
    m.share = STEM_SHARE_GROUP;
    const size_t cap = static_cast<size_t>(stem_sel_capacity_m(nb, &m));
    const size_t bytes = stem_workspace_size_m(1, kHq, 1, nb * 64, kD, 64, &m);
    auto* qbar = static_cast<float*>(device(sizeof(float) * kHq * nb * kD));
    auto* kbar = static_cast<float*>(device(sizeof(float) * nb * kD));
    auto* vnorm = static_cast<float*>(device(sizeof(float) * nb));
    auto* idx = static_cast<int32_t*>(device(sizeof(int32_t) * kHq * cap));
    auto* cnt = static_cast<int32_t*>(device(sizeof(int32_t) * kHq * nb));
    void* ws = device(bytes);
    cudaStream_t st = nullptr;
    int bad = cudaStreamCreate(&st) != cudaSuccess;
    auto call = [&] {
      return stem_select_m(qbar, kbar, vnorm, 1, kHq, 1, nb, kD, &m, idx, cnt, nullptr, ws, bytes,
                           st) != STEM_OK;
    };
    bad |= call() || cudaStreamSynchronize(st) != cudaSuccess;
    ++ready;
    while (ready < 2) std::this_thread::yield();
    for (int n = 0; n < kCalls && bad == 0; ++n) {
      bad = call();
      if (n % 50 == 0) cudaStreamSynchronize(st);
    }
    if (cudaStreamSynchronize(st) != cudaSuccess) bad = 1;
    failed += bad;
  };
  std::thread few(work, 64), many(work, 1024);
  few.join();
  many.join();
  std::printf(failed ? "failed\n" : "ok\n");
  return failed != 0;
}
