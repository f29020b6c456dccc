// First calls of the tensor-map encoder's lookup from many host threads, over a
// driver query that takes its time: all of them get the same pointer.
#include <cuda_runtime.h>

#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>

static int target;
static std::atomic<int> queries{0};
static cudaError_t slow_query(const char *, void **p, unsigned, unsigned long long, cudaDriverEntryPointQueryResult *q) {
  ++queries;
  std::this_thread::sleep_for(std::chrono::milliseconds(300));
  *p = &target;
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
#define cudaGetDriverEntryPointByVersion slow_query
#include "tcgen05.cuh"

int main() {
  constexpr int kThreads = 8;
  std::atomic<int> ready{0}, wrong{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < kThreads; ++i)
    threads.emplace_back([&] {
      ++ready;
      while (ready < kThreads) std::this_thread::yield();
      if ((void *)sv::encode_fn() != (void *)&target) ++wrong;
    });
  for (auto &t : threads) t.join();
  printf("%d wrong, %d queries\n", wrong.load(), queries.load());
  return wrong.load() != 0;
}
