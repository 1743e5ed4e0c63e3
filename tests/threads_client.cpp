// Calls of the C ABI from several host threads at once, without an interpreter's lock
// between them (driven by test_gpu_threads.py).
#include <atomic>
#include <thread>
#include <vector>

#include "ds_ragged.h"

struct AdjustCall {
  const ds_ragged_meta* meta;
  const void* logits;
  const ds_logit_rules* rules;
  void* out;
  void* stream;
  int64_t stride;
  int32_t dtype, vocab;
};

struct SampleCall {
  const ds_ragged_meta* meta;
  const void* logits;
  const ds_sampler* sampler;
  int32_t* tokens;
  void* stream;
  int64_t stride;
  int32_t dtype, vocab;
};

// A thread to each of the n calls, each made `times` times; how many failed.
template <class Call, class F>
static int together(const Call* calls, int n, int times, F one) {
  std::atomic<int> failed{0}, ready{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < n; ++i)
    threads.emplace_back([&, i] {
      ++ready;
      while (ready < n) std::this_thread::yield();
      for (int k = 0; k < times; ++k)
        if (one(calls[i]) != DS_OK) ++failed;
    });
  for (auto& t : threads) t.join();
  return failed;
}

extern "C" int adjust_together(decltype(&ds_ragged_adjust_logits) fn, const AdjustCall* calls, int n, int times) {
  return together(calls, n, times, [&](const AdjustCall& c) {
    return fn(c.meta, c.logits, c.dtype, c.vocab, c.stride, c.rules, c.out, c.stride, c.stream);
  });
}

extern "C" int sample_together(decltype(&ds_ragged_sample) fn, const SampleCall* calls, int n, int times) {
  return together(calls, n, times, [&](const SampleCall& c) {
    return fn(c.meta, c.logits, c.dtype, c.vocab, c.stride, c.sampler, c.tokens, nullptr, c.stream);
  });
}
