// Calls kda_residual_norm_bwd from several host threads at once, without an interpreter between the
// calls.  For test_gpu_layer_edges.py.
#include <atomic>
#include <thread>
#include <vector>

#include "kda.h"

using Call = decltype(&kda_residual_norm_bwd);

struct Args {                    // one thread's calls: the same call `times` times
  const kda_norm_params_t* p;
  const void *x, *h, *gate;
  const float *post_weight, *weight;
  const void *d_y, *d_h;
  void *dx, *d_residual, *d_gate;
  float *d_post_weight, *d_weight;
  void* workspace;
  size_t workspace_bytes;
  void* stream;
};

// The number of calls that failed.
extern "C" int call_from_threads(Call call, const Args* args, int threads, int times) {
  std::atomic<int> failed{0}, ready{0};
  std::vector<std::thread> pool;
  for (int i = 0; i < threads; ++i)
    pool.emplace_back([&, i] {
      const Args& a = args[i];
      for (++ready; ready < threads;) std::this_thread::yield();
      for (int n = 0; n < times; ++n)
        if (call(a.p, a.x, a.h, a.gate, a.post_weight, a.weight, a.d_y, a.d_h, a.dx, a.d_residual, a.d_gate,
                 a.d_post_weight, a.d_weight, a.workspace, a.workspace_bytes, a.stream) != KDA_OK)
          ++failed;
    });
  for (auto& t : pool) t.join();
  return failed;
}
