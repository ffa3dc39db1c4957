// Host driver of the 8-bit operators' entry points (csrc/fp8_ops.cpp) with the HIP
// runtime and the kernel launches replaced by stand-ins: what threads that share a
// stream do to the library's workspace of split products. Runs without a GPU.
#include "../../include/iris_local.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <chrono>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <mutex>
#include <new>
#include <set>
#include <string>
#include <thread>
#include <vector>

#include "../../gemm_collective_tile_amd/csrc/fp8.hpp"

namespace {
std::mutex mu;
std::set<void*> busy;                              // workspaces between a product's first and last launch
std::map<std::thread::id, std::set<void*>> used;   // by thread
int overlaps = 0;
std::atomic<int> mallocs{0}, frees{0};
bool no_memory = false;
}  // namespace

extern "C" {
hipError_t hipMalloc(void** p, size_t) {
  *p = malloc(64);
  ++mallocs;
  return hipSuccess;
}
hipError_t hipFree(void* p) {
  free(p);
  ++frees;
  return hipSuccess;
}
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipDeviceSynchronize() { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipThreadExchangeStreamCaptureMode(hipStreamCaptureMode*) { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return ""; }
}

namespace iris {
int set_error(int status, const char*) { return status; }
int use_device(int* dev, int* cus) {
  if (no_memory) throw std::bad_alloc();
  *dev = 0;
  *cus = 256;
  return 0;
}
int fp8_finalize();

Fp8MmPlan fp8_mm_plan(int64_t, int64_t, int64_t, bool) {
  Fp8MmPlan p;
  p.bm = p.bn = 64;
  p.splits = 4;
  p.ws_bytes = 1 << 20;
  return p;
}
// stands for the two launches of a split product
hipError_t launch_fp8_mm(const Fp8MmArgs&, const Fp8MmPlan&, void* ws, hipStream_t) {
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!busy.insert(ws).second) ++overlaps;
    used[std::this_thread::get_id()].insert(ws);
  }
  std::this_thread::sleep_for(std::chrono::microseconds(200));
  std::lock_guard<std::mutex> lk(mu);
  busy.erase(ws);
  return hipSuccess;
}
hipError_t launch_fp8_mm_few(const Fp8MmArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_fp8_quantize(const Fp8QuantArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_fp8_swiglu(const Fp8SwigluArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_fp8_swiglu_bwd(const Fp8SwigluBwdArgs&, hipStream_t) { return hipSuccess; }
}  // namespace iris

namespace {
// the addresses are placeholders: no kernel runs
int product(hipStream_t s) {
  const iris_fp8_t a{(void*)0x100000, (void*)0x200000, 4096, 32, 1}, b{(void*)0x300000, (void*)0x400000, 4096, 32, 128};
  return iris_fp8_mm((void*)0x500000, IRIS_TYPE_FP16, 512, &a, &b, nullptr, 256, 512, 4096, 0, nullptr, 0, s);
}

int check(bool ok, const char* what) {
  if (!ok) printf("failed: %s\n", what);
  return ok ? 0 : 1;
}

int from_threads(hipStream_t s) {
  std::atomic<int> bad{0};
  std::vector<std::thread> ts;
  used.clear();
  for (int t = 0; t < 6; ++t)
    ts.emplace_back([&] {
      for (int i = 0; i < 40; ++i) bad += product(s) != IRIS_OK;
    });
  for (auto& t : ts) t.join();
  return bad;
}
}  // namespace

int main() {
  int bad = 0;
  bad += check(from_threads(nullptr) == 0, "products on one stream");
  bad += check(overlaps == 0, "two products of one stream were enqueued into each other");
  bad += check(mallocs == 1, "one workspace for one stream");
  bad += check(from_threads(hipStreamPerThread) == 0, "products on per-thread streams");
  std::set<void*> all;
  size_t n = 0;
  for (auto& kv : used) {
    bad += check(kv.second.size() == 1, "one workspace for a thread's stream");
    all.insert(kv.second.begin(), kv.second.end());
    n += kv.second.size();
  }
  bad += check(n == 6 && all.size() == n, "per-thread streams share a workspace");
  bad += check(overlaps == 0, "products of different streams met in one workspace");
  bad += check(iris::fp8_finalize() == IRIS_OK && mallocs == frees, "everything is freed");
  bad += check(product(nullptr) == IRIS_OK && iris::fp8_finalize() == IRIS_OK && mallocs == frees, "use after finalize");
  no_memory = true;   // no exception leaves an entry
  const iris_fp8_t a{(void*)0x100000, (void*)0x200000, 4096, 32, 1}, b{(void*)0x300000, (void*)0x400000, 4096, 32, 1},
      c{(void*)0x600000, (void*)0x700000, 4096, 32, 1}, d{(void*)0x800000, (void*)0x900000, 4096, 32, 1};
  bad += check(product(nullptr) == IRIS_ERR_NO_MEMORY, "iris_fp8_mm without memory");
  bad += check(iris_fp8_quantize(&a, nullptr, (void*)0x500000, IRIS_TYPE_FP16, 4096, nullptr, 8, 4096, nullptr) ==
                   IRIS_ERR_NO_MEMORY, "iris_fp8_quantize without memory");
  bad += check(iris_fp8_swiglu(&a, nullptr, nullptr, (void*)0x500000, (void*)0x510000, IRIS_TYPE_FP16, 4096, 4096, 8, 4096,
                               nullptr) == IRIS_ERR_NO_MEMORY, "iris_fp8_swiglu without memory");
  bad += check(iris_fp8_swiglu_bwd(&a, &b, nullptr, nullptr, nullptr, (void*)0x500000, IRIS_TYPE_FP16, 4096, &c, &d, 8, 4096,
                                   nullptr) == IRIS_ERR_NO_MEMORY, "iris_fp8_swiglu_bwd without memory");
  if (!bad) printf("ok\n");
  return bad ? 1 : 0;
}
