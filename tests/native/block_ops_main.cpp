// Host driver of the block operators' entry points (csrc/block_ops.cpp beside csrc/fp8_ops.cpp)
// with the HIP runtime and the kernel launches replaced by stand-ins: threads that share a
// stream do not enqueue into each other's launches on the library's workspace, what does not
// fit it is refused, and no exception leaves an entry. Runs without a GPU.
#include "../../include/iris_local.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <chrono>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <new>
#include <set>
#include <thread>
#include <vector>

#include "../../gemm_collective_tile_amd/csrc/block_norm.hpp"
#include "../../gemm_collective_tile_amd/csrc/fp8_act.hpp"

namespace {
std::mutex mu;
std::set<void*> busy, used;
int overlaps = 0;
std::atomic<int> mallocs{0}, frees{0};
std::set<size_t> sizes;
bool no_memory = false;
size_t need = 1 << 20;

// stands for a call's launches, which write the workspace and read it again
hipError_t work(void* ws) {
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!busy.insert(ws).second) ++overlaps;
    used.insert(ws);
  }
  std::this_thread::sleep_for(std::chrono::microseconds(200));
  std::lock_guard<std::mutex> lk(mu);
  busy.erase(ws);
  return hipSuccess;
}
}  // namespace

extern "C" {
hipError_t hipMalloc(void** p, size_t n) {
  *p = malloc(64);
  ++mallocs;
  std::lock_guard<std::mutex> lk(mu);
  sizes.insert(n);
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

Fp8MmPlan fp8_mm_plan(int64_t, int64_t, int64_t, bool) { return {}; }
hipError_t launch_fp8_mm(const Fp8MmArgs&, const Fp8MmPlan&, void*, hipStream_t) { return hipSuccess; }
hipError_t launch_fp8_mm_few(const Fp8MmArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_fp8_quantize(const Fp8QuantArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_fp8_swiglu(const Fp8SwigluArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_fp8_swiglu_bwd(const Fp8SwigluBwdArgs&, hipStream_t) { return hipSuccess; }

DropoutPlan dropout_plan(int64_t, int64_t) { return {16, 1, 64, need}; }
hipError_t launch_dropout(const DropoutArgs&, const DropoutPlan&, void* sums, void* ws, hipStream_t) {
  return sums ? work(ws) : hipSuccess;
}
NormBwdPlan norm_bwd_plan(int64_t, int64_t, bool) { return {4, 16, need}; }
template <class T>
hipError_t launch_norm(const NormArgs&, bool, bool, hipStream_t) { return hipSuccess; }
template <class T>
hipError_t launch_norm_bwd(const NormBwdArgs& a, bool, bool, hipStream_t) { return work(a.part); }
template hipError_t launch_norm<f16>(const NormArgs&, bool, bool, hipStream_t);
template hipError_t launch_norm<bf16>(const NormArgs&, bool, bool, hipStream_t);
template hipError_t launch_norm_bwd<f16>(const NormBwdArgs&, bool, bool, hipStream_t);
template hipError_t launch_norm_bwd<bf16>(const NormBwdArgs&, bool, bool, hipStream_t);
hipError_t launch_norm_join(const NormBwdArgs& a, hipStream_t) { return work(a.part); }
Fp8ActPlan fp8_mm_act_plan(int64_t, int64_t, int64_t, bool, bool, bool) {
  Fp8ActPlan p{};
  p.ws_bytes = need;
  return p;
}
hipError_t launch_fp8_mm_act(const Fp8ActArgs&, const Fp8ActPlan&, void*, void* ws, hipStream_t) { return work(ws); }
}  // namespace iris

namespace {
// the addresses are placeholders: no kernel runs
int dropout(void* sums) {
  return iris_dropout((void*)0x100000, 64, (void*)0x200000, 64, nullptr, 0, IRIS_TYPE_FP16, 1.0f, nullptr, sums, 16, 64, nullptr, 0,
                      nullptr);
}
iris_norm_t norm() {
  iris_norm_t n{};
  n.kind = IRIS_NORM_RMS;
  n.type = n.stream_type = n.param_type = n.gate_type = IRIS_TYPE_FP16;
  n.eps = 1e-6f;
  n.alpha = 1.0f;
  return n;
}
int forward() {
  const iris_norm_t n = norm();
  return iris_block_norm(nullptr, 0, (void*)0x100000, 64, nullptr, nullptr, (void*)0x200000, 64, nullptr, 0, &n, 16, 64, nullptr);
}
int backward() {
  const iris_norm_t n = norm();
  return iris_block_norm_bwd((void*)0x100000, 64, nullptr, 0, (float*)0x600000, nullptr, nullptr, nullptr, nullptr, (void*)0x200000,
                             64, nullptr, 0, (void*)0x300000, 64, nullptr, 0, (float*)0x400000, &n, 16, 64, nullptr, 0, nullptr);
}
const iris_fp8_t A{(void*)0x1000000, (void*)0x2000000, 256, 4, 1}, B{(void*)0x3000000, (void*)0x4000000, 256, 4, 128};
int product() {
  return iris_fp8_mm_act((void*)0x500000, IRIS_TYPE_FP16, 64, nullptr, 0, nullptr, &A, &B, nullptr, IRIS_ACT_GELU, 1.0f, nullptr,
                         nullptr, 0, 16, 64, 256, nullptr, 0, nullptr);
}
int product_bwd() {
  return iris_fp8_mm_act_bwd((void*)0x500000, IRIS_TYPE_FP16, 64, nullptr, &A, &B, (void*)0x600000, 64, IRIS_ACT_SILU, 1.0f, nullptr,
                             16, 64, 256, nullptr, 0, nullptr);
}

int check(bool ok, const char* what) {
  if (!ok) printf("failed: %s\n", what);
  return ok ? 0 : 1;
}

// every operator that uses the workspace, on one stream
int from_threads() {
  std::atomic<int> bad{0};
  std::vector<std::thread> ts;
  for (int t = 0; t < 8; ++t)
    ts.emplace_back([&, t] {
      for (int i = 0; i < 20; ++i)
        bad += (t % 4 == 0 ? dropout((void*)0x700000) : t % 4 == 1 ? backward() : t % 4 == 2 ? product() : product_bwd()) != IRIS_OK;
    });
  for (auto& t : ts) t.join();
  return bad;
}
}  // namespace

int main() {
  int bad = 0;
  bad += check(dropout(nullptr) == IRIS_OK && forward() == IRIS_OK && mallocs == 0, "no workspace where none is needed");
  bad += check(from_threads() == 0 && overlaps == 0, "calls on one stream were enqueued into each other");
  bad += check(used.size() == 1 && mallocs == 1, "one workspace for one stream");
  need = (size_t)40 << 20;
  bad += check(from_threads() == 0 && overlaps == 0, "calls on one stream in the wide workspace");
  bad += check(used.size() == 2 && mallocs == 2 && sizes.size() == 2, "a second, wider workspace");
  need = ((size_t)128 << 20) + 1;
  bad += check(dropout((void*)0x700000) == IRIS_ERR_WORKSPACE && backward() == IRIS_ERR_WORKSPACE &&
                   product() == IRIS_ERR_WORKSPACE && product_bwd() == IRIS_ERR_WORKSPACE, "what fits neither is refused");
  bad += check(iris::fp8_finalize() == IRIS_OK && mallocs == frees, "everything is freed");
  need = 1 << 20;
  no_memory = true;   // no exception leaves an entry
  bad += check(dropout((void*)0x700000) == IRIS_ERR_NO_MEMORY, "iris_dropout without memory");
  bad += check(forward() == IRIS_ERR_NO_MEMORY, "iris_block_norm without memory");
  bad += check(backward() == IRIS_ERR_NO_MEMORY, "iris_block_norm_bwd without memory");
  bad += check(product() == IRIS_ERR_NO_MEMORY, "iris_fp8_mm_act without memory");
  bad += check(product_bwd() == IRIS_ERR_NO_MEMORY, "iris_fp8_mm_act_bwd without memory");
  if (!bad) printf("ok\n");
  return bad ? 1 : 0;
}
