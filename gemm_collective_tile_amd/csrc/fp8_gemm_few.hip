// C = A B^T + bias for few rows of A: the plain product. How it is multiplied is in
// fp8_gemm_few.hpp.
#include "fp8_gemm_few.hpp"

namespace iris {
namespace {

template <class OUT>
struct PutPlain {
  __device__ __forceinline__ void put(const Fp8MmArgs& g, int m, int n, float v) const {
    put_output((OUT*)g.C + (int64_t)m * g.ldc + n, v, (const OUT*)g.bias, g.bias_along_m ? m : n, g.accumulate);
  }
};

}  // namespace

hipError_t launch_fp8_mm_few(const Fp8MmArgs& a, hipStream_t s) {
  switch (a.c_type) {
    case T_FP16: return launch_few<PutPlain<f16>, false>(a, {}, s);
    case T_BF16: return launch_few<PutPlain<bf16>, false>(a, {}, s);
    default: return launch_few<PutPlain<float>, true>(a, {}, s);
  }
}

}  // namespace iris
