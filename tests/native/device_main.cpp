// Host driver of the library's device check (csrc/iris_local.cpp) on a machine whose
// GPU is another one than the library is built for. The HIP runtime is replaced by
// stand-ins; what else the file refers to is never called. Runs without a GPU.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>

#include "../../include/iris_local.h"

static const char* arch = "gfx942:sramecc+:xnack-";

extern "C" {
hipError_t hipGetDevice(int* d) {
  *d = 0;
  return hipSuccess;
}
hipError_t hipGetDeviceProperties(hipDeviceProp_t* p, int) {
  memset((void*)p, 0, sizeof *p);
  strncpy(p->gcnArchName, arch, sizeof p->gcnArchName - 1);
  return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) {
  *v = 100000;
  return hipSuccess;
}
}

namespace iris {
int use_device(int* dev, int* cus);
}

int main() {
  int dev = 0, cus = 0, bad = 0;
  for (int call = 0; call < 3; ++call)
    if (iris::use_device(&dev, &cus) != IRIS_ERR_NO_DEVICE) {
      printf("failed: call %d took a %s for a gfx950\n", call, arch);
      ++bad;
    }
  if (!bad) printf("ok\n");
  return bad ? 1 : 0;
}
