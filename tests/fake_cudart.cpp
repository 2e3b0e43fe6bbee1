// A stand-in for the CUDA runtime, for host tests of the launch code (no GPU): devices are
// numbers, kernels do nothing, and a launch is refused where the runtime would refuse it
// for its grid or for shared memory that was not asked for on that device.
#include <cuda.h>
#include <cuda_runtime_api.h>

#include <map>
#include <utility>

static int device = 0;
static std::map<std::pair<const void*, int>, int> shared;    // (kernel, device) -> bytes
static cudaLaunchConfig_t last = {};
static int launches = 0;
static void* handle = nullptr;

extern "C" {

void fake_set_device(int d) { device = d; }
int fake_launches(void) { return launches; }
// x, y, z of the last launch's grid
void fake_last_grid(unsigned* g) {
  g[0] = last.gridDim.x, g[1] = last.gridDim.y, g[2] = last.gridDim.z;
}

void** __cudaRegisterFatBinary(void*) { return &handle; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}

cudaError_t cudaGetDevice(int* d) { return *d = device, cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrMultiProcessorCount ? 152 : a == cudaDevAttrMaxSharedMemoryPerBlockOptin ? 232448 : 0;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) shared[{f, device}] = v;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t,
                                                                   unsigned) {
  return *n = 2, cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  const auto it = shared.find({f, device});
  if (c->dynamicSmemBytes > (it == shared.end() ? 48u * 1024 : static_cast<unsigned>(it->second)))
    return cudaErrorInvalidValue;
  if (c->gridDim.x < 1 || c->gridDim.x > 0x7fffffffu || c->gridDim.y < 1 || c->gridDim.y > 65535 ||
      c->gridDim.z < 1 || c->gridDim.z > 65535)
    return cudaErrorInvalidConfiguration;
  last = *c;
  ++launches;
  return cudaSuccess;
}

static CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                       const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                       CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *f = reinterpret_cast<void*>(&encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

}
