// A CUDA runtime that launches nothing: the library's objects are linked with it, so
// that tests without a GPU see which kernels a call would launch, how, and on which
// device (tests/fake_cuda.py). Devices, their attributes' failures and errors are
// set by the test.
#include <cuda_runtime.h>

#include <map>
#include <string>
#include <utility>
#include <vector>

namespace {
struct Launch {
  std::string kernel;
  dim3 grid, block;
  size_t smem;
  int cluster, device;
};
std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}
std::map<std::pair<int, const void*>, int> allowed;  // dynamic shared memory by device and kernel, for the process
std::vector<Launch> launches;
int device = 0, failures = 0;
int encode_ok(...) { return 0; }
}  // namespace

extern "C" {

void fake_reset() { launches.clear(), device = failures = 0; }
void fake_set_device(int d) { device = d; }
void fake_fail_attributes(int n) { failures = n; }  // the next n calls fail
int fake_launches() { return (int)launches.size(); }
const char* fake_launch(int i, int64_t* v) {  // grid x y z, block, shared bytes, cluster, device
  const Launch& l = launches[i];
  const int64_t all[7] = {l.grid.x, l.grid.y, l.grid.z, l.block.x, (int64_t)l.smem, l.cluster, l.device};
  for (int k = 0; k < 7; ++k) v[k] = all[k];
  return l.kernel.c_str();
}

cudaError_t cudaGetDevice(int* d) { return *d = device, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  if (failures > 0) return --failures, cudaErrorInvalidValue;
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) allowed[{device, f}] = v;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  const auto it = allowed.find({device, f});
  if (c->dynamicSmemBytes > (size_t)(it == allowed.end() ? 49152 : it->second)) return cudaErrorInvalidValue;
  if (c->gridDim.x < 1 || c->gridDim.x > 0x7FFFFFFFu || c->gridDim.y < 1 || c->gridDim.y > 65535) return cudaErrorInvalidConfiguration;
  Launch l{names()[f], c->gridDim, c->blockDim, c->dynamicSmemBytes, 1, device};
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) l.cluster = (int)c->attrs[i].val.clusterDim.x;
  launches.push_back(l);
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned int, unsigned long long, cudaDriverEntryPointQueryResult* r) {
  *p = (void*)encode_ok;
  if (r) *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

// what the compiler's stubs call
void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, uint3*, uint3*, dim3*, dim3*, int*) { names()[host] = name; }
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}

// what the operators under test do not call
#define UNUSED(name) \
  cudaError_t name() { return cudaErrorNotSupported; }
UNUSED(__cudaGetKernel)
UNUSED(__cudaLaunchKernel)
UNUSED(__cudaPushCallConfiguration)
UNUSED(__cudaPopCallConfiguration)
}
