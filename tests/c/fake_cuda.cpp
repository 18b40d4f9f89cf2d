// A CUDA runtime without a GPU, for tests of the library's host code: every call succeeds and does nothing, every
// pointer counts as memory of device 0, launches are counted, and a named call can be made to fail.
#include <cstddef>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "driver_types.h"

namespace {
char fail_name[64];
int fail_code, launches, registers = 168, cluster = 1;
alignas(256) char symbol[16 << 20];   // stands for every device symbol

int result(const char* name) { return std::strcmp(name, fail_name) ? 0 : fail_code; }
int pointer_attributes(unsigned n, const int* which, void** out, unsigned long long) {
  for (unsigned i = 0; i < n; ++i)
    *static_cast<int*>(out[i]) = which[i] == 2 ? 2 : 0;   // memory type: device; not managed; device 0
  return 0;
}
int encode_tiled() { return 0; }
}  // namespace

#define DONE(name) \
  int name() { return result(#name); }

extern "C" {
void fake_fail(const char* name, int code) {
  std::snprintf(fail_name, sizeof fail_name, "%s", name);
  fail_code = code;
}
int fake_launches() { return launches; }
int fake_cluster() { return cluster; }   // of the last launch
void fake_registers(int n) { registers = n; }

void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
DONE(__cudaRegisterFatBinaryEnd)
DONE(__cudaUnregisterFatBinary)
DONE(__cudaRegisterFunction)
DONE(__cudaRegisterVar)
DONE(__cudaPushCallConfiguration)
DONE(__cudaPopCallConfiguration)
int cudaGetDevice(int* d) {
  *d = 0;
  return result("cudaGetDevice");
}
int cudaDeviceGetAttribute(int* v, int attr, int) {
  *v = attr == cudaDevAttrMultiProcessorCount ? 148 : 227 << 10;
  return result("cudaDeviceGetAttribute");
}
int cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  std::memset(a, 0, sizeof *a);
  a->sharedSizeBytes = 1024;
  a->numRegs = registers;
  return result("cudaFuncGetAttributes");
}
int cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* cfg) {
  *n = 148 / static_cast<int>(cfg->gridDim.x);
  return result("cudaOccupancyMaxActiveClusters");
}
int cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n) {
  *n = 1;
  return result("cudaOccupancyMaxActiveBlocksPerMultiprocessor");
}
int cudaLaunchKernel() {
  ++launches;
  cluster = 1;
  return result("cudaLaunchKernel");
}
int cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg) {
  ++launches;
  cluster = 1;
  for (unsigned i = 0; i < cfg->numAttrs; ++i)
    if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = cfg->attrs[i].val.clusterDim.x;
  return result("cudaLaunchKernelExC");
}
int cudaGetSymbolAddress(void** p, const void*) {
  *p = symbol;
  return result("cudaGetSymbolAddress");
}
int cudaGetDriverEntryPoint(const char* name, void** fn, unsigned long long, cudaDriverEntryPointQueryResult* q) {
  *fn = std::strcmp(name, "cuPointerGetAttributes") ? reinterpret_cast<void*>(encode_tiled)
                                                    : reinterpret_cast<void*>(pointer_attributes);
  if (q) *q = cudaDriverEntryPointSuccess;
  return result("cudaGetDriverEntryPoint");
}
const char* cudaGetErrorString(int) { return "an error of the fake runtime"; }
int cudaMalloc(void** p, size_t n) {
  *p = std::malloc(n);
  return result("cudaMalloc");
}
int cudaFree(void* p) {
  std::free(p);
  return result("cudaFree");
}
DONE(cudaGetLastError)
DONE(cudaFuncSetAttribute)
DONE(cudaStreamSynchronize)
DONE(cudaMemcpyAsync)
DONE(cudaMemsetAsync)
DONE(cudaMemset)
DONE(cudaMemcpy)
DONE(cudaStreamEndCapture)
DONE(cudaStreamDestroy)
DONE(cudaStreamCreateWithFlags)
DONE(cudaStreamBeginCapture)
DONE(cudaSetDevice)
DONE(cudaGraphNodeGetType)
DONE(cudaGraphLaunch)
DONE(cudaGraphKernelNodeGetParams)
DONE(cudaGraphInstantiate)
DONE(cudaGraphGetNodes)
DONE(cudaGraphExecKernelNodeSetParams)
DONE(cudaGraphExecDestroy)
DONE(cudaGraphDestroy)
DONE(cudaDeviceSynchronize)
}
