// A CUDA runtime without a GPU: linked with the library's own objects in place of the real one, it records the launches
// and keeps the one rule that matters here, that a kernel's dynamic shared memory above 48 KB has to be allowed first, on
// every device and again after a reset.
#include <cstring>
#include <map>
#include <set>
#include <string>
#include <utility>

#include <cuda_runtime_api.h>

namespace {

int g_device = 0, g_sms = 148;
std::map<const void*, std::string> g_names;
std::map<std::pair<int, const void*>, int> g_allowed;
struct Launch {
  const void* kernel;
  dim3 grid, block;
  size_t smem;
  unsigned cluster;
};
Launch g_last;
int g_launches = 0;
Launch g_pushed;
cudaError_t g_error = cudaSuccess;
char g_symbols[1 << 16];

cudaError_t launch(const Launch& l) {
  const auto at = g_allowed.find({g_device, l.kernel});
  const size_t most = at == g_allowed.end() ? 48 * 1024 : size_t(at->second);
  if (l.smem > most) return g_error = cudaErrorInvalidValue;
  const unsigned long long blocks = 1ull * l.grid.x;
  if (blocks == 0 || blocks > 0x7fffffffull || l.grid.y == 0 || l.grid.y > 65535 || l.grid.z == 0 || l.grid.z > 65535)
    return g_error = cudaErrorInvalidConfiguration;
  g_last = l;
  ++g_launches;
  return cudaSuccess;
}

}  // namespace

extern "C" {

// what the tests ask
void fake_device(int device) { g_device = device; }
void fake_reset() { g_allowed.clear(); }
int fake_launches() { return g_launches; }
const char* fake_kernel() { return g_names[g_last.kernel].c_str(); }
void fake_last(unsigned* v) {
  v[0] = g_last.grid.x;
  v[1] = g_last.grid.y;
  v[2] = g_last.block.x;
  v[3] = unsigned(g_last.smem);
  v[4] = g_last.cluster;
}

cudaError_t cudaGetDevice(int* d) { return *d = g_device, cudaSuccess; }
cudaError_t cudaSetDevice(int d) { return g_device = d, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { return *v = g_sms, cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) g_allowed[{g_device, f}] = v;
  return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** p, const void*) { return *p = g_symbols, cudaSuccess; }
cudaError_t cudaMemcpyFromSymbol(void* to, const void*, size_t n, size_t, cudaMemcpyKind) { return memset(to, 0, n), cudaSuccess; }
cudaError_t cudaMemcpyToSymbol(const void*, const void*, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMalloc(void** p, size_t) { return *p = g_symbols, cudaSuccess; }
cudaError_t cudaFree(void*) { return cudaSuccess; }
cudaError_t cudaEventCreate(cudaEvent_t* e) { return *e = nullptr, cudaErrorNotSupported; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t cudaEventSynchronize(cudaEvent_t) { return cudaErrorNotSupported; }
cudaError_t cudaEventElapsedTime(float*, cudaEvent_t, cudaEvent_t) { return cudaErrorNotSupported; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
const char* cudaGetErrorName(cudaError_t) { return "fake"; }
const char* cudaGetErrorString(cudaError_t) { return "fake error"; }
cudaError_t cudaGetLastError(void) { return std::exchange(g_error, cudaSuccess); }

cudaError_t cudaLaunchKernel(const void* f, dim3 g, dim3 b, void**, size_t smem, cudaStream_t) { return launch({f, g, b, smem, 1}); }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  unsigned cluster = 1;
  for (unsigned k = 0; k < c->numAttrs; ++k)
    if (c->attrs[k].id == cudaLaunchAttributeClusterDimension) cluster = c->attrs[k].val.clusterDim.x;
  return launch({f, c->gridDim, c->blockDim, c->dynamicSmemBytes, cluster});
}

// what the compiler's host code calls
unsigned __cudaPushCallConfiguration(dim3 g, dim3 b, size_t smem, cudaStream_t) {
  g_pushed = {nullptr, g, b, smem, 1};
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* g, dim3* b, size_t* smem, void* stream) {
  *g = g_pushed.grid;
  *b = g_pushed.block;
  *smem = g_pushed.smem;
  *static_cast<cudaStream_t*>(stream) = nullptr;
  return cudaSuccess;
}
void** __cudaRegisterFatBinary(void*) {
  static void* handle = nullptr;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, uint3*, uint3*, dim3*, dim3*, int*) {
  g_names[host] = name;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}

}  // extern "C"
