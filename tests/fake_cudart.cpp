// A CUDA runtime without a GPU, for the library's host code: device memory is host
// memory, kernels are counted but not run, and what a call leaves queued is kept per
// stream until something waits for it.
//
// Linked with the library's objects in place of the CUDA runtime. fake_* is what a
// test looks at and sets.
#include <cuda_runtime_api.h>

#include <cstdlib>
#include <cstring>
#include <map>
#include <set>

namespace {

int g_device = 0;                            // the current one, of two
std::map<cudaStream_t, int> g_queued;        // memory operations not yet waited for
std::set<cudaStream_t> g_streams;            // those that the library made
std::map<void*, int> g_allocs;               // and the device of each
int g_alloc_calls = 0, g_launches = 0, g_launch_device = -1;

cudaError_t launched() {
  ++g_launches;
  g_launch_device = g_device;
  return cudaSuccess;
}

}  // namespace

extern "C" {

void fake_set_device(int d) { g_device = d; }
int fake_queued() {
  int n = 0;
  for (const auto& s : g_queued) n += s.second;
  return n;
}
int fake_streams() { return (int)g_streams.size(); }
int fake_alloc_calls() { return g_alloc_calls; }
int fake_allocs(int device) {
  int n = 0;
  for (const auto& a : g_allocs) n += a.second == device;
  return n;
}
int fake_launches() { return g_launches; }

cudaError_t cudaGetDevice(int* d) {
  *d = g_device;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  *v = 152;
  return cudaSuccess;
}
cudaError_t cudaMalloc(void** p, size_t n) {
  *p = std::aligned_alloc(256, (n + 255) / 256 * 256);
  std::memset(*p, 0xA5, n);
  g_allocs[*p] = g_device;
  ++g_alloc_calls;
  return cudaSuccess;
}
cudaError_t cudaFree(void* p) {
  g_queued.clear();
  g_allocs.erase(p);
  std::free(p);
  return cudaSuccess;
}
// (to device memory the host does not wait, and from pageable memory only for the
// copy out of it)
cudaError_t cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t s) {
  std::memset(p, v, n);
  ++g_queued[s];
  return cudaSuccess;
}
cudaError_t cudaMemset(void* p, int v, size_t n) { return cudaMemsetAsync(p, v, n, nullptr); }
cudaError_t cudaMemcpyAsync(void* d, const void* s, size_t n, cudaMemcpyKind, cudaStream_t st) {
  std::memcpy(d, s, n);
  ++g_queued[st];
  return cudaSuccess;
}
cudaError_t cudaMemcpy(void* d, const void* s, size_t n, cudaMemcpyKind k) {
  std::memcpy(d, s, n);
  if (k == cudaMemcpyDeviceToHost) g_queued.erase(nullptr);
  else ++g_queued[nullptr];
  return cudaSuccess;
}
cudaError_t cudaStreamCreateWithFlags(cudaStream_t* s, unsigned) {
  *s = reinterpret_cast<cudaStream_t>(std::malloc(1));
  g_streams.insert(*s);
  return cudaSuccess;
}
cudaError_t cudaStreamDestroy(cudaStream_t s) {
  g_streams.erase(s);
  std::free(s);
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t s) {
  g_queued.erase(s);
  return cudaSuccess;
}
cudaError_t cudaDeviceSynchronize() {
  g_queued.clear();
  return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** p, const void*) {
  static char scratch[256];
  *p = scratch;
  return cudaSuccess;
}
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  std::memset(a, 0, sizeof(*a));
  a->numRegs = 255;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* r) {
  *f = nullptr;
  if (r) *r = cudaDriverEntryPointSymbolNotFound;
  return cudaErrorNotSupported;
}
const char* cudaGetErrorString(cudaError_t) { return "an error of the test's runtime"; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) { return launched(); }

// what the compiler's launch stubs and registrations call
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, void*) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaSuccess; }
cudaError_t __cudaGetKernel(void** k, const void* f) {
  *k = const_cast<void*>(f);
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(void*, dim3, dim3, void**, size_t, cudaStream_t) { return launched(); }
void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}

}  // extern "C"
