// The runtime of fake_cudart.cpp, which also keeps each launch's kernel (its mangled name), grid
// and block.
#include <cuda_runtime_api.h>

#define __cudaRegisterFunction not_recorded_register
#define cudaLaunchKernelExC not_recorded_launch
#include "fake_cudart.cpp"
#undef __cudaRegisterFunction
#undef cudaLaunchKernelExC

#include <string>
#include <vector>

namespace {

struct Launch {
  std::string kernel;
  int grid, block;
};
std::vector<Launch> g_recorded;
std::map<const void*, std::string>& kernels() {
  static std::map<const void*, std::string> m;   // (filled by constructors of other files)
  return m;
}

}  // namespace

extern "C" {

void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, uint3*, uint3*, dim3*, dim3*,
                            int*) {
  kernels()[host] = name;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  g_recorded.push_back({kernels()[f], (int)c->gridDim.x, (int)c->blockDim.x});
  return launched();
}
void recorded_clear() { g_recorded.clear(); }
int recorded_launches() { return (int)g_recorded.size(); }
const char* recorded_kernel(int i) { return g_recorded[i].kernel.c_str(); }
int recorded_grid(int i) { return g_recorded[i].grid; }
int recorded_block(int i) { return g_recorded[i].block; }

}  // extern "C"
