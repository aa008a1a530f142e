// A HIP runtime that launches nothing and writes down what it is asked to launch, linked with
// the host side of libepget's sources: which kernel a call picks, on which grid, without a
// device.  Test infrastructure only.
#include <cxxabi.h>
#include <hip/hip_runtime.h>

#include <cstdlib>
#include <cstring>
#include <map>
#include <string>
#include <vector>

namespace {
struct Launch {
  std::string kernel;
  uint32_t grid[3], block[3];
};
std::map<const void*, std::string>& kernels() {
  static std::map<const void*, std::string> k;
  return k;
}
std::vector<Launch> launches;
struct {
  dim3 grid, block;
  size_t shared;
  hipStream_t stream;
} config;

// without the namespace and the arguments
std::string plain(const char* mangled) {
  int rc = 0;
  char* d = abi::__cxa_demangle(mangled, nullptr, nullptr, &rc);
  std::string s = rc == 0 ? d : mangled;
  free(d);
  for (size_t at; (at = s.find("(anonymous namespace)::")) != std::string::npos;) s.erase(at, 23);
  if (s.rfind("void ", 0) == 0) s.erase(0, 5);
  int depth = 0;
  for (size_t i = 0; i < s.size(); i++) {
    depth += (s[i] == '<') - (s[i] == '>');
    if (s[i] == '(' && depth == 0) return s.substr(0, i);
  }
  return s;
}
}  // namespace

extern "C" {

// ---- what the test reads
int recorder_kernels() { return (int)kernels().size(); }
const char* recorder_kernel(int i) { return std::next(kernels().begin(), i)->second.c_str(); }
int recorder_launches() { return (int)launches.size(); }
const char* recorder_launch(int i, uint32_t* sizes) {
  memcpy(sizes, launches[i].grid, 12);
  memcpy(sizes + 3, launches[i].block, 12);
  return launches[i].kernel.c_str();
}
void recorder_clear() { launches.clear(); }

// ---- what the sources call
void** __hipRegisterFatBinary(const void*) {
  static void* handle;
  return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*,
                           void*, void*, void*, int*) {
  kernels()[host] = plain(name);
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t stream) {
  config = {grid, block, shared, stream};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
  *grid = config.grid;
  *block = config.block;
  *shared = config.shared;
  *stream = config.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void**, size_t, hipStream_t) {
  launches.push_back({kernels()[f], {grid.x, grid.y, grid.z}, {block.x, block.y, block.z}});
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return ""; }
hipError_t hipGetDevice(int* device) {
  *device = 0;
  return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int) {
  memset(p, 0, sizeof *p);
  strcpy(p->gcnArchName, "gfx950");
  return hipSuccess;
}

}  // extern "C"
