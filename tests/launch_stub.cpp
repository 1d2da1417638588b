// A stand-in for the HIP runtime calls of libwqbmm.so, loaded before it on a machine
// without a GPU: device 0 is a gfx950, memory is never touched, and a launch notes its
// kernel's name and its sizes.  As the runtime does, it refuses 2^32 threads and more
// along x.
#include <hip/hip_runtime.h>

#include <cstring>
#include <map>
#include <string>
#include <vector>

namespace {
struct Launch {
  std::string kernel;
  uint32_t grid, block;
};
std::map<const void*, std::string>& kernels() {
  static std::map<const void*, std::string> all;      // filled while the library is loaded
  return all;
}
std::vector<Launch> launches;
int allocated = 0;
struct {
  dim3 grid, block;
  size_t shared;
  hipStream_t stream;
} configuration;
}  // namespace

extern "C" {

int stub_kernels() { return (int)kernels().size(); }
const char* stub_kernel(int i) { return std::next(kernels().begin(), i)->second.c_str(); }
int stub_launches() { return (int)launches.size(); }
const char* stub_launched(int i) { return launches[i].kernel.c_str(); }
uint32_t stub_grid(int i) { return launches[i].grid; }
uint32_t stub_block(int i) { return launches[i].block; }
void stub_reset() { launches.clear(); }

void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
  kernels()[host] = name;
}
hipError_t hipGetDevice(int* device) {
  *device = 0;
  return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int) {
  std::memset(p, 0, sizeof *p);
  std::strcpy(p->gcnArchName, "gfx950");
  return hipSuccess;
}
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) {
  *s = hipStreamCaptureStatusNone;
  return hipSuccess;
}
hipError_t hipMalloc(void** p, size_t) {
  *p = reinterpret_cast<void*>(uintptr_t(1) << 40 | uintptr_t(0x1000) * ++allocated);
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t stream) {
  configuration = {grid, block, shared, stream};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
  *grid = configuration.grid;
  *block = configuration.block;
  *shared = configuration.shared;
  *stream = configuration.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* host, dim3 grid, dim3 block, void**, size_t, hipStream_t) {
  launches.push_back({kernels()[host], grid.x, block.x});
  return (uint64_t)grid.x * block.x < (uint64_t(1) << 32) ? hipSuccess : hipErrorInvalidConfiguration;
}

}  // extern "C"
