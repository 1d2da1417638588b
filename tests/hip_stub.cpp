// A stand-in for the HIP runtime calls of libwqbmm.so, loaded before it on a
// machine without a GPU: device 0 is a gfx950, memory is never touched, and a launch
// notes which thread made it, on which stream, and takes a while.
#include <hip/hip_runtime.h>

#include <atomic>
#include <chrono>
#include <cstring>
#include <thread>

namespace {
struct Launch {
  int thread;
  hipStream_t stream;
};
constexpr int kMost = 4096;
Launch launches[kMost];
std::atomic<int> launched{0}, allocated{0};
thread_local int thread_number = -1;
thread_local struct {
  dim3 grid, block;
  size_t shared;
  hipStream_t stream;
} configuration;                       // of the launch that the compiler's own code is about to make
}  // namespace

extern "C" {

void stub_thread(int number) { thread_number = number; }
int stub_launches() { return launched; }
int stub_thread_of(int i) { return launches[i].thread; }
uintptr_t stub_stream_of(int i) { return reinterpret_cast<uintptr_t>(launches[i].stream); }
int stub_allocations() { return allocated; }
void stub_reset() { launched = allocated = 0; }

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
  *p = reinterpret_cast<void*>(uintptr_t(0x100000000) * ++allocated);
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
hipError_t hipLaunchKernel(const void*, dim3, dim3, void**, size_t, hipStream_t stream) {
  const int i = launched++;
  if (i < kMost) launches[i] = {thread_number, stream};
  std::this_thread::sleep_for(std::chrono::microseconds(200));
  return hipSuccess;
}

}  // extern "C"
