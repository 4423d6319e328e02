// A HIP runtime of the host alone: devices without a GPU behind them, memory
// that is never touched and launches that are only counted, any of which can be
// made to fail.  Loaded in the runtime's place it lets tests walk the host side
// of the library's calls.
#include <hip/hip_runtime.h>
#include <stdlib.h>
#include <string.h>

#include <map>

namespace {
hipError_t last = hipSuccess;
int device = 0, launches = 0, attributes = 0, live = 0;
int fail_launch = -1, fail_attribute = -1;  // the n-th from now, from 0
long long lds_launched = 0, bytes = 0;
int over = 0;                              // launches with more LDS than was asked for
std::map<const void*, size_t> limits;
struct {
  dim3 grid, block;
  size_t lds;
  hipStream_t stream;
} pushed;

hipError_t done(hipError_t e) {
  if (e != hipSuccess) last = e;
  return e;
}
}  // namespace

extern "C" {
void host_fail(int launch, int attribute) { fail_launch = launch, fail_attribute = attribute; }
void host_reset() {
  launches = attributes = over = 0, lds_launched = 0;
  limits.clear();
}
int host_launches() { return launches; }
int host_attributes() { return attributes; }
int host_allocations() { return live; }
long long host_bytes() { return bytes; }
int host_over() { return over; }
long long host_lds_launched() { return lds_launched; }

void** __hipRegisterFatBinary(const void*) { return (void**)&device; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, dim3*, dim3*, int*) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}

hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
  pushed = {grid, block, lds, stream};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
  *grid = pushed.grid, *block = pushed.block, *lds = pushed.lds, *stream = pushed.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* kernel, dim3, dim3, void**, size_t lds, hipStream_t) {
  if (fail_launch == 0) {
    fail_launch = -1;
    return done(hipErrorLaunchFailure);
  }
  if (fail_launch > 0) --fail_launch;
  ++launches;
  over += lds > 65536 && (!limits.count(kernel) || lds > limits[kernel]);
  if ((long long)lds > lds_launched) lds_launched = lds;
  return done(hipSuccess);
}
hipError_t hipFuncSetAttribute(const void* kernel, hipFuncAttribute, int value) {
  if (fail_attribute == 0) {
    fail_attribute = -1;
    return done(hipErrorInvalidValue);
  }
  if (fail_attribute > 0) --fail_attribute;
  ++attributes;
  limits[kernel] = value;
  return done(hipSuccess);
}

hipError_t hipGetDevice(int* d) { return *d = device, done(hipSuccess); }
hipError_t hipSetDevice(int d) { return device = d, done(hipSuccess); }
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int) {
  memset(p, 0, sizeof *p);
  strcpy(p->gcnArchName, "gfx950");
  return done(hipSuccess);
}
hipError_t hipDeviceGetAttribute(int* value, hipDeviceAttribute_t, int) { return *value = 256, done(hipSuccess); }
hipError_t hipDeviceSynchronize() { return done(hipSuccess); }
hipError_t hipMalloc(void** p, size_t n) {
  *p = malloc(16);
  ++live, bytes += n;
  return done(hipSuccess);
}
hipError_t hipFree(void* p) {
  free(p);
  if (p) --live;
  return done(hipSuccess);
}
hipError_t hipMemset(void*, int, size_t) { return done(hipSuccess); }
hipError_t hipGetLastError() {
  const hipError_t e = last;
  last = hipSuccess;
  return e;
}
hipError_t hipPeekAtLastError() { return last; }

// what the library links against besides
#define ABSENT(f)               \
  hipError_t f##_(...) asm(#f); \
  hipError_t f##_(...) { return done(hipErrorNotSupported); }
ABSENT(hipEventCreate)
ABSENT(hipEventCreateWithFlags)
ABSENT(hipEventDestroy)
ABSENT(hipEventElapsedTime)
ABSENT(hipEventRecord)
ABSENT(hipEventSynchronize)
ABSENT(hipExtLaunchKernel)
ABSENT(hipGetSymbolAddress)
ABSENT(hipGraphDestroy)
ABSENT(hipGraphExecDestroy)
ABSENT(hipGraphInstantiate)
ABSENT(hipGraphLaunch)
ABSENT(hipMemcpyAsync)
ABSENT(hipOccupancyMaxActiveBlocksPerMultiprocessor)
ABSENT(hipStreamBeginCapture)
ABSENT(hipStreamCreateWithFlags)
ABSENT(hipStreamDestroy)
ABSENT(hipStreamEndCapture)
const char* hipGetErrorString(hipError_t) { return "made to fail"; }
}
