// The calls of the HIP runtime that the library makes, for machines without a
// GPU: several devices, of which each has to allow a kernel's dynamic LDS past
// 64 KB before it takes a launch with it, and nothing is run.
#include <hip/hip_runtime_api.h>

#include <set>
#include <utility>

static int current = 0;
static std::set<std::pair<int, const void*>> allowed;
static dim3 grid, block;
static size_t shared;
static hipStream_t stream;
static hipError_t last = hipSuccess;

extern "C" {

int fake_launches[8] = {}, fake_refused[8] = {}, fake_large[8] = {};
void fake_device(int device) { current = device; }

hipError_t hipGetDevice(int* device) {
  *device = current;
  return hipSuccess;
}
hipError_t hipFuncSetAttribute(const void* f, hipFuncAttribute, int) {
  allowed.insert({current, f});
  return hipSuccess;
}
hipError_t __hipPushCallConfiguration(dim3 g, dim3 b, size_t s, hipStream_t st) {
  grid = g, block = b, shared = s, stream = st;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* g, dim3* b, size_t* s, hipStream_t* st) {
  *g = grid, *b = block, *s = shared, *st = stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3, dim3, void**, size_t s, hipStream_t) {
  const bool ok = s <= 64 * 1024 || allowed.count({current, f}) != 0;
  last = ok ? hipSuccess : hipErrorInvalidValue;
  if (s > 64 * 1024) ++fake_large[current];
  ++(ok ? fake_launches : fake_refused)[current];
  return last;
}
hipError_t hipGetLastError() {
  const hipError_t e = last;
  last = hipSuccess;
  return e;
}
hipError_t hipExtLaunchKernel(const void* f, dim3 g, dim3 b, void** args, size_t s, hipStream_t st,
                              hipEvent_t, hipEvent_t, int) {
  return hipLaunchKernel(f, g, b, args, s, st);
}
hipError_t hipEventRecord(hipEvent_t, hipStream_t) { return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* value, hipDeviceAttribute_t, int) {
  *value = 256;
  return hipSuccess;
}
hipError_t hipOccupancyMaxActiveBlocksPerMultiprocessor(int* blocks, const void*, int, size_t) {
  *blocks = 2;
  return hipSuccess;
}
void** __hipRegisterFatBinary(const void*) {
  static void* handle = nullptr;
  return &handle;
}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, dim3*,
                           dim3*, int*) {}
void __hipRegisterVar(void**, void*, char*, const char*, int, size_t, int, int) {}
void __hipUnregisterFatBinary(void**) {}

}  // extern "C"
