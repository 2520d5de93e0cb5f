// A CUDA runtime of host memory with two devices: enough to test the paged handle's host side without a GPU.
// hook_after_read sets bits in the status word right after it was copied to the host, as a kernel of another stream would;
// fake_* tell what happened where.
#include <cstdlib>
#include <cstring>

#include <cuda_runtime_api.h>

extern "C" {
int fake_device = 0, fake_freed_on = -1, fake_synced_on = -1, fake_allocs = 0;
unsigned hook_after_read = 0;

cudaError_t cudaGetDevice(int* d) { *d = fake_device; return cudaSuccess; }
cudaError_t cudaSetDevice(int d) {
  if (d < 0 || d > 1) return cudaErrorInvalidDevice;
  fake_device = d;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrMultiProcessorCount ? 148 : 0;
  return cudaSuccess;
}
cudaError_t cudaMalloc(void** p, size_t n) { *p = std::malloc(n); ++fake_allocs; return cudaSuccess; }
cudaError_t cudaFree(void* p) { std::free(p); --fake_allocs; fake_freed_on = fake_device; return cudaSuccess; }
cudaError_t cudaMemset(void* p, int v, size_t n) { std::memset(p, v, n); return cudaSuccess; }
cudaError_t cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t) { std::memset(p, v, n); return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void* to, const void* from, size_t n, cudaMemcpyKind, cudaStream_t) {
  std::memcpy(to, from, n);
  if (n == 4) *static_cast<unsigned*>(const_cast<void*>(from)) |= hook_after_read;
  hook_after_read = 0;
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { fake_synced_on = fake_device; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorName(cudaError_t) { return "name"; }
const char* cudaGetErrorString(cudaError_t) { return "text"; }
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
}
