// A CUDA runtime of host functions, preloaded under libmsa by the tests of its
// host side: device memory is host memory, kernels are only noted down, and any
// allocation on the host or the device can be made to fail.
#include <cuda_runtime_api.h>

#include <atomic>
#include <cstdlib>
#include <cstring>
#include <new>
#include <vector>

namespace {

struct Event {
  const void* func;
  int kind;  // 0: limit of dynamic shared memory set, 1: launch
  long bytes;
};
std::atomic<long> live_host{0}, live_device{0};
int device = 0;
std::atomic<long> host_left{-1}, device_left{-1};  // allocations until they fail; below 0: they do not

// a vector of its own allocator, outside the counts
template <typename T>
struct Raw {
  using value_type = T;
  Raw() = default;
  template <typename U>
  Raw(const Raw<U>&) {}
  T* allocate(size_t n) { return static_cast<T*>(malloc(n * sizeof(T))); }
  void deallocate(T* p, size_t) { free(p); }
  template <typename U>
  bool operator==(const Raw<U>&) const { return true; }
  template <typename U>
  bool operator!=(const Raw<U>&) const { return false; }
};
std::vector<Event, Raw<Event>> events;

bool fails(std::atomic<long>& left) {  // from the one asked for on, until told otherwise
  if (left < 0) return false;
  if (left == 0) return true;
  --left;
  return false;
}

int encode(void* map, ...) {
  memset(map, 0, 128);
  return 0;
}

}  // namespace

void* operator new(size_t n) {
  void* p = fails(host_left) ? nullptr : malloc(n ? n : 1);
  if (!p) throw std::bad_alloc();
  ++live_host;
  return p;
}
void* operator new(size_t n, const std::nothrow_t&) noexcept {
  void* p = fails(host_left) ? nullptr : malloc(n ? n : 1);
  live_host += p != nullptr;
  return p;
}
void operator delete(void* p) noexcept {
  live_host -= p != nullptr;
  free(p);
}
void operator delete(void* p, size_t) noexcept { operator delete(p); }
void operator delete(void* p, const std::nothrow_t&) noexcept { operator delete(p); }

extern "C" {

void fake_fail(long on_host, long on_device) { host_left = on_host, device_left = on_device; }
void fake_set_device(int d) { device = d; }
long fake_live_host() { return live_host; }
long fake_live_device() { return live_device; }
long fake_events(Event* out, long most) {
  const long n = static_cast<long>(events.size()) < most ? static_cast<long>(events.size()) : most;
  for (long i = 0; i < n; ++i) out[i] = events[i];
  return n;
}

cudaError_t cudaGetDevice(int* d) {
  *d = device;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  *v = 152;  // SMs: the only one that is asked for
  return cudaSuccess;
}
cudaError_t cudaMalloc(void** p, size_t n) {
  *p = fails(device_left) ? nullptr : malloc(n);
  if (!*p) return cudaErrorMemoryAllocation;
  ++live_device;
  return cudaSuccess;
}
cudaError_t cudaFree(void* p) {
  live_device -= p != nullptr;
  free(p);
  return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void* d, const void* s, size_t n, cudaMemcpyKind, cudaStream_t) {
  memcpy(d, s, n);
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void* d, int v, size_t n, cudaStream_t) {
  memset(d, v, n);
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  memset(a, 0, sizeof(*a));
  a->numRegs = 128;  // what the kernels with register splits are compiled for
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* func, cudaFuncAttribute attr, int value) {
  if (attr == cudaFuncAttributeMaxDynamicSharedMemorySize) events.push_back({func, 0, value});
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void* func, void**) {
  events.push_back({func, 1, static_cast<long>(cfg->dynamicSmemBytes)});
  return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *fn = reinterpret_cast<void*>(encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

}  // extern "C"
