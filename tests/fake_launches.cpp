// The runtime of host functions, that also counts the bytes that are uploaded and
// notes down grids and clusters.
#define cudaMemcpyAsync noted_memcpy_async
#define cudaLaunchKernelExC noted_launch
#include "fake_cudart.cpp"
#undef cudaMemcpyAsync
#undef cudaLaunchKernelExC

namespace {
long uploaded = 0;
struct Shape {
  int ctas, cluster;
};
std::vector<Shape, Raw<Shape>> shapes;
}  // namespace

extern "C" {

long fake_uploaded() { return uploaded; }
// the last launch: CTAs, kernel, cluster size
int fake_last_ctas() { return shapes.back().ctas; }
const void* fake_last_func() { return events.back().func; }
int fake_last_cluster() { return shapes.back().cluster; }

cudaError_t cudaMemcpyAsync(void* d, const void* s, size_t n, cudaMemcpyKind kind, cudaStream_t st) {
  uploaded += static_cast<long>(n);
  return noted_memcpy_async(d, s, n, kind, st);
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void* func, void** args) {
  Shape x{static_cast<int>(cfg->gridDim.x), 1};
  for (unsigned i = 0; i < cfg->numAttrs; ++i)
    if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension) x.cluster = static_cast<int>(cfg->attrs[i].val.clusterDim.x);
  shapes.push_back(x);
  return noted_launch(cfg, func, args);
}

}  // extern "C"
