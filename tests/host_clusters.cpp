// The launches of paged_tables_fork and paged_pages_compact, on a CUDA runtime made up
// here in front of the library's own: host_clusters LIBRARY prints a line for each call,
// its launches as CTAs or as "cluster CTAs".
#include <dlfcn.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <string>

#include "../include/pkv.h"
#include "pkv_internal.h"

static int g_device = 0, g_clusters = 0, g_asked = 0;
static cudaError_t g_answer = cudaSuccess;
static std::string g_launches;

extern "C" {
cudaError_t cudaGetDevice(int* device) { return *device = g_device, cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* value, cudaDeviceAttr, int) { return *value = 152, cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* cfg) {
  ++g_asked;
  if (cfg->numAttrs != 1 || cfg->attrs[0].id != cudaLaunchAttributeClusterDimension || cfg->attrs[0].val.clusterDim.x != 16) abort();
  return *n = g_clusters, g_answer;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void*, void**) {
  for (unsigned i = 0; i < cfg->numAttrs; ++i)
    if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension) g_launches += " cluster";
  g_launches += " " + std::to_string(cfg->gridDim.x);
  return cudaSuccess;
}
}

int main(int, char** argv) {
  void* lib = dlopen(argv[1], RTLD_NOW);
  if (!lib) return std::fprintf(stderr, "%s\n", dlerror()), 1;
  const auto fork = reinterpret_cast<decltype(&paged_tables_fork)>(dlsym(lib, "paged_tables_fork"));
  const auto compact = reinterpret_cast<decltype(&paged_pages_compact)>(dlsym(lib, "paged_pages_compact"));
  const auto bytes = reinterpret_cast<decltype(&paged_pages_workspace_bytes)>(dlsym(lib, "paged_pages_workspace_bytes"));
  auto at = [](uintptr_t i) { return reinterpret_cast<int32_t*>(i << 32); };  // no memory
  auto run = [&](const char* what, int device, long long pages, int batch, int listed) {
    static pkv_pool pool;
    pool.storage = at(1);
    pool.storage_bytes = 3 * 4096 * pages;
    pool.num_pages = pages;
    pool.num_kv_heads = 3;
    pool.device = g_device = device;
    g_launches.clear();
    const int rc = *what == 'f' ? fork(&pool, at(2), batch, at(3), batch, 1, at(4), 100, at(5), at(6), listed, at(7), at(8), at(9), at(10),
                                       at(11), at(12), at(13), bytes(&pool), nullptr)
                                : compact(&pool, at(3), batch, 1, at(4), 100, at(5), at(6), listed, at(7), at(8), at(10), at(11), at(12),
                                          at(13), bytes(&pool), nullptr);
    std::printf("%s of %d in %lld pages, %d listed, device %d: %d,%s; asked %d times\n", what, batch, pages, listed, device, rc,
                g_launches.c_str(), g_asked);
  };
  for (const char* what : {"fork", "compaction"}) {
    g_asked = 0;
    const int most = *what == 'f' ? 128 : 250, list = 6 * 128;  // 640 pieces of work; 256
    g_clusters = 5;
    run(what, 0, 24576, most, list);
    run(what, 0, 24576, most + 1, list);  // too much work
    run(what, 0, 24577, most, list);      // too many chunks
    run(what, 0, 2048, most, list);
    g_clusters = 0;  // a device that runs none
    run(what, 1, 24576, most, list);
    run(what, 1, 2048, 1, list);
    run(what, 0, 24576, most, list);  // the other one still does
    g_answer = cudaErrorInvalidValue;  // no answer
    run(what, 2, 2048, 1, list);
    g_answer = cudaSuccess;
    g_clusters = 1;
    run(what, 2, 2048, 1, list);
    run(what, 70, 2048, 1, list);
    run(what, 70, 2048, 1, list);
  }
}
