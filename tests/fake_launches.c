/* A CUDA runtime for host-side tests without a GPU whose launches are counted:
 * the program loads libmxsa.so (argv[1]) and prints, for each mxsa_tree_fwd
 * call given as "sequences,tokens of one,query heads,kv heads,keys" (tables
 * just wide enough for the keys, pages of 64), the launches that it made and
 * the first one's cluster size. */
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <dlfcn.h>
#include <stdio.h>
#include <string.h>

#include "../include/mxsa.h"

static int launches, cluster;

cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int d) {
  (void)d;
  return *v = a == cudaDevAttrMultiProcessorCount ? 152 : 1, cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) {
  return (void)f, (void)a, (void)v, cudaSuccess;
}
static CUresult encode() { return CUDA_SUCCESS; }
cudaError_t cudaGetDriverEntryPointByVersion(const char* s, void** p, unsigned v, unsigned long long fl,
                                             enum cudaDriverEntryPointQueryResult* q) {
  (void)s, (void)v, (void)fl;
  if (q) *q = cudaDriverEntryPointSuccess;
  return *p = (void*)encode, cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
  (void)f, (void)args;
  for (unsigned i = 0; i < c->numAttrs && !launches; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = (int)c->attrs[i].val.clusterDim.x;
  return ++launches, cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void* f, int threads, size_t smem) {
  return (void)f, (void)threads, (void)smem, *n = 1, cudaSuccess;
}
cudaError_t cudaPointerGetAttributes(struct cudaPointerAttributes* a, const void* p) {
  memset(a, 0, sizeof(*a));
  a->type = cudaMemoryTypeDevice;
  a->devicePointer = (void*)p;
  return cudaSuccess;
}

int main(int argc, char** argv) {
  void* lib = argc > 1 ? dlopen(argv[1], RTLD_NOW) : NULL;
  if (!lib) return fprintf(stderr, "%s\n", dlerror()), 2;
  __typeof__(&mxsa_shared_workspace_size) size = (__typeof__(size))dlsym(lib, "mxsa_shared_workspace_size");
  __typeof__(&mxsa_tree_fwd) tree = (__typeof__(tree))dlsym(lib, "mxsa_tree_fwd");
  void* const x = (void*)(1ul << 20); /* never read */
  for (int i = 2; i < argc; ++i) {
    int n, tq, hq, hkv, keys;
    if (sscanf(argv[i], "%d,%d,%d,%d,%d", &n, &tq, &hq, &hkv, &keys) != 5) return 3;
    mxsa_problem p;
    memset(&p, 0, sizeof(p));
    p.num_seqs = n, p.total_q = n * tq, p.num_q_heads = hq, p.num_kv_heads = hkv, p.head_dim = 128;
    p.page_size = 64, p.max_pages_per_seq = (keys + 63) / 64, p.num_pages = n * p.max_pages_per_seq;
    p.q_dtype = p.kv_dtype = MXSA_BF16;
    size_t bytes = 0;
    if (size(&p, &bytes) != MXSA_OK) return 4;
    launches = cluster = 0;
    if (tree(&p, x, x, x, x, x, x, x, 4, 0, NULL, NULL, x, bytes, x, NULL, NULL, NULL) != MXSA_OK) return 5;
    printf("%d %d\n", launches, cluster);
  }
  return 0;
}
