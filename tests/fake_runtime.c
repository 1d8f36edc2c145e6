/* A CUDA runtime for host-side tests without a GPU: devices are numbers, a
 * launch does nothing, and a kernel's shared-memory limit is kept per device,
 * as the real runtime keeps it -- a launch with more than 48 KB of dynamic
 * shared memory fails on a device where the limit was not raised.  The
 * program loads libmxsa.so (argv[1]), whose runtime calls resolve to the
 * functions here, and calls its entry points on several devices (argv[2]
 * "devices") or around a failure (argv[2] the kind, argv[3] the call). */
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <dlfcn.h>
#include <stdio.h>
#include <string.h>

#include "../include/mxsa.h"

static int device, fail_attributes, fail_entry_points;
static const void* raised[8][64];

static int is_raised(const void* f) {
  for (int i = 0; i < 64; ++i)
    if (raised[device][i] == f) return 1;
  return 0;
}

cudaError_t cudaGetDevice(int* d) { return *d = device, cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int d) {
  (void)d;
  *v = a == cudaDevAttrMultiProcessorCount ? 152 : 1;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) {
  (void)v;
  if (a != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaSuccess;
  if (fail_attributes > 0) return --fail_attributes, cudaErrorMemoryAllocation;
  for (int i = 0; i < 64 && !is_raised(f); ++i)
    if (!raised[device][i]) raised[device][i] = f;
  return cudaSuccess;
}
static CUresult encode() { return CUDA_SUCCESS; }
cudaError_t cudaGetDriverEntryPointByVersion(const char* s, void** p, unsigned v, unsigned long long fl,
                                             enum cudaDriverEntryPointQueryResult* q) {
  (void)s, (void)v, (void)fl;
  if (fail_entry_points > 0) return --fail_entry_points, cudaErrorInitializationError;
  *p = (void*)encode;
  if (q) *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
  (void)args;
  return c->dynamicSmemBytes > 48 * 1024 && !is_raised(f) ? cudaErrorInvalidValue : cudaSuccess;
}
cudaError_t cudaLaunchCooperativeKernel(const void* f, dim3 g, dim3 b, void** args, size_t smem, cudaStream_t st) {
  (void)f, (void)g, (void)b, (void)args, (void)smem, (void)st;
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t st) {
  (void)p, (void)v, (void)n, (void)st;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void* f, int threads, size_t smem) {
  (void)f, (void)threads, (void)smem;
  return *n = 1, cudaSuccess;
}
cudaError_t cudaPointerGetAttributes(struct cudaPointerAttributes* a, const void* p) {
  memset(a, 0, sizeof(*a));
  a->type = cudaMemoryTypeDevice;
  a->devicePointer = (void*)p;
  return cudaSuccess;
}

static void* lib;
static void* fn(const char* name) {
  void* p = dlsym(lib, name);
  if (!p) fprintf(stderr, "%s: %s\n", name, dlerror());
  return p;
}

/* one call of an entry point that launches kernels with raised limits */
static mxsa_status call(int which, int kv) {
  void* const x = (void*)(1ul << 20); /* never read */
  mxsa_problem p;
  memset(&p, 0, sizeof(p));
  p.num_seqs = 3, p.total_q = 5, p.num_q_heads = 16, p.num_kv_heads = 2, p.head_dim = 128, p.topk = 4;
  p.page_size = 64, p.num_pages = 10, p.max_pages_per_seq = 10, p.q_dtype = MXSA_BF16, p.kv_dtype = kv;
  size_t a = 0, b = 0, c = 0;
  switch (which) {
    case 0:
      return ((__typeof__(&mxsa_dense_fwd))fn("mxsa_dense_fwd"))(&p, x, x, x, x, x, x, x, x, NULL, NULL);
    case 1:
      ((__typeof__(&mxsa_shared_workspace_size))fn("mxsa_shared_workspace_size"))(&p, &a);
      return ((__typeof__(&mxsa_dense_shared_fwd))fn("mxsa_dense_shared_fwd"))(&p, x, x, x, x, x, x, 0, NULL, NULL, x,
                                                                             a, x, x, NULL, NULL);
    case 2:
      ((__typeof__(&mxsa_workspace_size))fn("mxsa_workspace_size"))(&p, &a, &b, &c);
      return ((__typeof__(&mxsa_kvouter_fwd))fn("mxsa_kvouter_fwd"))(&p, x, x, x, x, x, a, x, b, 0, x, c, NULL);
    default:
      ((__typeof__(&mxsa_select_workspace_size))fn("mxsa_select_workspace_size"))(&p, 64, &a);
      return ((__typeof__(&mxsa_select_blocks))fn("mxsa_select_blocks"))(&p, 64, x, x, x, x, x, x, a, x, NULL, NULL);
  }
}

static int bad;
static void expect(const char* what, int which, int kv, int ok) {
  static const char* names[4] = {"mxsa_dense_fwd", "mxsa_dense_shared_fwd", "mxsa_kvouter_fwd", "mxsa_select_blocks"};
  const mxsa_status s = call(which, kv);
  if ((s == MXSA_OK) == ok) return;
  printf("%s, device %d, kv type %d, %s: status %d\n", names[which], device, kv, what, s);
  bad = 1;
}

int main(int argc, char** argv) {
  lib = argc > 2 ? dlopen(argv[1], RTLD_NOW) : NULL;
  if (!lib) return fprintf(stderr, "%s\n", dlerror()), 2;
  if (!strcmp(argv[2], "devices")) {
    for (device = 0; device < 3; ++device)
      for (int which = 0; which < 4; ++which)
        for (int kv = 0; kv < 4; ++kv) {
          const int runs = kv == MXSA_BF16 || (which == 2 && kv != MXSA_FP16) || (which == 3 && kv == MXSA_FP8_E4M3);
          if (runs) expect("first call", which, kv, 1), expect("second call", which, kv, 1);
        }
  } else {  /* one failure of the runtime in the call argv[3], then none */
    const int which = argv[3][0] - '0';
    if (!strcmp(argv[2], "attributes")) fail_attributes = 1;
    else fail_entry_points = 1;
    expect("failing", which, MXSA_BF16, 0);
    fail_attributes = fail_entry_points = 0;
    expect("after the failure", which, MXSA_BF16, 1);
  }
  return bad;
}
