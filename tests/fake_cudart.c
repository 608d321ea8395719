/* A CUDA runtime for tests without a GPU, preloaded ahead of the real one: one sm_103
 * device of 152 multiprocessors whose calls all succeed, or, of cudaOccupancyMaxActiveClusters,
 * fail while a test asks for it.  Launches run nothing; their kernels' names are kept. */
#define _GNU_SOURCE
#include <dlfcn.h>
#include <string.h>

#include <cuda_runtime_api.h>

static int fail_occupancy, n_launches;
static const char* launched[64];
static struct { const void* host; const char* name; } kernels[1024];
static int n_kernels;
static int status_word;

void fake_fail_occupancy(int on) { fail_occupancy = on; }
int fake_launches(void) { return n_launches; }
const char* fake_launched(int i) { return launched[i]; }
void fake_forget(void) { n_launches = 0; }

static void launch(const void* f) {
  if (n_launches == 64) return;
  launched[n_launches] = "?";
  for (int i = 0; i < n_kernels; ++i)
    if (kernels[i].host == f) launched[n_launches] = kernels[i].name;
  ++n_launches;
}

/* the names of the kernels, as the library registers them when it is loaded */
void __cudaRegisterFunction(void** handle, const char* host, char* device, const char* name, int limit, void* tid,
                            void* bid, void* bd, void* gd, int* ws) {
  static void (*real)(void**, const char*, char*, const char*, int, void*, void*, void*, void*, int*);
  if (!real) *(void**)&real = dlsym(RTLD_NEXT, "__cudaRegisterFunction");
  if (n_kernels < 1024) {
    kernels[n_kernels].host = host;
    kernels[n_kernels++].name = strdup(name);
  }
  if (real) real(handle, host, device, name, limit, tid, bid, bd, gd, ws);
}

cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int d) {
  (void)d;
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3
       : a == cudaDevAttrMultiProcessorCount ? 152 : 0;
  return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** p, const void* s) { (void)s; *p = &status_word; return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(struct cudaFuncAttributes* a, const void* f) {
  (void)f;
  memset(a, 0, sizeof *a);
  a->numRegs = 80;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) { (void)f; (void)a; (void)v; return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* c) {
  (void)f; (void)c;
  if (fail_occupancy) return cudaErrorUnknown;
  *n = 74;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
  (void)c; (void)args;
  launch(f);
  return cudaSuccess;
}

/* tensor maps: any bytes do, nothing reads them */
static int encode(void* map, ...) { memset(map, 0, 128); return 0; }
cudaError_t cudaGetDriverEntryPointByVersion(const char* s, void** f, unsigned int v, unsigned long long flags,
                                             enum cudaDriverEntryPointQueryResult* q) {
  (void)s; (void)v; (void)flags;
  *f = (void*)encode;
  if (q) *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
