/* A CUDA runtime that launches nothing, for tests of the library's host code
 * without a GPU: its objects are linked against this file in place of the
 * runtime. It has two devices, of 152 and 100 SMs, and keeps what a launch
 * depends on apart for each: a kernel's limit of dynamic shared memory is 48 KB
 * on a device until it is raised there, and a launch or an occupancy query past
 * it fails, as on a GPU. Launches are recorded. */
#include <stddef.h>
#include <string.h>

typedef struct { unsigned x, y, z; } dim3_t;
typedef struct { int id; char pad[4]; union { char raw[64]; int value; dim3_t dim; } val; } attr_t;
typedef struct { dim3_t grid, block; size_t smem; void *stream; attr_t *attrs; unsigned num; } config_t;
typedef struct { const char *name; int device; unsigned grid[3], block, smem, cluster; } launch_t;

enum { MAX = 4096, ERR = 1 };
static const int sms[2] = {152, 100};
static struct { const void *host; const char *name; size_t limit[2]; } kernels[MAX];
static int n_kernels, device, refuse;
static launch_t launches[MAX];
static int n_launches;

/* ---- for the test */
void fake_device(int d) { device = d; }
void fake_refuse(int n) { refuse = n; } /* the next n settings of an attribute fail */
int fake_launches(void) { return n_launches; }
const launch_t *fake_launch(int i) { return &launches[i]; }
void fake_clear(void) { n_launches = 0; }

/* ---- registration of kernels */
void **__cudaRegisterFatBinary(void *f) { static void *h; (void)f; return &h; }
void __cudaRegisterFatBinaryEnd(void **h) { (void)h; }
void __cudaUnregisterFatBinary(void **h) { (void)h; }
void __cudaRegisterVar(void **h, char *v, char *a, const char *n, int e, size_t s, int c, int g) {
  (void)h; (void)v; (void)a; (void)n; (void)e; (void)s; (void)c; (void)g;
}
void __cudaRegisterFunction(void **h, const char *host, char *fun, const char *name, int limit, void *t, void *b, void *bd,
                            void *gd, int *w) {
  (void)h; (void)fun; (void)limit; (void)t; (void)b; (void)bd; (void)gd; (void)w;
  if (n_kernels == MAX) return;
  kernels[n_kernels].host = host;
  kernels[n_kernels].name = name;
  kernels[n_kernels].limit[0] = kernels[n_kernels].limit[1] = 48 * 1024;
  ++n_kernels;
}
static int find(const void *host) {
  for (int i = 0; i < n_kernels; ++i)
    if (kernels[i].host == host) return i;
  return -1;
}

/* ---- what the library's launches ask for */
int cudaGetDevice(int *d) { *d = device; return 0; }
int cudaDeviceGetAttribute(int *v, int attr, int d) { *v = attr == 16 ? sms[d] : 0; return 0; } /* 16: SM count */
int cudaFuncSetAttribute(const void *f, int attr, int v) {
  const int k = find(f);
  if (k < 0) return ERR;
  if (refuse > 0) { --refuse; return ERR; }
  if (attr == 8) kernels[k].limit[device] = (size_t)v; /* 8: dynamic shared memory */
  return 0;
}
int cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int *n, const void *f, int block, size_t smem, unsigned flags) {
  const int k = find(f);
  (void)block; (void)flags;
  if (k < 0 || smem > kernels[k].limit[device]) return ERR;
  *n = 4;
  return 0;
}
int cudaLaunchKernelExC(const config_t *c, const void *f, void **args) {
  const int k = find(f);
  (void)args;
  if (k < 0 || c->smem > kernels[k].limit[device] || !c->grid.x || !c->grid.y || !c->grid.z || n_launches == MAX) return ERR;
  launch_t *l = &launches[n_launches++];
  l->name = kernels[k].name;
  l->device = device;
  l->grid[0] = c->grid.x, l->grid[1] = c->grid.y, l->grid[2] = c->grid.z;
  l->block = c->block.x;
  l->smem = (unsigned)c->smem;
  l->cluster = 1;
  for (unsigned i = 0; i < c->num; ++i)
    if (c->attrs[i].id == 4) l->cluster = c->attrs[i].val.dim.x; /* 4: cluster dimension */
  return 0;
}

/* ---- what the calls under test do not reach */
#define NEVER(name) int name(void) { return ERR; }
NEVER(__cudaGetKernel) NEVER(__cudaLaunchKernel) NEVER(__cudaPopCallConfiguration) NEVER(__cudaPushCallConfiguration)
NEVER(cudaEventCreate) NEVER(cudaEventDestroy) NEVER(cudaEventElapsedTime) NEVER(cudaEventRecord) NEVER(cudaEventSynchronize)
NEVER(cudaGetDriverEntryPointByVersion) NEVER(cudaGetLastError) NEVER(cudaGetSymbolAddress) NEVER(cudaHostGetDevicePointer)
NEVER(cudaMemcpy) NEVER(cudaMemcpyAsync) NEVER(cudaMemsetAsync) NEVER(cudaStreamSynchronize)
