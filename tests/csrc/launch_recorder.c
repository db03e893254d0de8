/* Stand-ins for the HIP entry points that libdg.so uses on the host: kernels
 * are registered and launches recorded by name, nothing is run.  Loaded before
 * libdg.so, with global symbols, in a process of its own. */
#include <stddef.h>
#include <stdint.h>
#include <string.h>

typedef struct { uint32_t x, y, z; } dim3_;

enum { MAX = 4096 };
static struct { const void *host; const char *name; } kernels[MAX];
static const char *launched[1 << 16];
static int n_kernels, n_launched;
static struct { dim3_ grid, block; size_t shared; void *stream; } config;
static void *handle;

void **__hipRegisterFatBinary(const void *data) { (void)data; return &handle; }
void __hipUnregisterFatBinary(void **h) { (void)h; }
void __hipRegisterFunction(void **h, const void *host, char *device, const char *name, unsigned limit,
                           void *tid, void *bid, void *block, void *grid, int *wave) {
  (void)h; (void)device; (void)limit; (void)tid; (void)bid; (void)block; (void)grid; (void)wave;
  if (n_kernels < MAX) {
    kernels[n_kernels].host = host;
    kernels[n_kernels++].name = name;
  }
}
void __hipRegisterVar(void **h, void *var, char *host, char *device, int ext, size_t size, int constant,
                      int global) {
  (void)h; (void)var; (void)host; (void)device; (void)ext; (void)size; (void)constant; (void)global;
}
int __hipPushCallConfiguration(dim3_ grid, dim3_ block, size_t shared, void *stream) {
  config.grid = grid; config.block = block; config.shared = shared; config.stream = stream;
  return 0;
}
int __hipPopCallConfiguration(dim3_ *grid, dim3_ *block, size_t *shared, void **stream) {
  *grid = config.grid; *block = config.block; *shared = config.shared; *stream = config.stream;
  return 0;
}
int hipLaunchKernel(const void *host, dim3_ grid, dim3_ block, void **args, size_t shared, void *stream) {
  (void)grid; (void)block; (void)args; (void)shared; (void)stream;
  for (int i = 0; i < n_kernels; ++i)
    if (kernels[i].host == host && n_launched < 1 << 16) launched[n_launched++] = kernels[i].name;
  return 0;
}
int hipGetLastError(void) { return 0; }
int hipGetDevice(int *d) { *d = 0; return 0; }
int hipStreamGetDevice(void *s, int *d) { (void)s; *d = 0; return 0; }
int hipDeviceGetAttribute(int *v, int attribute, int device) { (void)attribute; (void)device; *v = 256; return 0; }
int hipGetSymbolAddress(void **p, const void *symbol) { (void)symbol; *p = (void *)0x100000; return 0; }

int recorded_kernels(void) { return n_kernels; }
const char *recorded_kernel(int i) { return kernels[i].name; }
int recorded_launches(void) { return n_launched; }
const char *recorded_launch(int i) { return launched[i]; }
