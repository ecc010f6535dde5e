/* Stands in for the HIP runtime's launch calls, so that the library's host code can be run without a
 * device: every launch is recorded with its kernel's name, grid, block and LDS bytes and the dynamic LDS
 * limit that the kernel has at that moment; nothing is launched. Loaded (RTLD_GLOBAL) before the library,
 * its definitions come first. The device it pretends to be has 256 compute units. */
#define _GNU_SOURCE
#include <dlfcn.h>
#include <stddef.h>
#include <stdint.h>

typedef struct { uint32_t x, y, z; } dim3_t;
typedef struct { const void* f; uint32_t grid, block; uint64_t lds, limit; } launch_t;

enum { MOST = 1 << 20, FUNCS = 512 };
static launch_t launches[MOST];
static int n_launches;
/* the dynamic LDS limit of each kernel: 64 KiB until it is set; how often it was set to another value */
static struct { const void* f; uint64_t limit; int changes; } limits[FUNCS];
static int n_limits;
static struct { dim3_t grid, block; size_t lds; void* stream; } config;

static int limit_of(const void* f) {
  for (int i = 0; i < n_limits; ++i)
    if (limits[i].f == f) return i;
  if (n_limits == FUNCS) __builtin_trap();
  limits[n_limits].f = f;
  limits[n_limits].limit = 64 << 10;
  return n_limits++;
}

int hipGetDevice(int* d) { *d = 0; return 0; }
int hipDeviceGetAttribute(int* v, int attr, int dev) { (void)attr; (void)dev; *v = 256; return 0; }
int hipGetLastError(void) { return 0; }
int hipFuncSetAttribute(const void* f, int attr, int value) {
  const int i = limit_of(f);
  if (attr != 8) return 1;                                 /* hipFuncAttributeMaxDynamicSharedMemorySize */
  if (limits[i].limit != (uint64_t)value) ++limits[i].changes;
  limits[i].limit = (uint64_t)value;
  return 0;
}
int __hipPushCallConfiguration(dim3_t grid, dim3_t block, size_t lds, void* stream) {
  config.grid = grid; config.block = block; config.lds = lds; config.stream = stream;
  return 0;
}
int __hipPopCallConfiguration(dim3_t* grid, dim3_t* block, size_t* lds, void** stream) {
  *grid = config.grid; *block = config.block; *lds = config.lds; *stream = config.stream;
  return 0;
}
int hipLaunchKernel(const void* f, dim3_t grid, dim3_t block, void** args, size_t lds, void* stream) {
  (void)args; (void)stream;
  if (n_launches == MOST) __builtin_trap();
  launch_t* l = &launches[n_launches++];
  l->f = f; l->grid = grid.x; l->block = block.x; l->lds = lds; l->limit = limits[limit_of(f)].limit;
  return 0;
}

void recorder_clear(void) { n_launches = 0; }
int recorder_count(void) { return n_launches; }
const char* recorder_get(int i, uint64_t out[4]) {
  Dl_info info;
  out[0] = launches[i].grid; out[1] = launches[i].block; out[2] = launches[i].lds; out[3] = launches[i].limit;
  return dladdr(launches[i].f, &info) && info.dli_sname ? info.dli_sname : "";
}
/* the kernel whose limit changed most often, and how often */
const char* recorder_most_changes(int* changes) {
  Dl_info info;
  int at = -1;
  for (int i = 0; i < n_limits; ++i)
    if (at < 0 || limits[i].changes > limits[at].changes) at = i;
  *changes = at < 0 ? 0 : limits[at].changes;
  return at >= 0 && dladdr(limits[at].f, &info) && info.dli_sname ? info.dli_sname : "";
}
