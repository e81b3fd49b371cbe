/* A CUDA runtime of two devices that runs nothing, for host-side tests: it
 * answers libnk's calls, keeps what each kernel was granted on each device, and
 * refuses the launches that the real one refuses for want of shared memory. */
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#define DEVICES 2
#define KERNELS 4096
enum { OK = 0, INVALID_VALUE = 1, SMEM_DEFAULT = 48 * 1024, ATTR_MAX_DYNAMIC_SMEM = 8 };

static struct {
  const void* f;
  int smem[DEVICES];
} kernels[KERNELS];
static int current, launches, refused;
static char memory[DEVICES][256] __attribute__((aligned(256)));

void fake_reset(int device) { current = device, launches = 0, refused = 0; }
int fake_launches(void) { return launches; }
int fake_refused(void) { return refused; }

static int* granted(const void* f) {
  for (int i = 0; i < KERNELS; ++i) {
    if (!kernels[i].f) kernels[i].f = f;
    if (kernels[i].f == f) return &kernels[i].smem[current];
  }
  return NULL;
}

int cudaGetDevice(int* d) { return *d = current, OK; }
int cudaDeviceGetAttribute(int* v, int attr, int d) { return (void)attr, (void)d, *v = 152, OK; }
int cudaGetSymbolAddress(void** p, const void* s) { return (void)s, *p = memory[current], OK; }
int cudaGetLastError(void) { return OK; }
const char* cudaGetErrorString(int e) { return e ? "invalid argument" : "no error"; }

int cudaFuncSetAttribute(const void* f, int attr, int value) {
  if (attr == ATTR_MAX_DYNAMIC_SMEM) *granted(f) = value;
  return OK;
}

int cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void* f, int threads, size_t smem, unsigned fl) {
  (void)threads, (void)fl;
  *n = smem > SMEM_DEFAULT && (int)smem > *granted(f) ? 0 : (int)(227 * 1024 / (smem + 1024));
  return OK;
}

/* the head of cudaLaunchConfig_t */
struct config {
  unsigned grid[3], block[3];
  size_t smem;
};

int cudaLaunchKernelExC(const struct config* c, const void* f, void** args) {
  (void)args;
  ++launches;
  if (c->smem > SMEM_DEFAULT && (int)c->smem > *granted(f)) return ++refused, INVALID_VALUE;
  return OK;
}

static int encode(void* map) { return memset(map, 0, 128), OK; }

int cudaGetDriverEntryPointByVersion(const char* name, void** p, unsigned version, unsigned long long flags, int* found) {
  (void)name, (void)version, (void)flags;
  return *p = (void*)encode, *found = 0, OK;
}

int cudaMemcpy2DAsync(void) { return INVALID_VALUE; }
int cudaMemcpyAsync(void) { return INVALID_VALUE; }
int cudaMemsetAsync(void) { return INVALID_VALUE; }
int cudaStreamSynchronize(void) { return INVALID_VALUE; }
int __cudaGetKernel(void** k, const void* f) { return *k = (void*)f, OK; }
int __cudaLaunchKernel(void) { return INVALID_VALUE; }
int __cudaPopCallConfiguration(void) { return INVALID_VALUE; }
unsigned __cudaPushCallConfiguration(void) { return INVALID_VALUE; }
void** __cudaRegisterFatBinary(void* b) { return (void**)b; }
void __cudaRegisterFatBinaryEnd(void** h) { (void)h; }
void __cudaUnregisterFatBinary(void** h) { (void)h; }
void __cudaRegisterFunction(void) {}
void __cudaRegisterVar(void) {}
