/* The part of the CUDA runtime that the cache and attention calls use on the host, without a GPU: preloaded before the real
 * one, it notes kernel launches and attribute settings by device, so that the host's choices can be tested on any machine.
 * Nothing is executed. */
#include <stddef.h>
#include <stdio.h>
#include <string.h>

typedef struct { unsigned x, y, z; } dim3;
typedef struct { dim3 grid, block; size_t smem; void* stream; void* attrs; unsigned n_attrs; } launch_config;

enum { kOk = 0, kInvalid = 1, kMaxKernels = 512, kMaxNotes = 256, kAttrSms = 16 };

static struct { const void* host; const char* name; } kernels[kMaxKernels];
static int n_kernels, device, fail_attributes, fail_entry_points, last_error;
static int sms[8] = {152, 100, 90, 80, 70, 60, 50, 40};
static char notes[kMaxNotes][400];
static int n_notes;

static const char* name_of(const void* host) {
  for (int i = 0; i < n_kernels; ++i)
    if (kernels[i].host == host) return kernels[i].name;
  return "?";
}

/* ---- what the tests set and read */
void fake_set_device(int d) { device = d; }
void fake_fail_attributes(int n) { fail_attributes = n; }
void fake_fail_entry_points(int n) { fail_entry_points = n; }
int fake_notes(void) { return n_notes; }
const char* fake_note(int i) { return i < n_notes ? notes[i] : ""; }
void fake_clear(void) { n_notes = 0; }

/* ---- registration and launches of kernels */
void** __cudaRegisterFatBinary(void* image) { static void* handle; (void)image; return &handle; }
void __cudaRegisterFatBinaryEnd(void** handle) { (void)handle; }
void __cudaUnregisterFatBinary(void** handle) { (void)handle; }
void __cudaRegisterVar(void** handle, char* host, char* dev, const char* name, int ext, size_t size, int constant, int global) {
  (void)handle, (void)host, (void)dev, (void)name, (void)ext, (void)size, (void)constant, (void)global;
}
void __cudaRegisterFunction(void** handle, const char* host, char* dev, const char* name, int limit, void* tid, void* bid,
                            void* bdim, void* gdim, int* wsize) {
  (void)handle, (void)dev, (void)limit, (void)tid, (void)bid, (void)bdim, (void)gdim, (void)wsize;
  if (n_kernels < kMaxKernels) kernels[n_kernels].host = host, kernels[n_kernels++].name = name;
}

static struct { dim3 grid, block; size_t smem; void* stream; } pushed;
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, void* stream) {
  pushed.grid = grid, pushed.block = block, pushed.smem = smem, pushed.stream = stream;
  return 0;
}
int __cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* smem, void* stream) {
  *grid = pushed.grid, *block = pushed.block, *smem = pushed.smem, *(void**)stream = pushed.stream;
  return kOk;
}
int __cudaGetKernel(const void** kernel, const void* host) { *kernel = host; return kOk; }

static int note_launch(const void* host, dim3 grid, dim3 block, size_t smem) {
  if (grid.x == 0 || block.x == 0) return last_error = kInvalid;
  if (n_notes < kMaxNotes)
    snprintf(notes[n_notes++], sizeof(notes[0]), "launch %d %u %u %zu %s", device, grid.x, block.x, smem, name_of(host));
  return kOk;
}
int __cudaLaunchKernel(const void* kernel, dim3 grid, dim3 block, void** args, size_t smem, void* stream) {
  (void)args, (void)stream;
  return note_launch(kernel, grid, block, smem);
}
int cudaLaunchKernelExC(const launch_config* cfg, const void* host, void** args) {
  (void)args;
  return note_launch(host, cfg->grid, cfg->block, cfg->smem);
}

/* ---- devices and errors */
int cudaGetDevice(int* d) { *d = device; return kOk; }
int cudaDeviceGetAttribute(int* value, int attr, int d) {
  *value = attr == kAttrSms ? sms[d & 7] : 0;
  return kOk;
}
int cudaFuncSetAttribute(const void* host, int attr, int value) {
  if (fail_attributes > 0) return --fail_attributes, last_error = kInvalid;
  if (n_notes < kMaxNotes)
    snprintf(notes[n_notes++], sizeof(notes[0]), "attribute %d %d %d %s", device, attr, value, name_of(host));
  return kOk;
}
int cudaGetLastError(void) { int e = last_error; last_error = kOk; return e; }

static int encode_tiled(void) { return 0; }
int cudaGetDriverEntryPointByVersion(const char* symbol, void** fn, unsigned version, unsigned long long flags, int* result) {
  (void)symbol, (void)version, (void)flags;
  if (fail_entry_points > 0) { --fail_entry_points; *fn = NULL; if (result) *result = 1; return kOk; }
  *fn = (void*)encode_tiled;
  if (result) *result = 0;
  return kOk;
}
