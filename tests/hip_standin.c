/* Stands in for the calls of the HIP runtime that a launch makes, and notes them: what the
 * library would do is seen without a GPU.  Loaded before the library, for all to find. */
#define _GNU_SOURCE
#include <dlfcn.h>
#include <stdio.h>
#include <string.h>

typedef struct { unsigned x, y, z; } dim3;

static char notes[1 << 20];
static size_t used;
static int refuse, last;
static dim3 grid, block;
static size_t lds;
static void* stream;

static const char* name_of(const void* f) {
  Dl_info i;
  return dladdr(f, &i) && i.dli_sname ? i.dli_sname : "?";
}

int standin_refuse(int error) { return refuse = error, last = 0; }
const char* standin_notes(void) { notes[used] = 0; used = 0; return notes; }

int hipFuncSetAttribute(const void* f, int what, int value) {
  used += (size_t)snprintf(notes + used, sizeof notes - used, "set %s %d %d\n", name_of(f), what, value);
  return refuse ? last = refuse : 0;
}
int hipLaunchKernel(const void* f, dim3 g, dim3 b, void** args, size_t shared, void* s) {
  (void)args, (void)s;
  used += (size_t)snprintf(notes + used, sizeof notes - used, "launch %s %zu %u %u\n", name_of(f),
                           shared, g.x, b.x);
  return 0;
}
int __hipPushCallConfiguration(dim3 g, dim3 b, size_t shared, void* s) {
  grid = g, block = b, lds = shared, stream = s;
  return 0;
}
int __hipPopCallConfiguration(dim3* g, dim3* b, size_t* shared, void** s) {
  *g = grid, *b = block, *shared = lds, *s = stream;
  return 0;
}
int hipGetLastError(void) {
  const int e = last;
  last = 0;
  return e;
}
