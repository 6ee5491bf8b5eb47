/*
 * Stands in for the HIP runtime's launch on a host without a GPU (preloaded):
 * launches are counted, none runs, and the one that fail_at names (from 0)
 * fails.
 */
#include <stddef.h>
#include <stdint.h>

typedef struct {
  uint32_t x, y, z;
} dim3;

enum { SUCCESS = 0, LAUNCH_FAILURE = 719 };

int launches, fail_at;
static int last_error = SUCCESS;

int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, void *stream) {
  (void)grid, (void)block, (void)lds, (void)stream;
  return SUCCESS;
}

int __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, void **stream) {
  *grid = *block = (dim3){1, 1, 1};
  *lds = 0;
  *stream = NULL;
  return SUCCESS;
}

int hipGetDeviceCount(int *count) {
  *count = 1;
  return SUCCESS;
}

int hipGetLastError(void) {
  const int e = last_error;
  last_error = SUCCESS;
  return e;
}

int hipLaunchKernel(const void *fn, dim3 grid, dim3 block, void **args, size_t lds, void *stream) {
  (void)fn, (void)grid, (void)block, (void)args, (void)lds, (void)stream;
  if (launches++ == fail_at) last_error = LAUNCH_FAILURE;
  return last_error;
}
