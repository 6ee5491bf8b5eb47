/*
 * Stands in for the HIP runtime's launch on a host without a GPU (preloaded):
 * every launch is recorded, none runs, and one that breaks HIP's limit on a
 * grid's work-items (fewer than 2^32 in each dimension) fails as it would on
 * a device.
 */
#include <stddef.h>
#include <stdint.h>

typedef struct {
  uint32_t x, y, z;
} dim3;

enum { SUCCESS = 0, INVALID_CONFIGURATION = 9 };

static int last_error = SUCCESS;
static uint64_t launches, items_largest;

static dim3 pushed_grid, pushed_block;
static size_t pushed_lds;
static void *pushed_stream;

int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, void *stream) {
  pushed_grid = grid;
  pushed_block = block;
  pushed_lds = lds;
  pushed_stream = stream;
  return SUCCESS;
}

int __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, void **stream) {
  *grid = pushed_grid;
  *block = pushed_block;
  *lds = pushed_lds;
  *stream = pushed_stream;
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
  (void)fn, (void)args, (void)lds, (void)stream;
  const uint64_t items = (uint64_t)grid.x * block.x;
  ++launches;
  if (items > items_largest) items_largest = items;
  const int bad = grid.x == 0 || block.x == 0 || block.x > 1024 || items > 0xffffffffu || grid.y != 1 || grid.z != 1 ||
                  block.y != 1 || block.z != 1;
  if (bad) last_error = INVALID_CONFIGURATION;
  return last_error;
}

uint64_t recorded_launches(void) { return launches; }
uint64_t recorded_largest(void) { return items_largest; }
void recorded_clear(void) { launches = items_largest = 0; }
