// Few-rows paged attention: fp16 queries, e4m3 cache.
#include "paged_few.h"
namespace kmi {
void few_f16_e4m3(const AttendArgs &a, int dim, int row_tiles, dim3 grid, hipStream_t st) { launch_few<F16, true>(a, dim, row_tiles, grid, st); }
}  // namespace kmi
