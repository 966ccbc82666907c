// Few-rows paged attention: fp16 queries, a cache of the same type.
#include "paged_few.h"
namespace kmi {
void few_f16(const AttendArgs &a, int dim, int row_tiles, dim3 grid, hipStream_t st) { launch_few<F16, false>(a, dim, row_tiles, grid, st); }
}  // namespace kmi
