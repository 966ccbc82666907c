// Few-rows paged attention: fp16 queries, a cache of the same type.
#include "paged_few.h"
namespace kmi {
int few_f16(const AttendArgs &a, int dim, int row_tiles, int grid, int join_rows, hipStream_t st) {
  return launch_few<F16, false>(a, dim, row_tiles, grid, join_rows, st);
}
}  // namespace kmi
