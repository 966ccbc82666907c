// Few-rows paged attention: bf16 queries, a cache of the same type.
#include "paged_few.h"
namespace kmi {
int few_bf16(const AttendArgs &a, int dim, int row_tiles, int grid, int join_rows, hipStream_t st) {
  return launch_few<Bf16, 16>(a, dim, row_tiles, grid, join_rows, st);
}
}  // namespace kmi
