// Few-rows paged attention: bf16 queries, e4m3 cache.
#include "paged_few.h"
namespace kmi {
int few_bf16_e4m3(const AttendArgs &a, int dim, int row_tiles, int grid, int join_rows, hipStream_t st) {
  return launch_few<Bf16, true>(a, dim, row_tiles, grid, join_rows, st);
}
}  // namespace kmi
