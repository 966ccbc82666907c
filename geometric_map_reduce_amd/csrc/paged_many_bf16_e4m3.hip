// Many-rows paged attention and column sums: bf16 queries, e4m3 cache.
#include "paged_many.h"
namespace kmi {
void many_bf16_e4m3(const AttendArgs &a, int dim, bool sums, dim3 grid, hipStream_t st) {
  if (sums) launch_sums<Bf16, 8>(a, dim, grid, st);
  else launch_many<Bf16, 8>(a, dim, grid, st);
}
}  // namespace kmi
