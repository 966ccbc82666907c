// Many-rows paged attention and column sums: fp16 queries, e2m1 cache.
#include "paged_many.h"
namespace kmi {
void many_f16_e2m1(const AttendArgs &a, int dim, bool sums, dim3 grid, hipStream_t st) {
  if (sums) launch_sums<F16, 4>(a, dim, grid, st);
  else launch_many<F16, 4>(a, dim, grid, st);
}
}  // namespace kmi
