// Many-rows paged attention and column sums: bf16 queries, e2m1 cache.
#include "paged_many.h"
namespace kmi {
void many_bf16_e2m1(const AttendArgs &a, int dim, bool sums, dim3 grid, hipStream_t st) {
  if (sums) launch_sums<Bf16, 4>(a, dim, grid, st);
  else launch_many<Bf16, 4>(a, dim, grid, st);
}
}  // namespace kmi
