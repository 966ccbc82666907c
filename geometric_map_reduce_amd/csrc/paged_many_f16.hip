// Many-rows paged attention and column sums: fp16 queries, a cache of the same type.
#include "paged_many.h"
namespace kmi {
void many_f16(const AttendArgs &a, int dim, bool sums, dim3 grid, hipStream_t st) {
  if (sums) launch_sums<F16, 16>(a, dim, grid, st);
  else launch_many<F16, 16>(a, dim, grid, st);
}
}  // namespace kmi
