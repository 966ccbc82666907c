// Few-rows paged attention: bf16 queries, a cache of the same type.
#include "paged_few.h"
namespace kmi {
void few_bf16(const AttendArgs &a, int dim, int row_tiles, dim3 grid, hipStream_t st) { launch_few<Bf16, false>(a, dim, row_tiles, grid, st); }
}  // namespace kmi
