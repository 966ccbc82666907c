// Few-rows paged attention: bf16 queries, e4m3 cache.
#include "paged_few.h"
namespace kmi {
void few_bf16_e4m3(const AttendArgs &a, int dim, int row_tiles, dim3 grid, hipStream_t st) { launch_few<Bf16, true>(a, dim, row_tiles, grid, st); }
}  // namespace kmi
