// sdv_paged_wide_i8.cu - the many-row attention over pages of i8 rows (one translation unit per type: they compile
// beside each other).
#include "sdv_paged_wide.cuh"

namespace sdv {

cudaError_t paged_wide_i8(const PagedArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, int D, int rows, int grid,
                          cudaStream_t s) {
    return D == 128 ? wide_launch_c<SD_KV_I8, 128>(a, tmk, tmv, rows, grid, s)
                    : wide_launch_c<SD_KV_I8, 64>(a, tmk, tmv, rows, grid, s);
}

}  // namespace sdv
