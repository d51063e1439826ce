// sdv_paged_wide_f16.cu - the many-row attention over pages of f16 rows (one translation unit per type: they compile
// beside each other).
#include "sdv_paged_wide.cuh"

namespace sdv {

cudaError_t paged_wide_f16(const PagedArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, int D, int rows,
                           int grid, cudaStream_t s) {
    return D == 128 ? wide_launch_c<SD_KV_F16, 128, PA_ALL>(a, tmk, tmv, rows, grid, s)
                    : wide_launch_c<SD_KV_F16, 64, PA_ALL>(a, tmk, tmv, rows, grid, s);
}

}  // namespace sdv
