// sdv_paged_shared_f16.cu - the many-row attention over pages of f16 rows, where sequences share prefixes.
#include "sdv_paged_wide.cuh"

namespace sdv {

cudaError_t paged_shared_f16(PaMode mode, const PagedArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, int D, int rows,
                             int grid, cudaStream_t s) {
    if (mode == PA_PREFIX)
        return D == 128 ? wide_launch_c<SD_KV_F16, 128, PA_PREFIX>(a, tmk, tmv, rows, grid, s)
                        : wide_launch_c<SD_KV_F16, 64, PA_PREFIX>(a, tmk, tmv, rows, grid, s);
    return D == 128 ? wide_launch_c<SD_KV_F16, 128, PA_OWN>(a, tmk, tmv, rows, grid, s)
                    : wide_launch_c<SD_KV_F16, 64, PA_OWN>(a, tmk, tmv, rows, grid, s);
}

}  // namespace sdv
