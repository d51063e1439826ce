// sdv_paged_shared_i8.cu - the many-row attention over pages of i8 rows, where sequences share prefixes.
#include "sdv_paged_wide.cuh"

namespace sdv {

cudaError_t paged_shared_i8(PaMode mode, const PagedArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, int D, int rows,
                            int grid, cudaStream_t s) {
    if (mode == PA_PREFIX)
        return D == 128 ? wide_launch_c<SD_KV_I8, 128, PA_PREFIX>(a, tmk, tmv, rows, grid, s)
                        : wide_launch_c<SD_KV_I8, 64, PA_PREFIX>(a, tmk, tmv, rows, grid, s);
    return D == 128 ? wide_launch_c<SD_KV_I8, 128, PA_OWN>(a, tmk, tmv, rows, grid, s)
                    : wide_launch_c<SD_KV_I8, 64, PA_OWN>(a, tmk, tmv, rows, grid, s);
}

}  // namespace sdv
