// sdv_paged_wide_bf16.cu - the many-row attention over pages of bf16 rows (one translation unit per type: they compile
// beside each other).
#include "sdv_paged_wide.cuh"

namespace sdv {

cudaError_t paged_wide_bf16(const PagedArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, int D, int rows,
                            int grid, cudaStream_t s) {
    return D == 128 ? wide_launch_c<SD_KV_BF16, 128>(a, tmk, tmv, rows, grid, s)
                    : wide_launch_c<SD_KV_BF16, 64>(a, tmk, tmv, rows, grid, s);
}

}  // namespace sdv
