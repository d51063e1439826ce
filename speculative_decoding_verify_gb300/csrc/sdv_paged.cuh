// sdv_paged.cuh - what the calls on a cache in pages share: the checked view of sd_kv_pages, row
// addresses through a sequence's table, and the per-row 8-bit codes.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "sdv_common.cuh"

namespace sdv {

constexpr int PG_MAX_B = 1024;  // sequences per call (their schedule is held in shared memory)
constexpr int PG_MAX_PAGES = 1 << 30;

// The CUDA driver's tensor-map encoder (sdv_attn.cu), looked up once; null if it has none.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

inline int kv_type_bytes(int type) { return type == SD_KV_I8 ? 1 : 2; }

// Whether a description of pages is one that every call takes: the sizes, the row counts that tile
// 64-row stages, 16-byte rows and strides, and pages that do not overlap themselves.
inline sd_status pages_check(const sd_kv_pages *p) {
    if (!p || !p->k || !p->v) return SD_EINVAL;
    if (p->type != SD_KV_F16 && p->type != SD_KV_BF16 && p->type != SD_KV_I8) return SD_EUNSUPPORTED;
    if (p->n_pages < 1 || p->n_pages > PG_MAX_PAGES || p->H_kv < 1 || p->page_rows < 1 || p->D < 1) return SD_EINVAL;
    if (p->D != 64 && p->D != 128 && p->D != 256) return SD_EUNSUPPORTED;
    if (!(p->page_rows == 8 || p->page_rows == 16 || p->page_rows == 32 || p->page_rows % 64 == 0))
        return SD_EUNSUPPORTED;
    const int eb = kv_type_bytes(p->type);
    const int64_t s[3] = {p->page_stride, p->head_stride, p->row_stride};
    for (int i = 0; i < 3; ++i)
        if (s[i] < p->D || (s[i] * eb) % 16 || s[i] > (int64_t(1) << 38)) return SD_EINVAL;
    // rows of all heads together ([page][row][head][D]) or heads apart ([page][head][row][D])
    const bool hnd = p->head_stride >= p->row_stride * p->page_rows && p->page_stride >= p->head_stride * p->H_kv;
    const bool nhd = p->row_stride >= p->head_stride * p->H_kv && p->page_stride >= p->row_stride * p->page_rows;
    if (!hnd && !nhd && p->n_pages > 1) return SD_EINVAL;
    if (!hnd && !nhd && !(p->head_stride >= p->row_stride * p->page_rows || p->row_stride >= p->head_stride * p->H_kv))
        return SD_EINVAL;
    if (!aligned(p->k, 16) || !aligned(p->v, 16)) return SD_EINVAL;
    if (p->type == SD_KV_I8) {
        if (!p->k_scale || !p->v_scale) return SD_EINVAL;
        if (!aligned(p->k_scale, 16) || !aligned(p->v_scale, 16)) return SD_EINVAL;
    }
    return SD_OK;
}

// A sequence's rows of the cache: the row of position pos, head h starts at element
// page * page_stride + h * head_stride + (pos % P) * row_stride, page = table[pos / P].
struct PageView {
    int64_t ps, hs, rs;  // strides in elements
    int32_t n_pages, P, H_kv, D;
};

inline PageView page_view(const sd_kv_pages *p) {
    return {p->page_stride, p->head_stride, p->row_stride, p->n_pages, p->page_rows, p->H_kv, p->D};
}

}  // namespace sdv
