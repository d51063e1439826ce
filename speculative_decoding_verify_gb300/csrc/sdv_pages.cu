// sdv_pages.cu - a KV cache in pages: writing and committing rows, and taking, sharing, releasing and
// moving pages.
//
// The pool's whole state is a count per page (how many table entries name it); a free page is one whose count is
// 0 and allocation takes the lowest free ones, so every call's outcome is a function of counts and tables
// alone, whatever order the threads run in (counts change by integer atomics, which commute).  Plans (which
// pages to take, copy or move) are made by one CTA in one pass over the counts; the copies they list are made by a
// second launch over the whole GPU, which reads how many there are from the plan, so nothing returns to the host.
#include "sdv_paged.cuh"

namespace sdv {

// ---------------------------------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------------------------------

// 8 fp32 values as 8 codes of a row whose scale is d (0 codes where d is 0, NaN or infinite)
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float d) {
    uint32_t w[2] = {0, 0};
    if (d > 0.0f && d < INFINITY) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            int v = static_cast<int>(roundf(__fdiv_rn(x[i], d)));
            v = v > 127 ? 127 : (v < -127 ? -127 : v);
            w[i >> 2] |= (static_cast<uint32_t>(v) & 255u) << (8 * (i & 3));
        }
    }
    return make_uint2(w[0], w[1]);
}

// One group of D / 8 lanes per (sequence, row, KV head): K and V, 8 elements a lane (two 16-byte loads, one store
// each).  Bound by HBM: 4 bytes read and `elt` written per element; the row's page is looked up once per group.
template <int T, int D>
__global__ void __launch_bounds__(256) paged_append_kernel(PageView pv, void *k, void *v, float *k_scale,
                                                           float *v_scale, const int32_t *table, int32_t width,
                                                           const int32_t *lens, const int32_t *n_new, int32_t B,
                                                           int32_t M, const float *k_new, const float *v_new,
                                                           int64_t sb, int64_t sm, int *status) {
    constexpr int LR = D / 8, RB = 256 / LR;  // lanes per row, rows per block
    pdl_wait();
    pdl_launch_dependents();
    const int l = static_cast<int>(threadIdx.x) % LR;
    const int64_t items = static_cast<int64_t>(B) * M * pv.H_kv;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * RB + threadIdx.x / LR; it < items;
         it += static_cast<int64_t>(gridDim.x) * RB) {
        const int64_t y = it / pv.H_kv;
        const int h = static_cast<int>(it - y * pv.H_kv), b = static_cast<int>(y / M);
        const int i = static_cast<int>(y - static_cast<int64_t>(b) * M);
        const int n = n_new ? n_new[b] : M;
        const int len = lens[b];
        if (n < 0 || n > M || len < 0 || static_cast<int64_t>(len) + n > static_cast<int64_t>(width) * pv.P) {
            set_status(status, SD_EDEVICE);
            continue;
        }
        if (i >= n) continue;
        const int pos = len + i, slot = pos / pv.P;
        const int page = table[static_cast<int64_t>(b) * width + slot];
        if (page < 0 || page >= pv.n_pages) {
            set_status(status, SD_EDEVICE);
            continue;
        }
        const int r = pos - slot * pv.P;
        if (!SD_INB(b < B && i < M && h >= 0 && h < pv.H_kv && slot >= 0 && slot < width && r >= 0 && r < pv.P && 8 * l + 8 <= D,
                    status, 109))  // site 109: appended row
            continue;
        const int64_t src = b * sb + i * sm + static_cast<int64_t>(h) * D + 8 * l;
        const int64_t dst = page * pv.ps + h * pv.hs + r * pv.rs + 8 * l;
        float x[2][8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float4 *s = reinterpret_cast<const float4 *>((e ? v_new : k_new) + src);
            const float4 a = __ldcs(s), c = __ldcs(s + 1);
            x[e][0] = a.x, x[e][1] = a.y, x[e][2] = a.z, x[e][3] = a.w;
            x[e][4] = c.x, x[e][5] = c.y, x[e][6] = c.z, x[e][7] = c.w;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if constexpr (T == SD_KV_I8) {
                // the largest magnitude by its bits, where an infinity is above every number and a NaN above that
                uint32_t a = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(fabsf(x[e][j])));
                const unsigned mask = LR == 32 ? 0xffffffffu : ((1u << (LR & 31)) - 1u) << ((threadIdx.x & 31) / LR * LR);
#pragma unroll
                for (int o = LR / 2; o >= 1; o >>= 1) a = max(a, __shfl_xor_sync(mask, a, o));
                const float d = __fdiv_rn(__uint_as_float(a), 127.0f);
                *reinterpret_cast<uint2 *>(static_cast<int8_t *>(e ? v : k) + dst) = codes8(x[e], d);
                if (l == 0) (e ? v_scale : k_scale)[(static_cast<int64_t>(page) * pv.H_kv + h) * pv.P + r] = d;
            } else {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (T == SD_KV_BF16) {
                        const __nv_bfloat162 p = __floats2bfloat162_rn(x[e][2 * j], x[e][2 * j + 1]);
                        w[j] = *reinterpret_cast<const uint32_t *>(&p);
                    } else {
                        const __half2 p = __floats2half2_rn(x[e][2 * j], x[e][2 * j + 1]);
                        w[j] = *reinterpret_cast<const uint32_t *>(&p);
                    }
                }
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(e ? v : k) + dst) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

// One CTA per sequence, a thread per 16-byte column of a row (K and V of all heads).  path increases and path[t] >= t,
// so moving the rows in the order of t never overwrites a row that is still to be read: no staging.  The row addresses
// are looked up once by the first threads.
__global__ void __launch_bounds__(256) paged_commit_kernel(PageView pv, uint8_t *k, uint8_t *v, float *k_scale,
                                                           float *v_scale, int eb, const int32_t *table, int32_t width,
                                                           int32_t *lens, int32_t M, const int32_t *path,
                                                           const int32_t *count, int *status) {
    __shared__ int32_t from[16], spage[16], srow[16], dpage[16], drow[16];
    pdl_wait();
    pdl_launch_dependents();
    const int b = static_cast<int>(blockIdx.x), t = static_cast<int>(threadIdx.x);
    const int n = count[b], len = lens[b];
    bool bad = n < 0 || n > M || len < 0 || static_cast<int64_t>(len) + (path ? M : n) > static_cast<int64_t>(INT32_MAX) ||
               static_cast<int64_t>(len) + n > static_cast<int64_t>(width) * pv.P;
    if (path && !bad && t < n) {
        const int f = path[static_cast<int64_t>(b) * M + t];
        bad = f < t || f >= M || (t > 0 && f <= path[static_cast<int64_t>(b) * M + t - 1]);
        if (!bad) {
            const int sp = len + f, dp = len + t;
            bad = sp / pv.P >= width || !SD_INB(f < M && t < 16 && t <= f && dp / pv.P < width, status, 110);  // site 110: moved row
            if (!bad) {
                from[t] = f;
                spage[t] = table[static_cast<int64_t>(b) * width + sp / pv.P];
                dpage[t] = table[static_cast<int64_t>(b) * width + dp / pv.P];
                srow[t] = sp % pv.P;
                drow[t] = dp % pv.P;
                bad = f != t && (spage[t] < 0 || spage[t] >= pv.n_pages || dpage[t] < 0 || dpage[t] >= pv.n_pages);
            }
        }
    }
    if (__syncthreads_or(bad)) {
        if (t == 0) set_status(status, SD_EDEVICE);
        return;
    }
    if (path) {
        const int cols = pv.D * eb / 16;
        for (int x = t; x < 2 * pv.H_kv * cols; x += blockDim.x) {
            const int c = x % cols, y = x / cols, h = y % pv.H_kv;
            uint8_t *base = y / pv.H_kv ? v : k;
            const int64_t at = h * pv.hs * eb + 16 * c;
            for (int i0 = 0; i0 < n; i0 += 8) {  // eight loads in flight
                uint4 r[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (i0 + j < n && from[i0 + j] != i0 + j)
                        r[j] =
                            *reinterpret_cast<const uint4 *>(base + (spage[i0 + j] * pv.ps + srow[i0 + j] * pv.rs) * eb + at);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (i0 + j < n && from[i0 + j] != i0 + j)
                        *reinterpret_cast<uint4 *>(base + (dpage[i0 + j] * pv.ps + drow[i0 + j] * pv.rs) * eb + at) = r[j];
            }
        }
        if (k_scale)
            for (int x = t; x < 2 * pv.H_kv; x += blockDim.x) {
                float *s = x / pv.H_kv ? v_scale : k_scale;
                const int64_t h = x % pv.H_kv;
                for (int i = 0; i < n; ++i)
                    if (from[i] != i)
                        s[(static_cast<int64_t>(dpage[i]) * pv.H_kv + h) * pv.P + drow[i]] =
                            s[(static_cast<int64_t>(spage[i]) * pv.H_kv + h) * pv.P + srow[i]];
            }
    }
    if (t == 0) lens[b] = len + n;
}

// ---------------------------------------------------------------------------------------------------
// plans
// ---------------------------------------------------------------------------------------------------

constexpr int PL_T = 1024;    // threads of the planning CTA
constexpr int PL_ROUND = 8 * PL_T;  // pages per round: each warp 256 in order, 8 coalesced loads in flight

// The workspace: a header, two arrays that are zero between calls, and scratch.
struct PagesWs {
    int32_t *n_copies;  // header: copies listed
    int32_t *cnt, *last;  // [n_pages]: writers of a shared page in this call, and 1 + the last one's item
    int32_t *freel;       // [n_pages]: free pages (or holes) in order
    int32_t *movers;      // [n_pages]
    int4 *list;           // [n_pages]: (from, to, rows, 0)
    int32_t *dec;         // [B * width]: what each item of a reservation does
    size_t total;
};
__host__ __device__ inline PagesWs pages_ws(void *base, int64_t n_pages, int64_t items) {
    uint8_t *p = static_cast<uint8_t *>(base);
    PagesWs w;
    size_t at = 256;
    w.n_copies = reinterpret_cast<int32_t *>(p);
    w.list = reinterpret_cast<int4 *>(p + at);
    at += static_cast<size_t>(n_pages) * 16;
    w.cnt = reinterpret_cast<int32_t *>(p + at);
    at += static_cast<size_t>(n_pages) * 4;
    w.last = reinterpret_cast<int32_t *>(p + at);
    at += static_cast<size_t>(n_pages) * 4;
    w.freel = reinterpret_cast<int32_t *>(p + at);
    at += static_cast<size_t>(n_pages) * 4;
    w.movers = reinterpret_cast<int32_t *>(p + at);
    at += static_cast<size_t>(n_pages) * 4;
    w.dec = reinterpret_cast<int32_t *>(p + at);
    at += static_cast<size_t>(items) * 4;
    w.total = at;
    return w;
}

// exclusive sum over the CTA of one number per warp (given by its lane 0's value `x`, equal in all lanes); the total
// in `sum`.  Two barriers; sh has 33 entries.
__device__ __forceinline__ int warps_before(int x, int *sh, int &sum) {
    const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
    __syncthreads();
    if (lane == 0) sh[warp] = x;
    __syncthreads();
    int v = sh[lane];  // PL_T / 32 = 32 warps
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    sum = __shfl_sync(0xffffffffu, inc, 31);
    return __shfl_sync(0xffffffffu, inc - v, warp);
}

// pages p in [lo, hi) with (refs[p] > 0) == live, in order, into out[at ..]; stops once `most` are there.  Returns how
// many.
__device__ int list_pages(const int32_t *refs, int lo, int hi, bool live, int32_t *out, int most, int *sh) {
    const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
    int at = 0;
    for (int r0 = lo; r0 < hi && at < most; r0 += PL_ROUND) {
        uint32_t mask[8];
        int32_t v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int p = r0 + warp * 256 + k * 32 + lane;
            v[k] = p < hi ? refs[p] : (live ? 0 : 1);
        }
        int n = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            mask[k] = __ballot_sync(0xffffffffu, (v[k] > 0) == live);
            n += __popc(mask[k]);
        }
        int sum;
        int o = at + warps_before(n, sh, sum);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if ((mask[k] >> lane) & 1u) {
                const int x = o + __popc(mask[k] & ((1u << lane) - 1u));
                if (x < most) out[x] = r0 + warp * 256 + k * 32 + lane;
            }
            o += __popc(mask[k]);
        }
        at += sum;
    }
    return at;
}

__global__ void __launch_bounds__(PL_T) pages_reserve_kernel(int32_t *refs, int32_t n_pages, int32_t *table,
                                                             int32_t width, int32_t P, const int32_t *lens,
                                                             const int32_t *n_new, int32_t B, int32_t M, int32_t per,
                                                             int32_t *missing, PagesWs ws, int *status) {
    __shared__ int sh[33];
    __shared__ int n_list;
    pdl_wait();
    pdl_launch_dependents();
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
    const int items = B * per;
    if (tid == 0) n_list = 0;
    // the slot and page of an item; -2: nothing to do
    auto look = [&](int it, int &b, int &slot, int &len) {
        b = it / per;
        len = lens[b];
        const int n = n_new ? n_new[b] : M;
        if (n < 0 || n > M || len < 0 || static_cast<int64_t>(len) + n > static_cast<int64_t>(width) * P) {
            set_status(status, SD_EDEVICE);
            return -2;
        }
        slot = len / P + it % per;
        if (n == 0 || static_cast<int64_t>(slot) * P >= len + n) return -2;
        const int pg = table[static_cast<int64_t>(b) * width + slot];
        if (pg >= n_pages) {
            set_status(status, SD_EDEVICE);
            return -2;
        }
        return pg < 0 ? -1 : pg;
    };
    // who writes to pages that others hold too
    for (int it = tid; it < items; it += PL_T) {
        int b, slot, len;
        const int pg = look(it, b, slot, len);
        if (pg >= 0 && refs[pg] > 1) {
            atomicAdd(&ws.cnt[pg], 1);
            atomicMax(&ws.last[pg], it + 1);
        }
    }
    __syncthreads();
    int takes = 0;
    for (int r0 = 0; r0 < items; r0 += PL_T) {
        const int it = r0 + tid;
        int d = 0;
        if (it < items) {
            int b, slot, len;
            const int pg = look(it, b, slot, len);
            if (pg == -1) d = 1;
            else if (pg >= 0 && refs[pg] > 1 && !(__ldcg(&ws.cnt[pg]) == refs[pg] && __ldcg(&ws.last[pg]) == it + 1))
                d = 2;
            ws.dec[it] = d;
        }
        int sum;
        warps_before(__popc(__ballot_sync(0xffffffffu, d != 0)), sh, sum);
        takes += sum;
    }
    __syncthreads();
    for (int it = tid; it < items; it += PL_T) {  // the arrays back to zero
        int b, slot, len;
        const int pg = look(it, b, slot, len);
        if (pg >= 0 && refs[pg] > 1) {
            ws.cnt[pg] = 0;
            ws.last[pg] = 0;
        }
    }
    const int found = takes ? list_pages(refs, 0, n_pages, false, ws.freel, takes, sh) : 0;
    __syncthreads();
    if (found < takes) {
        if (tid == 0) {
            *missing = takes - found;
            *ws.n_copies = 0;
        }
        return;
    }
    int at = 0;
    for (int r0 = 0; r0 < items && takes; r0 += PL_T) {
        const int it = r0 + tid;
        const int d = it < items ? ws.dec[it] : 0;
        const uint32_t mask = __ballot_sync(0xffffffffu, d != 0);
        int sum;
        const int o = at + warps_before(__popc(mask), sh, sum) + __popc(mask & ((1u << lane) - 1u));
        at += sum;
        if (d) {
            const int b = it / per, slot = lens[b] / P + it % per;
            if (!SD_INB(b < B && slot >= 0 && slot < width && o >= 0 && o < found && o < n_pages && ws.freel[o] >= 0 &&
                            ws.freel[o] < n_pages,
                        status, 111))  // site 111: a plan's pages
                continue;
            int32_t *e = table + static_cast<int64_t>(b) * width + slot;
            const int to = ws.freel[o];
            if (d == 2) {
                const int from = *e, rows = min(max(lens[b] - slot * P, 0), P);
                atomicSub(&refs[from], 1);
                if (rows > 0) ws.list[atomicAdd(&n_list, 1)] = make_int4(from, to, rows, 0);
            }
            refs[to] = 1;
            *e = to;
        }
    }
    __syncthreads();
    if (tid == 0) {
        *missing = 0;
        *ws.n_copies = n_list;
    }
}

__global__ void __launch_bounds__(PL_T) pages_compact_kernel(int32_t *refs, int32_t n_pages, int32_t P, int32_t *remap,
                                                             int32_t *n_live, PagesWs ws, int *status) {
    __shared__ int sh[33];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5;
    int live = 0;
    for (int r0 = 0; r0 < n_pages; r0 += PL_ROUND) {
        int n = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int p = r0 + warp * 256 + k * 32 + (tid & 31);
            const int v = p < n_pages ? refs[p] : 0;
            if (p < n_pages) remap[p] = v > 0 ? p : -1;
            n += __popc(__ballot_sync(0xffffffffu, v > 0));
        }
        int sum;
        warps_before(n, sh, sum);
        live += sum;
    }
    const int holes = list_pages(refs, 0, live, false, ws.freel, n_pages, sh);
    list_pages(refs, live, n_pages, true, ws.movers, n_pages, sh);
    __syncthreads();
    for (int i = tid; i < holes; i += PL_T) {  // as many movers as holes: live pages = live
        const int from = ws.movers[i], to = ws.freel[i];
        if (!SD_INB(i < n_pages && from >= live && from < n_pages && to >= 0 && to < live, status, 111)) continue;
        ws.list[i] = make_int4(from, to, P, 0);
        remap[from] = to;
        refs[to] = refs[from];
        refs[from] = 0;
    }
    if (tid == 0) {
        *n_live = live;
        *ws.n_copies = holes;
    }
}

// ---------------------------------------------------------------------------------------------------
// copies
// ---------------------------------------------------------------------------------------------------

// The listed rows of K and V, in parts of CP_T * CP_U * 16 bytes so that one large page spreads over CTAs; 16 bytes a
// thread, four loads in flight.  Rows of one head are taken in a row where heads lie apart, heads of one row
// where they lie together.  With a table, its entries follow remap.  HBM-bound: every byte read and written once.
constexpr int CP_T = 256, CP_U = 4;

__global__ void __launch_bounds__(CP_T) pages_copy_kernel(PageView pv, uint8_t *k, uint8_t *v, float *k_scale,
                                                          float *v_scale, int eb, const int32_t *n_copies,
                                                          const int4 *list, int32_t *table, int64_t entries,
                                                          const int32_t *remap, int *status) {
    pdl_wait();
    pdl_launch_dependents();
    if (table)
        for (int64_t x = static_cast<int64_t>(blockIdx.x) * CP_T + threadIdx.x; x < entries;
             x += static_cast<int64_t>(gridDim.x) * CP_T) {
            const int t = table[x];
            if (t >= 0 && t < pv.n_pages) table[x] = remap[t];
        }
    const int n = min(*n_copies, pv.n_pages);  // a plan lists a page at most once as a target
    const int cols = pv.D * eb / 16;  // a power of two
    const int cs = __ffs(cols) - 1;
    const int parts = static_cast<int>((static_cast<int64_t>(pv.P) * pv.H_kv * cols + CP_T * CP_U - 1) / (CP_T * CP_U));
    const bool together = pv.hs < pv.rs;
    for (int64_t w = blockIdx.x; w < static_cast<int64_t>(n) * 2 * parts; w += gridDim.x) {
        const int64_t y = w / parts;
        const int part = static_cast<int>(w - y * parts);
        const int4 e = list[y >> 1];
        // a plan for another pool's sizes
        if (e.x < 0 || e.x >= pv.n_pages || e.y < 0 || e.y >= pv.n_pages || e.z > pv.P) {
            set_status(status, SD_EDEVICE);
            continue;
        }
        const int total = e.z * pv.H_kv * cols;
        if (part * (CP_T * CP_U) >= total) continue;
        uint8_t *base = (y & 1) ? v : k;
        const uint8_t *src = base + e.x * pv.ps * eb;
        uint8_t *dst = base + e.y * pv.ps * eb;
        uint4 r[CP_U];
        int64_t off[CP_U];
#pragma unroll
        for (int u = 0; u < CP_U; ++u) {
            const int x = part * (CP_T * CP_U) + u * CP_T + static_cast<int>(threadIdx.x);
            off[u] = -1;
            if (x < total) {
                const int c = x & (cols - 1), z = x >> cs;
                const int div = together ? pv.H_kv : e.z;
                const int hi = z / div, low = z - hi * div;
                const int h = together ? low : hi, row = together ? hi : low;
                if (!SD_INB(h >= 0 && h < pv.H_kv && row >= 0 && row < e.z && c < cols, status, 112)) continue;  // site 112: copy
                off[u] = (h * pv.hs + row * pv.rs) * eb + 16 * c;
                r[u] = __ldcs(reinterpret_cast<const uint4 *>(src + off[u]));
            }
        }
#pragma unroll
        for (int u = 0; u < CP_U; ++u)
            if (off[u] >= 0) __stcs(reinterpret_cast<uint4 *>(dst + off[u]), r[u]);
        if (k_scale && part == 0) {
            float *s = (y & 1) ? v_scale : k_scale;
            const int64_t page = static_cast<int64_t>(pv.H_kv) * pv.P;
            for (int x = threadIdx.x; x < e.z * pv.H_kv; x += CP_T) {
                const int64_t at = static_cast<int64_t>(x / e.z) * pv.P + x % e.z;
                s[e.y * page + at] = s[e.x * page + at];
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------------
// tables and counts
// ---------------------------------------------------------------------------------------------------

// whether a sequence's length is one that its table can hold
__device__ __forceinline__ bool len_ok(int len, int32_t width, int32_t P) {
    return len >= 0 && len <= static_cast<int64_t>(width) * P;
}

// one holder fewer; a count that was not there is put back and recorded
__device__ __forceinline__ void drop_page(int32_t *refs, int32_t n_pages, int pg, int *status) {
    if (pg < 0) return;
    if (pg >= n_pages) {
        set_status(status, SD_EDEVICE);
        return;
    }
    if (atomicSub(&refs[pg], 1) <= 0) {
        atomicAdd(&refs[pg], 1);
        set_status(status, SD_EDEVICE);
    }
}

// one CTA per pair
__global__ void __launch_bounds__(256) pages_fork_kernel(int32_t *refs, int32_t n_pages, int32_t *table, int32_t width,
                                                         int32_t *lens, int32_t B, int32_t P, const int32_t *src,
                                                         const int32_t *dst, int32_t n, int *status) {
    pdl_wait();
    pdl_launch_dependents();
    const int i = static_cast<int>(blockIdx.x), s = src[i], d = dst[i];
    bool bad = s < 0 || s >= B || d < 0 || d >= B || !len_ok(lens[s], width, P);
    for (int j = threadIdx.x; j < n; j += blockDim.x) bad |= src[j] == d || (j != i && dst[j] == d);
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) set_status(status, SD_EDEVICE);
        return;
    }
    const int len = lens[s];
    int32_t *to = table + static_cast<int64_t>(d) * width;
    const int32_t *from = table + static_cast<int64_t>(s) * width;
    for (int x = threadIdx.x; x < width; x += blockDim.x) {
        int pg = static_cast<int64_t>(x) * P < len ? from[x] : -1;
        if (pg >= n_pages) {
            set_status(status, SD_EDEVICE);
            pg = -1;
        }
        drop_page(refs, n_pages, to[x], status);
        to[x] = pg < 0 ? -1 : pg;
        if (pg >= 0) atomicAdd(&refs[pg], 1);
    }
    if (threadIdx.x == 0) lens[d] = len;
}

// one CTA per named sequence; entries are exchanged, so that a sequence named twice releases its pages once
__global__ void __launch_bounds__(256) pages_free_kernel(int32_t *refs, int32_t n_pages, int32_t *table, int32_t width,
                                                         int32_t *lens, int32_t B, int32_t P, const int32_t *seqs,
                                                         const int32_t *keep, int *status) {
    pdl_wait();
    pdl_launch_dependents();
    const int b = seqs[blockIdx.x], rows = keep ? keep[blockIdx.x] : 0;
    if (b < 0 || b >= B || rows < 0 || !len_ok(lens[b], width, P)) {
        if (threadIdx.x == 0) set_status(status, SD_EDEVICE);
        return;
    }
    int32_t *t = table + static_cast<int64_t>(b) * width;
    for (int64_t x = (static_cast<int64_t>(rows) + P - 1) / P + threadIdx.x; x < width; x += blockDim.x)
        if (t[x] != -1) drop_page(refs, n_pages, atomicExch(&t[x], -1), status);
    if (threadIdx.x == 0) atomicMin(&lens[b], rows);
}

// one CTA per sequence
__global__ void __launch_bounds__(256) pages_trim_kernel(int32_t *refs, int32_t n_pages, int32_t *table, int32_t width,
                                                         const int32_t *lens, int32_t P, int32_t window, int32_t sinks,
                                                         int *status) {
    pdl_wait();
    pdl_launch_dependents();
    const int b = static_cast<int>(blockIdx.x);
    if (!len_ok(lens[b], width, P)) {
        if (threadIdx.x == 0) set_status(status, SD_EDEVICE);
        return;
    }
    const int lo = lens[b] - window + 1;  // the first row that a later row sees
    int32_t *t = table + static_cast<int64_t>(b) * width;
    const int end = lo > 0 ? min(lo / P, width) : 0;
    for (int64_t x = (static_cast<int64_t>(sinks) + P - 1) / P + threadIdx.x; x < end; x += blockDim.x) {
        const int pg = t[x];
        if (pg == -1) continue;
        t[x] = -1;
        drop_page(refs, n_pages, pg, status);
    }
}

template <int T>
static cudaError_t append_launch(const sd_kv_pages *p, const int32_t *table, int32_t width, const int32_t *lens,
                                 const int32_t *n_new, int32_t B, int32_t M, const float *kn, const float *vn,
                                 int64_t sb, int64_t sm, int *status, cudaStream_t s) {
    const int rb = 256 / (p->D / 8);
    const int64_t blocks = (static_cast<int64_t>(B) * M * p->H_kv + rb - 1) / rb;
    const int64_t cap = static_cast<int64_t>(num_sms()) * 32;
    const dim3 grid(static_cast<unsigned>(blocks < cap ? blocks : cap));
    const PageView pv = page_view(p);
    float *ks = T == SD_KV_I8 ? p->k_scale : nullptr, *vs = T == SD_KV_I8 ? p->v_scale : nullptr;
    if (p->D == 64)
        return launch(paged_append_kernel<T, 64>, grid, dim3(256), 0, s, pv,
                      p->k, p->v, ks, vs, table, width, lens, n_new, B, M, kn, vn, sb, sm, status);
    if (p->D == 128)
        return launch(paged_append_kernel<T, 128>, grid, dim3(256), 0, s, pv,
                      p->k, p->v, ks, vs, table, width, lens, n_new, B, M, kn, vn, sb, sm, status);
    return launch(paged_append_kernel<T, 256>, grid, dim3(256), 0, s, pv,
                  p->k, p->v, ks, vs, table, width, lens, n_new, B, M, kn, vn, sb, sm, status);
}

static cudaError_t copy_launch(const sd_kv_pages *p, const PagesWs &ws, int32_t *table, int64_t entries,
                               const int32_t *remap, cudaStream_t s) {
    int *status = status_ptr();
    if (!status) return cudaErrorUnknown;
    const bool i8 = p->type == SD_KV_I8;
    return launch(pages_copy_kernel, dim3(static_cast<unsigned>(num_sms()) * 16), dim3(CP_T), 0, s, page_view(p),
                  static_cast<uint8_t *>(p->k),
                  static_cast<uint8_t *>(p->v), i8 ? p->k_scale : nullptr, i8 ? p->v_scale : nullptr, kv_type_bytes(p->type),
                  static_cast<const int32_t *>(ws.n_copies), static_cast<const int4 *>(ws.list), table, entries, remap, status);
}

static bool table_ok(const void *refs, int32_t n_pages, const void *table, int32_t width, int32_t B, int32_t P) {
    return refs && table && n_pages >= 1 && n_pages <= PG_MAX_PAGES && width >= 1 && B >= 1 && P >= 1 &&
           static_cast<int64_t>(width) * P <= INT32_MAX - 128;
}

}  // namespace sdv

using namespace sdv;

extern "C" {

sd_status sd_paged_append(const sd_kv_pages *pages, const int32_t *table, int32_t width, const int32_t *lens,
                          const int32_t *n_new, int32_t B, int32_t M, const float *k_new, const float *v_new,
                          int64_t seq_stride, int64_t row_stride, sd_stream_t stream) {
    SD_NVTX("sd_paged_append");
    const sd_status st = pages_check(pages);
    if (st != SD_OK) return st;
    if (!table || !lens || !k_new || !v_new || width < 1 || B < 1 || M < 1) return SD_EINVAL;
    if (B > PG_MAX_B) return SD_EUNSUPPORTED;
    const int64_t line = static_cast<int64_t>(pages->H_kv) * pages->D;
    if ((M > 1 && row_stride < line) || (B > 1 && seq_stride < line) || row_stride % 4 || seq_stride % 4)
        return SD_EINVAL;
    if (!aligned(k_new, 16) || !aligned(v_new, 16)) return SD_EINVAL;
    if (static_cast<int64_t>(width) * pages->page_rows > INT32_MAX - 128) return SD_EUNSUPPORTED;
    int *status = status_ptr();
    if (!status) return SD_ECUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e =
        pages->type == SD_KV_F16    ? append_launch<SD_KV_F16>(pages, table, width, lens, n_new, B, M, k_new, v_new,
                                                               seq_stride, row_stride, status, s)
        : pages->type == SD_KV_BF16 ? append_launch<SD_KV_BF16>(pages, table, width, lens, n_new, B, M, k_new, v_new,
                                                                seq_stride, row_stride, status, s)
                                    : append_launch<SD_KV_I8>(pages, table, width, lens, n_new, B, M, k_new, v_new,
                                                              seq_stride, row_stride, status, s);
    return e == cudaSuccess ? SD_OK : SD_ECUDA;
}

sd_status sd_paged_commit(const sd_kv_pages *pages, const int32_t *table, int32_t width, int32_t *lens, int32_t B,
                          int32_t M, const int32_t *path, const int32_t *count, sd_stream_t stream) {
    SD_NVTX("sd_paged_commit");
    const sd_status st = pages_check(pages);
    if (st != SD_OK) return st;
    if (!table || !lens || !count || width < 1 || B < 1 || M < 1) return SD_EINVAL;
    if (B > PG_MAX_B || (path && M > 16)) return SD_EUNSUPPORTED;
    if (static_cast<int64_t>(width) * pages->page_rows > INT32_MAX - 128) return SD_EUNSUPPORTED;
    int *status = status_ptr();
    if (!status) return SD_ECUDA;
    const bool i8 = pages->type == SD_KV_I8;
    const cudaError_t e = launch(paged_commit_kernel, dim3(B), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream),
                                 page_view(pages),
                                 static_cast<uint8_t *>(pages->k), static_cast<uint8_t *>(pages->v),
                                 i8 ? pages->k_scale : nullptr, i8 ? pages->v_scale : nullptr,
                                 kv_type_bytes(pages->type), table, width, lens, M, path, count, status);
    return e == cudaSuccess ? SD_OK : SD_ECUDA;
}

size_t sd_pages_workspace_bytes(int32_t n_pages, int32_t B, int32_t width) {
    if (n_pages < 1 || B < 1 || width < 1) return 0;
    return pages_ws(nullptr, n_pages, static_cast<int64_t>(B) * width).total;
}

sd_status sd_pages_reserve(const sd_kv_pages *pages, int32_t *refs, int32_t *table, int32_t width, const int32_t *lens,
                           const int32_t *n_new, int32_t B, int32_t M, int32_t *missing, void *workspace, size_t ws_bytes,
                           sd_stream_t stream) {
    SD_NVTX("sd_pages_reserve");
    const sd_status st = pages_check(pages);
    if (st != SD_OK) return st;
    const int P = pages->page_rows;
    if (!table_ok(refs, pages->n_pages, table, width, B, P) || !lens || !missing || !workspace || M < 1)
        return SD_EINVAL;
    if (!aligned(workspace, 256) || ws_bytes < sd_pages_workspace_bytes(pages->n_pages, B, width)) return SD_EINVAL;
    // slots that M rows can touch; items are counted in 32 bits
    const int64_t most = (static_cast<int64_t>(M) + P - 2) / P + 1, per = most < width ? most : width;
    if (B > PG_MAX_B || per * B > INT32_MAX / 2) return SD_EUNSUPPORTED;
    int *status = status_ptr();
    if (!status) return SD_ECUDA;
    const PagesWs ws = pages_ws(workspace, pages->n_pages, static_cast<int64_t>(B) * width);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch(pages_reserve_kernel, dim3(1), dim3(PL_T), 0, s, refs,
                           pages->n_pages, table, width, P, lens, n_new, B, M, static_cast<int32_t>(per), missing,
                           ws, status);
    if (e == cudaSuccess) e = copy_launch(pages, ws, nullptr, 0, nullptr, s);
    return e == cudaSuccess ? SD_OK : SD_ECUDA;
}

sd_status sd_pages_copy(const sd_kv_pages *pages, const void *workspace, size_t ws_bytes, sd_stream_t stream) {
    SD_NVTX("sd_pages_copy");
    const sd_status st = pages_check(pages);
    if (st != SD_OK) return st;
    if (!workspace || !aligned(workspace, 256) || ws_bytes < sd_pages_workspace_bytes(pages->n_pages, 1, 1))
        return SD_EINVAL;
    const PagesWs ws = pages_ws(const_cast<void *>(workspace), pages->n_pages, 1);
    return copy_launch(pages, ws, nullptr, 0, nullptr,
                       reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? SD_OK : SD_ECUDA;
}

sd_status sd_pages_fork(int32_t *refs, int32_t n_pages, int32_t *table, int32_t width, int32_t *lens, int32_t B,
                        int32_t page_rows, const int32_t *src, const int32_t *dst, int32_t n, sd_stream_t stream) {
    SD_NVTX("sd_pages_fork");
    if (!table_ok(refs, n_pages, table, width, B, page_rows) || !lens || n < 0 || (n > 0 && (!src || !dst)))
        return SD_EINVAL;
    if (n == 0) return SD_OK;
    if (n > B) return SD_EINVAL;  // some dst would be named twice
    int *status = status_ptr();
    if (!status) return SD_ECUDA;
    return launch(pages_fork_kernel, dim3(n), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), refs, n_pages,
                  table, width, lens, B, page_rows, src, dst, n, status) == cudaSuccess
               ? SD_OK
               : SD_ECUDA;
}

sd_status sd_pages_free(int32_t *refs, int32_t n_pages, int32_t *table, int32_t width, int32_t *lens, int32_t B,
                        int32_t page_rows, const int32_t *seqs, const int32_t *keep, int32_t n, sd_stream_t stream) {
    SD_NVTX("sd_pages_free");
    if (!table_ok(refs, n_pages, table, width, B, page_rows) || !lens || n < 0 || (n > 0 && !seqs)) return SD_EINVAL;
    if (n == 0) return SD_OK;
    int *status = status_ptr();
    if (!status) return SD_ECUDA;
    return launch(pages_free_kernel, dim3(n), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), refs, n_pages,
                  table, width, lens, B, page_rows, seqs, keep, status) == cudaSuccess
               ? SD_OK
               : SD_ECUDA;
}

sd_status sd_pages_trim(int32_t *refs, int32_t n_pages, int32_t *table, int32_t width, const int32_t *lens, int32_t B,
                        int32_t page_rows, int32_t window, int32_t sinks, sd_stream_t stream) {
    SD_NVTX("sd_pages_trim");
    if (!table_ok(refs, n_pages, table, width, B, page_rows) || !lens || window < 1 || sinks < 0) return SD_EINVAL;
    int *status = status_ptr();
    if (!status) return SD_ECUDA;
    return launch(pages_trim_kernel, dim3(B), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), refs, n_pages,
                  table, width, lens, page_rows, window, sinks, status) == cudaSuccess
               ? SD_OK
               : SD_ECUDA;
}

sd_status sd_pages_compact(const sd_kv_pages *pages, int32_t *refs, int32_t *table, int32_t width, int32_t B,
                           int32_t *remap, int32_t *n_live, void *workspace, size_t ws_bytes, sd_stream_t stream) {
    SD_NVTX("sd_pages_compact");
    const sd_status st = pages_check(pages);
    if (st != SD_OK) return st;
    if (!table_ok(refs, pages->n_pages, table, width, B, pages->page_rows) || !remap || !n_live || !workspace)
        return SD_EINVAL;
    if (!aligned(workspace, 256) || ws_bytes < sd_pages_workspace_bytes(pages->n_pages, B, width)) return SD_EINVAL;
    int *status = status_ptr();
    if (!status) return SD_ECUDA;
    const PagesWs ws = pages_ws(workspace, pages->n_pages, static_cast<int64_t>(B) * width);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch(pages_compact_kernel, dim3(1), dim3(PL_T), 0, s, refs,
                           pages->n_pages, pages->page_rows, remap, n_live, ws, status);
    if (e == cudaSuccess) e = copy_launch(pages, ws, table, static_cast<int64_t>(B) * width, remap, s);
    return e == cudaSuccess ? SD_OK : SD_ECUDA;
}

}  // extern "C"
