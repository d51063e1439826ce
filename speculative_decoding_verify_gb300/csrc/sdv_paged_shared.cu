// sdv_paged_shared.cu - attention of a batch whose sequences share prefixes of pages, each prefix computed once for all.
//
// The softmax over a sequence's rows is split behind its group's shared rows: with (m, l, o) the maximum, the sum and
// the normalised output of either part,
//   out = (2^(m_p - m) l_p o_p + 2^(m_o - m) l_o o_o) / (2^(m_p - m) l_p + 2^(m_o - m) l_o),  m = max(m_p, m_o).
// Three launches on the stream:
//   the plan: what the tables say is shared, whether that is worth it, and the lists of the groups' query rows;
//   the prefixes: the many-row kernel with all new rows of a group as the rows of one "sequence" (128 of them share each
//   64-row tile of keys), into the workspace;
//   each sequence's rows behind its prefix, as sd_paged_attn computes them, joined where an output row is finished.  It starts
//   beside the prefixes, as their CTAs leave the SMs, and waits for them only where it reads what they came to.
// So a prefix is read from HBM once per group (per 128 query rows from L2), where sd_paged_attn reads it once per sequence.
#include "sdv_paged_attn.cuh"

namespace sdv {

constexpr int SP_THREADS = 256;
// Tiles of keys (per KV head and member) that have to be left out for the prefixes' launch to pay: it costs about as long as
// 3000 of them.  (A test may set another number.)
static int64_t g_worth = 3000;

// The plan, in the workspace.
struct SharedPlan {
    int32_t *head;  // CTAs that are done (0 between calls)
    int32_t *ref, *common;                       // [B]: a sequence's group as its lowest member (-1: none), slots that it shares with it
    int32_t *skip, *start;                       // [B] tiles of the prefix, and where its rows are in rows_of
    int32_t *first, *rows, *len, *leader;        // [B / 2]: the groups
    int32_t *rows_of;                            // [B * M]
};
struct SharedWs {
    SharedPlan p;
    uint8_t *attn;  // the workspace of the launch for the sequences; the prefixes' has counters and partials of its own
    int32_t *counters;
    uint8_t *partials;
    float2 *prefix_ml;
    float *prefix_o;
    size_t total;
};
static SharedWs shared_ws(void *base, int B, int M, int H, int D) {
    uint8_t *p = static_cast<uint8_t *>(base);
    SharedWs w;
    // what has to be zero between calls comes first, at places that no size moves
    size_t at = 256;
    auto take = [&](size_t n) {
        uint8_t *x = p + at;
        at += (n + 255) / 256 * 256;
        return x;
    };
    auto ints = [&](size_t n) { return reinterpret_cast<int32_t *>(take(4 * n)); };
    w.p.head = reinterpret_cast<int32_t *>(p);
    w.counters = reinterpret_cast<int32_t *>(take(pa_counters()));
    w.attn = take(pa_workspace(D, nullptr, nullptr));
    w.partials = take(pa_workspace(D, nullptr, nullptr));
    w.p.ref = ints(B);
    w.p.common = ints(B);
    w.p.skip = ints(B);
    w.p.start = ints(B);
    w.p.first = ints(B);
    w.p.rows = ints(B);
    w.p.len = ints(B);
    w.p.leader = ints(B);
    const size_t rows = static_cast<size_t>(B) * M;
    w.p.rows_of = ints(rows);
    w.prefix_ml = reinterpret_cast<float2 *>(take(rows * H * 8));
    w.prefix_o = reinterpret_cast<float *>(take(rows * H * D * 4));
    w.total = at;
    return w;
}

// One CTA per sequence compares its table with that of its group's lowest member; the last one to finish makes the lists.
__global__ void __launch_bounds__(SP_THREADS) shared_plan_kernel(SharedPlan pl, const int32_t *table, int32_t width,
                                                                 const int32_t *lens, const int32_t *n_new,
                                                                 const int32_t *group, int32_t B, int32_t M, int32_t P,
                                                                 int32_t H_kv, int32_t n_pages, int64_t worth_it, int *status) {
    __shared__ int32_t s_ref[PG_MAX_B], s_n[PG_MAX_B], s_min[PG_MAX_B];
    __shared__ uint32_t s_at[PG_MAX_B], s_warp[SP_THREADS / 32];
    __shared__ int32_t s_low, s_last;
    pdl_wait();
    pdl_launch_dependents();
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5, b = static_cast<int>(blockIdx.x);
    auto news = [&](int j) {  // its new rows; 0 where the sequence takes no part
        const int n = n_new ? n_new[j] : M, len = lens[j];
        return n < 0 || n > M || len < 0 || static_cast<int64_t>(len) + n > static_cast<int64_t>(width) * P ? 0 : n;
    };
    const int grp = group[b], mine = news(b);
    if (tid == 0) {
        s_low = INT32_MAX;
        if (grp < -1 || grp >= B) set_status(status, SD_EDEVICE);
    }
    __syncthreads();
    int ref = mine > 0 ? b : -1;
    if (mine > 0 && grp >= 0 && grp < B) {
        for (int j = tid; j < b; j += SP_THREADS)
            if (group[j] == grp && news(j) > 0) {
                atomicMin(&s_low, j);
                break;
            }
        __syncthreads();
        ref = min(b, s_low);
    }
    // slots of whole committed pages that both hold
    int slots = 0;
    if (ref >= 0 && ref != b) {
        slots = min(lens[b], lens[ref]) / P;
        __syncthreads();
        if (tid == 0) s_low = slots;
        __syncthreads();
        const int32_t *ta = table + static_cast<int64_t>(b) * width, *tb = table + static_cast<int64_t>(ref) * width;
        for (int s0 = 0; s0 < slots; s0 += 8 * SP_THREADS) {  // eight loads in flight, until they differ
            int32_t x[8], y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int s = s0 + k * SP_THREADS + tid;
                const bool on = s < slots && SD_INB(s < width && ref < B, status, 128);  // site 128: table entry
                x[k] = on ? ta[s] : 0;
                y[k] = on ? tb[s] : 0;
            }
            bool differ = false;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (x[k] != y[k] || x[k] < 0 || x[k] >= n_pages) {
                    atomicMin(&s_low, s0 + k * SP_THREADS + tid);
                    differ = true;
                }
            if (__syncthreads_or(differ)) break;
        }
        __syncthreads();
        slots = s_low;
    }
    if (tid == 0) {
        pl.ref[b] = ref;
        pl.common[b] = slots;
        __threadfence();
        s_last = atomicAdd(&pl.head[0], 1) == B - 1;
    }
    __syncthreads();
    if (!s_last) return;
    // ---- the lists
    __threadfence();
    if (tid == 0) pl.head[0] = 0;
    for (int j = tid; j < B; j += SP_THREADS) {
        s_ref[j] = __ldcg(&pl.ref[j]);
        s_n[j] = s_ref[j] >= 0 ? news(j) : 0;
        s_min[j] = INT32_MAX;
        s_at[j] = 0;
    }
    __syncthreads();
    for (int j = tid; j < B; j += SP_THREADS)
        if (s_ref[j] >= 0) {
            if (s_ref[j] != j) atomicMin(&s_min[s_ref[j]], __ldcg(&pl.common[j]));
            atomicAdd(&s_at[s_ref[j]], static_cast<uint32_t>(s_n[j]));
        }
    __syncthreads();
    // a group's prefix in whole tiles (a group of one has none), and what all members but one of each leave out
    if (tid == 0) s_low = 0;
    __syncthreads();
    for (int j = tid; j < B; j += SP_THREADS)
        s_min[j] = s_ref[j] == j && s_min[j] != INT32_MAX ? static_cast<int32_t>(static_cast<int64_t>(s_min[j]) * P / PA_KT) : 0;
    __syncthreads();
    int64_t less = 0;
    for (int j = tid; j < B; j += SP_THREADS)
        if (s_ref[j] >= 0 && s_ref[j] != j) less += static_cast<int64_t>(s_min[s_ref[j]]) * H_kv;
    if (less > 0) atomicAdd(&s_low, static_cast<int32_t>(min(less, static_cast<int64_t>(1 << 20))));  // (1024 of them at most)
    __syncthreads();
    const bool worth = s_low >= worth_it;
    // groups in the order of their lowest members: each thread takes neighbours, (groups << 16 | rows) summed over all before
    const int per = (B + SP_THREADS - 1) / SP_THREADS, j0 = min(B, tid * per), j1 = min(B, j0 + per);
    uint32_t sum = 0;
    for (int j = j0; j < j1; ++j) {
        if (!worth) s_min[j] = 0;
        if (s_min[j] > 0) sum += 1u << 16 | s_at[j];
    }
    uint32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    uint32_t at = inc - sum, all = 0;
    for (int i = 0; i < SP_THREADS / 32; ++i) {
        if (i < warp) at += s_warp[i];
        all += s_warp[i];
    }
    for (int j = j0; j < j1; ++j)
        if (s_min[j] > 0) {
            const uint32_t n = s_at[j], v = at >> 16;
            if (SD_INB(v < static_cast<uint32_t>(B) / 2 && (at & 0xffffu) + n <= static_cast<uint32_t>(B) * M, status, 126)) {  // site 126: group
                pl.first[v] = static_cast<int32_t>(at & 0xffffu);
                pl.rows[v] = static_cast<int32_t>(n);
                pl.len[v] = s_min[j] * PA_KT;
                pl.leader[v] = j;
            }
            s_at[j] = at & 0xffffu;  // where its rows begin
            at += 1u << 16 | n;
        }
    for (int v = static_cast<int>(all >> 16) + tid; v < B / 2; v += SP_THREADS) pl.rows[v] = pl.len[v] = 0;
    __syncthreads();
    for (int j = tid; j < B; j += SP_THREADS) {
        const int r = s_ref[j], tiles = r >= 0 ? s_min[r] : 0;
        pl.skip[j] = tiles;
        if (tiles == 0) continue;
        int to = static_cast<int>(s_at[r]);
        for (int i = r; i < j; ++i) to += s_ref[i] == r ? s_n[i] : 0;
        pl.start[j] = to;
        for (int i = 0; i < s_n[j]; ++i)
            if (SD_INB(to + i < B * M, status, 127)) pl.rows_of[to + i] = j * M + i;  // site 127: query row of a group
    }
}

}  // namespace sdv

using namespace sdv;

extern "C" {

void sd_debug_share_from(int64_t tiles) { g_worth = tiles < 1 ? 1 : tiles > (1 << 20) ? (1 << 20) : tiles; }

size_t sd_paged_attn_shared_workspace_bytes(int32_t B, int32_t M, int32_t H, int32_t H_kv, int32_t D) {
    if (!sd_paged_attn_workspace_bytes(B, M, H, H_kv, D)) return 0;
    return shared_ws(nullptr, B, M, H, D).total;
}

sd_status sd_paged_attn_shared(const sd_kv_pages *pages, const int32_t *table, int32_t width, const int32_t *lens,
                               const int32_t *n_new, const int32_t *group, int32_t B, int32_t M, int32_t H, const float *q,
                               int64_t q_seq_stride, int64_t q_row_stride, const int32_t *parent, float *out,
                               int64_t out_seq_stride, int64_t out_row_stride, void *workspace, size_t ws_bytes,
                               sd_stream_t stream) {
    SD_NVTX("sd_paged_attn_shared");
    const size_t ahead = 256 + pa_counters();
    if (!group || !workspace || !aligned(workspace, 256) || ws_bytes < ahead) return SD_EINVAL;
    PaCall c;
    const sd_status st = pa_call(pages, table, width, lens, n_new, B, M, H, q, q_seq_stride, q_row_stride, parent, 0, 0, out,
                                 out_seq_stride, out_row_stride, static_cast<uint8_t *>(workspace) + ahead, ws_bytes - ahead, c);
    if (st != SD_OK) return st;
    const SharedWs w = shared_ws(workspace, B, M, H, c.D);
    if (ws_bytes < w.total) return SD_EINVAL;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // the most tiles that could be left out
    const int64_t most = static_cast<int64_t>(B - 1) * (static_cast<int64_t>(width) * c.a.P / PA_KT) * c.a.H_kv;
    if (most < g_worth) return pa_rows(c, PA_ALL, s);
    if (launch(shared_plan_kernel, dim3(B), dim3(SP_THREADS), 0, s, w.p, table, width, lens, n_new, group, B, M, c.a.P, c.a.H_kv,
               c.a.n_pages, g_worth, c.a.status) != cudaSuccess)
        return SD_ECUDA;
    PaCall g = c;
    size_t off_ml, off_o;
    pa_workspace(c.D, &off_ml, &off_o);
    g.a.B = B / 2;
    g.a.lens = w.p.len;
    g.a.n_new = w.p.rows;
    g.a.parent = nullptr;
    g.a.first = w.p.first;
    g.a.leader = w.p.leader;
    g.a.rows_of = w.p.rows_of;
    g.a.out = w.prefix_o;
    g.a.pre_ml = w.prefix_ml;
    g.a.counters = w.counters;
    g.a.part_ml = reinterpret_cast<float2 *>(w.partials + off_ml);
    g.a.part_o = reinterpret_cast<float *>(w.partials + off_o);
    const sd_status r = pa_prefix(g, B * M * c.a.g, s);
    if (r != SD_OK) return r;
    c.a.skip = w.p.skip;
    c.a.start = w.p.start;
    c.a.pre_ml = w.prefix_ml;
    c.a.pre_o = w.prefix_o;
    return pa_rows(c, PA_OWN, s);
}

}  // extern "C"
