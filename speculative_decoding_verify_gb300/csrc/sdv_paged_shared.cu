// sdv_paged_shared.cu - attention of a batch whose sequences share prefixes of pages, each prefix computed once for all.
//
// The softmax over a sequence's rows is split behind its group's shared rows: with (m, l, o) the maximum, the sum and
// the normalised output of either part,
//   out = (2^(m_p - m) l_p o_p + 2^(m_o - m) l_o o_o) / (2^(m_p - m) l_p + 2^(m_o - m) l_o),  m = max(m_p, m_o).
// On the stream:
//   the plan: what the tables say is shared, whether that is worth it, and the lists of the groups' query rows;
//   the prefixes: the many-row kernel with all new rows of a group as the rows of one "sequence" (128 of them share each
//   64-row tile of keys), into the workspace; a run that is cut between CTAs stays as partials (joined there, 128 rows
//   of up to a dozen of them were one CTA's work: 17 us behind the others);
//   each sequence's rows behind its prefix, as sd_paged_attn computes them, beside the prefixes as those leave the SMs
//   (after_plan: what orders them behind the plan);
//   the join, a warp per query row and head: its prefix's partials and its own.
// So a prefix is read from HBM once per group (per 128 query rows from L2), where sd_paged_attn reads it once per sequence.
#include "sdv_paged_attn.cuh"

namespace sdv {

constexpr int SP_THREADS = 256;
// Tiles of keys (per KV head and member) that have to be left out for the prefixes' launch to pay: it and the join cost
// about as long as 3000 of them.  Where the tables cannot hold SP_LOOK of them, which the plan costs too, nobody looks.  (A
// test may set another number for both.)  us of sd_paged_attn / with the prefix shared, 8 KV heads, one new row a member:
//   tiles left out         D = 128 fp16   D = 64 int8    D = 256 fp16
//    6000 (4 x 16000 rows)  42.4 / 42.1    42.8 / 42.9    96 / 81
//    7440 (16 x 4000)       41.3 / 40.4    42.3 / 41.0    94 / 65
//    7560 (64 x 1000)       45.9 / 51.6    45.6 / 49.9   104 / 84
//   14000 (8 x 16000)       70.5 / 45.4    74.2 / 46.9   175 / 113
// A tile counts the same whatever its bytes, its members' query rows and the number of members: many members of a short
// prefix lose up to 12 % there, and D = 256 would gain from fewer tiles on.
constexpr int64_t SP_WORTH = 3000, SP_LOOK = 6000;
static int64_t g_share_from = 0;

// The plan, in the workspace.
struct SharedPlan {
    int32_t *head;  // [0] CTAs that are done (0 between calls), [1] rows of rows_of
    int32_t *tickets;  // of the CTAs of the sequences' launch (0 between calls)
    int32_t *ref, *common;  // [B]: a sequence's group as its lowest member (-1: none), slots that it shares with it
    int32_t *skip;          // [B] tiles of the prefix
    int4 *at;       // [B] its group's first tile in the line of the prefixes' tiles (two words), row groups per KV head, the
                    // sequence's first row in the group
    int64_t *line;  // that line's length
    int32_t *first, *rows, *len, *leader;  // [B / 2]: the groups
    int32_t *rows_of;                      // [B * M]
};
struct SharedWs {
    SharedPlan p;
    uint8_t *attn;  // the workspace of the launch for the sequences; the prefixes' has partials of its own
    uint8_t *partials;
    float2 *prefix_ml, *own_ml;
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
    w.p.tickets = reinterpret_cast<int32_t *>(take(pa_counters()));
    w.attn = take(pa_workspace(D, nullptr, nullptr));
    w.partials = take(pa_workspace(D, nullptr, nullptr));
    w.p.ref = ints(B);
    w.p.common = ints(B);
    w.p.skip = ints(B);
    w.p.at = reinterpret_cast<int4 *>(take(16 * static_cast<size_t>(B)));
    w.p.line = reinterpret_cast<int64_t *>(take(8));
    w.p.first = ints(B);
    w.p.rows = ints(B);
    w.p.len = ints(B);
    w.p.leader = ints(B);
    const size_t rows = static_cast<size_t>(B) * M;
    w.p.rows_of = ints(rows);
    w.prefix_ml = reinterpret_cast<float2 *>(take(rows * H * 8));
    w.own_ml = reinterpret_cast<float2 *>(take(rows * H * 8));
    w.prefix_o = reinterpret_cast<float *>(take(rows * H * D * 4));
    w.total = at;
    return w;
}

// One CTA per sequence compares its table with that of its group's lowest member; the last one to finish makes the lists.
__global__ void __launch_bounds__(SP_THREADS) shared_plan_kernel(SharedPlan pl, const int32_t *table, int32_t width,
                                                                 const int32_t *lens, const int32_t *n_new,
                                                                 const int32_t *group, int32_t B, int32_t M, int32_t P,
                                                                 int32_t H_kv, int32_t g, int32_t rp, int32_t n_pages,
                                                                 int64_t worth_it, int32_t n_tickets, int *status) {
    __shared__ int32_t s_ref[PG_MAX_B], s_n[PG_MAX_B], s_min[PG_MAX_B];
    __shared__ uint32_t s_at[PG_MAX_B], s_warp[SP_THREADS / 32];
    __shared__ int32_t s_low, s_last;
    __shared__ int64_t s_line[PG_MAX_B], s_sum[SP_THREADS / 32];
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
        s_min[j] = s_ref[j] == j && s_min[j] != INT32_MAX
                       ? static_cast<int32_t>(static_cast<int64_t>(s_min[j]) * P / PA_KT) : 0;
    __syncthreads();
    int64_t less = 0;
    for (int j = tid; j < B; j += SP_THREADS)
        if (s_ref[j] >= 0 && s_ref[j] != j) less += static_cast<int64_t>(s_min[s_ref[j]]) * H_kv;
    // (256 threads' at most: no sum passes 32 bits)
    if (less > 0) atomicAdd(&s_low, static_cast<int32_t>(min(less, static_cast<int64_t>(1 << 20))));
    __syncthreads();
    const bool worth = s_low >= worth_it;
    // groups in the order of their lowest members: each thread takes neighbours, (groups << 16 | rows) summed over all before
    const int per = (B + SP_THREADS - 1) / SP_THREADS, j0 = min(B, tid * per), j1 = min(B, j0 + per);
    uint32_t sum = 0;
    int64_t tiles_of = 0;  // and the tiles of their runs
    auto group_tiles = [&](int j) {
        return static_cast<int64_t>((static_cast<int>(s_at[j]) * g + rp - 1) / rp) * H_kv * s_min[j];
    };
    for (int j = j0; j < j1; ++j) {
        if (!worth) s_min[j] = 0;
        if (s_min[j] > 0) {
            sum += 1u << 16 | s_at[j];
            tiles_of += group_tiles(j);
        }
    }
    uint32_t inc = sum;
    int64_t tinc = tiles_of;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        const int64_t z = __shfl_up_sync(0xffffffffu, tinc, o);
        if (lane >= o) {
            inc += y;
            tinc += z;
        }
    }
    if (lane == 31) {
        s_warp[warp] = inc;
        s_sum[warp] = tinc;
    }
    __syncthreads();
    uint32_t at = inc - sum, all = 0;
    int64_t line = tinc - tiles_of, whole = 0;
    for (int i = 0; i < SP_THREADS / 32; ++i) {
        if (i < warp) {
            at += s_warp[i];
            line += s_sum[i];
        }
        all += s_warp[i];
        whole += s_sum[i];
    }
    if (tid == 0) {
        *pl.line = whole;
        pl.head[1] = static_cast<int32_t>(all & 0xffffu);
    }
    for (int j = j0; j < j1; ++j)
        if (s_min[j] > 0) {
            const uint32_t n = s_at[j], v = at >> 16;
            if (SD_INB(v < static_cast<uint32_t>(B) / 2 && (at & 0xffffu) + n <= static_cast<uint32_t>(B) * M, status,
                       126)) {  // site 126: group
                pl.first[v] = static_cast<int32_t>(at & 0xffffu);
                pl.rows[v] = static_cast<int32_t>(n);
                pl.len[v] = s_min[j] * PA_KT;
                pl.leader[v] = j;
            }
            s_line[j] = line;
            line += group_tiles(j);
            s_n[j] |= static_cast<int32_t>((n * g + rp - 1) / rp) << 5;  // row groups, above its own new rows
            s_at[j] = at & 0xffffu;  // where its rows begin
            at += 1u << 16 | n;
        }
    for (int v = static_cast<int>(all >> 16) + tid; v < B / 2; v += SP_THREADS) pl.rows[v] = pl.len[v] = 0;
    __syncthreads();
    for (int j = tid; j < B; j += SP_THREADS) {
        const int r = s_ref[j], tiles = r >= 0 ? s_min[r] : 0;
        pl.skip[j] = tiles;
        if (tiles == 0) continue;
        // (a walk over the group: 9 us in all for 72 sequences in groups of 16, 15 for 1024, 37 for 1024 in one group)
        int to = 0;
        for (int i = r; i < j; ++i) to += s_ref[i] == r ? s_n[i] & 31 : 0;
        pl.at[j] = make_int4(static_cast<int32_t>(s_line[r] & 0xffffffff), static_cast<int32_t>(s_line[r] >> 32),
                             s_n[r] >> 5, to);
        to += static_cast<int>(s_at[r]);
        for (int i = 0; i < (s_n[j] & 31); ++i)
            if (SD_INB(to + i < B * M, status, 127)) pl.rows_of[to + i] = j * M + i;  // site 127: query row of a group
    }
    __syncthreads();
    __threadfence();  // (with it the stores release what the CTA has written and seen)
    for (int i = tid; i < n_tickets; i += SP_THREADS)
        asm volatile("st.relaxed.gpu.b32 [%0], %1;" ::"l"(pl.tickets + i), "r"(1) : "memory");
}

struct JoinArgs {
    SharedPlan pl;
    PrefixLayout lay;
    const float2 *prefix_ml, *own_ml, *part_ml;
    const float *prefix_o, *part_o;
    float *out;
    int64_t o_sb, o_sm;
    int32_t B, M, H, g;
    int *status;
};

// A warp per query row and head: with (m, l, o) the maximum, the sum and the outputs (weights' sum times the average row) of
// each part, n the largest m,
//   out = sum 2^(m - n) o / sum 2^(m - n) l.
// The parts' statistics are a lane's each, 32 at a time; the outputs of the first few are on their way beside them.
template <int D>
__global__ void __launch_bounds__(256, 4) shared_join_kernel(const JoinArgs a) {
    constexpr int NV = D / 128 > 0 ? D / 128 : 1;  // 16-byte columns of a lane (D = 64: half a warp has one)
    constexpr int FLY = 4 / NV;                    // parts whose outputs are on their way
    pdl_wait();
    pdl_launch_dependents();
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const bool on = lane < D / 4;
    const int64_t items = static_cast<int64_t>(__ldcg(&a.pl.head[1])) * a.H, W = *a.pl.line;
    const int64_t G = min(static_cast<int64_t>(a.lay.grid), W);
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < items;
         it += static_cast<int64_t>(gridDim.x) * 8) {
        const int x = static_cast<int>(it / a.H), h = static_cast<int>(it - static_cast<int64_t>(x) * a.H);
        const int code = a.pl.rows_of[x], b = code / a.M, i = code - b * a.M;
        if (!SD_INB(x < a.B * a.M && code >= 0 && b < a.B, a.status, 129)) continue;  // site 129: joined row
        const int4 y = a.pl.at[b];
        const int T = a.pl.skip[b], kh = h / a.g, tg = (y.w + i) * a.g + h - kh * a.g;
        const int rg = tg / a.lay.rp, r = tg - rg * a.lay.rp;
        const int64_t run0 = (static_cast<int64_t>(static_cast<uint32_t>(y.x)) | static_cast<int64_t>(y.y) << 32) +
                             (static_cast<int64_t>(kh) * y.z + rg) * T;
        const int c0 = static_cast<int>(((run0 + 1) * G - 1) / W), n = static_cast<int>(((run0 + T) * G - 1) / W) - c0 + 1;
        // the sequence's own part, normalised
        const float2 own = a.own_ml[static_cast<int64_t>(code) * a.H + h];
        float4 *to = reinterpret_cast<float4 *>(a.out + b * a.o_sb + i * a.o_sm + static_cast<int64_t>(h) * D) + lane;
        float4 v[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) v[k] = on ? to[32 * k] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        auto slot_of = [&](int p) { return static_cast<int64_t>(2 * (c0 + p) + (p == 0)); };
        // part p: (maximum, sum, what its outputs are multiplied with); one that was never cut is normalised
        auto stats = [&](int p) {
            if (n == 1) {
                const float2 z = a.prefix_ml[it];
                return make_float3(z.x, z.y, z.y);
            }
            const float2 z = a.part_ml[slot_of(p) * a.lay.rp + r];
            return make_float3(z.x, z.y * a.lay.unit, a.lay.unit);
        };
        auto outs = [&](int p, int c4) {
            return n == 1 ? reinterpret_cast<const float4 *>(a.prefix_o) + it * (D / 4) + c4
                          : reinterpret_cast<const float4 *>(a.part_o) + (slot_of(p) * a.lay.rp + r) * (D / 4) + c4;
        };
        // (the first outputs are on their way beside the statistics)
        float4 t[FLY][NV];
        auto load = [&](int p0) {
#pragma unroll
            for (int q = 0; q < FLY; ++q)
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    t[q][k] = on && p0 + q < n ? __ldcg(outs(p0 + q, lane + 32 * k)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        };
        load(0);
        float m = own.x;
        for (int p = lane; p < n; p += 32) m = fmaxf(m, stats(p).x);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float w = own.y * exp2f(own.x - m);
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) v[k] = make_float4(v[k].x * w, v[k].y * w, v[k].z * w, v[k].w * w);
        for (int p0 = 0; p0 < n; p0 += 32) {
            const float3 z = p0 + lane < n ? stats(p0 + lane) : make_float3(m, 0.0f, 0.0f);
            const float e = exp2f(z.x - m), f = e * z.z;
            sum = fmaf(z.y, e, sum);
            const int np = min(32, n - p0);
            for (int q0 = 0; q0 < np; q0 += FLY) {
                if (p0 + q0 > 0) load(p0 + q0);
#pragma unroll
                for (int q = 0; q < FLY; ++q) {
                    const float g = __shfl_sync(0xffffffffu, f, (q0 + q) & 31);
                    if (q0 + q < np)
#pragma unroll
                        for (int k = 0; k < NV; ++k)
                            v[k] = make_float4(fmaf(t[q][k].x, g, v[k].x), fmaf(t[q][k].y, g, v[k].y), fmaf(t[q][k].z, g, v[k].z),
                                               fmaf(t[q][k].w, g, v[k].w));
                }
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        // (no weight at all: every score is below fp32's range)
        const float all = sum + w, inv = all == 0.0f ? 0.0f : 1.0f / all;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (on) to[32 * k] = make_float4(v[k].x * inv, v[k].y * inv, v[k].z * inv, v[k].w * inv);
    }
}

}  // namespace sdv

using namespace sdv;

extern "C" {

void sd_debug_share_from(int64_t tiles) { g_share_from = tiles < 0 ? 0 : tiles > (1 << 20) ? (1 << 20) : tiles; }

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
    if (!group || !workspace || !aligned(workspace, 256) || ws_bytes < ahead || (out && out == q)) return SD_EINVAL;
    PaCall c;
    const sd_status st = pa_call(pages, table, width, lens, n_new, B, M, H, q, q_seq_stride, q_row_stride, parent, 0, 0, out,
                                 out_seq_stride, out_row_stride, static_cast<uint8_t *>(workspace) + ahead, ws_bytes - ahead, c);
    if (st != SD_OK) return st;
    const SharedWs w = shared_ws(workspace, B, M, H, c.D);
    if (ws_bytes < w.total) return SD_EINVAL;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // the most tiles that could be left out
    const int64_t most = static_cast<int64_t>(B - 1) * (static_cast<int64_t>(width) * c.a.P / PA_KT) * c.a.H_kv;
    if (most < (g_share_from ? g_share_from : SP_LOOK)) return pa_rows(c, PA_ALL, s);
    const int rows = B * M * c.a.g;
    const PrefixLayout lay = pa_prefix_layout(c, rows);
    if (launch(shared_plan_kernel, dim3(B), dim3(SP_THREADS), 0, s, w.p, table, width, lens, n_new, group, B, M, c.a.P, c.a.H_kv,
               c.a.g, lay.rp, c.a.n_pages, g_share_from ? g_share_from : SP_WORTH, pa_own_grid(c), c.a.status) != cudaSuccess)
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
    g.a.row_ml = w.prefix_ml;
    g.a.counters = nullptr;  // (nothing is joined there)
    g.a.part_ml = reinterpret_cast<float2 *>(w.partials + off_ml);
    g.a.part_o = reinterpret_cast<float *>(w.partials + off_o);
    sd_status r = pa_prefix(g, rows, s);
    if (r != SD_OK) return r;
    c.a.skip = w.p.skip;
    c.a.row_ml = w.own_ml;
    c.a.tickets = w.p.tickets;
    r = pa_rows(c, PA_OWN, s);
    if (r != SD_OK) return r;
    JoinArgs ja = {w.p, lay, w.prefix_ml, w.own_ml, g.a.part_ml, w.prefix_o, g.a.part_o, out, out_seq_stride, out_row_stride,
                   B, M, H, c.a.g, c.a.status};
    const int64_t warps = static_cast<int64_t>(B) * M * H, most_ctas = static_cast<int64_t>(num_sms()) * 8;
    const int grid = static_cast<int>((warps + 7) / 8 < most_ctas ? (warps + 7) / 8 : most_ctas);
    const auto join = c.D == 64 ? shared_join_kernel<64> : c.D == 128 ? shared_join_kernel<128> : shared_join_kernel<256>;
    return launch(join, dim3(grid), dim3(256), 0, s, ja) == cudaSuccess ? SD_OK : SD_ECUDA;
}

}  // extern "C"
