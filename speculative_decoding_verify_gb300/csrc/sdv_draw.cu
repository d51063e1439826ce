// sdv_draw.cu - one token per row of logits: temperature, top-k, top-p and min-p, from given random numbers.
//
// With m the row's largest logit, token c weighs w_c = exp((l_c - m) / T), held as a whole number of 2^-44: sums of them
// are exact, so that no result depends on how the row is cut or in which order threads add.  The filters keep a
// prefix of the order (larger logit first, lower index among equals), so each is a threshold in that order and the strictest
// one counts; the token is the first in index order whose running sum of kept weights exceeds u times their total.
//
// A row is read from HBM once, by a cluster of CTAs that hold it in shared memory; what follows works there:
//   the thresholds by histograms over the distance d = m - l (128 bins per octave first; bins with more than DR_LIST tokens
//   are cut again, by the bits of d, then of l, then of the index), their bins added up over the cluster, each CTA a slice
//   of them; the last few tokens are listed in every CTA and ranked by comparing all with all;
//   the draw by one sum per thread over neighbouring tokens and a scan of those sums.
// Bound by the exchanges over the cluster for few rows, by the passes over shared memory for many.
#include <cooperative_groups.h>

#include "sdv_common.cuh"

namespace cg = cooperative_groups;

namespace sdv {

constexpr int DR_THREADS = 512, DR_WARPS = DR_THREADS / 32;
constexpr int DR_BINS = 2048;
constexpr int DR_LIST = 256;               // tokens that are ranked directly
constexpr int DR_MOST_CTAS = 8;
constexpr int DR_CHUNK = 45056;            // most tokens of a CTA
constexpr uint32_t DR_FIRST = 0x3b800000u;  // bits of 2^-8: where the first histogram's octaves start (16 of them)
constexpr float DR_UNIT = 17592186044416.0f;  // 2^44

struct DrawArgs {
    const float *logits;
    int64_t ld;
    int32_t V, chunk;  // chunk: tokens per CTA, a multiple of 4
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *tokens;
    float *prob, *probs;
    int64_t ldp;
    int *status;
};

// order of logits as whole numbers
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

// counts and weights of a histogram's slice, or of everything before it
struct Tally {
    uint32_t n;
    uint64_t w;
};

// what a search gives all CTAs: the bin, what is before it and how many are in it
struct Found {
    uint64_t before_w;
    uint32_t before_n, bin, n;
};

struct alignas(16) DrawShared {
    uint32_t hist_n[DR_BINS], hist_lo[DR_BINS], hist_hi[DR_BINS];
    uint64_t list_w[DR_LIST];
    uint64_t list_at[DR_LIST];  // key and index in the order's terms
    Tally total[2][DR_MOST_CTAS];  // of the first histogram and of the later ones
    uint64_t warp_w[DR_WARPS + 1];
    uint32_t warp_n[DR_WARPS + 1];
    uint64_t sums[DR_MOST_CTAS];
    float maxima[DR_MOST_CTAS];
    float warp_max[DR_WARPS];
    Found found;
    uint64_t thr, thr_sum;
    uint32_t list_n;
    float c_hi, c_lo;
    uint32_t key_low;
    int32_t k;
    float p, u;
    int bad;
};

// 2^x by its series in f ln 2 for x = round(x) + f: the terms behind the eighth power are under 2^-32
__device__ __forceinline__ float exp2_parts(float xh, float xl) {
    const float k = rintf(xh), f = (xh - k) + xl;
    float p = 1.3215487e-6f;
    p = fmaf(p, f, 1.5252734e-5f);
    p = fmaf(p, f, 1.5403530e-4f);
    p = fmaf(p, f, 1.3333558e-3f);
    p = fmaf(p, f, 9.6181291e-3f);
    p = fmaf(p, f, 5.5504109e-2f);
    p = fmaf(p, f, 2.4022651e-1f);
    p = fmaf(p, f, 6.9314718e-1f);
    p = fmaf(p, f, 1.0f);
    return p * __int_as_float((static_cast<int>(k) + 127) << 23);
}

// exp((l - m) / T): the difference and its product with log2(e) / T in two floats each, so that a far token's weight is as
// good as a near one's; nothing below 2^-60
__device__ __forceinline__ float weight_of(float l, float m, float c_hi, float c_lo) {
    if (l == m) return 1.0f;
    const float s = l - m, xh = s * c_hi;
    if (!(xh > -60.0f)) return 0.0f;
    const float bb = s - l, left = (l - (s - bb)) + (-m - bb);
    const float xl = fmaf(s, c_hi, -xh) + fmaf(s, c_lo, left * c_hi);
    return exp2_parts(xh, xl);
}
__device__ __forceinline__ uint64_t units(float w) { return __float2ull_rn(w * DR_UNIT); }

// floor(f * x) for 0 <= f <= 1 (up: the least whole number not below f * x)
template <bool UP>
__device__ __forceinline__ uint64_t whole_times(float f, uint64_t x) {
    const uint32_t b = __float_as_uint(f);
    const int e = static_cast<int>(b >> 23);
    const unsigned __int128 y = static_cast<unsigned __int128>(e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu) * x;
    const int down = 150 - (e ? e : 1);  // f = mantissa * 2^-down
    const uint64_t floor = down >= 128 ? 0 : static_cast<uint64_t>(y >> down);
    const bool rest = down >= 128 ? y != 0 : (static_cast<unsigned __int128>(floor) << down) != y;
    return floor + (UP && rest ? 1 : 0);
}

// What one CTA of a row's cluster works with.
struct Draw {
    const DrawArgs &a;
    DrawShared &sh;
    float *x;       // this CTA's logits
    Tally *first, *later;  // this CTA's slice of the first histogram and of a later one
    int rank, ctas, lo, n;  // tokens [lo, lo + n) of the row
    float m;
};

// Which tokens a search still goes through: ranges of the bits of d, of the key from above, and of the index.
struct Range {
    uint32_t lo[3], hi[3];
};
__device__ __forceinline__ uint32_t value_of(int phase, float l, float m, int idx) {
    if (phase == 0) return __float_as_uint(l == m ? 0.0f : m - l);
    return phase == 1 ? ~order_key(l) : static_cast<uint32_t>(idx);
}
__device__ __forceinline__ bool in_range(const Range &r, float l, float m, int idx) {
    const uint32_t d = value_of(0, l, m, idx), k = value_of(1, l, m, idx), i = static_cast<uint32_t>(idx);
    return d >= r.lo[0] && d <= r.hi[0] && k >= r.lo[1] && k <= r.hi[1] && i >= r.lo[2] && i <= r.hi[2];
}

// The row's histogram over the values of one phase (first: of all tokens over the octaves of d), added up over the
// cluster: each CTA is left with its slice in `slice`, and every CTA with all slices' totals.
__device__ void histogram(const Draw &w, bool first, int phase, const Range &r, int shift, bool mass, Tally *slice) {
    DrawShared &sh = w.sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < DR_BINS; i += DR_THREADS) sh.hist_n[i] = sh.hist_lo[i] = sh.hist_hi[i] = 0;
    __syncthreads();
    for (int i = tid; i < w.n; i += DR_THREADS) {
        const float l = w.x[i];
        uint32_t bin;
        if (first) {
            const uint32_t d = value_of(0, l, w.m, 0);
            bin = d < DR_FIRST ? 0u : min((d - DR_FIRST) >> 16, static_cast<uint32_t>(DR_BINS - 1));
        } else {
            if (!in_range(r, l, w.m, w.lo + i)) continue;
            bin = (value_of(phase, l, w.m, w.lo + i) - r.lo[phase]) >> shift;
        }
        if (!SD_INB(bin < DR_BINS, w.a.status, 123)) continue;  // site 123: bin
        atomicAdd(&sh.hist_n[bin], 1u);
        if (mass) {  // a 64-bit sum in two words, by the carry of the lower one
            const uint64_t u = units(weight_of(l, w.m, sh.c_hi, sh.c_lo));
            const uint32_t low = static_cast<uint32_t>(u);
            uint32_t high = static_cast<uint32_t>(u >> 32);
            if (low) high += atomicAdd(&sh.hist_lo[bin], low) > ~low;
            if (high) atomicAdd(&sh.hist_hi[bin], high);
        }
    }
    cluster.sync();
    const int bins = DR_BINS / w.ctas;  // of a slice
    Tally sum = {0, 0};
    for (int i = tid; i < bins; i += DR_THREADS) {
        Tally t = {0, 0};
        const int bin = w.rank * bins + i;
#pragma unroll 1
        for (int c = 0; c < w.ctas; ++c) {
            t.n += *cluster.map_shared_rank(&sh.hist_n[bin], c);
            if (mass) {
                t.w += *cluster.map_shared_rank(&sh.hist_lo[bin], c);
                t.w += static_cast<uint64_t>(*cluster.map_shared_rank(&sh.hist_hi[bin], c)) << 32;
            }
        }
        slice[i] = t;
        sum.n += t.n;
        sum.w += t.w;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        sum.n += __shfl_xor_sync(0xffffffffu, sum.n, o);
        sum.w += __shfl_xor_sync(0xffffffffu, sum.w, o);
    }
    if (lane == 0) {
        sh.warp_n[warp] = sum.n;
        sh.warp_w[warp] = sum.w;
    }
    __syncthreads();
    if (tid < w.ctas) {
        Tally t = {0, 0};
        for (int i = 0; i < DR_WARPS; ++i) {
            t.n += sh.warp_n[i];
            t.w += sh.warp_w[i];
        }
        *cluster.map_shared_rank(&sh.total[first ? 0 : 1][w.rank], tid) = t;
    }
    cluster.sync();
}

// The bin of the token that brings the count (or, by_mass, the weight) to `target`, and what is before that bin.
__device__ Found locate(const Draw &w, bool first, bool by_mass, uint64_t target) {
    DrawShared &sh = w.sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const Tally *slice = first ? w.first : w.later;
    const int bins = DR_BINS / w.ctas, per = (bins + DR_THREADS - 1) / DR_THREADS, b0 = tid * per, b1 = min(bins, b0 + per);
    Tally mine = {0, 0};
    for (int i = b0; i < b1; ++i) {
        mine.n += slice[i].n;
        mine.w += slice[i].w;
    }
    Tally inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t yn = __shfl_up_sync(0xffffffffu, inc.n, o);
        const uint64_t yw = __shfl_up_sync(0xffffffffu, inc.w, o);
        if (lane >= o) {
            inc.n += yn;
            inc.w += yw;
        }
    }
    __syncthreads();
    if (lane == 31) {
        sh.warp_n[warp] = inc.n;
        sh.warp_w[warp] = inc.w;
    }
    __syncthreads();
    Tally at = {inc.n - mine.n, inc.w - mine.w};
    for (int i = 0; i < warp; ++i) {
        at.n += sh.warp_n[i];
        at.w += sh.warp_w[i];
    }
    for (int c = 0; c < w.rank; ++c) {
        at.n += sh.total[first ? 0 : 1][c].n;
        at.w += sh.total[first ? 0 : 1][c].w;
    }
    for (int i = b0; i < b1; ++i) {
        const Tally t = slice[i];
        const uint64_t before = by_mass ? at.w : at.n, here = by_mass ? t.w : t.n;
        if (before < target && target <= before + here) {
            const Found f = {at.w, at.n, static_cast<uint32_t>(w.rank * bins + i), t.n};
            for (int c = 0; c < w.ctas; ++c) *cluster.map_shared_rank(&sh.found, c) = f;
        }
        at.n += t.n;
        at.w += t.w;
    }
    cluster.sync();
    return sh.found;
}

// The token at which the count reaches `target` (by_mass: at which the weight does), as (key, ~index) in one number, and
// the weight of all up to it.  The first histogram is there already.
__device__ void select(const Draw &w, bool by_mass, uint64_t target, bool mass, uint64_t &thr, uint64_t &thr_sum) {
    DrawShared &sh = w.sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = static_cast<int>(threadIdx.x);
    Range r;
    for (int i = 0; i < 3; ++i) {
        r.lo[i] = 0;
        r.hi[i] = i == 2 ? static_cast<uint32_t>(w.a.V - 1) : 0xffffffffu;
    }
    Found f = locate(w, true, by_mass, target);
    uint64_t before_w = f.before_w, before_n = f.before_n;
    if (f.bin > 0) r.lo[0] = DR_FIRST + (f.bin << 16);
    if (f.bin < DR_BINS - 1) r.hi[0] = DR_FIRST + ((f.bin + 1) << 16) - 1;
    int phase = 0;
    while (f.n > DR_LIST) {
        while (phase < 2 && r.lo[phase] == r.hi[phase]) ++phase;
        const uint32_t width = r.hi[phase] - r.lo[phase];
        const int shift = max(0, 32 - __clz(width) - 11);
        histogram(w, false, phase, r, shift, mass, w.later);
        f = locate(w, false, by_mass, target - (by_mass ? before_w : before_n));
        before_w += f.before_w;
        before_n += f.before_n;
        const uint32_t at = r.lo[phase] + (f.bin << shift);
        r.lo[phase] = at;
        r.hi[phase] = min(r.hi[phase], at + ((1u << shift) - 1u));
    }
    // the few that are left, in every CTA
    uint32_t *counter = cluster.map_shared_rank(&sh.list_n, 0);
    for (int i = tid; i < w.n; i += DR_THREADS) {
        const float l = w.x[i];
        if (!in_range(r, l, w.m, w.lo + i)) continue;
        const uint32_t slot = atomicAdd(counter, 1u);
        if (slot >= DR_LIST || !SD_INB(slot < DR_LIST, w.a.status, 124)) continue;  // site 124: listed token
        const uint64_t at = static_cast<uint64_t>(order_key(l)) << 32 | (0xffffffffu - static_cast<uint32_t>(w.lo + i));
        const uint64_t u = mass ? units(weight_of(l, w.m, sh.c_hi, sh.c_lo)) : 0;
        for (int c = 0; c < w.ctas; ++c) {
            *cluster.map_shared_rank(&sh.list_at[slot], c) = at;
            *cluster.map_shared_rank(&sh.list_w[slot], c) = u;
        }
    }
    cluster.sync();
    const int n = static_cast<int>(min(f.n, static_cast<uint32_t>(DR_LIST)));
    if (tid < n) {
        const uint64_t at = sh.list_at[tid], u = sh.list_w[tid];
        uint64_t bw = before_w, bn = before_n;
        for (int j = 0; j < n; ++j)
            if (sh.list_at[j] > at) {
                bw += sh.list_w[j];
                ++bn;
            }
        if (by_mass ? bw < target && target <= bw + u : bn + 1 == target) {
            sh.thr = at;
            sh.thr_sum = bw + u;
        }
    }
    if (tid == 0 && w.rank == 0) sh.list_n = 0;  // (the next list comes behind another exchange)
    __syncthreads();
    thr = sh.thr;
    thr_sum = sh.thr_sum;
}

__global__ void __launch_bounds__(DR_THREADS) sample_kernel(const DrawArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    DrawShared &sh = *reinterpret_cast<DrawShared *>(smem_raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    Tally *slices = reinterpret_cast<Tally *>(smem_raw + sizeof(DrawShared));
    float *x = reinterpret_cast<float *>(slices + 2 * (DR_BINS / ctas));
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / ctas;
    const int lo = min(a.V, rank * a.chunk), n = min(a.V, lo + a.chunk) - lo;
    const float *from = a.logits + row * a.ld + lo;

    pdl_wait();
    pdl_launch_dependents();
    // ---- the row's tokens of this CTA; a NaN counts as minus infinity, -0 as 0
    float top = -INFINITY;
    auto clean = [](float v) { return v != v ? -INFINITY : v + 0.0f; };
    const bool wide = (reinterpret_cast<uintptr_t>(from) & 15) == 0;
    const int n4 = wide ? n / 4 : 0;
    constexpr int FLY = 8;
    for (int i = tid; i < n4; i += FLY * DR_THREADS) {
        float4 v[FLY];
#pragma unroll
        for (int j = 0; j < FLY; ++j)
            if (i + j * DR_THREADS < n4) v[j] = __ldcs(reinterpret_cast<const float4 *>(from) + i + j * DR_THREADS);
#pragma unroll
        for (int j = 0; j < FLY; ++j)
            if (i + j * DR_THREADS < n4 && SD_INB(4 * (i + j * DR_THREADS) + 4 <= a.chunk, a.status, 125)) {  // site 125: logits
                const float4 c = make_float4(clean(v[j].x), clean(v[j].y), clean(v[j].z), clean(v[j].w));
                reinterpret_cast<float4 *>(x)[i + j * DR_THREADS] = c;
                top = fmaxf(top, fmaxf(fmaxf(c.x, c.y), fmaxf(c.z, c.w)));
            }
    }
    for (int i = 4 * n4 + tid; i < n; i += FLY * DR_THREADS) {
        float v[FLY];
#pragma unroll
        for (int j = 0; j < FLY; ++j)
            if (i + j * DR_THREADS < n) v[j] = __ldcs(from + i + j * DR_THREADS);
#pragma unroll
        for (int j = 0; j < FLY; ++j)
            if (i + j * DR_THREADS < n && SD_INB(i + j * DR_THREADS < a.chunk, a.status, 125)) {
                x[i + j * DR_THREADS] = clean(v[j]);
                top = fmaxf(top, x[i + j * DR_THREADS]);
            }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) sh.warp_max[warp] = top;
    if (tid == 0) sh.list_n = 0;
    __syncthreads();
    if (tid < ctas)
        for (int i = 0; i < DR_WARPS; ++i) top = fmaxf(top, sh.warp_max[i]);
    cluster.sync();  // every CTA of the cluster runs before another writes to its shared memory
    if (tid < ctas) *cluster.map_shared_rank(&sh.maxima[rank], tid) = top;
    cluster.sync();
    float m = -INFINITY;
    for (int c = 0; c < ctas; ++c) m = fmaxf(m, sh.maxima[c]);

    // ---- the row's settings
    if (tid == 0) {
        const float T = a.temperature ? a.temperature[row] : 1.0f, p = a.top_p ? a.top_p[row] : 1.0f;
        const float low = a.min_p ? a.min_p[row] : 0.0f, u = a.u[row];
        const int k = a.top_k ? a.top_k[row] : 0;
        sh.bad = !(T >= 0.0f && T < INFINITY) || !(p > 0.0f && p <= 1.0f) || !(low >= 0.0f && low <= 1.0f) ||
                 !(u >= 0.0f && u < 1.0f) || k < 0 || m == -INFINITY;
        const double c = T > 0.0f ? 1.4426950408889634 / static_cast<double>(T) : 1.4426950408889634;
        sh.c_hi = static_cast<float>(c);
        sh.c_lo = sh.c_hi < INFINITY ? static_cast<float>(c - static_cast<double>(sh.c_hi)) : 0.0f;
        sh.k = T == 0.0f ? 1 : k >= a.V ? 0 : k;
        sh.p = p;
        sh.u = u;
        // the lowest logit that min-p keeps; minus infinity never is
        sh.key_low = order_key(-INFINITY) + 1;
        if (low > 0.0f && T > 0.0f && m < INFINITY) {
            const float at = __double2float_ru(static_cast<double>(m) + static_cast<double>(T) * log(static_cast<double>(low)));
            sh.key_low = max(sh.key_low, order_key(at + 0.0f));
        }
        if (sh.bad && rank == 0) {
            set_status(a.status, SD_EDEVICE);
            a.tokens[row] = -1;
            if (a.prob) a.prob[row] = 0.0f;
        }
    }
    __syncthreads();
    const float c_hi = sh.c_hi, c_lo = sh.c_lo;
    const bool bad = sh.bad != 0;
    float inv = 0.0f;
    if (!bad) {
        const Draw w = {a, sh, x, slices, slices + DR_BINS / ctas, rank, ctas, lo, n, m};
        // ---- the thresholds
        uint64_t thr = static_cast<uint64_t>(sh.key_low) << 32;
        const int k = sh.k;
        const float p = sh.p;
        if (k > 0 || p < 1.0f) {
            const bool mass = p < 1.0f;
            histogram(w, true, 0, Range{}, 0, mass, w.first);
            uint64_t total = 0, at;
            for (int c = 0; c < ctas; ++c) total += sh.total[0][c].w;
            if (k > 0) {
                select(w, false, static_cast<uint64_t>(k), mass, at, total);
                thr = max(thr, at);
            }
            if (p < 1.0f) {
                uint64_t sum;
                select(w, true, whole_times<true>(p, total), mass, at, sum);
                thr = max(thr, at);
            }
        }
        // ---- the kept tokens' weights, over their logits; a thread sums neighbours (an odd number: no bank conflicts)
        const int per = ((n + DR_THREADS - 1) / DR_THREADS) | 1, i0 = min(n, tid * per), i1 = min(n, i0 + per);
        uint64_t mine = 0;
        for (int i = i0; i < i1; ++i) {
            const float l = x[i];
            const uint64_t at = static_cast<uint64_t>(order_key(l)) << 32 | (0xffffffffu - static_cast<uint32_t>(lo + i));
            const float e = at >= thr ? weight_of(l, m, c_hi, c_lo) : 0.0f;
            x[i] = e;
            mine += units(e);
        }
        uint64_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        __syncthreads();
        if (lane == 31) sh.warp_w[warp] = inc;
        __syncthreads();
        uint64_t at = inc - mine, all = 0;
        for (int i = 0; i < DR_WARPS; ++i) {
            if (i < warp) at += sh.warp_w[i];
            all += sh.warp_w[i];
        }
        if (tid < ctas) *cluster.map_shared_rank(&sh.sums[rank], tid) = all;
        cluster.sync();
        uint64_t total = 0;
        for (int c = 0; c < ctas; ++c) {
            if (c < rank) at += sh.sums[c];
            total += sh.sums[c];
        }
        // ---- the draw
        const uint64_t want = whole_times<false>(sh.u, total);  // (under the total: u < 1)
        inv = DR_UNIT / static_cast<float>(total);
        if (at <= want && want < at + mine) {
            int i = i0;
            for (; i < i1; ++i) {
                at += units(x[i]);
                if (at > want) break;
            }
            a.tokens[row] = lo + i;
            if (a.prob) a.prob[row] = x[i] * inv;
        }
    }
    if (a.probs) {
        __syncthreads();
        float *to = a.probs + row * a.ldp + lo;
        const int m4 = (reinterpret_cast<uintptr_t>(to) & 15) == 0 ? n / 4 : 0;
        for (int i = tid; i < m4; i += DR_THREADS) {
            const float4 e = reinterpret_cast<const float4 *>(x)[i];
            __stcs(reinterpret_cast<float4 *>(to) + i,
                   bad ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : make_float4(e.x * inv, e.y * inv, e.z * inv, e.w * inv));
        }
        for (int i = 4 * m4 + tid; i < n; i += DR_THREADS) to[i] = bad ? 0.0f : x[i] * inv;
    }
    cluster.sync();  // no CTA leaves while another may read its shared memory
}

}  // namespace sdv

using namespace sdv;

extern "C" {

sd_status sd_sample(const float *logits, int64_t ld, int64_t vocab, int32_t N, const float *u, const float *temperature,
                    const int32_t *top_k, const float *top_p, const float *min_p, int32_t *out_tokens, float *out_prob,
                    float *out_probs, int64_t ld_probs, sd_stream_t stream) {
    SD_NVTX("sd_sample");
    if (!logits || !u || !out_tokens || N < 1 || vocab < 1) return SD_EINVAL;
    if (ld < vocab || (out_probs && ld_probs < vocab)) return SD_EINVAL;
    if (!aligned(logits, 4) || (out_probs && !aligned(out_probs, 4))) return SD_EINVAL;
    if (vocab > static_cast<int64_t>(DR_MOST_CTAS) * DR_CHUNK || N > INT32_MAX / DR_MOST_CTAS) return SD_EUNSUPPORTED;
    int *status = status_ptr();
    if (!status) return SD_ECUDA;
    int ctas = DR_MOST_CTAS;
    while (ctas > 1 && vocab <= static_cast<int64_t>(ctas) * 1024) ctas /= 2;
    DrawArgs a = {};
    a.logits = logits;
    a.ld = ld;
    a.V = static_cast<int32_t>(vocab);
    a.chunk = static_cast<int32_t>((vocab + ctas - 1) / ctas + 3) / 4 * 4;
    a.u = u;
    a.temperature = temperature;
    a.top_p = top_p;
    a.min_p = min_p;
    a.top_k = top_k;
    a.tokens = out_tokens;
    a.prob = out_prob;
    a.probs = out_probs;
    a.ldp = ld_probs;
    a.status = status;
    if (allow_max_dynamic_smem(sample_kernel) != cudaSuccess) return SD_ECUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(N) * ctas);
    cfg.blockDim = dim3(DR_THREADS);
    cfg.dynamicSmemBytes = sizeof(DrawShared) + 2 * static_cast<size_t>(DR_BINS / ctas) * sizeof(Tally) +
                           static_cast<size_t>(a.chunk) * 4;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel, a) == cudaSuccess ? SD_OK : SD_ECUDA;
}

}  // extern "C"
