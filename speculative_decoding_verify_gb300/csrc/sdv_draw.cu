// sdv_draw.cu - one token per row of logits: temperature, top-k, top-p and min-p, from given random numbers.
//
// With m the row's largest logit, token c weighs w_c = exp((l_c - m) / T), held as a whole number of 2^-44: sums of them
// are exact, so that no result depends on how the row is cut or in which order threads add.  The filters keep a
// prefix of the order (larger logit first, lower index among equals), so each is a threshold in that order and the strictest
// one counts; the token is the first in index order whose running sum of kept weights exceeds u times their total.
//
// A row is read from HBM once, by a cluster of CTAs that hold it in shared memory; what follows works there.  A warp has a
// run of neighbouring tokens, a lane four of each 128 of them; a lane whose largest logit is out of a pass's reach
// leaves its tokens out.  A filter's threshold is the token at a given count, or at a given sum of weights:
//   a small top-k looks at the lanes' largest logits first: no more tokens than about k are as large as the k-th of those.
//   They are listed in every CTA and ranked by comparing all with all, and everything else is done on the list;
//   otherwise histograms over the distance d = m - l (128 bins per octave first, or 512; a bin with more than DR_LIST tokens
//   is cut again, by the bits of d, then of l, then of the index): each CTA makes its own, one exchange later every CTA adds
//   up the few bins that decide.  Counts are exact; a bin's weights are 13- to 15-bit parts of its first token's, so their
//   sum only says where to look (about a token off in a flat row): a pass over the tokens then takes the exact sum of all before the
//   bin and lists those in it and beside it, and where the threshold is not among them the search goes on at the next token
//   before or behind, then by halves.
// A pass leaves the sum of each warp's kept tokens, so the draw is a search among those and a scan of one run.
// Every exchange is one cluster barrier: two for a row without top-k or top-p, three with a small top-k, four with top-p of a
// flat row, and one at each end.
#include <cooperative_groups.h>

#include <type_traits>

#include "sdv_common.cuh"

namespace cg = cooperative_groups;

namespace sdv {

constexpr int DR_THREADS = 512, DR_WARPS = DR_THREADS / 32;
// Bins of a histogram, 32 to a coarse one: 1024 beside a row that is held in shared memory; 4096 for one that is read again,
// where a bin of the first level mostly has few enough tokens to be listed (a level more is a pass more: 256 flat rows with
// top-p 174 -> 141 us; beside a held row as many would leave no place for it).
constexpr int bits_of(bool held) { return held ? 10 : 12; }
constexpr int DR_LIST = 256;      // tokens that are ranked directly
constexpr int DR_MOST_CTAS = 8;
constexpr int DR_VOCAB = 360448;  // most tokens of a row
constexpr int DR_ORDER = 4096;    // most rows that are put in order
constexpr uint32_t DR_BESIDE = 100;  // tokens on either side of a threshold that are listed with it
constexpr int DR_SMALL_K = 192;   // top-k for which about as many tokens are worth listing
constexpr uint32_t DR_FIRST = 0x3e000000u;  // the first histogram: 8 octaves of d from 2^-3 on, by the bits of d

struct DrawArgs {
    const float *logits;
    int64_t ld;
    int32_t V, chunk;  // chunk: tokens per CTA, a multiple of 4
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *tokens;
    float *prob, *probs;
    int64_t ldp;
    int32_t N, order;  // order: the rows that take longest come first
    int *status;
};

// the order of logits as whole numbers (-0 as 0), and back
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k ^ (static_cast<uint32_t>(static_cast<int32_t>(~k) >> 31) | 0x80000000u));
}
// a token in the order: larger first
__device__ __forceinline__ uint64_t place_of(float l, int idx) {
    return static_cast<uint64_t>(order_key(l)) << 32 | (0xffffffffu - static_cast<uint32_t>(idx));
}
__device__ __forceinline__ int place_idx(uint64_t at) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(at)); }

// Which tokens a search has come down to: ranges of the bits of d, of the key from above, and of the index.
struct Range {
    uint32_t lo[3], hi[3];
};

// what a histogram says of the bin that was looked for: the tokens before it and in it (a search by counts); or about the
// weight before it and the least number of tokens that the bins' weights take (a search by weights, where bins beside it come
// along as long as the tokens stay few: the sums are a little off)
struct Found {
    uint32_t bin, last, before_n, n;
    float before_m, target_m;  // in units of 2^-MASS
};

// What a pass over the tokens tells of a CTA: the sums of all weights, of those before the range and of the kept ones, and
// how many tokens are in the range.
struct Passed {
    uint64_t all, before, kept;
    uint32_t n;
};

template <bool HELD>
struct alignas(16) DrawShared {
    // ---- read or written by the cluster's other CTAs (what they write has two turns: a slow CTA still reads one)
    uint32_t bins[2][1 << bits_of(HELD)];                     // a level's histogram: tokens, or parts of weights
    uint32_t coarse[2][DR_MOST_CTAS][1 << (bits_of(HELD) - 5)];  // every CTA's: tokens, or weights (floats' bits)
    uint64_t list[2][DR_LIST];                   // this CTA's tokens in a pass's range
    Passed passed[2][DR_MOST_CTAS];              // every CTA's
    float tops[DR_MOST_CTAS];                    // every CTA's largest logit
    // ---- of this CTA alone
    uint64_t at[DR_LIST], w[DR_LIST];  // the cluster's list
    uint64_t cta_sum[DR_MOST_CTAS];
    uint64_t part[3][DR_WARPS];  // the warps' sums: of all, of those before, of the kept ones
    float warp_f[DR_WARPS];
    Found found;
    uint64_t thr, thr_sum;
    double low_log;
    float c_hi, c_lo, p, u;
    uint32_t heavy[DR_ORDER / 32];
    uint32_t listed;
    uint32_t after, upto;  // top-p's threshold is among tokens after+1 .. upto of the order
    bool walked;           // and a search by counts has been made for it
    int32_t k, bad;
};

__device__ __forceinline__ float ex2_approx(float x) {  // 2^x to about 2^-22, 0 below the normal numbers
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// exp((l - m) / T) of two tokens: the difference and its product with c = log2(e) / T in two floats each, so that a far
// token's weight is as good as a near one's; nothing below 2^-60
__device__ __forceinline__ float2 weights_of(float2 l, float m, float c_hi, float c_lo) {
    const float2 one = make_float2(-1.0f, -1.0f), c = make_float2(c_hi, c_hi);
    const float2 s = fadd2_rn(l, make_float2(-m, -m)), bb = ffma2_rn(l, one, s);
    const float2 left = fadd2_rn(ffma2_rn(ffma2_rn(bb, one, s), one, l), ffma2_rn(bb, one, make_float2(-m, -m)));
    const float2 down = fmul2_rn(s, make_float2(-c_hi, -c_hi));
    const float2 xl = ffma2_rn(left, c, ffma2_rn(s, make_float2(c_lo, c_lo), ffma2_rn(s, c, down)));
    const float2 g = ffma2_rn(xl, make_float2(0.693147182f, 0.693147182f), make_float2(1.0f, 1.0f));
    const float2 e = fmul2_rn(make_float2(ex2_approx(-down.x), ex2_approx(-down.y)), g);
    return make_float2(down.x < 60.0f ? e.x : 0.0f, down.y < 60.0f ? e.y : 0.0f);
}
__device__ __forceinline__ float weight_of(float l, float m, float c_hi, float c_lo) {
    return weights_of(make_float2(l, l), m, c_hi, c_lo).x;
}

// Weights as whole numbers of 2^-44, summed in two words: adding 4 leaves the multiples of 2^-21 in the bits, adding
// 1.5 * 2^-21 to the rest those of 2^-44 (under 2^22 of them, either sign).  What is added twice per weight comes off at
// the end.
constexpr uint32_t DR_ADDS = 511;  // (the second word's sum stays under 2^31)
struct Units {
    uint32_t hi, lo;
    __device__ __forceinline__ void add(float2 e) {
        const float2 t = fadd2_rn(e, make_float2(4.0f, 4.0f));
        const float2 r = ffma2_rn(fadd2_rn(t, make_float2(-4.0f, -4.0f)), make_float2(-1.0f, -1.0f), e);
        const float2 q = fadd2_rn(r, make_float2(7.152557373046875e-07f, 7.152557373046875e-07f));
        hi += __float_as_uint(t.x) + __float_as_uint(t.y);
        lo += __float_as_uint(q.x) + __float_as_uint(q.y);
    }
    __device__ __forceinline__ uint64_t sum(uint32_t n) const {  // n weights were added, at most DR_ADDS
        const uint32_t h = hi - n * 0x40800000u;
        const int32_t l = static_cast<int32_t>(lo - n * 0x35400000u);
        return (static_cast<uint64_t>(h) << 23) + static_cast<uint64_t>(static_cast<int64_t>(l));
    }
};
__device__ __forceinline__ uint64_t units(float e) {
    Units u = {0, 0};
    u.add(make_float2(e, 0.0f));
    return u.sum(2);
}
constexpr float DR_UNIT = 17592186044416.0f;  // 2^44

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

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <class T>
__device__ __forceinline__ T warp_scan(T v) {  // inclusive
    const int lane = static_cast<int>(threadIdx.x) & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}
template <class T>
__device__ __forceinline__ T before_me(T v) {  // the sum of the lanes before
    const T y = __shfl_up_sync(0xffffffffu, warp_scan(v), 1);
    return (threadIdx.x & 31) ? y : T(0);
}
// A search for a threshold so far: the range, the phase that cuts it next, and what the last histogram said.
struct Search {
    Range r;
    int phase;
    Found f;
};

// a logit as it counts: a NaN as minus infinity; in a row with plus infinities those share everything
__device__ __forceinline__ float clean(float v) { return fmaxf(v, -INFINITY); }
__device__ __forceinline__ float4 clean_of(float4 v, bool infinite) {
    if (infinite)
        return make_float4(v.x == INFINITY ? 0.0f : -INFINITY, v.y == INFINITY ? 0.0f : -INFINITY,
                           v.z == INFINITY ? 0.0f : -INFINITY, v.w == INFINITY ? 0.0f : -INFINITY);
    return make_float4(clean(v.x), clean(v.y), clean(v.z), clean(v.w));
}

// Four logits of a CTA from i (a multiple of four) on, minus infinity from `end` on.
__device__ __forceinline__ float4 four_of(const float *from, bool wide, int i, int end) {
    if (wide && i + 4 <= end) return *reinterpret_cast<const float4 *>(from + i);
    float4 v;
    v.x = i < end ? from[i] : -INFINITY;
    v.y = i + 1 < end ? from[i + 1] : -INFINITY;
    v.z = i + 2 < end ? from[i + 2] : -INFINITY;
    v.w = i + 3 < end ? from[i + 3] : -INFINITY;
    return v;
}

// What one CTA of a row's cluster of CS works with.  HELD: its logits are in shared memory, cleaned; else they are read
// again.
template <int CS, bool HELD>
struct Draw {
    const DrawArgs &a;
    DrawShared<HELD> &sh;
    const float *x;       // this CTA's logits (HELD: minus infinity up to a multiple of four)
    bool wide, infinite;  // not HELD: 16-byte loads; plus infinities
    int rank, lo, n;   // tokens [lo, lo + n) of the row
    int w0, w1;        // of these, this warp's
    float m, top, c_hi, c_lo;  // the row's largest logit, this thread's
    int level, turn;   // histograms and passes so far

    static constexpr int DR_BITS = bits_of(HELD), DR_BINS = 1 << DR_BITS, DR_COARSE = DR_BINS / 32, DR_SHIFT = 26 - DR_BITS;
    // a token's weight in a histogram: a part of its bin's first token's, in units of 2^-MASS (no CTA's sum passes 32 bits)
    static constexpr int MASS_BITS = CS == 1 ? 13 : CS == 2 ? 14 : 15;
    static_assert(static_cast<uint64_t>((DR_VOCAB + CS - 1) / CS + 3) << MASS_BITS < 1ull << 32, "a bin's sum");
    static constexpr float MASS_ONE = static_cast<float>(1 << (23 - MASS_BITS));  // adding it leaves the units in the bits
    static constexpr float PER_UNIT = static_cast<float>(1 << MASS_BITS) / 17592186044416.0f;  // of weights' units into these

    template <class T>
    __device__ __forceinline__ T *of(T *mine, int c) const {
        return cg::this_cluster().map_shared_rank(mine, c);
    }

    __device__ __forceinline__ float4 four(int i) const {
        if constexpr (HELD) return *reinterpret_cast<const float4 *>(x + i);
        return clean_of(four_of(x, wide, i, n), infinite);
    }

    // f(i, four logits from i on) for this lane's tokens.  Those that are read again come four loads at a time (a load that
    // may be cut short would wait for the one before: two branches write the same registers)
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        const int at = w0 + 4 * (static_cast<int>(threadIdx.x) & 31);
        if constexpr (HELD) {
#pragma unroll 2
            for (int i = at; i < w1; i += 128) f(i, *reinterpret_cast<const float4 *>(x + i));
        } else {
            constexpr int BATCH = 4;
            for (int i0 = at; i0 < w1; i0 += 128 * BATCH) {
                if (wide && i0 + 128 * (BATCH - 1) + 4 <= w1) {
                    float4 v[BATCH];
#pragma unroll
                    for (int j = 0; j < BATCH; ++j) v[j] = *reinterpret_cast<const float4 *>(x + i0 + 128 * j);
#pragma unroll
                    for (int j = 0; j < BATCH; ++j) f(i0 + 128 * j, clean_of(v[j], infinite));
                } else {
#pragma unroll 1
                    for (int j = 0; j < BATCH && i0 + 128 * j < w1; ++j) f(i0 + 128 * j, four(i0 + 128 * j));
                }
            }
        }
    }

    // bits of d, key from above, or index
    __device__ __forceinline__ uint32_t value(int phase, float l, int idx) const {
        if (phase == 0) return __float_as_uint(fabsf(l - m));
        return phase == 1 ? ~order_key(l) : static_cast<uint32_t>(idx);
    }
    // -1: before the range, 0: in it, 1: behind (d: the bits of its distance)
    __device__ __forceinline__ int side(const Range &r, uint32_t d, float l, int idx) const {
        if (d < r.lo[0]) return -1;
        if (d > r.hi[0]) return 1;
        const uint32_t k = value(1, l, idx), i = static_cast<uint32_t>(idx);
        if (k < r.lo[1]) return -1;
        if (k > r.hi[1]) return 1;
        return i < r.lo[2] ? -1 : i > r.hi[2] ? 1 : 0;
    }
    // where a bin of a level begins, as a distance
    __device__ __forceinline__ float edge(bool first, int phase, const Range &r, int shift, uint32_t bin) const {
        if (first) return bin == 0 ? 0.0f : __uint_as_float(DR_FIRST + (bin << DR_SHIFT));
        return __uint_as_float(phase == 0 ? r.lo[0] + (bin << shift) : r.lo[0]);
    }

    // A level: the tokens of the range (FIRST: all) counted, or weighed, by bins.  Ends with the exchange.
    template <bool FIRST, bool MASS>
    __device__ void histogram(int phase, const Range &r, int shift) {
        const int tid = static_cast<int>(threadIdx.x), b = level & 1;
        uint32_t *bins = sh.bins[b];
        for (int i = tid; i < DR_BINS; i += DR_THREADS) bins[i] = 0;
        __syncthreads();
        if (FIRST || value(0, top, 0) <= r.hi[0])
            each([&](int i, float4 v) {
                const float l[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t d = value(0, l[j], 0);
                    uint32_t bin;
                    float from = 0.0f;
                    if constexpr (FIRST) {
                        bin = first_bin(d);
                        if constexpr (MASS) {
                            constexpr uint32_t LAST = DR_FIRST + (static_cast<uint32_t>(DR_BINS - 1) << DR_SHIFT);
                            from = __uint_as_float(min(d & (0xffffffffu << DR_SHIFT), LAST));
                            if (bin == 0) from = 0.0f;
                        }
                    } else {
                        if (d < r.lo[0] || d > r.hi[0] || side(r, d, l[j], lo + i + j) != 0) continue;
                        bin = (value(phase, l[j], lo + i + j) - r.lo[phase]) >> shift;
                        if constexpr (MASS) from = edge(false, phase, r, shift, bin);
                    }
                    if (!SD_INB(bin < DR_BINS && i + 3 < a.chunk, a.status, 123)) continue;  // site 123: bin
                    if constexpr (MASS) {  // its weight as a part of the bin's first
                        const float part = ex2_approx((from - __uint_as_float(d)) * c_hi);
                        atomicAdd(&bins[bin], __float_as_uint(part + MASS_ONE) - __float_as_uint(MASS_ONE));
                    } else {
                        atomicAdd(&bins[bin], 1u);
                    }
                }
            });
        share<FIRST, MASS>(phase, r, shift);
    }
    // The first level over the threads' largest logits alone: as many different tokens.
    __device__ void histogram_of_tops() {
        const int tid = static_cast<int>(threadIdx.x);
        uint32_t *bins = sh.bins[level & 1];
        for (int i = tid; i < DR_BINS; i += DR_THREADS) bins[i] = 0;
        __syncthreads();
        atomicAdd(&bins[first_bin(value(0, top, 0))], 1u);
        share<true, false>(0, whole(), DR_SHIFT);
    }
    __device__ __forceinline__ static uint32_t first_bin(uint32_t d) {
        const int bin = (static_cast<int32_t>(d) - static_cast<int32_t>(DR_FIRST)) >> DR_SHIFT;
        return static_cast<uint32_t>(min(max(bin, 0), DR_BINS - 1));
    }
    // The coarse bins; every CTA gets them.
    template <bool FIRST, bool MASS>
    __device__ void share(int phase, const Range &r, int shift) {
        const int tid = static_cast<int>(threadIdx.x), b = level & 1;
        constexpr int OWN = DR_BINS / DR_THREADS, TEAM = 32 / OWN;  // bins of a thread, threads of a coarse bin
        const uint32_t *bins = sh.bins[b];
        __syncthreads();
        uint32_t cn = 0;
        float cm = 0.0f;
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            const uint32_t bin = OWN * tid + j;
            if constexpr (MASS) cm += static_cast<float>(bins[bin]) * ex2_approx(-c_hi * edge(FIRST, phase, r, shift, bin));
            else cn += bins[bin];
        }
#pragma unroll
        for (int o = TEAM / 2; o >= 1; o >>= 1) {
            if constexpr (MASS) cm += __shfl_xor_sync(0xffffffffu, cm, o);
            else cn += __shfl_xor_sync(0xffffffffu, cn, o);
        }
#pragma unroll
        for (int c = tid % TEAM; c < CS; c += TEAM) *of(&sh.coarse[b][rank][tid / TEAM], c) = MASS ? __float_as_uint(cm) : cn;
        cluster_arrive();
        cluster_wait();
        ++level;
    }

    // The bin of the last level with the token that brings the count (MASS: about the weight; a share of the whole level's
    // where target_m is under 0) to the target, from the CTAs' coarse bins and the bins of three of them.  Every CTA
    // finds the same.
    template <bool MASS>
    __device__ Found locate(bool first, int phase, const Range &r, int shift, uint32_t target_n, float target_m) {
        const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, b = (level - 1) & 1;
        if (tid < 32) {
            using Sum = typename std::conditional<MASS, float, uint32_t>::type;
            // NC coarse bins a lane: each one's sum, and that of all before it
            constexpr int NC = DR_COARSE / 32;
            Sum cs[NC], pre[NC], sum_c = 0;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                cs[i] = 0;
#pragma unroll
                for (int c = 0; c < CS; ++c) {
                    const uint32_t y = sh.coarse[b][c][NC * lane + i];
                    if constexpr (MASS) cs[i] += __uint_as_float(y);
                    else cs[i] += y;
                }
                pre[i] = sum_c;
                sum_c += cs[i];
            }
            const Sum pre_c = before_me(sum_c);
            Sum target;
            if constexpr (MASS) target = target_m < 0.0f ? -target_m * __shfl_sync(0xffffffffu, pre_c + sum_c, 31) : target_m;
            else target = target_n;
            // (rounded sums may fall short of their own total: the last bin that has any, then)
            int at = INT_MAX, there = 0;
#pragma unroll
            for (int i = NC - 1; i >= 0; --i) {
                pre[i] += pre_c;
                if (cs[i] > 0 && pre[i] + cs[i] >= target) at = NC * lane + i;
                if (cs[i] > 0) there = max(there, NC * lane + i);
            }
            at = __reduce_min_sync(0xffffffffu, at);
            there = __reduce_max_sync(0xffffffffu, there);
            const int q = at != INT_MAX ? at : there;
            // that coarse bin's and its neighbours' bins, three a lane
            const int g0 = min(max(q - 1, 0), DR_COARSE - 3), bin0 = 32 * g0 + 3 * lane;
            uint64_t raw[3] = {0, 0, 0};
#pragma unroll
            for (int c = 0; c < CS; ++c)
#pragma unroll
                for (int i = 0; i < 3; ++i) raw[i] += *of(&sh.bins[b][bin0 + i], c);
            Sum f[3], upto[3], mine = 0;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                if constexpr (MASS)
                    f[i] = static_cast<float>(raw[i]) * ex2_approx(-c_hi * edge(first, phase, r, shift, bin0 + i));
                else f[i] = static_cast<uint32_t>(raw[i]);
                mine += f[i];
                upto[i] = mine;
            }
            Sum pre_g = pre[0];
#pragma unroll
            for (int i = 1; i < NC; ++i)
                if (g0 % NC == i) pre_g = pre[i];
            const Sum ahead = __shfl_sync(0xffffffffu, pre_g, g0 / NC) + before_me(mine);
            int hit = INT_MAX, some = -1;
#pragma unroll
            for (int i = 2; i >= 0; --i) {
                upto[i] += ahead;
                if (f[i] > 0 && upto[i] >= target) hit = 3 * lane + i;
                if (f[i] > 0) some = max(some, 3 * lane + i);
            }
            hit = __reduce_min_sync(0xffffffffu, hit);
            some = __reduce_max_sync(0xffffffffu, some);
            const int who = hit != INT_MAX ? hit : max(some, 0);
            // value x[i] of bin k of the 96
            auto of_bin = [&](auto (&x)[3], int k) {
                return __shfl_sync(0xffffffffu, k % 3 == 0 ? x[0] : k % 3 == 1 ? x[1] : x[2], k / 3);
            };
            int lo = who, hi = who;
            uint32_t n[3], sum[3], all = 0;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                n[i] = static_cast<uint32_t>(MASS ? (raw[i] + ((1u << MASS_BITS) - 1)) >> MASS_BITS : raw[i]);
                all += n[i];
                sum[i] = all;
            }
            const uint32_t n_ahead = warp_scan(all) - all;
#pragma unroll
            for (int i = 0; i < 3; ++i) sum[i] += n_ahead;
            if constexpr (MASS) {
                const uint32_t who_sum = of_bin(sum, who), who_n = of_bin(n, who);
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const int k = 3 * lane + i;
                    if (k < who && who_sum - sum[i] + n[i] <= DR_BESIDE) lo = min(lo, k);
                    if (k > who && sum[i] - who_sum + who_n <= DR_BESIDE) hi = max(hi, k);
                }
                lo = __reduce_min_sync(0xffffffffu, lo);
                hi = __reduce_max_sync(0xffffffffu, hi);
            }
            const uint32_t inside = of_bin(sum, hi) - (of_bin(sum, lo) - of_bin(n, lo));
            const Sum before = of_bin(upto, lo) - of_bin(f, lo);
            if (lane == 0) {
                sh.found.bin = 32 * g0 + lo;
                sh.found.last = 32 * g0 + hi;
                sh.found.n = inside;
                if constexpr (MASS) {
                    sh.found.before_n = 0;
                    sh.found.before_m = before;
                    sh.found.target_m = target;
                } else {
                    sh.found.before_n = before;
                    sh.found.before_m = sh.found.target_m = 0.0f;
                }
            }
        }
        __syncthreads();
        const Found f = sh.found;
        __syncthreads();
        return f;
    }

    __device__ Range whole() const {
        Range r;
        for (int i = 0; i < 3; ++i) {
            r.lo[i] = 0;
            r.hi[i] = i == 2 ? static_cast<uint32_t>(a.V - 1) : 0xffffffffu;
        }
        return r;
    }
    // the first level and its bin's range
    template <bool MASS>
    __device__ Search start(uint32_t target_n, float target_m) {
        Search q = {whole(), 0, {}};
        histogram<true, MASS>(0, q.r, DR_SHIFT);
        q.f = locate<MASS>(true, 0, q.r, DR_SHIFT, target_n, target_m);
        if (q.f.bin > 0) q.r.lo[0] = DR_FIRST + (q.f.bin << DR_SHIFT);
        q.r.hi[0] = bin_end(q.f.last);
        return q;
    }
    __device__ __forceinline__ static uint32_t bin_end(uint32_t bin) {
        return bin < DR_BINS - 1 ? DR_FIRST + ((bin + 1) << DR_SHIFT) - 1 : 0xffffffffu;
    }
    // one level more
    template <bool MASS>
    __device__ void refine(Search &q, uint32_t target_n, float target_m) {
        while (q.phase < 2 && q.r.lo[q.phase] == q.r.hi[q.phase]) ++q.phase;
        const int phase = q.phase, shift = max(0, 32 - __clz(q.r.hi[phase] - q.r.lo[phase]) - DR_BITS);
        histogram<false, MASS>(phase, q.r, shift);
        const Found g = locate<MASS>(false, phase, q.r, shift, target_n - q.f.before_n, fmaxf(target_m - q.f.before_m, 0.0f));
        q.f = {g.bin, g.last, q.f.before_n + g.before_n, g.n, q.f.before_m + g.before_m, target_m};
        q.r.hi[phase] = min(q.r.hi[phase], q.r.lo[phase] + (g.last << shift) + ((1u << shift) - 1u));
        q.r.lo[phase] += g.bin << shift;
    }
    // by counts, to a range of at most DR_LIST tokens
    __device__ Search search_count(uint32_t target) {
        Search q = start<false>(target, 0.0f);
        while (q.f.n > DR_LIST) refine<false>(q, target, 0.0f);
        return q;
    }

    // A pass over the tokens: the sum of the weights before the range (not RANGED: of logits from `low` on) in every CTA, and
    // with TOTAL of all; of the kept ones (those before; with LOW only from `low` on) each warp's in sh.part[2] and each
    // CTA's in sh.cta_sum; the range's tokens in sh.at, sh.w (`listed` of them), false in `fits` if they are too many.
    template <bool RANGED, bool TOTAL, bool LOW>
    __device__ void pass(const Range &r, float low, uint64_t &before, uint64_t &all) {
        const int tid = static_cast<int>(threadIdx.x), t = turn++ & 1;
        if (tid == 0) sh.listed = 0;
        __syncthreads();
        uint64_t sum_a = 0, sum_b = 0, sum_k = 0;
        const bool reach = TOTAL || (RANGED ? value(0, top, 0) <= r.hi[0] : top >= low);
        Units sa = {0, 0}, sb = {0, 0}, sk = {0, 0};
        uint32_t added = 0;
        auto fold = [&]() {
            if (TOTAL) sum_a += sa.sum(added);
            sum_b += sb.sum(added);
            if (LOW) sum_k += sk.sum(added);
            sa = sb = sk = {0, 0};
            added = 0;
        };
        if (reach)
            each([&](int i, float4 v) {  // (behind the row's end: minus infinity)
                if (added > DR_ADDS - 4) fold();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 l = h ? make_float2(v.z, v.w) : make_float2(v.x, v.y);
                    const int at = i + 2 * h;
                    bool b0, b1;
                    if constexpr (RANGED) {
                        const uint32_t d0 = value(0, l.x, 0), d1 = value(0, l.y, 0);
                        b0 = d0 < r.lo[0];
                        b1 = d1 < r.lo[0];
                        if (!b0 && d0 <= r.hi[0]) b0 = list(r, t, d0, l.x, lo + at);
                        if (!b1 && d1 <= r.hi[0]) b1 = list(r, t, d1, l.y, lo + at + 1);
                    } else {
                        b0 = l.x >= low;
                        b1 = l.y >= low;
                    }
                    if (!TOTAL && !(b0 || b1)) continue;
                    const float2 e = weights_of(l, m, c_hi, c_lo);
                    const float2 eb = make_float2(b0 ? e.x : 0.0f, b1 ? e.y : 0.0f);
                    if constexpr (TOTAL) sa.add(e);
                    sb.add(eb);
                    if constexpr (LOW) sk.add(make_float2(l.x >= low ? eb.x : 0.0f, l.y >= low ? eb.y : 0.0f));
                    added += 2;
                }
            });
        fold();
        tell<TOTAL, LOW>(t, sum_a, sum_b, sum_k);
        hear<RANGED>(t, before, all);
    }
    // a listed token goes into the list; whether it is before the range
    __device__ __forceinline__ bool list(const Range &r, int t, uint32_t d, float l, int idx) {
        const int s = side(r, d, l, idx);
        if (s == 0) put(t, l, idx);
        return s < 0;
    }
    // the CTA's sums and list to all CTAs
    template <bool TOTAL, bool LOW>
    __device__ __forceinline__ void tell(int t, uint64_t sa, uint64_t sb, uint64_t sk) {
        const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
        if (TOTAL) sa = warp_sum(sa);
        sb = warp_sum(sb);
        sk = LOW ? warp_sum(sk) : sb;
        if (lane == 0) {
            sh.part[0][warp] = sa;
            sh.part[1][warp] = sb;
            sh.part[2][warp] = sk;
        }
        __syncthreads();
        if (warp == 0) {
            Passed p = {0, 0, 0, sh.listed};
            if (TOTAL) p.all = warp_sum(lane < DR_WARPS ? sh.part[0][lane] : uint64_t(0));
            p.before = warp_sum(lane < DR_WARPS ? sh.part[1][lane] : uint64_t(0));
            p.kept = LOW ? warp_sum(lane < DR_WARPS ? sh.part[2][lane] : uint64_t(0)) : p.before;
            if (lane < CS) *of(&sh.passed[t][rank], lane) = p;
        }
        cluster_arrive();
        cluster_wait();
    }
    template <bool LISTED>
    __device__ __forceinline__ void hear(int t, uint64_t &before, uint64_t &all) {
        const int tid = static_cast<int>(threadIdx.x);
        before = all = 0;
        if (tid < CS) sh.cta_sum[tid] = sh.passed[t][tid].kept;
        uint32_t from = 0;
        const uint64_t *src = nullptr;
#pragma unroll
        for (int c = 0; c < CS; ++c) {
            const uint32_t nc = sh.passed[t][c].n;
            before += sh.passed[t][c].before;
            all += sh.passed[t][c].all;
            if (LISTED && static_cast<uint32_t>(tid) >= from && static_cast<uint32_t>(tid) - from < nc && tid < DR_LIST)
                src = of(&sh.list[t][tid - from], c);
            from += nc;
        }
        fits = from <= DR_LIST;
        listed = LISTED && fits ? static_cast<int>(from) : 0;
        if (LISTED && tid < DR_LIST) {
            const uint64_t at = src && fits ? *src : 0;
            sh.at[tid] = at;
            sh.w[tid] = src && fits ? units(weight_of(key_logit(static_cast<uint32_t>(at >> 32)), m, c_hi, c_lo)) : 0;
        }
        __syncthreads();
    }
    // The tokens whose distance has at most the bits d_end, listed.
    __device__ void gather(uint32_t d_end) {
        const int tid = static_cast<int>(threadIdx.x), t = turn++ & 1;
        if (tid == 0) sh.listed = 0;
        __syncthreads();
        if (value(0, top, 0) <= d_end)
            each([&](int i, float4 v) {
                const float l[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (value(0, l[j], 0) <= d_end && i + j < n) put(t, l[j], lo + i + j);
            });
        __syncthreads();
        if (tid < DR_WARPS) sh.part[2][tid] = 0;
        if (tid < CS) *of(&sh.passed[t][rank], tid) = Passed{0, 0, 0, sh.listed};
        cluster_arrive();
        cluster_wait();
        uint64_t before, all;
        hear<true>(t, before, all);
    }
    __device__ __forceinline__ void put(int t, float l, int idx) {
        const uint32_t slot = atomicAdd(&sh.listed, 1u);
        if (slot < DR_LIST && SD_INB(slot < DR_LIST, a.status, 124))  // site 124: listed token
            sh.list[t][slot] = place_of(l, idx);
    }
    // how many tokens are before a range, in every CTA
    __device__ uint32_t count_before(const Range &r) {
        const int t = turn++ & 1;
        uint64_t mine = 0;
        each([&](int i, float4 v) {
            const float l[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) mine += side(r, value(0, l[j], 0), l[j], lo + i + j) < 0 ? 1 : 0;
        });
        tell<false, false>(t, 0, mine, 0);
        uint32_t sum = 0;
        for (int c = 0; c < CS; ++c) sum += static_cast<uint32_t>(sh.passed[t][c].before);
        return sum;
    }

    // The rank of this thread's listed token: weight and number of those before it (in the list, and as many more).
    __device__ __forceinline__ void ranks(uint64_t before_w, uint32_t before_n) {
        const int tid = static_cast<int>(threadIdx.x);
        rank_w = before_w;
        rank_n = before_n;
        if (tid >= listed) return;
        const uint64_t at = sh.at[tid];
#pragma unroll 8
        for (int j = 0; j < listed; ++j)
            if (sh.at[j] > at) {
                rank_w += sh.w[j];
                ++rank_n;
            }
    }
    // The listed token at which the count (by_mass: the weight) reaches `target` becomes the threshold; false: not listed.
    __device__ bool pick(bool by_mass, uint64_t target) {
        const int tid = static_cast<int>(threadIdx.x);
        bool hit = false;
        if (tid < listed) {
            hit = by_mass ? rank_w < target && target <= rank_w + sh.w[tid] : rank_n + 1 == target;
            if (hit) {
                sh.thr = sh.at[tid];
                sh.thr_sum = rank_w + sh.w[tid];
            }
        }
        return __syncthreads_or(hit) != 0;
    }
    int listed;
    bool fits;
    uint64_t rank_w;
    uint32_t rank_n;
};

// The row of a cluster where there are more than the GPU holds at once: first those that may have to be ordered by weight,
// then the others (a late one of the first kind is several times as long behind the rest: 96 -> 86 us for 256 rows with
// settings of their own).
__device__ __forceinline__ int row_in_order(const DrawArgs &a, uint32_t *heavies, int q) {
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
    for (int r = tid; r < DR_ORDER; r += DR_THREADS) {
        bool heavy = false;
        if (r < a.N) {
            const int k = a.top_k ? a.top_k[r] : 0;
            heavy = a.top_p[r] < 1.0f && (k == 0 || k > DR_SMALL_K) && !(a.temperature && a.temperature[r] == 0.0f);
        }
        const uint32_t word = __ballot_sync(0xffffffffu, heavy);
        if (lane == 0) heavies[r >> 5] = word;
    }
    __syncthreads();
    constexpr int PER = DR_ORDER / 32 / 32;  // words of a lane
    uint32_t w[PER], first = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) first += __popc(heavies[PER * lane + i]);
    first = warp_sum(first);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r0 = 32 * (PER * lane + i);
        const uint32_t there = r0 >= a.N ? 0u : a.N - r0 >= 32 ? 0xffffffffu : (1u << (a.N - r0)) - 1u;
        w[i] = (q < static_cast<int>(first) ? heavies[PER * lane + i] : ~heavies[PER * lane + i]) & there;
        sum += __popc(w[i]);
    }
    uint32_t rank = q < static_cast<int>(first) ? q : q - first;
    const uint32_t upto = warp_scan(sum);
    int row = 0;
    if (rank < upto && rank >= upto - sum) {
        rank -= upto - sum;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t n = __popc(w[i]);
            if (rank < n) {
                row = 32 * (PER * lane + i) + static_cast<int>(__fns(w[i], 0, static_cast<int>(rank) + 1));
                rank = 0xffffffffu;
            } else if (rank != 0xffffffffu) {
                rank -= n;
            }
        }
    }
    return static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(row)));
}

// (Two CTAs per SM have 64 registers a thread: where a row is held nothing is spilled, where it is read again 32 to 64 bytes a
// thread are, beside 176 to 192 of stack.)
template <int CS, bool HELD>
__global__ void __launch_bounds__(DR_THREADS, 2) sample_kernel(const DrawArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    DrawShared<HELD> &sh = *reinterpret_cast<DrawShared<HELD> *>(smem_raw);
    float *held = reinterpret_cast<float *>(smem_raw + sizeof(DrawShared<HELD>));
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    int64_t row = blockIdx.x / CS;
    const int rank = static_cast<int>(blockIdx.x % CS);  // (the clusters are made of neighbours)
    const int lo = min(a.V, rank * a.chunk), n = min(a.V, lo + a.chunk) - lo;

    cluster_arrive();  // that this CTA runs, and may be written to
    pdl_wait();
    pdl_launch_dependents();
    if (a.order) row = row_in_order(a, sh.heavy, static_cast<int>(row));
    const float *from = a.logits + row * a.ld + lo;
    if (tid == 0) {  // the row's settings
        const float T = a.temperature ? a.temperature[row] : 1.0f, p = a.top_p ? a.top_p[row] : 1.0f;
        const float low = a.min_p ? a.min_p[row] : 0.0f, u = a.u[row];
        const int k = a.top_k ? a.top_k[row] : 0;
        sh.bad = !(T >= 0.0f && T < INFINITY) || !(p > 0.0f && p <= 1.0f) || !(low >= 0.0f && low <= 1.0f) ||
                 !(u >= 0.0f && u < 1.0f) || k < 0;
        // (held under 10^36: temperatures below 2^-119 count as that)
        const double c = T > 0.0f ? fmin(1.4426950408889634 / static_cast<double>(T), 1e36) : 1.4426950408889634;
        sh.c_hi = static_cast<float>(c);
        sh.c_lo = static_cast<float>(c - static_cast<double>(sh.c_hi));
        sh.k = T == 0.0f ? 1 : k >= a.V ? 0 : k;
        sh.p = p;
        sh.u = u;
        sh.low_log = low > 0.0f && T > 0.0f ? static_cast<double>(T) * log(static_cast<double>(low)) : -INFINITY;
    }
    // ---- the row's tokens of this CTA; a NaN counts as minus infinity, and minus infinity fills up the last four
    const int run = (n + 4 * DR_WARPS - 1) / (4 * DR_WARPS) * 4, w0 = min(n, warp * run), w1 = min(n, w0 + run);
    float mine = -INFINITY;
    const bool wide = (reinterpret_cast<uintptr_t>(from) & 15) == 0;
    auto take = [&](int i, float4 v) {
        if (!SD_INB(i + 4 <= a.chunk, a.status, 125)) return;  // site 125: logits
        const float4 c = make_float4(clean(v.x), clean(v.y), clean(v.z), clean(v.w));
        if constexpr (HELD) *reinterpret_cast<float4 *>(held + i) = c;
        mine = fmaxf(mine, fmaxf(fmaxf(c.x, c.y), fmaxf(c.z, c.w)));
    };
    constexpr int FLY = HELD ? 5 : 8;
    const int whole = wide ? w0 + (w1 - w0) / 4 * 4 : w0;
    for (int i0 = w0 + 4 * lane; i0 < w1; i0 += FLY * 128) {
        float4 v[FLY];
#pragma unroll
        for (int j = 0; j < FLY; ++j)
            if (i0 + 128 * j < whole) v[j] = *reinterpret_cast<const float4 *>(from + i0 + 128 * j);
#pragma unroll
        for (int j = 0; j < FLY; ++j) {
            const int i = i0 + 128 * j;
            if (i < whole) take(i, v[j]);
            else if (i < w1) take(i, four_of(from, false, i, w1));
        }
    }
    float top = mine;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) sh.warp_f[warp] = top;
    __syncthreads();
    cluster_wait();
    if (tid < CS) {
        for (int i = 0; i < DR_WARPS; ++i) top = fmaxf(top, sh.warp_f[i]);
        *cg::this_cluster().map_shared_rank(&sh.tops[rank], tid) = top;
    }
    cluster_arrive();
    cluster_wait();
    float m = -INFINITY;
#pragma unroll
    for (int c = 0; c < CS; ++c) m = fmaxf(m, sh.tops[c]);
    const bool bad = sh.bad || m == -INFINITY;
    const bool infinite = m == INFINITY;
    if (infinite) {
        if constexpr (HELD)
            for (int i = tid; i < n; i += DR_THREADS) held[i] = held[i] == INFINITY ? 0.0f : -INFINITY;
        mine = mine == INFINITY ? 0.0f : -INFINITY;
        m = 0.0f;
    }
    // the lowest logit that min-p keeps; minus infinity never is
    float low = -3.402823466e38f;
    if (sh.low_log > -INFINITY) low = fmaxf(__double2float_ru(static_cast<double>(m) + sh.low_log), low) + 0.0f;
    __syncthreads();

    float inv = 0.0f;
    uint64_t thr = ~uint64_t(0);
    const float c_hi = sh.c_hi, c_lo = sh.c_lo;
    if (bad) {
        if (tid == 0 && rank == 0) {
            set_status(a.status, SD_EDEVICE);
            a.tokens[row] = -1;
            if (a.prob) a.prob[row] = 0.0f;
        }
    } else {
        Draw<CS, HELD> w = {a, sh, HELD ? held : from, wide, infinite, rank, lo, n, w0, w1, m, mine, c_hi, c_lo, 0, 0};
        const float p = sh.p;
        const uint32_t k = static_cast<uint32_t>(sh.k), low_d = __float_as_uint(fabsf(low - m));
        const bool has_low = low > -3.402823466e38f;
        uint64_t before, all = 0, target = 0;
        thr = static_cast<uint64_t>(order_key(low)) << 32;
        bool nucleus = p < 1.0f;  // top-p still to be done
        bool few = false;         // the list holds all that may be kept
        const Range none = w.whole();
        if (k > 0) {
            few = k <= DR_SMALL_K;
            if (few) {
                w.histogram_of_tops();
                const Found f = w.template locate<false>(true, 0, none, Draw<CS, HELD>::DR_SHIFT, k, 0.0f);
                w.gather(Draw<CS, HELD>::bin_end(f.bin));
                few = w.fits;
                w.ranks(0, 0);
            }
            if (!few) {
                const Search q = w.search_count(k);
                if (has_low && low_d <= q.r.hi[0]) w.template pass<true, false, true>(q.r, low, before, all);
                else w.template pass<true, false, false>(q.r, low, before, all);
                w.ranks(before, q.f.before_n);
            }
            w.pick(false, k);
            thr = max(thr, sh.thr);
            if (nucleus) target = whole_times<true>(p, sh.thr_sum);
            if (few && nucleus) {
                __syncthreads();
                w.pick(true, target);
                thr = max(thr, sh.thr);
                nucleus = false;
            }
        } else if (!nucleus || has_low) {
            // no order is needed where min-p alone keeps no more than top-p would
            if (nucleus) w.template pass<false, true, false>(none, low, before, all);
            else w.template pass<false, false, false>(none, low, before, all);
            if (nucleus) {
                target = whole_times<true>(p, all);
                nucleus = before > target;
            }
        }
        if (nucleus) {
            if (tid == 0) {
                sh.after = 0;
                sh.upto = static_cast<uint32_t>(a.V);
                sh.walked = false;
            }
            const bool known = target != 0;  // else the histogram's own sum says about where to look
            const float per_unit = Draw<CS, HELD>::PER_UNIT;
            Search q = w.template start<true>(0, known ? static_cast<float>(target) * per_unit : -p);
            const float about = q.f.target_m;
            while (q.f.n > DR_LIST - 32) w.template refine<true>(q, 0, about);
            bool found = false;
            for (int turn = 0; !found; ++turn) {
                const bool cut = has_low && low_d <= q.r.hi[0];
                if (!known && turn == 0) w.template pass<true, true, false>(q.r, low, before, all);
                else if (cut) w.template pass<true, false, true>(q.r, low, before, all);
                else w.template pass<true, false, false>(q.r, low, before, all);
                if (!known && turn == 0) target = whole_times<true>(p, all);
                if (!w.fits) {
                    w.template refine<true>(q, 0, static_cast<float>(target) * per_unit);
                    continue;
                }
                w.ranks(before, 0);
                found = w.pick(true, target);
                if (!found) {
                    // the threshold is before the range or behind it, among tokens after+1 .. upto: the next token there,
                    // by counts (the sums are mostly a token off), then the middle (where a temperature is so low that a
                    // bin's weights differ by more than its parts' bits, they may be off by most of the row)
                    const uint32_t ahead = w.count_before(q.r);
                    const bool back = target <= before, again = sh.walked;
                    const uint32_t after = back ? sh.after : ahead + w.listed, upto = back ? ahead : sh.upto;
                    __syncthreads();
                    if (tid == 0) {
                        sh.after = after;
                        sh.upto = upto;
                        sh.walked = true;
                    }
                    if (after >= upto) break;  // (never: the weights of all reach the target)
                    q = w.search_count(again ? after + (upto - after + 1) / 2 : back ? upto : after + 1);
                }
            }
            thr = max(thr, sh.thr);
        }
        __syncthreads();
        const uint64_t at = tid < w.listed ? sh.at[tid] : 0;
        const bool kept = tid < w.listed && at >= thr;
        if (few) {
            // ---- the draw from a list: each kept token's running sum in index order (the first CTA draws; where all
            // probabilities are wanted each needs the total)
            if (rank == 0 || a.probs) {
                if (tid < w.listed && !kept) sh.w[tid] = 0;
                __syncthreads();
                uint64_t total = 0, upto = 0;
#pragma unroll 8
                for (int j = 0; j < w.listed; ++j) {
                    const uint64_t y = sh.w[j];
                    total += y;
                    // (a lower index is a larger second half of the place)
                    upto += static_cast<uint32_t>(sh.at[j]) >= static_cast<uint32_t>(at) ? y : 0;
                }
                inv = DR_UNIT / static_cast<float>(total);
                const uint64_t want = whole_times<false>(sh.u, total);  // (under the total: u < 1)
                if (rank == 0 && kept && want < upto && upto - sh.w[tid] <= want) {
                    a.tokens[row] = place_idx(at);
                    if (a.prob) a.prob[row] = weight_of(key_logit(static_cast<uint32_t>(at >> 32)), m, c_hi, c_lo) * inv;
                }
            }
        } else {
            // ---- the draw: the listed tokens that are kept join their CTAs' and warps' sums
            if (kept) {
                const int idx = place_idx(at);
                atomicAdd(reinterpret_cast<unsigned long long *>(&sh.cta_sum[CS == 1 ? 0 : idx / a.chunk]), sh.w[tid]);
                if (idx >= lo && idx < lo + n)
                    atomicAdd(reinterpret_cast<unsigned long long *>(&sh.part[2][(idx - lo) / run]), sh.w[tid]);
            }
            __syncthreads();
            uint64_t total = 0, base = 0;
#pragma unroll
            for (int c = 0; c < CS; ++c) {
                if (c == rank) base = total;
                total += sh.cta_sum[c];
            }
            const uint64_t want = whole_times<false>(sh.u, total);
            inv = DR_UNIT / static_cast<float>(total);
            if (base <= want && want < base + sh.cta_sum[rank]) {
                // the warp whose run it falls on; the CTA's threads take four of its tokens each
                const uint64_t own = lane < DR_WARPS ? sh.part[2][lane] : 0, upto = base + warp_scan(own);
                const int q = __ffs(__ballot_sync(0xffffffffu, upto > want)) - 1;
                uint64_t done = __shfl_sync(0xffffffffu, upto - own, q);
                const int r0 = min(n, q * run), r1 = min(n, r0 + run);
                for (int i0 = r0; i0 < r1; i0 += 4 * DR_THREADS) {
                    const int i = i0 + 4 * tid;
                    float e[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    uint64_t s = 0;
                    if (i < r1) {
                        const float4 v = w.four(i);
                        const float l[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (i + j < r1 && place_of(l[j], lo + i + j) >= thr) e[j] = weight_of(l[j], m, c_hi, c_lo);
                            s += units(e[j]);
                        }
                    }
                    const uint64_t inc = warp_scan(s);
                    __syncthreads();
                    if (lane == 31) sh.part[0][warp] = inc;
                    __syncthreads();
                    const uint64_t pw = warp_scan(lane < DR_WARPS ? sh.part[0][lane] : uint64_t(0));
                    const uint64_t ahead = __shfl_sync(0xffffffffu, pw, max(warp - 1, 0));
                    uint64_t y = done + inc - s + (warp > 0 ? ahead : 0);
                    if (y <= want && want < y + s) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint64_t z = y + units(e[j]);
                            if (y <= want && want < z) {
                                a.tokens[row] = lo + i + j;
                                if (a.prob) a.prob[row] = e[j] * inv;
                            }
                            y = z;
                        }
                    }
                    done += __shfl_sync(0xffffffffu, pw, DR_WARPS - 1);
                }
            }
        }
    }
    if (a.probs) {
        float *to = a.probs + row * a.ldp + lo;
        const float tl = key_logit(static_cast<uint32_t>(thr >> 32));
        const int ti = place_idx(thr);  // (the last index where all of that logit are kept)
        auto prob = [&](float l, int i) {
            const bool in = !bad && (l > tl || (l == tl && (lo + i <= ti || ti < 0)));
            return in ? weight_of(l, m, c_hi, c_lo) * inv : 0.0f;
        };
        const bool wide_to = (reinterpret_cast<uintptr_t>(to) & 15) == 0;
        const Draw<CS, HELD> w = {a, sh, HELD ? held : from, wide, infinite, rank, lo, n};
        for (int i = 4 * tid; i < n; i += 4 * DR_THREADS) {
            const float4 v = w.four(i);
            const float4 e = make_float4(prob(v.x, i), prob(v.y, i + 1), prob(v.z, i + 2), prob(v.w, i + 3));
            if (wide_to && i + 4 <= n) {
                __stcs(reinterpret_cast<float4 *>(to + i), e);
            } else {
                to[i] = e.x;
                if (i + 1 < n) to[i + 1] = e.y;
                if (i + 2 < n) to[i + 2] = e.z;
                if (i + 3 < n) to[i + 3] = e.w;
            }
        }
    }
    cluster_arrive();  // no CTA leaves while another may read its shared memory
    cluster_wait();
}

template <int CS, bool HELD>
static cudaError_t sample_launch(const DrawArgs &a, int N, cudaStream_t s) {
    const cudaError_t e = allow_max_dynamic_smem(sample_kernel<CS, HELD>);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(N) * CS);
    cfg.blockDim = dim3(DR_THREADS);
    cfg.dynamicSmemBytes = sizeof(DrawShared<HELD>) + (HELD ? static_cast<size_t>(a.chunk) * 4 : 0);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CS;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<CS, HELD>, a);
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
    if (vocab > DR_VOCAB || N > INT32_MAX / DR_MOST_CTAS) return SD_EUNSUPPORTED;
    if (out_probs == logits) return SD_EINVAL;
    // (in a large batch every row's settings are read for its place in the order, by then rows may be drawn)
    if (top_k && out_tokens == top_k) return SD_EINVAL;
    if (out_prob && (out_prob == temperature || out_prob == top_p)) return SD_EINVAL;
    int *status = status_ptr();
    if (!status) return SD_ECUDA;
    // As many CTAs per row as the GPU holds at once beside the other rows', two per SM; two at least where top-p may have to
    // order a flat row; no more than the row has 1024 tokens for.  us by 1 / 2 / 4 / 8 CTAs, rows of 151936 tokens:
    //               64 rows            256 rows              1024 rows
    //   top-k 50    30 / 20 / 18 / 26  58 / 62 / 78 / 100    209 / 210 / 268 / 376
    //   T alone     36 / 22 / 21 / 27  76 / 74 / 76 / 93     252 / 233 / 277 / 348  (256 rows at once are read twice from HBM)
    //   flat top-p  78 / 47 / 41 / 66  137 / 142 / 153 / 239 459 / 457 / 571 / 916
    //   mixed                          123 / 83 / 85 / 117  (a setting of its own for each row)
    const int slots = 2 * num_sms(), least = top_p ? 2 : 1;
    int ctas = DR_MOST_CTAS;
    while (ctas > 1 &&
           (vocab <= static_cast<int64_t>(ctas) * 1024 || (ctas > least && static_cast<int64_t>(N) * ctas > slots)))
        ctas /= 2;
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
    a.N = N;
    a.order = top_p && static_cast<int64_t>(N) * ctas > slots && N <= DR_ORDER;
    a.status = status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // (two CTAs of an SM hold their logits in its shared memory where they fit)
    const bool held = (sizeof(DrawShared<true>) + static_cast<size_t>(a.chunk) * 4 + 1024) * 2 <= 228 * 1024;
    auto run = [&](auto h) {
        constexpr bool H = decltype(h)::value;
        return ctas == 1 ? sample_launch<1, H>(a, N, s) : ctas == 2 ? sample_launch<2, H>(a, N, s)
               : ctas == 4 ? sample_launch<4, H>(a, N, s) : sample_launch<8, H>(a, N, s);
    };
    const cudaError_t e = held ? run(std::true_type()) : run(std::false_type());
    return e == cudaSuccess ? SD_OK : SD_ECUDA;
}

}  // extern "C"
