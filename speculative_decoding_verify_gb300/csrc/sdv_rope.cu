// sdv_rope.cu - rotary positions: of rows beside each other, and of a batch's new queries and keys on their way into the
// pages.
//
// A pair (a, b) of frequency f (radians per position) at position p becomes (a cos pf - b sin pf, a sin pf + b cos pf).
// The angle comes from whole numbers: f / 2 pi as a 64-bit fraction of a turn, times the position modulo 2^64, is the
// angle's fraction of a turn to 2^-64 of a turn per position, exact for the rest, at any position (a fp32 product p f is 0.06
// radians off at a position of a million; fp64 would run on a pipe that is a 64th as wide).  It is rounded to fp32 as a
// signed half turn, where sincospif takes it.
//
// A block takes one row's heads, RP_HEADS a lane with all their loads in flight, LR = D / 8 lanes a head: a lane has the same
// 8 elements (4 pairs) of each, and the block's threads form the row's sines and cosines once, a pair each, into shared
// memory (by every lane for itself they were half of the instructions: 16384 rows of 8 + 8 + 8 heads into 8-bit rows 97 -> 69
// us).  Bound by HBM for many rows, by the launch and one chain of loads for few.
#include <math.h>

#include "sdv_paged.cuh"

namespace sdv {

constexpr int RP_THREADS = 128;
constexpr int RP_HEADS = 4;  // heads of one lane's turn

struct RopeArgs {
    const uint64_t *turns;
    int32_t rot, interleaved;
    float scale;
};

// sines and cosines of a row's pairs, times the factor; ends with a barrier
struct Turns {
    float c[512], s[512];
};
__device__ __forceinline__ void turns_of(const RopeArgs &r, int64_t pos, Turns &t) {
    for (int p = static_cast<int>(threadIdx.x); p < r.rot / 2; p += RP_THREADS) {
        const int64_t part = static_cast<int64_t>(r.turns[p] * static_cast<uint64_t>(pos));  // of 2^64, signed
        float s, c;
        sincospif(__ll2float_rn(part) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
        t.c[p] = c * r.scale;
        t.s[p] = s * r.scale;
    }
    __syncthreads();
}
// lane l's four pairs
struct Turn {
    float c[4], s[4];
};
__device__ __forceinline__ Turn turn_of(const Turns &t, int l) {
    const float4 c = reinterpret_cast<const float4 *>(t.c)[l], s = reinterpret_cast<const float4 *>(t.s)[l];
    return {{c.x, c.y, c.z, c.w}, {s.x, s.y, s.z, s.w}};
}

// where lane l's two groups of four elements stand in a head: the halves of its pairs, or 8 in a row
__device__ __forceinline__ int2 lane_at(const RopeArgs &r, int l) {
    return !r.interleaved && l < r.rot / 8 ? make_int2(4 * l, r.rot / 2 + 4 * l) : make_int2(8 * l, 8 * l + 4);
}

__device__ __forceinline__ void turn_pair(float &a, float &b, float c, float s) {
    const float x = a;
    a = fmaf(x, c, -__fmul_rn(b, s));
    b = fmaf(x, s, __fmul_rn(b, c));
}
__device__ __forceinline__ void turn_lane(float4 &x, float4 &y, const Turn &t, bool interleaved) {
    if (interleaved) {
        turn_pair(x.x, x.y, t.c[0], t.s[0]);
        turn_pair(x.z, x.w, t.c[1], t.s[1]);
        turn_pair(y.x, y.y, t.c[2], t.s[2]);
        turn_pair(y.z, y.w, t.c[3], t.s[3]);
    } else {
        turn_pair(x.x, y.x, t.c[0], t.s[0]);
        turn_pair(x.y, y.y, t.c[1], t.s[1]);
        turn_pair(x.z, y.z, t.c[2], t.s[2]);
        turn_pair(x.w, y.w, t.c[3], t.s[3]);
    }
}

// Rows: block (n, y) takes the y-th `per` heads of row n; the threads behind the last whole head of a block only help with
// the sines.
__global__ void __launch_bounds__(RP_THREADS) rope_rows_kernel(RopeArgs r, const float *x, int64_t xs, const int32_t *pos,
                                                               int32_t N, int32_t heads, int32_t LR, int32_t per,
                                                               float *out, int64_t os, int *status) {
    __shared__ __align__(16) Turns turns;
    pdl_wait();
    pdl_launch_dependents();
    const int slots = RP_THREADS / LR, slot = static_cast<int>(threadIdx.x) / LR, l = static_cast<int>(threadIdx.x) % LR;
    const int64_t n = blockIdx.x;
    const int h0 = static_cast<int>(blockIdx.y) * per + slot, h1 = min(heads, static_cast<int>(blockIdx.y + 1) * per);
    const int D = 8 * LR;
    const int2 at = lane_at(r, l);
    const bool work = slot < slots;
    float4 a[RP_HEADS], b[RP_HEADS];
#pragma unroll
    for (int j = 0; j < RP_HEADS; ++j) {
        const int hj = h0 + j * slots;
        if (work && hj < h1 && SD_INB(n < N && hj < heads && at.x + 4 <= D && at.y + 4 <= D, status, 119)) {  // site 119: row
            const float *p = x + n * xs + static_cast<int64_t>(hj) * D;
            a[j] = __ldcs(reinterpret_cast<const float4 *>(p + at.x));
            b[j] = __ldcs(reinterpret_cast<const float4 *>(p + at.y));
        }
    }
    turns_of(r, pos[n], turns);
    const bool on = l < r.rot / 8;
    Turn t = {};
    if (on) t = turn_of(turns, l);
#pragma unroll
    for (int j = 0; j < RP_HEADS; ++j) {
        const int hj = h0 + j * slots;
        if (work && hj < h1 && SD_INB(n < N && hj < heads && at.x + 4 <= D && at.y + 4 <= D, status, 119)) {
            if (on) turn_lane(a[j], b[j], t, r.interleaved != 0);
            float *p = out + n * os + static_cast<int64_t>(hj) * D;
            __stcs(reinterpret_cast<float4 *>(p + at.x), a[j]);
            __stcs(reinterpret_cast<float4 *>(p + at.y), b[j]);
        }
    }
}

struct AppendRopeArgs {
    PageView pv;
    void *k, *v;
    float *k_scale, *v_scale;
    const int32_t *table, *lens, *n_new, *parent;
    int32_t width, B, M, H, per;  // per: heads (of Q, K and V together) of a block's turn
    const float *q, *k_new, *v_new;
    float *q_out;
    int64_t q_sb, q_sm, o_sb, o_sm, sb, sm;
    RopeArgs r;
    int *status;
};

template <int T>
__device__ __forceinline__ uint2 pack4(float4 x) {
    uint2 w;
    if constexpr (T == SD_KV_BF16) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
        w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
        const __half2 a = __floats2half2_rn(x.x, x.y), b = __floats2half2_rn(x.z, x.w);
        w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
    return w;
}
// 4 codes of a row whose scale is d (0 codes where d is 0, NaN or infinite; inv: its rounded inverse), as sd_paged_append
// makes them: the nearest whole numbers to the rounded quotients x / d, halves away from 0.  x times inv is within
// 127 * 4 * 2^-24 < 2^-15 of that quotient and not above 127 + 2^-15, so the whole number is in the low bits of the product
// plus 1.5 * 2^23, and only where it is as near as 2^-10 to a half are the divisions themselves made.
__device__ __forceinline__ uint32_t codes4(float4 x, float d, float inv) {
    if (!(d > 0.0f && d < INFINITY)) return 0;
    const float f[4] = {x.x, x.y, x.z, x.w};
    uint32_t b[4];
    float off = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float q = __fmul_rn(f[i], inv), t = __fadd_rn(q, 12582912.0f);
        b[i] = __float_as_uint(t);
        off = fmaxf(off, fabsf(__fsub_rn(q, __fsub_rn(t, 12582912.0f))));
    }
    if (!(off < 0.4990234375f && d > 1e-37f)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int v = static_cast<int>(roundf(__fdiv_rn(f[i], d)));
            b[i] = static_cast<uint32_t>(v > 127 ? 127 : v < -127 ? -127 : v);
        }
    }
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t magnitude4(float4 x) {  // by its bits: an infinity above every number, a NaN above that
    return max(max(__float_as_uint(fabsf(x.x)), __float_as_uint(fabsf(x.y))),
               max(__float_as_uint(fabsf(x.z)), __float_as_uint(fabsf(x.w))));
}

// Block (y, z) takes the z-th `per` of the H + 2 H_kv heads [Q | K | V] of new row y.
template <int T, int D>
__global__ void __launch_bounds__(RP_THREADS) paged_append_rope_kernel(const AppendRopeArgs a) {
    constexpr int LR = D / 8, SLOTS = RP_THREADS / LR;
    __shared__ __align__(16) Turns turns;
    pdl_wait();
    pdl_launch_dependents();
    const int slot = static_cast<int>(threadIdx.x) / LR, l = static_cast<int>(threadIdx.x) % LR, lane = threadIdx.x & 31;
    const int HK = a.pv.H_kv, heads = a.H + 2 * HK;
    const int h0 = static_cast<int>(blockIdx.y) * a.per + slot, h1 = min(heads, static_cast<int>(blockIdx.y + 1) * a.per);
    const int b = static_cast<int>(blockIdx.x) / a.M, i = static_cast<int>(blockIdx.x) - b * a.M;
    const int n = a.n_new ? a.n_new[b] : a.M, len = a.lens[b];
    // a tree's parents, one a lane
    const int par = a.parent && lane < a.M ? a.parent[static_cast<int64_t>(b) * a.M + lane] : lane - 1;
    if (n < 0 || n > a.M || len < 0 || static_cast<int64_t>(len) + n > static_cast<int64_t>(a.width) * a.pv.P) {
        set_status(a.status, SD_EDEVICE);
        return;
    }
    if (i >= n) return;
    const int2 at = lane_at(a.r, l);
    float4 x[RP_HEADS], z[RP_HEADS];
#pragma unroll
    for (int j = 0; j < RP_HEADS; ++j) {
        const int hj = h0 + j * SLOTS;
        if (hj < h1 && SD_INB(b < a.B && i < a.M && hj < heads && at.y + 4 <= D, a.status, 120)) {  // site 120: new row
            const float *p = hj < a.H ? a.q + b * a.q_sb + i * a.q_sm + static_cast<int64_t>(hj) * D
                             : hj < a.H + HK ? a.k_new + b * a.sb + i * a.sm + static_cast<int64_t>(hj - a.H) * D
                                             : a.v_new + b * a.sb + i * a.sm + static_cast<int64_t>(hj - a.H - HK) * D;
            const int2 w = hj < a.H + HK ? at : make_int2(8 * l, 8 * l + 4);
            x[j] = __ldcs(reinterpret_cast<const float4 *>(p + w.x));
            z[j] = __ldcs(reinterpret_cast<const float4 *>(p + w.y));
        }
    }
    const int place = len + i, sl = place / a.pv.P, row = place - sl * a.pv.P;
    int page = -1;
    if (static_cast<int>(blockIdx.y + 1) * a.per > a.H) {  // the block has heads of K or V
        page = a.table[static_cast<int64_t>(b) * a.width + sl];
        if (page < 0 || page >= a.pv.n_pages) {
            set_status(a.status, SD_EDEVICE);
            page = -1;
        }
    }
    int depth = i;
    if (a.parent) {  // M <= 16
        int up = i;
        depth = 0;
        for (;; ++depth) {
            const int y = __shfl_sync(0xffffffffu, par, up);
            if (y >= up) set_status(a.status, SD_EDEVICE);  // parents come before their children
            if (y < 0 || y >= up) break;
            up = y;
        }
    }
    turns_of(a.r, static_cast<int64_t>(len) + depth, turns);
    const bool turned = l < a.r.rot / 8;
    Turn t = {};
    if (turned) t = turn_of(turns, l);
    const int64_t into = page * a.pv.ps + row * a.pv.rs;
#pragma unroll
    for (int j = 0; j < RP_HEADS; ++j) {
        const int hj = h0 + j * SLOTS;
        const bool isv = hj >= a.H + HK;
        if (hj >= h1) continue;
        if (turned && !isv) turn_lane(x[j], z[j], t, a.r.interleaved != 0);
        if (hj < a.H) {
            if (!SD_INB(b < a.B && i < n && at.y + 4 <= D, a.status, 121)) continue;  // site 121: turned query
            float *p = a.q_out + b * a.o_sb + i * a.o_sm + static_cast<int64_t>(hj) * D;
            *reinterpret_cast<float4 *>(p + at.x) = x[j];
            *reinterpret_cast<float4 *>(p + at.y) = z[j];
        } else if (page >= 0) {
            const int hk = hj - a.H - (isv ? HK : 0);
            if (!SD_INB(hk >= 0 && hk < HK && sl < a.width && row >= 0 && row < a.pv.P && page < a.pv.n_pages, a.status,
                        122))  // site 122: row in its page
                continue;
            const int64_t dst = into + hk * a.pv.hs;
            const int2 w = isv ? make_int2(8 * l, 8 * l + 4) : at;
            if constexpr (T == SD_KV_I8) {  // the largest magnitude of the row, over its lanes
                uint32_t top = max(magnitude4(x[j]), magnitude4(z[j]));
                const unsigned mask = LR == 32 ? 0xffffffffu : ((1u << (LR & 31)) - 1u) << (lane / LR * LR);
#pragma unroll
                for (int o = LR / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(mask, top, o));
                const float d = __fdiv_rn(__uint_as_float(top), 127.0f), inv = __frcp_rn(d);
                int8_t *to = static_cast<int8_t *>(isv ? a.v : a.k) + dst;
                *reinterpret_cast<uint32_t *>(to + w.x) = codes4(x[j], d, inv);
                *reinterpret_cast<uint32_t *>(to + w.y) = codes4(z[j], d, inv);
                if (l == 0) (isv ? a.v_scale : a.k_scale)[(static_cast<int64_t>(page) * HK + hk) * a.pv.P + row] = d;
            } else {
                uint16_t *to = static_cast<uint16_t *>(isv ? a.v : a.k) + dst;
                *reinterpret_cast<uint2 *>(to + w.x) = pack4<T>(x[j]);
                *reinterpret_cast<uint2 *>(to + w.y) = pack4<T>(z[j]);
            }
        }
    }
}

// Heads of a block's turn: all RP_HEADS of its lanes' where there are blocks enough for every SM all the same, one
// otherwise (the launch and the loads' latency are all there is).
// (A block per row and turn: a grid that stays, 16 blocks per SM, took 118 us for 16384 rows of 40 heads and 148 us for 8
// prompts of 2048 rows, this 97 and 131.)
static int heads_per_block(int64_t rows, int64_t heads, int slots) {
    const int64_t full = rows * ((heads + RP_HEADS * slots - 1) / (RP_HEADS * slots));
    return full >= 2 * num_sms() ? RP_HEADS * slots : slots;
}
static sd_status rope_check(const sd_rope *r, int D) {
    if (!r || !r->turns || !aligned(r->turns, 16)) return SD_EINVAL;
    if (r->rot < 2 || r->rot > D || (r->interleaved != 0 && r->interleaved != 1) || !isfinite(r->scale)) return SD_EINVAL;
    return r->rot % 8 ? SD_EUNSUPPORTED : SD_OK;
}

template <int T>
static cudaError_t append_rope_launch(int D, const AppendRopeArgs &a, dim3 grid, cudaStream_t s) {
    if (D == 64) return launch(paged_append_rope_kernel<T, 64>, grid, dim3(RP_THREADS), 0, s, a);
    if (D == 128) return launch(paged_append_rope_kernel<T, 128>, grid, dim3(RP_THREADS), 0, s, a);
    return launch(paged_append_rope_kernel<T, 256>, grid, dim3(RP_THREADS), 0, s, a);
}

}  // namespace sdv

using namespace sdv;

extern "C" {

sd_status sd_rope_freqs(int32_t rot, double base, int32_t scaling, double factor, double original, double low, double high,
                        double *inv_freq, float *scale) {
    const double tau = 6.283185307179586476925;
    if (!inv_freq || !scale || rot < 2 || rot % 2 || rot > (1 << 20) || !(base > 1.0) || !isfinite(base)) return SD_EINVAL;
    if (scaling < SD_ROPE_PLAIN || scaling > SD_ROPE_YARN) return SD_EUNSUPPORTED;
    if (scaling != SD_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return SD_EINVAL;
    if ((scaling == SD_ROPE_BANDS || scaling == SD_ROPE_YARN) &&
        (!(original > 0.0) || !isfinite(original) || !(low > 0.0) || !(high > low) || !isfinite(high)))
        return SD_EINVAL;
    if (scaling == SD_ROPE_NTK && rot > 2) base *= pow(factor, static_cast<double>(rot) / (rot - 2));
    *scale = scaling == SD_ROPE_YARN ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.0f;
    double first = 0.0, last = 0.0;
    if (scaling == SD_ROPE_YARN) {  // the pairs that make `high` and `low` turns within the trained length
        first = fmax(0.0, floor(rot * log(original / (high * tau)) / (2.0 * log(base))));
        last = fmin(rot - 1.0, ceil(rot * log(original / (low * tau)) / (2.0 * log(base))));
        last = fmax(last, first + 0.001);
    }
    for (int i = 0; i < rot / 2; ++i) {
        const double f = pow(base, -2.0 * i / rot);
        double keep = 1.0;  // the share of the unstretched frequency
        if (scaling == SD_ROPE_LINEAR) keep = 0.0;
        if (scaling == SD_ROPE_BANDS) keep = (original * f / tau - low) / (high - low);
        if (scaling == SD_ROPE_YARN) keep = 1.0 - (i - first) / (last - first);
        keep = fmin(1.0, fmax(0.0, keep));
        inv_freq[i] = keep == 1.0 ? f : f / factor * (1.0 - keep) + f * keep;
    }
    return SD_OK;
}

sd_status sd_rope_turns(const double *inv_freq, int32_t n, uint64_t *turns) {
    // 1 / 2 pi in two doubles
    const double hi = 0.15915494309189535, lo = -9.839338337591e-18;
    if (!inv_freq || !turns || n < 1) return SD_EINVAL;
    for (int32_t i = 0; i < n; ++i)
        if (!isfinite(inv_freq[i]) || fabs(inv_freq[i]) > 1048576.0) return SD_EINVAL;
    for (int32_t i = 0; i < n; ++i) {
        const double f = fabs(inv_freq[i]), t = f * hi, rest = fma(f, hi, -t) + f * lo;  // the product, and what it leaves
        const double part = t - floor(t);                                                // exact
        // the first as 2^64ths by its upper and lower half; the second is small
        const double up = floor(part * 4294967296.0), down = (part * 4294967296.0 - up) * 4294967296.0;
        const uint64_t whole = (static_cast<uint64_t>(up) << 32) + static_cast<uint64_t>(down);
        const uint64_t sum = whole + static_cast<uint64_t>(llrint((down - floor(down)) + rest * 18446744073709551616.0));
        turns[i] = inv_freq[i] < 0.0 ? 0 - sum : sum;
    }
    return SD_OK;
}

sd_status sd_rope_rows(const sd_rope *rope, const float *x, int64_t x_stride, const int32_t *pos, int32_t N, int32_t heads,
                       int32_t D, float *out, int64_t out_stride, sd_stream_t stream) {
    SD_NVTX("sd_rope_rows");
    if (!x || !pos || !out || N < 1 || heads < 1 || D < 8) return SD_EINVAL;
    if (D % 8 || D > 1024) return SD_EUNSUPPORTED;
    const sd_status st = rope_check(rope, D);
    if (st != SD_OK) return st;
    const int64_t line = static_cast<int64_t>(heads) * D;
    if ((N > 1 && (x_stride < line || out_stride < line)) || x_stride % 4 || out_stride % 4) return SD_EINVAL;
    if (!aligned(x, 16) || !aligned(out, 16)) return SD_EINVAL;
    if (x == out && N > 1 && x_stride != out_stride) return SD_EINVAL;  // (a row would go where another is still read)
    const int LR = D / 8, per = heads_per_block(N, heads, RP_THREADS / LR);
    const int64_t turns = (static_cast<int64_t>(heads) + per - 1) / per;
    if (turns > 65535) return SD_EUNSUPPORTED;
    int *status = status_ptr();
    if (!status) return SD_ECUDA;
    const RopeArgs r = {rope->turns, rope->rot, rope->interleaved, rope->scale};
    return launch(rope_rows_kernel, dim3(N, static_cast<unsigned>(turns)), dim3(RP_THREADS), 0,
                  reinterpret_cast<cudaStream_t>(stream), r, x, x_stride, pos, N, heads,
                  static_cast<int32_t>(LR), static_cast<int32_t>(per), out, out_stride, status) == cudaSuccess
               ? SD_OK
               : SD_ECUDA;
}

sd_status sd_paged_append_rope(const sd_kv_pages *pages, const int32_t *table, int32_t width, const int32_t *lens,
                               const int32_t *n_new, int32_t B, int32_t M, int32_t H, const float *q, int64_t q_seq_stride,
                               int64_t q_row_stride, const float *k_new, const float *v_new, int64_t seq_stride,
                               int64_t row_stride, const int32_t *parent, const sd_rope *rope, float *q_out,
                               int64_t out_seq_stride, int64_t out_row_stride, sd_stream_t stream) {
    SD_NVTX("sd_paged_append_rope");
    sd_status st = pages_check(pages);
    if (st != SD_OK) return st;
    if (!table || !lens || !k_new || !v_new || width < 1 || B < 1 || M < 1 || H < 0) return SD_EINVAL;
    if (B > PG_MAX_B || (parent && M > 16)) return SD_EUNSUPPORTED;
    st = rope_check(rope, pages->D);
    if (st != SD_OK) return st;
    const int64_t line = static_cast<int64_t>(pages->H_kv) * pages->D, qline = static_cast<int64_t>(H) * pages->D;
    if (seq_stride % 4 || row_stride % 4 || (M > 1 && row_stride < line) || (B > 1 && seq_stride < line)) return SD_EINVAL;
    if (!aligned(k_new, 16) || !aligned(v_new, 16)) return SD_EINVAL;
    if (H > 0) {
        if (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16)) return SD_EINVAL;
        if (q_seq_stride % 4 || q_row_stride % 4 || out_seq_stride % 4 || out_row_stride % 4) return SD_EINVAL;
        if (M > 1 && (q_row_stride < qline || out_row_stride < qline)) return SD_EINVAL;
        if (B > 1 && (q_seq_stride < qline || out_seq_stride < qline)) return SD_EINVAL;
    }
    if (static_cast<int64_t>(width) * pages->page_rows > INT32_MAX - 128) return SD_EUNSUPPORTED;
    if (H > 0 && q == q_out && ((M > 1 && q_row_stride != out_row_stride) || (B > 1 && q_seq_stride != out_seq_stride)))
        return SD_EINVAL;
    const int64_t rows = static_cast<int64_t>(B) * M, heads = static_cast<int64_t>(H) + 2 * static_cast<int64_t>(pages->H_kv);
    const int per = heads_per_block(rows, heads, RP_THREADS / (pages->D / 8));
    const int64_t turns = (heads + per - 1) / per;
    if (rows > INT32_MAX || turns > 65535) return SD_EUNSUPPORTED;
    int *status = status_ptr();
    if (!status) return SD_ECUDA;
    AppendRopeArgs a = {};
    a.pv = page_view(pages);
    a.k = pages->k;
    a.v = pages->v;
    a.k_scale = pages->k_scale;
    a.v_scale = pages->v_scale;
    a.table = table;
    a.lens = lens;
    a.n_new = n_new;
    a.parent = parent;
    a.width = width;
    a.B = B;
    a.M = M;
    a.H = H;
    a.per = per;
    a.q = q;
    a.k_new = k_new;
    a.v_new = v_new;
    a.q_out = q_out;
    a.q_sb = q_seq_stride;
    a.q_sm = q_row_stride;
    a.o_sb = out_seq_stride;
    a.o_sm = out_row_stride;
    a.sb = seq_stride;
    a.sm = row_stride;
    a.r = {rope->turns, rope->rot, rope->interleaved, rope->scale};
    a.status = status;
    const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>(turns));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = pages->type == SD_KV_F16    ? append_rope_launch<SD_KV_F16>(pages->D, a, grid, s)
                          : pages->type == SD_KV_BF16 ? append_rope_launch<SD_KV_BF16>(pages->D, a, grid, s)
                                                      : append_rope_launch<SD_KV_I8>(pages->D, a, grid, s);
    return e == cudaSuccess ? SD_OK : SD_ECUDA;
}

}  // extern "C"
