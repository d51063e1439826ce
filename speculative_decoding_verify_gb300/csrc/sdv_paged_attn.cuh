// sdv_paged_attn.cuh - what the two kernels of the attention over pages share: the arguments, the cut of the work into
// pieces, the producer warp and the join of partials.
#pragma once

#include "sdv_paged.cuh"

namespace sdv {

constexpr int PA_KT = 64;          // keys per tile
constexpr int PA_CW = 4;           // consumer warps, 16 keys of a tile each
constexpr int PA_THREADS = 32 * (PA_CW + 1);
constexpr float PA_NEG = -3.402823466e38f;  // running-max start: finite, below every score
constexpr float PA_PS = 16384.0f;  // fp16 weights are scaled by 2^14 (exact)
constexpr float PW_UNIT = 6.103515625e-05f;  // 2^-14: what the many-row kernel's weights and their sums are in
constexpr uint64_t PA_WAIT_NS = 2000000000ull;

// What a launch goes over: whole sequences (sd_paged_attn); or of a batch that shares prefixes (sd_paged_attn_shared) each
// sequence's rows behind its group's prefix, or the groups' prefixes, where a "sequence" is a group's shared rows and its
// new rows are those of all its members.  (The first is a mode of its own because the others' few instructions per piece
// cost it 4 %: 515 against 535 us, 16 sequences of 20000-60000 8-bit rows.)
enum PaMode { PA_ALL = 0, PA_OWN = 1, PA_PREFIX = 2 };

struct PagedArgs {
    const float *q;  // row i of sequence b at b * q_sb + i * q_sm, heads contiguous
    float *out;
    const int32_t *table, *lens, *n_new, *parent;
    const float *k_scale, *v_scale;  // 8-bit rows: [n_pages][H_kv][P]
    int64_t q_sb, q_sm, o_sb, o_sm;
    int32_t B, M, H, H_kv, g, P, n_pages, width, window, sinks;
    int32_t nst;          // ring stages
    float qscale;         // log2(e) / sqrt(D)
    // partials, two per CTA (of a run cut at the start of its share, and at the end), RPG query rows each (8 NT, or the
    // many-row kernel's 128 / C, whose 128-row partials keep the order of lanes, [D / 4][128] columns of four)
    float *part_o;        // [2 * grid][RPG][D]
    float2 *part_ml;      // [2 * grid][RPG]: maximum and sum
    int32_t *counters;    // [grid], zero between calls
    int32_t part_rows;    // rows of D floats that part_o holds (part_ml: as many pairs)
    int *status;
    // PA_PREFIX: lens, n_new hold the groups' shared rows and numbers of new rows, first[v] where group v's begin in
    // rows_of (sequence * M + row), leader[v] a sequence whose table names the group's pages; out [row of rows_of][H][D]
    const int32_t *first, *leader, *rows_of;
    // maximum and sum behind each row of out and head: PA_PREFIX [row of rows_of][H] (of runs inside one CTA; those that are
    // cut stay as partials), PA_OWN [B * M][H]
    float2 *row_ml;
    const int32_t *skip;          // PA_OWN: [B] tiles of a sequence's prefix
    int32_t *tickets;             // PA_OWN: [grid], 1 from the plan's end until the CTA takes it
    int32_t own_min, own_max;     // PA_OWN: the sequences of so many tiles behind their prefix
};

// query and output row of new row i of sequence (or group) b
template <int MODE>
__device__ __forceinline__ const float *q_row(const PagedArgs &a, int b, int i) {
    if constexpr (MODE == PA_PREFIX) {
        const int at = a.rows_of[a.first[b] + i], sb = at / a.M;
        return a.q + sb * a.q_sb + (at - sb * a.M) * a.q_sm;
    } else {
        return a.q + b * a.q_sb + i * a.q_sm;
    }
}
template <int MODE>
__device__ __forceinline__ float *out_row(const PagedArgs &a, int b, int i, int h, int D) {
    if constexpr (MODE == PA_PREFIX) return a.out + (static_cast<int64_t>(a.first[b] + i) * a.H + h) * D;
    else return a.out + b * a.o_sb + i * a.o_sm + static_cast<int64_t>(h) * D;
}
// the softmax statistics behind a finished row
template <int MODE>
__device__ __forceinline__ void put_ml(const PagedArgs &a, int b, int i, int h, float m, float l) {
    if constexpr (MODE == PA_PREFIX) a.row_ml[static_cast<int64_t>(a.first[b] + i) * a.H + h] = make_float2(m, l);
    if constexpr (MODE == PA_OWN) a.row_ml[(static_cast<int64_t>(b) * a.M + i) * a.H + h] = make_float2(m, l);
}

// PA_OWN, the kernel of few rows: it runs beside the prefixes' launch, for whose end griddepcontrol.wait would wait.  What
// it reads is the plan's, or older, and the plan has waited for all that is older: its last CTA releases a ticket per CTA
// behind its lists, and the exchange that takes it acquires all of that (the proxy fence: for the tensor copies too).  A CTA
// that finds none waits like any other.  The exchange leaves zero, so a ticket is never an earlier call's, replayed graphs
// included.  `word` is in shared memory.  All threads call it, and griddepcontrol.wait ahead of their end: what comes next
// finds the prefixes done as well.  (Waiting here instead: 106.5 -> 115 us for 4 x 16 + 8 sequences, 178 -> 180 for 64 x 5
// rows.)
__device__ __forceinline__ void after_plan(const PagedArgs &a, volatile int *word) {
    int32_t *ticket = a.tickets + blockIdx.x;
    if (threadIdx.x == 0) {
        int32_t got;
        asm volatile("atom.acquire.gpu.exch.b32 %0, [%1], %2;" : "=r"(got) : "l"(ticket), "r"(0) : "memory");
        *word = got;
    }
    __syncthreads();
    if (*word == 0) {
        pdl_wait();
        if (threadIdx.x == 0) *ticket = 0;
    }
    fence_proxy_async_global();
}

// the scales of 8-bit rows where there is no page
static __device__ __align__(16) float pa_zeros[PA_KT];

template <int T, int D>
struct PaLayout {
    static constexpr int ELT = T == SD_KV_I8 ? 1 : 2;
    static constexpr int ROWB = D * ELT < 128 ? D * ELT : 128;  // bytes of a row in one tensor tile
    static constexpr int NB = D * ELT / ROWB;                   // tensor tiles across a row
    static constexpr int TILE = PA_KT * ROWB;
    static constexpr int KV = NB * TILE;                        // K (or V) rows of a stage
    static constexpr int SCALES = T == SD_KV_I8 ? 1024 : 0;     // 64 + 64 row scales, padded to the swizzle's alignment
    static constexpr int STAGE = 2 * KV + SCALES;
    static constexpr int SW = ROWB / 16 - 1;                    // swizzle mask over the 16-byte chunks
    static constexpr int SSH = ROWB == 128 ? 0 : 1;             // 64-byte rows: two rows per 128-byte line
};

// byte offset inside a stage's K (or V) rows of the 16-byte chunk that holds bytes x .. of row r
template <int T, int D>
__device__ __forceinline__ uint32_t pa_off(int r, int x) {
    using L = PaLayout<T, D>;
    return static_cast<uint32_t>((x / L::ROWB) * L::TILE + r * L::ROWB +
                                 ((((x % L::ROWB) >> 4) ^ ((r >> L::SSH) & L::SW)) << 4));
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *tm, int x, int y, int z, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void pa_ldsm(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void pa_ldsm_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t pa_movm(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <int T>
__device__ __forceinline__ void pa_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (T == SD_KV_BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An fp32 pair as 16-bit parts that add up to it: two fp16 (each halves the rounding 2^-11 left by the part
// before: 2^-22 in all) or three bf16 (2^-8 each: 2^-24).
template <int T>
struct Parts {
    static constexpr int N = T == SD_KV_BF16 ? 3 : 2;
    uint32_t r[N];
};
template <int T>
__device__ __forceinline__ Parts<T> split2(float x0, float x1) {
    Parts<T> p;
#pragma unroll
    for (int i = 0; i < Parts<T>::N; ++i) {
        if constexpr (T == SD_KV_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
            const float2 f = __bfloat1622float2(h);
            p.r[i] = *reinterpret_cast<const uint32_t *>(&h);
            x0 -= f.x;
            x1 -= f.y;
        } else {
            const __half2 h = __floats2half2_rn(x0, x1);
            const float2 f = __half22float2(h);
            p.r[i] = *reinterpret_cast<const uint32_t *>(&h);
            x0 -= f.x;
            x1 -= f.y;
        }
    }
    return p;
}

// 8-bit rows: a power of two above a finite scale's magnitude (the least normal number where there is none), at most
// 2^126 so that its inverse is a normal number too: the unit in which weights times V scales are split
__device__ __forceinline__ uint32_t unit_above(uint32_t bits) { return min((bits & 0x7f800000u) + 0x00800000u, 0x7e800000u); }
__device__ __forceinline__ float unit_inverse(uint32_t unit) { return __uint_as_float(0x7f000000u - unit); }
__device__ __forceinline__ uint32_t scale_bits(float x) {  // (magnitudes order as their bits; 0: counts for nothing)
    return fabsf(x) < INFINITY ? __float_as_uint(fabsf(x)) : 0u;
}

// two of a word's four int8 codes (bytes picked by sel, as selector nibbles 0..3) as an exact fp16 pair:
// the code plus 128 in the mantissa of 1024, minus 1152
template <int B0, int B1>
__device__ __forceinline__ uint32_t codes2(uint32_t biased) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(biased), "r"(0x64646464u), "n"(B0 | (4 << 4) | (B1 << 8) | (4 << 12)));
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&r), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The tiles of one sequence: [0, n_sink) and from tile lo_tile on, T in all.
struct SeqTiles {
    int32_t n_sink, lo_tile, T;
};
__device__ __forceinline__ SeqTiles seq_tiles(int len, int n, int window, int sinks) {
    SeqTiles s;
    const int total = len + n;
    int lo = 0;
    if (window > 0 && len - window + 1 > 0) lo = len - window + 1;  // the first row (depth 0) reaches furthest back
    s.lo_tile = lo / PA_KT;
    const int st = window > 0 ? min((min(sinks, lo) + PA_KT - 1) / PA_KT, s.lo_tile) : 0;
    s.n_sink = st;
    s.T = st + (total + PA_KT - 1) / PA_KT - s.lo_tile;
    return s;
}

// the tiles of a launch's sequence (or group); skip: of its shared prefix (full context alone has one)
template <int MODE>
__device__ __forceinline__ SeqTiles tiles_of(const PagedArgs &a, int len, int n, int skip) {
    if constexpr (MODE == PA_PREFIX) return {0, 0, len / PA_KT};  // whole tiles
    SeqTiles s = seq_tiles(len, n, a.window, a.sinks);
    if constexpr (MODE == PA_OWN) {
        s.lo_tile += skip;
        s.T -= skip;
    }
    return s;
}

// new rows that position i of a sequence sees: its path, cut by the window (the path's k-th node stands at depth k)
__device__ __forceinline__ uint32_t new_rows_seen(const PagedArgs &a, int b, int i, int len, int &depth) {
    uint32_t path = 0;
    if (!a.parent) {
        path = (2u << i) - 1u;
    } else {
        int x = i;
        for (int step = 0; step <= i && x >= 0; ++step) {
            path |= 1u << x;
            const int p = a.parent[static_cast<int64_t>(b) * a.M + x];
            if (p >= x) {  // parents come before their children; anything else is a bad tree
                set_status(a.status, SD_EDEVICE);
                break;
            }
            x = p;
        }
    }
    depth = __popc(path) - 1;
    if (a.window > 0) {
        uint32_t keep = 0, left = path;
        for (int k = 0; left; ++k) {
            const uint32_t bit = left & (0u - left);
            left ^= bit;
            if (k > depth - a.window || len + k < a.sinks) keep |= bit;
        }
        path = keep;
    }
    return path;
}

// One piece of a CTA's share: tiles [t0, t1) of the run of (b, kh, rg).
struct Piece {
    int32_t b, kh, rg, t0, t1, len, n;
    SeqTiles st;
    int64_t run0;  // the run's first tile in the whole line
    int64_t next;  // PA_OWN: where the CTA's next piece begins
};
// PA_OWN: what a run costs beside its tiles, in tiles.  The line has as many places ahead of the run's own, so that a CTA
// gets fewer short runs than long ones' tiles.
constexpr int PA_RUN = 3;
// and the tiles up to which it is one CTA's: a short run that is cut costs its CTAs a partial, a fence and a join each
constexpr int PA_WHOLE = 12;

struct Sched {
    const int64_t *prefix;  // [B + 1]: tiles of the sequences before
    const int2 *ln;         // [B]: (len, n_new; PA_OWN: n_new + 32 * skipped tiles), n_new 0 where nothing is to be done
    int64_t u0, u1, W;
    int32_t G;              // CTAs that share the line
};

template <int RPG, int MODE>
__device__ __forceinline__ Piece piece_at(const PagedArgs &a, const Sched &s, int64_t u, int b) {
    Piece p;
    while (s.prefix[b + 1] <= u) ++b;
    p.b = b;
    const int2 ln = s.ln[b];
    p.len = ln.x;
    p.n = MODE == PA_OWN ? ln.y & 31 : ln.y;
    p.st = tiles_of<MODE>(a, p.len, p.n, MODE == PA_OWN ? ln.y >> 5 : 0);
    const int64_t rem = u - s.prefix[b];
    const int RG = (p.n * a.g + RPG - 1) / RPG;
    if constexpr (MODE == PA_OWN) {
        const int all = p.st.T + PA_RUN;
        const int64_t run = rem / all;
        const int at = static_cast<int>(rem - run * all);
        p.run0 = u - at + PA_RUN;
        p.kh = static_cast<int32_t>(run / RG);
        p.rg = static_cast<int32_t>(run - static_cast<int64_t>(p.kh) * RG);
        p.next = min(s.u1, u - at + all);
        p.t0 = max(0, at - PA_RUN);
        p.t1 = static_cast<int32_t>(p.next - (u - at)) - PA_RUN;  // (no tiles where it is not above t0)
    } else {
        const int64_t run = rem / p.st.T;
        p.t0 = static_cast<int32_t>(rem - run * p.st.T);
        p.run0 = u - p.t0;
        p.kh = static_cast<int32_t>(run / RG);
        p.rg = static_cast<int32_t>(run - static_cast<int64_t>(p.kh) * RG);
        const int64_t left = s.u1 - u;
        p.t1 = left < p.st.T - p.t0 ? p.t0 + static_cast<int32_t>(left) : p.st.T;
    }
    return p;
}
// the place behind a piece
template <int MODE>
__device__ __forceinline__ int64_t behind(const Piece &p, int64_t u) {
    return MODE == PA_OWN ? p.next : u + (p.t1 - p.t0);
}
__device__ __forceinline__ int cta_of(const Sched &s, int64_t u) { return static_cast<int>(((u + 1) * s.G - 1) / s.W); }

// The whole line of tiles and this CTA's share of it; false: the CTA has none.  All NTHR threads call it.
template <int RPG, int NTHR, int MODE>
__device__ bool make_sched(const PagedArgs &a, int64_t *prefix, int2 *ln, Sched &sc) {
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    for (int b = tid; b < a.B; b += NTHR) {
        int len = a.lens[b], n = a.n_new ? a.n_new[b] : a.M;
        if constexpr (MODE != PA_PREFIX) {  // (the groups are made of sequences that pass this)
            if (len < 0 || n < 0 || n > a.M || static_cast<int64_t>(len) + n > static_cast<int64_t>(a.width) * a.P) {
                set_status(a.status, SD_EDEVICE);
                n = 0;
            }
        }
        const int skip = MODE == PA_OWN && n > 0 ? a.skip[b] : 0;
        int64_t cost = 0;
        if (n > 0) {
            const int tiles = tiles_of<MODE>(a, len, n, skip).T;
            if (MODE == PA_OWN && (tiles < a.own_min || tiles > a.own_max)) n = 0;
            else cost = static_cast<int64_t>(tiles + (MODE == PA_OWN ? PA_RUN : 0)) * ((n * a.g + RPG - 1) / RPG) * a.H_kv;
        }
        ln[b] = make_int2(len, n + 32 * skip);
        prefix[b + 1] = cost;
    }
    if (tid == 0) prefix[0] = 0;
    __syncthreads();
    if (warp == 0) {  // the tiles' running sum
        int64_t run = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + lane;
            int64_t v = b < a.B ? prefix[b + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += y;
            }
            if (b < a.B) prefix[b + 1] = run + v;
            run += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    __syncthreads();
    sc.prefix = prefix;
    sc.ln = ln;
    sc.W = prefix[a.B];
    sc.G = static_cast<int32_t>(min(static_cast<int64_t>(gridDim.x), sc.W));
    if (static_cast<int64_t>(blockIdx.x) >= sc.W) return false;
    sc.u0 = static_cast<int64_t>(blockIdx.x) * sc.W / sc.G;
    sc.u1 = static_cast<int64_t>(blockIdx.x + 1) * sc.W / sc.G;
    if constexpr (MODE == PA_OWN) {
        // an end inside a short run moves to its start, which leaves the ends inside the others, and so cta_of there, as they
        // are
        auto whole = [&](int64_t u) {
            if (u >= sc.W) return u;
            int lo = 0, hi = a.B - 1;
            while (lo < hi) {  // the sequence of u
                const int mid = (lo + hi) / 2;
                if (prefix[mid + 1] <= u) lo = mid + 1;
                else hi = mid;
            }
            const int T = tiles_of<MODE>(a, ln[lo].x, ln[lo].y & 31, ln[lo].y >> 5).T;
            return T <= PA_WHOLE ? u - (u - prefix[lo]) % (T + PA_RUN) : u;
        };
        sc.u0 = whole(sc.u0);
        sc.u1 = whole(sc.u1);
        return sc.u0 < sc.u1;
    }
    return true;
}

// The producer warp's loop: the tiles of the CTA's pieces into the ring's stages, running ahead of whoever empties
// them.  QS > 0: each piece's query rows come first, in QS stages of QR rows, each row D floats and 16 bytes apart (so
// that threads of consecutive rows read them without bank conflicts).
template <int T, int D, int RPG, int QS, int QR, int MODE>
__device__ void produce_tiles(const PagedArgs &a, const Sched &sc, const CUtensorMap *tmk, const CUtensorMap *tmv,
                              uint8_t *ring, int nst, uint64_t *full, uint64_t *empty, volatile int *abort) {
    using LY = PaLayout<T, D>;
    const int lane = static_cast<int>(threadIdx.x) & 31;
    // lane l issues copies l, l + 32, .. of a tile (page, K or V, 128 bytes of row)
    const int rows = min(a.P, PA_KT), npt = PA_KT / rows;  // rows of a page in a tile, pages per tile
    const int lg = __ffs(npt) - 1;
    const int ncopy = npt * 2 * LY::NB;
    int64_t u = sc.u0;
    int b = 0, slot = 0, issued = 0;
    uint32_t ph = 0;
    bool ok = true;
    // the next stage, free; false: given up
    auto take = [&]() {
        if (issued >= nst && !mbar_wait_bounded(&empty[slot], ph ^ 1u, PA_WAIT_NS, abort)) {
            set_status(a.status, SD_ETIMEOUT);
            *abort = 1;
        }
        return __all_sync(0xffffffffu, *abort == 0) != 0;
    };
    auto taken = [&]() {
        ++issued;
        if (++slot == nst) {
            slot = 0;
            ph ^= 1u;
        }
    };
    while (ok && u < sc.u1) {
        const Piece p = piece_at<RPG, MODE>(a, sc, u, b);
        b = p.b;
        if (MODE == PA_OWN && p.t1 <= p.t0) {
            u = p.next;
            continue;
        }
        for (int s = 0; ok && s < QS; ++s) {
            ok = take();
            if (!ok) break;
            // rows of this stage
            const int r0 = s * QR, n = max(0, min(min(QR, RPG - r0), p.n * a.g - p.rg * RPG - r0));
            if (lane == 0) {
                if (n) mbar_arrive_expect_tx(&full[slot], static_cast<uint32_t>(n) * D * 4);
                else mbar_arrive(&full[slot]);
            }
            __syncwarp();
            for (int i = lane; i < n; i += 32) {
                const int tg = p.rg * RPG + r0 + i;
                if (!SD_INB(p.b >= 0 && p.b < a.B && tg >= 0 && tg / a.g < (MODE == PA_PREFIX ? p.n : a.M) && p.kh >= 0 &&
                                p.kh < a.H_kv && slot < nst,
                            a.status, 113))  // site 113: query row
                    continue;
                bulk_g2s_l2keep(ring + static_cast<size_t>(slot) * LY::STAGE + i * (D * 4 + 16),
                                q_row<MODE>(a, p.b, tg / a.g) + static_cast<int64_t>(p.kh * a.g + tg % a.g) * D,
                                D * 4, &full[slot]);
            }
            taken();
        }
        if (!ok) break;
        const int32_t *tab = a.table + static_cast<int64_t>(MODE == PA_PREFIX ? a.leader[b] : b) * a.width;
        const int total = MODE == PA_PREFIX ? p.len : p.len + p.n;
        const int lo = a.window > 0 ? max(0, p.len - a.window + 1) : 0, sink = a.window > 0 ? a.sinks : 0;
        // the pages of the piece's places in order, npt to a tile, 32 at a time and 32 more on their way: a table entry
        // fetched per tile would cost the tile its latency.  (A place without rows, or an entry that is no page, reads
        // as zeros.)
        auto page_of = [&](int e) {
            const int t = p.t0 + (e >> lg);
            if (t >= p.t1) return a.n_pages;
            const int key = (t < p.st.n_sink ? t : t - p.st.n_sink + p.st.lo_tile) * PA_KT + (e & (npt - 1)) * rows;
            if (key >= total) return a.n_pages;
            if (!SD_INB(key >= 0 && key / a.P < a.width && b < a.B, a.status, 114)) return a.n_pages;  // site 114: table entry
            const int pg = tab[key / a.P];
            if (pg >= 0 && pg < a.n_pages) return pg;
            if (key + rows > lo || key < sink) set_status(a.status, SD_EDEVICE);  // a row of it is visible
            return a.n_pages;
        };
        int pages = page_of(lane), later = page_of(32 + lane);
        for (int t = p.t0; t < p.t1; ++t) {
            const int e = (t - p.t0) << lg;
            if (e && (e & 31) == 0) {
                pages = later;
                later = page_of(e + 32 + lane);
            }
            const int pg = __shfl_sync(0xffffffffu, pages, (e & 31) + (lane & (npt - 1)));
            const int key0 = (t < p.st.n_sink ? t : t - p.st.n_sink + p.st.lo_tile) * PA_KT;
            ok = take();
            if (!ok) break;
            uint8_t *stp = ring + static_cast<size_t>(slot) * LY::STAGE;
            if (lane == 0)
                mbar_arrive_expect_tx(&full[slot], 2 * LY::KV + (T == SD_KV_I8 ? 2 * PA_KT * 4 : 0));
            __syncwarp();
            for (int i = lane; i < ncopy; i += 32) {
                // page place i % npt: this lane's own (npt divides 32)
                const int place = i % npt, half = (i / npt) % LY::NB, kv = i / npt / LY::NB;
                const uint32_t dst = smem_u32(stp) + kv * LY::KV + half * LY::TILE + place * rows * LY::ROWB;
                if (!SD_INB(slot < nst && key0 >= 0 && key0 % a.P + rows <= a.P && p.kh >= 0 && p.kh < a.H_kv && pg >= 0 &&
                                pg <= a.n_pages && kv < 2 && (place + 1) * rows <= PA_KT,
                            a.status, 115))  // site 115: a page's rows (and its scales)
                    continue;
                tma_4d(dst, kv ? tmv : tmk, half * (LY::ROWB / LY::ELT), key0 % a.P, p.kh, pg, &full[slot]);
            }
            if constexpr (T == SD_KV_I8) {
                if (lane < 2 * npt) {
                    const int place = lane % npt, kv = lane / npt;
                    const float *src = pg >= a.n_pages ? pa_zeros
                                                       : (kv ? a.v_scale : a.k_scale) +
                                                             (static_cast<int64_t>(pg) * a.H_kv + p.kh) * a.P + key0 % a.P;
                    bulk_g2s_l2keep(stp + 2 * LY::KV + kv * PA_KT * 4 + place * rows * 4, src, rows * 4, &full[slot]);
                }
            }
            taken();
        }
        u = behind<MODE>(p, u);
    }
    if (!ok && lane == 0) {  // never leave with copies in flight
        for (int i = max(0, issued - nst); i < issued; ++i)
            mbar_wait_bounded(&full[i % nst], (i / nst) & 1u, PA_WAIT_NS);
    }
    __syncwarp();
}

// The partials of one run's CTAs c0 .. c1, joined in the order of their keys by the NTHR threads that call it (named
// barrier `bar` among them; l_unit: what their sums are in).  A warp reads whole rows (a row of D = 64 half a warp), JC
// CTAs at a time: the weights of all rows come first, through shared memory (RPG * (JC + 2) floats), then every load of a
// pass is in flight at once.
constexpr int JC = 8;
template <int RPG, int D, int NTHR, int MODE>
__device__ void join_partials(const PagedArgs &a, const Piece &p, int c0, int c1, int tid, float *sm, int bar,
                              float l_unit = 1.0f) {
    constexpr int LR = D / 4 < 32 ? D / 4 : 32, NV = D / 4 / LR;  // lanes of a row, 16-byte columns per lane
    constexpr int RT = NTHR / LR, NR = (RPG + RT - 1) / RT;       // rows at a time, rows per thread
    constexpr int XU = 16 / (NR * NV) > 0 ? (16 / (NR * NV) < JC ? 16 / (NR * NV) : JC) : 1;
    const int rows = min(RPG, p.n * a.g - p.rg * RPG);
    float *mx_of = sm, *sum_of = sm + RPG, *weight = sm + 2 * RPG;  // weight [JC][RPG]
    __threadfence();
    auto ml_of = [&](int x, int tr) { return __ldcg(&a.part_ml[static_cast<int64_t>(2 * x + (x == c0)) * RPG + tr]); };
    if (tid < rows) {
        float mx = PA_NEG, lv = 0.0f;
#pragma unroll 8
        for (int x = c0; x <= c1; ++x) {
            const float2 ml = ml_of(x, tid);
            const float n = fmaxf(mx, ml.x);
            lv = fmaf(lv, exp2f(mx - n), ml.y * exp2f(ml.x - n));
            mx = n;
        }
        mx_of[tid] = mx;
        sum_of[tid] = lv == 0.0f ? 0.0f : 1.0f / lv;
        if constexpr (MODE == PA_OWN) {
            const int tg = p.rg * RPG + tid;
            put_ml<MODE>(a, p.b, tg / a.g, p.kh * a.g + tg % a.g, mx, lv * l_unit);
        }
    }
    const int r0 = tid / LR, col = tid % LR;
    float4 v[NR][NV];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int k = 0; k < NV; ++k) v[i][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (!SD_INB(c0 >= 0 && c0 < c1 && c1 < static_cast<int>(gridDim.x) && (2 * c1 + 2) * RPG <= a.part_rows && rows <= RPG &&
                    (p.rg * RPG + rows - 1) / a.g < a.M,
                a.status, 116))  // site 116: partials of a join, its output rows
        c1 = c0 - 1;
    for (int x0 = c0; x0 <= c1; x0 += JC) {
        const int nx = min(JC, c1 - x0 + 1);
        named_bar_sync(bar, NTHR);
        for (int i = tid; i < nx * rows; i += NTHR) {
            const int x = i / rows, tr = i - x * rows;
            weight[x * RPG + tr] = exp2f(ml_of(x0 + x, tr).x - mx_of[tr]);
        }
        named_bar_sync(bar, NTHR);
        for (int xs = 0; xs < nx; xs += XU) {
            float4 y[XU][NR][NV];
            float f[XU][NR];
#pragma unroll
            for (int x = 0; x < XU; ++x)
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const int tr = r0 + i * RT, xc = x0 + xs + x;
                    const bool on = xs + x < nx && tr < rows;
                    f[x][i] = on ? weight[(xs + x) * RPG + tr] : 0.0f;
                    const float4 *from =
                        reinterpret_cast<const float4 *>(
                            a.part_o + (static_cast<int64_t>(2 * xc + (xc == c0)) * RPG + tr) * D) +
                        col;
#pragma unroll
                    for (int k = 0; k < NV; ++k)
                        y[x][i][k] = on ? __ldcg(from + k * LR) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
#pragma unroll
            for (int x = 0; x < XU; ++x)
#pragma unroll
                for (int i = 0; i < NR; ++i)
#pragma unroll
                    for (int k = 0; k < NV; ++k) {
                        v[i][k].x = fmaf(y[x][i][k].x, f[x][i], v[i][k].x);
                        v[i][k].y = fmaf(y[x][i][k].y, f[x][i], v[i][k].y);
                        v[i][k].z = fmaf(y[x][i][k].z, f[x][i], v[i][k].z);
                        v[i][k].w = fmaf(y[x][i][k].w, f[x][i], v[i][k].w);
                    }
        }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int tr = r0 + i * RT, tg = p.rg * RPG + tr;
        if (tr < rows) {
            const float inv = sum_of[tr];
            float4 *to = reinterpret_cast<float4 *>(out_row<MODE>(a, p.b, tg / a.g, p.kh * a.g + tg % a.g, D)) + col;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                to[k * LR] = make_float4(v[i][k].x * inv, v[i][k].y * inv, v[i][k].z * inv, v[i][k].w * inv);
        }
    }
    named_bar_sync(bar, NTHR);
}

// A checked call of the attention over pages (sdv_paged_attn.cu): what its launches share.
struct PaCall {
    PagedArgs a;
    CUtensorMap tmk, tmv;
    int32_t type, D;
};
size_t pa_workspace(int D, size_t *off_ml, size_t *off_o);
size_t pa_counters();  // bytes of a counter for each CTA of the largest grid (at the workspace's start)
sd_status pa_call(const sd_kv_pages *pages, const int32_t *table, int32_t width, const int32_t *lens, const int32_t *n_new,
                  int32_t B, int32_t M, int32_t H, const float *q, int64_t q_seq_stride, int64_t q_row_stride,
                  const int32_t *parent, int32_t window, int32_t sinks, float *out, int64_t out_seq_stride,
                  int64_t out_row_stride, void *workspace, size_t ws_bytes, PaCall &c);
// the new rows of the sequences of c.a (PA_ALL or PA_OWN)
sd_status pa_rows(const PaCall &c, PaMode mode, cudaStream_t s);
// CTAs of its first launch (PA_OWN): at most pa_counters() / 4
int pa_own_grid(const PaCall &c);
// the prefixes of the groups of c.a (at most PG_MAX_B / 2), of at most `rows` query rows per KV head each, and how their
// partials are left: rows of one, the CTAs that share the line of tiles, and what the sums and outputs are in
struct PrefixLayout {
    int32_t rp, grid;
    float unit;
};
PrefixLayout pa_prefix_layout(const PaCall &c, int rows);
sd_status pa_prefix(const PaCall &c, int rows, cudaStream_t s);

// The many-row kernel (sdv_paged_wide.cuh): D = 64 or 128, `rows` the most query rows of a KV head, one CTA per SM.
cudaError_t paged_wide_f16(const PagedArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, int D, int rows,
                           int grid, cudaStream_t s);
cudaError_t paged_wide_bf16(const PagedArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, int D, int rows,
                            int grid, cudaStream_t s);
cudaError_t paged_wide_i8(const PagedArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, int D, int rows, int grid,
                          cudaStream_t s);
// the same in the modes of shared prefixes
cudaError_t paged_shared_f16(PaMode mode, const PagedArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, int D, int rows,
                             int grid, cudaStream_t s);
cudaError_t paged_shared_bf16(PaMode mode, const PagedArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, int D, int rows,
                              int grid, cudaStream_t s);
cudaError_t paged_shared_i8(PaMode mode, const PagedArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, int D, int rows,
                            int grid, cudaStream_t s);

}  // namespace sdv
