// sdv_paged_wide.cuh - the attention over pages for many query rows per KV head (a tree of drafts, grouped
// heads): the same work, cut, masks and partials as paged_attn_kernel, on the 5th-generation tensor cores.
//
// The rows of one (sequence, KV head) are the 128 lanes of tensor memory.  With at most 64 (32) of them the lanes hold
// C = 2 (4) groups of the same rows, which hold different 16-bit parts of the weights (one pass of the product instead
// of two or three) or weigh different keys of a tile; the lane groups join at the end of a piece as the splits of a run
// do.
//   S = Q K^T: tcgen05.mma kind::f16, M = 128, N = 64, Q in tensor memory as A (written once per piece, in 16-bit parts
//     that add up to the fp32 value: two fp16, or three bf16), K as B from shared memory as the tensor copy left it
//     (K-major, 128-byte swizzle);
//   softmax: two threads per lane, half of the lane's keys each, their maximum shared through shared memory; the
//     weights go back to tensor memory over the scores, in parts;
//   O_t = P V: the weights as A, V as B (MN-major, the same swizzle), from zero for each tile; the softmax threads add
//     half of the columns each to their fp32 outputs in registers with the rescale of the running maximum (a
//     tensor-core accumulator kept over the tiles would truncate at every step, and rescaling it would cost the same
//     loads and more stores).
// One thread issues all MMAs: scores two tiles ahead of the weights, so the tensor cores work while the softmax
// runs.  Measured on the way (16 sequences of 8000 rows, 8 KV heads, 128 query rows, fp16): one softmax group of four
// warps 215 us, two that take the tiles in turn 149 us (each waits for its own product: the chain scores - softmax -
// product is longer than two tiles).  8-bit rows pass through four more warps that write them as fp16 into operand
// buffers (exact) and their scales beside them.
//
// What bounds it: at 128 rows of D = 128 a 64-key fp16 tile is 32 KB of HBM (about 1400 SM cycles of one SM's share)
// against 4 x 128 x 64 x 128 multiply-adds (about 1050 cycles) and 64 weights a thread.
#pragma once

#include "sdv_paged_attn.cuh"

namespace sdv {

constexpr int PW_NG = 2;       // softmax groups of four warps (the lane quarters of tensor memory)
constexpr int PW_SOFT = 128 * PW_NG;
constexpr float PW_UP = 14.0f; // weights are in units of 2^-14 throughout (their sum too): fp16 parts stay normal

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
                 : "memory");
}
// one thread of a converged warp.  MMAs issued under `lane == 0` instead cost 116 cycles each (the compiler does
// not know that one thread runs and serialises over the lanes), under this 44 at N = 64 and 76 at N = 128.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred q;\nelect.sync _|q, 0xffffffff;\nselp.u32 %0, 1, 0, q;\n}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define PW_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), \
                    "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
#define PW_I8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), \
                    "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])
#define PW_W8(r, o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), \
                    "+r"(r[o + 4]), "+r"(r[o + 5]), "+r"(r[o + 6]), "+r"(r[o + 7])

// N consecutive columns of this warp's lanes; the values are there after tc_wait_ld on the same registers
__device__ __forceinline__ void tc_ld(uint32_t (&r)[16], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : PW_R8(r, 0), PW_R8(r, 8)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : PW_W8(r, 0), PW_W8(r, 8)::"memory");
}
__device__ __forceinline__ void tc_ld(uint32_t (&r)[32], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
                 "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : PW_R8(r, 0), PW_R8(r, 8), PW_R8(r, 16), PW_R8(r, 24)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : PW_W8(r, 0), PW_W8(r, 8), PW_W8(r, 16), PW_W8(r, 24)::"memory");
}
__device__ __forceinline__ void tc_st(const uint32_t (&r)[8], uint32_t addr) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), PW_I8(r, 0) : "memory");
}
__device__ __forceinline__ void tc_st(const uint32_t (&r)[16], uint32_t addr) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
                 PW_I8(r, 0), PW_I8(r, 8)
                 : "memory");
}
__device__ __forceinline__ float ex2(float x) {  // 2^x to about 2^-22, 0 below the normal numbers
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// one 16-bit part of a pair, and what it leaves over
template <int T>
__device__ __forceinline__ uint32_t part_bits(float2 x) {
    if constexpr (T == SD_KV_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(x.x, x.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
template <int T>
__device__ __forceinline__ float2 part_left(float2 x, uint32_t bits) {
    const float2 f = T == SD_KV_BF16 ? make_float2(__uint_as_float(bits << 16), __uint_as_float(bits & 0xffff0000u))
                                     : __half22float2(*reinterpret_cast<const __half2 *>(&bits));
    return ffma2_rn(f, make_float2(-1.0f, -1.0f), x);
}

// a pair of weights in all its parts, as split2 (the differences are exact)
template <int T>
__device__ __forceinline__ Parts<T> split_pair(float2 x) {
    Parts<T> p;
#pragma unroll
    for (int i = 0; i < Parts<T>::N; ++i) {
        p.r[i] = part_bits<T>(x);
        if (i + 1 < Parts<T>::N) x = part_left<T>(x, p.r[i]);
    }
    return p;
}

// shared-memory operand with the 128-byte swizzle: 8-row groups of 1024 bytes; lbo is the step between 64-element
// blocks along N of an MN-major operand (unused for K-major)
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr, uint32_t lbo) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | static_cast<uint64_t>((lbo >> 4) & 0x3FFF) << 16 |
           static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}

template <int T, int D, int C>
struct WideLayout {
    static constexpr bool I8 = T == SD_KV_I8;
    static constexpr int NP = Parts<T>::N;
    static constexpr int RP = 128 / C;              // rows of a group
    // of the C lane groups, CP hold different parts of the same weights and C / CP different keys
    static constexpr int CP = C == 4 && NP == 2 ? 2 : C;
    static constexpr int KL = PA_KT * CP / C;       // keys of a tile that a lane weighs
    static constexpr int NC = KL / PW_NG;           // of these, a thread
    static constexpr int DO = D / PW_NG;            // output columns of a thread
    static constexpr int NR = (NP + CP - 1) / CP;   // parts that a lane holds: passes of the product
    static constexpr int OTILE = PA_KT * 128;       // 64 keys x 64 halves
    static constexpr int OKV = D / 64 * OTILE;      // K (or V) operand of a tile
    // scales of K [64], of V [64] in the tile's unit, that unit
    static constexpr int OSCALES = I8 ? 1024 : 0;
    static constexpr int OSTAGE = 2 * OKV + OSCALES;
    // operand stages (8-bit rows: written by the converting warps)
    static constexpr int NOP = I8 ? (D == 64 ? 4 : 3) : (D == 64 ? 8 : 6);
    static constexpr int NRAW = I8 ? (D == 64 ? 8 : 5) : 0;                 // 8-bit stages as copied
    // the query rows of a piece take stages of the copies' ring before its tiles
    static constexpr int QROW = D * 4 + 16;
    static constexpr int QR = PaLayout<T, D>::STAGE / QROW < RP ? PaLayout<T, D>::STAGE / QROW : RP, QS = (RP + QR - 1) / QR;
    static_assert(QS < (I8 ? NRAW : NOP), "a piece's queries fit in the ring");
    static constexpr int THREADS = PW_SOFT + 128 + (I8 ? 128 : 0);
    // producer, MMAs, scales and first converting warp (8-bit rows)
    static constexpr int WARP_P = 4 * PW_NG, WARP_M = WARP_P + 1, WARP_S = WARP_P + 2, WARP_C = WARP_P + 4;
    // tensor memory columns
    static constexpr int TQ = 0, QCOLS = NP * D / 2;
    static constexpr int SCOLS = NR == 3 ? 96 : 64;  // scores (64), then the weights' parts over them (32 each)
    static constexpr int TS = QCOLS;
    static constexpr int NPV = QCOLS + 2 * SCOLS + 2 * D <= 512 ? 2 : 1;  // product buffers
    static constexpr int TO = TS + 2 * SCOLS;
    static_assert(TO + NPV * D <= 512, "tensor memory");
    // shared memory after the rings: 16 columns of every softmax thread's outputs, the threads' maxima (two turns) and
    // sums
    static constexpr int SCRATCH = PW_SOFT * 20 * 4 + 3 * PW_SOFT * 4;
    static constexpr int NBAR = 2 * NOP + 2 * NRAW + 8 + 3;
    static constexpr size_t fixed() {
        return 1024 + static_cast<size_t>(NOP) * OSTAGE +
               static_cast<size_t>(NRAW) * PaLayout<T, D>::STAGE + SCRATCH + NBAR * 8 + 64;
    }
    // registers per thread as launched, then of the softmax, of producer and MMA, of the converting warps
    static constexpr int REG_L = I8 ? 128 : 168, REG_S = I8 ? 192 : 224, REG_P = I8 ? 64 : 56, REG_C = 64;
    static_assert(PW_SOFT * REG_S + 128 * REG_P + (I8 ? 128 * REG_C : 0) <= THREADS * REG_L, "registers");
};

// bits e < 32 of the keys key0 + e in [lo, hi)
__device__ __forceinline__ uint32_t key_range(int key0, int lo, int hi) {
    const int l = min(max(lo - key0, 0), 32), h = min(max(hi - key0, 0), 32);
    return h <= l ? 0u : (0xffffffffu >> (32 - (h - l))) << l;
}
// bits e < 32: whether a row sees key key0 + e.  low: the first committed row of its window (INT32_MAX: no row at
// all), sink: the first rows that stay visible, vis: the new rows on its path
__device__ __forceinline__ uint32_t seen_keys(int key0, int len, int low, int sink, uint32_t vis) {
    uint32_t m = key_range(key0, low, len);
    if (low != INT32_MAX) m |= key_range(key0, 0, min(sink, len));
    const int d = len - key0;
    return m | (d >= 32 || d <= -32 ? 0u : d >= 0 ? vis << d : vis >> -d);
}

// What V rows with a NaN or infinity (bits of bad) add to the outputs acc of this thread: weight times value where the
// row sees the key and has a weight for it, and nothing elsewhere.  Rare: kept out of the tile's code.
template <int T, int D, int DO>
__device__ __noinline__ void add_bad_rows(float *acc, const uint8_t *v_rows, uint2 bad, uint2 seen, uint32_t scores,
                                          float back, float off, int d0) {
    for (int j = 0; j < PA_KT; ++j) {
        if (!(((j < 32 ? bad.x : bad.y) >> (j & 31)) & 1u)) continue;
        uint32_t y;
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(y) : "r"(scores + j) : "memory");
        asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(y)::"memory");
        const float w = ((j < 32 ? seen.x : seen.y) >> (j & 31)) & 1u ? ex2(fmaf(__uint_as_float(y), back, off)) : 0.0f;
#pragma unroll 1
        for (int d = 0; d < DO; ++d) {
            const int x = 2 * (d0 + d);
            const uint16_t h = *reinterpret_cast<const volatile uint16_t *>(v_rows + pa_off<T, D>(j, x) + (x & 15));
            float v;
            if constexpr (T == SD_KV_BF16) v = __bfloat162float(__ushort_as_bfloat16(h));
            else v = __half2float(__ushort_as_half(h));
            if (w > 0.0f) acc[d] += w * v;
        }
    }
}

template <int R>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

template <int T, int D, int C>
__global__ void __launch_bounds__(WideLayout<T, D, C>::THREADS, 1)
    paged_wide_kernel(const PagedArgs a, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv) {
    using W = WideLayout<T, D, C>;
    using LY = PaLayout<T, D>;
    constexpr int NP = W::NP, RP = W::RP, NC = W::NC, KS = D / 16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ops = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *raw = ops + static_cast<size_t>(W::NOP) * W::OSTAGE;  // 8-bit rows: the copies' ring
    float *scratch = reinterpret_cast<float *>(raw + static_cast<size_t>(W::NRAW) * LY::STAGE);
    float *sm_m = scratch + PW_SOFT * 20, *sm_l = sm_m + 2 * PW_SOFT;
    uint64_t *op_full = reinterpret_cast<uint64_t *>(sm_l + PW_SOFT), *op_empty = op_full + W::NOP;
    uint64_t *raw_full = op_empty + W::NOP, *raw_empty = raw_full + W::NRAW;
    // in turns of two tiles, whatever the number of product buffers
    uint64_t *s_full = raw_empty + W::NRAW, *p_ready = s_full + 2, *pv_full = p_ready + 2, *pv_free = pv_full + 2;
    uint64_t *q_ready = pv_free + 2, *done = q_ready + 1, *mask_bar = done + 1;
    uint32_t *tbase = reinterpret_cast<uint32_t *>(mask_bar + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tbase + 1);
    volatile int *last = abort + 1;
    uint32_t *badw = tbase + 4;  // [3 turns][2]: rows of a tile with a NaN or infinity in V
    int64_t *prefix = reinterpret_cast<int64_t *>(tbase + 10);
    int2 *ln = reinterpret_cast<int2 *>(prefix + a.B + 1);
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < W::NOP; ++i) {
            mbar_init(&op_full[i], W::I8 ? 5 : 1);
            mbar_init(&op_empty[i], 1);
        }
        for (int i = 0; i < W::NRAW; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], 5);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 4 * PW_NG);
            mbar_init(&pv_full[i], 1);
            mbar_init(&pv_free[i], 4 * PW_NG);
        }
        mbar_init(mask_bar, 4 * PW_NG);
        mbar_init(q_ready, 4 * PW_NG);
        mbar_init(done, 1);
        *abort = 0;
        for (int i = 0; i < 6; ++i) badw[i] = 0;
        fence_barrier_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    Sched sc;
    if (!make_sched<RP, W::THREADS>(a, prefix, ln, sc)) return;
    if (warp == W::WARP_M) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tbase)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tbase;
    auto wait = [&](uint64_t *bar, uint32_t parity) {  // false: given up, and every role unwinds
        if (mbar_wait_bounded(bar, parity, PA_WAIT_NS, abort)) return true;
        set_status(a.status, SD_ETIMEOUT);
        *abort = 1;
        return false;
    };

    if (warp >= W::WARP_P && warp < W::WARP_P + 4) regs_dec<W::REG_P>();
    if (warp == W::WARP_P) {
        if constexpr (W::I8)
            produce_tiles<T, D, RP, W::QS, W::QR>(a, sc, &tmk, &tmv, raw, W::NRAW, raw_full, raw_empty, abort);
        else
            produce_tiles<T, D, RP, W::QS, W::QR>(a, sc, &tmk, &tmv, ops, W::NOP, op_full, op_empty, abort);
    } else if (warp == W::WARP_M) {
        // ---- the thread that issues the MMAs: tiles are numbered over the whole share
        if (elect_one()) {
            constexpr uint32_t FMT = T == SD_KV_BF16 ? 1u : 0u;
            constexpr uint32_t ID = (1u << 4) | (FMT << 7) | (FMT << 10) | (8u << 24);  // fp32 sums, M = 128
            // B K-major; B MN-major
            constexpr uint32_t ID_QK = ID | (PA_KT / 8 << 17), ID_PV = ID | (1u << 16) | (D / 8 << 17);
            const uint32_t ob = smem_u32(ops);
            int64_t u = sc.u0;
            int b = 0;
            uint32_t qk_slot = 0, qk_ph = 0, pv_slot = 0;  // operand stages of the next scores and the next product
            uint32_t nqk = 0, npv = 0, np = 0;             // tiles and pieces so far
            bool ok = true;
            while (ok && u < sc.u1) {
                const Piece p = piece_at<RP>(a, sc, u, b);
                b = p.b;
                const int n = p.t1 - p.t0;
                if (!wait(q_ready, np & 1u)) break;
                ++np;
                if constexpr (!W::I8)
                    for (int s = 0; s < W::QS; ++s) {  // the queries' stages are read
                        mbar_arrive(&op_empty[qk_slot]);
                        if (++qk_slot == W::NOP) {
                            qk_slot = 0;
                            qk_ph ^= 1u;
                        }
                        if (++pv_slot == W::NOP) pv_slot = 0;
                    }
                auto scores = [&]() {
                    if (!wait(&op_full[qk_slot], qk_ph)) return false;
                    tc_fence_after();
                    const uint32_t kb = ob + qk_slot * W::OSTAGE, d = tm + W::TS + (nqk & 1u) * W::SCOLS;
                    bool acc = false;
                    // the smallest parts first: the accumulation truncates at the size that the sum has by then
#pragma unroll
                    for (int x = NP - 1; x >= 0; --x)
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) {
                            tc_mma_ts(d, tm + W::TQ + x * (D / 2) + ks * 8,
                                      sw128_desc(kb + (ks >> 2) * W::OTILE + (ks & 3) * 32, 0), ID_QK, acc);
                            acc = true;
                        }
                    tc_commit(&s_full[nqk & 1u]);
                    ++nqk;
                    if (++qk_slot == W::NOP) {
                        qk_slot = 0;
                        qk_ph ^= 1u;
                    }
                    return true;
                };
                ok = scores() && (n < 2 || scores());
                for (int i = 0; ok && i < n; ++i) {
                    const uint32_t sb = npv & 1u, ob2 = npv % W::NPV;
                    ok = npv < W::NPV || wait(&pv_free[(npv - W::NPV) & 1u], ((npv - W::NPV) >> 1) & 1u);
                    ok = ok && wait(&p_ready[sb], (npv >> 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t vb = ob + pv_slot * W::OSTAGE + W::OKV, d = tm + W::TO + ob2 * D,
                                   pa = tm + W::TS + sb * W::SCOLS;
                    bool acc = false;
#pragma unroll
                    for (int x = W::NR - 1; x >= 0; --x)
#pragma unroll
                        for (int ks = 0; ks < PA_KT / 16; ++ks) {
                            tc_mma_ts(d, pa + x * 32 + ks * 8, sw128_desc(vb + ks * 2048, W::OTILE), ID_PV, acc);
                            acc = true;
                        }
                    tc_commit(&pv_full[sb]);
                    tc_commit(&op_empty[pv_slot]);
                    ++npv;
                    if (++pv_slot == W::NOP) pv_slot = 0;
                    // the scores of tile i + 2 go where the weights of tile i are; MMAs of one thread execute in order
                    if (i + 2 < n) ok = scores();
                }
                u += n;
            }
            tc_commit(done);  // no MMA is left when the tensor memory goes
            (void)mbar_wait_bounded(done, 0, PA_WAIT_NS);
        }
        __syncwarp();
    } else if (warp == W::WARP_S || warp >= W::WARP_C) {
        if constexpr (W::I8) {
            // ---- 8-bit rows to fp16 operands: thread ct takes row ct % 64 of K (ct < 64) or V; a warp of its own
            // writes the scales (on a converting warp they were the longest way through a tile: 254 -> 221 us for 16
            // sequences of 16000 rows)
            if (warp >= W::WARP_C) regs_dec<W::REG_C>();
            const int ct = tid - 32 * W::WARP_C, row = ct & 63;
            const bool isv = ct >= 64;
            // 16-byte chunk x of a row is at its row's offset with x in the swizzled bits: exclusive-ors of one base
            const uint32_t from = (isv ? LY::KV : 0) + pa_off<T, D>(row, 0);
            const uint32_t to = (isv ? W::OKV : 0) + pa_off<SD_KV_F16, D>(row, 0);
            uint32_t rs = 0, rph = 0, os = 0, oph = 0, np = 0;
            int64_t u = sc.u0, i = 0;
            int b = 0, left = 0;  // tiles of the piece still to come
            Piece p = {};
            // the unit of the tiles of the piece that every row sees, so far: a power of two above their V scales (its bits)
            uint32_t unit = 0x00800000u;
            for (; left > 0 || u < sc.u1; ++i, --left) {
                if (left == 0) {  // the next piece: its queries' stages go back once they are read
                    p = piece_at<RP>(a, sc, u, b);
                    b = p.b;
                    left = p.t1 - p.t0;
                    u += left;
                    unit = 0x00800000u;
                    if (!mbar_wait_bounded(q_ready, np++ & 1u, PA_WAIT_NS, abort)) {
                        set_status(a.status, SD_ETIMEOUT);
                        *abort = 1;
                    }
                    for (int s = 0; s < W::QS; ++s) {
                        if (lane == 0) mbar_arrive(&raw_empty[rs]);
                        if (++rs == W::NRAW) {
                            rs = 0;
                            rph ^= 1u;
                        }
                    }
                }
                bool ok = mbar_wait_bounded(&raw_full[rs], rph, PA_WAIT_NS, abort);
                if (ok && i >= W::NOP) ok = mbar_wait_bounded(&op_empty[os], oph ^ 1u, PA_WAIT_NS, abort);
                if (!ok) {  // (the loop goes on: every later wait gives up at once)
                    set_status(a.status, SD_ETIMEOUT);
                    *abort = 1;
                }
                __syncwarp();
                const uint8_t *src = raw + static_cast<size_t>(rs) * LY::STAGE;
                uint8_t *dst = ops + static_cast<size_t>(os) * W::OSTAGE;
                if (warp >= W::WARP_C) {
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        // (a row's 16-byte chunks beyond 128 bytes are in the next tensor tile)
                        const uint4 v =
                            *reinterpret_cast<const uint4 *>(src + ((from + (x * 16 / LY::ROWB) * LY::TILE) ^ (x * 16 % LY::ROWB)));
                        const uint32_t w[4] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u, v.w ^ 0x80808080u};
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            *reinterpret_cast<uint4 *>(
                                dst + ((to + ((32 * x + 16 * y) / 128) * W::OTILE) ^ ((32 * x + 16 * y) % 128))) =
                                make_uint4(codes2<0, 1>(w[2 * y]), codes2<2, 3>(w[2 * y]), codes2<0, 1>(w[2 * y + 1]),
                                           codes2<2, 3>(w[2 * y + 1]));
                    }
                } else {
                    const float *ss = reinterpret_cast<const float *>(src + 2 * LY::KV);
                    float *ds = reinterpret_cast<float *>(dst + 2 * W::OKV);
                    const float k0 = ss[lane], k1 = ss[lane + 32], v0 = ss[PA_KT + lane], v1 = ss[PA_KT + 32 + lane];
                    ds[lane] = k0 + 0.0f * k0;  // an infinite K scale makes a row of NaN
                    ds[lane + 32] = k1 + 0.0f * k1;
                    // V scales in the tile's unit: of a tile that every row sees a power of two above those of all such tiles
                    // so far in the piece; of another, whose scales may be of any size where a row does not look, 1
                    const int t = p.t1 - left, tile0 = (t < p.st.n_sink ? t : t - p.st.n_sink + p.st.lo_tile) * PA_KT;
                    const bool whole = tile0 + PA_KT <= p.len &&
                                       (a.window == 0 || tile0 >= p.len + p.n - a.window || tile0 + PA_KT <= a.sinks);
                    const uint32_t above = unit_above(__reduce_max_sync(0xffffffffu, max(scale_bits(v0), scale_bits(v1))));
                    if (whole) unit = max(unit, above);
                    const float down = whole ? unit_inverse(unit) : 1.0f;
                    ds[PA_KT + lane] = v0 * down;
                    ds[PA_KT + 32 + lane] = v1 * down;
                    if (lane == 0) ds[2 * PA_KT] = whole ? __uint_as_float(unit) : 1.0f;
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&raw_empty[rs]);
                    mbar_arrive(&op_full[os]);
                }
                if (++rs == W::NRAW) {
                    rs = 0;
                    rph ^= 1u;
                }
                if (++os == W::NOP) {
                    os = 0;
                    oph ^= 1u;
                }
            }
        }
    } else if (warp < 4 * PW_NG) {
        regs_inc<W::REG_S>();
        // ---- softmax: thread = lane of tensor memory (row lt % RP, lane group lt / RP), of which each of the PW_NG
        // groups weighs some keys of every tile and adds some columns of its product; a lane's maximum is shared by its
        // PW_NG threads
        const int grp = warp >> 2, lt = tid & 127, quarter = warp & 3;
        const uint32_t tq = tm + (static_cast<uint32_t>(32 * quarter) << 16);
        const int lg = lt / RP, r = lt % RP;
        // this lane's part and keys; this thread's keys
        const int part = lg % W::CP, l_at = (lg / W::CP) * W::KL, k_at = l_at + grp * NC;
        int64_t u = sc.u0;
        int b = 0;
        uint32_t nt = 0, nsync = 0, nmask = 0, nmax = 0, slot_n = 0, slot_ph = 0, q_slot = 0, q_ph = 0;
        bool ok = true;
        auto sync_all = [&]() {  // all softmax warps (an mbarrier: waits that give up)
            __syncwarp();
            if (lane == 0) mbar_arrive(mask_bar);
            return __all_sync(0xffffffffu, wait(mask_bar, nsync++ & 1u)) != 0;
        };
        // the largest of a lane's PW_NG values; `ok` false in any of its warps makes it false in all: they leave
        // together
        auto lane_max = [&](float x) {
            float *turn = sm_m + (nmax++ & 1u) * PW_SOFT;
            turn[tid] = x;
            tc_fence_before();  // the lane's scores are read; its weights may go over them
            ok = !bar_any(1 + quarter, 32 * PW_NG, !ok);
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < PW_NG; ++g) x = fmaxf(x, turn[g * 128 + lt]);
            return x;
        };
        while (u < sc.u1) {
            const Piece p = piece_at<RP>(a, sc, u, b);
            b = p.b;
            const int rows = p.n * a.g, tg = p.rg * RP + r;
            const bool real = tg < rows;
            float2 o[W::DO / 2];
            float back = 1.0f;
            {
                // this thread's columns of the row's query into tensor memory, in parts; fp16 parts scaled by a power
                // of two as in paged_attn_kernel.  The producer has put the rows into the first stages of the piece
                if constexpr (!W::I8) q_slot = slot_n, q_ph = slot_ph;
                uint64_t *qfull = W::I8 ? raw_full : op_full;
                const uint8_t *qring = W::I8 ? raw : ops;
                const float4 *qp = nullptr;
#pragma unroll
                for (int s = 0; s < W::QS; ++s) {
                    ok = ok && __all_sync(0xffffffffu, wait(&qfull[q_slot], q_ph));
                    if (r / W::QR == s)
                        qp = reinterpret_cast<const float4 *>(qring + static_cast<size_t>(q_slot) * LY::STAGE +
                                                              (r - s * W::QR) * W::QROW + grp * W::DO * 4);
                    if (++q_slot == (W::I8 ? W::NRAW : W::NOP)) {
                        q_slot = 0;
                        q_ph ^= 1u;
                    }
                }
                if constexpr (!W::I8) slot_n = q_slot, slot_ph = q_ph;
                float mx = 0.0f;
#pragma unroll
                for (int d = 0; d < W::DO; d += 4) {
                    const float4 f = real && ok ? qp[d / 4] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    o[d / 2] = make_float2(f.x * a.qscale, f.y * a.qscale);
                    o[d / 2 + 1] = make_float2(f.z * a.qscale, f.w * a.qscale);
#pragma unroll
                    for (int e = 0; e < 2; ++e) mx = fmaxf(mx, fmaxf(fabsf(o[d / 2 + e].x), fabsf(o[d / 2 + e].y)));
                }
                float up = 1.0f;
                if constexpr (T != SD_KV_BF16) {
                    mx = lane_max(mx);
                    // 2^ex above a finite maximum, by its exponent; powers of two by theirs
                    const int ex = mx < INFINITY ? max(static_cast<int>(__float_as_uint(mx) >> 23) - 126, -100) : 0;
                    up = __int_as_float((127 + 11 - ex) << 23);
                    back = __int_as_float((127 + ex - 11) << 23);
                }
#pragma unroll
                for (int d = 0; d < W::DO; d += 16) {
                    uint32_t f16[NP][8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const Parts<T> f = split_pair<T>(fmul2_rn(o[d / 2 + e], make_float2(up, up)));
#pragma unroll
                        for (int x = 0; x < NP; ++x) f16[x][e] = f.r[x];
                    }
#pragma unroll
                    for (int x = 0; x < NP; ++x) tc_st(f16[x], tq + W::TQ + x * (D / 2) + (grp * W::DO + d) / 2);
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_ready);
            }
            uint32_t vis = 0;
            int low = INT32_MAX;
            if (real) {
                int depth;
                vis = new_rows_seen(a, p.b, tg / a.g, p.len, depth);
                low = a.window > 0 ? p.len + depth - a.window + 1 : 0;
            }
            const int full_lo = a.window > 0 ? p.len + p.n - a.window : 0, full_sink = a.window > 0 ? a.sinks : 0;
            // al: rescale of the outputs before the product still to be added; vunit: their unit (8-bit rows), a power of
            // two above every V scale that this lane's row has seen so far, as in paged_attn_kernel
            float m = PA_NEG, l = 0.0f, al = 0.0f;
            uint32_t vunit = 0x00800000u;
#pragma unroll
            for (int d = 0; d < W::DO / 2; ++d) o[d] = make_float2(0.0f, 0.0f);
            // adds this thread's columns of the product of tile number i to the outputs
            auto add_product = [&](uint32_t i) {
                const bool got = wait(&pv_full[i & 1u], (i >> 1) & 1u);
                tc_fence_after();
                const uint32_t at = tq + W::TO + (i % W::NPV) * D + grp * W::DO;
                uint32_t y[W::DO / 32][32];
#pragma unroll
                for (int d = 0; d < W::DO / 32; ++d) tc_ld(y[d], at + 32 * d);
#pragma unroll
                for (int d = 0; d < W::DO / 32; ++d) {
                    tc_wait_ld(y[d]);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 f = make_float2(__uint_as_float(y[d][2 * e]), __uint_as_float(y[d][2 * e + 1]));
                            o[16 * d + e] = ffma2_rn(o[16 * d + e], make_float2(al, al), f);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pv_free[i & 1u]);
                return got;
            };
            for (int t = p.t0; t < p.t1; ++t, ++nt) {
                const uint32_t sb = nt & 1u, slot = slot_n, slot_par = slot_ph;
                if (++slot_n == W::NOP) {
                    slot_n = 0;
                    slot_ph ^= 1u;
                }
                if constexpr (W::I8) {  // the copies' ring, which holds the queries, goes on beside the operands'
                    if (++q_slot == W::NRAW) {
                        q_slot = 0;
                        q_ph ^= 1u;
                    }
                }
                // (each lane's own answer: lane_max brings them together)
                ok = wait(&s_full[sb], (nt >> 1) & 1u) && ok;
                tc_fence_after();
                const uint32_t sc_at = tq + W::TS + sb * W::SCOLS;
                const int tile0 = (t < p.st.n_sink ? t : t - p.st.n_sink + p.st.lo_tile) * PA_KT, key0 = tile0 + k_at;
                const uint8_t *stage = ops + static_cast<size_t>(slot) * W::OSTAGE;
                const float *scales = reinterpret_cast<const float *>(stage + 2 * W::OKV);
                const bool whole = tile0 + PA_KT <= p.len && (tile0 >= full_lo || tile0 + PA_KT <= full_sink);
                if (W::I8 || !whole)  // what stands in the stage is read below: its barrier makes it visible here too
                    ok = wait(&op_full[slot], slot_par) && ok;
                // 8-bit rows: `above` is what the outputs' unit has to reach.  Outputs in a unit 2^k times the tile's take
                // weights that are smaller by that, in the exponent; the sum of weights gets it back
                // (k is from -104, where 2^(14 + 104) is left of the largest weights, to 112, where 2^(14 - 112) is: the weights
                // that count and their sum stay normal numbers)
                uint32_t above = 0, tile_unit = 0;
                if constexpr (W::I8) above = tile_unit = __float_as_uint(scales[2 * PA_KT]);
                float2 s[NC / 2];
                {
                    uint32_t y[NC];
                    tc_ld(y, sc_at + k_at);
                    tc_wait_ld(y);
#pragma unroll
                    for (int e = 0; e < NC / 2; ++e)
                        s[e] = make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1]));
                }
                if constexpr (W::I8) {
#pragma unroll
                    for (int e = 0; e < NC / 2; e += 2) {
                        const float4 f = *reinterpret_cast<const float4 *>(scales + k_at + 2 * e);
                        s[e] = fmul2_rn(s[e], make_float2(f.x, f.y));
                        s[e + 1] = fmul2_rn(s[e + 1], make_float2(f.z, f.w));
                    }
                }
                if (!whole) {
                    const uint32_t seen = seen_keys(key0, p.len, low, full_sink, vis);
#pragma unroll
                    for (int e = 0; e < NC; ++e)
                        if (!((seen >> e) & 1u)) (e & 1 ? s[e / 2].y : s[e / 2].x) = -INFINITY;
                    if constexpr (W::I8) {  // (the tile's unit is 1)
                        uint32_t top = 0;
                        // (rolled in the longest kernel: 432 -> 412 us for 256 sequences of 500 rows, 128 query rows; the
                        // others are faster unrolled, 10 query rows over 16000-row contexts 221 us against 227)
                        if constexpr (D == 128 && C == 1) {
#pragma unroll 2
                            for (int e = 0; e < NC; e += 4) {
                                const float4 f = *reinterpret_cast<const float4 *>(scales + PA_KT + k_at + e);
                                const uint32_t m = seen >> e;
                                const uint32_t a0 = max(m & 1u ? scale_bits(f.x) : 0u, m & 2u ? scale_bits(f.y) : 0u);
                                const uint32_t a1 = max(m & 4u ? scale_bits(f.z) : 0u, m & 8u ? scale_bits(f.w) : 0u);
                                top = max(top, max(a0, a1));
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < NC; ++e)
                                if ((seen >> e) & 1u) top = max(top, scale_bits(scales[PA_KT + k_at + e]));
                        }
                        above = max(unit_above(__float_as_uint(lane_max(__uint_as_float(top)))), tile_unit - (104u << 23));
                    }
                }
                float shrink = 1.0f, k = 0.0f, two_k = 1.0f;
                if constexpr (W::I8) {
                    const uint32_t was = vunit;
                    vunit = min(max(was, above), tile_unit + (112u << 23));
                    shrink = __uint_as_float(was) * unit_inverse(vunit);
                    k = static_cast<float>(static_cast<int>(vunit - tile_unit) >> 23);
                    two_k = __uint_as_float(0x3f800000u + (vunit - tile_unit));
                }
                float x2[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < NC / 2; ++e) x2[e & 1] = fmaxf(fmaxf(x2[e & 1], s[e].x), s[e].y);
                const float n = fmaxf(m, lane_max(fmaxf(x2[0], x2[1])) * back);
                if (!ok) break;
                const float an = ex2(m - n), off = PW_UP - k - n;
                m = n;
                bool rescaled = false;
                if constexpr (!W::I8) {
                    if (!whole) {
                        // V rows with a NaN or infinity reach the rows that see them alone: added here, and cleared
                        // before the product
                        uint32_t bw[2] = {0, 0};
#pragma unroll 1
                        for (int x = tid; x < PA_KT * (2 * D / 16); x += PW_SOFT) {
                            const int vr = x % PA_KT;
                            const uint4 v =
                                *reinterpret_cast<const uint4 *>(stage + W::OKV + pa_off<T, D>(vr, (x / PA_KT) * 16));
                            constexpr uint32_t EX = T == SD_KV_BF16 ? 0x7f80u : 0x7c00u;
                            const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int w = 0; w < 4; ++w)
                                if ((q[w] & EX) == EX || ((q[w] >> 16) & EX) == EX) bw[vr >> 5] |= 1u << (vr & 31);
                        }
                        // the words of the next turn are cleared ahead of this one's barrier: they were read before the last
                        // one, and are written behind this one
                        uint32_t *words = badw + 2 * nmask;
                        nmask = nmask == 2 ? 0 : nmask + 1;
                        if (tid == 0) badw[2 * nmask] = badw[2 * nmask + 1] = 0;
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            const uint32_t any = __reduce_or_sync(0xffffffffu, bw[w]);
                            if (lane == 0 && any) atomicOr(&words[w], any);
                        }
                        ok = sync_all() && ok;
                        const uint32_t bad[2] = {*reinterpret_cast<volatile uint32_t *>(&words[0]),
                                                 *reinterpret_cast<volatile uint32_t *>(&words[1])};
                        if (__all_sync(0xffffffffu, ok) && (bad[0] | bad[1])) {
                            if (t > p.t0) ok = add_product(nt - 1) && ok;
                            float acc[W::DO];
#pragma unroll
                            for (int d = 0; d < W::DO / 2; ++d) {
                                acc[2 * d] = o[d].x * an;
                                acc[2 * d + 1] = o[d].y * an;
                            }
                            rescaled = true;
                            uint2 seen = make_uint2(seen_keys(tile0, p.len, low, full_sink, vis),
                                                    seen_keys(tile0 + 32, p.len, low, full_sink, vis));
                            // this lane's keys, once for all parts
                            seen.x &= part == 0 ? key_range(0, l_at, l_at + W::KL) : 0u;
                            seen.y &= part == 0 ? key_range(32, l_at, l_at + W::KL) : 0u;
                            add_bad_rows<T, D, W::DO>(acc, stage + W::OKV, make_uint2(bad[0], bad[1]), seen, sc_at,
                                                      back, off, grp * W::DO);
#pragma unroll
                            for (int d = 0; d < W::DO / 2; ++d) o[d] = make_float2(acc[2 * d], acc[2 * d + 1]);
                            ok = sync_all() && ok;
#pragma unroll 1
                            for (int x = tid; x < PA_KT * (2 * D / 16); x += PW_SOFT) {
                                const int vr = x % PA_KT;
                                if ((bad[vr >> 5] >> (vr & 31)) & 1u)
                                    *reinterpret_cast<uint4 *>(const_cast<uint8_t *>(stage) + W::OKV +
                                                               pa_off<T, D>(vr, (x / PA_KT) * 16)) =
                                        make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async_shared();
                        }
                    }
                }
                // weights in parts, over the scores: the lane's threads read theirs before any writes (lane_max is
                // behind them)
                float2 l2 = make_float2(0.0f, 0.0f);
                uint32_t keep[W::NR][NC / 2];
#pragma unroll
                for (int e = 0; e < NC / 2; ++e) {
                    const float2 x = ffma2_rn(s[e], make_float2(back, back), make_float2(off, off));
                    s[e] = make_float2(ex2(x.x), ex2(x.y));
                    l2 = fadd2_rn(l2, s[e]);
                }
                l = fmaf(l, an, W::I8 ? (l2.x + l2.y) * two_k : l2.x + l2.y);
                if constexpr (W::I8) {
#pragma unroll
                    for (int e = 0; e < NC / 2; e += 2) {
                        const float4 f = *reinterpret_cast<const float4 *>(scales + PA_KT + k_at + 2 * e);
                        const float2 was = s[e], was1 = s[e + 1];
                        s[e] = fmul2_rn(s[e], make_float2(f.x, f.y));
                        s[e + 1] = fmul2_rn(s[e + 1], make_float2(f.z, f.w));
                        if (!whole) {  // a key with no weight keeps none, whatever its scale is
                            s[e] = make_float2(was.x > 0.0f ? s[e].x : was.x, was.y > 0.0f ? s[e].y : was.y);
                            s[e + 1] = make_float2(was1.x > 0.0f ? s[e + 1].x : was1.x, was1.y > 0.0f ? s[e + 1].y : was1.y);
                        }
                    }
                }
                if constexpr (W::CP == 1) {
#pragma unroll
                    for (int e = 0; e < NC / 2; ++e) {
                        const Parts<T> f = split_pair<T>(s[e]);
#pragma unroll
                        for (int x = 0; x < W::NR; ++x) keep[x][e] = f.r[x];
                    }
                } else {
                    // one part, the same for the whole warp (lane groups are whole warps): part `part` of what the
                    // parts before leave
                    static_assert(W::NR == 1 && RP % 32 == 0, "one part a lane, one lane group a warp");
                    for (int k = 0; k < part && k < NP - 1; ++k)
#pragma unroll
                        for (int e = 0; e < NC / 2; ++e) s[e] = part_left<T>(s[e], part_bits<T>(s[e]));
                    if (part < NP) {
#pragma unroll
                        for (int e = 0; e < NC / 2; ++e) keep[0][e] = part_bits<T>(s[e]);
                    } else {
#pragma unroll
                        for (int e = 0; e < NC / 2; ++e) keep[0][e] = 0;
                    }
                }
#pragma unroll
                for (int x = 0; x < W::NR; ++x) tc_st(keep[x], sc_at + x * 32 + k_at / 2);
                if constexpr (W::KL < PA_KT) {  // the other lanes' keys weigh nothing in this one
                    uint32_t zero[NC / 2];
#pragma unroll
                    for (int e = 0; e < NC / 2; ++e) zero[e] = 0;
#pragma unroll
                    for (int x = 0; x < W::NR; ++x) tc_st(zero, sc_at + x * 32 + (W::KL - l_at + grp * NC) / 2);
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[sb]);
                // the product of the tile before, while this one's runs
                if (t > p.t0 && !rescaled) ok = add_product(nt - 1) && ok;
                al = rescaled ? 1.0f : W::I8 ? an * shrink : an;
            }
            ok = add_product(nt - 1) && ok;
            if (bar_any(5, PW_SOFT, !ok)) break;  // all softmax warps leave together
            // ---- write the piece: a run that is whole goes out, others become partials
            const bool complete = p.t0 == 0 && p.t1 == p.st.T;
            const int pslot = 2 * static_cast<int>(blockIdx.x) + (p.t0 == 0 ? 1 : 0);
            sm_m[tid] = m;
            sm_l[tid] = l;
            named_bar_sync(5, PW_SOFT);
            // a lane's threads have the same maximum, lanes with parts of the same weights the same sums too
            float mx = PA_NEG, lv = 0.0f;
#pragma unroll
            for (int j = 0; j < C; j += W::CP) mx = fmaxf(mx, sm_m[j * RP + r]);
#pragma unroll
            for (int j = 0; j < C; j += W::CP) {
                float x = 0.0f;
#pragma unroll
                for (int g = 0; g < PW_NG; ++g) x += sm_l[g * 128 + j * RP + r];
                lv = fmaf(x, ex2(sm_m[j * RP + r] - mx), lv);
            }
            const float unit = W::I8 ? __uint_as_float(vunit) : 1.0f;
            const float f = ex2(m - mx) * unit * (!complete ? 1.0f : lv == 0.0f ? 0.0f : 1.0f / lv);
            if (!complete && real && lg == 0 && grp == 0) a.part_ml[pslot * RP + r] = make_float2(mx, lv);
            // rows of D floats from the threads' columns times fac, 16 columns of every group at a time through shared
            // memory: thread = 4 columns of row tid / 8 (and of the rows RW further on), group (tid / 4) % 2
            auto write_rows = [&](bool final, float fac) {
                constexpr int RW = PW_SOFT / (4 * PW_NG), NK = (RP + RW - 1) / RW;
                const int wg = (tid >> 2) % PW_NG, wc = wg * W::DO + 4 * (tid & 3), wr = tid / (4 * PW_NG);
                float *to[NK];
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    const int tr = wr + RW * k, y = p.rg * RP + tr;
                    to[k] = tr >= RP || y >= rows ? nullptr
                            : final ? a.out + p.b * a.o_sb + (y / a.g) * a.o_sm +
                                          static_cast<int64_t>(p.kh * a.g + y % a.g) * D + wc
                                    : a.part_o + (static_cast<int64_t>(pslot) * RP + tr) * D + wc;
                }
#pragma unroll
                for (int d = 0; d < W::DO; d += 16) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 x = fmul2_rn(o[d / 2 + 2 * e], make_float2(fac, fac));
                        const float2 y = fmul2_rn(o[d / 2 + 2 * e + 1], make_float2(fac, fac));
                        *reinterpret_cast<float4 *>(scratch + tid * 20 + 4 * e) = make_float4(x.x, x.y, y.x, y.y);
                    }
                    named_bar_sync(5, PW_SOFT);
#pragma unroll
                    for (int k = 0; k < NK; ++k)
                        if (to[k] && SD_INB(p.b < a.B && (p.rg * RP + wr + RW * k) / a.g < a.M && p.kh < a.H_kv &&
                                                (final || (pslot + 1) * RP <= a.part_rows),
                                            a.status, 117)) {  // site 117: rows of a piece
                            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                            for (int j = 0; j < C; ++j) {
                                const float4 x = *reinterpret_cast<const float4 *>(
                                    scratch + (wg * 128 + j * RP + wr + RW * k) * 20 + 4 * (tid & 3));
                                v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
                            }
                            *reinterpret_cast<float4 *>(to[k] + d) = v;
                        }
                    named_bar_sync(5, PW_SOFT);
                }
            };
            // C = 1: a thread's columns of a partial as they are, [D / 4][128] 16-byte columns (lanes beside each
            // other: whole lines, no exchange); the joining CTA's threads read the same places.
            // (Rows are written at one place in the code: 127 KB of instructions instead of 137.)
            float4 *lanes = reinterpret_cast<float4 *>(a.part_o) + grp * (W::DO / 4) * 128 + lt;
            bool rows_ready = complete;
            float fac = f;
            if constexpr (C > 1) {
                write_rows(complete, f);
            } else if (!complete) {
#pragma unroll
                for (int d = 0; d < W::DO / 4; ++d)
                    lanes[static_cast<int64_t>(pslot) * (RP * D / 4) + d * 128] =
                        make_float4(o[2 * d].x * unit, o[2 * d].y * unit, o[2 * d + 1].x * unit, o[2 * d + 1].y * unit);
            }
            if (!complete) {
                const int c0 = cta_of(sc, p.run0), c1 = cta_of(sc, p.run0 + p.st.T - 1);
                __threadfence();
                named_bar_sync(5, PW_SOFT);
                if (tid == 0 && SD_INB(c0 >= 0 && c0 < c1 && c1 < static_cast<int>(gridDim.x) && (2 * c1 + 2) * RP <= a.part_rows,
                                       a.status, 118)) {  // site 118: counter, partials
                    const int was = atomicAdd(&a.counters[c0], 1);
                    *last = was == c1 - c0;
                    if (was == c1 - c0) a.counters[c0] = 0;
                }
                named_bar_sync(5, PW_SOFT);
                if (*last) {
                    if constexpr (C > 1) {
                        join_partials<RP, D, PW_SOFT>(a, p, c0, c1, tid, scratch, 5);
                    } else {
                        // as join_partials: in the order of the keys, with a running maximum; two partials' loads in
                        // flight at once
                        __threadfence();
                        float jm = PA_NEG, jl = 0.0f;
#pragma unroll
                        for (int d = 0; d < W::DO / 2; ++d) o[d] = make_float2(0.0f, 0.0f);
                        for (int x0 = c0; x0 <= c1; x0 += 2) {
                            float2 ml[2];
                            float4 y[2][W::DO / 4];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int x = min(x0 + h, c1);  // (past the last: read again, and weighed by 0)
                                const int64_t sl = 2 * x + (x == c0);
                                ml[h] = __ldcg(&a.part_ml[sl * RP + r]);
#pragma unroll
                                for (int d = 0; d < W::DO / 4; ++d)
                                    y[h][d] = __ldcg(lanes + sl * (RP * D / 4) + d * 128);
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (x0 + h > c1) break;
                                const float n = fmaxf(jm, ml[h].x), w0 = ex2(jm - n), w = ex2(ml[h].x - n);
                                jm = n;
                                jl = fmaf(jl, w0, ml[h].y * w);
#pragma unroll
                                for (int d = 0; d < W::DO / 4; ++d) {
                                    const float2 lo = fmul2_rn(o[2 * d], make_float2(w0, w0));
                                    const float2 hi = fmul2_rn(o[2 * d + 1], make_float2(w0, w0));
                                    o[2 * d] = ffma2_rn(make_float2(y[h][d].x, y[h][d].y), make_float2(w, w), lo);
                                    o[2 * d + 1] = ffma2_rn(make_float2(y[h][d].z, y[h][d].w), make_float2(w, w), hi);
                                }
                            }
                        }
                        fac = jl == 0.0f ? 0.0f : 1.0f / jl;
                        rows_ready = true;
                    }
                }
            }
            if constexpr (C == 1)
                if (rows_ready) write_rows(true, fac);
            u += p.t1 - p.t0;
        }
    }
    // ---- every role is done
    tc_fence_before();
    __syncthreads();
    if (warp == W::WARP_M) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
    }
}

template <int T, int D, int C>
cudaError_t wide_launch(const PagedArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, int grid, cudaStream_t s) {
    using W = WideLayout<T, D, C>;
    const size_t smem = W::fixed() + (static_cast<size_t>(a.B) + 1) * 8 + static_cast<size_t>(a.B) * 8;
    const cudaError_t e = allow_max_dynamic_smem(paged_wide_kernel<T, D, C>);
    if (e != cudaSuccess) return e;
    return launch(paged_wide_kernel<T, D, C>, dim3(grid), dim3(W::THREADS), smem, s, a, tmk, tmv);
}
template <int T, int D>
cudaError_t wide_launch_c(const PagedArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, int rows, int grid,
                          cudaStream_t s) {
    if (rows <= 32) return wide_launch<T, D, 4>(a, tmk, tmv, grid, s);
    // (two lane groups for three bf16 parts make two passes of the product: 346 us against 264 us with one group, 64
    // rows, 16 sequences of 16000 rows)
    if constexpr (T != SD_KV_BF16)
        if (rows <= 64) return wide_launch<T, D, 2>(a, tmk, tmv, grid, s);
    return wide_launch<T, D, 1>(a, tmk, tmv, grid, s);
}

}  // namespace sdv
