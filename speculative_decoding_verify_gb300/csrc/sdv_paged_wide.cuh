// sdv_paged_wide.cuh - the attention over pages for many query rows per KV head (a tree of drafts, grouped
// heads): the same work, cut, masks and partials as paged_attn_kernel, on the 5th-generation tensor cores.
//
// The rows of one (sequence, KV head) are the 128 lanes of tensor memory.  With at most 64 (32) of them the lanes hold
// C = 2 (4) groups of the same rows, which hold different 16-bit parts of the weights (one pass of the product instead of
// two or three) or weigh different keys of a tile; the lane groups join at the end of a piece as the splits of a run do.
//   S = Q K^T: tcgen05.mma kind::f16, M = 128, N = 64, Q in tensor memory as A (written once per piece, in 16-bit parts
//     that add up to the fp32 value: two fp16, or three bf16), K as B from shared memory as the tensor copy left it
//     (K-major, 128-byte swizzle);
//   softmax: one thread per lane, so a row's maximum and sum need no exchange; the weights go back to tensor memory
//     over the scores, in parts; two groups of four warps take the tiles in turn, each with a state of its own;
//   O_t = P V: the weights as A, V as B (MN-major, the same swizzle), from zero for each tile; the softmax threads add
//     it to their fp32 outputs in registers with the rescale of the running maximum (a tensor-core accumulator kept
//     over the tiles would truncate at every step, and rescaling it would cost the same loads and more stores).
// One thread issues all MMAs: scores two tiles ahead of the weights, so the tensor cores work while the softmax of
// two tiles runs.  8-bit rows pass through four more warps that write them as fp16 into operand
// buffers (exact) and their scales beside them.
//
// What bounds it: at 128 rows of D = 128 a 64-key fp16 tile is 32 KB of HBM (about 1400 SM cycles of one SM's share)
// against 4 x 128 x 64 x 128 multiply-adds (about 1050 cycles) and 64 weights a thread.
#pragma once

#include "sdv_paged_attn.cuh"

namespace sdv {

constexpr int PW_SOFT = 128;   // threads of a softmax group (four warps: the lane quarters of tensor memory)
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

#define PW_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
#define PW_I8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])
#define PW_W8(r, o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), "+r"(r[o + 4]), "+r"(r[o + 5]), "+r"(r[o + 6]), "+r"(r[o + 7])

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
__device__ __forceinline__ void tc_st(const uint32_t (&r)[32], uint32_t addr) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
                 "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
                 PW_I8(r, 0), PW_I8(r, 8), PW_I8(r, 16), PW_I8(r, 24)
                 : "memory");
}
__device__ __forceinline__ float ex2(float x) {  // 2^x to about 2^-22, 0 below the normal numbers
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a pair of weights in 16-bit parts, as split2 (the differences are exact)
template <int T>
__device__ __forceinline__ Parts<T> split_pair(float2 x) {
    Parts<T> p;
#pragma unroll
    for (int i = 0; i < Parts<T>::N; ++i) {
        float2 f;
        if constexpr (T == SD_KV_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
            p.r[i] = *reinterpret_cast<const uint32_t *>(&h);
            f = make_float2(__uint_as_float(p.r[i] << 16), __uint_as_float(p.r[i] & 0xffff0000u));
        } else {
            const __half2 h = __floats2half2_rn(x.x, x.y);
            p.r[i] = *reinterpret_cast<const uint32_t *>(&h);
            f = __half22float2(h);
        }
        if (i + 1 < Parts<T>::N) x = ffma2_rn(f, make_float2(-1.0f, -1.0f), x);
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
    static constexpr int NC = PA_KT * CP / C;       // keys of a tile that a thread weighs
    static constexpr int NR = (NP + CP - 1) / CP;   // parts that a lane holds: passes of the product
    static constexpr int OTILE = PA_KT * 128;       // 64 keys x 64 halves
    static constexpr int OKV = D / 64 * OTILE;      // K (or V) operand of a tile
    static constexpr int OSCALES = I8 ? 1024 : 0;   // scales of K [64], of V [64] in units of the tile's, that unit
    static constexpr int OSTAGE = 2 * OKV + OSCALES;
    static constexpr int NOP = I8 ? (D == 64 ? 4 : 3) : (D == 64 ? 8 : 6);  // operand stages (8-bit rows: written by the converting warps)
    static constexpr int NRAW = I8 ? (D == 64 ? 8 : 5) : 0;                 // 8-bit stages as copied
    static constexpr int THREADS = 32 * (I8 ? 16 : 12);
    static constexpr int WARP_P = 8, WARP_M = 9, WARP_C = 12;  // producer, MMAs, first converting warp
    // tensor memory columns
    static constexpr int TQ = 0, QCOLS = NP * D / 2;
    static constexpr int SCOLS = NR == 3 ? 96 : 64;  // scores (64), then the weights' parts over them (32 each)
    static constexpr int TS = QCOLS;
    static constexpr int NPV = QCOLS + 2 * SCOLS + 2 * D <= 512 ? 2 : 1;  // product buffers
    static constexpr int TO = TS + 2 * SCOLS;
    static_assert(TO + NPV * D <= 512, "tensor memory");
    // shared memory after the rings: 16 columns of every softmax thread's outputs, m and l of each, the rows' scales
    static constexpr int SCRATCH = 256 * 20 * 4 + 2 * 256 * 4 + 128 * 4;
    static constexpr int NBAR = 2 * NOP + 2 * NRAW + 8 + 4;
    static constexpr size_t fixed() { return 1024 + static_cast<size_t>(NOP) * OSTAGE + static_cast<size_t>(NRAW) * PaLayout<T, D>::STAGE + SCRATCH + NBAR * 8 + 64; }
    // registers per thread of the softmax, of producer and MMA, of the converting warps: as many as are launched
    static constexpr int REG_S = I8 ? 200 : 224, REG_P = 56, REG_C = 56;
    static_assert(I8 ? 256 * REG_S + 128 * REG_P + 128 * REG_C <= 512 * 128 : 256 * REG_S + 128 * REG_P <= 384 * 168, "registers");
};

template <int R>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

template <int T, int D, int C>
__global__ void __launch_bounds__(WideLayout<T, D, C>::THREADS, 1)
    paged_wide_kernel(const PagedArgs a, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    using W = WideLayout<T, D, C>;
    using LY = PaLayout<T, D>;
    constexpr int NP = W::NP, RP = W::RP, NC = W::NC, KS = D / 16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ops = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *raw = ops + static_cast<size_t>(W::NOP) * W::OSTAGE;  // 8-bit rows: the copies' ring
    float *scratch = reinterpret_cast<float *>(raw + static_cast<size_t>(W::NRAW) * LY::STAGE);
    float *sm_m = scratch + 256 * 20, *sm_l = sm_m + 256, *sm_back = sm_l + 256;
    uint64_t *op_full = reinterpret_cast<uint64_t *>(sm_back + 128), *op_empty = op_full + W::NOP;
    uint64_t *raw_full = op_empty + W::NOP, *raw_empty = raw_full + W::NRAW;
    // per group (tile parity), whatever the number of product buffers: a wait knows its phase from the group's own tiles
    uint64_t *s_full = raw_empty + W::NRAW, *p_ready = s_full + 2, *pv_full = p_ready + 2, *pv_free = pv_full + 2;
    uint64_t *q_ready = pv_free + 2, *done = q_ready + 1, *mask_bar = done + 1;
    uint32_t *tbase = reinterpret_cast<uint32_t *>(mask_bar + 2);
    volatile int *abort = reinterpret_cast<volatile int *>(tbase + 1);
    volatile int *last = abort + 1;
    uint32_t *badw = tbase + 4;  // [group][turn][2]: rows of a tile with a NaN or infinity in V
    int64_t *prefix = reinterpret_cast<int64_t *>(tbase + 12);
    int2 *ln = reinterpret_cast<int2 *>(prefix + a.B + 1);
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < W::NOP; ++i) {
            mbar_init(&op_full[i], W::I8 ? 4 : 1);
            mbar_init(&op_empty[i], 1);
        }
        for (int i = 0; i < W::NRAW; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 4);
            mbar_init(&mask_bar[i], 4);
            mbar_init(&pv_full[i], 1);
            mbar_init(&pv_free[i], 4);
        }
        mbar_init(q_ready, 4);
        mbar_init(done, 1);
        *abort = 0;
        for (int i = 0; i < 8; ++i) badw[i] = 0;
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

    if (warp >= 8 && warp < 12) regs_dec<W::REG_P>();
    if (warp == W::WARP_P) {
        if constexpr (W::I8)
            produce_tiles<T, D, RP>(a, sc, &tmk, &tmv, raw, W::NRAW, raw_full, raw_empty, abort);
        else
            produce_tiles<T, D, RP>(a, sc, &tmk, &tmv, ops, W::NOP, op_full, op_empty, abort);
    } else if (warp == W::WARP_M) {
        // ---- the thread that issues the MMAs: tiles are numbered over the whole share
        if (elect_one()) {
            constexpr uint32_t FMT = T == SD_KV_BF16 ? 1u : 0u;
            constexpr uint32_t ID = (1u << 4) | (FMT << 7) | (FMT << 10) | (8u << 24);  // fp32 sums, M = 128
            constexpr uint32_t ID_QK = ID | (PA_KT / 8 << 17), ID_PV = ID | (1u << 16) | (D / 8 << 17);  // B K-major; B MN-major
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
                auto scores = [&]() {
                    if (!wait(&op_full[qk_slot], qk_ph)) return false;
                    tc_fence_after();
                    const uint32_t kb = ob + qk_slot * W::OSTAGE, d = tm + W::TS + (nqk & 1u) * W::SCOLS;
                    bool acc = false;
#pragma unroll
                    for (int x = 0; x < NP; ++x)
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) {
                            tc_mma_ts(d, tm + W::TQ + x * (D / 2) + ks * 8, sw128_desc(kb + (ks >> 2) * W::OTILE + (ks & 3) * 32, 0), ID_QK, acc);
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
                    ok = wait(&p_ready[sb], (npv >> 1) & 1u);
                    if (ok && npv >= W::NPV) ok = wait(&pv_free[(npv - W::NPV) & 1u], ((npv - W::NPV) >> 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t vb = ob + pv_slot * W::OSTAGE + W::OKV, d = tm + W::TO + ob2 * D, pa = tm + W::TS + sb * W::SCOLS;
                    bool acc = false;
#pragma unroll
                    for (int x = 0; x < W::NR; ++x)
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
    } else if (warp >= W::WARP_C) {
        if constexpr (W::I8) {
            regs_dec<W::REG_C>();
            // ---- 8-bit rows to fp16 operands: thread ct takes row ct % 64 of K (ct < 64) or V
            const int ct = tid - 32 * W::WARP_C, row = ct & 63;
            const bool isv = ct >= 64;
            const int64_t tiles = sc.u1 - sc.u0;
            uint32_t rs = 0, rph = 0, os = 0, oph = 0;
            for (int64_t i = 0; i < tiles; ++i) {
                bool ok = mbar_wait_bounded(&raw_full[rs], rph, PA_WAIT_NS, abort);
                if (ok && i >= W::NOP) ok = mbar_wait_bounded(&op_empty[os], oph ^ 1u, PA_WAIT_NS, abort);
                if (!__all_sync(0xffffffffu, ok)) {
                    set_status(a.status, SD_ETIMEOUT);
                    *abort = 1;
                    break;
                }
                const uint8_t *src = raw + static_cast<size_t>(rs) * LY::STAGE;
                uint8_t *dst = ops + static_cast<size_t>(os) * W::OSTAGE + (isv ? W::OKV : 0);
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(src + (isv ? LY::KV : 0) + pa_off<T, D>(row, 16 * x));
                    const uint32_t w[4] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u, v.w ^ 0x80808080u};
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        *reinterpret_cast<uint4 *>(dst + pa_off<SD_KV_F16, D>(row, 32 * x + 16 * y)) =
                            make_uint4(codes2<0, 1>(w[2 * y]), codes2<2, 3>(w[2 * y]), codes2<0, 1>(w[2 * y + 1]), codes2<2, 3>(w[2 * y + 1]));
                }
                const float *ss = reinterpret_cast<const float *>(src + 2 * LY::KV);
                float *ds = reinterpret_cast<float *>(ops + static_cast<size_t>(os) * W::OSTAGE + 2 * W::OKV);
                if (ct < 32) {  // K scales; an infinite one makes a row of NaN
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float s = ss[lane + 32 * y];
                        ds[lane + 32 * y] = s + 0.0f * s;
                    }
                } else if (ct < 64) {  // V scales in units of a power of two that none exceeds
                    float s[2] = {ss[PA_KT + lane], ss[PA_KT + 32 + lane]};
                    int e = -126;
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        if (s[y] > 0.0f && s[y] < INFINITY) {
                            int x;
                            (void)frexpf(s[y], &x);
                            e = max(e, x);
                        }
                    e = __reduce_max_sync(0xffffffffu, e);
                    const float down = ldexpf(1.0f, -e);
                    ds[PA_KT + lane] = s[0] * down;
                    ds[PA_KT + 32 + lane] = s[1] * down;
                    if (lane == 0) ds[2 * PA_KT] = ldexpf(1.0f, e);
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
    } else if (warp < 8) {
        regs_inc<W::REG_S>();
        // ---- softmax: two groups of four warps take the tiles in turn, each with a running state of its own; thread =
        // lane of tensor memory = row lt % RP of the rows, lane group lt / RP
        const int grp = warp >> 2, lt = tid & 127;
        const uint32_t tq = tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const int lg = lt / RP, r = lt % RP;
        const int part = lg % W::CP, k_at = (lg / W::CP) * NC;  // this lane group's part, and its keys of a tile
        int64_t u = sc.u0;
        int b = 0;
        uint32_t base = 0, nsync = 0, nmask = 0;  // tiles before this piece
        bool ok = true;
        auto sync_group = [&]() {  // the group's four warps (an mbarrier: waits that give up)
            __syncwarp();
            if (lane == 0) mbar_arrive(&mask_bar[grp]);
            return __all_sync(0xffffffffu, wait(&mask_bar[grp], nsync++ & 1u)) != 0;
        };
        while (u < sc.u1) {
            const Piece p = piece_at<RP>(a, sc, u, b);
            b = p.b;
            const int rows = p.n * a.g, total = p.len + p.n, tg = p.rg * RP + r;
            const bool real = tg < rows;
            float2 o[D / 2];
            if (grp == 0) {
                // the row's query into tensor memory, in parts; fp16 parts scaled by a power of two as in paged_attn_kernel
                const float4 *qp = reinterpret_cast<const float4 *>(
                    a.q + p.b * a.q_sb + (real ? tg / a.g : 0) * a.q_sm + static_cast<int64_t>(p.kh * a.g + (real ? tg % a.g : 0)) * D);
                float mx = 0.0f;
#pragma unroll
                for (int d = 0; d < D; d += 4) {
                    const float4 f = real ? qp[d / 4] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    o[d / 2] = make_float2(f.x * a.qscale, f.y * a.qscale);
                    o[d / 2 + 1] = make_float2(f.z * a.qscale, f.w * a.qscale);
#pragma unroll
                    for (int e = 0; e < 2; ++e) mx = fmaxf(mx, fmaxf(fabsf(o[d / 2 + e].x), fabsf(o[d / 2 + e].y)));
                }
                float up = 1.0f, down = 1.0f;
                if constexpr (T != SD_KV_BF16) {
                    int ex = 0;
                    if (mx > 0.0f && mx < INFINITY) (void)frexpf(mx, &ex);
                    ex = max(ex, -100);
                    up = ldexpf(1.0f, 11 - ex);
                    down = ldexpf(1.0f, ex - 11);
                }
#pragma unroll
                for (int d = 0; d < D; d += 32) {
                    uint32_t f16[NP][16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const Parts<T> f = split_pair<T>(fmul2_rn(o[d / 2 + e], make_float2(up, up)));
#pragma unroll
                        for (int x = 0; x < NP; ++x) f16[x][e] = f.r[x];
                    }
#pragma unroll
                    for (int x = 0; x < NP; ++x) tc_st(f16[x], tq + W::TQ + x * (D / 2) + d / 2);
                }
                sm_back[lt] = down;  // read by the other group once scores are there
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
            float m = PA_NEG, l = 0.0f, al = 0.0f, unit = 1.0f, back = 1.0f;  // al, unit: rescale of the outputs and unit of the next product
#pragma unroll
            for (int d = 0; d < D / 2; ++d) o[d] = make_float2(0.0f, 0.0f);
            // adds the product of tile number i to the outputs
            auto add_product = [&](uint32_t i) {
                const uint32_t ob2 = i % W::NPV;
                const bool got = wait(&pv_full[grp], (i >> 1) & 1u);
                if (!__all_sync(0xffffffffu, got)) return false;
                tc_fence_after();
                // 32 columns at a time, the next ones on their way
                uint32_t y[2][32];
                tc_ld(y[0], tq + W::TO + ob2 * D);
#pragma unroll
                for (int d = 0; d < D; d += 32) {
                    tc_wait_ld(y[(d / 32) & 1]);
                    if (d + 32 < D) tc_ld(y[(d / 32 + 1) & 1], tq + W::TO + ob2 * D + d + 32);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 f = make_float2(__uint_as_float(y[(d / 32) & 1][2 * e]), __uint_as_float(y[(d / 32) & 1][2 * e + 1]));
                        if constexpr (W::I8) f = fmul2_rn(f, make_float2(unit, unit));
                        o[d / 2 + e] = ffma2_rn(o[d / 2 + e], make_float2(al, al), f);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pv_free[grp]);
                return true;
            };
            const uint32_t n_tiles = static_cast<uint32_t>(p.t1 - p.t0);
            for (uint32_t i = (base & 1u) ^ static_cast<uint32_t>(grp); i < n_tiles; i += 2) {
                const uint32_t nt = base + i, slot = nt % W::NOP, sph = (nt / W::NOP) & 1u;
                const int t = p.t0 + static_cast<int>(i);
                ok = __all_sync(0xffffffffu, wait(&s_full[grp], (nt >> 1) & 1u));
                if (!ok) break;
                tc_fence_after();
                back = sm_back[lt];
                const uint32_t sc_at = tq + W::TS + grp * W::SCOLS;
                const int tile0 = (t < p.st.n_sink ? t : t - p.st.n_sink + p.st.lo_tile) * PA_KT, key0 = tile0 + k_at;
                const uint8_t *stage = ops + static_cast<size_t>(slot) * W::OSTAGE;
                const float *scales = reinterpret_cast<const float *>(stage + 2 * W::OKV);
                const bool whole = tile0 + PA_KT <= p.len && (tile0 >= full_lo || tile0 + PA_KT <= full_sink);
                if (W::I8 || !whole) {  // what stands in the stage is read below: its barrier makes it visible here too
                    ok = __all_sync(0xffffffffu, wait(&op_full[slot], sph));
                    if (!ok) break;
                }
                float tunit = 1.0f;
                if constexpr (W::I8) tunit = scales[2 * PA_KT];
                // 32 scores from the h-th of this thread's keys on: K's scale, and -inf where the row does not see the key
                float2 s[16];
                auto load = [&](int h) {
                    uint32_t y[32];
                    tc_ld(y, sc_at + k_at + h);
                    tc_wait_ld(y);
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[e] = make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1]));
                    if constexpr (W::I8) {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float4 f = *reinterpret_cast<const float4 *>(scales + k_at + h + 2 * e);
                            s[e] = fmul2_rn(s[e], make_float2(f.x, f.y));
                            s[e + 1] = fmul2_rn(s[e + 1], make_float2(f.z, f.w));
                        }
                    }
                    if (!whole) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const int j = key0 + h + e;
                            const bool seen = j >= p.len ? j < total && ((vis >> (j - p.len)) & 1u) != 0
                                                         : j >= low || (j < full_sink && low != INT32_MAX);
                            if (!seen) (e & 1 ? s[e / 2].y : s[e / 2].x) = -INFINITY;
                        }
                    }
                };
                float x4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int h = NC - 32; h >= 0; h -= 32) {  // the first 32 stay in s
                    load(h);
#pragma unroll
                    for (int e = 0; e < 16; ++e) x4[e & 3] = fmaxf(fmaxf(x4[e & 3], s[e].x), s[e].y);
                }
                const float n = fmaxf(m, fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3])) * back);
                const float an = ex2(m - n), off = PW_UP - n;
                m = n;
                bool rescaled = false;
                if constexpr (!W::I8) {
                    if (!whole) {
                        // V rows with a NaN or infinity reach the rows that see them alone: added here, and cleared before the product
                        uint32_t bw[2] = {0, 0};
                        for (int x = lt; x < PA_KT * (2 * D / 16); x += PW_SOFT) {
                            const int vr = x % PA_KT;
                            const uint4 v = *reinterpret_cast<const uint4 *>(stage + W::OKV + pa_off<T, D>(vr, (x / PA_KT) * 16));
                            constexpr uint32_t EX = T == SD_KV_BF16 ? 0x7f80u : 0x7c00u;
                            const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int w = 0; w < 4; ++w)
                                if ((q[w] & EX) == EX || ((q[w] >> 16) & EX) == EX) bw[vr >> 5] |= 1u << (vr & 31);
                        }
                        uint32_t *words = badw + 4 * grp + 2 * (nmask & 1u), *other = badw + 4 * grp + 2 * ((nmask + 1) & 1u);
                        ++nmask;
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            const uint32_t any = __reduce_or_sync(0xffffffffu, bw[w]);
                            if (lane == 0 && any) atomicOr(&words[w], any);
                        }
                        ok = sync_group();
                        if (!ok) break;
                        const uint32_t bad[2] = {*reinterpret_cast<volatile uint32_t *>(&words[0]), *reinterpret_cast<volatile uint32_t *>(&words[1])};
                        if (lt == 0) other[0] = other[1] = 0;  // read by all before the barrier above
                        if (bad[0] | bad[1]) {
#pragma unroll
                            for (int d = 0; d < D / 2; ++d) o[d] = fmul2_rn(o[d], make_float2(an, an));
                            rescaled = true;
                            for (int j = 0; j < PA_KT; ++j) {
                                if (!((bad[j >> 5] >> (j & 31)) & 1u)) continue;
                                uint32_t y;  // this row's weight of key j, from its score once more
                                asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(y) : "r"(sc_at + j) : "memory");
                                asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(y)::"memory");
                                const int jj = tile0 + j;
                                const bool seen = jj >= p.len ? jj < total && ((vis >> (jj - p.len)) & 1u) != 0
                                                              : jj >= low || (jj < full_sink && low != INT32_MAX);
                                const float w = seen && part == 0 && j >= k_at && j < k_at + NC ? ex2(fmaf(__uint_as_float(y), back, off)) : 0.0f;
#pragma unroll
                                for (int d = 0; d < D; ++d) {
                                    const uint16_t h = *reinterpret_cast<const volatile uint16_t *>(stage + W::OKV + pa_off<T, D>(j, 2 * d) + ((2 * d) & 15));
                                    float v;
                                    if constexpr (T == SD_KV_BF16) v = __bfloat162float(__ushort_as_bfloat16(h));
                                    else v = __half2float(__ushort_as_half(h));
                                    if (w > 0.0f) (d & 1 ? o[d / 2].y : o[d / 2].x) += w * v;
                                }
                            }
                            ok = sync_group();
                            if (!ok) break;
                            for (int x = lt; x < PA_KT * (2 * D / 16); x += PW_SOFT) {
                                const int vr = x % PA_KT;
                                if ((bad[vr >> 5] >> (vr & 31)) & 1u)
                                    *reinterpret_cast<uint4 *>(const_cast<uint8_t *>(stage) + W::OKV + pa_off<T, D>(vr, (x / PA_KT) * 16)) = make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async_shared();
                        }
                    }
                }
                // weights in parts, over the scores: 32 keys at a time, the second 32 scores read before parts go over them
                float2 l2[2] = {};
                uint32_t keep[W::NR][16];
                auto weigh = [&](int h) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 x = ffma2_rn(s[e], make_float2(back, back), make_float2(off, off));
                        s[e] = make_float2(ex2(x.x), ex2(x.y));
                        l2[e & 1] = fadd2_rn(l2[e & 1], s[e]);
                    }
                    if constexpr (W::I8) {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float4 f = *reinterpret_cast<const float4 *>(scales + PA_KT + k_at + h + 2 * e);
                            // a key with no weight keeps none, whatever its scale is
                            s[e] = make_float2(s[e].x > 0.0f ? s[e].x * f.x : s[e].x, s[e].y > 0.0f ? s[e].y * f.y : s[e].y);
                            s[e + 1] = make_float2(s[e + 1].x > 0.0f ? s[e + 1].x * f.z : s[e + 1].x, s[e + 1].y > 0.0f ? s[e + 1].y * f.w : s[e + 1].y);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const Parts<T> f = split_pair<T>(s[e]);
                        if constexpr (W::CP == 1) {
#pragma unroll
                            for (int x = 0; x < W::NR; ++x) keep[x][e] = f.r[x];
                        } else {
#pragma unroll
                            for (int x = 0; x < W::NR; ++x) {
                                uint32_t v = 0;
#pragma unroll
                                for (int y = 0; y < NP; ++y) v = x * W::CP + part == y ? f.r[y] : v;
                                keep[x][e] = v;
                            }
                        }
                    }
                };
                weigh(0);
                if constexpr (NC == 64) {
                    tc_st(keep[0], sc_at);  // over the first 32 scores
                    if constexpr (W::NR > 1) {
                        uint32_t held[W::NR][16];
#pragma unroll
                        for (int x = 1; x < W::NR; ++x)
#pragma unroll
                            for (int e = 0; e < 16; ++e) held[x][e] = keep[x][e];
                        load(32);
#pragma unroll
                        for (int x = 1; x < W::NR; ++x) tc_st(held[x], sc_at + x * 32);
                    } else {
                        load(32);
                    }
                    weigh(32);
#pragma unroll
                    for (int x = 0; x < W::NR; ++x) tc_st(keep[x], sc_at + x * 32 + 16);
                } else {
                    uint32_t zero[16];  // the other lane groups' keys weigh nothing in these lanes
#pragma unroll
                    for (int e = 0; e < 16; ++e) zero[e] = 0;
#pragma unroll
                    for (int x = 0; x < W::NR; ++x) {
                        tc_st(keep[x], sc_at + x * 32 + k_at / 2);
                        tc_st(zero, sc_at + x * 32 + 16 - k_at / 2);
                    }
                }
                l = fmaf(l, an, (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y));
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[grp]);
                // this tile's product; the other group's softmax runs meanwhile
                al = rescaled ? 1.0f : an;
                unit = tunit;
                ok = add_product(nt);
                if (!ok) break;
            }
            if (bar_any(1, 256, !ok)) break;  // the eight warps leave together
            base += n_tiles;
            // ---- write the piece: a run that is whole goes out, others become partials
            const bool complete = p.t0 == 0 && p.t1 == p.st.T;
            const int pslot = 2 * static_cast<int>(blockIdx.x) + (p.t0 == 0 ? 1 : 0);
            sm_m[tid] = m;
            sm_l[tid] = l;
            named_bar_sync(1, 256);
            // lane groups that hold parts of the same weights have the same m and l
            float mx = PA_NEG, lv = 0.0f;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int j = 0; j < C; j += W::CP) mx = fmaxf(mx, sm_m[x * 128 + j * RP + r]);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int j = 0; j < C; j += W::CP) lv = fmaf(sm_l[x * 128 + j * RP + r], ex2(sm_m[x * 128 + j * RP + r] - mx), lv);
            const float f = ex2(m - mx) * (!complete ? 1.0f : lv == 0.0f ? 0.0f : 1.0f / lv);
            if (!complete && real && lg == 0 && grp == 0) a.part_ml[pslot * RP + r] = make_float2(mx, lv);
            // 16 columns at a time through shared memory: thread = 4 columns of row tid / 4 (and of the row 64 further on)
            float *to[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int tr = (tid >> 2) + 64 * k, y = p.rg * RP + tr;
                to[k] = tr >= RP || y >= rows ? nullptr
                        : complete ? a.out + p.b * a.o_sb + (y / a.g) * a.o_sm + static_cast<int64_t>(p.kh * a.g + y % a.g) * D + 4 * (tid & 3)
                                   : a.part_o + (static_cast<int64_t>(pslot) * RP + tr) * D + 4 * (tid & 3);
            }
#pragma unroll
            for (int d = 0; d < D; d += 16) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 x = fmul2_rn(o[d / 2 + 2 * e], make_float2(f, f)), y = fmul2_rn(o[d / 2 + 2 * e + 1], make_float2(f, f));
                    *reinterpret_cast<float4 *>(scratch + tid * 20 + 4 * e) = make_float4(x.x, x.y, y.x, y.y);
                }
                named_bar_sync(1, 256);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (to[k]) {
                        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                        for (int j = 0; j < 2 * C; ++j) {
                            const float4 x = *reinterpret_cast<const float4 *>(scratch + (j * RP + (tid >> 2) + 64 * k) * 20 + 4 * (tid & 3));
                            v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
                        }
                        *reinterpret_cast<float4 *>(to[k] + d) = v;
                    }
                named_bar_sync(1, 256);
            }
            if (!complete) {
                const int c0 = cta_of(sc, p.run0), c1 = cta_of(sc, p.run0 + p.st.T - 1);
                __threadfence();
                named_bar_sync(1, 256);
                if (tid == 0) {
                    const int was = atomicAdd(&a.counters[c0], 1);
                    *last = was == c1 - c0;
                    if (was == c1 - c0) a.counters[c0] = 0;
                }
                named_bar_sync(1, 256);
                if (*last) join_partials<RP, D, 256>(a, p, c0, c1, tid);
            }
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
cudaError_t wide_launch_c(const PagedArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv, int rows, int grid, cudaStream_t s) {
    if (rows <= 32) return wide_launch<T, D, 4>(a, tmk, tmv, grid, s);
    if (rows <= 64) return wide_launch<T, D, 2>(a, tmk, tmv, grid, s);
    return wide_launch<T, D, 1>(a, tmk, tmv, grid, s);
}

}  // namespace sdv
