// sdv_paged_wide.cuh - the attention over pages for many query rows per KV head (a tree of drafts, grouped
// heads): the same work, cut, masks and partials as paged_attn_kernel, on the 5th-generation tensor cores.
//
// The rows of one (sequence, KV head) are the 128 lanes of tensor memory.  With at most 64 (32) of them the lanes hold
// C = 2 (4) copies of the rows, and copy j weighs keys [j 64/C, (j+1) 64/C) of each 64-key tile alone: the softmax of a
// tile spreads over all four warps, and the copies join at the end of a piece as the splits of a run do.
//   S = Q K^T: tcgen05.mma kind::f16, M = 128, N = 64, Q in tensor memory as A (written once per piece, in 16-bit parts
//     that add up to the fp32 value: two fp16, or three bf16), K as B from shared memory as the tensor copy left it
//     (K-major, 128-byte swizzle);
//   softmax: one thread per lane, so a row's maximum and sum need no exchange; the weights go back to tensor memory
//     over the scores, in parts;
//   O_t = P V: the weights as A, V as B (MN-major, the same swizzle), from zero for each tile; the softmax threads add
//     it to their fp32 outputs in registers with the rescale of the running maximum (a tensor-core accumulator kept
//     over the tiles would truncate at every step, and rescaling it would cost the same loads and more stores).
// One thread issues all MMAs: scores two tiles ahead of the weights, so the tensor cores work while the softmax of
// the tile between runs.  8-bit rows pass through four more warps that write them as fp16 into operand
// buffers (exact) and their scales beside them.
//
// What bounds it: at 128 rows of D = 128 a 64-key fp16 tile is 32 KB of HBM (about 1400 SM cycles of one SM's share)
// against 4 x 128 x 64 x 128 multiply-adds (about 1050 cycles) and 64 weights a thread.
#pragma once

#include "sdv_paged_attn.cuh"

namespace sdv {

constexpr int PW_SOFT = 128;   // softmax threads (warps 0..3: the four lane quarters of tensor memory)
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
    static constexpr int NC = PA_KT / C;            // keys of a tile that a thread weighs
    static constexpr int OTILE = PA_KT * 128;       // 64 keys x 64 halves
    static constexpr int OKV = D / 64 * OTILE;      // K (or V) operand of a tile
    static constexpr int OSCALES = I8 ? 1024 : 0;   // scales of K [64], of V [64] in units of the tile's, that unit
    static constexpr int OSTAGE = 2 * OKV + OSCALES;
    static constexpr int NOP = I8 ? 3 : (D == 64 ? 8 : 6);  // operand stages (8-bit rows: written by the converting warps)
    static constexpr int NRAW = I8 ? (D == 64 ? 8 : 5) : 0; // 8-bit stages as copied
    static constexpr int THREADS = 32 * (I8 ? 12 : 6);
    // tensor memory columns
    static constexpr int TQ = 0, QCOLS = NP * D / 2;
    static constexpr int SCOLS = NP == 3 ? 96 : 64;  // scores (64), then the weights' parts over them (32 each)
    static constexpr int TS = QCOLS;
    static constexpr int NPV = T == SD_KV_BF16 && D == 128 ? 1 : 2;  // product buffers
    static constexpr int TO = TS + 2 * SCOLS;
    static_assert(TO + NPV * D <= 512, "tensor memory");
    // shared memory after the rings: join scratch [128][33] floats, m and l [128] each
    static constexpr int SCRATCH = 128 * 33 * 4 + 2 * 128 * 4;
    static constexpr int NBAR = 2 * NOP + 2 * NRAW + 2 + 2 + 2 * NPV + 2;
    static constexpr size_t fixed() { return 1024 + static_cast<size_t>(NOP) * OSTAGE + static_cast<size_t>(NRAW) * PaLayout<T, D>::STAGE + SCRATCH + NBAR * 8 + 64; }
};

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
    float *sm_m = scratch + 128 * 33, *sm_l = sm_m + 128;
    uint64_t *op_full = reinterpret_cast<uint64_t *>(sm_l + 128), *op_empty = op_full + W::NOP;
    uint64_t *raw_full = op_empty + W::NOP, *raw_empty = raw_full + W::NRAW;
    uint64_t *s_full = raw_empty + W::NRAW, *p_ready = s_full + 2, *pv_full = p_ready + 2, *pv_free = pv_full + W::NPV;
    uint64_t *q_ready = pv_free + W::NPV, *done = q_ready + 1;
    uint32_t *tbase = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tbase + 1);
    volatile int *last = abort + 1;
    uint32_t *badw = tbase + 4;  // [2][2]: rows of a tile with a NaN or infinity in V
    int64_t *prefix = reinterpret_cast<int64_t *>(tbase + 8);
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
        }
        for (int i = 0; i < W::NPV; ++i) {
            mbar_init(&pv_full[i], 1);
            mbar_init(&pv_free[i], 4);
        }
        mbar_init(q_ready, 4);
        mbar_init(done, 1);
        *abort = 0;
        for (int i = 0; i < 4; ++i) badw[i] = 0;
        fence_barrier_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    Sched sc;
    if (!make_sched<RP, W::THREADS>(a, prefix, ln, sc)) return;
    if (warp == 5) {
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

    // 8-bit rows: 384 threads of 160 registers or more are launched; 128 x (240 + 104 + 136) are used
    if (W::I8 && warp >= 4 && warp < 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 4) {
        if constexpr (W::I8)
            produce_tiles<T, D, RP>(a, sc, &tmk, &tmv, raw, W::NRAW, raw_full, raw_empty, abort);
        else
            produce_tiles<T, D, RP>(a, sc, &tmk, &tmv, ops, W::NOP, op_full, op_empty, abort);
    } else if (warp == 5) {
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
                    if (ok && npv >= W::NPV) ok = wait(&pv_free[ob2], (npv / W::NPV - 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t vb = ob + pv_slot * W::OSTAGE + W::OKV, d = tm + W::TO + ob2 * D, pa = tm + W::TS + sb * W::SCOLS;
                    bool acc = false;
#pragma unroll
                    for (int x = 0; x < NP; ++x)
#pragma unroll
                        for (int ks = 0; ks < PA_KT / 16; ++ks) {
                            tc_mma_ts(d, pa + x * 32 + ks * 8, sw128_desc(vb + ks * 2048, W::OTILE), ID_PV, acc);
                            acc = true;
                        }
                    tc_commit(&pv_full[ob2]);
                    tc_commit(&op_empty[pv_slot]);
                    ++npv;
                    if (++pv_slot == W::NOP) pv_slot = 0;
                    // the scores of tile i + 2 go where the weights of tile i are: after their product
                    if (i + 2 < n) ok = wait(&pv_full[ob2], ((npv - 1) / W::NPV) & 1u) && scores();
                }
                u += n;
            }
            tc_commit(done);  // no MMA is left when the tensor memory goes
            (void)mbar_wait_bounded(done, 0, PA_WAIT_NS);
        }
        __syncwarp();
    } else if (warp >= 8) {
        if constexpr (W::I8) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 136;");
            // ---- 8-bit rows to fp16 operands: thread ct takes row ct % 64 of K (ct < 64) or V
            const int ct = tid - 256, row = ct & 63;
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
                if (warp == 8) {  // K scales; an infinite one makes a row of NaN
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float s = ss[lane + 32 * y];
                        ds[lane + 32 * y] = s + 0.0f * s;
                    }
                } else if (warp == 9) {  // V scales in units of a power of two that none exceeds
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
    } else if (warp < 4) {
        if constexpr (W::I8) asm volatile("setmaxnreg.inc.sync.aligned.u32 240;");
        // ---- softmax: thread = lane of tensor memory = row tid % RP of the group, copy tid / RP
        const uint32_t tq = tm + (static_cast<uint32_t>(32 * warp) << 16);
        const int copy = tid / RP, r = tid % RP;
        int64_t u = sc.u0;
        int b = 0;
        uint32_t nt = 0, npv = 0, slot = 0, sph = 0, nmask = 0;
        bool ok = true, gone = false;
        // a barrier of the four warps; false: one of them has given up, and all leave at this very barrier
        auto meet = [&]() {
            gone = bar_any(1, PW_SOFT, false);
            return !gone;
        };
        while (u < sc.u1) {
            const Piece p = piece_at<RP>(a, sc, u, b);
            b = p.b;
            const int rows = p.n * a.g, total = p.len + p.n, tg = p.rg * RP + r;
            const bool real = tg < rows;
            float o[D];
            // the row's query into tensor memory, in parts; fp16 parts scaled by a power of two as in paged_attn_kernel
            float back = 1.0f;
            {
                const float4 *qp = reinterpret_cast<const float4 *>(
                    a.q + p.b * a.q_sb + (real ? tg / a.g : 0) * a.q_sm + static_cast<int64_t>(p.kh * a.g + (real ? tg % a.g : 0)) * D);
                float mx = 0.0f;
#pragma unroll
                for (int d = 0; d < D; d += 4) {
                    const float4 f = real ? qp[d / 4] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    o[d] = f.x * a.qscale;
                    o[d + 1] = f.y * a.qscale;
                    o[d + 2] = f.z * a.qscale;
                    o[d + 3] = f.w * a.qscale;
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(o[d + e]));
                }
                float up = 1.0f;
                if constexpr (T != SD_KV_BF16) {
                    int ex = 0;
                    if (mx > 0.0f && mx < INFINITY) (void)frexpf(mx, &ex);
                    ex = max(ex, -100);
                    up = ldexpf(1.0f, 11 - ex);
                    back = ldexpf(1.0f, ex - 11);
                }
#pragma unroll
                for (int d = 0; d < D; d += 32) {
                    uint32_t part[NP][16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const Parts<T> f = split2<T>(o[d + 2 * e] * up, o[d + 2 * e + 1] * up);
#pragma unroll
                        for (int x = 0; x < NP; ++x) part[x][e] = f.r[x];
                    }
#pragma unroll
                    for (int x = 0; x < NP; ++x) tc_st(part[x], tq + W::TQ + x * (D / 2) + d / 2);
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
            float m = PA_NEG, l = 0.0f, al = 0.0f, unit = 1.0f;  // al, unit: rescale and unit of the product still to be added
#pragma unroll
            for (int d = 0; d < D; ++d) o[d] = 0.0f;
            // adds the product of the tile before to the outputs
            auto add_product = [&]() {
                const uint32_t ob2 = npv % W::NPV;
                const bool got = wait(&pv_full[ob2], (npv / W::NPV) & 1u);
                if (!__all_sync(0xffffffffu, got)) return false;
                tc_fence_after();
#pragma unroll
                for (int d = 0; d < D; d += 32) {
                    uint32_t y[32];
                    tc_ld(y, tq + W::TO + ob2 * D + d);
                    tc_wait_ld(y);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float f = __uint_as_float(y[e]);
                        o[d + e] = fmaf(o[d + e], al, W::I8 ? f * unit : f);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pv_free[ob2]);
                ++npv;
                return true;
            };
            for (int t = p.t0; ok && t < p.t1; ++t) {
                const uint32_t sb = nt & 1u;
                ok = __all_sync(0xffffffffu, wait(&s_full[sb], (nt >> 1) & 1u));
                if (!ok) break;
                tc_fence_after();
                const uint32_t sc_at = tq + W::TS + sb * W::SCOLS;
                float s[NC];
                if constexpr (NC == 16) {
                    uint32_t y[16];
                    tc_ld(y, sc_at + copy * NC);
                    tc_wait_ld(y);
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[e] = __uint_as_float(y[e]);
                } else {
#pragma unroll
                    for (int h = 0; h < NC; h += 32) {
                        uint32_t y[32];
                        tc_ld(y, sc_at + copy * NC + h);
                        tc_wait_ld(y);
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[h + e] = __uint_as_float(y[e]);
                    }
                }
                const int key0 = (t < p.st.n_sink ? t : t - p.st.n_sink + p.st.lo_tile) * PA_KT + copy * NC;  // this thread's first
                const uint8_t *stage = ops + static_cast<size_t>(slot) * W::OSTAGE;
                const float *scales = reinterpret_cast<const float *>(stage + 2 * W::OKV);
                float tunit = 1.0f;
                if constexpr (W::I8) {
                    // the operand barrier makes the converting warps' scales visible here too
                    ok = __all_sync(0xffffffffu, wait(&op_full[slot], sph));
                    if (!ok) break;
#pragma unroll
                    for (int e = 0; e < NC; e += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(scales + copy * NC + e);
                        s[e] *= f.x;
                        s[e + 1] *= f.y;
                        s[e + 2] *= f.z;
                        s[e + 3] *= f.w;
                    }
                    tunit = scales[2 * PA_KT];
                }
                const int tile0 = key0 - copy * NC;
                const bool whole = tile0 + PA_KT <= p.len && (tile0 >= full_lo || tile0 + PA_KT <= full_sink);
                if (!whole) {
#pragma unroll
                    for (int e = 0; e < NC; ++e) {
                        const int j = key0 + e;
                        const bool seen = j >= p.len ? j < total && ((vis >> (j - p.len)) & 1u) != 0
                                                     : j >= low || (j < full_sink && low != INT32_MAX);
                        if (!seen) s[e] = -INFINITY;
                    }
                }
                float x4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int e = 4; e < NC; ++e) x4[e & 3] = fmaxf(x4[e & 3], s[e]);
                const float n = fmaxf(m, fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3])) * back);
                const float an = ex2(m - n), off = PW_UP - n;
                m = n;
                float l4[4] = {};
#pragma unroll
                for (int e = 0; e < NC; ++e) {
                    s[e] = ex2(fmaf(s[e], back, off));
                    l4[e & 3] += s[e];
                }
                l = fmaf(l, an, (l4[0] + l4[1]) + (l4[2] + l4[3]));
                if constexpr (W::I8) {
#pragma unroll
                    for (int e = 0; e < NC; e += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(scales + PA_KT + copy * NC + e);
                        // a key with no weight keeps none, whatever its scale is
                        s[e] = s[e] > 0.0f ? s[e] * f.x : s[e];
                        s[e + 1] = s[e + 1] > 0.0f ? s[e + 1] * f.y : s[e + 1];
                        s[e + 2] = s[e + 2] > 0.0f ? s[e + 2] * f.z : s[e + 2];
                        s[e + 3] = s[e + 3] > 0.0f ? s[e + 3] * f.w : s[e + 3];
                    }
                } else if (!whole) {
                    // V rows with a NaN or infinity reach the rows that see them alone: added here, and cleared before the product
                    ok = __all_sync(0xffffffffu, wait(&op_full[slot], sph));  // the copy's writes, seen by these threads too
                    if (!ok) break;
                    uint32_t bw[2] = {0, 0};
                    for (int i = tid; i < PA_KT * (2 * D / 16); i += PW_SOFT) {
                        const int vr = i % PA_KT, x = (i / PA_KT) * 16;
                        const uint4 v = *reinterpret_cast<const uint4 *>(stage + W::OKV + pa_off<T, D>(vr, x));
                        constexpr uint32_t EX = T == SD_KV_BF16 ? 0x7f80u : 0x7c00u;
                        const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            if ((q[w] & EX) == EX || ((q[w] >> 16) & EX) == EX) bw[vr >> 5] |= 1u << (vr & 31);
                    }
                    uint32_t *words = badw + 2 * (nmask & 1u);
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const uint32_t any = __reduce_or_sync(0xffffffffu, bw[w]);
                        if (lane == 0 && any) atomicOr(&words[w], any);
                    }
                    ok = meet();
                    if (!ok) break;
                    uint32_t bad[2] = {*reinterpret_cast<volatile uint32_t *>(&words[0]), *reinterpret_cast<volatile uint32_t *>(&words[1])};
                    if (tid == 0) badw[2 * ((nmask + 1) & 1u)] = badw[2 * ((nmask + 1) & 1u) + 1] = 0;  // every thread has read it: the barrier above
                    ++nmask;
                    if (bad[0] | bad[1]) {
                        if (t > p.t0) {
                            ok = add_product();
                            if (!ok) break;
                        }
#pragma unroll
                        for (int d = 0; d < D; ++d) o[d] *= an;
                        for (int j = 0; j < PA_KT; ++j) {
                            if (!((bad[j >> 5] >> (j & 31)) & 1u)) continue;
                            float w = 0.0f;  // this thread's weight of key j
#pragma unroll
                            for (int e = 0; e < NC; ++e) w = j == copy * NC + e ? s[e] : w;
#pragma unroll
                            for (int d = 0; d < D; ++d) {
                                const uint16_t h = *reinterpret_cast<const volatile uint16_t *>(stage + W::OKV + pa_off<T, D>(j, 2 * d) + ((2 * d) & 15));
                                float v;
                                if constexpr (T == SD_KV_BF16) v = __bfloat162float(__ushort_as_bfloat16(h));
                                else v = __half2float(__ushort_as_half(h));
                                if (w > 0.0f) o[d] += w * v;
                            }
                        }
                        ok = meet();
                        if (!ok) break;
                        for (int i = tid; i < PA_KT * (2 * D / 16); i += PW_SOFT) {
                            const int vr = i % PA_KT, x = (i / PA_KT) * 16;
                            if ((bad[vr >> 5] >> (vr & 31)) & 1u)
                                *reinterpret_cast<uint4 *>(const_cast<uint8_t *>(stage) + W::OKV + pa_off<T, D>(vr, x)) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_shared();
                    }
                    if (bad[0] | bad[1]) al = -1.0f;  // the rescale is done
                }
                // the weights in parts over the scores; the other copies' keys weigh nothing in these lanes
#pragma unroll
                for (int h = 0; h < NC; h += (NC < 32 ? NC : 32)) {
                    constexpr int HW = (NC < 32 ? NC : 32) / 2;
                    uint32_t part[NP][HW];
#pragma unroll
                    for (int e = 0; e < HW; ++e) {
                        const Parts<T> f = split2<T>(s[h + 2 * e], s[h + 2 * e + 1]);
#pragma unroll
                        for (int x = 0; x < NP; ++x) part[x][e] = f.r[x];
                    }
#pragma unroll
                    for (int x = 0; x < NP; ++x) tc_st(part[x], sc_at + x * 32 + (copy * NC + h) / 2);
                }
                if constexpr (C > 1) {
                    uint32_t zero[NC / 2];
#pragma unroll
                    for (int e = 0; e < NC / 2; ++e) zero[e] = 0;
#pragma unroll
                    for (int x = 0; x < NP; ++x)
#pragma unroll
                        for (int j = 1; j < C; ++j) tc_st(zero, sc_at + x * 32 + ((copy + j) % C) * (NC / 2));
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[sb]);
                if (al < 0.0f) {
                    al = 1.0f;
                } else {
                    if (t > p.t0) {
                        ok = add_product();
                        if (!ok) break;
                    }
                    al = an;
                }
                unit = tunit;
                ++nt;
                if (++slot == W::NOP) {
                    slot = 0;
                    sph ^= 1u;
                }
            }
            if (ok) ok = add_product();
            if (gone || bar_any(1, PW_SOFT, !ok)) break;  // the four warps leave together
            // ---- write the piece: a run that is whole goes out, others become partials
            const bool complete = p.t0 == 0 && p.t1 == p.st.T;
            const int pslot = 2 * static_cast<int>(blockIdx.x) + (p.t0 == 0 ? 1 : 0);
            float *base = complete ? a.out + p.b * a.o_sb : a.part_o + static_cast<int64_t>(pslot) * RP * D;
            auto row_at = [&](int tr) {
                const int x = p.rg * RP + tr;
                return complete ? base + (x / a.g) * a.o_sm + static_cast<int64_t>(p.kh * a.g + x % a.g) * D : base + static_cast<int64_t>(tr) * D;
            };
            if constexpr (C == 1) {
                if (real) {
                    const float inv = !complete ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
                    float4 *op = reinterpret_cast<float4 *>(row_at(r));
#pragma unroll
                    for (int d = 0; d < D; d += 4) op[d / 4] = make_float4(o[d] * inv, o[d + 1] * inv, o[d + 2] * inv, o[d + 3] * inv);
                    if (!complete) a.part_ml[pslot * RP + r] = make_float2(m, l);
                }
            } else {
                sm_m[tid] = m;
                sm_l[tid] = l;
                named_bar_sync(1, PW_SOFT);
                float mx = PA_NEG, lv = 0.0f;
#pragma unroll
                for (int j = 0; j < C; ++j) mx = fmaxf(mx, sm_m[j * RP + r]);
#pragma unroll
                for (int j = 0; j < C; ++j) lv = fmaf(sm_l[j * RP + r], ex2(sm_m[j * RP + r] - mx), lv);
                const float f = ex2(m - mx) * (!complete ? 1.0f : lv == 0.0f ? 0.0f : 1.0f / lv);
                if (!complete && real && copy == 0) a.part_ml[pslot * RP + r] = make_float2(mx, lv);
#pragma unroll
                for (int d = 0; d < D; d += 32) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) scratch[tid * 33 + e] = o[d + e] * f;
                    named_bar_sync(1, PW_SOFT);
                    for (int i = tid; i < RP * 32; i += PW_SOFT) {
                        const int tr = i / 32, e = i % 32;
                        if (p.rg * RP + tr < rows) {
                            float v = scratch[tr * 33 + e];
#pragma unroll
                            for (int j = 1; j < C; ++j) v += scratch[(j * RP + tr) * 33 + e];
                            row_at(tr)[d + e] = v;
                        }
                    }
                    named_bar_sync(1, PW_SOFT);
                }
            }
            if (!complete) {
                const int c0 = cta_of(sc, p.run0), c1 = cta_of(sc, p.run0 + p.st.T - 1);
                __threadfence();
                named_bar_sync(1, PW_SOFT);
                if (tid == 0) {
                    const int was = atomicAdd(&a.counters[c0], 1);
                    *last = was == c1 - c0;
                    if (was == c1 - c0) a.counters[c0] = 0;
                }
                named_bar_sync(1, PW_SOFT);
                if (*last) join_partials<RP, D, PW_SOFT>(a, p, c0, c1, tid);
            }
            u += p.t1 - p.t0;
        }
    }
    // ---- every role is done
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
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
