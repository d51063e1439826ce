// sdv_paged_attn.cu - attention of the new rows of a batch of sequences over a cache in pages.
//
// Row i of sequence b (i < n_new[b]) stands at position len[b] + depth(i) and sees
//   the committed rows j < len[b] with j > its position - window (all of them without a window), and
//   the first `sinks` rows, and the new rows on its own path that the same rule lets it see;
// out = softmax(q k^T / sqrt(D)) v over what it sees, query head h reading KV head h / g, g = H / H_kv.
//
// The work of one (sequence, KV head, group of 8 NT query rows) is a run of 64-key tiles (with a window: the
// tiles of the first rows, then those from the window's start on).  All runs laid end to end are cut into
// one equal piece per CTA of a persistent grid, so that lengths that differ balance whatever the batch is, and
// a single long context spreads over the whole GPU.  A run inside one CTA is written out at once; a run cut between
// CTAs leaves (max, sum, unnormalised output) partials in the workspace, and the CTA that arrives last joins
// them in the order of their keys: a counter decides who joins, never in which order, so results repeat.
//
// Inside a CTA: one producer warp, its lanes fetching the tile's pages (a tensor copy per page, K or V and
// 128 bytes of row, 128-byte swizzled) into a ring of 64-key stages that runs ahead over the piece's runs; four
// consumer warps with 16 keys each.  S^T = K Q^T and O^T += V^T P^T on mma m16n8k16 with fp32 accumulation.  The
// fp32 operands are split so that a product keeps about 2^-22 of relative error: into two fp16 parts
// for fp16 and 8-bit rows (codes are exact in fp16; the row scales multiply scores and weights in
// fp32), into three bf16 parts for bf16 rows.  Softmax statistics are fp32 in exp2 units.  A tile's product
// starts from zero and is added to the rescaled outputs by fp32 FMAs: the tensor cores' own accumulation
// truncates, a bias that grows with the tiles (1.2e-5 of the result at 40000 rows against 64 bits).
#include "sdv_paged_attn.cuh"

namespace sdv {

// (Five warps a CTA put three of ten on one scheduler: above 168 registers one CTA runs per SM.  At D = 64 the 16-row
// form is held to that, 162 -> 125 us for 16 sequences of 16000 bf16 rows; at D = 128 it would spill 60 registers and
// take 20 % longer.)
template <int T, int D, int NT>
__global__ void __launch_bounds__(PA_THREADS, D == 64 ? 2 : 0)
    paged_attn_kernel(const PagedArgs a, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv) {
    using LY = PaLayout<T, D>;
    constexpr int KS = D / 16, RPG = 8 * NT, NP = Parts<T>::N, SD = 64 + 4;
    // 16 rows of D = 256: their query fragments do not fit beside the outputs in registers, and all four warps need the
    // same ones
    constexpr bool QSM = D == 256 && NT == 2;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);  // the swizzle wants 1024 B
    // [PA_CW][8][SD]: 64 columns of the warps' outputs
    float *sm_o = reinterpret_cast<float *>(ring + static_cast<size_t>(a.nst) * LY::STAGE);
    float *sm_m = sm_o + PA_CW * 8 * SD, *sm_l = sm_m + PA_CW * RPG;                         // [PA_CW][RPG]
    uint32_t *sm_q = reinterpret_cast<uint32_t *>(sm_l + PA_CW * RPG);  // [NT][KS][2 NP][32]
    uint64_t *full = reinterpret_cast<uint64_t *>(sm_q + (QSM ? NT * KS * 2 * NP * 32 : 0)), *empty = full + a.nst;
    int64_t *prefix = reinterpret_cast<int64_t *>(empty + a.nst);
    int2 *ln = reinterpret_cast<int2 *>(prefix + a.B + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(ln + a.B);
    volatile int *last = abort + 1;
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;

    if (tid == 0) {
        for (int i = 0; i < a.nst; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], PA_CW);
        }
        *abort = 0;
        fence_barrier_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    Sched sc;
    if (!make_sched<RPG, PA_THREADS>(a, prefix, ln, sc)) return;

    if (warp == PA_CW) {
        produce_tiles<T, D, RPG, 0, 1>(a, sc, &tmk, &tmv, ring, a.nst, full, empty, abort);
        return;
    }

    // ---- consumer warps
    const uint32_t sbase = smem_u32(ring);
    // ldmatrix row addresses of this lane: K (keys x d) and, transposed, V
    const int kr = 16 * warp + (lane & 7) + ((lane >> 3) & 1) * 8, kx = (lane >> 4) * 16;
    const int vr = 16 * warp + (lane & 7) + (T == SD_KV_I8 ? ((lane >> 3) & 1) : (lane >> 4)) * 8;
    const int vx = (T == SD_KV_I8 ? (lane >> 4) : ((lane >> 3) & 1)) * 16;
    int64_t u = sc.u0;
    int b = 0, slot = 0;
    uint32_t ph = 0;
    while (u < sc.u1) {
        const Piece p = piece_at<RPG>(a, sc, u, b);
        b = p.b;
        const int rows = p.n * a.g, total = p.len + p.n;
        // B fragments of query row g of each 8-row tile, in parts; fp16 parts of a row scaled by 2^(11-e) for
        // max |q| in [2^(e-1), 2^e), so that neither part is subnormal
        uint32_t qf[QSM ? 1 : NT][QSM ? 1 : KS][2][NP];
        if constexpr (QSM) named_bar_sync(1, 32 * PA_CW);  // the piece before is done with them
        float rs[NT][2];            // the scale back of rows 2c, 2c+1
        uint32_t vis[NT][2];        // new rows that rows 2c, 2c+1 see
        int low[NT][2];             // the first row of their window
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int tg = p.rg * RPG + nt * 8 + g;
            const bool real = tg < rows;
            const int i = real ? tg / a.g : 0, h = p.kh * a.g + (real ? tg % a.g : 0);
            const float *qp = a.q + p.b * a.q_sb + i * a.q_sm + static_cast<int64_t>(h) * D;
            float qv[KS][4];
            float mx = 0.0f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                float2 x, y;
                if constexpr (T == SD_KV_I8) {  // the order in which a word of four codes is unpacked
                    const float4 f = *reinterpret_cast<const float4 *>(qp + 16 * ks + 4 * c);
                    x = make_float2(f.x, f.y);
                    y = make_float2(f.z, f.w);
                } else {
                    x = *reinterpret_cast<const float2 *>(qp + 16 * ks + 2 * c);
                    y = *reinterpret_cast<const float2 *>(qp + 16 * ks + 2 * c + 8);
                }
                qv[ks][0] = real ? x.x * a.qscale : 0.0f;
                qv[ks][1] = real ? x.y * a.qscale : 0.0f;
                qv[ks][2] = real ? y.x * a.qscale : 0.0f;
                qv[ks][3] = real ? y.y * a.qscale : 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(qv[ks][e]));
            }
            float up = 1.0f, back = 1.0f;
            if constexpr (T != SD_KV_BF16) {
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                int ex = 0;
                if (mx > 0.0f && mx < INFINITY) (void)frexpf(mx, &ex);
                ex = max(ex, -100);  // below that the parts may go subnormal: such scores are 0 anyway
                up = ldexpf(1.0f, 11 - ex);
                back = ldexpf(1.0f, ex - 11);
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const Parts<T> f0 = split2<T>(qv[ks][0] * up, qv[ks][1] * up), f1 = split2<T>(qv[ks][2] * up, qv[ks][3] * up);
#pragma unroll
                for (int i2 = 0; i2 < NP; ++i2) {
                    if constexpr (QSM) {
                        if (ks % PA_CW == warp) {
                            sm_q[((nt * KS + ks) * 2 * NP + i2) * 32 + lane] = f0.r[i2];
                            sm_q[((nt * KS + ks) * 2 * NP + NP + i2) * 32 + lane] = f1.r[i2];
                        }
                    } else {
                        qf[nt][ks][0][i2] = f0.r[i2];
                        qf[nt][ks][1][i2] = f1.r[i2];
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                rs[nt][r] = __shfl_sync(0xffffffffu, back, 8 * c + 4 * r);
                const int tr = p.rg * RPG + nt * 8 + 2 * c + r;
                vis[nt][r] = 0;
                low[nt][r] = INT32_MAX;
                if (tr < rows) {
                    int depth;
                    vis[nt][r] = new_rows_seen(a, p.b, tr / a.g, p.len, depth);
                    low[nt][r] = a.window > 0 ? p.len + depth - a.window + 1 : 0;
                }
            }
        }
        if constexpr (QSM) named_bar_sync(1, 32 * PA_CW);
        // a query fragment in its parts
        auto q_of = [&](int nt, int ks, int half, int x) {
            if constexpr (QSM) return sm_q[((nt * KS + ks) * 2 * NP + half * NP + x) * 32 + lane];
            else return qf[nt][ks][half][x];
        };
        float m[NT][2], l[NT][2], o[NT][KS][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = PA_NEG;
            l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
            for (int dt = 0; dt < KS; ++dt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][dt][e] = 0.0f;
        }
        // 8-bit rows: the unit of a row's outputs, a power of two above every V scale that it has seen so far (its bits).
        // One for all rows while they have seen the same scales; after a tile that they see parts of one for each
        // (`apart`, in shared memory): a scale that a row does not see may be of any size, and in a unit above it nothing
        // would be left of the row's weights.  (A unit per row in every tile: 194 -> 219 us, 16 sequences of 8000 rows of
        // D = 256, 16 query rows.)
        uint32_t vunit = 0x00800000u;
        uint32_t *sm_unit = reinterpret_cast<uint32_t *>(sm_m) + warp * RPG;  // (the maxima come there at the piece's end)
        bool apart = false;
        // keys from full_lo on (or below full_sink) and below p.len are seen by every row
        const int full_lo = a.window > 0 ? p.len + p.n - a.window : 0, full_sink = a.window > 0 ? a.sinks : 0;
        bool ok = true;
        for (int t = p.t0; t < p.t1; ++t) {
            const bool ready = mbar_wait_bounded(&full[slot], ph, PA_WAIT_NS, abort);
            if (!__all_sync(0xffffffffu, ready)) {
                if (lane == 0) {
                    set_status(a.status, SD_ETIMEOUT);
                    *abort = 1;
                }
                ok = false;
                break;
            }
            const uint32_t st = sbase + static_cast<uint32_t>(slot) * LY::STAGE;
            const int key0 = (t < p.st.n_sink ? t : t - p.st.n_sink + p.st.lo_tile) * PA_KT;
            float s[NT][4];
            {
                float sa[NT][2][4] = {};  // two accumulator chains (even / odd k step)
#pragma unroll
                for (int k0 = 0; k0 < KS; k0 += (T == SD_KV_I8 ? 2 : 1)) {
                    uint32_t ka[4];
                    pa_ldsm(st + pa_off<T, D>(kr, (T == SD_KV_I8 ? 16 : 32) * k0 + kx), ka);
                    if constexpr (T == SD_KV_I8) {
                        const uint32_t w0 = ka[0] ^ 0x80808080u, w1 = ka[1] ^ 0x80808080u, w2 = ka[2] ^ 0x80808080u,
                                       w3 = ka[3] ^ 0x80808080u;
                        const uint32_t k1[4] = {codes2<0, 1>(w0), codes2<0, 1>(w1), codes2<2, 3>(w0), codes2<2, 3>(w1)};
                        const uint32_t k2[4] = {codes2<0, 1>(w2), codes2<0, 1>(w3), codes2<2, 3>(w2), codes2<2, 3>(w3)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int x = 0; x < NP; ++x) {
                                pa_mma<T>(sa[nt][0], k1, q_of(nt, k0, 0, x), q_of(nt, k0, 1, x));
                                pa_mma<T>(sa[nt][1], k2, q_of(nt, k0 + 1, 0, x), q_of(nt, k0 + 1, 1, x));
                            }
                    } else {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int x = 0; x < NP; ++x)
                                pa_mma<T>(sa[nt][k0 & 1], ka, q_of(nt, k0, 0, x), q_of(nt, k0, 1, x));
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[nt][e] = (sa[nt][0][e] + sa[nt][1][e]) * rs[nt][e & 1];
            }
            const int ja = key0 + 16 * warp + g, jb = ja + 8;  // s[.][0..1]: key ja, rows 2c, 2c+1; s[.][2..3]: key jb
            float vs0 = 1.0f, vs1 = 1.0f;
            if constexpr (T == SD_KV_I8) {
                const float *scales =
                    reinterpret_cast<const float *>(ring + static_cast<size_t>(slot) * LY::STAGE + 2 * LY::KV);
                float ks0 = scales[16 * warp + g], ks1 = scales[16 * warp + g + 8];
                // an infinite scale makes a row of NaN (0 codes times infinity), not a score of -inf
                ks0 += 0.0f * ks0;
                ks1 += 0.0f * ks1;
                vs0 = scales[PA_KT + 16 * warp + g];
                vs1 = scales[PA_KT + 16 * warp + g + 8];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    s[nt][0] *= ks0;
                    s[nt][1] *= ks0;
                    s[nt][2] *= ks1;
                    s[nt][3] *= ks1;
                }
            }
            const bool whole = key0 + PA_KT <= p.len && (key0 >= full_lo || key0 + PA_KT <= full_sink);
            if (!whole) {
                auto seen = [&](int j, int nt, int r) {
                    if (j >= p.len) return j < total && ((vis[nt][r] >> (j - p.len)) & 1u) != 0;
                    return j >= low[nt][r] || (j < full_sink && low[nt][r] != INT32_MAX);
                };
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (!seen(ja, nt, 0)) s[nt][0] = -INFINITY;
                    if (!seen(ja, nt, 1)) s[nt][1] = -INFINITY;
                    if (!seen(jb, nt, 0)) s[nt][2] = -INFINITY;
                    if (!seen(jb, nt, 1)) s[nt][3] = -INFINITY;
                }
            }
            // weights of the keys, running max and sum
            float pr[NT][4], al[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float x0 = fmaxf(s[nt][0], s[nt][2]), x1 = fmaxf(s[nt][1], s[nt][3]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
                    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
                }
                const float n0 = fmaxf(m[nt][0], x0), n1 = fmaxf(m[nt][1], x1);
                const float al0 = exp2f(m[nt][0] - n0), al1 = exp2f(m[nt][1] - n1);
                pr[nt][0] = exp2f(s[nt][0] - n0);
                pr[nt][1] = exp2f(s[nt][1] - n1);
                pr[nt][2] = exp2f(s[nt][2] - n0);
                pr[nt][3] = exp2f(s[nt][3] - n1);
                l[nt][0] = fmaf(l[nt][0], al0, pr[nt][0] + pr[nt][2]);  // this lane's keys; lanes are added at the end
                l[nt][1] = fmaf(l[nt][1], al1, pr[nt][1] + pr[nt][3]);
                m[nt][0] = n0;
                m[nt][1] = n1;
                al[nt][0] = al0;
                al[nt][1] = al1;
            }
            if constexpr (T == SD_KV_I8) {
                const uint32_t t0 = scale_bits(vs0), t1 = scale_bits(vs1);
                if (whole && !apart) {
                    const uint32_t was = vunit;
                    vunit = max(was, unit_above(__reduce_max_sync(0xffffffffu, max(t0, t1))));
                    const float down = unit_inverse(vunit), shrink = __uint_as_float(was) * down;
                    const float vmul0 = vs0 * down, vmul1 = vs1 * down;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        al[nt][0] *= shrink;
                        al[nt][1] *= shrink;
                        pr[nt][0] *= vmul0;
                        pr[nt][1] *= vmul0;
                        pr[nt][2] *= vmul1;
                        pr[nt][3] *= vmul1;
                    }
                } else {
                    uint32_t hi = 0, lo = 0xffffffffu;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            // the largest scale of a key that the row sees (what it does not see scores -inf)
                            uint32_t top = max(s[nt][r] == -INFINITY ? 0u : t0, s[nt][2 + r] == -INFINITY ? 0u : t1);
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
                            const uint32_t was = apart ? sm_unit[nt * 8 + 2 * c + r] : vunit, now = max(was, unit_above(top));
                            __syncwarp();
                            if (g == 0) sm_unit[nt * 8 + 2 * c + r] = now;
                            if (low[nt][r] != INT32_MAX) {
                                hi = max(hi, now);
                                lo = min(lo, now);
                            }
                            const float down = unit_inverse(now);
                            al[nt][r] *= __uint_as_float(was) * down;
                            // a key with no weight keeps none, whatever its scale is
                            if (!(pr[nt][r] == 0.0f)) pr[nt][r] *= vs0 * down;
                            if (!(pr[nt][2 + r] == 0.0f)) pr[nt][2 + r] *= vs1 * down;
                        }
                    __syncwarp();
                    vunit = __reduce_max_sync(0xffffffffu, hi);
                    apart = __reduce_min_sync(0xffffffffu, lo) != vunit;
                }
            }
            const uint32_t vst = st + LY::KV;
            if constexpr (T != SD_KV_I8) {
                if (!whole) {
                    // a row that some query row does not see may hold anything, and 0 times a NaN or infinity is no 0:
                    // such rows are added here, to the query rows that see them alone, and cleared before the product
                    uint32_t bad = 0;
                    for (int i = lane; i < 16 * LY::NB * (LY::ROWB / 16); i += 32) {
                        const int r = i % 16, x = (i / 16) * 16;
                        uint4 v;
                        const uint32_t ad = vst + pa_off<T, D>(16 * warp + r, x);
                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                     : "r"(ad)
                                     : "memory");
                        constexpr uint32_t EX = T == SD_KV_BF16 ? 0x7f80u : 0x7c00u;
                        bool any = false;
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t q = w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
                            any |= (q & EX) == EX || ((q >> 16) & EX) == EX;
                        }
                        if (any) bad |= 1u << r;
                    }
                    bad = __reduce_or_sync(0xffffffffu, bad);
                    if (bad) {  // the rescale that the product below makes otherwise
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                            for (int dt = 0; dt < KS; ++dt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[nt][dt][e] *= al[nt][e & 1];
                            al[nt][0] = al[nt][1] = 1.0f;
                        }
                    }
                    for (uint32_t left = bad; left; left &= left - 1) {
                        const int key = __ffs(left) - 1, src = (key & 7) * 4 + c;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const float w0 = __shfl_sync(0xffffffffu, key < 8 ? pr[nt][0] : pr[nt][2], src);
                            const float w1 = __shfl_sync(0xffffffffu, key < 8 ? pr[nt][1] : pr[nt][3], src);
                            const float f = T == SD_KV_BF16 ? 1.0f : PA_PS;
#pragma unroll
                            for (int dt = 0; dt < KS; ++dt)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const int x = 2 * (16 * dt + g + 8 * e);
                                    uint16_t raw;
                                    asm volatile("ld.shared.u16 %0, [%1];"
                                                 : "=h"(raw)
                                                 : "r"(vst + pa_off<T, D>(16 * warp + key, x) + (x & 15))
                                                 : "memory");
                                    float v;
                                    if constexpr (T == SD_KV_BF16) v = __bfloat162float(__ushort_as_bfloat16(raw));
                                    else v = __half2float(__ushort_as_half(raw));
                                    if (w0 > 0.0f) o[nt][dt][2 * e] += w0 * f * v;
                                    if (w1 > 0.0f) o[nt][dt][2 * e + 1] += w1 * f * v;
                                }
                        }
                        __syncwarp();
                        for (int x = 16 * lane; x < 2 * D; x += 512)
                            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(vst + pa_off<T, D>(16 * warp + key, x)),
                                         "r"(0u)
                                         : "memory");
                        __syncwarp();
                    }
                    if (bad) fence_proxy_async_shared();  // before the stage's next copy
                }
            }
            uint32_t b0[NT][NP], b1[NT][NP];  // the weights as B fragments (keys x rows), in parts
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                constexpr float PS = T == SD_KV_BF16 ? 1.0f : PA_PS;
                const Parts<T> pa = split2<T>(pr[nt][0] * PS, pr[nt][1] * PS), pb = split2<T>(pr[nt][2] * PS, pr[nt][3] * PS);
#pragma unroll
                for (int x = 0; x < NP; ++x) {
                    b0[nt][x] = pa_movm(pa.r[x]);
                    b1[nt][x] = pa_movm(pb.r[x]);
                }
            }
#pragma unroll
            for (int dt = 0; dt < KS; dt += (T == SD_KV_I8 ? 2 : 1)) {
                uint32_t va[4];
                pa_ldsm_t(vst + pa_off<T, D>(vr, (T == SD_KV_I8 ? 16 : 32) * dt + vx), va);
                if constexpr (T == SD_KV_I8) {
                    const uint32_t w0 = va[0] ^ 0x80808080u, w1 = va[1] ^ 0x80808080u, w2 = va[2] ^ 0x80808080u,
                                   w3 = va[3] ^ 0x80808080u;
                    const uint32_t v1[4] = {codes2<0, 2>(w0), codes2<1, 3>(w0), codes2<0, 2>(w1), codes2<1, 3>(w1)};
                    const uint32_t v2[4] = {codes2<0, 2>(w2), codes2<1, 3>(w2), codes2<0, 2>(w3), codes2<1, 3>(w3)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                            float y1[4] = {}, y2[4] = {};
#pragma unroll
                            for (int x = 0; x < NP; ++x) {
                                pa_mma<T>(y1, v1, b0[nt][x], b1[nt][x]);
                                pa_mma<T>(y2, v2, b0[nt][x], b1[nt][x]);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                o[nt][dt][e] = fmaf(o[nt][dt][e], al[nt][e & 1], y1[e]);
                                o[nt][dt + 1][e] = fmaf(o[nt][dt + 1][e], al[nt][e & 1], y2[e]);
                            }
                    }
                } else {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float y[4] = {};
#pragma unroll
                        for (int x = 0; x < NP; ++x) pa_mma<T>(y, va, b0[nt][x], b1[nt][x]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[nt][dt][e] = fmaf(o[nt][dt][e], al[nt][e & 1], y[e]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[slot]);
            if (++slot == a.nst) {
                slot = 0;
                ph ^= 1u;
            }
        }
        if (bar_any(1, 32 * PA_CW, !ok)) return;  // every consumer warp leaves together
        // ---- join the warps' states and write the piece: rows that are whole go out, others become partials
        const bool complete = p.t0 == 0 && p.t1 == p.st.T;
        const int pslot = 2 * static_cast<int>(blockIdx.x) + (p.t0 == 0 ? 1 : 0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float unit[2];
#pragma unroll
            for (int r = 0; r < 2; ++r)
                unit[r] = T == SD_KV_BF16 ? 1.0f
                          : T == SD_KV_I8 ? __uint_as_float(apart ? sm_unit[nt * 8 + 2 * c + r] : vunit) / PA_PS : 1.0f / PA_PS;
            if constexpr (T == SD_KV_I8) __syncwarp();  // read before the maxima come there
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = l[nt][r];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
                if (g == 0) {
                    sm_m[warp * RPG + nt * 8 + 2 * c + r] = m[nt][r];
                    sm_l[warp * RPG + nt * 8 + 2 * c + r] = x;
                }
            }
            const int r = tid >> 4, tr = nt * 8 + r, tg = p.rg * RPG + tr;
            float f[PA_CW], mx = PA_NEG, lv = 0.0f, inv = 0.0f;
#pragma unroll
            for (int cc = 0; cc < D / 64; ++cc) {  // 64 columns at a time
                float *ow = sm_o + warp * 8 * SD;
#pragma unroll
                for (int dx = 0; dx < 4; ++dx) {
                    const int dt = 4 * cc + dx;
                    const int d0 = 16 * dx + (T == SD_KV_I8 ? 2 * g : g), d1 = d0 + (T == SD_KV_I8 ? 1 : 8);
                    ow[(2 * c) * SD + d0] = o[nt][dt][0] * unit[0];
                    ow[(2 * c + 1) * SD + d0] = o[nt][dt][1] * unit[1];
                    ow[(2 * c) * SD + d1] = o[nt][dt][2] * unit[0];
                    ow[(2 * c + 1) * SD + d1] = o[nt][dt][3] * unit[1];
                }
                named_bar_sync(1, 32 * PA_CW);
                if (cc == 0) {
#pragma unroll
                    for (int w = 0; w < PA_CW; ++w) mx = fmaxf(mx, sm_m[w * RPG + tr]);
#pragma unroll
                    for (int w = 0; w < PA_CW; ++w) {
                        f[w] = exp2f(sm_m[w * RPG + tr] - mx);
                        lv = fmaf(sm_l[w * RPG + tr], f[w], lv);
                    }
                    inv = lv == 0.0f ? 0.0f : 1.0f / lv;
                    if (!complete && tg < rows && (tid & 15) == 0) a.part_ml[pslot * RPG + tr] = make_float2(mx, lv);
                }
                if (tg < rows && SD_INB(p.b < a.B && tg / a.g < a.M && p.kh < a.H_kv && (complete || (pslot + 1) * RPG <= a.part_rows),
                                        a.status, 117)) {  // site 117: rows of a piece
                    const int i = tg / a.g, h = p.kh * a.g + tg % a.g, d = 4 * (tid & 15);
                    float *op = complete ? a.out + p.b * a.o_sb + i * a.o_sm + static_cast<int64_t>(h) * D
                                         : a.part_o + (static_cast<int64_t>(pslot) * RPG + tr) * D;
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int w = 0; w < PA_CW; ++w) {
                        const float4 x = *reinterpret_cast<const float4 *>(sm_o + (w * 8 + r) * SD + d);
                        v.x = fmaf(x.x, f[w], v.x);
                        v.y = fmaf(x.y, f[w], v.y);
                        v.z = fmaf(x.z, f[w], v.z);
                        v.w = fmaf(x.w, f[w], v.w);
                    }
                    if (complete) v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                    *reinterpret_cast<float4 *>(op + 64 * cc + d) = v;
                }
                named_bar_sync(1, 32 * PA_CW);
            }
        }
        if (!complete) {
            // the last of the run's CTAs to come here joins their partials, in the order of their keys
            const int c0 = cta_of(sc, p.run0), c1 = cta_of(sc, p.run0 + p.st.T - 1);
            __threadfence();
            named_bar_sync(1, 32 * PA_CW);
            if (tid == 0 && SD_INB(c0 >= 0 && c0 <= c1 && c1 < static_cast<int>(gridDim.x), a.status, 118)) {  // site 118: counter
                const int was = atomicAdd(&a.counters[c0], 1);
                *last = was == c1 - c0;
                if (was == c1 - c0) a.counters[c0] = 0;
            }
            named_bar_sync(1, 32 * PA_CW);
            if (*last) {
                join_partials<RPG, D, 32 * PA_CW>(a, p, c0, c1, tid, sm_o, 1);
            }
        }
        u += p.t1 - p.t0;
    }
}

struct PaPlan {
    int nt, grid, nst;
    size_t smem, off_ml, off_o, total;
};

static size_t pa_stage(int type, int D) {
    return 2 * static_cast<size_t>(PA_KT) * D * kv_type_bytes(type) + (type == SD_KV_I8 ? 1024 : 0);
}

// Rows beside each other in one 8- or 16-row group; a persistent grid of two CTAs per SM, or one where their registers
// or two stages of the ring each do not fit.
static bool pa_plan(int type, int B, int M, int H, int H_kv, int D, PaPlan &p) {
    const int sms = num_sms();
    if (sms < 1) return false;
    const int rows = M * (H / H_kv);
    p.nt = rows > 8 ? 2 : 1;
    const int parts = type == SD_KV_BF16 ? 3 : 2;
    const size_t fixed = 1024 + static_cast<size_t>(PA_CW) * 8 * 68 * 4 + 2 * static_cast<size_t>(PA_CW) * 8 * p.nt * 4 +
                         (D == 256 && p.nt == 2 ? static_cast<size_t>(2) * (D / 16) * 2 * parts * 32 * 4 : 0) +
                         (static_cast<size_t>(B) + 1) * 8 + static_cast<size_t>(B) * 8 + 16;
    const size_t per = pa_stage(type, D) + 16;
    const size_t half = (228 * 1024) / 2 - 1024, whole = 227 * 1024;
    // two CTAs where their registers fit (above) and two stages each do
    int per_sm = D == 256 || (D == 128 && p.nt == 2) ? 1 : 2;
    int64_t n = (static_cast<int64_t>(per_sm == 2 ? half : whole) - static_cast<int64_t>(fixed)) / static_cast<int64_t>(per);
    if (n < 2) {
        per_sm = 1;
        n = (static_cast<int64_t>(whole) - static_cast<int64_t>(fixed)) / static_cast<int64_t>(per);
    }
    p.nst = static_cast<int>(n < 8 ? n : 8);
    p.grid = per_sm * sms;
    p.smem = fixed + per * p.nst;
    return true;
}

// Query rows of a KV head above which the tensor-memory kernel runs: its cost per 64-key tile hardly depends on D or on
// the rows (up to 32 of them), the other's grows with both.  16 sequences of 16000 rows, 8 KV heads, 16 query rows,
// this kernel / the tensor-memory one: D = 64 fp16 100 / 158 us, bf16 125 / 205, int8 117 / 207; D = 128 fp16 184 / 197,
// bf16 246 / 229, int8 221 / 219.  The other's shared memory holds the schedule of PA_WIDE_B sequences; more are two
// launches (this kernel in its place took 2731 us for 513 sequences of 500 rows, 128 query rows; 512 take 510).
constexpr int PA_WIDE_ROWS = 8, PA_WIDE_ROWS_64 = 16, PA_WIDE_B = 512;

static bool pa_wide(int rows, int D) { return rows > (D == 64 ? PA_WIDE_ROWS_64 : PA_WIDE_ROWS) && D <= 128; }

// workspace: counters of the largest grid, then the partials: two per CTA, of 16 rows on two CTAs per SM or
// of 128 rows on one
static size_t pa_workspace(int D, size_t *off_ml, size_t *off_o) {
    const size_t sms = num_sms() > 0 ? num_sms() : 0;
    if (!sms) return 0;
    const size_t rows = sms * 2 * 128;  // 4 x 16 rows per SM take less
    const size_t ml = (2 * sms * 4 + 255) / 256 * 256, o = ml + (rows * 8 + 255) / 256 * 256;
    if (off_ml) *off_ml = ml;
    if (off_o) *off_o = o;
    return o + rows * static_cast<size_t>(D) * 4;
}

// K or V pages as a 4-d tensor (x = element of a row, y = row in its page, z = KV head, w = page): boxes of
// up to 64 rows of one page by 128 bytes, zeros for a page past the last
static bool pages_map(CUtensorMap *tm, const sd_kv_pages *p, void *base) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const int eb = kv_type_bytes(p->type);
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(p->D), static_cast<cuuint64_t>(p->page_rows),
                                static_cast<cuuint64_t>(p->H_kv), static_cast<cuuint64_t>(p->n_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(p->row_stride) * eb, static_cast<cuuint64_t>(p->head_stride) * eb,
                                   static_cast<cuuint64_t>(p->page_stride) * eb};
    const int rowb = p->D * eb < 128 ? p->D * eb : 128;
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(rowb / eb),
                               static_cast<cuuint32_t>(p->page_rows < PA_KT ? p->page_rows : PA_KT), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUtensorMapDataType dt = p->type == SD_KV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                   : p->type == SD_KV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    return enc(tm, dt, 4, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               rowb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int T, int D, int NT>
static cudaError_t pa_launch(const PaPlan &p, const PagedArgs &a, const CUtensorMap &tmk, const CUtensorMap &tmv,
                             cudaStream_t s) {
    const cudaError_t e = allow_max_dynamic_smem(paged_attn_kernel<T, D, NT>);
    if (e != cudaSuccess) return e;
    return launch(paged_attn_kernel<T, D, NT>, dim3(p.grid), dim3(PA_THREADS), p.smem, s, a, tmk, tmv);
}
template <int T>
static cudaError_t pa_launch_d(int D, const PaPlan &p, const PagedArgs &a, const CUtensorMap &tmk,
                               const CUtensorMap &tmv, cudaStream_t s) {
    if (D == 256) return p.nt == 1 ? pa_launch<T, 256, 1>(p, a, tmk, tmv, s) : pa_launch<T, 256, 2>(p, a, tmk, tmv, s);
    if (D == 128) return p.nt == 1 ? pa_launch<T, 128, 1>(p, a, tmk, tmv, s) : pa_launch<T, 128, 2>(p, a, tmk, tmv, s);
    return p.nt == 1 ? pa_launch<T, 64, 1>(p, a, tmk, tmv, s) : pa_launch<T, 64, 2>(p, a, tmk, tmv, s);
}

}  // namespace sdv

using namespace sdv;

extern "C" {

size_t sd_paged_attn_workspace_bytes(int32_t B, int32_t M, int32_t H, int32_t H_kv, int32_t D) {
    if (B < 1 || B > PG_MAX_B || M < 1 || M > 16 || H_kv < 1 || H < H_kv || H % H_kv || (D != 64 && D != 128 && D != 256))
        return 0;
    return pa_workspace(D, nullptr, nullptr);
}

sd_status sd_paged_attn(const sd_kv_pages *pages, const int32_t *table, int32_t width, const int32_t *lens,
                        const int32_t *n_new, int32_t B, int32_t M, int32_t H, const float *q, int64_t q_seq_stride,
                        int64_t q_row_stride, const int32_t *parent, int32_t window, int32_t sinks, float *out,
                        int64_t out_seq_stride, int64_t out_row_stride, void *workspace, size_t ws_bytes,
                        sd_stream_t stream) {
    SD_NVTX("sd_paged_attn");
    const sd_status st = pages_check(pages);
    if (st != SD_OK) return st;
    const int H_kv = pages->H_kv, D = pages->D;
    if (!table || !lens || !q || !out || !workspace || width < 1) return SD_EINVAL;
    if (B < 1 || M < 1 || H < H_kv || H % H_kv || window < 0 || sinks < 0) return SD_EINVAL;
    if (M > 16 || B > PG_MAX_B) return SD_EUNSUPPORTED;
    const int64_t line = static_cast<int64_t>(H) * D;
    if (q_row_stride < line || out_row_stride < line || q_row_stride % 4 || out_row_stride % 4 ||
        q_seq_stride % 4 || out_seq_stride % 4)
        return SD_EINVAL;
    if (B > 1 && (q_seq_stride < line || out_seq_stride < line)) return SD_EINVAL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256)) return SD_EINVAL;
    // positions are 32-bit
    if (static_cast<int64_t>(width) * pages->page_rows > INT32_MAX - 2 * PA_KT) return SD_EUNSUPPORTED;
    PaPlan p;
    size_t off_ml, off_o;
    const size_t need = pa_workspace(D, &off_ml, &off_o);
    if (!need || !pa_plan(pages->type, B, M, H, H_kv, D, p)) return SD_ECUDA;
    if (ws_bytes < need) return SD_EINVAL;
    CUtensorMap tmk, tmv;
    if (!pages_map(&tmk, pages, pages->k) || !pages_map(&tmv, pages, pages->v)) return SD_ECUDA;
    int *status = status_ptr();
    if (!status) return SD_ECUDA;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    PagedArgs a = {};
    a.q = q;
    a.out = out;
    a.table = table;
    a.lens = lens;
    a.n_new = n_new;
    a.parent = parent;
    a.k_scale = pages->k_scale;
    a.v_scale = pages->v_scale;
    a.q_sb = q_seq_stride;
    a.q_sm = q_row_stride;
    a.o_sb = out_seq_stride;
    a.o_sm = out_row_stride;
    a.B = B;
    a.M = M;
    a.H = H;
    a.H_kv = H_kv;
    a.g = H / H_kv;
    a.P = pages->page_rows;
    a.n_pages = pages->n_pages;
    a.width = width;
    a.window = window;
    a.sinks = sinks;
    a.nst = p.nst;
    a.qscale = 1.4426950408889634f / sqrtf(static_cast<float>(D));
    a.counters = reinterpret_cast<int32_t *>(ws);
    a.part_rows = static_cast<int32_t>((need - off_o) / (static_cast<size_t>(D) * 4));
    a.part_ml = reinterpret_cast<float2 *>(ws + off_ml);
    a.part_o = reinterpret_cast<float *>(ws + off_o);
    a.status = status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int rows = M * a.g;
    if (pa_wide(rows, D)) {
        const auto run = pages->type == SD_KV_F16 ? paged_wide_f16
                         : pages->type == SD_KV_BF16 ? paged_wide_bf16
                                                      : paged_wide_i8;
        const int part = B <= PA_WIDE_B ? B : (B + 1) / 2;
        static_assert(PG_MAX_B <= 2 * PA_WIDE_B, "two launches hold the most sequences");
        for (int b0 = 0; b0 < B; b0 += part) {
            a.B = B - b0 < part ? B - b0 : part;
            a.table = table + static_cast<int64_t>(b0) * width;
            a.lens = lens + b0;
            a.n_new = n_new ? n_new + b0 : nullptr;
            a.parent = parent ? parent + static_cast<int64_t>(b0) * M : nullptr;
            a.q = q + b0 * q_seq_stride;
            a.out = out + b0 * out_seq_stride;
            if (run(a, tmk, tmv, D, rows, num_sms(), s) != cudaSuccess) return SD_ECUDA;
        }
        return SD_OK;
    }
    const cudaError_t e = pages->type == SD_KV_F16    ? pa_launch_d<SD_KV_F16>(D, p, a, tmk, tmv, s)
                          : pages->type == SD_KV_BF16 ? pa_launch_d<SD_KV_BF16>(D, p, a, tmk, tmv, s)
                                                      : pa_launch_d<SD_KV_I8>(D, p, a, tmk, tmv, s);
    return e == cudaSuccess ? SD_OK : SD_ECUDA;
}

}  // extern "C"
