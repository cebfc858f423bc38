// Backward of the selective scan (lizard_scan_bwd).
//
// With e = dy silu(z), a = exp(d A) and G[t] the gradient of h[t]:
//   G[t] = Cm[t] e[t] + a[t+1] G[t+1],   q[t] = a[t] G[t] h[t-1]
//   dBm[t, n] = sum_c G d x,   dCm[t, n] = sum_c e h,   dA = sum_t q d,
//   gb = sum_n G Bm,   dx = d gb + D e,   dd = x gb + sum_n q A,   ddt = dd sigmoid(dt + bias),
//   dz = dy (sum_n Cm h + D x) silu'(z),   dh0 = a[first] G[first].
//
// A CTA of 128 threads owns a block of channels (lanes and states as in the forward) and walks a
// segment backwards, 16 tokens at a time from the state the forward kept at their start: the
// second eight tokens' states are recomputed into registers and walked backwards, then the first
// eight's.  The decays are computed again on the way back, which costs less than holding them.
// Sums over states go over a channel's lanes, sums over channels over the other lanes and then
// over the CTA's warps in shared memory; the CTA's part of dBm and dCm, of dA, dD and ddt_bias
// goes to the workspace and is added in a fixed order.
#include <type_traits>

#include "scan.cuh"

namespace lz {
namespace scan {
namespace {

constexpr int HB = CK / 2;  // tokens whose states are held at once

template <int LPC>
struct Lay {
    static constexpr int CPT = LPC >= 4 ? 2 : 1;  // channels a thread
    static constexpr int LC = 32 / LPC;
    static constexpr int CH = NT / 32 * LC * CPT;
    static constexpr int NP = NS * LPC;
    static constexpr int NV = CH / 8;
    static constexpr int PX = (CK * NV + NT - 1) / NT;
    static constexpr int PB = (CK * (NP + 7) / 8 + NT - 1) / NT;
    static constexpr int OS = CH + 8;  // row stride of the outputs' tiles
};

template <int LPC>
struct Smem {
    using L = Lay<LPC>;
    float2 dx[CK][L::CH];  // d, d x
    float e[CK][L::CH];
    float2 b[CK][2][LPC], c[CK][2][LPC];
    float gb[CK][L::OS], qa[CK][L::OS], ch[CK][L::OS];  // sums over states
    float bc[NT / 32][CK][2][L::NP];                    // a warp's sums over channels
};

template <typename T, int LPC>
__global__ void __launch_bounds__(NT) scan_bwd_kernel(const ScanArgs a, const Cut cut,
                                                      const float* rec_g, float* pbc, float* pA,
                                                      float* pD, float* pbias) {
    using L = Lay<LPC>;
    constexpr int CPT = L::CPT, LC = L::LC, CH = L::CH, NP = L::NP, NV = L::NV, PX = L::PX, PB = L::PB;
    constexpr int NQ = (NP + 7) / 8;
    constexpr bool FAST = is_fast<T>();
    extern __shared__ __align__(16) unsigned char smraw[];
    Smem<LPC>& sm = *reinterpret_cast<Smem<LPC>*>(smraw);
    const Where<CH> w(a, cut);
    check_offsets(a.seqs, a.header);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int q = lane & (LPC - 1), cl = lane / LPC;
    const int N = (int)a.N, nn = max(0, min(NS, N - NS * q));
    const bool v4 = N % 4 == 0;
    const int64_t t0 = w.seg * cut.seg_len, t1 = min64(t0 + cut.seg_len, a.seqs.L);
    const int64_t row0 = w.b * a.seqs.L, C = a.C, nck = (a.seqs.L + CK - 1) / CK;
    const int lch = warp * (LC * CPT) + cl;  // channel k of this thread: lch + k LC

    float A2[CPT][NS], dA[CPT][NS], gn[CPT][NS];
    int64_t ch[CPT];
    bool own[CPT];
    auto load_state = [&](const float* p, float (*f)[NS]) {  // p: [C, N] or null
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
#pragma unroll
            for (int i = 0; i < NS; ++i) f[k][i] = 0.0f;
            if (p != nullptr && own[k]) load4(p + ch[k] * N + NS * q, nn, v4, f[k]);
        }
    };
    auto put_state = [&](float* p, float (*f)[NS]) {
#pragma unroll
        for (int k = 0; k < CPT; ++k)
            if (own[k]) store4(p + ch[k] * N + NS * q, nn, v4, f[k]);
    };
    auto seq_state = [&](const float* p, int64_t seq) { return p == nullptr ? p : p + seq * C * N; };
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        ch[k] = w.c0 + lch + k * LC;
        own[k] = ch[k] < w.clim;
    }
    load_state(a.A, A2);
#pragma unroll
    for (int k = 0; k < CPT; ++k)
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            A2[k][i] *= kLog2e;
            dA[k][i] = 0.0f;
        }
    // gn: the gradient that reaches the state after a token from later ones
    SeqAt sq = seq_at(a.seqs, w.b, t1 - 1);
    if (t1 == sq.end) load_state(seq_state(a.dh_out, sq.seq), gn);
    else load_state(rec_g + (w.b * cut.segs + w.seg) * C * N, gn);

    const bool vec = C % 8 == 0 && (C / a.G) % 8 == 0 && a.ldx % 8 == 0 && a.lddt % 8 == 0 &&
                     a.ldz % 8 == 0 && a.ldy % 8 == 0 && a.lddx % 8 == 0 && a.ldddt % 8 == 0 &&
                     a.lddz % 8 == 0;
    const bool vecb = N % 8 == 0 && a.ldb % 8 == 0 && a.ldc % 8 == 0;
    const int pc = tid % NV * 8, pt = tid / NV;
    const int64_t pch = w.c0 + pc;
    const int pn = (int)max64(0, min64(8, w.clim - pch));
    constexpr int DT = NT / NV;
    float sD[8], sbias[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sD[j] = sbias[j] = 0.0f;

    auto step = [&](int tl, float (*h)[NS]) {  // the recurrence, one token on
        const float2 b0 = sm.b[tl][0][q], b1 = sm.b[tl][1][q];
        const float bb[4] = {b0.x, b0.y, b1.x, b1.y};
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const float2 d = sm.dx[tl][lch + k * LC];
#pragma unroll
            for (int i = 0; i < NS; ++i) h[k][i] = fmaf(ex2(d.x * A2[k][i]), h[k][i], d.y * bb[i]);
        }
    };

    for (int64_t tt = t0 + (t1 - 1 - t0) / CK * CK; tt >= t0; tt -= CK) {
        Raw<T> rx[PX], rdt[PX], rz[PX], rdy[PX];
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            const int tl = pt + i * DT;
            const int n = tl < CK && tt + tl < t1 ? pn : 0;
            const int64_t r = row0 + tt + tl;
            rx[i].load((const T*)a.x + r * a.ldx + pch, n, vec);
            rdt[i].load((const T*)a.dt + r * a.lddt + pch, n, vec);
            rdy[i].load((const T*)a.dy + r * a.ldy + pch, n, vec);
            if (a.z != nullptr) rz[i].load((const T*)a.z + r * a.ldz + pch, n, vec);
        }
        float hs[CPT][NS];  // the state before the chunk
        load_state(a.states + (w.b * nck + tt / CK) * C * N, hs);
        __syncthreads();  // the last chunk's tiles have been read
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int e = tid + i * NT, tl = e / NQ, n0 = e % NQ * 8;
            if (tl >= CK) break;
            const int n = tt + tl < t1 ? max(0, min(8, N - n0)) : 0;
            const int64_t r = row0 + tt + tl;
            Raw<T> v;
            float f[8];
            v.load((const T*)a.Bm + r * a.ldb + w.grp * N + n0, n, vecb);
            v.get(f);
#pragma unroll
            for (int j = 0; j < 8 && j < NP; j += 2)
                sm.b[tl][j / 2 % 2][(n0 + j) / 4] = make_float2(f[j], f[j + 1]);
            v.load((const T*)a.Cm + r * a.ldc + w.grp * N + n0, n, vecb);
            v.get(f);
#pragma unroll
            for (int j = 0; j < 8 && j < NP; j += 2)
                sm.c[tl][j / 2 % 2][(n0 + j) / 4] = make_float2(f[j], f[j + 1]);
        }
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            const int tl = pt + i * DT;
            if (tl >= CK) break;
            const bool live = tt + tl < t1;
            float fx[8], fd[8], fe[8], fz[8];
            rx[i].get(fx);
            rdt[i].get(fd);
            rdy[i].get(fe);
            if (a.z != nullptr) rz[i].get(fz);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = fd[j] + (a.dt_bias != nullptr && j < pn ? a.dt_bias[pch + j] : 0.0f);
                // a place past the segment's end must leave the state and its gradient as they are
                const float d = live ? (a.softplus ? softplus_(v) : v) : 0.0f;
                sm.dx[tl][pc + j] = make_float2(d, d * fx[j]);
                sm.e[tl][pc + j] = a.z != nullptr ? fe[j] * (fz[j] * sigm<FAST>(fz[j])) : fe[j];
            }
        }
        __syncthreads();
#pragma unroll 1
        for (int half = 1; half >= 0; --half) {
            const int l0 = half * HB;
            if (tt + l0 >= t1) continue;
            float h[CPT][NS], hist[HB][CPT][NS];
#pragma unroll
            for (int k = 0; k < CPT; ++k)
#pragma unroll
                for (int i = 0; i < NS; ++i) h[k][i] = hs[k][i];
            // whether a sequence begins among the chunk's tokens up to the half's end
            const bool plain = sq.begin < tt;
            auto enter = [&](int64_t t) {  // the state before token t
                const SeqAt s = seq_at(a.seqs, w.b, t);
                if (s.begin == t) load_state(seq_state(a.h0, s.seq), h);
            };
            for (int tl = 0; tl < l0; ++tl) {
                if (!plain) enter(tt + tl);
                step(tl, h);
            }
            float hb0[CPT][NS];  // the state before the half
#pragma unroll
            for (int k = 0; k < CPT; ++k)
#pragma unroll
                for (int i = 0; i < NS; ++i) hb0[k][i] = h[k][i];
#pragma unroll
            for (int u = 0; u < HB; ++u) {
                if (!plain && tt + l0 + u < t1) enter(tt + l0 + u);
                step(l0 + u, h);
#pragma unroll
                for (int k = 0; k < CPT; ++k)
#pragma unroll
                    for (int i = 0; i < NS; ++i) hist[u][k][i] = h[k][i];
            }
#pragma unroll
            for (int u4 = HB - 4; u4 >= 0; u4 -= 4) {
                float pgb[4][CPT], pqa[4][CPT], pch[4][CPT];
#pragma unroll
                for (int u3 = 3; u3 >= 0; --u3) {
                    const int u = u4 + u3, tl = l0 + u;
                    const int64_t t = tt + tl;
                    const float2 b0 = sm.b[tl][0][q], b1 = sm.b[tl][1][q];
                    const float2 c0 = sm.c[tl][0][q], c1 = sm.c[tl][1][q];
                    const float bb[4] = {b0.x, b0.y, b1.x, b1.y}, cc[4] = {c0.x, c0.y, c1.x, c1.y};
                    const bool first = !plain && t == sq.begin && t < t1;
                    float hp[CPT][NS];
#pragma unroll
                    for (int k = 0; k < CPT; ++k)
#pragma unroll
                        for (int i = 0; i < NS; ++i) hp[k][i] = u > 0 ? hist[u > 0 ? u - 1 : 0][k][i] : hb0[k][i];
                    if (first) load_state(seq_state(a.h0, sq.seq), hp);
                    float v[8];  // dBm, dCm of this lane's states, over its channels
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
#pragma unroll
                    for (int k = 0; k < CPT; ++k) {
                        const float2 d = sm.dx[tl][lch + k * LC];
                        const float e = sm.e[tl][lch + k * LC];
                        float gb = 0.0f, qa = 0.0f, cs = 0.0f;
#pragma unroll
                        for (int i = 0; i < NS; ++i) {
                            const float g = fmaf(cc[i], e, gn[k][i]);
                            const float ag = ex2(d.x * A2[k][i]) * g;
                            const float qq = ag * hp[k][i];
                            gn[k][i] = ag;
                            dA[k][i] = fmaf(qq, d.x, dA[k][i]);
                            qa = fmaf(qq, A2[k][i], qa);
                            gb = fmaf(g, bb[i], gb);
                            cs = fmaf(cc[i], hist[u][k][i], cs);
                            v[i] = fmaf(g, d.y, v[i]);
                            v[4 + i] = fmaf(e, hist[u][k][i], v[4 + i]);
                        }
                        pgb[u3][k] = gb;
                        pqa[u3][k] = qa;
                        pch[u3][k] = cs;
                    }
                    if (first) {
                        if (a.dh0 != nullptr) put_state(a.dh0 + sq.seq * C * N, gn);
                        if (t > t0) {
                            sq = seq_at(a.seqs, w.b, t - 1);
                            load_state(seq_state(a.dh_out, sq.seq), gn);
                        }
                    }
                    // over the lanes with the same states: each stage hands half of the values
                    // over, and a lane ends with one (or, with few such lanes, some) of the eight
                    int at = 0, cnt = 8;
#pragma unroll
                    for (int o = LPC; o < 32; o *= 2) {
                        const bool up = lane & o;
                        if (cnt > 1) {
                            cnt /= 2;
#pragma unroll
                            for (int i = 0; i < cnt; ++i) {
                                const float send = up ? v[i] : v[cnt + i], keep = up ? v[cnt + i] : v[i];
                                v[i] = keep + __shfl_xor_sync(~0u, send, o);
                            }
                            at += up ? cnt : 0;
                        } else {
                            v[0] += __shfl_xor_sync(~0u, v[0], o);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < cnt; ++i)
                        if (LPC >= 4 || cl < 8) sm.bc[warp][tl][(at + i) / 4][NS * q + (at + i) % 4] = v[i];
                }
                // over a channel's lanes, four tokens together; a lane keeps one token of four
                auto put = [&](float (*p)[CPT], float* o) {
#pragma unroll
                    for (int k = 0; k < CPT; ++k) {
                        float* y = o + k * LC;
                        if constexpr (LPC == 1) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) y[i * L::OS] = p[i][k];
                        } else {
                            const bool b0 = q & 1;
                            float u = b0 ? p[1][k] : p[0][k], v = b0 ? p[3][k] : p[2][k];
                            u += __shfl_xor_sync(~0u, b0 ? p[0][k] : p[1][k], 1);
                            v += __shfl_xor_sync(~0u, b0 ? p[2][k] : p[3][k], 1);
                            if constexpr (LPC == 2) {
                                y[(q & 1) * L::OS] = u;
                                y[(2 + (q & 1)) * L::OS] = v;
                            } else {
                                const bool b1 = q & 2;
                                float s = b1 ? v : u;
                                s += __shfl_xor_sync(~0u, b1 ? u : v, 2);
#pragma unroll
                                for (int x = 4; x < LPC; x *= 2) s += __shfl_xor_sync(~0u, s, x);
                                if (q < 4) y[(q & 3) * L::OS] = s;
                            }
                        }
                    }
                };
                put(pgb, &sm.gb[l0 + u4][lch]);
                put(pqa, &sm.qa[l0 + u4][lch]);
                if (a.z != nullptr) put(pch, &sm.ch[l0 + u4][lch]);
            }
        }
        __syncthreads();
        // the CTA's part of dBm and dCm
        float* o = pbc + (((w.cb % cut.cbg) * a.B * a.seqs.L + row0 + tt) * a.G + w.grp) * 2 * N;
        for (int e = tid; e < CK * 2 * NP; e += NT) {
            const int tl = e / (2 * NP), m = e / NP % 2, n = e % NP;
            if (tt + tl >= t1 || n >= N) continue;
            float s = sm.bc[0][tl][m][n];
#pragma unroll
            for (int k = 1; k < NT / 32; ++k) s += sm.bc[k][tl][m][n];
            o[((int64_t)tl * a.G * 2 + m) * N + n] = s;
        }
        // the gradients of x, dt and z
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            const int tl = pt + i * DT;
            if (tl >= CK) break;
            const int n = tt + tl < t1 ? pn : 0;
            float fx[8], fd[8], fy[8], fz[8], ox[8], ot[8], oz[8];
            rx[i].get(fx);
            rdt[i].get(fd);
            rdy[i].get(fy);
            if (a.z != nullptr) rz[i].get(fz);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float D = a.D != nullptr && j < n ? a.D[pch + j] : 0.0f;
                const float d = sm.dx[tl][pc + j].x, e = sm.e[tl][pc + j], gb = sm.gb[tl][pc + j];
                ox[j] = fmaf(d, gb, D * e);
                // qa was summed with A log2(e)
                float dd = fmaf(fx[j], gb, sm.qa[tl][pc + j] * 0.69314718055994531f);
                if (a.softplus) {
                    const float v = fd[j] + (a.dt_bias != nullptr && j < n ? a.dt_bias[pch + j] : 0.0f);
                    dd *= sigm<FAST>(v);
                }
                ot[j] = dd;
                if (j < n) {
                    sD[j] = fmaf(e, fx[j], sD[j]);
                    sbias[j] += dd;
                }
                if (a.z != nullptr) {
                    const float sg = sigm<FAST>(fz[j]);
                    oz[j] = fy[j] * fmaf(D, fx[j], sm.ch[tl][pc + j]) * dsilu(fz[j], sg);
                }
            }
            const int64_t r = row0 + tt + tl;
            store8((T*)a.dx + r * a.lddx + pch, ox, n, vec);
            store8((T*)a.ddt + r * a.ldddt + pch, ot, n, vec);
            if (a.z != nullptr) store8((T*)a.dz + r * a.lddz + pch, oz, n, vec);
        }
    }
    // the CTA's part of dA, dD and ddt_bias
    const int64_t part = w.b * cut.segs + w.seg;
    put_state(pA + part * C * N, dA);
    __syncthreads();
    float* red = reinterpret_cast<float*>(smraw);  // [2][DT][CH]
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        red[pt * CH + pc + j] = sD[j];
        red[(DT + pt) * CH + pc + j] = sbias[j];
    }
    __syncthreads();
    for (int e = tid; e < 2 * CH; e += NT) {
        const int c = e % CH, m = e / CH;
        if (w.c0 + c >= w.clim) continue;
        float s = 0.0f;
        for (int k = 0; k < DT; ++k) s += red[(m * DT + k) * CH + c];
        (m == 0 ? pD : pbias)[part * C + w.c0 + c] = s;
    }
}

// A segment's own contribution to the gradient of the state before it: sum over its tokens of
// (the decays up to and with the token) Cm e, up to the first place where a sequence ends; and
// the sum of its step sizes (NaN where a sequence begins in it, whose decays let nothing pass).
template <typename T, int LPC>
__global__ void __launch_bounds__(NT) scan_adj_kernel(const ScanArgs a, const Cut cut, float* rec_g,
                                                      float* rec_d) {
    using L = Lay<LPC>;
    constexpr int CPT = L::CPT, LC = L::LC, CH = L::CH, NP = L::NP, NV = L::NV, PX = L::PX, PB = L::PB;
    constexpr int NQ = (NP + 7) / 8, DT = NT / NV;
    constexpr bool FAST = is_fast<T>();
    __shared__ float2 sde[CK][CH];  // d, e
    __shared__ float2 sc[CK][2][LPC];
    const Where<CH> w(a, cut);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int q = lane & (LPC - 1), lch = warp * (LC * CPT) + lane / LPC;
    const int N = (int)a.N, nn = max(0, min(NS, N - NS * q));
    const bool v4 = N % 4 == 0;
    const int64_t t0 = w.seg * cut.seg_len, t1 = min64(t0 + cut.seg_len, a.seqs.L);
    const int64_t row0 = w.b * a.seqs.L, C = a.C;
    float A2[CPT][NS], p[CPT][NS], acc[CPT][NS], sd[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        const int64_t c = w.c0 + lch + k * LC;
        if (c < w.clim) load4(a.A + c * N + NS * q, nn, v4, f);
        sd[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            A2[k][i] = f[i] * kLog2e;
            p[k][i] = 1.0f;
            acc[k][i] = 0.0f;
        }
    }
    const SeqAt sq = seq_at(a.seqs, w.b, t0);
    const bool vec = C % 8 == 0 && (C / a.G) % 8 == 0 && a.lddt % 8 == 0 && a.ldz % 8 == 0 && a.ldy % 8 == 0;
    const bool vecb = N % 8 == 0 && a.ldc % 8 == 0;
    const int pc = tid % NV * 8, pt = tid / NV;
    const int64_t pch = w.c0 + pc;
    const int pn = (int)max64(0, min64(8, w.clim - pch));
    // a segment that begins a sequence hands nothing on
    const int64_t stop = sq.begin == t0 ? t0 : min64(t1, sq.end);
    for (int64_t tt = t0; tt < stop; tt += CK) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            const int tl = pt + i * DT;
            if (tl >= CK) break;
            const bool live = tt + tl < stop;
            const int64_t r = row0 + tt + tl;
            Raw<T> v;
            float fd[8], fe[8], fz[8];
            v.load((const T*)a.dt + r * a.lddt + pch, live ? pn : 0, vec);
            v.get(fd);
            v.load((const T*)a.dy + r * a.ldy + pch, live ? pn : 0, vec);
            v.get(fe);
            if (a.z != nullptr) {
                v.load((const T*)a.z + r * a.ldz + pch, live ? pn : 0, vec);
                v.get(fz);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = fd[j] + (a.dt_bias != nullptr && j < pn ? a.dt_bias[pch + j] : 0.0f);
                const float d = live ? (a.softplus ? softplus_(x) : x) : 0.0f;
                sde[tl][pc + j] = make_float2(d, a.z != nullptr ? fe[j] * (fz[j] * sigm<FAST>(fz[j])) : fe[j]);
            }
        }
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int e = tid + i * NT, tl = e / NQ, n0 = e % NQ * 8;
            if (tl >= CK) break;
            Raw<T> v;
            float f[8];
            v.load((const T*)a.Cm + (row0 + tt + tl) * a.ldc + w.grp * N + n0,
                   tt + tl < stop ? max(0, min(8, N - n0)) : 0, vecb);
            v.get(f);
#pragma unroll
            for (int j = 0; j < 8 && j < NP; j += 2)
                sc[tl][j / 2 % 2][(n0 + j) / 4] = make_float2(f[j], f[j + 1]);
        }
        __syncthreads();
#pragma unroll 4
        for (int tl = 0; tl < CK; ++tl) {
            const float2 c0 = sc[tl][0][q], c1 = sc[tl][1][q];
            const float cc[4] = {c0.x, c0.y, c1.x, c1.y};
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const float2 d = sde[tl][lch + k * LC];
                sd[k] += d.x;
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    p[k][i] *= ex2(d.x * A2[k][i]);
                    acc[k][i] = fmaf(p[k][i], cc[i] * d.y, acc[k][i]);
                }
            }
        }
    }
    const bool ends = stop > t0 && stop == sq.end;
    const int64_t rec = (w.b * cut.segs + w.seg) * C;
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int64_t c = w.c0 + lch + k * LC;
        if (c >= w.clim) continue;
        if (ends && a.dh_out != nullptr) {
            float g[4];
            load4(a.dh_out + (sq.seq * C + c) * N + NS * q, nn, v4, g);
#pragma unroll
            for (int i = 0; i < NS; ++i) acc[k][i] = fmaf(p[k][i], g[i], acc[k][i]);
        }
        store4(rec_g + (rec + c) * N + NS * q, nn, v4, acc[k]);
        if (q == 0) rec_d[rec + c] = stop < t1 || ends ? __int_as_float(0x7fc00000) : sd[k];
    }
}

// Joins the segments of a row from the last: the gradient of the state after each, in place.
__global__ void __launch_bounds__(256) scan_adj_join_kernel(const ScanArgs a, int64_t segs, float* rec_g,
                                                            const float* rec_d) {
    const int64_t CN = a.C * a.N, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= a.B * CN) return;
    const int64_t b = id / CN, cn = id % CN, c = cn / a.N;
    const float A2 = a.A[cn] * kLog2e;
    float g = 0.0f;
    for (int64_t s = segs - 1; s >= 0; --s) {
        float* p = rec_g + (b * segs + s) * CN + cn;
        const float own = *p, d = rec_d[(b * segs + s) * a.C + c];
        *p = g;
        g = isnan(d) ? own : fmaf(ex2(d * A2), g, own);
    }
}

// dBm and dCm: the sums over a group's channel blocks.
template <typename T>
__global__ void __launch_bounds__(256) scan_bc_kernel(const ScanArgs a, int64_t cbg, const float* pbc) {
    const int64_t rows = a.B * a.seqs.L, width = a.G * 2 * a.N, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= rows * width) return;
    const int64_t row = id / width, g = id % width / (2 * a.N), m = id / a.N % 2, n = id % a.N;
    float s = 0.0f;
#pragma unroll 8
    for (int64_t k = 0; k < cbg; ++k) s += pbc[k * rows * width + id];
    if (m == 0) st((T*)a.dBm + row * a.lddb + g * a.N + n, s);
    else st((T*)a.dCm + row * a.lddc + g * a.N + n, s);
}

__global__ void __launch_bounds__(256) scan_bwd_empty_kernel(const ScanArgs a) {
    const int64_t CN = a.C * a.N, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= a.nstate * CN) return;
    int64_t end;
    if (seq_tokens(a.seqs, id / CN, &end) > 0) return;
    a.dh0[id] = a.dh_out != nullptr ? a.dh_out[id] : 0.0f;
}

template <int LPC = 1, typename F>
cudaError_t with_lanes(int l, F&& f) {
    if constexpr (LPC > 16) return cudaErrorInvalidValue;
    else return l == LPC ? f(std::integral_constant<int, LPC>()) : with_lanes<LPC * 2>(l, f);
}

Cut bwd_cut(const ScanArgs& a) {
    const int lanes = lanes_for(a.N), ch = NT / lanes * (lanes >= 4 ? 2 : 1);
    Cut k;
    k.cbg = (a.C / a.G + ch - 1) / ch;
    k.cblocks = k.cbg * a.G;
    k.segs = 1;
    k.seg_len = a.seqs.L;
    const int64_t ctas = a.B * k.cblocks;
    if (ctas >= 304 || a.seqs.L <= SEG) return k;
    const int64_t want = (3 * 152 + ctas - 1) / ctas;
    k.seg_len = ((a.seqs.L + want - 1) / want + SEG - 1) / SEG * SEG;
    k.segs = (a.seqs.L + k.seg_len - 1) / k.seg_len;
    return k;
}

struct BwdWs {
    size_t rec_g, rec_d, bc, A, D, bias, total;
};
BwdWs bwd_ws(const ScanArgs& a, const Cut& k) {
    BwdWs o;
    const size_t parts = (size_t)(a.B * k.segs), CN = (size_t)(a.C * a.N);
    auto up = [](size_t n) { return (n + 3) & ~(size_t)3; };
    size_t at = 0;
    o.rec_g = at, at += k.segs > 1 ? up(parts * CN) : 0;
    o.rec_d = at, at += k.segs > 1 ? up(parts * a.C) : 0;
    o.bc = at, at += up((size_t)(k.cbg * a.B * a.seqs.L * a.G * 2 * a.N));
    o.A = at, at += up(parts * CN);
    o.D = at, at += up(parts * a.C);
    o.bias = at, at += up(parts * a.C);
    o.total = at;
    return o;
}

template <typename T>
cudaError_t scan_bwd(const ScanArgs& a, cudaStream_t s) {
    const Cut k = bwd_cut(a);
    const BwdWs o = bwd_ws(a, k);
    float* f = a.ws;
    const int64_t CN = a.C * a.N;
    cudaError_t e = cudaSuccess;
    if (a.dh0 != nullptr && (a.seqs.cu != nullptr || a.seqs.L == 0))
        scan_bwd_empty_kernel<<<(unsigned)((a.nstate * CN + 255) / 256), 256, 0, s>>>(a);
    int64_t parts = 0;
    if (a.seqs.L > 0) {
        parts = a.B * k.segs;
        e = with_lanes(lanes_for(a.N), [&](auto ll) {
            constexpr int LPC = decltype(ll)::value;
            const unsigned g = (unsigned)(parts * k.cblocks);
            if (k.segs > 1) {
                scan_adj_kernel<T, LPC><<<g, NT, 0, s>>>(a, k, f + o.rec_g, f + o.rec_d);
                scan_adj_join_kernel<<<(unsigned)((a.B * CN + 255) / 256), 256, 0, s>>>(a, k.segs, f + o.rec_g, f + o.rec_d);
            }
            const int bytes = (int)sizeof(Smem<LPC>);
            cudaError_t r = cudaFuncSetAttribute(scan_bwd_kernel<T, LPC>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (r != cudaSuccess) return r;
            scan_bwd_kernel<T, LPC><<<g, NT, bytes, s>>>(a, k, f + o.rec_g, f + o.bc, f + o.A, f + o.D, f + o.bias);
            const int64_t n = a.B * a.seqs.L * a.G * 2 * a.N;
            scan_bc_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a, k.cbg, f + o.bc);
            return cudaGetLastError();
        });
        if (e != cudaSuccess) return e;
    }
    e = launch_sum_partials(f + o.A, parts, CN, a.dA, CN, s);
    if (e == cudaSuccess && a.dD != nullptr) e = launch_sum_partials(f + o.D, parts, a.C, a.dD, a.C, s);
    if (e == cudaSuccess && a.ddt_bias != nullptr)
        e = launch_sum_partials(f + o.bias, parts, a.C, a.ddt_bias, a.C, s);
    return e;
}

}  // namespace
}  // namespace scan

size_t scan_bwd_ws_floats(const ScanArgs& a) { return scan::bwd_ws(a, scan::bwd_cut(a)).total; }

cudaError_t launch_scan_bwd(const ScanArgs& a, cudaStream_t s) {
    return a.dtype == LIZARD_BF16 ? scan::scan_bwd<__nv_bfloat16>(a, s) : scan::scan_bwd<float>(a, s);
}

}  // namespace lz
