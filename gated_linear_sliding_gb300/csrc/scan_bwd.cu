// Backward of the selective scan (lizard_scan_bwd).
//
// With e = dy silu(z), a = exp(d A) and G[t] the gradient of h[t]:
//   G[t] = Cm[t] e[t] + a[t+1] G[t+1],   q[t] = a[t] G[t] h[t-1]
//   dBm[t, n] = sum_c G d x,   dCm[t, n] = sum_c e h,   dA = sum_t q d,
//   gb = sum_n G Bm,   dx = d gb + D e,   dd = x gb + sum_n q A,   ddt = dd sigmoid(dt + bias),
//   dz = dy (sum_n Cm h + D x) silu'(z),   dh0 = a[first] G[first].
//
// A CTA of 128 threads owns a block of channels and walks a segment backwards, 16 tokens at a time
// from the state the forward kept at their start: one walk forward leaves the states before each
// four tokens in shared memory, then four tokens at a time, from the last, are walked forward
// again into registers and backwards.  The decays are computed again on the way back, which costs
// less than holding them.  A thread holds four states of two channels.
//
// What bounds it is the number of instructions, and of those a third are the sums that cross
// lanes: over states (three values a token and channel) and over channels (dBm and dCm).  Each
// stage of such a sum hands half of the values to another lane.  Which half is free of selects
// where it goes by an order that the lanes do not share: neighbouring lanes of a channel hold the
// two channels in opposite order, and neighbouring channels hold the two pairs of states in
// opposite order, so that every lane sends its second one and keeps its first.
//
// 8 x 2048 x 4096 x 16 bf16: 1656 us, 239 instructions for the eight elements of a thread's token
// at half of the issue slots; the floor is 139 us of bytes or 114 us of exponentials (each is taken
// 2.75 times).  Before: states of eight tokens in registers (two CTAs a SM) 2850 us, unpaired 3056
// us.  The chunk ahead by asynchronous copies 1702 us, in registers 1853 us (spilled).
//
// The CTA's parts of dBm and dCm, of dA, dD and ddt_bias go to the workspace and are added in a
// fixed order.
#include <type_traits>

#include "scan.cuh"

namespace lz {
namespace scan {
namespace {

constexpr int QT = 4, QN = CK / QT;  // tokens whose states are held at once, and how often a chunk
constexpr int NS = 4, H = 2;  // states a lane holds of a channel, and pairs of them

template <int LPC>
struct Lay {
    static constexpr int CPT = LPC > 1 ? 2 : 1;  // channels a thread
    static constexpr int LC = 32 / LPC;
    static constexpr int CW = LC * CPT;          // channels a warp
    static constexpr int CH = NT / 32 * CW;
    static constexpr int NP = NS * LPC;
    static constexpr int NV = CH / 8;
    static constexpr int PX = (CK * NV + NT - 1) / NT;
    static constexpr int NQ = (NP + 7) / 8;
    static constexpr int PB = (CK * NQ + NT - 1) / NT;
    static constexpr int KEEP = spread_left(16, 32 / NV > 1 ? 32 / NV : 1);
    using P = Plane<CK, CH, CW>;
};

template <int LPC>
struct Smem {
    using L = Lay<LPC>;
    // (d, d), (d x, d x), (e, e); once a token has been walked back, the second becomes its sums
    // over states (gb, qa) and the last one's first half that of Cm h
    f2 d[L::P::SIZE], dx[L::P::SIZE], e[L::P::SIZE];
    f2 b[CK][H * LPC], c[CK][H * LPC];
    float bc[NT / 32][CK][2][L::NP];         // a warp's sums over channels
    __align__(8) float bias[L::CH], skip[L::CH];  // dt_bias and D of the channels
    f2 start[QN][L::CPT * H][NT];            // a thread's states before each four tokens
    f2 dA[L::CPT * H][NT];                   // a thread's dA: a chunk's terms are added up first
};

template <typename T, int LPC>
__global__ void __launch_bounds__(NT, LPC > 2 ? 4 : 2) scan_bwd_kernel(const ScanArgs a, const Cut cut,
                                                      const float* rec_g, float* pbc, float* pparam,
                                                      int64_t param_stride) {
    using L = Lay<LPC>;
    using P = typename L::P;
    constexpr int CPT = L::CPT, LC = L::LC, CH = L::CH, NP = L::NP, NV = L::NV, PX = L::PX, PB = L::PB;
    constexpr int NQ = L::NQ, KEEP = L::KEEP;
    constexpr bool FAST = is_fast<T>();
    extern __shared__ __align__(16) unsigned char smraw[];
    Smem<LPC>& sm = *reinterpret_cast<Smem<LPC>*>(smraw);
    const Where<CH> w(a, cut);
    check_offsets(a.seqs, a.header);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int q = lane & (LPC - 1), cl = lane / LPC;
    const bool swap = cl & 1;  // this lane's pairs of states are held in reverse order
    const int N = (int)a.N, nn = max(0, min(NS, N - NS * q));
    const bool v4 = N % 4 == 0;
    const int64_t t0 = w.seg * cut.seg_len, t1 = min64(t0 + cut.seg_len, a.seqs.L);
    const int64_t row0 = w.b * a.seqs.L, C = a.C, nck = (a.seqs.L + CK - 1) / CK;
    int lch[CPT], pl[CPT];  // channel k of this thread (the order goes by the lane), its place in a plane
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        lch[k] = warp * L::CW + (CPT == 2 ? (k ^ (q & 1)) * LC : 0) + cl;
        pl[k] = P::at(0, lch[k]);
    }
    const int pair0 = (swap ? LPC : 0) + q, pair1 = (swap ? 0 : LPC) + q;  // of a row of b and c

    auto load_state = [&](const float* p, f2 (*f)[H]) {  // p: [C, N] or null
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            f2 v[H] = {0, 0};
            if (p != nullptr && w.c0 + lch[k] < w.clim)
                load_pairs<NS>(p + (w.c0 + lch[k]) * N + NS * q, nn, v4, v);
            f[k][0] = swap ? v[1] : v[0];
            f[k][1] = swap ? v[0] : v[1];
        }
    };
    auto put_state = [&](float* p, f2 (*f)[H]) {
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const f2 v[H] = {swap ? f[k][1] : f[k][0], swap ? f[k][0] : f[k][1]};
            if (w.c0 + lch[k] < w.clim) store_pairs<NS>(p + (w.c0 + lch[k]) * N + NS * q, nn, v4, v);
        }
    };
    auto seq_state = [&](const float* p, int64_t seq) { return p == nullptr ? p : p + seq * C * N; };
    f2 A2[CPT][H], gn[CPT][H];
    load_state(a.A, A2);
#pragma unroll
    for (int k = 0; k < CPT; ++k)
#pragma unroll
        for (int i = 0; i < H; ++i) A2[k][i] = mul2(A2[k][i], pack(kLog2e, kLog2e));
    // gn: the gradient that reaches the state after a token from later ones
    SeqAt sq = seq_at(a.seqs, w.b, t1 - 1);
    if (t1 == sq.end) load_state(seq_state(a.dh_out, sq.seq), gn);
    else load_state(rec_g + (w.b * cut.segs + w.seg) * C * N, gn);

    const int64_t cg = C / a.G;
    const bool vec = rows16<T>(cg, a.ldx) && rows16<T>(cg, a.lddt) && rows16<T>(cg, a.ldz) && rows16<T>(cg, a.ldy) &&
                     rows16<T>(cg, a.lddx) && rows16<T>(cg, a.ldddt) && rows16<T>(cg, a.lddz);
    const bool vecb = rows16<T>(N, a.ldb) && rows16<T>(N, a.ldc);
    const int pv = tid % NV, pt = tid / NV;
    const int64_t pch = w.c0 + pv * 8;
    const int pn = (int)max64(0, min64(8, w.clim - pch));
    constexpr int DT = NT / NV;
    for (int c = tid; c < CH; c += NT) {
        const bool in = w.c0 + c < w.clim;
        sm.bias[c] = in && a.dt_bias != nullptr ? a.dt_bias[w.c0 + c] : 0.0f;
        sm.skip[c] = in && a.D != nullptr ? a.D[w.c0 + c] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < CPT * H; ++i) sm.dA[i][tid] = 0;
    float keep[KEEP];  // sums of dD's and ddt_bias's terms: see below
#pragma unroll
    for (int i = 0; i < KEEP; ++i) keep[i] = 0.0f;
    // places of this lane's shares of the sums across lanes
    float dummy[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int at_t = spread_sum<4, 2, LPC>(dummy, lane), at_n = spread_sum<4, LPC * 2, 32>(dummy, lane);
    constexpr int LEFT_T = spread_left(4, LPC / 2 > 0 ? LPC / 2 : 1), LEFT_N = spread_left(4, LC / 2);
    const bool put_t = LPC <= 8 || q < 8, put_n = LC <= 8 || cl < 8;

    auto step = [&](int tl, f2 (*h)[H]) {  // the recurrence, one token on
        const f2 b[H] = {sm.b[tl][pair0], sm.b[tl][pair1]};
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const f2 d = sm.d[pl[k] + tl * NV], dx = sm.dx[pl[k] + tl * NV];
#pragma unroll
            for (int i = 0; i < H; ++i) h[k][i] = fma2(decay2(d, A2[k][i]), h[k][i], mul2(dx, b[i]));
        }
    };

    // The tokens [tt, tt + 16) of which those before t1 are walked.  PLAIN: none of them begins a
    // sequence.
    f2 dA[CPT][H];
    auto chunk = [&](int64_t tt, auto plain) {
        constexpr bool PLAIN = decltype(plain)::value;
        f2 h[CPT][H];
        load_state(a.states + (w.b * nck + tt / CK) * C * N, h);
        auto enter = [&](int tl) {  // the state before a token
            if (PLAIN || tt + tl >= t1) return;
            const SeqAt s = seq_at(a.seqs, w.b, tt + tl);
            if (s.begin == tt + tl) load_state(seq_state(a.h0, s.seq), h);
        };
        // a segment's short last chunk stops at its end
        const int quarters = (int)((min64(tt + CK, t1) - tt + QT - 1) / QT);
#pragma unroll 1
        for (int j = 0; j < quarters; ++j) {
#pragma unroll
            for (int k = 0; k < CPT; ++k)
#pragma unroll
                for (int i = 0; i < H; ++i) sm.start[j][k * H + i][tid] = h[k][i];
            if (j + 1 == quarters) break;
#pragma unroll
            for (int u = 0; u < QT; ++u) {
                enter(j * QT + u);
                step(j * QT + u, h);
            }
        }
#pragma unroll 1
        for (int j = quarters - 1; j >= 0; --j) {
            const int l0 = j * QT;
            f2 hist[QT + 1][CPT][H];
#pragma unroll
            for (int k = 0; k < CPT; ++k)
#pragma unroll
                for (int i = 0; i < H; ++i) h[k][i] = hist[0][k][i] = sm.start[j][k * H + i][tid];
#pragma unroll
            for (int u = 0; u < QT; ++u) {
                enter(l0 + u);
                step(l0 + u, h);
#pragma unroll
                for (int k = 0; k < CPT; ++k)
#pragma unroll
                    for (int i = 0; i < H; ++i) hist[u + 1][k][i] = h[k][i];
            }
            float pgb[QT], pqa[QT], pch[QT];  // of the first channel in this lane's order
#pragma unroll
            for (int u = QT - 1; u >= 0; --u) {
                const int tl = l0 + u;
                const f2 b[H] = {sm.b[tl][pair0], sm.b[tl][pair1]};
                const f2 c[H] = {sm.c[tl][pair0], sm.c[tl][pair1]};
                const bool first = !PLAIN && tt + tl == sq.begin && tt + tl < t1;
                f2 hp[CPT][H];  // the state before the token
#pragma unroll
                for (int k = 0; k < CPT; ++k)
#pragma unroll
                    for (int i = 0; i < H; ++i) hp[k][i] = hist[u][k][i];
                if (first) load_state(seq_state(a.h0, sq.seq), hp);
                f2 vb[H], vc[H];  // dBm, dCm of this lane's states, over its channels
                float gb[CPT], qa[CPT], cs[CPT];
#pragma unroll
                for (int k = 0; k < CPT; ++k) {
                    const f2 d = sm.d[pl[k] + tl * NV], dx = sm.dx[pl[k] + tl * NV], e = sm.e[pl[k] + tl * NV];
                    f2 sgb, sqa, scs;
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const f2 g = fma2(c[i], e, gn[k][i]), hh = hist[u + 1][k][i];
                        const f2 ag = mul2(decay2(d, A2[k][i]), g), qq = mul2(ag, hp[k][i]);
                        gn[k][i] = ag;
                        dA[k][i] = fma2(qq, d, dA[k][i]);
                        sqa = i == 0 ? mul2(qq, A2[k][i]) : fma2(qq, A2[k][i], sqa);
                        sgb = i == 0 ? mul2(g, b[i]) : fma2(g, b[i], sgb);
                        scs = i == 0 ? mul2(c[i], hh) : fma2(c[i], hh, scs);
                        vb[i] = k == 0 ? mul2(g, dx) : fma2(g, dx, vb[i]);
                        vc[i] = k == 0 ? mul2(hh, e) : fma2(hh, e, vc[i]);
                    }
                    gb[k] = sum2(sgb);
                    qa[k] = sum2(sqa);
                    cs[k] = sum2(scs);
                }
                if (first) {
                    if (a.dh0 != nullptr) put_state(a.dh0 + sq.seq * C * N, gn);
                    if (tt + tl > t0) {
                        sq = seq_at(a.seqs, w.b, tt + tl - 1);
                        load_state(seq_state(a.dh_out, sq.seq), gn);
                    }
                }
                // over states, first stage: the second channel goes to the neighbouring lane,
                // whose first it is
                if constexpr (CPT == 2) {
                    gb[0] += __shfl_xor_sync(~0u, gb[1], 1);
                    qa[0] += __shfl_xor_sync(~0u, qa[1], 1);
                    cs[0] += __shfl_xor_sync(~0u, cs[1], 1);
                }
                pgb[u] = gb[0];
                pqa[u] = qa[0];
                pch[u] = cs[0];
                // over channels: the second pair of states goes to the lane that has it first
                float v[4], s0, s1;
                unpack(vb[1], s0, s1);
                f2 x = pack(__shfl_xor_sync(~0u, s0, LPC), __shfl_xor_sync(~0u, s1, LPC));
                unpack(add2(vb[0], x), v[0], v[1]);
                unpack(vc[1], s0, s1);
                x = pack(__shfl_xor_sync(~0u, s0, LPC), __shfl_xor_sync(~0u, s1, LPC));
                unpack(add2(vc[0], x), v[2], v[3]);
                spread_sum<4, LPC * 2, 32>(v, lane);
#pragma unroll
                for (int i = 0; i < LEFT_N; ++i)
                    if (put_n) sm.bc[warp][tl][(at_n + i) / 2][NS * q + (swap ? 2 : 0) + (at_n + i) % 2] = v[i];
            }
            // over states, the other stages: four tokens together, of which a lane keeps some.
            // All lanes of a channel have read the tokens' planes by now.
            spread_sum<4, 2, LPC>(pgb, lane);
            spread_sum<4, 2, LPC>(pqa, lane);
            spread_sum<4, 2, LPC>(pch, lane);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < LEFT_T; ++i)
                if (put_t) {
                    const int o = pl[0] + (l0 + at_t + i) * NV;
                    sm.dx[o] = pack(pgb[i], pqa[i]);
                    reinterpret_cast<float*>(&sm.e[o])[0] = pch[i];
                }
        }
    };

#pragma unroll 1
    for (int64_t tt = t0 + (t1 - 1 - t0) / CK * CK; tt >= t0; tt -= CK) {
        // the chunk before is fetched into L2 meanwhile: registers for it are not to be had
        if (tt > t0 && vec && pn > 0) {
#pragma unroll
            for (int i = 0; i < PX; ++i) {
                const int tl = pt + i * DT - CK;
                if (tl >= 0) break;
                const int64_t r = row0 + tt + tl;
                prefetch_l2((const T*)a.x + r * a.ldx + pch);
                prefetch_l2((const T*)a.dt + r * a.lddt + pch);
                prefetch_l2((const T*)a.dy + r * a.ldy + pch);
                if (a.z != nullptr) prefetch_l2((const T*)a.z + r * a.ldz + pch);
            }
            // and the state before it, a 128-byte line each
            if (tid < CH * N / 32 && w.c0 * N + tid * 32 < w.clim * N)
                prefetch_l2(a.states + (w.b * nck + tt / CK - 1) * C * N + w.c0 * N + tid * 32);
        }
        __syncthreads();  // the last chunk's tiles have been read
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            const int tl = pt + i * DT;
            if (tl >= CK) break;
            const bool live = tt + tl < t1;
            const int n = live ? pn : 0;
            const int64_t r = row0 + tt + tl;
            Raw<T> rx, rdt, rz, rdy;
            rx.load((const T*)a.x + r * a.ldx + pch, n, vec);
            rdt.load((const T*)a.dt + r * a.lddt + pch, n, vec);
            rdy.load((const T*)a.dy + r * a.ldy + pch, n, vec);
            if (a.z != nullptr) rz.load((const T*)a.z + r * a.ldz + pch, n, vec);
            f2 fx[4], fd[4], fe[4], fz[4];
            rx.get(fx);
            rdt.get(fd);
            rdy.get(fe);
            if (a.z != nullptr) rz.get(fz);
            const f2* bias = reinterpret_cast<const f2*>(&sm.bias[pv * 8]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f2 v = add2(fd[j], bias[j]);
                // a place past the segment's end must leave the state and its gradient as they are
                const f2 d = live ? (a.softplus ? softplus2(v) : v) : 0;
                if (a.z != nullptr) fe[j] = mul2(fe[j], mul2(fz[j], sigm2<FAST>(fz[j])));
                put_doubled<P>(sm.d, tl, pv * 8 + 2 * j, d);
                put_doubled<P>(sm.dx, tl, pv * 8 + 2 * j, mul2(d, fx[j]));
                put_doubled<P>(sm.e, tl, pv * 8 + 2 * j, fe[j]);
            }
        }
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int e = tid + i * NT, tl = e / NQ, n0 = e % NQ * 8;
            if (tl >= CK) break;
            const int n = tt + tl < t1 ? max(0, min(8, N - n0)) : 0;
            const int64_t r = row0 + tt + tl;
            Raw<T> rb, rc;
            float f[8];
            rb.load((const T*)a.Bm + r * a.ldb + w.grp * N + n0, n, vecb);
            rc.load((const T*)a.Cm + r * a.ldc + w.grp * N + n0, n, vecb);
            rb.get(f);
            put_states<NS, LPC>(sm.b[tl], n0, f);
            rc.get(f);
            put_states<NS, LPC>(sm.c[tl], n0, f);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < CPT; ++k)
#pragma unroll
            for (int i = 0; i < H; ++i) dA[k][i] = 0;
        if (sq.begin < tt) chunk(tt, std::true_type());
        else chunk(tt, std::false_type());
#pragma unroll
        for (int k = 0; k < CPT; ++k)
#pragma unroll
            for (int i = 0; i < H; ++i) sm.dA[k * H + i][tid] = add2(sm.dA[k * H + i][tid], dA[k][i]);
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
        float terms[16];  // of dD and ddt_bias, this thread's channels
#pragma unroll
        for (int j = 0; j < 16; ++j) terms[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            const int tl = pt + i * DT;
            if (tl >= CK) break;
            const int n = tt + tl < t1 ? pn : 0;
            const int64_t r = row0 + tt + tl;
            Raw<T> rx, rdt, rz, rdy;
            rx.load((const T*)a.x + r * a.ldx + pch, n, vec);
            rdt.load((const T*)a.dt + r * a.lddt + pch, n, vec);
            rdy.load((const T*)a.dy + r * a.ldy + pch, n, vec);
            if (a.z != nullptr) rz.load((const T*)a.z + r * a.ldz + pch, n, vec);
            f2 fx[4], fd[4], fy[4], fz[4], ox[4], ot[4], oz[4];
            rx.get(fx);
            rdt.get(fd);
            rdy.get(fy);
            if (a.z != nullptr) rz.get(fz);
            const f2* bias = reinterpret_cast<const f2*>(&sm.bias[pv * 8]);
            const f2* skip = reinterpret_cast<const f2*>(&sm.skip[pv * 8]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int o0 = P::at(tl, pv * 8 + 2 * j), o1 = P::at(tl, pv * 8 + 2 * j + 1);
                float d0, d1, g0, g1, q0, q1, x;
                unpack(sm.d[o0], d0, x);
                unpack(sm.d[o1], d1, x);
                unpack(sm.dx[o0], g0, q0);
                unpack(sm.dx[o1], g1, q1);
                const f2 d = pack(d0, d1), gb = pack(g0, g1), D = skip[j];
                f2 e = fy[j];
                if (a.z != nullptr) {
                    const f2 sg = sigm2<FAST>(fz[j]);
                    float c0, c1;
                    unpack(sm.e[o0], c0, x);
                    unpack(sm.e[o1], c1, x);
                    oz[j] = mul2(mul2(fy[j], fma2(D, fx[j], pack(c0, c1))), dsilu2(fz[j], sg));
                    e = mul2(e, mul2(fz[j], sg));
                }
                ox[j] = fma2(d, gb, mul2(D, e));
                // qa was summed with A log2(e)
                f2 dd = fma2(fx[j], gb, mul2(pack(q0, q1), pack(0.69314718055994531f, 0.69314718055994531f)));
                if (a.softplus) dd = mul2(dd, sigm2<FAST>(add2(fd[j], bias[j])));
                ot[j] = dd;
                float e0, e1;
                unpack(mul2(e, fx[j]), e0, e1);
                unpack(dd, d0, d1);
                if (2 * j < n) terms[2 * j] += e0, terms[8 + 2 * j] += d0;
                if (2 * j + 1 < n) terms[2 * j + 1] += e1, terms[9 + 2 * j] += d1;
            }
            store8((T*)a.dx + r * a.lddx + pch, ox, n, vec);
            store8((T*)a.ddt + r * a.ldddt + pch, ot, n, vec);
            if (a.z != nullptr) store8((T*)a.dz + r * a.lddz + pch, oz, n, vec);
        }
        // over the warp's threads of the same channels; a thread keeps KEEP of the sixteen sums
        spread_sum<16, NV, 32>(terms, lane);
#pragma unroll
        for (int i = 0; i < KEEP; ++i) keep[i] += terms[i];
    }
    // the CTA's part of dA, dD and ddt_bias
    const int64_t part = w.b * cut.segs + w.seg;
    f2 tA[CPT][H];
#pragma unroll
    for (int k = 0; k < CPT; ++k)
#pragma unroll
        for (int i = 0; i < H; ++i) tA[k][i] = sm.dA[k * H + i][tid];
    float* pp = pparam + part * param_stride;  // dA [C, N], dD [C], ddt_bias [C]
    put_state(pp, tA);
    __syncthreads();
    float* red = reinterpret_cast<float*>(smraw);  // [warps][2][CH]
    {
        float none[16] = {};
        const int at = spread_sum<16, NV, 32>(none, lane);
        // where a warp holds a channel's threads once or less often than its lanes, every lane has
        // its own sums; else lanes that ended with the same ones write the same values
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            red[(warp * 2 + (at + i) / 8) * CH + pv * 8 + (at + i) % 8] = keep[i];
    }
    __syncthreads();
    for (int e = tid; e < 2 * CH; e += NT) {
        const int c = e % CH, m = e / CH;
        if (w.c0 + c >= w.clim) continue;
        float s = 0.0f;
        for (int k = 0; k < NT / 32; ++k) s += red[(k * 2 + m) * CH + c];
        pp[C * N + m * C + w.c0 + c] = s;
    }
}

// A segment's own contribution to the gradient of the state before it: sum over its tokens of
// (the decays up to and with the token) Cm e, up to the first place where a sequence ends; and
// the sum of its step sizes (NaN where a sequence begins in it, whose decays let nothing pass).
template <typename T, int LPC>
__global__ void __launch_bounds__(NT) scan_adj_kernel(const ScanArgs a, const Cut cut, float* rec_g,
                                                      float* rec_d) {
    using L = Lay<LPC>;
    using P = typename L::P;
    constexpr int CPT = L::CPT, LC = L::LC, CH = L::CH, NV = L::NV, PX = L::PX, PB = L::PB, NQ = L::NQ;
    constexpr int DT = NT / NV;
    constexpr bool FAST = is_fast<T>();
    __shared__ __align__(16) f2 sd[P::SIZE];  // (d, d)
    __shared__ __align__(16) f2 se[P::SIZE];  // (e, e)
    __shared__ __align__(16) f2 sc[CK][H * LPC];
    const Where<CH> w(a, cut);
    if (w.seg == 0) return;  // nothing is before the first segment
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int q = lane & (LPC - 1), lch = warp * L::CW + lane / LPC;
    const int N = (int)a.N, nn = max(0, min(NS, N - NS * q));
    const bool v4 = N % 4 == 0;
    const int64_t t0 = w.seg * cut.seg_len, t1 = min64(t0 + cut.seg_len, a.seqs.L);
    const int64_t row0 = w.b * a.seqs.L, C = a.C;
    f2 A2[CPT][H], p[CPT][H], acc[CPT][H];
    float sum[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int64_t c = w.c0 + lch + k * LC;
        A2[k][0] = A2[k][1] = 0;
        if (c < w.clim) load_pairs<NS>(a.A + c * N + NS * q, nn, v4, A2[k]);
        sum[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            A2[k][i] = mul2(A2[k][i], pack(kLog2e, kLog2e));
            p[k][i] = pack(1.0f, 1.0f);
            acc[k][i] = 0;
        }
    }
    const SeqAt sq = seq_at(a.seqs, w.b, t0);
    const int64_t cg = C / a.G;
    const bool vec = rows16<T>(cg, a.lddt) && rows16<T>(cg, a.ldz) && rows16<T>(cg, a.ldy);
    const bool vecb = rows16<T>(N, a.ldc);
    const int pv = tid % NV, pt = tid / NV;
    const int64_t pch = w.c0 + pv * 8;
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
            Raw<T> rdt, rdy, rz;
            f2 fd[4], fe[4], fz[4];
            rdt.load((const T*)a.dt + r * a.lddt + pch, live ? pn : 0, vec);
            rdy.load((const T*)a.dy + r * a.ldy + pch, live ? pn : 0, vec);
            if (a.z != nullptr) {
                rz.load((const T*)a.z + r * a.ldz + pch, live ? pn : 0, vec);
                rz.get(fz);
            }
            rdt.get(fd);
            rdy.get(fe);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float b0 = 0.0f, b1 = 0.0f;
                if (a.dt_bias != nullptr) {
                    if (2 * j < pn) b0 = a.dt_bias[pch + 2 * j];
                    if (2 * j + 1 < pn) b1 = a.dt_bias[pch + 2 * j + 1];
                }
                const f2 v = add2(fd[j], pack(b0, b1));
                if (a.z != nullptr) fe[j] = mul2(fe[j], mul2(fz[j], sigm2<FAST>(fz[j])));
                put_doubled<P>(sd, tl, pv * 8 + 2 * j, live ? (a.softplus ? softplus2(v) : v) : 0);
                put_doubled<P>(se, tl, pv * 8 + 2 * j, fe[j]);
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
            put_states<NS, LPC>(sc[tl], n0, f);
        }
        __syncthreads();
#pragma unroll 4
        for (int tl = 0; tl < CK; ++tl) {
            const f2 c[H] = {sc[tl][q], sc[tl][LPC + q]};
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const f2 d = sd[P::at(tl, lch + k * LC)], e = se[P::at(tl, lch + k * LC)];
                float u, v;
                unpack(d, u, v);
                sum[k] += u;
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    p[k][i] = mul2(p[k][i], decay2(d, A2[k][i]));
                    acc[k][i] = fma2(p[k][i], mul2(c[i], e), acc[k][i]);
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
            f2 g[H];
            load_pairs<NS>(a.dh_out + (sq.seq * C + c) * N + NS * q, nn, v4, g);
#pragma unroll
            for (int i = 0; i < H; ++i) acc[k][i] = fma2(p[k][i], g[i], acc[k][i]);
        }
        store_pairs<NS>(rec_g + (rec + c) * N + NS * q, nn, v4, acc[k]);
        if (q == 0) rec_d[rec + c] = stop < t1 || ends ? __int_as_float(0x7fc00000) : sum[k];
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
    float* p = rec_g + b * segs * CN + cn;
    const float* pd = rec_d + b * segs * a.C + c;
    constexpr int U = 8;  // records read together
    for (int64_t s = segs - 1; s >= 0; s -= U) {
        float own[U], d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            own[u] = s > u ? p[(s - u) * CN] : 0.0f;  // the first segment's own is not needed
            d[u] = s > u ? pd[(s - u) * a.C] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s < u) break;
            p[(s - u) * CN] = g;
            g = isnan(d[u]) ? own[u] : fmaf(ex2(d[u] * A2), g, own[u]);
        }
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

// dA, dD and ddt_bias from the CTAs' parts [n][stride].
template <int KT>
__global__ void __launch_bounds__(32 * KT) scan_param_kernel(const ScanArgs a, int64_t n, const float* in, int64_t stride) {
    const int64_t i0 = (int64_t)blockIdx.x * 32, CN = a.C * a.N;
    sum_columns<KT>(
        n, (int)min64(32, CN + 2 * a.C - i0), [&](int64_t p, int i) { return in[p * stride + i0 + i]; },
        [&](int k, float s) {
            const int64_t i = i0 + k;
            if (i < CN) a.dA[i] = s;
            else if (i < CN + a.C) {
                if (a.dD != nullptr) a.dD[i - CN] = s;
            } else if (a.ddt_bias != nullptr) {
                a.ddt_bias[i - CN - a.C] = s;
            }
        });
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

// As the forward's cut: segments where there are fewer than two CTAs a SM.  The pass over the
// segments' gradients costs about a fifth of the walk.
Cut bwd_cut(const ScanArgs& a) {
    const int lanes = padded_states(a.N) / NS, ch = NT / lanes * (lanes > 1 ? 2 : 1);
    Cut k;
    k.cbg = (a.C / a.G + ch - 1) / ch;
    k.cblocks = k.cbg * a.G;
    k.segs = 1;
    k.seg_len = a.seqs.L;
    const int64_t ctas = a.B * k.cblocks;
    if (ctas > 304 || a.seqs.L <= SEG) return k;
    const int64_t want = (4 * 152 + ctas - 1) / ctas;
    k.seg_len = ((a.seqs.L + want - 1) / want + SEG - 1) / SEG * SEG;
    k.segs = (a.seqs.L + k.seg_len - 1) / k.seg_len;
    return k;
}

struct BwdWs {
    size_t rec_g, rec_d, bc, param, param_stride, total;
};
BwdWs bwd_ws(const ScanArgs& a, const Cut& k) {
    BwdWs o;
    const size_t parts = (size_t)(a.B * k.segs), CN = (size_t)(a.C * a.N);
    auto up = [](size_t n) { return (n + 3) & ~(size_t)3; };
    size_t at = 0;
    o.rec_g = at, at += k.segs > 1 ? up(parts * CN) : 0;
    o.rec_d = at, at += k.segs > 1 ? up(parts * a.C) : 0;
    o.bc = at, at += up((size_t)(k.cbg * a.B * a.seqs.L * a.G * 2 * a.N));
    o.param_stride = up(CN + 2 * (size_t)a.C);
    o.param = at, at += parts * o.param_stride;
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
        e = with_lanes(padded_states(a.N) / NS, [&](auto ll) {
            constexpr int LPC = decltype(ll)::value;
            const unsigned g = (unsigned)(parts * k.cblocks);
            if (k.segs > 1) {
                scan_adj_kernel<T, LPC><<<g, NT, 0, s>>>(a, k, f + o.rec_g, f + o.rec_d);
                scan_adj_join_kernel<<<(unsigned)((a.B * CN + 255) / 256), 256, 0, s>>>(a, k.segs, f + o.rec_g, f + o.rec_d);
            }
            const int bytes = (int)sizeof(Smem<LPC>);
            cudaError_t r = cudaFuncSetAttribute(scan_bwd_kernel<T, LPC>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (r != cudaSuccess) return r;
            scan_bwd_kernel<T, LPC><<<g, NT, bytes, s>>>(a, k, f + o.rec_g, f + o.bc, f + o.param, (int64_t)o.param_stride);
            const int64_t n = a.B * a.seqs.L * a.G * 2 * a.N;
            scan_bc_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a, k.cbg, f + o.bc);
            return cudaGetLastError();
        });
        if (e != cudaSuccess) return e;
    }
    const unsigned g = (unsigned)((CN + 2 * a.C + 31) / 32);
    if (many_partials(parts, g)) scan_param_kernel<32><<<g, 1024, 0, s>>>(a, parts, f + o.param, o.param_stride);
    else scan_param_kernel<8><<<g, 256, 0, s>>>(a, parts, f + o.param, o.param_stride);
    return cudaGetLastError();
}

}  // namespace
}  // namespace scan

size_t scan_bwd_ws_floats(const ScanArgs& a) { return scan::bwd_ws(a, scan::bwd_cut(a)).total; }

cudaError_t launch_scan_bwd(const ScanArgs& a, cudaStream_t s) {
    return a.dtype == LIZARD_BF16 ? scan::scan_bwd<__nv_bfloat16>(a, s) : scan::scan_bwd<float>(a, s);
}

}  // namespace lz
