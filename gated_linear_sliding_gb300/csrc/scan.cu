// The selective scan (lizard_scan_*): forward and single-token step.
//
//   h[t, c, n] = exp(d A[c, n]) h[t-1, c, n] + d x[t, c] Bm[t, n],   d = softplus(dt + bias)
//   y[t, c]    = (sum_n Cm[t, n] h[t, c, n] + D[c] x[t, c]) silu(z[t, c])
//
// Four lanes (N = 16) share a channel, four states each in registers; a CTA of 128 threads walks
// its channels through a segment of the time axis, a tile of 32 tokens at a time: the tile's step sizes and
// d x are computed once and put into shared memory with Bm and Cm in fp32, while the next tile's
// rows are already on their way into registers.
#include <type_traits>

#include "scan.cuh"

namespace lz {
namespace scan {
namespace {

template <int LPC, int CPT>
struct Lay {
    static constexpr int TT = LPC == 1 ? 16 : 32;    // tokens a tile
    static constexpr int LC = 32 / LPC;              // channels side by side in a warp
    static constexpr int CH = NT / 32 * LC * CPT;    // channels a CTA
    static constexpr int NP = NS * LPC;              // states, padded
    static constexpr int NV = CH / 8;                // 8-channel pieces of a row
    static constexpr int PX = (TT * NV + NT - 1) / NT;       // pieces a thread stages of x, dt, z
    static constexpr int PB = (TT * (NP + 7) / 8 + NT - 1) / NT;  // and of Bm, Cm
    static constexpr int YS = CH + 8;                // row stride of the outputs' tile: four
                                                     // rows x eight channels in distinct banks
};

template <int LPC, int CPT>
struct Smem {
    using L = Lay<LPC, CPT>;
    static constexpr int TT = L::TT;
    float2 dx[TT][L::CH];          // d, d x
    float2 b[TT][2][LPC], c[TT][2][LPC];  // [half][lane]: states 4 lane + 2 half + {0, 1}
    float y[TT][L::YS];
};

// MAIN: the outputs (and states).  Otherwise only a segment's own end state from a zero start and
// the sum of its step sizes, for the join.
template <typename T, int LPC, int CPT, bool MAIN>
__global__ void __launch_bounds__(NT) scan_fwd_kernel(const ScanArgs a, const Cut cut,
                                                      float* rec_h, float* rec_d,
                                                      const float* h0) {
    using L = Lay<LPC, CPT>;
    constexpr int TT = L::TT, LC = L::LC, CH = L::CH, NP = L::NP, NV = L::NV, PX = L::PX, PB = L::PB;
    constexpr int NQ = (NP + 7) / 8;  // 8-state pieces of a row of Bm
    __shared__ __align__(16) Smem<LPC, CPT> sm;
    const Where<CH> w(a, cut);
    if (MAIN) check_offsets(a.seqs, a.header);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int q = lane & (LPC - 1), cl = lane / LPC;
    const int N = (int)a.N, nn = max(0, min(NS, N - NS * q));  // this lane's states
    const bool v4 = N % 4 == 0;
    const int64_t t0 = w.seg * cut.seg_len, t1 = min64(t0 + cut.seg_len, a.seqs.L);
    const int64_t row0 = w.b * a.seqs.L;
    const int64_t C = a.C;

    float A2[CPT][NS], h[CPT][NS], sd[CPT];
    int64_t ch[CPT];
    bool own[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        ch[k] = w.c0 + warp * (LC * CPT) + k * LC + cl;
        own[k] = ch[k] < w.clim;
        sd[k] = 0.0f;
        float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (own[k]) load4(a.A + ch[k] * N + NS * q, nn, v4, f);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            A2[k][i] = f[i] * kLog2e;
            h[k][i] = 0.0f;
        }
    }
    // a sequence's first state
    auto begin_state = [&](int64_t seq) {
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
#pragma unroll
            for (int i = 0; i < NS; ++i) h[k][i] = 0.0f;
            if (h0 != nullptr && own[k]) load4(h0 + (seq * C + ch[k]) * N + NS * q, nn, v4, h[k]);
        }
    };
    auto put_state = [&](float* p) {  // p: [C, N]
#pragma unroll
        for (int k = 0; k < CPT; ++k)
            if (own[k]) store4(p + ch[k] * N + NS * q, nn, v4, h[k]);
    };
    SeqAt sq = seq_at(a.seqs, w.b, t0);
    bool cutoff = false;  // a sequence begins in this segment: nothing before it reaches its end
    const int64_t rec = (w.b * cut.segs + w.seg) * C;
    if (t0 == sq.begin) {
        begin_state(sq.seq);
        cutoff = true;
    } else if (MAIN) {
#pragma unroll
        for (int k = 0; k < CPT; ++k)
            if (own[k]) load4(rec_h + (rec + ch[k]) * N + NS * q, nn, v4, h[k]);
    }

    // staging: thread's pieces of a tile
    const bool vec = a.C % 8 == 0 && (C / a.G) % 8 == 0 && a.ldx % 8 == 0 && a.lddt % 8 == 0 &&
                     a.ldz % 8 == 0 && a.ldy % 8 == 0;
    const bool vecb = N % 8 == 0 && a.ldb % 8 == 0 && a.ldc % 8 == 0;
    const int pc = tid % NV * 8, pt = tid / NV;  // channel and first token of the x pieces
    const int64_t pch = w.c0 + pc;
    const int pn = (int)max64(0, min64(8, w.clim - pch));
    constexpr int DT = NT / NV;  // tokens between a thread's pieces
    Raw<T> rx[PX], rdt[PX], rz[PX], rb[PB], rc[PB];
    auto fetch = [&](int64_t tt) {
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            const int64_t t = tt + pt + i * DT;
            const int n = t < t1 && pt + i * DT < TT ? pn : 0;
            const int64_t r = row0 + t;
            rx[i].load((const T*)a.x + r * a.ldx + pch, n, vec);
            rdt[i].load((const T*)a.dt + r * a.lddt + pch, n, vec);
            if (MAIN && a.z != nullptr) rz[i].load((const T*)a.z + r * a.ldz + pch, n, vec);
        }
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int e = tid + i * NT, tl = e / NQ, n0 = e % NQ * 8;
            const int n = tl < TT && tt + tl < t1 ? max(0, min(8, N - n0)) : 0;
            const int64_t r = row0 + tt + tl;
            rb[i].load((const T*)a.Bm + r * a.ldb + w.grp * N + n0, n, vecb);
            if (MAIN) rc[i].load((const T*)a.Cm + r * a.ldc + w.grp * N + n0, n, vecb);
        }
    };
    Raw<T> kx[PX], kz[PX];  // the current tile's x and z, for its outputs
    auto commit = [&]() {
        float bias[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) bias[i] = a.dt_bias != nullptr && i < pn ? a.dt_bias[pch + i] : 0.0f;
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            if (pt + i * DT >= TT) break;
            float fx[8], fd[8];
            rx[i].get(fx);
            rdt[i].get(fd);
            float2* o = &sm.dx[pt + i * DT][pc];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = fd[j] + bias[j], d = a.softplus ? softplus_(v) : v;
                o[j] = make_float2(d, d * fx[j]);
            }
            if (MAIN) {
                kx[i] = rx[i];
                kz[i] = rz[i];
            }
        }
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int e = tid + i * NT, tl = e / NQ, n0 = e % NQ * 8;
            if (tl >= TT) break;
            float f[8];
            rb[i].get(f);
#pragma unroll
            for (int j = 0; j < 8 && j < NP; j += 2)
                sm.b[tl][j / 2 % 2][(n0 + j) / 4] = make_float2(f[j], f[j + 1]);
            if (MAIN) {
                rc[i].get(f);
#pragma unroll
                for (int j = 0; j < 8 && j < NP; j += 2)
                    sm.c[tl][j / 2 % 2][(n0 + j) / 4] = make_float2(f[j], f[j + 1]);
            }
        }
    };
    // one token: the recurrence, and this lane's part of the output
    auto step = [&](int tl, float* part) {
        const float2 b0 = sm.b[tl][0][q], b1 = sm.b[tl][1][q];
        const float bb[4] = {b0.x, b0.y, b1.x, b1.y};
        float cc[4];
        if (MAIN) {
            const float2 c0 = sm.c[tl][0][q], c1 = sm.c[tl][1][q];
            cc[0] = c0.x, cc[1] = c0.y, cc[2] = c1.x, cc[3] = c1.y;
        }
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const float2 d = sm.dx[tl][warp * (LC * CPT) + k * LC + cl];
            float p = 0.0f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                h[k][i] = fmaf(ex2(d.x * A2[k][i]), h[k][i], d.y * bb[i]);
                if (MAIN) p = fmaf(cc[i], h[k][i], p);
            }
            if (MAIN) part[k] = p;
            else sd[k] += d.x;
        }
    };
    // sums over a channel's lanes of four tokens' parts; each lane keeps one token of four
    // (two of four with two lanes a channel)
    auto reduce = [&](float (*p)[CPT], int tl) {
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            float* yc = &sm.y[tl][warp * (LC * CPT) + k * LC + cl];
            if constexpr (LPC == 1) {
#pragma unroll
                for (int i = 0; i < 4; ++i) yc[i * L::YS] = p[i][k];
            } else {
                const bool b0 = q & 1;
                float u = b0 ? p[1][k] : p[0][k], v = b0 ? p[3][k] : p[2][k];
                u += __shfl_xor_sync(~0u, b0 ? p[0][k] : p[1][k], 1);
                v += __shfl_xor_sync(~0u, b0 ? p[2][k] : p[3][k], 1);
                if constexpr (LPC == 2) {
                    yc[(q & 1) * L::YS] = u;
                    yc[(2 + (q & 1)) * L::YS] = v;
                } else {
                    const bool b1 = q & 2;
                    float s = b1 ? v : u;
                    s += __shfl_xor_sync(~0u, b1 ? u : v, 2);
#pragma unroll
                    for (int o = 4; o < LPC; o *= 2) s += __shfl_xor_sync(~0u, s, o);
                    if (q < 4) yc[(q & 3) * L::YS] = s;
                }
            }
        }
    };

    fetch(t0);
    for (int64_t tt = t0; tt < t1; tt += TT) {
        commit();
        __syncthreads();
        if (tt + TT < t1) fetch(tt + TT);
        const int n = (int)min64(TT, t1 - tt);
        for (int tl = 0; tl < n; tl += 4) {
            const int64_t t = tt + tl;
            if (MAIN && a.states != nullptr && tl % CK == 0)
                put_state(a.states + (w.b * ((a.seqs.L + CK - 1) / CK) + t / CK) * C * N);
            float part[4][CPT];
            if (t + 4 <= sq.end) {  // then t + 4 <= t1 too: a segment ends on a group or with its row
#pragma unroll
                for (int i = 0; i < 4; ++i) step(tl + i, part[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int k = 0; k < CPT; ++k) part[i][k] = 0.0f;
                    if (t + i >= t1) continue;
                    if (t + i == sq.end) {
                        if (MAIN && a.h_out != nullptr) put_state(a.h_out + sq.seq * C * N);
                        sq = seq_at(a.seqs, w.b, t + i);
                        begin_state(sq.seq);
                        cutoff = true;
                    }
                    step(tl + i, part[i]);
                }
            }
            if (MAIN) reduce(part, tl);
        }
        if (MAIN) {
            __syncthreads();
            float dd[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) dd[i] = a.D != nullptr && i < pn ? a.D[pch + i] : 0.0f;
#pragma unroll
            for (int i = 0; i < PX; ++i) {
                const int tl = pt + i * DT;
                if (tl >= TT) break;
                float fx[8], o[8];
                kx[i].get(fx);
                const float4 y0 = *reinterpret_cast<const float4*>(&sm.y[tl][pc]);
                const float4 y1 = *reinterpret_cast<const float4*>(&sm.y[tl][pc + 4]);
                const float yy[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = fmaf(dd[j], fx[j], yy[j]);
                if (a.z != nullptr) {
                    float fz[8];
                    kz[i].get(fz);
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] *= fz[j] * sigm<is_fast<T>()>(fz[j]);
                }
                store8((T*)a.y + (row0 + tt + tl) * a.ldy + pch, o, tt + tl < t1 ? pn : 0, vec);
            }
        } else {
            __syncthreads();
        }
    }
    if (MAIN) {
        if (t1 == sq.end && a.h_out != nullptr) put_state(a.h_out + sq.seq * C * N);
    } else {
        put_state(rec_h + rec * N);
#pragma unroll
        for (int k = 0; k < CPT; ++k)
            if (own[k] && q == 0) rec_d[rec + ch[k]] = cutoff ? __int_as_float(0x7fc00000) : sd[k];
    }
}

// Joins the segments of a row: the state before each, in place of each one's own end state.  A
// sum of NaN marks a segment in which a sequence begins.
__global__ void __launch_bounds__(256) scan_join_kernel(const ScanArgs a, int64_t segs, float* rec_h,
                                                        const float* rec_d) {
    const int64_t CN = a.C * a.N, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= a.B * CN) return;
    const int64_t b = id / CN, cn = id % CN, c = cn / a.N;
    const float A2 = a.A[cn] * kLog2e;
    float h = 0.0f;
    for (int64_t s = 0; s < segs; ++s) {
        float* p = rec_h + (b * segs + s) * CN + cn;
        float own = 0.0f, d = 0.0f;
        if (s + 1 < segs) {  // the last segment's own end state is not needed
            own = *p;
            d = rec_d[(b * segs + s) * a.C + c];
        }
        *p = h;
        h = isnan(d) ? own : fmaf(ex2(d * A2), h, own);
    }
}

// Sequences without tokens hand their state on; with `all`, a plain copy of every state.
__global__ void __launch_bounds__(256) scan_pass_kernel(Seqs seqs, int64_t nstate, int64_t w, const float* from,
                                                        float* to, bool all) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= nstate * w) return;
    int64_t end;
    if (!all && seq_tokens(seqs, id / w, &end) > 0) return;
    to[id] = from != nullptr ? from[id] : 0.0f;
}

// One token a sequence.  Bound by reading and writing the state once.
template <typename T, int LPC>
__global__ void __launch_bounds__(NT) scan_step_kernel(const ScanArgs a) {
    constexpr int LC = NT / LPC;
    const int q = threadIdx.x & (LPC - 1);
    const int64_t cbs = (a.C + LC - 1) / LC, b = blockIdx.x / cbs;
    const int64_t c = blockIdx.x % cbs * LC + threadIdx.x / LPC;
    const bool own = c < a.C;
    const int N = (int)a.N, nn = own ? max(0, min(NS, N - NS * q)) : 0;
    const int64_t slot = a.slots != nullptr ? a.slots[b] : b;
    if (slot < 0 || slot >= a.nslots) {  // an idle row
        if (slot >= 0) report(a.header, LIZARD_ERR_INVALID_ARG, 33);
        if (own && q == 0) st((T*)a.y + b * a.ldy + c, 0.0f);
        return;
    }
    float h[NS] = {}, A[NS] = {}, bb[NS] = {}, cc[NS] = {}, d = 0.0f, x = 0.0f;
    if (own) {
        const bool v4 = N % 4 == 0;
        load4(a.state + (slot * a.C + c) * N + NS * q, nn, v4, h);
        load4(a.A + c * N + NS * q, nn, v4, A);
        const int64_t grp = c / (a.C / a.G);
        const T* pb = (const T*)a.Bm + b * a.ldb + grp * N + NS * q;
        const T* pc = (const T*)a.Cm + b * a.ldc + grp * N + NS * q;
        if (v4 && a.ldb % 4 == 0 && a.ldc % 4 == 0 && nn == NS) {
            Vec<4>::ld(pb, bb);
            Vec<4>::ld(pc, cc);
        } else {
#pragma unroll
            for (int i = 0; i < NS; ++i)
                if (i < nn) bb[i] = ld(pb + i), cc[i] = ld(pc + i);
        }
        x = ld((const T*)a.x + b * a.ldx + c);
        const float v = ld((const T*)a.dt + b * a.lddt + c) + (a.dt_bias != nullptr ? a.dt_bias[c] : 0.0f);
        d = a.softplus ? softplus_(v) : v;
    }
    const float dx = d * x;
    float y = 0.0f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        h[i] = fmaf(ex2(d * (A[i] * kLog2e)), h[i], dx * bb[i]);
        y = fmaf(cc[i], h[i], y);
    }
#pragma unroll
    for (int o = 1; o < LPC; o *= 2) y += __shfl_xor_sync(~0u, y, o);
    if (!own) return;
    store4(a.state + (slot * a.C + c) * N + NS * q, nn, N % 4 == 0, h);
    if (q != 0) return;
    if (a.D != nullptr) y = fmaf(a.D[c], x, y);
    if (a.z != nullptr) {
        const float z = ld((const T*)a.z + b * a.ldz + c);
        y *= z * sigm<is_fast<T>()>(z);
    }
    st((T*)a.y + b * a.ldy + c, y);
}

template <int LPC = 1, typename F>
cudaError_t with_lanes(int l, F&& f) {
    if constexpr (LPC > 16) return cudaErrorInvalidValue;
    else return l == LPC ? f(std::integral_constant<int, LPC>()) : with_lanes<LPC * 2>(l, f);
}

// The forward's cut.  One pass over the whole time axis costs the least; where that leaves too
// few warps, the axis is cut into segments, whose end states take a pass of their own.
Cut fwd_cut(const ScanArgs& a) {
    const int lanes = lanes_for(a.N), ch = NT / lanes;
    Cut k;
    k.cbg = (a.C / a.G + ch - 1) / ch;
    k.cblocks = k.cbg * a.G;
    k.segs = 1;
    k.seg_len = a.seqs.L;
    const int64_t ctas = a.B * k.cblocks;
    if (ctas >= 96 || a.seqs.L <= 4 * SEG) return k;
    int64_t want = (4 * 152 + ctas - 1) / ctas;
    k.seg_len = ((a.seqs.L + want - 1) / want + SEG - 1) / SEG * SEG;
    k.segs = (a.seqs.L + k.seg_len - 1) / k.seg_len;
    return k;
}

size_t rec_floats(const ScanArgs& a, const Cut& k) {
    return k.segs > 1 ? (size_t)(a.B * k.segs * a.C) * (a.N + 1) : 0;
}

template <typename T>
cudaError_t scan_fwd(const ScanArgs& a, cudaStream_t s) {
    const Cut k = fwd_cut(a);
    float *rec_h = a.ws, *rec_d = a.ws + (size_t)(a.B * k.segs * a.C) * a.N;
    const float* h0 = a.h0;
    const int64_t w = a.C * a.N;
    const unsigned gs = (unsigned)((a.nstate * w + 255) / 256);
    if (k.segs > 1 && h0 != nullptr && h0 == a.h_out) {
        // a sequence's end is written while another segment may still read its beginning
        float* copy = a.ws + rec_floats(a, k);
        scan_pass_kernel<<<gs, 256, 0, s>>>(a.seqs, a.nstate, w, h0, copy, true);
        h0 = copy;
    }
    if (a.h_out != nullptr && a.h_out != a.h0 && (a.seqs.cu != nullptr || a.seqs.L == 0))
        scan_pass_kernel<<<gs, 256, 0, s>>>(a.seqs, a.nstate, w, a.h0, a.h_out, false);
    if (a.seqs.L == 0) return cudaGetLastError();
    return with_lanes(lanes_for(a.N), [&](auto ll) {
        constexpr int LPC = decltype(ll)::value;
        const unsigned g = (unsigned)(a.B * k.segs * k.cblocks);
        if (k.segs > 1) {
            scan_fwd_kernel<T, LPC, 1, false><<<g, NT, 0, s>>>(a, k, rec_h, rec_d, h0);
            scan_join_kernel<<<(unsigned)((a.B * w + 255) / 256), 256, 0, s>>>(a, k.segs, rec_h, rec_d);
        }
        scan_fwd_kernel<T, LPC, 1, true><<<g, NT, 0, s>>>(a, k, rec_h, rec_d, h0);
        return cudaGetLastError();
    });
}

template <typename T>
cudaError_t scan_step(const ScanArgs& a, cudaStream_t s) {
    return with_lanes(lanes_for(a.N), [&](auto ll) {
        constexpr int LPC = decltype(ll)::value, LC = NT / LPC;
        scan_step_kernel<T, LPC><<<(unsigned)(a.B * ((a.C + LC - 1) / LC)), NT, 0, s>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace
}  // namespace scan

size_t scan_fwd_ws_floats(const ScanArgs& a) {
    const scan::Cut k = scan::fwd_cut(a);
    // and room for a copy of the first states where they are updated in place
    return k.segs > 1 ? scan::rec_floats(a, k) + (size_t)(a.nstate * a.C * a.N) : 0;
}

cudaError_t launch_scan_fwd(const ScanArgs& a, cudaStream_t s) {
    return a.dtype == LIZARD_BF16 ? scan::scan_fwd<__nv_bfloat16>(a, s) : scan::scan_fwd<float>(a, s);
}

cudaError_t launch_scan_step(const ScanArgs& a, cudaStream_t s) {
    return a.dtype == LIZARD_BF16 ? scan::scan_step<__nv_bfloat16>(a, s) : scan::scan_step<float>(a, s);
}

}  // namespace lz
