// The selective scan (lizard_scan_*): forward and single-token step.
//
//   h[t, c, n] = exp(d A[c, n]) h[t-1, c, n] + d x[t, c] Bm[t, n],   d = softplus(dt + bias)
//   y[t, c]    = (sum_n Cm[t, n] h[t, c, n] + D[c] x[t, c]) silu(z[t, c])
//
// Two lanes (N = 16) share a channel, eight states each in registers; a CTA of 128 threads walks its
// channels through a segment of the time axis, a tile of tokens at a time: the tile's step sizes
// and d x are computed once and put into shared memory with Bm and Cm in fp32, while the next
// tile's rows are already on their way into registers.
//
// The floor is the exponentials: one for each token, channel and state, 32 a cycle and SM (57 us
// for 8192 x 4096 x 16; the bytes take 40 us).  An element takes 8.5 instruction slots: the
// exponential, two products, two multiply-adds (paired, half a slot each), a quarter each of four
// loads from shared memory and its share of the staging (softplus, gate, conversions: about 27 slots a
// token and channel).  8 x 2048 x 4096 x 16 bf16: 453 us at 55% of the issue slots, no pipe above
// 63%: the warps wait for one another's shared-memory loads and for the fixed latency of dependent
// instructions; more warps with fewer registers, exponentials ahead by a group of tokens, tiles by
// asynchronous copies, and single instead of paired arithmetic all measured the same or slower.
#include <type_traits>

#include "scan.cuh"

namespace lz {
namespace scan {
namespace {

template <int LPC, int NS>
struct Lay {
    static constexpr int LC = 32 / LPC;            // channels side by side in a warp
    static constexpr int CH = NT / 32 * LC;        // channels a CTA
    static constexpr int NP = NS * LPC;            // states, padded
    static constexpr int NV = CH / 8;              // 8-channel pieces of a row
    // tokens a tile: one piece of x, dt and z a thread where Bm and Cm leave room for it
    static constexpr int TT = 1024 / CH < 2048 / NP ? 1024 / CH : 2048 / NP;
    static constexpr int NQ = (NP + 7) / 8;        // 8-state pieces of a row of Bm
    static constexpr int PB = (TT * NQ + NT - 1) / NT;  // of which a thread stages so many
    static constexpr int U = 8;                    // tokens whose outputs are summed together
    using P = Plane<TT, CH, LC>;
};

template <int LPC, int NS>
struct Smem {
    using L = Lay<LPC, NS>;
    f2 d[L::P::SIZE], dx[L::P::SIZE];        // (d, d), (d x, d x)
    f2 b[L::TT][NS / 2 * LPC], c[L::TT][NS / 2 * LPC];
    float y[L::P::SIZE];
    __align__(8) float bias[L::CH], skip[L::CH];  // dt_bias and D of the channels
};

// MAIN: the outputs (and states).  Otherwise only a segment's own end state from a zero start and
// the sum of its step sizes, for the join.
template <typename T, int LPC, int NS, bool MAIN>
__global__ void __launch_bounds__(NT, 4) scan_fwd_kernel(const ScanArgs a, const Cut cut,
                                                      float* rec_h, float* rec_d,
                                                      const float* h0) {
    using L = Lay<LPC, NS>;
    using P = typename L::P;
    constexpr int TT = L::TT, LC = L::LC, CH = L::CH, NV = L::NV, PB = L::PB, NQ = L::NQ, U = L::U;
    constexpr int H = NS / 2;
    __shared__ __align__(16) Smem<LPC, NS> sm;
    const Where<CH> w(a, cut);
    if (MAIN) check_offsets(a.seqs, a.header);
    else if (w.seg + 1 == cut.segs) return;  // nothing follows the last segment
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int q = lane & (LPC - 1), lch = warp * LC + lane / LPC;
    const int N = (int)a.N, nn = max(0, min(NS, N - NS * q));  // this lane's states
    const bool vn = N % (NS < 4 ? NS : 4) == 0;
    const int64_t t0 = w.seg * cut.seg_len, t1 = min64(t0 + cut.seg_len, a.seqs.L);
    const int64_t row0 = w.b * a.seqs.L, C = a.C, c = w.c0 + lch;
    const bool own = c < w.clim;
    const int64_t off = c * N + NS * q;  // of this lane's states in [C, N]

    f2 A2[H], h[H];
    float sd = 0.0f;
#pragma unroll
    for (int i = 0; i < H; ++i) A2[i] = h[i] = 0;
    if (own) load_pairs<NS>(a.A + off, nn, vn, A2);
#pragma unroll
    for (int i = 0; i < H; ++i) A2[i] = mul2(A2[i], pack(kLog2e, kLog2e));
    auto begin_state = [&](int64_t seq) {  // a sequence's first state
#pragma unroll
        for (int i = 0; i < H; ++i) h[i] = 0;
        if (h0 != nullptr && own) load_pairs<NS>(h0 + seq * C * N + off, nn, vn, h);
    };
    auto put_state = [&](float* p) {  // p: [C, N]
        if (own) store_pairs<NS>(p + off, nn, vn, h);
    };
    SeqAt sq = seq_at(a.seqs, w.b, t0);
    bool cutoff = false;  // a sequence begins in this segment: nothing before it reaches its end
    const int64_t rec = (w.b * cut.segs + w.seg) * C;
    if (t0 == sq.begin) {
        begin_state(sq.seq);
        cutoff = true;
    } else if (MAIN && own) {
        load_pairs<NS>(rec_h + rec * N + off, nn, vn, h);
    }

    // staging: one piece of eight channels of one token
    const int64_t cg = C / a.G;
    const bool vec = rows16<T>(cg, a.ldx) && rows16<T>(cg, a.lddt) && rows16<T>(cg, a.ldz) && rows16<T>(cg, a.ldy);
    const bool vecb = rows16<T>(N, a.ldb) && rows16<T>(N, a.ldc);
    const int pv = tid % NV, pt = tid / NV;
    const bool stages = pt < TT;
    const int64_t pch = w.c0 + pv * 8;
    const int pn = stages ? (int)max64(0, min64(8, w.clim - pch)) : 0;
    for (int k = tid; k < CH; k += NT) {
        const bool in = w.c0 + k < w.clim;
        sm.bias[k] = in && a.dt_bias != nullptr ? a.dt_bias[w.c0 + k] : 0.0f;
        sm.skip[k] = MAIN && in && a.D != nullptr ? a.D[w.c0 + k] : 0.0f;
    }
    __syncthreads();
    const T *px = (const T*)a.x + (row0 + t0 + pt) * a.ldx + pch;
    const T *pdt = (const T*)a.dt + (row0 + t0 + pt) * a.lddt + pch;
    const T *pz = (const T*)a.z + (row0 + t0 + pt) * a.ldz + pch;
    T* py = (T*)a.y + (row0 + t0 + pt) * a.ldy + pch;
    const T *pb[PB], *pc[PB];
    int bn[PB], bt[PB];  // states of a piece of Bm and Cm, its token in a tile
#pragma unroll
    for (int i = 0; i < PB; ++i) {
        const int e = tid + i * NT, n0 = e % NQ * 8;
        bt[i] = e / NQ;
        bn[i] = bt[i] < TT ? max(0, min(8, N - n0)) : 0;
        pb[i] = (const T*)a.Bm + (row0 + t0 + bt[i]) * a.ldb + w.grp * N + n0;
        pc[i] = (const T*)a.Cm + (row0 + t0 + bt[i]) * a.ldc + w.grp * N + n0;
    }
    Raw<T> rx, rdt, rz, rb[PB], rc[PB];
    auto fetch = [&](int left) {  // the next tile, of which `left` tokens are the segment's
        const int n = pt < left ? pn : 0;
        rx.load(px, n, vec);
        rdt.load(pdt, n, vec);
        px += TT * a.ldx;
        pdt += TT * a.lddt;
        if (MAIN && a.z != nullptr) {
            rz.load(pz, n, vec);
            pz += TT * a.ldz;
        }
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int m = bt[i] < left ? bn[i] : 0;
            rb[i].load(pb[i], m, vecb);
            pb[i] += TT * a.ldb;
            if (MAIN) {
                rc[i].load(pc[i], m, vecb);
                pc[i] += TT * a.ldc;
            }
        }
    };
    Raw<T> kx, kz;  // the current tile's x and z, for its outputs
    auto commit = [&]() {
        if (stages) {
            f2 fx[4], fd[4];
            rx.get(fx);
            rdt.get(fd);
            const f2* bias = reinterpret_cast<const f2*>(&sm.bias[pv * 8]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f2 v = add2(fd[j], bias[j]), d = a.softplus ? softplus2(v) : v;
                put_doubled<P>(sm.d, pt, pv * 8 + 2 * j, d);
                put_doubled<P>(sm.dx, pt, pv * 8 + 2 * j, mul2(d, fx[j]));
            }
        }
        if (MAIN) {
            kx = rx;
            kz = rz;
        }
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int e = tid + i * NT, tl = e / NQ, n0 = e % NQ * 8;
            if (tl >= TT) break;
            float f[8];
            rb[i].get(f);
            put_states<NS, LPC>(sm.b[tl], n0, f);
            if (MAIN) {
                rc[i].get(f);
                put_states<NS, LPC>(sm.c[tl], n0, f);
            }
        }
    };
    // one token: the recurrence, and this lane's part of the output
    auto step = [&](int tl) {
        const f2 d = sm.d[P::at(tl, lch)], dx = sm.dx[P::at(tl, lch)];
        f2 part = 0, half = 0;  // two chains of sums
#pragma unroll
        for (int i = 0; i < H; ++i) {
            h[i] = fma2(decay2(d, A2[i]), h[i], mul2(dx, sm.b[tl][i * LPC + q]));
            if (MAIN) {
                f2& p = i < (H + 1) / 2 ? part : half;
                p = i == 0 || i == (H + 1) / 2 ? mul2(h[i], sm.c[tl][i * LPC + q]) : fma2(h[i], sm.c[tl][i * LPC + q], p);
            }
        }
        if (H > 1) part = add2(part, half);
        if (!MAIN) {
            float u, v;
            unpack(d, u, v);
            sd += u;
        }
        return sum2(part);
    };

    auto outputs = [&](float* part, int tl) {  // over the channel's lanes; a lane keeps some of the tokens
        if (MAIN) {
            const int at = spread_sum<U, 1, LPC>(part, lane);
#pragma unroll
            for (int i = 0; i < spread_left(U, LPC); ++i)
                if (LPC <= U || q < U) sm.y[P::at(tl + at + i, lch)] = part[i];
        }
    };

    // tokens left in the segment and in the sequence (a row has less than 2^31)
    int left = (int)(t1 - t0), inside = (int)(sq.end - t0);
    // where the states before each 16 tokens go
    float* keep = MAIN && a.states != nullptr
                      ? a.states + (w.b * ((a.seqs.L + CK - 1) / CK) + t0 / CK) * C * N + off : nullptr;
    int until = 0;  // tokens until the next of them
    auto keep_state = [&]() {
        if (!MAIN || keep == nullptr) return;
        if (until == 0) {
            if (own) store_pairs<NS>(keep, nn, vn, h);
            keep += C * N;
            until = CK;
        }
        until -= U;
    };
    fetch(left);
    for (; left > 0; left -= TT, inside -= TT) {
        commit();
        __syncthreads();
        if (left > TT) fetch(left - TT);
        if (left >= TT && inside >= TT) {
#pragma unroll 1
            for (int tl = 0; tl < TT; tl += U) {
                keep_state();
                float part[U];
#pragma unroll
                for (int i = 0; i < U; ++i) part[i] = step(tl + i);
                outputs(part, tl);
            }
        } else {
            const int n = min(TT, left);
#pragma unroll 1
            for (int tl = 0; tl < n; tl += U) {
                keep_state();
                float part[U];
#pragma unroll
                for (int i = 0; i < U; ++i) part[i] = 0.0f;
#pragma unroll 1
                for (int i = 0; i < U && tl + i < n; ++i) {
                    if (tl + i == inside) {
                        if (MAIN && a.h_out != nullptr) put_state(a.h_out + sq.seq * C * N);
                        const int64_t at = sq.end;
                        sq = seq_at(a.seqs, w.b, at);
                        inside += (int)(sq.end - at);
                        begin_state(sq.seq);
                        cutoff = true;
                    }
                    const float p = step(tl + i);
#pragma unroll
                    for (int k = 0; k < U; ++k)
                        if (k == i) part[k] = p;
                }
                outputs(part, tl);
            }
        }
        __syncthreads();
        if (MAIN && stages) {
            f2 fx[4], o[4];
            kx.get(fx);
            const f2* skip = reinterpret_cast<const f2*>(&sm.skip[pv * 8]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = pv * 8 + 2 * j;
                o[j] = fma2(skip[j], fx[j], pack(sm.y[P::at(pt, k)], sm.y[P::at(pt, k + 1)]));
            }
            if (a.z != nullptr) {
                f2 fz[4];
                kz.get(fz);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = mul2(o[j], mul2(fz[j], sigm2<is_fast<T>()>(fz[j])));
            }
            store8(py, o, pt < left ? pn : 0, vec);
            py += TT * a.ldy;
        }
    }
    if (MAIN) {
        if (t1 == sq.end && a.h_out != nullptr) put_state(a.h_out + sq.seq * C * N);
    } else {
        put_state(rec_h + rec * N);
        if (own && q == 0) rec_d[rec + c] = cutoff ? __int_as_float(0x7fc00000) : sd;
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
    float* p = rec_h + b * segs * CN + cn;
    const float* pd = rec_d + b * segs * a.C + c;
    constexpr int U = 8;  // records read together: each is a trip to memory
    for (int64_t s = 0; s < segs; s += U) {
        float own[U], d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = s + u + 1 < segs;  // the last segment's own end state is not needed
            own[u] = in ? p[(s + u) * CN] : 0.0f;
            d[u] = in ? pd[(s + u) * a.C] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= segs) break;
            p[(s + u) * CN] = h;
            h = isnan(d[u]) ? own[u] : fmaf(ex2(d[u] * A2), h, own[u]);
        }
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
    constexpr int NS = 4;
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
        load_n<NS>(a.state + (slot * a.C + c) * N + NS * q, nn, v4, h);
        load_n<NS>(a.A + c * N + NS * q, nn, v4, A);
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
        h[i] = fmaf(ex2(fmaf(d, A[i] * kLog2e, kDecayShift)), h[i], dx * bb[i]);
        y = fmaf(cc[i], h[i], y);
    }
#pragma unroll
    for (int o = 1; o < LPC; o *= 2) y += __shfl_xor_sync(~0u, y, o);
    if (!own) return;
    store_n<NS>(a.state + (slot * a.C + c) * N + NS * q, nn, N % 4 == 0, h);
    if (q != 0) return;
    if (a.D != nullptr) y = fmaf(a.D[c], x, y);
    if (a.z != nullptr) {
        const float z = ld((const T*)a.z + b * a.ldz + c);
        y *= z * sigm<is_fast<T>()>(z);
    }
    st((T*)a.y + b * a.ldy + c, y);
}

// Calls f with l, one of LPC, 2 LPC, ... MOST, as a constant.
template <int LPC, int MOST, typename F>
cudaError_t with_lanes(int l, F&& f) {
    if constexpr (LPC > MOST) return cudaErrorInvalidValue;
    else return l == LPC ? f(std::integral_constant<int, LPC>()) : with_lanes<LPC * 2, MOST>(l, f);
}

// Calls f with the lanes a channel and the states a lane, as constants.  Eight states a lane keep
// the sums over a channel's lanes cheapest (8 x 2048 x 4096 x 16: 451 us, with four a lane 490).
template <typename F>
cudaError_t with_lay(const ScanArgs& a, F&& f) {
    using std::integral_constant;
    const int np = padded_states(a.N);
    if (np == 4) return f(integral_constant<int, 1>(), integral_constant<int, 4>());
    if (np == 8) return f(integral_constant<int, 2>(), integral_constant<int, 4>());
    return with_lanes<2, 8>(np / 8, [&](auto l) { return f(l, integral_constant<int, 8>()); });
}
int channels_of(const ScanArgs& a) {
    const int np = padded_states(a.N);
    return NT * (np >= 16 ? 8 : 4) / np;
}

// The forward's cut.  One pass over the whole time axis computes the least; where that leaves
// about a CTA for each of 152 SMs or fewer, the axis is cut into segments for two rounds of the
// four CTAs a SM holds, although their end states then take a pass of their own, half as long as
// the outputs' (8192 x 4096 x 16: 64 CTAs 1000 us, cut into 16 x 64 335 us; 65536 x 1024 x 16:
// 16 CTAs cut into 32 x 16 793 us, 64 x 16 686 us, 128 x 16 717 us).
Cut fwd_cut(const ScanArgs& a) {
    const int ch = channels_of(a);
    Cut k;
    k.cbg = (a.C / a.G + ch - 1) / ch;
    k.cblocks = k.cbg * a.G;
    k.segs = 1;
    k.seg_len = a.seqs.L;
    const int64_t ctas = a.B * k.cblocks;
    if (ctas > 180 || a.seqs.L <= 4 * SEG) return k;
    const int64_t want = (8 * 152 + ctas - 1) / ctas;
    k.seg_len = ((a.seqs.L + want - 1) / want + SEG - 1) / SEG * SEG;
    k.segs = (a.seqs.L + k.seg_len - 1) / k.seg_len;
    return k;
}

// The segments' records, rounded up to 16 bytes: the copy of the first states after them is read in
// pieces of four values.
size_t rec_floats(const ScanArgs& a, const Cut& k) {
    return k.segs > 1 ? ((size_t)(a.B * k.segs * a.C) * (a.N + 1) + 3) & ~(size_t)3 : 0;
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
    return with_lay(a, [&](auto ll, auto nn) {
        constexpr int LPC = decltype(ll)::value, NS = decltype(nn)::value;
        const unsigned g = (unsigned)(a.B * k.segs * k.cblocks);
        if (k.segs > 1) {
            scan_fwd_kernel<T, LPC, NS, false><<<g, NT, 0, s>>>(a, k, rec_h, rec_d, h0);
            scan_join_kernel<<<(unsigned)((a.B * w + 255) / 256), 256, 0, s>>>(a, k.segs, rec_h, rec_d);
        }
        scan_fwd_kernel<T, LPC, NS, true><<<g, NT, 0, s>>>(a, k, rec_h, rec_d, h0);
        return cudaGetLastError();
    });
}

template <typename T>
cudaError_t scan_step(const ScanArgs& a, cudaStream_t s) {
    return with_lanes<1, 16>(padded_states(a.N) / 4, [&](auto ll) {
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
