// Norm after a block, gate, residual scale and add, and the norm before the next block
// (lizard_block_norm_*), one pass over the row.
//
//   u = o [act(gate)],  n = w_post u / rms_group(u),  n [act(gate)],  rr = r + scale n,
//   r_out = rr,  n_out = w_pre rr / rms(rr)
//
// Bound by HBM: each row is read once (V neighbouring columns a piece, NV pieces a thread), the sums
// of squares are reduced inside the CTA, and both outputs leave from registers.  16384 x 4096 bf16
// with gate, residual and both norms: 129 us, 5.2 TB/s; without the next row on its way 153 us; the
// norm over 32 heads with its gate, 8192 x 4096: 38 us, 5.3 TB/s.  Backward of the former: 283 us,
// 3.8 TB/s: one row at a time a SM, three sums over the row, each with a barrier, between its loads
// and its stores; with the parameters read again for each row and their sums in shared memory
// 366 us, with four columns a thread 402 us.
#include <type_traits>

#include "selective.h"

namespace lz {
namespace {

constexpr int kSumsWidth = 8192;  // widest row whose parameter sums fit into shared memory

// Sum over a CTA's (TPR > 32) or a warp's threads, the same value in each of them.  Consecutive
// sums of a CTA alternate between two buffers: the barrier of the one in between is what lets a
// buffer be written again.
template <int TPR, int NVAL>
__device__ __forceinline__ void row_sum(float* v, float (*red)[32]) {
#pragma unroll
    for (int k = 0; k < NVAL; ++k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(~0u, v[k], o);
    if constexpr (TPR > 32) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < NVAL; ++k) red[k][warp] = v[k];
        __syncthreads();
        constexpr int W = TPR / 32;
#pragma unroll
        for (int k = 0; k < NVAL; ++k) {
            if constexpr (W >= 4 && W <= 16) {  // broadcast loads and a tree: shorter than a second round of shuffles
                f2 t[W / 2];
#pragma unroll
                for (int i = 0; i < W / 4; ++i) {
                    const float4 q = reinterpret_cast<const float4*>(red[k])[i];
                    t[2 * i] = pack(q.x, q.y);
                    t[2 * i + 1] = pack(q.z, q.w);
                }
#pragma unroll
                for (int o = W / 4; o > 0; o >>= 1)
#pragma unroll
                    for (int i = 0; i < o; ++i) t[i] = add2(t[i], t[i + o]);
                v[k] = sum2(t[0]);
            } else {
                v[k] = lane < W ? red[k][lane] : 0.0f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(~0u, v[k], o);
            }
        }
    }
}

// Sums over the groups of a row: p[i] is this thread's sum over piece i, and becomes the sum over
// that piece's whole group.  gv pieces make a group.
template <int TPR, int NV>
__device__ __forceinline__ void group_sum(float* p, int nvec, int gv, float* sm, int lane_in_row) {
    if (gv <= 32 && (gv & (gv - 1)) == 0) {  // a group's pieces are neighbouring lanes
#pragma unroll
        for (int i = 0; i < NV; ++i)
            for (int o = 1; o < gv; o <<= 1) p[i] += __shfl_xor_sync(~0u, p[i], o);
        return;
    }
    float *part = sm, *sum = sm + nvec;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int vi = i * TPR + lane_in_row;
        if (vi < nvec) part[vi] = p[i];
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, groups = nvec / gv;
    for (int g = warp; g < groups; g += TPR / 32) {
        float s = 0.0f;
        for (int e = lane; e < gv; e += 32) s += part[g * gv + e];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        if (lane == 0) sum[g] = s;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int vi = i * TPR + lane_in_row;
        if (vi < nvec) p[i] = sum[vi / gv];
    }
}

// A thread's columns of a row, in pairs: NV pieces of V neighbouring columns each, piece i at
// column (i TPR + lane) V.  With V = 1 a pair is two pieces.
template <int V, int TPR, int NV>
struct Cols {
    static constexpr int NP = V * NV / 2;
    template <typename T>
    static __device__ __forceinline__ void ld(const T* row, int lr, int nvec, f2* f) {
        if constexpr (V == 1) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int c = 2 * k * TPR + lr;
                f[k] = pack(c < nvec ? lz::ld(row + c) : 0.0f, c + TPR < nvec ? lz::ld(row + c + TPR) : 0.0f);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i * TPR + lr < nvec) {
                    get2(*reinterpret_cast<const Pack<T, V>*>(row + (i * TPR + lr) * V), f + i * V / 2);
                } else {
#pragma unroll
                    for (int k = 0; k < V / 2; ++k) f[i * V / 2 + k] = 0;
                }
            }
        }
    }
    template <typename T>
    static __device__ __forceinline__ void st(T* row, int lr, int nvec, const f2* f) {
        if constexpr (V == 1) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int c = 2 * k * TPR + lr;
                float x, y;
                unpack(f[k], x, y);
                if (c < nvec) lz::st(row + c, x);
                if (c + TPR < nvec) lz::st(row + c + TPR, y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i * TPR + lr >= nvec) continue;
                float v[V];
#pragma unroll
                for (int k = 0; k < V / 2; ++k) unpack(f[i * V / 2 + k], v[2 * k], v[2 * k + 1]);
                Vec<V>::st(row + (i * TPR + lr) * V, v);
            }
        }
    }
    // the sum of a b over each piece
    static __device__ __forceinline__ void pieces(const f2* a, const f2* b, float* p) {
        if constexpr (V == 1) {
#pragma unroll
            for (int k = 0; k < NP; ++k) unpack(mul2(a[k], b[k]), p[2 * k], p[2 * k + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                f2 s = mul2(a[i * V / 2], b[i * V / 2]);
#pragma unroll
                for (int k = 1; k < V / 2; ++k) s = fma2(a[i * V / 2 + k], b[i * V / 2 + k], s);
                p[i] = sum2(s);
            }
        }
    }
    // piece i's value at pair k
    static __device__ __forceinline__ f2 at(const float* p, int k) {
        if constexpr (V == 1) return pack(p[2 * k], p[2 * k + 1]);
        else return pack(p[k / (V / 2)], p[k / (V / 2)]);
    }
};

// The next row's pieces of one tensor on their way into shared memory, each thread's own; not ON:
// rows are read directly.
template <typename T, int V, int TPR, int NV, bool ON>
struct Ahead {
    T* at;  // [nvec V]
    __device__ __forceinline__ void fetch(const T* row, int lr, int nvec, size_t offset = 0) const {
        if constexpr (ON) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + lr) * V;
                if (i * TPR + lr < nvec) copy_async<T, V>((T*)((char*)at + offset) + c, row + c);
            }
        }
    }
    __device__ __forceinline__ void get(const T* row, int lr, int nvec, f2* f, size_t offset = 0) const {
        Cols<V, TPR, NV>::ld(ON ? (const T*)((const char*)at + offset) : row, lr, nvec, f);
    }
};

// Whether the backward's rows fit ahead, next to the parameter sums, into a SM's 227 KB.
template <typename T, int V, int TPR>
constexpr bool rows_ahead() { return V > 1 && (TPR < 512 || (TPR == 512 && sizeof(T) == 2)); }

template <int NP>
__device__ __forceinline__ float dot_of(const f2* a, const f2* b) {
    f2 s = mul2(a[0], b[0]);
#pragma unroll
    for (int k = 1; k < NP; ++k) s = fma2(a[k], b[k], s);
    return sum2(s);
}

// TPR threads a row (32: four rows a CTA of 128, else one row a CTA), which walk rows at a distance
// of all rows that are worked on at once, the next row's values on their way meanwhile.
template <typename T, typename R, int V, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, TPR < 768 ? 768 / (TPR < 128 ? 128 : TPR) : 1)
    norm_fwd_kernel(const NormArgs a) {
    using C = Cols<V, TPR, NV>;
    constexpr int NP = C::NP, RPC = TPR < 128 ? 128 / TPR : 1;
    constexpr bool FAST = is_fast<T>();
    __shared__ __align__(16) float red[2][1][32];
    extern __shared__ __align__(16) float gsm[];  // the group sums' space, then the rows ahead
    const int lr = threadIdx.x % TPR, rc = threadIdx.x / TPR;
    const int D = (int)a.D, nvec = D / V, gv = nvec / (int)a.groups;
    char* ahead = (char*)gsm + a.group_bytes + (size_t)rc * D * (2 * sizeof(T) + sizeof(R));
    const Ahead<R, V, TPR, NV, (V > 1)> ar{(R*)ahead};
    const Ahead<T, V, TPR, NV, (V > 1)> ao{(T*)(ahead + D * sizeof(R))}, ag{ao.at + D};
    const int64_t step = (int64_t)gridDim.x * RPC;
    auto fetch = [&](int64_t row) {  // two groups: what a row begins with, and its residual
        if (row < a.T) {
            ao.fetch((const T*)a.o + row * a.ldo, lr, nvec);
            if (a.gate != nullptr) ag.fetch((const T*)a.gate + row * a.ldg, lr, nvec);
        }
        copy_commit();
    };
    auto fetch_r = [&](int64_t row) {
        if (row < a.T && a.r != nullptr) ar.fetch((const R*)a.r + row * a.ldr, lr, nvec);
        copy_commit();
    };
    int64_t row = (int64_t)blockIdx.x * RPC + rc;
    fetch(row);
    fetch_r(row);
    int buf = 0;
    for (; row < a.T; row += step) {
        f2 n[NP], ga[NP], rr[NP], w[NP];
        copy_wait<1>();
        ao.get((const T*)a.o + row * a.ldo, lr, nvec, n);
        if (a.gate != nullptr) ag.get((const T*)a.gate + row * a.ldg, lr, nvec, ga);
        fetch(row + step);
        if (a.gate != nullptr) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const f2 sg = sigm2<FAST>(ga[k]);
                ga[k] = a.act == LIZARD_ACT_SILU ? mul2(ga[k], sg) : sg;
                if (a.gate_first) n[k] = mul2(n[k], ga[k]);
            }
        }
        if (a.w_post != nullptr) {
            C::ld(a.w_post, lr, nvec, w);
            if (a.groups == 1) {
                float all[1] = {dot_of<NP>(n, n)};
                row_sum<TPR, 1>(all, red[buf]);
                buf ^= 1;
                const float rs = rsqrtf(all[0] / (float)D + a.eps_post);
#pragma unroll
                for (int k = 0; k < NP; ++k) n[k] = mul2(n[k], mul2(w[k], pack(rs, rs)));
            } else {
                float p[NV];
                C::pieces(n, n, p);
                group_sum<TPR, NV>(p, nvec, gv, gsm, lr);
                const float inv = 1.0f / (float)(gv * V);
#pragma unroll
                for (int i = 0; i < NV; ++i)  // columns past the row stay zero, whatever eps is
                    p[i] = i * TPR + lr < nvec ? rsqrtf(fmaf(p[i], inv, a.eps_post)) : 0.0f;
#pragma unroll
                for (int k = 0; k < NP; ++k) n[k] = mul2(n[k], mul2(w[k], C::at(p, k)));
            }
        }
        if (a.gate != nullptr && !a.gate_first) {
#pragma unroll
            for (int k = 0; k < NP; ++k) n[k] = mul2(n[k], ga[k]);
        }
        copy_wait<1>();
        if (a.r != nullptr) ar.get((const R*)a.r + row * a.ldr, lr, nvec, rr);
        fetch_r(row + step);
        if (a.scale != nullptr) {
            C::ld(a.scale, lr, nvec, w);
#pragma unroll
            for (int k = 0; k < NP; ++k) n[k] = a.r != nullptr ? fma2(w[k], n[k], rr[k]) : mul2(w[k], n[k]);
        } else if (a.r != nullptr) {
#pragma unroll
            for (int k = 0; k < NP; ++k) n[k] = add2(n[k], rr[k]);
        }
        if (a.r_out != nullptr) C::st((R*)a.r_out + row * a.ldro, lr, nvec, n);
        if (a.n_out == nullptr) continue;
        C::ld(a.w_pre, lr, nvec, w);
        float all[1] = {dot_of<NP>(n, n)};
        row_sum<TPR, 1>(all, red[buf]);
        buf ^= 1;
        const float rs = rsqrtf(all[0] / (float)D + a.eps_pre);
#pragma unroll
        for (int k = 0; k < NP; ++k) n[k] = mul2(n[k], mul2(w[k], pack(rs, rs)));
        C::st((T*)a.n_out + row * a.ldn, lr, nvec, n);
    }
    copy_wait<0>();
}

// One CTA walks rows b, b + grid, ...  The parameter gradients of a thread's columns are summed as
// the rows go by and leave once.  HOLD (rows up to 4096 columns, eight a thread): the parameters
// and their sums stay in registers, and two rows are on their way in shared memory.  Otherwise
// sixteen columns a thread, the sums in shared memory (the widest rows: in the CTA's partial sums
// themselves), in the thread's own places, the parameters read again for each row.
template <typename T, typename R, int V, int TPR, int NV, bool HOLD>
__global__ void __launch_bounds__(TPR, TPR >= 512 ? 1 : 512 / TPR) norm_bwd_kernel(const NormArgs a) {
    using C = Cols<V, TPR, NV>;
    constexpr int NP = C::NP;
    constexpr bool ON = HOLD || rows_ahead<T, V, TPR>();
    constexpr int S = HOLD ? 2 : 1;  // rows on their way
    constexpr bool FAST = is_fast<T>();
    __shared__ __align__(16) float red[2][2][32];
    // [3][D] up to kSumsWidth columns, the group sums' space, the row ahead
    extern __shared__ __align__(16) float gsm[];
    const int lr = threadIdx.x;
    const int D = (int)a.D, nvec = D / V, gv = nvec / (int)a.groups;
    float* partial = a.partial + (int64_t)blockIdx.x * 3 * D;
    const bool near = !HOLD && D <= kSumsWidth;
    float *sums = near ? gsm : partial, *gspace = near ? gsm + 3 * D : gsm;
    f2 held[3][HOLD ? NP : 1], param[3][HOLD ? NP : 1];  // sums of, and w_post, scale, w_pre
    const float* const params[3] = {a.w_post, a.scale, a.w_pre};
#pragma unroll
    for (int m = 0; m < 3; ++m) {
        if constexpr (HOLD) {
#pragma unroll
            for (int k = 0; k < NP; ++k) held[m][k] = 0;
            if (params[m] != nullptr) C::ld(params[m], lr, nvec, param[m]);
        } else {
            f2 zero[NP];
#pragma unroll
            for (int k = 0; k < NP; ++k) zero[k] = 0;
            C::st(sums + m * D, lr, nvec, zero);
        }
    }
    auto get_param = [&](auto m, f2* w) {
        if constexpr (HOLD) {
#pragma unroll
            for (int k = 0; k < NP; ++k) w[k] = param[decltype(m)::value][k];
        } else {
            C::ld(params[decltype(m)::value], lr, nvec, w);
        }
    };
    using W0 = std::integral_constant<int, 0>;  // w_post
    using W1 = std::integral_constant<int, 1>;  // scale
    using W2 = std::integral_constant<int, 2>;  // w_pre
    auto add_to = [&](auto mm, const f2* v) {
        constexpr int m = decltype(mm)::value;
        if constexpr (HOLD) {
#pragma unroll
            for (int k = 0; k < NP; ++k) held[m][k] = add2(held[m][k], v[k]);
            return;
        }
        f2 s[NP];
        C::ld(sums + m * D, lr, nvec, s);
#pragma unroll
        for (int k = 0; k < NP; ++k) s[k] = add2(s[k], v[k]);
        C::st(sums + m * D, lr, nvec, s);
    };
    const bool gate = a.gate != nullptr, gfirst = gate && a.gate_first, glast = gate && !a.gate_first;
    const float ginv = 1.0f / (float)(gv * V), dinv = 1.0f / (float)D;
    char* ahead = (char*)gspace + a.group_bytes;
    const size_t row_bytes = (size_t)D * (3 * sizeof(T) + 2 * sizeof(R));
    const Ahead<R, V, TPR, NV, ON> ad{(R*)ahead}, ar{ad.at + D};
    const Ahead<T, V, TPR, NV, ON> ao{(T*)(ar.at + D)}, ag{ao.at + D}, an{ag.at + D};
    // two groups of a row: what it begins with, and what comes later
    auto fetch = [&](int64_t row, int slot) {
        if (row < a.T) {
            ao.fetch((const T*)a.o + row * a.ldo, lr, nvec, slot * row_bytes);
            if (gate) ag.fetch((const T*)a.gate + row * a.ldg, lr, nvec, slot * row_bytes);
        }
        copy_commit();
    };
    auto fetch_later = [&](int64_t row, int slot) {
        if (row < a.T) {
            if (a.dr_out != nullptr) ad.fetch((const R*)a.dr_out + row * a.ldro, lr, nvec, slot * row_bytes);
            if (a.w_pre != nullptr) {
                if (a.r != nullptr) ar.fetch((const R*)a.r + row * a.ldr, lr, nvec, slot * row_bytes);
                an.fetch((const T*)a.dn_out + row * a.ldn, lr, nvec, slot * row_bytes);
            }
        }
        copy_commit();
    };
    const int64_t next = (int64_t)gridDim.x * S;  // from a row to the one its place is for next
    for (int k = 0; k < S; ++k) {
        fetch(blockIdx.x + (int64_t)k * gridDim.x, k);
        fetch_later(blockIdx.x + (int64_t)k * gridDim.x, k);
    }
    int slot = 0;
    int buf = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        // u: the normalised row (the plain one without a norm); ga, gd: act(gate), its derivative
        f2 u[NP], ga[NP], gd[NP], dr[NP], w[NP];
        copy_wait<2 * S - 1>();
        ao.get((const T*)a.o + row * a.ldo, lr, nvec, u, slot * row_bytes);
        if (gate) ag.get((const T*)a.gate + row * a.ldg, lr, nvec, ga, slot * row_bytes);
        fetch(row + next, slot);
        if (gate) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const f2 sg = sigm2<FAST>(ga[k]);
                if (a.act == LIZARD_ACT_SILU) {
                    gd[k] = dsilu2(ga[k], sg);
                    ga[k] = mul2(ga[k], sg);
                } else {
                    gd[k] = mul2(sg, fma2(sg, pack(-1.0f, -1.0f), pack(1.0f, 1.0f)));
                    ga[k] = sg;
                }
                if (gfirst) {
                    gd[k] = mul2(gd[k], u[k]);
                    u[k] = mul2(u[k], ga[k]);
                }
            }
        }
        float rs[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) rs[i] = 1.0f;
        if (a.w_post != nullptr) {
            if (a.groups == 1) {
                float all[1] = {dot_of<NP>(u, u)};
                row_sum<TPR, 1>(all, red[buf]);
                buf ^= 1;
#pragma unroll
                for (int i = 0; i < NV; ++i) rs[i] = rsqrtf(fmaf(all[0], ginv, a.eps_post));
            } else {
                C::pieces(u, u, rs);
                group_sum<TPR, NV>(rs, nvec, gv, gspace, lr);
#pragma unroll
                for (int i = 0; i < NV; ++i)  // columns past the row stay zero, whatever eps is
                    rs[i] = i * TPR + lr < nvec ? rsqrtf(fmaf(rs[i], ginv, a.eps_post)) : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < NP; ++k) u[k] = mul2(u[k], C::at(rs, k));
        }
        // the gradient of rr
        copy_wait<2 * S - 1>();
        if (a.dr_out != nullptr) {
            ad.get((const R*)a.dr_out + row * a.ldro, lr, nvec, dr, slot * row_bytes);
        } else {
#pragma unroll
            for (int k = 0; k < NP; ++k) dr[k] = 0;
        }
        // what the block adds to the residual, before its scale, times f
        auto added = [&](const f2* f, f2* n) {
            if (a.w_post != nullptr) {
                get_param(W0(), n);
#pragma unroll
                for (int k = 0; k < NP; ++k) n[k] = mul2(n[k], mul2(u[k], f[k]));
            } else {
#pragma unroll
                for (int k = 0; k < NP; ++k) n[k] = mul2(u[k], f[k]);
            }
            if (glast) {
#pragma unroll
                for (int k = 0; k < NP; ++k) n[k] = mul2(n[k], ga[k]);
            }
        };
        if (a.w_pre != nullptr) {
            f2 rr[NP], dn[NP];
            if (a.scale != nullptr) {
                get_param(W1(), w);
            } else {
#pragma unroll
                for (int k = 0; k < NP; ++k) w[k] = pack(1.0f, 1.0f);
            }
            added(w, rr);
            if (a.r != nullptr) {
                ar.get((const R*)a.r + row * a.ldr, lr, nvec, w, slot * row_bytes);
#pragma unroll
                for (int k = 0; k < NP; ++k) rr[k] = add2(rr[k], w[k]);
            }
            an.get((const T*)a.dn_out + row * a.ldn, lr, nvec, dn, slot * row_bytes);
            get_param(W2(), w);
#pragma unroll
            for (int k = 0; k < NP; ++k) w[k] = mul2(w[k], dn[k]);
            float all[2] = {dot_of<NP>(rr, rr), dot_of<NP>(w, rr)};
            row_sum<TPR, 2>(all, red[buf]);
            buf ^= 1;
            const float rp = rsqrtf(fmaf(all[0], dinv, a.eps_pre)), c = -all[1] * dinv * rp * rp;
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                dr[k] = fma2(fma2(rr[k], pack(c, c), w[k]), pack(rp, rp), dr[k]);
                dn[k] = mul2(dn[k], mul2(rr[k], pack(rp, rp)));
            }
            add_to(W2(), dn);
        }
        fetch_later(row + next, slot);
        if (S > 1) slot ^= 1;
        if (a.dr != nullptr) C::st((R*)a.dr + row * a.lddr, lr, nvec, dr);
        f2 t[NP];
        if (a.scale != nullptr) {
            added(dr, t);
            add_to(W1(), t);
            get_param(W1(), w);
#pragma unroll
            for (int k = 0; k < NP; ++k) dr[k] = mul2(dr[k], w[k]);
        }
        if (glast) {
            if (a.w_post != nullptr) {
                get_param(W0(), t);
#pragma unroll
                for (int k = 0; k < NP; ++k) t[k] = mul2(t[k], u[k]);
            } else {
#pragma unroll
                for (int k = 0; k < NP; ++k) t[k] = u[k];
            }
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                t[k] = mul2(t[k], mul2(dr[k], gd[k]));
                dr[k] = mul2(dr[k], ga[k]);
            }
            C::st((T*)a.dgate + row * a.lddg, lr, nvec, t);
        }
        if (a.w_post != nullptr) {
#pragma unroll
            for (int k = 0; k < NP; ++k) t[k] = mul2(dr[k], u[k]);
            add_to(W0(), t);
            get_param(W0(), w);
#pragma unroll
            for (int k = 0; k < NP; ++k) dr[k] = mul2(dr[k], w[k]);
            float dot[NV];
            if (a.groups == 1) {
                float all[1] = {dot_of<NP>(dr, u)};
                row_sum<TPR, 1>(all, red[buf]);
                buf ^= 1;
#pragma unroll
                for (int i = 0; i < NV; ++i) dot[i] = all[0];
            } else {
                C::pieces(dr, u, dot);
                group_sum<TPR, NV>(dot, nvec, gv, gspace, lr);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) dot[i] *= -ginv;
#pragma unroll
            for (int k = 0; k < NP; ++k) dr[k] = mul2(fma2(u[k], C::at(dot, k), dr[k]), C::at(rs, k));
        }
        if (gfirst) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                t[k] = mul2(dr[k], gd[k]);
                dr[k] = mul2(dr[k], ga[k]);
            }
            C::st((T*)a.dgate + row * a.lddg, lr, nvec, t);
        }
        C::st((T*)a.d_o + row * a.lddo, lr, nvec, dr);
    }
    copy_wait<0>();
    if constexpr (HOLD) {
#pragma unroll
        for (int m = 0; m < 3; ++m) C::st(partial + m * D, lr, nvec, held[m]);
    } else if (near) {
        f2 s[NP];
        for (int m = 0; m < 3; ++m) {
            C::ld(sums + m * D, lr, nvec, s);
            C::st(partial + m * D, lr, nvec, s);
        }
    }
}

// dw_post, dscale and dw_pre from the CTAs' partial sums [n][3][D].
template <int KT>
__global__ void __launch_bounds__(32 * KT) norm_bwd_sum_kernel(const NormArgs a, int64_t n) {
    const int m = blockIdx.y;
    float* out = m == 0 ? a.dw_post : m == 1 ? a.dscale : a.dw_pre;
    if (out == nullptr) return;
    const int64_t i0 = (int64_t)blockIdx.x * 32;
    sum_columns<KT>(
        n, (int)min64(32, a.D - i0), [&](int64_t p, int i) { return a.partial[(p * 3 + m) * a.D + i0 + i]; },
        [&](int i, float s) { out[i0 + i] = s; });
}

// Raises a kernel's limit of dynamic shared memory where this launch's bytes need it, always to the
// most that any of its launches takes: the limit is the process's, and another thread may launch the
// same kernel with other sizes between this call and the launch.
template <size_t most, typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
    static_assert(most <= 226 * 1024, "with the static part within a SM's 227 KB");
    if (bytes <= 40 * 1024) return cudaSuccess;  // with the static part below the default 48 KB
    if (bytes > most) return cudaErrorInvalidValue;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}

// Shared memory of the group sums that neighbouring lanes cannot do.
size_t group_bytes(const NormArgs& a, int V) {
    const int64_t nvec = a.D / V, gv = nvec / a.groups;
    if (a.groups == 1 || a.w_post == nullptr || (gv <= 32 && (gv & (gv - 1)) == 0)) return 0;
    return (sizeof(float) * (size_t)(nvec + a.groups) + 15) / 16 * 16;
}
// The most of it for rows of nvec pieces: such groups have three pieces or more.
constexpr size_t most_group_bytes(size_t nvec) { return (sizeof(float) * (nvec + nvec / 3) + 15) / 16 * 16; }

template <typename T, typename R, int V, int TPR, int NV>
cudaError_t fwd_go(NormArgs a, cudaStream_t s) {
    constexpr int RPC = TPR < 128 ? 128 / TPR : 1;
    a.group_bytes = group_bytes(a, V);
    const size_t sm = a.group_bytes + (V > 1 ? RPC * (size_t)a.D * (2 * sizeof(T) + sizeof(R)) : 0);
    const auto kernel = norm_fwd_kernel<T, R, V, TPR, NV>;
    constexpr size_t D = V * TPR * NV;  // widest row
    constexpr size_t most_smem = most_group_bytes(D / V) + (V > 1 ? RPC * D * (2 * sizeof(T) + sizeof(R)) : 0);
    const cudaError_t e = allow_smem<most_smem>(kernel, sm);
    if (e != cudaSuccess) return e;
    // as many CTAs as are resident: 768 threads a SM
    const int64_t ctas = (a.T + RPC - 1) / RPC, most = 152 * (TPR >= 768 ? 1 : 768 / (TPR < 128 ? 128 : TPR));
    kernel<<<(unsigned)(ctas < most ? ctas : most), TPR * RPC, sm, s>>>(a);
    return cudaGetLastError();
}

template <typename T, typename R, int V, int TPR, int NV, bool HOLD = false>
cudaError_t bwd_go(NormArgs a, cudaStream_t s) {
    a.group_bytes = group_bytes(a, V);
    const size_t row = (size_t)a.D * (3 * sizeof(T) + 2 * sizeof(R));
    const size_t sm = a.group_bytes + (HOLD ? 2 * row
                                            : sizeof(float) * (a.D <= kSumsWidth ? 3 * (size_t)a.D : 0) +
                                                  (rows_ahead<T, V, TPR>() ? row : 0));
    const auto kernel = norm_bwd_kernel<T, R, V, TPR, NV, HOLD>;
    constexpr size_t D = V * TPR * NV, wide = D * (3 * sizeof(T) + 2 * sizeof(R));  // widest row
    constexpr size_t most_smem = most_group_bytes(D / V) + (HOLD ? 2 * wide
                                                            : sizeof(float) * 3 * (D < kSumsWidth ? D : kSumsWidth) +
                                                                  (rows_ahead<T, V, TPR>() ? wide : 0));
    const cudaError_t e = allow_smem<most_smem>(kernel, sm);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)norm_bwd_ctas(a.T, a.D), TPR, sm, s>>>(a);
    return cudaGetLastError();
}

// Eight columns a piece where the rows and groups allow it, else one.
template <typename T, typename R>
cudaError_t fwd(const NormArgs& a, cudaStream_t s) {
    const bool v8 = a.D % 8 == 0 && (a.D / a.groups) % 8 == 0 && a.ldo % 8 == 0 && a.ldg % 8 == 0 &&
                    a.ldr % 8 == 0 && a.ldro % 8 == 0 && a.ldn % 8 == 0;
    if (v8) {
        if (a.D <= 512 && a.groups == 1) return fwd_go<T, R, 8, 32, 2>(a, s);
        if (a.D <= 1024) return fwd_go<T, R, 8, 128, 1>(a, s);
        if (a.D <= 2048) return fwd_go<T, R, 8, 128, 2>(a, s);
        if (a.D <= 4096) return fwd_go<T, R, 8, 256, 2>(a, s);
        if (a.D <= 8192) return fwd_go<T, R, 8, 512, 2>(a, s);
        return fwd_go<T, R, 8, 1024, 2>(a, s);
    }
    if (a.D <= 1024) return fwd_go<T, R, 1, 256, 4>(a, s);
    if (a.D <= 4096) return fwd_go<T, R, 1, 512, 8>(a, s);
    return fwd_go<T, R, 1, 1024, 16>(a, s);
}

template <typename T, typename R>
cudaError_t bwd(const NormArgs& a, cudaStream_t s) {
    const bool v8 = a.D % 8 == 0 && (a.D / a.groups) % 8 == 0 && a.ldo % 8 == 0 && a.ldg % 8 == 0 &&
                    a.ldr % 8 == 0 && a.ldro % 8 == 0 && a.ldn % 8 == 0 && a.lddo % 8 == 0 &&
                    a.lddg % 8 == 0 && a.lddr % 8 == 0;
    cudaError_t e;
    if (v8) {
        if (a.D <= 512) e = bwd_go<T, R, 8, 64, 1, true>(a, s);
        else if (a.D <= 1024) e = bwd_go<T, R, 8, 128, 1, true>(a, s);
        else if (a.D <= 2048) e = bwd_go<T, R, 8, 256, 1, true>(a, s);
        else if (a.D <= 4096) e = bwd_go<T, R, 8, 512, 1, true>(a, s);
        else if (a.D <= 8192) e = bwd_go<T, R, 8, 512, 2>(a, s);
        else e = bwd_go<T, R, 8, 1024, 2>(a, s);
    } else {
        if (a.D <= 1024) e = bwd_go<T, R, 1, 64, 16>(a, s);
        else if (a.D <= 4096) e = bwd_go<T, R, 1, 256, 16>(a, s);
        else e = bwd_go<T, R, 1, 1024, 16>(a, s);
    }
    if (e != cudaSuccess) return e;
    const int64_t n = norm_bwd_ctas(a.T, a.D);
    const dim3 g((unsigned)((a.D + 31) / 32), 3);
    if (many_partials(n, 3 * (int64_t)g.x)) norm_bwd_sum_kernel<32><<<g, 1024, 0, s>>>(a, n);
    else norm_bwd_sum_kernel<8><<<g, 256, 0, s>>>(a, n);
    return cudaGetLastError();
}

}  // namespace

int64_t norm_bwd_ctas(int64_t T, int64_t D) {
    // 512 threads a SM, eight columns a thread
    const int64_t most = 152 * (D <= 512 ? 8 : D <= 1024 ? 4 : D <= 2048 ? 2 : 1);
    return T < 1 ? 1 : T < most ? T : most;
}

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t s) {
    if (a.dtype == LIZARD_F32) return fwd<float, float>(a, s);
    return a.res_dtype == LIZARD_F32 ? fwd<__nv_bfloat16, float>(a, s)
                                     : fwd<__nv_bfloat16, __nv_bfloat16>(a, s);
}

cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t s) {
    if (a.dtype == LIZARD_F32) return bwd<float, float>(a, s);
    return a.res_dtype == LIZARD_F32 ? bwd<__nv_bfloat16, float>(a, s)
                                     : bwd<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace lz
