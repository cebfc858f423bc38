// Norm after a block, gate, residual scale and add, and the norm before the next block
// (lizard_block_norm_*), one pass over the row.
//
//   u = o [act(gate)],  n = w_post u / rms_group(u),  n [act(gate)],  rr = r + scale n,
//   r_out = rr,  n_out = w_pre rr / rms(rr)
//
// Bound by HBM: each row is read once into registers (V neighbouring columns a piece, NV pieces a
// thread), the sums of squares are reduced inside the CTA, and both outputs leave from registers.
#include <type_traits>

#include "selective.h"

namespace lz {
namespace {

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
#pragma unroll
        for (int k = 0; k < NVAL; ++k) {
            v[k] = lane < TPR / 32 ? red[k][lane] : 0.0f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(~0u, v[k], o);
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

__device__ __forceinline__ float act_of(int act, float g, float sg) { return act == LIZARD_ACT_SILU ? g * sg : sg; }
__device__ __forceinline__ float dact_of(int act, float g, float sg) {
    return act == LIZARD_ACT_SILU ? dsilu(g, sg) : sg * (1.0f - sg);
}

// TPR threads a row; 32: four rows a CTA of 128, else one row a CTA.
template <typename T, typename R, int V, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_fwd_kernel(const NormArgs a) {
    constexpr int RPC = TPR < 128 ? 128 / TPR : 1;
    constexpr bool FAST = is_fast<T>();
    __shared__ float red[2][1][32];
    extern __shared__ __align__(16) float gsm[];
    const int lr = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPC + threadIdx.x / TPR;
    if (TPR == 32 && row >= a.T) return;  // a whole warp
    const int D = (int)a.D, nvec = D / V, gv = nvec / (int)a.groups;
    const T* o = (const T*)a.o + row * a.ldo;
    const T* gate = (const T*)a.gate + row * a.ldg;
    const R* r = (const R*)a.r + row * a.ldr;
    float n[NV][V], ga[NV][V], rr[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int vi = i * TPR + lr;
        const bool in = vi < nvec;
#pragma unroll
        for (int j = 0; j < V; ++j) n[i][j] = ga[i][j] = rr[i][j] = 0.0f;
        if (in) Vec<V>::ld(o + vi * V, n[i]);
        if (in && a.gate != nullptr) Vec<V>::ld(gate + vi * V, ga[i]);
        if (in && a.r != nullptr) Vec<V>::ld(r + vi * V, rr[i]);
    }
    if (a.gate != nullptr) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                ga[i][j] = act_of(a.act, ga[i][j], sigm<FAST>(ga[i][j]));
                if (a.gate_first) n[i][j] *= ga[i][j];
            }
    }
    if (a.w_post != nullptr) {
        float ss[NV];
        float all[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            ss[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) ss[i] = fmaf(n[i][j], n[i][j], ss[i]);
            all[0] += ss[i];
        }
        if (a.groups == 1) {
            row_sum<TPR, 1>(all, red[0]);
#pragma unroll
            for (int i = 0; i < NV; ++i) ss[i] = all[0];
        } else {
            group_sum<TPR, NV>(ss, nvec, gv, gsm, lr);
        }
        const float inv = 1.0f / (float)(gv * V);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int vi = i * TPR + lr;
            const float rs = rsqrtf(fmaf(ss[i], inv, a.eps_post));
            float w[V];
            if (vi < nvec) Vec<V>::ld(a.w_post + vi * V, w);
#pragma unroll
            for (int j = 0; j < V; ++j) n[i][j] *= rs * w[j];
        }
    }
    float all[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int vi = i * TPR + lr;
        if (vi >= nvec) continue;
        float w[V];
        if (a.scale != nullptr) Vec<V>::ld(a.scale + vi * V, w);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (a.gate != nullptr && !a.gate_first) n[i][j] *= ga[i][j];
            rr[i][j] = a.scale != nullptr ? fmaf(w[j], n[i][j], rr[i][j]) : rr[i][j] + n[i][j];
            all[0] = fmaf(rr[i][j], rr[i][j], all[0]);
        }
        if (a.r_out != nullptr) Vec<V>::st((R*)a.r_out + row * a.ldro + vi * V, rr[i]);
    }
    if (a.n_out == nullptr) return;
    row_sum<TPR, 1>(all, red[1]);
    const float rs = rsqrtf(all[0] / (float)D + a.eps_pre);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int vi = i * TPR + lr;
        if (vi >= nvec) continue;
        float w[V];
        Vec<V>::ld(a.w_pre + vi * V, w);
#pragma unroll
        for (int j = 0; j < V; ++j) rr[i][j] *= rs * w[j];
        Vec<V>::st((T*)a.n_out + row * a.ldn + vi * V, rr[i]);
    }
}

// One CTA walks rows b, b + grid, ..., the next row's values on their way while one is worked on.
// The parameter gradients of a thread's columns are summed in shared memory, in the thread's own
// places, and leave once, as the CTA's partial sums.
template <typename T, typename R, int V, int TPR, int NV>
__global__ void __launch_bounds__(TPR, V * NV <= 4 ? 1024 / TPR : 1)
    norm_bwd_kernel(const NormArgs a) {
    constexpr bool FAST = is_fast<T>();
    // hold the next row where registers allow it: 64 a thread at 1024 threads a SM
    constexpr bool AHEAD = sizeof(T) == 2 && V * NV <= 4;
    __shared__ float red[2][2][32];
    extern __shared__ __align__(16) float gsm[];  // [3][D], then the group sums' space
    const int lr = threadIdx.x;
    const int D = (int)a.D, nvec = D / V, gv = nvec / (int)a.groups;
    float *apost = gsm, *ascale = gsm + D, *apre = gsm + 2 * D, *gspace = gsm + 3 * D;
    for (int i = lr; i < 3 * D; i += TPR) gsm[i] = 0.0f;
    __syncthreads();
    const bool gate = a.gate != nullptr, gfirst = gate && a.gate_first, glast = gate && !a.gate_first;
    const float ginv = 1.0f / (float)(gv * V), dinv = 1.0f / (float)D;
    Pack<T, V> po[NV], pg[NV], pn[NV];
    Pack<R, V> pr[NV], pd[NV];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int vi = i * TPR + lr;
            if (vi >= nvec) continue;
            po[i] = *reinterpret_cast<const Pack<T, V>*>((const T*)a.o + row * a.ldo + vi * V);
            if (gate) pg[i] = *reinterpret_cast<const Pack<T, V>*>((const T*)a.gate + row * a.ldg + vi * V);
            if (a.dr_out != nullptr) pd[i] = *reinterpret_cast<const Pack<R, V>*>((const R*)a.dr_out + row * a.ldro + vi * V);
            if (a.w_pre != nullptr) {
                if (a.r != nullptr) pr[i] = *reinterpret_cast<const Pack<R, V>*>((const R*)a.r + row * a.ldr + vi * V);
                pn[i] = *reinterpret_cast<const Pack<T, V>*>((const T*)a.dn_out + row * a.ldn + vi * V);
            }
        }
    };
    auto add_to = [](float* sum, const float* v) {
        float s[V];
        Vec<V>::ld(sum, s);
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] += v[j];
        Vec<V>::st(sum, s);
    };
    int buf = 0;
    if (AHEAD && (int64_t)blockIdx.x < a.T) fetch(blockIdx.x);
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        if (!AHEAD) fetch(row);
        float u[NV][V], ga[NV][V], gd[NV][V], dr[NV][V], rr[NV][V], dn[NV][V];
        float ss[NV], rs[NV], all[2] = {0.0f, 0.0f};
        // u: the normalised row (the plain one without a norm); a thread's columns past the row
        // stay zero and count nowhere
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = i * TPR + lr < nvec;
#pragma unroll
            for (int j = 0; j < V; ++j) u[i][j] = ga[i][j] = gd[i][j] = dr[i][j] = rr[i][j] = dn[i][j] = 0.0f;
            if (in) {
                po[i].get(u[i]);
                if (gate) pg[i].get(ga[i]);
                if (a.dr_out != nullptr) pd[i].get(dr[i]);
                if (a.w_pre != nullptr) {
                    if (a.r != nullptr) pr[i].get(rr[i]);
                    pn[i].get(dn[i]);
                }
            }
            ss[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (gate) {  // ga: act(gate), gd: its derivative
                    const float g = ga[i][j], sg = sigm<FAST>(g);
                    ga[i][j] = act_of(a.act, g, sg);
                    gd[i][j] = dact_of(a.act, g, sg);
                }
                if (gfirst) {
                    gd[i][j] *= u[i][j];
                    u[i][j] *= ga[i][j];
                }
                ss[i] = fmaf(u[i][j], u[i][j], ss[i]);
            }
            all[0] += ss[i];
            rs[i] = 1.0f;
        }
        if (AHEAD && row + gridDim.x < a.T) fetch(row + gridDim.x);
        if (a.w_post != nullptr) {
            if (a.groups == 1) {
                row_sum<TPR, 1>(all, red[buf]);
                buf ^= 1;
#pragma unroll
                for (int i = 0; i < NV; ++i) ss[i] = all[0];
            } else {
                group_sum<TPR, NV>(ss, nvec, gv, gspace, lr);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                rs[i] = rsqrtf(fmaf(ss[i], ginv, a.eps_post));
#pragma unroll
                for (int j = 0; j < V; ++j) u[i][j] *= rs[i];
            }
        }
        // the gradient of rr
        if (a.w_pre != nullptr) {
            all[0] = all[1] = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int vi = i * TPR + lr;
                if (vi >= nvec) continue;
                float w[V];
                if (a.w_post != nullptr) Vec<V>::ld(a.w_post + vi * V, w);
                float n[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    n[j] = a.w_post != nullptr ? u[i][j] * w[j] : u[i][j];
                    if (glast) n[j] *= ga[i][j];
                }
                if (a.scale != nullptr) {
                    Vec<V>::ld(a.scale + vi * V, w);
#pragma unroll
                    for (int j = 0; j < V; ++j) n[j] *= w[j];
                }
                Vec<V>::ld(a.w_pre + vi * V, w);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    rr[i][j] += n[j];
                    all[0] = fmaf(rr[i][j], rr[i][j], all[0]);
                    all[1] = fmaf(dn[i][j] * w[j], rr[i][j], all[1]);
                }
            }
            row_sum<TPR, 2>(all, red[buf]);
            buf ^= 1;
            const float rp = rsqrtf(fmaf(all[0], dinv, a.eps_pre)), k = all[1] * dinv * rp * rp;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int vi = i * TPR + lr;
                if (vi >= nvec) continue;
                float w[V];
                Vec<V>::ld(a.w_pre + vi * V, w);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    dr[i][j] += rp * (dn[i][j] * w[j] - rr[i][j] * k);
                    dn[i][j] *= rr[i][j] * rp;
                }
                add_to(apre + vi * V, dn[i]);
            }
        }
        float dot[NV];
        all[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int vi = i * TPR + lr;
            dot[i] = 0.0f;
            if (vi >= nvec) continue;
            if (a.dr != nullptr) Vec<V>::st((R*)a.dr + row * a.lddr + vi * V, dr[i]);
            float w[V], t[V];
            if (a.w_post != nullptr) Vec<V>::ld(a.w_post + vi * V, w);
            if (a.scale != nullptr) {
                float sc[V];
                Vec<V>::ld(a.scale + vi * V, sc);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float n = a.w_post != nullptr ? u[i][j] * w[j] : u[i][j];
                    if (glast) n *= ga[i][j];
                    t[j] = dr[i][j] * n;
                    dr[i][j] *= sc[j];
                }
                add_to(ascale + vi * V, t);
            }
            if (glast) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float n = a.w_post != nullptr ? u[i][j] * w[j] : u[i][j];
                    t[j] = dr[i][j] * n * gd[i][j];
                    dr[i][j] *= ga[i][j];
                }
                Vec<V>::st((T*)a.dgate + row * a.lddg + vi * V, t);
            }
            if (a.w_post != nullptr) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    t[j] = dr[i][j] * u[i][j];
                    dr[i][j] *= w[j];
                    dot[i] = fmaf(dr[i][j], u[i][j], dot[i]);
                }
                add_to(apost + vi * V, t);
            }
            all[0] += dot[i];
        }
        if (a.w_post != nullptr) {
            if (a.groups == 1) {
                row_sum<TPR, 1>(all, red[buf]);
                buf ^= 1;
#pragma unroll
                for (int i = 0; i < NV; ++i) dot[i] = all[0];
            } else {
                group_sum<TPR, NV>(dot, nvec, gv, gspace, lr);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int vi = i * TPR + lr;
            if (vi >= nvec) continue;
            float dg[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (a.w_post != nullptr) dr[i][j] = rs[i] * (dr[i][j] - u[i][j] * (dot[i] * ginv));
                if (gfirst) {
                    dg[j] = dr[i][j] * gd[i][j];
                    dr[i][j] *= ga[i][j];
                }
            }
            Vec<V>::st((T*)a.d_o + row * a.lddo + vi * V, dr[i]);
            if (gfirst) Vec<V>::st((T*)a.dgate + row * a.lddg + vi * V, dg);
        }
    }
    float* p = a.partial + (int64_t)blockIdx.x * 3 * D;
    __syncthreads();
    for (int i = lr; i < 3 * D; i += TPR) p[i] = gsm[i];
}

// dw_post, dscale and dw_pre from the CTAs' partial sums [n][3][D], each added in the same order.
__global__ void __launch_bounds__(256) norm_bwd_sum_kernel(const NormArgs a, int64_t n) {
    // 32 columns a CTA, eight threads a column: thread k adds partials k, k + 8, ..., then the
    // eight are added in order
    __shared__ float part[8][33];
    const int col = threadIdx.x & 31, k = threadIdx.x >> 5, m = blockIdx.y;
    float* out = m == 0 ? a.dw_post : m == 1 ? a.dscale : a.dw_pre;
    if (out == nullptr) return;
    const int64_t i = (int64_t)blockIdx.x * 32 + col;
    float s = 0.0f;
    if (i < a.D) {
#pragma unroll 8
        for (int64_t p = k; p < n; p += 8) s += a.partial[(p * 3 + m) * a.D + i];
    }
    part[k][col] = s;
    __syncthreads();
    if (k == 0 && i < a.D) {
#pragma unroll
        for (int j = 1; j < 8; ++j) s += part[j][col];
        out[i] = s;
    }
}

template <typename K>
cudaError_t group_smem(K kernel, size_t bytes) {
    if (bytes <= 40 * 1024) return cudaSuccess;  // with the static part below the default 48 KB
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// Shared memory of the group sums that neighbouring lanes cannot do.
size_t group_bytes(const NormArgs& a, int V) {
    const int64_t nvec = a.D / V, gv = nvec / a.groups;
    if (a.groups == 1 || a.w_post == nullptr || (gv <= 32 && (gv & (gv - 1)) == 0)) return 0;
    return sizeof(float) * (size_t)(nvec + a.groups);
}

template <typename T, typename R, int V, int TPR, int NV>
cudaError_t fwd_go(const NormArgs& a, cudaStream_t s) {
    constexpr int RPC = TPR < 128 ? 128 / TPR : 1;
    const size_t sm = group_bytes(a, V);
    const cudaError_t e = group_smem(norm_fwd_kernel<T, R, V, TPR, NV>, sm);
    if (e != cudaSuccess) return e;
    norm_fwd_kernel<T, R, V, TPR, NV><<<(unsigned)((a.T + RPC - 1) / RPC), TPR * RPC, sm, s>>>(a);
    return cudaGetLastError();
}

template <typename T, typename R, int V, int TPR, int NV>
cudaError_t bwd_go(const NormArgs& a, cudaStream_t s) {
    const size_t sm = sizeof(float) * 3 * (size_t)a.D + group_bytes(a, V);
    // the odd-width path at its widest, with both the sums and one value a column
    const cudaError_t e = group_smem(norm_bwd_kernel<T, R, V, TPR, NV>, sm);
    if (e != cudaSuccess) return e;
    norm_bwd_kernel<T, R, V, TPR, NV><<<(unsigned)norm_bwd_ctas(a.T, a.D), TPR, sm, s>>>(a);
    return cudaGetLastError();
}

// Eight columns a piece where the rows and groups allow it, else one.
template <typename T, typename R>
cudaError_t fwd(const NormArgs& a, cudaStream_t s) {
    const bool v8 = a.D % 8 == 0 && (a.D / a.groups) % 8 == 0 && a.ldo % 8 == 0 && a.ldg % 8 == 0 &&
                    a.ldr % 8 == 0 && a.ldro % 8 == 0 && a.ldn % 8 == 0;
    if (v8) {
        if (a.D <= 256 && a.groups == 1) return fwd_go<T, R, 8, 32, 1>(a, s);
        if (a.D <= 1024) return fwd_go<T, R, 8, 128, 1>(a, s);
        if (a.D <= 2048) return fwd_go<T, R, 8, 256, 1>(a, s);
        if (a.D <= 4096) return fwd_go<T, R, 8, 256, 2>(a, s);
        if (a.D <= 8192) return fwd_go<T, R, 8, 512, 2>(a, s);
        return fwd_go<T, R, 8, 1024, 2>(a, s);
    }
    if (a.D <= 1024) return fwd_go<T, R, 1, 256, 4>(a, s);
    if (a.D <= 8192) return fwd_go<T, R, 1, 1024, 8>(a, s);
    return fwd_go<T, R, 1, 1024, 16>(a, s);
}

template <typename T, typename R>
cudaError_t bwd(const NormArgs& a, cudaStream_t s) {
    const bool v4 = a.D % 4 == 0 && (a.D / a.groups) % 4 == 0 && a.ldo % 4 == 0 && a.ldg % 4 == 0 &&
                    a.ldr % 4 == 0 && a.ldro % 4 == 0 && a.ldn % 4 == 0 && a.lddo % 4 == 0 &&
                    a.lddg % 4 == 0 && a.lddr % 4 == 0;
    cudaError_t e;
    if (v4) {
        if (a.D <= 512) e = bwd_go<T, R, 4, 128, 1>(a, s);
        else if (a.D <= 1024) e = bwd_go<T, R, 4, 256, 1>(a, s);
        else if (a.D <= 2048) e = bwd_go<T, R, 4, 512, 1>(a, s);
        else if (a.D <= 4096) e = bwd_go<T, R, 4, 1024, 1>(a, s);
        else if (a.D <= 8192) e = bwd_go<T, R, 4, 1024, 2>(a, s);
        else e = bwd_go<T, R, 4, 1024, 4>(a, s);
    } else {
        if (a.D <= 1024) e = bwd_go<T, R, 1, 256, 4>(a, s);
        else if (a.D <= 8192) e = bwd_go<T, R, 1, 1024, 8>(a, s);
        else e = bwd_go<T, R, 1, 1024, 16>(a, s);
    }
    if (e != cudaSuccess) return e;
    norm_bwd_sum_kernel<<<dim3((unsigned)((a.D + 31) / 32), 3), 256, 0, s>>>(a, norm_bwd_ctas(a.T, a.D));
    return cudaGetLastError();
}

}  // namespace

int64_t norm_bwd_ctas(int64_t T, int64_t D) {
    // 1024 threads a SM, as far as the widths' CTAs go
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
