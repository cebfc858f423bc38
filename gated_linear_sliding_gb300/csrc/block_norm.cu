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

// Sum over a CTA's (TPR > 32) or a warp's threads, the same value in each of them.
template <int TPR, int NVAL>
__device__ __forceinline__ void row_sum(float* v, float (*red)[32]) {
#pragma unroll
    for (int k = 0; k < NVAL; ++k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(~0u, v[k], o);
    if constexpr (TPR > 32) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        __syncthreads();  // the last sum's readers are done
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

template <bool FAST>
__device__ __forceinline__ float act_of(int act, float g, float sg) { return act == LIZARD_ACT_SILU ? g * sg : sg; }
__device__ __forceinline__ float dact_of(int act, float g, float sg) {
    return act == LIZARD_ACT_SILU ? dsilu(g, sg) : sg * (1.0f - sg);
}

// TPR threads a row; 32: four rows a CTA of 128, else one row a CTA.
template <typename T, typename R, int V, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_fwd_kernel(const NormArgs a) {
    constexpr int RPC = TPR < 128 ? 128 / TPR : 1;
    constexpr bool FAST = is_fast<T>();
    __shared__ float red[2][32];
    extern __shared__ float gsm[];
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
                ga[i][j] = act_of<FAST>(a.act, ga[i][j], sigm<FAST>(ga[i][j]));
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
            row_sum<TPR, 1>(all, red);
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
    row_sum<TPR, 1>(all, red);
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

// One CTA walks rows b, b + grid, ...; the parameter gradients of its columns stay in registers
// and leave once, as the CTA's partial sums.
template <typename T, typename R, int V, int TPR, int NV>
__global__ void __launch_bounds__(TPR, TPR == 512 ? 2 : 1) norm_bwd_kernel(const NormArgs a) {
    constexpr bool FAST = is_fast<T>();
    __shared__ float red[2][32];
    extern __shared__ float gsm[];
    const int lr = threadIdx.x;
    const int D = (int)a.D, nvec = D / V, gv = nvec / (int)a.groups;
    float apost[NV][V], ascale[NV][V], apre[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) apost[i][j] = ascale[i][j] = apre[i][j] = 0.0f;
    const float ginv = 1.0f / (float)(gv * V), dinv = 1.0f / (float)D;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        float u[NV][V], ga[NV][V], dr[NV][V];
        float ss[NV], rs[NV], all[2] = {0.0f, 0.0f};
        // u: the normalised row (the plain one without a norm)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int vi = i * TPR + lr;
            const bool in = vi < nvec;
#pragma unroll
            for (int j = 0; j < V; ++j) u[i][j] = ga[i][j] = dr[i][j] = 0.0f;
            if (in) Vec<V>::ld((const T*)a.o + row * a.ldo + vi * V, u[i]);
            if (in && a.gate != nullptr) Vec<V>::ld((const T*)a.gate + row * a.ldg + vi * V, ga[i]);
            if (in && a.dr_out != nullptr) Vec<V>::ld((const R*)a.dr_out + row * a.ldro + vi * V, dr[i]);
            ss[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (a.gate != nullptr && a.gate_first) u[i][j] *= act_of<FAST>(a.act, ga[i][j], sigm<FAST>(ga[i][j]));
                ss[i] = fmaf(u[i][j], u[i][j], ss[i]);
            }
            all[0] += ss[i];
            rs[i] = 1.0f;
        }
        if (a.w_post != nullptr) {
            if (a.groups == 1) {
                row_sum<TPR, 1>(all, red);
#pragma unroll
                for (int i = 0; i < NV; ++i) ss[i] = all[0];
            } else {
                group_sum<TPR, NV>(ss, nvec, gv, gsm, lr);
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
            float rr[NV][V], dn[NV][V];
            all[0] = all[1] = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int vi = i * TPR + lr;
                if (vi >= nvec) continue;
                float wp[V], sc[V], w[V];
                if (a.r != nullptr) Vec<V>::ld((const R*)a.r + row * a.ldr + vi * V, rr[i]);
                Vec<V>::ld((const T*)a.dn_out + row * a.ldn + vi * V, dn[i]);
                if (a.w_post != nullptr) Vec<V>::ld(a.w_post + vi * V, wp);
                if (a.scale != nullptr) Vec<V>::ld(a.scale + vi * V, sc);
                Vec<V>::ld(a.w_pre + vi * V, w);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float n = u[i][j];
                    if (a.w_post != nullptr) n *= wp[j];
                    if (a.gate != nullptr && !a.gate_first) n *= act_of<FAST>(a.act, ga[i][j], sigm<FAST>(ga[i][j]));
                    if (a.scale != nullptr) n *= sc[j];
                    rr[i][j] = a.r != nullptr ? rr[i][j] + n : n;
                    all[0] = fmaf(rr[i][j], rr[i][j], all[0]);
                    all[1] = fmaf(dn[i][j] * w[j], rr[i][j], all[1]);
                }
            }
            row_sum<TPR, 2>(all, red);
            const float rp = rsqrtf(fmaf(all[0], dinv, a.eps_pre)), k = all[1] * dinv * rp * rp;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int vi = i * TPR + lr;
                if (vi >= nvec) continue;
                float w[V];
                Vec<V>::ld(a.w_pre + vi * V, w);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    apre[i][j] = fmaf(dn[i][j], rr[i][j] * rp, apre[i][j]);
                    dr[i][j] += rp * (dn[i][j] * w[j] - rr[i][j] * k);
                }
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
            float wp[V], sc[V], dg[V];
            if (a.w_post != nullptr) Vec<V>::ld(a.w_post + vi * V, wp);
            if (a.scale != nullptr) Vec<V>::ld(a.scale + vi * V, sc);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float n = a.w_post != nullptr ? u[i][j] * wp[j] : u[i][j];  // before a later gate
                float act = 1.0f, dact = 0.0f;
                if (a.gate != nullptr && !a.gate_first) {
                    const float sg = sigm<FAST>(ga[i][j]);
                    act = act_of<FAST>(a.act, ga[i][j], sg);
                    dact = dact_of(a.act, ga[i][j], sg);
                }
                ascale[i][j] = fmaf(dr[i][j], n * act, ascale[i][j]);
                float dm = a.scale != nullptr ? dr[i][j] * sc[j] : dr[i][j];
                dg[j] = dm * n * dact;
                dm *= act;
                apost[i][j] = fmaf(dm, u[i][j], apost[i][j]);
                if (a.w_post != nullptr) dm *= wp[j];
                dr[i][j] = dm;
                dot[i] = fmaf(dm, u[i][j], dot[i]);
            }
            if (a.gate != nullptr && !a.gate_first) Vec<V>::st((T*)a.dgate + row * a.lddg + vi * V, dg);
            all[0] += dot[i];
        }
        if (a.w_post != nullptr) {
            if (a.groups == 1) {
                row_sum<TPR, 1>(all, red);
#pragma unroll
                for (int i = 0; i < NV; ++i) dot[i] = all[0];
            } else {
                group_sum<TPR, NV>(dot, nvec, gv, gsm, lr);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int vi = i * TPR + lr;
            if (vi >= nvec) continue;
            float dg[V], ov[V];
            if (a.gate != nullptr && a.gate_first) Vec<V>::ld((const T*)a.o + row * a.ldo + vi * V, ov);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (a.w_post != nullptr) dr[i][j] = rs[i] * (dr[i][j] - u[i][j] * (dot[i] * ginv));
                if (a.gate != nullptr && a.gate_first) {
                    const float sg = sigm<FAST>(ga[i][j]);
                    dg[j] = dr[i][j] * ov[j] * dact_of(a.act, ga[i][j], sg);
                    dr[i][j] *= act_of<FAST>(a.act, ga[i][j], sg);
                }
            }
            Vec<V>::st((T*)a.d_o + row * a.lddo + vi * V, dr[i]);
            if (a.gate != nullptr && a.gate_first) Vec<V>::st((T*)a.dgate + row * a.lddg + vi * V, dg);
        }
    }
    float* p = a.partial + (int64_t)blockIdx.x * 3 * D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int vi = i * TPR + lr;
        if (vi >= nvec) continue;
        Vec<V>::st(p + vi * V, apost[i]);
        Vec<V>::st(p + D + vi * V, ascale[i]);
        Vec<V>::st(p + 2 * D + vi * V, apre[i]);
    }
}

constexpr int kBwdCtas = 304;  // two a SM

template <typename K>
cudaError_t group_smem(K kernel, size_t bytes) {
    if (bytes <= 48 * 1024) return cudaSuccess;
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
    const size_t sm = group_bytes(a, V);
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
    const bool v8 = a.D % 8 == 0 && (a.D / a.groups) % 8 == 0 && a.ldo % 8 == 0 && a.ldg % 8 == 0 &&
                    a.ldr % 8 == 0 && a.ldro % 8 == 0 && a.ldn % 8 == 0 && a.lddo % 8 == 0 &&
                    a.lddg % 8 == 0 && a.lddr % 8 == 0;
    cudaError_t e;
    if (v8) {
        if (a.D <= 1024) e = bwd_go<T, R, 8, 128, 1>(a, s);
        else if (a.D <= 2048) e = bwd_go<T, R, 8, 256, 1>(a, s);
        else if (a.D <= 4096) e = bwd_go<T, R, 8, 512, 1>(a, s);
        else if (a.D <= 8192) e = bwd_go<T, R, 8, 1024, 1>(a, s);
        else e = bwd_go<T, R, 8, 1024, 2>(a, s);
    } else {
        if (a.D <= 1024) e = bwd_go<T, R, 1, 256, 4>(a, s);
        else if (a.D <= 8192) e = bwd_go<T, R, 1, 1024, 8>(a, s);
        else e = bwd_go<T, R, 1, 1024, 16>(a, s);
    }
    const int64_t n = norm_bwd_ctas(a.T, a.D);
    if (e == cudaSuccess && a.dw_post != nullptr)
        e = launch_sum_partials(a.partial, n, 3 * a.D, a.dw_post, a.D, s);
    if (e == cudaSuccess && a.dscale != nullptr)
        e = launch_sum_partials(a.partial + a.D, n, 3 * a.D, a.dscale, a.D, s);
    if (e == cudaSuccess && a.dw_pre != nullptr)
        e = launch_sum_partials(a.partial + 2 * a.D, n, 3 * a.D, a.dw_pre, a.D, s);
    return e;
}

}  // namespace

int64_t norm_bwd_ctas(int64_t T, int64_t D) {
    const int64_t most = D <= 1024 ? 8 * 152 : D <= 2048 ? 4 * 152 : kBwdCtas;
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
