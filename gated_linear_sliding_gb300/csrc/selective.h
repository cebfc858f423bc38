// Host-side interface between the entry points of the selective state space block
// (lizard_conv_*, lizard_scan_*, lizard_block_norm_*) and their kernels, and the device helpers
// these kernels share.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"
#include "lizard.h"

namespace lz {

// Sequences of a batch: B dense rows of L tokens, or (cu != null) nseq packed ones in a single
// row of L tokens.  Tokens are counted within a row of the batch.
struct Seqs {
    int64_t L, nseq;
    const int64_t* cu;  // device, [nseq + 1]
};

// The sequence that holds a token: its index (of the per-sequence states) and token range.
struct SeqAt {
    int64_t seq, begin, end;
};

// The threads of a call's first CTA look the packed offsets over, once a call.
__device__ __forceinline__ void check_offsets(const Seqs& s, WsHeader* h) {
    if (s.cu == nullptr || h == nullptr || blockIdx.x != 0) return;
    bool bad = threadIdx.x == 0 && (s.cu[0] != 0 || s.cu[s.nseq] != s.L);
    for (int64_t i = threadIdx.x; i < s.nseq; i += blockDim.x) bad |= s.cu[i + 1] < s.cu[i];
    if (bad) report(h, LIZARD_ERR_INVALID_ARG, 32);
}

// Sequence of token t (0 <= t < L) of batch row b.  Whatever the offsets hold, the index is one
// of the batch's and the range lies in the row around t.
__device__ __forceinline__ SeqAt seq_at(const Seqs& s, int64_t b, int64_t t) {
    SeqAt a;
    if (s.cu == nullptr) {
        a.seq = b;
        a.begin = 0;
        a.end = s.L;
        return a;
    }
    int64_t lo = 0, hi = s.nseq;  // the last sequence that begins at or before t
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (s.cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    a.seq = lo;
    a.begin = s.cu[lo];
    a.end = s.cu[lo + 1];
    if (a.begin < 0 || a.begin > t || a.end <= t || a.end > s.L) {
        a.begin = t;
        a.end = s.L;
    }
    return a;
}

// Tokens of sequence i, 0 where the offsets are inconsistent; *end is its end, in [0, L].
__device__ __forceinline__ int64_t seq_tokens(const Seqs& s, int64_t i, int64_t* end) {
    if (s.cu == nullptr) {
        *end = s.L;
        return s.L;
    }
    const int64_t a = s.cu[i], e = s.cu[i + 1];
    const bool ok = a >= 0 && e >= a && e <= s.L;
    *end = ok ? e : 0;
    return ok ? e - a : 0;
}

// Eight consecutive elements as fp32 (16-byte aligned), or one element.
template <int V>
struct Vec;
template <>
struct Vec<8> {
    static __device__ __forceinline__ void ld(const __nv_bfloat16* p, float* f) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void ld(const float* p, float* f) {
        const float4 a = reinterpret_cast<const float4*>(p)[0];
        const float4 b = reinterpret_cast<const float4*>(p)[1];
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    static __device__ __forceinline__ void st(__nv_bfloat16* p, const float* f) {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
    }
    static __device__ __forceinline__ void st(float* p, const float* f) {
        reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};
template <>
struct Vec<4> {
    static __device__ __forceinline__ void ld(const __nv_bfloat16* p, float* f) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        f[0] = __uint_as_float(u.x << 16), f[1] = __uint_as_float(u.x & 0xffff0000u);
        f[2] = __uint_as_float(u.y << 16), f[3] = __uint_as_float(u.y & 0xffff0000u);
    }
    static __device__ __forceinline__ void ld(const float* p, float* f) {
        const float4 a = *reinterpret_cast<const float4*>(p);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    }
    static __device__ __forceinline__ void st(__nv_bfloat16* p, const float* f) {
        __nv_bfloat162 h[2] = {__floats2bfloat162_rn(f[0], f[1]), __floats2bfloat162_rn(f[2], f[3])};
        *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(h);
    }
    static __device__ __forceinline__ void st(float* p, const float* f) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
};
template <>
struct Vec<1> {
    template <typename T>
    static __device__ __forceinline__ void ld(const T* p, float* f) { f[0] = lz::ld(p); }
    template <typename T>
    static __device__ __forceinline__ void st(T* p, const float* f) { lz::st(p, f[0]); }
};

// Vec<V>'s elements as they lie in memory.
template <typename T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Pack {
    T e[V];
    __device__ __forceinline__ void get(float* f) const { Vec<V>::ld(e, f); }
};

// sigmoid(v), and the derivative of v sigmoid(v) given it.  The fp32 path divides, takes expf and
// never e^|v|, which overflows where the sigmoid is still a number; the bf16 path takes the fast
// exponential and division, whose error (a few 2^-23) is far below bf16's step.
template <bool FAST>
__device__ __forceinline__ float sigm(float v) {
    if constexpr (FAST) return __fdividef(1.0f, 1.0f + __expf(-v));
    const float e = expf(-fabsf(v));
    return (v >= 0.0f ? 1.0f : e) / (1.0f + e);
}
__device__ __forceinline__ float dsilu(float v, float sg) { return sg * fmaf(v, 1.0f - sg, 1.0f); }

template <typename T>
constexpr bool is_fast() { return sizeof(T) == 2; }

struct ConvArgs {
    int64_t B, C;
    Seqs seqs;
    int64_t nstate;  // per-sequence states: B or nseq
    int K, act, dtype;
    int64_t ldx, ldy, lddx;
    const void* x;
    const float *w, *bias;
    const void* state_in;
    void *y, *state_out;
    const void *dy, *dstate_out;
    void *dx, *dstate_in;
    float *dw, *dbias;
    void* state;  // step
    int64_t nslots;
    const int64_t* slots;
    WsHeader* header;
    float* partial;  // backward: [runs, K + 1, C]
};
cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t s);
cudaError_t launch_conv_step(const ConvArgs& a, cudaStream_t s);
int64_t conv_bwd_runs(int64_t B, int64_t L, int64_t C);
cudaError_t launch_conv_bwd(const ConvArgs& a, cudaStream_t s);

struct ScanArgs {
    int64_t B, C, N, G;
    Seqs seqs;
    int64_t nstate;
    int dtype, softplus;
    int64_t ldx, lddt, ldz, ldb, ldc, ldy, lddx, ldddt, lddz, lddb, lddc;
    const void *x, *dt, *Bm, *Cm, *z;
    const float *A, *D, *dt_bias, *h0;
    void* y;
    float* h_out;
    float* states;
    // backward
    const void* dy;
    const float* dh_out;
    void *dx, *ddt, *dz, *dBm, *dCm;
    float *dA, *dD, *ddt_bias, *dh0;
    // step
    float* state;
    int64_t nslots;
    const int64_t* slots;
    WsHeader* header;
    float* ws;  // after the header
};
size_t scan_fwd_ws_floats(const ScanArgs& a);
size_t scan_bwd_ws_floats(const ScanArgs& a);
cudaError_t launch_scan_fwd(const ScanArgs& a, cudaStream_t s);
cudaError_t launch_scan_bwd(const ScanArgs& a, cudaStream_t s);
cudaError_t launch_scan_step(const ScanArgs& a, cudaStream_t s);

struct NormArgs {
    int64_t T, D, groups;
    int64_t ldo, ldg, ldr, ldro, ldn, lddo, lddg, lddr;
    float eps_post, eps_pre;
    int dtype, res_dtype, act, gate_first;
    const void *o, *gate, *r;
    const float *w_post, *scale, *w_pre;
    void *r_out, *n_out;
    const void *dr_out, *dn_out;
    void *d_o, *dgate, *dr;
    float *dw_post, *dscale, *dw_pre;
    float* partial;  // backward: [CTAs, 3, D]
};
int64_t norm_bwd_ctas(int64_t T, int64_t D);
cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t s);

// out[i] = sum over p < n of in[p * stride + i], i < count, in the order of p.
cudaError_t launch_sum_partials(const float* in, int64_t n, int64_t stride, float* out,
                                int64_t count, cudaStream_t s);

}  // namespace lz
