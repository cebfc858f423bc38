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

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// Two fp32 values in a register pair, and the paired instructions on them.  One issue slot does
// two operations; measured, a pair takes 2.1 cycles of a scheduler with up to two operands of its
// own and 3.1 with three, against 1.03 for each single fused multiply-add, so that pairs cost the
// same multiplier time and leave slots for the loads, exponentials and shuffles between them.
typedef uint64_t f2;
__device__ __forceinline__ f2 pack(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack(f2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 exp2_2(f2 v) {
    float a, b;
    unpack(v, a, b);
    return pack(ex2(a), ex2(b));
}
__device__ __forceinline__ float sum2(f2 v) {
    float a, b;
    unpack(v, a, b);
    return a + b;
}

// 1 / x of a value from 1 on, within one ulp (0 from 2^126 on)
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// sigmoid(v), and the derivative of v sigmoid(v) given it.  The fp32 path divides, takes expf and
// never e^|v|, which overflows where the sigmoid is still a number; the bf16 path takes the
// hardware's exponential and reciprocal, whose error (a few 2^-23) is far below bf16's step.
template <bool FAST>
__device__ __forceinline__ float sigm(float v) {
    if constexpr (FAST) return rcp(1.0f + ex2(-kLog2e * v));
    const float e = expf(-fabsf(v));
    return (v >= 0.0f ? 1.0f : e) / (1.0f + e);
}
__device__ __forceinline__ float dsilu(float v, float sg) { return sg * fmaf(v, 1.0f - sg, 1.0f); }

// The same for two values, and the derivative of v sigmoid(v) given the sigmoid.
template <bool FAST>
__device__ __forceinline__ f2 sigm2(f2 v) {
    float x, y;
    if constexpr (FAST) {
        unpack(mul2(v, pack(-kLog2e, -kLog2e)), x, y);
        unpack(add2(pack(ex2(x), ex2(y)), pack(1.0f, 1.0f)), x, y);
        return pack(rcp(x), rcp(y));
    } else {
        unpack(v, x, y);
        return pack(sigm<false>(x), sigm<false>(y));
    }
}
__device__ __forceinline__ f2 dsilu2(f2 v, f2 sg) {
    const f2 one = pack(1.0f, 1.0f), less = fma2(sg, pack(-1.0f, -1.0f), one);
    return fma2(mul2(v, sg), less, sg);
}
// V consecutive elements as V / 2 pairs, for V of 2 or more.
template <typename T, int V>
__device__ __forceinline__ void get2(const Pack<T, V>& p, f2* f) {
    float v[V];
    p.get(v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) f[i] = pack(v[2 * i], v[2 * i + 1]);
}

template <typename T>
constexpr bool is_fast() { return sizeof(T) == 2; }

// A thread's own copy of V elements from global to shared memory, asynchronous where its size
// allows it (4, 8, 16 or 32 bytes): rows ahead wait in shared memory and not in registers, and
// since each thread reads back only what it copied, waiting for its own copies is enough.
template <typename T, int V>
__device__ __forceinline__ void copy_async(T* to, const T* from) {
    constexpr int bytes = sizeof(T) * V;
    const uint32_t s = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (bytes == 32) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(from) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s + 16), "l"((const char*)from + 16) : "memory");
    } else if constexpr (bytes == 16) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(from) : "memory");
    } else if constexpr (bytes >= 4) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(s), "l"(from), "n"(bytes) : "memory");
    } else {
        *to = *from;
    }
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most LEFT of the thread's committed groups are under way.
template <int LEFT>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// Sums of 32 columns' n partial values by a CTA of 32 KT threads, always in the same order: thread
// (k, column) adds partials k, k + KT, ..., then a column's KT sums are added across a warp's lanes.
// value(p, column) is a partial, put(column, sum) takes a column's sum; columns count from the
// CTA's first, `columns` of them.
template <int KT, typename F, typename G>
__device__ __forceinline__ void sum_columns(int64_t n, int columns, F&& value, G&& put) {
    __shared__ float part[KT][33];
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    float s = 0.0f;
    if (lane < columns) {
#pragma unroll 8
        for (int64_t p = k; p < n; p += KT) s += value(p, lane);
    }
    part[k][lane] = s;
    __syncthreads();
    for (int c = k; c < 32; c += KT) {
        s = lane < KT ? part[lane][c] : 0.0f;
#pragma unroll
        for (int o = KT / 2; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        if (lane == 0 && c < columns) put(c, s);
    }
}
// Whether 32 threads a column pay, not eight: where a column's partials are a long chain of loads
// and the columns leave SMs idle (347 partials of 198 columns: 3.8 against 9.8 us; 152 of 12288:
// 6.1 against 4.2).
inline bool many_partials(int64_t n, int64_t ctas) { return (n >= 64 && ctas <= 152) || n >= 2048; }

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
    size_t group_bytes;  // set by the launch: shared memory of the group sums
};
int64_t norm_bwd_ctas(int64_t T, int64_t D);
cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t s);

}  // namespace lz
