// What the scan's forward, backward and step kernels share.
#pragma once

#include "selective.h"

namespace lz {
namespace scan {

constexpr int NT = 128;      // threads a CTA
constexpr int NS = 4;        // states a thread holds for each of its channels
constexpr int CK = 16;       // tokens between the states kept for the backward
constexpr int SEG = 64;      // segments are whole multiples of this many tokens

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// log(1 + e^x) = max(x, 0) + log1p(u), u = e^-|x| <= 1, and log1p(u) = 2 atanh(s) with
// s = u / (2 + u) <= 1/3: the odd series to s^13 leaves 2 (1/3)^15 / 15, below 2^-26 of the
// result.  (A logarithm of 1 + u would lose the digits of a small step size.)
__device__ __forceinline__ float softplus_(float x) {
    const float u = ex2(-kLog2e * fabsf(x));
    const float s = __fdividef(u, 2.0f + u), s2 = s * s;
    float p = 1.0f / 13.0f;
    p = fmaf(p, s2, 1.0f / 11.0f);
    p = fmaf(p, s2, 1.0f / 9.0f);
    p = fmaf(p, s2, 1.0f / 7.0f);
    p = fmaf(p, s2, 1.0f / 5.0f);
    p = fmaf(p, s2, 1.0f / 3.0f);
    p = fmaf(p, s2, 1.0f);
    return fmaf(2.0f * s, p, fmaxf(x, 0.0f));
}

// Eight storage elements in registers.
template <typename T>
struct Raw {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void get(float* f) const { Vec<8>::ld(reinterpret_cast<const T*>(v), f); }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = make_uint4(0, 0, 0, 0);
    }
    // n (0..8) elements at p, zeros after them; vec: p is 16-byte aligned and n is 0 or 8
    __device__ __forceinline__ void load(const T* p, int n, bool vec) {
        if (vec) {
            if (n > 0) {
#pragma unroll
                for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
            } else {
                zero();
            }
            return;
        }
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < n) e[i] = p[i];
            else lz::st(&e[i], 0.0f);
        }
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                v[i] = make_uint4(__float_as_uint(e[4 * i]), __float_as_uint(e[4 * i + 1]),
                                  __float_as_uint(e[4 * i + 2]), __float_as_uint(e[4 * i + 3]));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (uint32_t)__bfloat16_as_ushort(e[2 * i]) |
                       (uint32_t)__bfloat16_as_ushort(e[2 * i + 1]) << 16;
            v[0] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
};

template <typename T>
__device__ __forceinline__ void store8(T* p, const float* f, int n, bool vec) {
    if (vec) {
        if (n > 0) Vec<8>::st(p, f);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) lz::st(p + i, f[i]);
}

// Up to four consecutive fp32 values (n of them; the rest read as zero).
__device__ __forceinline__ void load4(const float* p, int n, bool vec, float* f) {
    if (vec && n == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < n ? p[i] : 0.0f;
}
__device__ __forceinline__ void store4(float* p, int n, bool vec, const float* f) {
    if (vec && n == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) p[i] = f[i];
}

// Lanes that share a channel: the power of two that holds N states, four a lane.
inline int lanes_for(int64_t N) {
    int l = 1;
    while (l * NS < N) l *= 2;
    return l;
}

// How a call is cut into CTAs: blocks of channels (none across two groups) x segments of the
// time axis x rows of the batch.
struct Cut {
    int64_t cbg;       // channel blocks of a group
    int64_t cblocks;   // of all groups
    int64_t segs, seg_len;
};

// Where a CTA is.
template <int CH>
struct Where {
    int64_t grp, cb, seg, b;
    int64_t c0, clim;  // first channel, end of the group's channels
    __device__ __forceinline__ Where(const ScanArgs& a, const Cut& k) {
        cb = blockIdx.x % k.cblocks;
        const int64_t r = blockIdx.x / k.cblocks;
        seg = r % k.segs;
        b = r / k.segs;
        grp = cb / k.cbg;
        const int64_t cg = a.C / a.G;
        c0 = grp * cg + cb % k.cbg * CH;
        clim = (grp + 1) * cg;
    }
};

}  // namespace scan
}  // namespace lz
