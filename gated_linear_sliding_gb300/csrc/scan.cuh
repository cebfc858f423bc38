// What the scan's forward, backward and step kernels share.
#pragma once

#include "selective.h"

namespace lz {
namespace scan {

constexpr int NT = 128;      // threads a CTA
constexpr int CK = 16;       // tokens between the states kept for the backward
constexpr int SEG = 64;      // segments are whole multiples of this many tokens

// The decays exp(d A) of two states, A2 = A log2(e).  ex2.approx errs downwards, and a state that
// remembers n tokens multiplies n decays.  The exponent is moved up by 2e-8 (1.4e-8 of the result) on
// the product's own instruction.  Mean error in 1e-8 of the result, by the exponent of two's size,
// without and with it (2^24 arguments a decade):
//   1e-6 -1.1 +0.3 | 1e-5 -0.8 +0.6 | 1e-4 -0.6 +0.8 | 1e-3 -1.2 +0.2 | 1e-2 -2.2 -0.8 | 0.1 -2.1 -1.0
// so from 1e-4 to 1e-3 it errs upwards by a little more than the exponential alone errs downwards, and
// elsewhere less.  With step sizes from 0.001 to 0.1 and rates from 1 to 16 the error of dA against
// 64 bits falls from 1.9e-6 to 0.9e-6 on 8 x 2048 tokens, of the last states from 4.5e-7 to 2.5e-7 on
// 8192.  Prompts, training and single tokens take the same decays, so that a state drifts alike
// whichever of them moves it.
constexpr float kDecayShift = 2e-8f;
__device__ __forceinline__ f2 decay2(f2 d, f2 A2) { return exp2_2(fma2(d, A2, pack(kDecayShift, kDecayShift))); }

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// The smaller of the two, NaN where one is.
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// log(1 + e^x) = max(x, 0) + log1p(u), u = e^-|x| <= 1, and log1p(u) = 2 atanh(s) with
// s = u / (2 + u) <= 1/3: s times a polynomial in s^2, five coefficients fitted for the least
// relative error on [0, 1/9], which rounded to fp32 is 2^-26.9.  (A logarithm of 1 + u would lose the digits of a small step size.)  For a small step size
// the result is u itself, whose exponent |x| log2(e) would bring |x| 2^-24 of it as the product's
// rounding and as much as that of the constant: what the product leaves, by the multiply-add, and
// the constant's second part are put back to first order.  Two at a time.
__device__ __forceinline__ f2 softplus2(f2 v) {
    float x, y;
    unpack(v, x, y);
    // from 128 on, infinity included, e^-|x| is 0
    const f2 a = pack(min_nan(fabsf(x), 128.0f), min_nan(fabsf(y), 128.0f));
    const f2 p2 = mul2(a, pack(-kLog2e, -kLog2e));  // -|x| log2(e) = p2 - left
    const float low = 1.9259629911e-8f;             // log2(e) - kLog2e
    const f2 left = fma2(a, pack(low, low), fma2(a, pack(kLog2e, kLog2e), p2));
    f2 u = exp2_2(p2);
    u = fma2(mul2(u, left), pack(-0.69314718055994531f, -0.69314718055994531f), u);
    float m, n;
    unpack(add2(u, pack(2.0f, 2.0f)), m, n);
    const f2 s = mul2(u, pack(rcp(m), rcp(n))), s2 = mul2(s, s);
    const float c[5] = {0.281783342f, 0.279606014f, 0.400249094f, 0.66666317f, 2.0f};
    f2 p = pack(c[0], c[0]);
#pragma unroll
    for (int i = 1; i < 5; ++i) p = fma2(p, s2, pack(c[i], c[i]));
    return fma2(s, p, pack(fmaxf(x, 0.0f), fmaxf(y, 0.0f)));
}

__device__ __forceinline__ float softplus_(float v) {
    float x, y;
    unpack(softplus2(pack(v, 0.0f)), x, y);
    return x;
}

// Eight storage elements in registers.
template <typename T>
struct Raw {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void get(float* f) const { Vec<8>::ld(reinterpret_cast<const T*>(v), f); }
    __device__ __forceinline__ void get(f2* f) const {
        float v[8];
        get(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = pack(v[2 * i], v[2 * i + 1]);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = make_uint4(0, 0, 0, 0);
    }
    // n (0..8) elements at p, zeros after them; vec: p is 16-byte aligned
    __device__ __forceinline__ void load(const T* p, int n, bool vec) {
        if (vec && n == 8) {
#pragma unroll
            for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
            return;
        }
        if (n <= 0) {
            zero();
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
__device__ __forceinline__ void store8(T* p, const f2* v, int n, bool vec) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack(v[i], f[2 * i], f[2 * i + 1]);
    if (vec && n == 8) {
        Vec<8>::st(p, f);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) lz::st(p + i, f[i]);
}

// NS consecutive fp32 values, n of them in the array (the rest read as zero); vec: p is aligned
// to min(NS, 4) values.
template <int NS>
__device__ __forceinline__ void load_n(const float* p, int n, bool vec, float* f) {
    if (vec && n == NS) {
        if constexpr (NS % 4 == 0) {
#pragma unroll
            for (int i = 0; i < NS / 4; ++i) {
                const float4 v = reinterpret_cast<const float4*>(p)[i];
                f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
            }
        } else {
            const float2 v = *reinterpret_cast<const float2*>(p);
            f[0] = v.x, f[1] = v.y;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) f[i] = i < n ? p[i] : 0.0f;
}
template <int NS>
__device__ __forceinline__ void store_n(float* p, int n, bool vec, const float* f) {
    if (vec && n == NS) {
        if constexpr (NS % 4 == 0) {
#pragma unroll
            for (int i = 0; i < NS / 4; ++i)
                reinterpret_cast<float4*>(p)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        } else {
            *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < NS; ++i)
        if (i < n) p[i] = f[i];
}
// The same as pairs.
template <int NS>
__device__ __forceinline__ void load_pairs(const float* p, int n, bool vec, f2* f) {
    float v[NS];
    load_n<NS>(p, n, vec, v);
#pragma unroll
    for (int i = 0; i < NS / 2; ++i) f[i] = pack(v[2 * i], v[2 * i + 1]);
}
template <int NS>
__device__ __forceinline__ void store_pairs(float* p, int n, bool vec, const f2* f) {
    float v[NS];
#pragma unroll
    for (int i = 0; i < NS / 2; ++i) unpack(f[i], v[2 * i], v[2 * i + 1]);
    store_n<NS>(p, n, vec, v);
}

// A row of Bm or Cm, eight states from n0 on, into a tile of pairs [state pair of a lane][lane].
template <int NS, int LPC>
__device__ __forceinline__ void put_states(f2* row, int n0, const float* f) {
#pragma unroll
    for (int j = 0; j < 8 && j < NS * LPC; j += 2) {
        const int n = n0 + j;
        row[n % NS / 2 * LPC + n / NS] = pack(f[j], f[j + 1]);
    }
}

// States of a channel, padded: the power of two from 4 that holds N.
inline int padded_states(int64_t N) {
    int n = 4;
    while (n < N) n *= 2;
    return n;
}

// Values of a tile by (token, channel), staged by the thread that loads eight neighbouring
// channels of a token and read by the lanes of a warp's LC channels: index [channel of eight]
// [token][piece of eight], so that the writing lanes are neighbours and, with PAD more values
// after each of the eight planes, the reading ones fall into different banks.
template <int TT, int CH, int LC>
struct Plane {
    static constexpr int NV = CH / 8, PAD = LC >= 8 ? LC / 8 : 1, STEP = TT * NV + PAD, SIZE = 8 * STEP;
    static __device__ __forceinline__ int at(int t, int c) { return (c & 7) * STEP + t * NV + (c >> 3); }
};

// Puts two neighbouring channels' values (channels 2 j and 2 j + 1 of a piece) into a plane of
// pairs, each doubled, as the recurrence's paired instructions want them.
template <typename P>
__device__ __forceinline__ void put_doubled(f2* plane, int t, int c, f2 v) {
    float x, y;
    unpack(v, x, y);
    plane[P::at(t, c)] = pack(x, x);
    plane[P::at(t, c + 1)] = pack(y, y);
}

// Sums over the lanes `o`, 2 o, ... < END of U values at once: each stage hands half of the
// values to the other lane.  Leaves CNT values in v[0 .. CNT), those from index `at` on, the same
// in the lanes of any further stages.
template <int U, int O, int END, int CNT = U>
__device__ __forceinline__ int spread_sum(float* v, int lane, int at = 0) {
    if constexpr (O >= END) return at;
    else if constexpr (CNT > 1) {
        constexpr int H = CNT / 2;
        const bool up = lane & O;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float send = up ? v[i] : v[H + i], keep = up ? v[H + i] : v[i];
            v[i] = keep + __shfl_xor_sync(~0u, send, O);
        }
        return spread_sum<U, O * 2, END, H>(v, lane, at + (up ? H : 0));
    } else {
        v[0] += __shfl_xor_sync(~0u, v[0], O);
        return spread_sum<U, O * 2, END, 1>(v, lane, at);
    }
}
// How many values spread_sum leaves: U over the lanes' number, at least one.
constexpr int spread_left(int U, int lanes) { return U > lanes ? U / lanes : 1; }

// Whether rows of this width and distance keep 16-byte alignment at every eighth element (of each
// of their groups).
template <typename T>
__device__ __forceinline__ bool rows16(int64_t width, int64_t ld) {
    constexpr int E = 16 / sizeof(T);
    return width % E == 0 && ld % E == 0;
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
