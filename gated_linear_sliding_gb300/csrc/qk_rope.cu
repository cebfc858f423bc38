// Norms of queries and keys for each head with the rotation by position, and their gradients (sm_103a).
//
//   n = w x / sqrt(mean(x^2) + eps),   (y1, y2) = (n1 cos a - n2 sin a, n2 cos a + n1 sin a)
//   dn = the rotation of dy by -a,   dw = sum dn xhat,   dx = rs (w dn - xhat mean(w dn xhat)),  xhat = rs x
//
// Bound by HBM: each value is read and written once.  A warp takes one token and walks its heads, so that
// the angles, which depend on the token alone, stay in registers; a lane holds the same pairs of each
// head (2 E values: both members of a pair, so the rotation needs no exchange), and as few lanes as
// that allows make a head, so that its sum of squares takes three steps for 128 values.
//
// Angles.  A frequency is kept as a 64-bit fraction of a turn (2^64 freq / 2 pi, made from the fp32 mantissa
// by integer products), so a position times it modulo 2^64 is the angle's fraction of a turn with an
// error of |position| 2^-64 turns, at any position; its upper 32 bits go through sincospi.
#include "heads.h"

namespace lz {
namespace {

// 2^64 freq / (2 pi) modulo 2^64; 2^64 / (2 pi) = 2935890503282001226 + 0x7f09 / 2^16 + ...
__device__ __forceinline__ uint64_t turns(float freq) {
    constexpr uint64_t kPer = 2935890503282001226ull, kRest = 0x7f09ull;  // 64 + 16 bits of 2^64 / 2 pi
    const uint32_t u = __float_as_uint(freq);
    const int e = (int)((u >> 23) & 255u);
    const uint64_t m = (u & 0x7fffffu) | (e > 0 ? 0x800000u : 0u);  // freq = m 2^(e' - 150)
    const int sh = (e > 0 ? e : 1) - 150 - 16;                      // of m * (kPer : kRest), 104 bits
    const uint64_t lo_part = m * kRest;                             // 40 bits
    // hi : lo = m * (kPer 2^16 + kRest)
    uint64_t lo = m * kPer, hi = __umul64hi(m, kPer);
    hi = (hi << 16) | (lo >> 48);
    lo <<= 16;
    lo += lo_part;
    hi += lo < lo_part ? 1u : 0u;
    uint64_t f;
    if (sh >= 64) f = 0;
    else if (sh >= 0) f = lo << sh;
    else if (sh > -64) f = (hi << (64 + sh)) | (lo >> -sh);
    else if (sh == -64) f = hi;
    else if (sh > -128) f = hi >> (-sh - 64);
    else f = 0;
    return (u >> 31) ? 0 - f : f;
}

struct RopePlan {
    int groups, rot_groups;  // pieces of 2 V values of a head, and how many of them turn
    int lph;                 // lanes a head
    int64_t items;           // (token, block of heads)
    int blocks, heads;       // blocks of heads a token, heads a block
};

template <int V, int NG>
RopePlan plan_of(const RopeArgs& a, int64_t want_items) {
    RopePlan p;
    p.groups = (a.d + 2 * V - 1) / (2 * V);
    p.rot_groups = a.rot / (2 * V);
    p.lph = 1;
    while (p.lph * NG < p.groups) p.lph *= 2;
    const int hpw = 32 / p.lph;
    const int64_t tokens = a.B * a.L, heads = a.Hq + a.Hkv, rounds = (heads + hpw - 1) / hpw;
    int64_t blocks = (want_items + tokens - 1) / (tokens > 0 ? tokens : 1);
    blocks = blocks < 1 ? 1 : blocks > rounds ? rounds : blocks;
    const int64_t per = (rounds + blocks - 1) / blocks;
    p.heads = (int)(per * hpw);
    p.blocks = (int)((rounds + per - 1) / per);
    p.items = tokens * p.blocks;
    return p;
}

// NEAR: pairs of neighbours.  U heads are under way in a lane at a time.
template <typename T, int V, int NG, bool NEAR, bool BWD, int U>
__global__ void __launch_bounds__(256, 2) rope_kernel(const RopeArgs a, const RopePlan p) {
    constexpr int E = V * NG;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hpw = 32 / p.lph, slot = lane / p.lph, in = lane % p.lph;
    const float inv_d = 1.0f / (float)a.d;
    // the places of this lane's pieces in a head, and their frequencies
    int at1[NG], at2[NG];
    bool has1[NG], has2[NG], turn[NG];
    uint64_t freq[E];
    unsigned wild = 0;  // frequencies that are not finite
    int axis[E];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const int i = in + p.lph * g;
        turn[g] = i < p.rot_groups;
        at1[g] = turn[g] ? (NEAR ? 2 * V * i : V * i) : a.rot + 2 * V * (i - p.rot_groups);
        at2[g] = turn[g] && !NEAR ? a.rot / 2 + V * i : at1[g] + V;
        has1[g] = i < p.groups;
        has2[g] = has1[g] && at2[g] < a.d;
#pragma unroll
        for (int m = 0; m < V; ++m) {
            const int e = g * V + m, pair = V * i + m;
            freq[e] = 0;
            axis[e] = 0;
            if (turn[g]) {
                const float f = a.freqs[pair];
                if (!isfinite(f)) wild |= 1u << e;
                freq[e] = turns(f);
                axis[e] = a.axes == 1 ? 0 : (pair >= a.section[0]) + (pair >= a.section[1]) + (pair >= a.section[2]);
            }
        }
    }
    float dw[BWD ? 2 : 1][2 * E];  // sums of dn xhat: queries, keys
    if constexpr (BWD) {
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) dw[0][e] = dw[1][e] = 0.0f;
    }

    const int64_t stride = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t item = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp; item < p.items; item += stride) {
        const int64_t tok = item / p.blocks;
        const int h0 = (int)(item - tok * p.blocks) * p.heads;
        const int h1 = h0 + p.heads < a.Hq + a.Hkv ? h0 + p.heads : (int)(a.Hq + a.Hkv);
        float cs[E], sn[E];
        int64_t pos[4];
        if (a.positions != nullptr) {
#pragma unroll
            for (int x = 0; x < 4; ++x) pos[x] = x < a.axes ? a.positions[tok * a.axes + x] : 0;
        } else {
            pos[0] = pos[1] = pos[2] = pos[3] = a.start + tok % a.L;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t at = axis[e] == 0 ? pos[0] : axis[e] == 1 ? pos[1] : axis[e] == 2 ? pos[2] : pos[3];
            const int64_t frac = (int64_t)((uint64_t)at * freq[e]);
            sincospif((float)(int32_t)(frac >> 32) * 4.656612873077393e-10f, &sn[e], &cs[e]);  // 2^-31
            if ((wild >> e) & 1u) cs[e] = sn[e] = __int_as_float(0x7fc00000);
        }
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const int lo = part == 0 ? h0 : (h0 > (int)a.Hq ? h0 : (int)a.Hq);
            const int hi = part == 0 ? (h1 < (int)a.Hq ? h1 : (int)a.Hq) : h1;
            if (lo >= hi) continue;
            const int64_t first = part == 0 ? 0 : a.Hq;
            const T* x = (const T*)(part == 0 ? a.q : a.k) + tok * (part == 0 ? a.ldq : a.ldk) - first * a.d;
            const T* dy = nullptr;
            T* out;
            if constexpr (BWD) {
                dy = (const T*)(part == 0 ? a.dq_out : a.dk_out) + tok * (part == 0 ? a.ldqo : a.ldko) - first * a.d;
                out = (T*)(part == 0 ? a.dq : a.dk) + tok * (part == 0 ? a.lddq : a.lddk) - first * a.d;
            } else {
                out = (T*)(part == 0 ? a.q_out : a.k_out) + tok * (part == 0 ? a.ldqo : a.ldko) - first * a.d;
            }
            const float* w = part == 0 ? a.w_q : a.w_k;
            float wv[2 * E];
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int m = 0; m < V; ++m) {
                    wv[2 * g * V + m] = w != nullptr && has1[g] ? w[at1[g] + m] : 1.0f;
                    wv[(2 * g + 1) * V + m] = w != nullptr && has2[g] ? w[at2[g] + m] : 1.0f;
                }
            for (int hb = lo + slot; hb - slot < hi; hb += U * hpw) {
                Pack<T, V> rx[U][2 * NG], ry[BWD ? U : 1][2 * NG];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = hb + u * hpw;
#pragma unroll
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int two = 0; two < 2; ++two) {
                            const bool on = h < hi && (two ? has2[g] : has1[g]);
                            const int64_t off = (int64_t)h * a.d + (two ? at2[g] : at1[g]);
                            Pack<T, V>& r = rx[u][2 * g + two];
                            r = Pack<T, V>{};
                            if (on && (!BWD || a.norm)) r = *reinterpret_cast<const Pack<T, V>*>(x + off);
                            if constexpr (BWD) {
                                Pack<T, V>& s = ry[u][2 * g + two];
                                s = Pack<T, V>{};
                                if (on) s = *reinterpret_cast<const Pack<T, V>*>(dy + off);
                            }
                        }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = hb + u * hpw;
                    float v[2 * E], rs = 1.0f;
#pragma unroll
                    for (int i = 0; i < 2 * NG; ++i) rx[u][i].get(v + i * V);
                    if (a.norm) {
                        float ss = 0.0f;
#pragma unroll
                        for (int e = 0; e < 2 * E; ++e) ss = fmaf(v[e], v[e], ss);
                        for (int o = p.lph / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
                        rs = rsqrtf(fmaf(ss, inv_d, a.eps));
                    }
                    float y[2 * E];
                    if constexpr (!BWD) {
#pragma unroll
                        for (int e = 0; e < 2 * E; ++e) v[e] = v[e] * rs * wv[e];
                    } else {
#pragma unroll
                        for (int i = 0; i < 2 * NG; ++i) ry[u][i].get(y + i * V);
                    }
                    float* n = BWD ? y : v;  // what turns
#pragma unroll
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int m = 0; m < V; ++m) {
                            const int e = g * V + m, i1 = 2 * g * V + (NEAR ? 2 * m : m), i2 = i1 + (NEAR ? 1 : V);
                            const float s = BWD ? -sn[e] : sn[e], n1 = n[i1], n2 = n[i2];
                            const float t1 = fmaf(n1, cs[e], -n2 * s), t2 = fmaf(n2, cs[e], n1 * s);
                            n[i1] = turn[g] ? t1 : n1;  // not by cos 1, sin 0: 0 times infinity is NaN
                            n[i2] = turn[g] ? t2 : n2;
                        }
                    if constexpr (BWD) {
                        if (a.norm) {
                            float c = 0.0f;
#pragma unroll
                            for (int e = 0; e < 2 * E; ++e) {
                                v[e] *= rs;  // xhat
                                dw[part][e] = fmaf(y[e], v[e], dw[part][e]);
                                y[e] *= wv[e];
                                c = fmaf(y[e], v[e], c);
                            }
                            for (int o = p.lph / 2; o > 0; o >>= 1) c += __shfl_xor_sync(~0u, c, o);
                            c *= inv_d;
#pragma unroll
                            for (int e = 0; e < 2 * E; ++e) y[e] = rs * fmaf(-v[e], c, y[e]);
                        }
                    }
                    if (h < hi) {
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const int64_t off = (int64_t)h * a.d;
                            if (has1[g]) Vec<V>::st(out + off + at1[g], n + 2 * g * V);
                            if (has2[g]) Vec<V>::st(out + off + at2[g], n + (2 * g + 1) * V);
                        }
                    }
                }
            }
        }
    }
    if constexpr (BWD) {
        if (a.dw_q == nullptr && a.dw_k == nullptr) return;
        // the CTA's sums, warps and their heads in a fixed order
        extern __shared__ float sums[];  // [8 warps][32 / lph][d] at most 8 * 512
#pragma unroll
        for (int part = 0; part < 2; ++part) {
#pragma unroll
            for (int e = 0; e < 2 * E; ++e)
                for (int o = p.lph; o < 32; o <<= 1) dw[part][e] += __shfl_xor_sync(~0u, dw[part][e], o);
            __syncthreads();
            if (slot == 0) {
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int m = 0; m < V; ++m) {
                        if (has1[g]) sums[warp * a.d + at1[g] + m] = dw[part][2 * g * V + m];
                        if (has2[g]) sums[warp * a.d + at2[g] + m] = dw[part][(2 * g + 1) * V + m];
                    }
            }
            __syncthreads();
            for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
                float s = 0.0f;
                for (int i = 0; i < (int)(blockDim.x >> 5); ++i) s += sums[i * a.d + c];
                a.partial[((int64_t)blockIdx.x * 2 + part) * a.d + c] = s;
            }
        }
    }
}

// dw_q and dw_k from the CTAs' sums, in a fixed order.
__global__ void __launch_bounds__(1024) rope_sum_kernel(const RopeArgs a, int64_t n) {
    float* dw = blockIdx.y == 0 ? a.dw_q : a.dw_k;
    if (dw == nullptr) return;
    const int c0 = blockIdx.x * 32, part = blockIdx.y;
    sum_columns<32>(n, a.d - c0 < 32 ? a.d - c0 : 32,
                    [&](int64_t i, int c) { return a.partial[(i * 2 + part) * a.d + c0 + c]; },
                    [&](int c, float s) { dw[c0 + c] = s; });
}

constexpr int64_t kBwdCtas = 304;  // two of 256 threads a SM

template <typename T, int V, int NG, bool NEAR, bool BWD>
cudaError_t go(const RopeArgs& a, cudaStream_t s) {
    constexpr int U = BWD ? 1 : 2;
    // eight warps a CTA; blocks of heads where the tokens alone do not make 16 warps a SM
    const RopePlan p = plan_of<V, NG>(a, 152 * 16);
    const int64_t ctas = (p.items + 7) / 8, most = BWD ? rope_bwd_ctas(a) : 152 * 8;
    const size_t sm = BWD ? sizeof(float) * 8 * (size_t)a.d : 0;
    const int64_t grid = BWD ? most : ctas < most ? ctas : most;
    rope_kernel<T, V, NG, NEAR, BWD, U><<<(unsigned)grid, 256, sm, s>>>(a, p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !BWD || (a.dw_q == nullptr && a.dw_k == nullptr)) return e;
    rope_sum_kernel<<<dim3((unsigned)((a.d + 31) / 32), 2), 1024, 0, s>>>(a, grid);
    return cudaGetLastError();
}

// Pieces of eight values where heads, halves and rows allow 16-byte accesses, of four, or single ones.
template <typename T, bool NEAR, bool BWD>
cudaError_t sized(const RopeArgs& a, cudaStream_t s) {
    const int64_t rows = a.ldq | a.ldk | a.ldqo | a.ldko | (BWD ? a.lddq | a.lddk : 0);
    if (a.d % 16 == 0 && a.rot % 16 == 0 && rows % 8 == 0) return go<T, 8, 1, NEAR, BWD>(a, s);
    if (a.d % 8 == 0 && a.rot % 8 == 0 && rows % 4 == 0) return go<T, 4, 2, NEAR, BWD>(a, s);
    return go<T, 1, 8, NEAR, BWD>(a, s);
}

template <bool BWD>
cudaError_t typed(const RopeArgs& a, cudaStream_t s) {
    if (a.dtype == LIZARD_F32)
        return a.neighbours ? sized<float, true, BWD>(a, s) : sized<float, false, BWD>(a, s);
    return a.neighbours ? sized<__nv_bfloat16, true, BWD>(a, s) : sized<__nv_bfloat16, false, BWD>(a, s);
}

}  // namespace

int64_t rope_bwd_ctas(const RopeArgs& a) {
    // a CTA for every eight tokens' worth of heads, at most what is resident
    const double work = (double)a.B * (double)a.L * (double)(a.Hq + a.Hkv) / 32.0;
    return work < 1.0 ? 1 : work < (double)kBwdCtas ? (int64_t)work : kBwdCtas;
}

cudaError_t launch_rope_fwd(const RopeArgs& a, cudaStream_t s) { return typed<false>(a, s); }
cudaError_t launch_rope_bwd(const RopeArgs& a, cudaStream_t s) { return typed<true>(a, s); }

}  // namespace lz
