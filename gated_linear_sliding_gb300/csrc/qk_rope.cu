// Norms of queries and keys for each head with the rotation by position, and their gradients (sm_103a).
//
//   n = w x / sqrt(mean(x^2) + eps),   (y1, y2) = (n1 cos a - n2 sin a, n2 cos a + n1 sin a)
//   dn = the rotation of dy by -a,   dw = sum dn xhat,   dx = rs (w dn - xhat mean(w dn xhat)),  xhat = rs x
//
// Each value is read and written once: 8192 tokens of 32 + 8 heads of 128 take 39 us, of which HBM needs 25; what else
// it is bound by is the issue of instructions, 54 % of the slots, with 16 warps a SM, and the wait for a token's loads.
// Weights folded into cosine and sine take fewer instructions and more registers, and 41 us.
// The gradients' kernels spill (112 bytes a thread in the main form): a warp holds the weights' sums of queries and of keys.
// A warp takes one token and walks its heads.  The token's
// cosines and sines are made by the warp's lanes once, lie in shared memory, and go to registers for all heads; a
// lane holds the same pairs of each head (both members, so the rotation needs no exchange), and as few lanes as that
// allows make a head, so that its sum of squares takes three steps for 128 values.  What a lane does is in pairs of
// fp32 registers, and the norm's factor goes into cosine and sine.
//
// Angles.  A frequency is kept as a 64-bit fraction of a turn (2^64 freq / 2 pi, made from the fp32 mantissa
// by integer products, once a CTA), so a position times it modulo 2^64 is the angle's fraction of a turn with an
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

// A pair's frequency.
struct Freq {
    uint64_t turn;
    float wild;  // NaN for a frequency that is not finite, else 0
    int axis;
};

// E pairs of a head, the first members and the second ones, as pairs of registers.
template <int E>
struct Pairs {
    f2 a[E / 2], b[E / 2];
};
// From a lane's pieces as they lie in memory: piece 2 g holds the first members and 2 g + 1 the second ones, or
// (NEAR) the two hold neighbours.
template <int V, int NG, bool NEAR>
__device__ __forceinline__ Pairs<V * NG> sorted(const float* v) {
    Pairs<V * NG> r;
#pragma unroll
    for (int e = 0; e < V * NG; e += 2) {
        const int i = 2 * (e / V) * V, m = e % V;
        if (V == 1) {
            r.a[e / 2] = pack(v[2 * e], v[2 * e + 2]);
            r.b[e / 2] = pack(v[2 * e + 1], v[2 * e + 3]);
        } else if (NEAR) {
            r.a[e / 2] = pack(v[i + 2 * m], v[i + 2 * m + 2]);
            r.b[e / 2] = pack(v[i + 2 * m + 1], v[i + 2 * m + 3]);
        } else {
            r.a[e / 2] = pack(v[i + m], v[i + m + 1]);
            r.b[e / 2] = pack(v[i + V + m], v[i + V + m + 1]);
        }
    }
    return r;
}
template <int V, int NG, bool NEAR>
__device__ __forceinline__ void unsorted(const Pairs<V * NG>& r, float* v) {
#pragma unroll
    for (int e = 0; e < V * NG; e += 2) {
        const int i = 2 * (e / V) * V, m = e % V;
        if (V == 1) {
            unpack(r.a[e / 2], v[2 * e], v[2 * e + 2]);
            unpack(r.b[e / 2], v[2 * e + 1], v[2 * e + 3]);
        } else if (NEAR) {
            unpack(r.a[e / 2], v[i + 2 * m], v[i + 2 * m + 2]);
            unpack(r.b[e / 2], v[i + 2 * m + 1], v[i + 2 * m + 3]);
        } else {
            unpack(r.a[e / 2], v[i + m], v[i + m + 1]);
            unpack(r.b[e / 2], v[i + V + m], v[i + V + m + 1]);
        }
    }
}

// NEAR: pairs of neighbours.  U heads are under way in a lane at a time.
template <typename T, int V, int NG, bool NEAR, bool BWD, int U>
__global__ void __launch_bounds__(256, 2) rope_kernel(const RopeArgs a, const RopePlan p) {
    constexpr int E = V * NG, H = E / 2;
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = a.rot / 2;
    const int hpw = 32 / p.lph, slot = lane / p.lph, in = lane % p.lph;
    const float inv_d = 1.0f / (float)a.d;
    Freq* freqs = reinterpret_cast<Freq*>(smem);                            // [half]
    float2* trig = reinterpret_cast<float2*>(freqs + half) + warp * half;  // cosine and sine of the warp's token
    for (int i = threadIdx.x; i < half; i += 256) {
        const float f = a.freqs[i];
        Freq q;
        q.turn = turns(f);
        q.wild = isfinite(f) ? 0.0f : __int_as_float(0x7fc00000);
        q.axis = a.axes == 1 ? 0 : (i >= a.section[0]) + (i >= a.section[1]) + (i >= a.section[2]);
        freqs[i] = q;
    }
    __syncthreads();
    // the places of this lane's pieces in a head, and of its pairs among the angles
    int at1[NG], at2[NG];
    bool has1[NG], has2[NG], turn[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const int i = in + p.lph * g;
        turn[g] = i < p.rot_groups;
        at1[g] = turn[g] ? (NEAR ? 2 * V * i : V * i) : a.rot + 2 * V * (i - p.rot_groups);
        at2[g] = turn[g] && !NEAR ? half + V * i : at1[g] + V;
        has1[g] = i < p.groups;
        has2[g] = has1[g] && at2[g] < a.d;
    }
    Pairs<E> dw[BWD ? 2 : 1];  // sums of dn xhat: queries, keys
    if constexpr (BWD) {
#pragma unroll
        for (int e = 0; e < H; ++e) dw[0].a[e] = dw[0].b[e] = dw[1].a[e] = dw[1].b[e] = pack(0.0f, 0.0f);
    }

    const int64_t stride = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t item = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp; item < p.items; item += stride) {
        const int64_t tok = item / p.blocks;
        const int h0 = (int)(item - tok * p.blocks) * p.heads;
        const int h1 = h0 + p.heads < a.Hq + a.Hkv ? h0 + p.heads : (int)(a.Hq + a.Hkv);
        __syncwarp();
        for (int i = lane; i < half; i += 32) {
            const Freq q = freqs[i];
            const int64_t at = a.positions != nullptr ? a.positions[tok * a.axes + q.axis] : a.start + tok % a.L;
            const int64_t frac = (int64_t)((uint64_t)at * q.turn);
            float2 t;
            sincospif((float)(int32_t)(frac >> 32) * 4.656612873077393e-10f, &t.y, &t.x);  // 2^-31
            t.x += q.wild, t.y += q.wild;
            trig[i] = t;
        }
        __syncwarp();
        f2 cs[H], sn[H];
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            float2 t[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int g = (e + k) / V, m = (e + k) % V;
                t[k] = turn[g] ? trig[V * (in + p.lph * g) + m] : make_float2(1.0f, 0.0f);
            }
            cs[e / 2] = pack(t[0].x, t[1].x);
            sn[e / 2] = BWD ? pack(-t[0].y, -t[1].y) : pack(t[0].y, t[1].y);
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
            Pairs<E> wp;
            {
                float wv[2 * E];
#pragma unroll
                for (int e = 0; e < 2 * E; ++e) wv[e] = 1.0f;
                if (w != nullptr) {
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        if (has1[g]) Vec<V>::ld(w + at1[g], wv + 2 * g * V);
                        if (has2[g]) Vec<V>::ld(w + at2[g], wv + (2 * g + 1) * V);
                    }
                }
                wp = sorted<V, NG, NEAR>(wv);
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
                    const Pairs<E> xp = sorted<V, NG, NEAR>(v);
                    if (a.norm) {
                        f2 s2 = mul2(xp.a[0], xp.a[0]);
                        s2 = fma2(xp.b[0], xp.b[0], s2);
#pragma unroll
                        for (int e = 1; e < H; ++e) s2 = fma2(xp.b[e], xp.b[e], fma2(xp.a[e], xp.a[e], s2));
                        float ss = sum2(s2);
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1)
                            if (o < p.lph) ss += __shfl_xor_sync(~0u, ss, o);
                        rs = rsqrtf(fmaf(ss, inv_d, a.eps));
                    }
                    const f2 rs2 = pack(rs, rs);
                    Pairs<E> n;  // what turns
                    if constexpr (BWD) {
#pragma unroll
                        for (int i = 0; i < 2 * NG; ++i) ry[u][i].get(v + i * V);
                        n = sorted<V, NG, NEAR>(v);
                    } else {
#pragma unroll
                        for (int e = 0; e < H; ++e) n.a[e] = mul2(xp.a[e], wp.a[e]), n.b[e] = mul2(xp.b[e], wp.b[e]);
                    }
                    Pairs<E> y;  // turned, times rs
#pragma unroll
                    for (int e = 0; e < H; ++e) {
                        const f2 c = mul2(cs[e], rs2), s = mul2(sn[e], rs2);
                        const f2 t1 = fma2(n.a[e], c, mul2(mul2(n.b[e], s), pack(-1.0f, -1.0f))), t2 = fma2(n.b[e], c, mul2(n.a[e], s));
                        y.a[e] = t1;
                        y.b[e] = t2;
                    }
                    if (p.rot_groups < p.groups) {  // beyond the rotation: not by cosine 1 and sine 0, 0 times infinity is NaN
#pragma unroll
                        for (int e = 0; e < E; e += 2) {
                            float t[4], k[4];
                            unpack(y.a[e / 2], t[0], t[1]);
                            unpack(y.b[e / 2], t[2], t[3]);
                            unpack(mul2(n.a[e / 2], rs2), k[0], k[1]);
                            unpack(mul2(n.b[e / 2], rs2), k[2], k[3]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) t[i] = turn[(e + (i & 1)) / V] ? t[i] : k[i];
                            y.a[e / 2] = pack(t[0], t[1]);
                            y.b[e / 2] = pack(t[2], t[3]);
                        }
                    }
                    if constexpr (BWD) {
                        if (a.norm) {  // y is rs dn: dw += y x, u = y w, dx = u - x rs^2 mean(u x)
                            f2 c2 = pack(0.0f, 0.0f);
#pragma unroll
                            for (int e = 0; e < H; ++e) {
                                if (h < hi) {  // (behind the last head lie zeros, and with eps 0 rs is infinite there)
                                    dw[part].a[e] = fma2(y.a[e], xp.a[e], dw[part].a[e]);
                                    dw[part].b[e] = fma2(y.b[e], xp.b[e], dw[part].b[e]);
                                }
                                y.a[e] = mul2(y.a[e], wp.a[e]);
                                y.b[e] = mul2(y.b[e], wp.b[e]);
                                c2 = fma2(y.b[e], xp.b[e], fma2(y.a[e], xp.a[e], c2));
                            }
                            float c = sum2(c2);
#pragma unroll
                            for (int o = 16; o > 0; o >>= 1)
                                if (o < p.lph) c += __shfl_xor_sync(~0u, c, o);
                            c *= -inv_d * rs * rs;
                            const f2 cc = pack(c, c);
#pragma unroll
                            for (int e = 0; e < H; ++e) y.a[e] = fma2(xp.a[e], cc, y.a[e]), y.b[e] = fma2(xp.b[e], cc, y.b[e]);
                        }
                    }
                    if (h < hi) {
                        unsorted<V, NG, NEAR>(y, v);
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const int64_t off = (int64_t)h * a.d;
                            if (has1[g]) Vec<V>::st(out + off + at1[g], v + 2 * g * V);
                            if (has2[g]) Vec<V>::st(out + off + at2[g], v + (2 * g + 1) * V);
                        }
                    }
                }
            }
        }
    }
    if constexpr (BWD) {
        if (a.dw_q == nullptr && a.dw_k == nullptr) return;
        // the CTA's sums, warps and their heads in a fixed order
        float* sums = reinterpret_cast<float*>(smem);  // [8 warps][d]
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            float v[2 * E];
            unsorted<V, NG, NEAR>(dw[part], v);
#pragma unroll
            for (int e = 0; e < 2 * E; ++e)
                for (int o = p.lph; o < 32; o <<= 1) v[e] += __shfl_xor_sync(~0u, v[e], o);
            __syncthreads();
            if (slot == 0) {
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int m = 0; m < V; ++m) {
                        if (has1[g]) sums[warp * a.d + at1[g] + m] = v[2 * g * V + m];
                        if (has2[g]) sums[warp * a.d + at2[g] + m] = v[(2 * g + 1) * V + m];
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
    // heads under way: registers for loads beat more warps (forwards 39 us against 42 with three CTAs of two heads;
    // with the gradients 187 against 191 with one head, 231 with three CTAs)
    constexpr int U = BWD ? 2 : 4;
    // eight warps a CTA; blocks of heads where the tokens alone do not make 16 warps a SM
    const RopePlan p = plan_of<V, NG>(a, 152 * 16);
    const int64_t ctas = (p.items + 7) / 8, most = BWD ? rope_bwd_ctas(a) : 152 * 2;
    const size_t half = (size_t)a.rot / 2, table = half * (sizeof(Freq) + 8 * sizeof(float2));
    const size_t sums = BWD ? sizeof(float) * 8 * (size_t)a.d : 0;
    const int64_t grid = BWD ? most : ctas < most ? ctas : most;
    rope_kernel<T, V, NG, NEAR, BWD, U><<<(unsigned)grid, 256, table > sums ? table : sums, s>>>(a, p);
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
