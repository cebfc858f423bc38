// Linear attention with a decay for each head: the kernels in fp32 arithmetic for every type and shape,
// the join of segments and the single-token step (sm_103a).
//
//   S[t] = e^l S[t-1] + k[t] v[t]^T,   o[t] = scale q[t] S[t]
// In tiles of 64 tokens, with S in front of the tile and i, j places in it:
//   o[i] = scale (e^(l (i+1)) q[i] S + sum_{j <= i} e^(l (i-j)) (q[i].k[j]) v[j])
//   S'   = e^(l n) S + sum_j e^(l (n-1-j)) k[j] v[j]^T
// Every exponent is a difference of places, so no factor exceeds 1 and none needs a rescue.  The
// gradients are passes of the same form (DecayPass).  The time axis is cut into segments where sequences
// and heads are few: each segment's own end state first, a join, then the outputs.
#include "decay.cuh"

namespace lz {
namespace {

constexpr int NT = 256;
constexpr int ZS = 64;       // columns of z a CTA works on
constexpr int PS = kTile + 4;  // row of pair weights in shared memory

// A thread's pieces of a tile's rows: piece c of row r, then dr rows and dc of a row's n pieces on.
struct Pieces {
    int r, c, dr, dc, n;
};
__device__ __forceinline__ Pieces pieces_of(int n) {
    Pieces q;
    q.n = n;
    q.r = threadIdx.x / n;
    q.c = threadIdx.x - q.r * n;
    q.dr = NT / n;
    q.dc = NT - q.dr * n;
    return q;
}

// Rows [0, n) of a tile of `cols` columns as fp32 with row distance `ld` in shared memory; other places 0.  *zero, if
// asked for, becomes NaN when this thread's values are not all finite.  Pieces of V values, eight of a thread under way.
// (In line: as a function its callers spill, 16 heads on 8 of 128 in fp32, 8 x 1024 tokens, forward and gradients: 2266
// against 1949 us.)
template <typename T, int V>
__device__ __forceinline__ void load_pieces(float* to, int ld, const T* from, int64_t dist, int n, int cols, Pieces q, float* zero) {
    while (q.r < kTile) {
        float v[8][V];
        int at[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[u][i] = 0.0f;
            if (q.r < n && q.c * V < cols) Vec<V>::ld(from + q.r * dist + q.c * V, v[u]);
            at[u] = q.r < kTile ? q.r * ld + q.c * V : -1;
            q.r += q.dr;
            q.c += q.dc;
            if (q.c >= q.n) q.c -= q.n, ++q.r;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (at[u] >= 0) Vec<V>::st(to + at[u], v[u]);
        if (zero != nullptr) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int i = 0; i < V; ++i) *zero = fmaf(v[u][i], 0.0f, *zero);
        }
    }
}
__device__ __forceinline__ void load_rows(const DecayPass& p, float* to, int ld, const void* base, int64_t at, int64_t dist, int n, int cols, const Pieces& q,
                                          float* zero = nullptr) {
    if (p.f32) {
        if (p.fours) load_pieces<float, 4>(to, ld, (const float*)base + at, dist, n, cols, q, zero);
        else load_pieces<float, 1>(to, ld, (const float*)base + at, dist, n, cols, q, zero);
    } else {
        if (p.fours) load_pieces<__nv_bfloat16, 4>(to, ld, (const __nv_bfloat16*)base + at, dist, n, cols, q, zero);
        else load_pieces<__nv_bfloat16, 1>(to, ld, (const __nv_bfloat16*)base + at, dist, n, cols, q, zero);
    }
}

// acc += sum over rows j of f[j] y[j] z[j]^T: rows 4 (ty + 16 m) .. + 3 of the sum and columns 4 tx .. + 3.
template <int M>
__device__ __forceinline__ void add_products(float (&acc)[M][4][4], const float* ys, int ldx, const float* zs, const float* f, int n, int dxp) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
        float4 z = *reinterpret_cast<const float4*>(zs + j * ZS + tx * 4);
        const float w = f[j];
        z.x *= w, z.y *= w, z.z *= w, z.w *= w;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int row = 4 * (ty + 16 * m);
            if (row >= dxp) continue;
            const float4 y4 = *reinterpret_cast<const float4*>(ys + j * ldx + row);
            const float y[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[m][i][0] = fmaf(y[i], z.x, acc[m][i][0]);
                acc[m][i][1] = fmaf(y[i], z.y, acc[m][i][1]);
                acc[m][i][2] = fmaf(y[i], z.z, acc[m][i][2]);
                acc[m][i][3] = fmaf(y[i], z.w, acc[m][i][3]);
            }
        }
    }
}

struct Where {  // of a CTA's segment
    int64_t unit, b, h, lo, hi;
    int seg, slice;
};
template <bool ENDS>
__device__ __forceinline__ Where where_of(const DecayPass& p, int slices) {
    Where w;
    int64_t id = blockIdx.x;
    w.slice = (int)(id % slices);
    id /= slices;
    w.unit = id % p.units;
    w.seg = (int)(id / p.units);
    if (ENDS) w.seg = ending_segment(p, w.seg);
    w.b = w.unit / p.Hkv;
    w.h = w.unit - w.b * p.Hkv;
    w.lo = (int64_t)w.seg * p.seg_len;
    w.hi = min64(w.lo + p.seg_len, p.seqs.L);
    return w;
}

// Entry (i, j) of a state [dx][dz] as it lies in memory.
__device__ __forceinline__ int64_t state_at(const DecayPass& p, int i, int j) {
    return p.transposed ? (int64_t)j * p.dx + i : (int64_t)i * p.dz + j;
}

// A segment's own contribution to the state that leaves it (always [dk][dv]: never transposed).
template <int M>
__global__ void __launch_bounds__(NT) decay_ends_kernel(const DecayPass p, float* recs) {
    extern __shared__ float sm[];
    const int slices = (p.dz + ZS - 1) / ZS;
    const Where w = where_of<true>(p, slices);
    check_offsets(p.seqs, p.header);
    const int dxp = (p.dx + 3) / 4 * 4, ldx = dxp + 4;
    float *ys = sm, *zs = ys + kTile * ldx, *fs = zs + kTile * ZS;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int z0 = w.slice * ZS, zn = min(ZS, p.dz - z0);
    const float l2 = log2_decay(p.log_decay, w.h);
    const int v = p.fours ? 4 : 1;
    const Pieces qy = pieces_of(dxp / v), qz = pieces_of(ZS / v);
    float acc[M][4][4] = {};
    const Reach r = reach(p.seqs, w.b, w.lo, w.hi, p.rev);
    if (r.whole && p.init != nullptr) {
        const float f = power(l2, r.to - r.from);
        const float* s = p.init + (r.seq * p.Hkv + w.h) * p.dx * p.dz;
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int row = 4 * (ty + 16 * m) + i, col = tx * 4 + c;
                    if (row < p.dx && col < zn) acc[m][i][c] = f * s[state_at(p, row, z0 + col)];
                }
    }
    for (int64_t t0 = r.from; t0 < r.to; t0 += kTile) {
        const int n = (int)min64(kTile, r.to - t0);
        for (int g = 0; g < p.gy; ++g) {
            __syncthreads();
            const int64_t row = w.b * p.seqs.L + t0, head = w.h * p.gy + g;
            load_rows(p, ys, ldx, p.y, row * p.ldy + head * p.dx, p.ldy, n, p.dx, qy);
            load_rows(p, zs, ZS, p.z, row * p.ldz + head * p.dz + z0, p.ldz, n, zn, qz);
            if (g == 0 && threadIdx.x < n) fs[threadIdx.x] = power(l2, p.rev ? t0 + threadIdx.x - r.from + 1 : r.to - 1 - t0 - threadIdx.x) * p.in_scale;
            __syncthreads();
            add_products<M>(acc, ys, ldx, zs, fs, n, dxp);
        }
    }
    float* out = recs + (w.unit * p.nseg + (p.parts > 0 ? 0 : w.seg)) * p.dx * p.dz;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int row = 4 * (ty + 16 * m) + i, col = tx * 4 + c;
                if (row < p.dx && col < zn) out[(int64_t)row * p.dz + z0 + col] = acc[m][i][c];
            }
}

// The states in front of the segments from their own contributions, in place: an element a thread,
// segments in the order of time (rev: against it).  Bound by latency, so single elements, many threads, and
// some segments' loads ahead (19 segments of 8 heads: 12 us with four elements a thread, 11 with 32 segments ahead,
// whose registers cost threads).
__global__ void __launch_bounds__(256) decay_join_kernel(const DecayPass p, float* recs) {
    extern __shared__ float pass[];  // [nseg]: what of the state in front of a segment leaves it
    const int64_t size = (int64_t)p.dx * p.dz, blocks = (size + 255) / 256;
    const int64_t unit = blockIdx.x / blocks, e = (blockIdx.x % blocks) * 256 + threadIdx.x;
    const int64_t b = unit / p.Hkv;
    const float l2 = log2_decay(p.log_decay, unit - b * p.Hkv);
    for (int s = threadIdx.x; s < p.nseg; s += 256) {
        const int64_t lo = s * p.seg_len, hi = min64(lo + p.seg_len, p.seqs.L);
        pass[s] = reach(p.seqs, b, lo, hi, p.rev).whole ? -1.0f : power(l2, hi - lo);
    }
    grid_dep_launch();
    grid_dep_wait();
    __syncthreads();
    if (e >= size) return;
    float* r = recs + unit * p.nseg * size + e;
    float carry = 0.0f;
    constexpr int AHEAD = 10;
    for (int s0 = 0; s0 < p.nseg; s0 += AHEAD) {
        float own[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int s = p.rev ? p.nseg - 1 - s0 - k : s0 + k;
            if (s0 + k < p.nseg - 1 + p.all_ends) own[k] = r[s * size];  // the last segment's is nobody's first state
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int s = p.rev ? p.nseg - 1 - s0 - k : s0 + k;
            if (s0 + k < p.nseg) {
                r[s * size] = carry;
                // a sequence that begins in the segment lets nothing pass, not even NaN
                if (s0 + k < p.nseg - 1 + p.all_ends) carry = pass[s] < 0.0f ? own[k] : fmaf(pass[s], carry, own[k]);
            }
        }
    }
    if (p.all_ends) p.fin[unit * size + e] = carry;  // (of a dense batch: units are states)
}

// One pass over a segment's tiles, 64 columns of z to a CTA; M: rows of the state by 64.  Bound by the fp32 pipes and
// the latency between barriers: a thread has 4 x 4 pairs, 4 x 4 outputs and 4 M x 4 of the state, 16 products for each
// two or three 16-byte reads of shared memory.  8192 tokens of 16 heads on 8, 128 values, fp32: 595 us forwards.
// A masked pair adds 0 times its z, so a tile whose z is not all finite takes its pairs one by one (looking for that
// costs up to 1.6 %: gradients of 8 x 1024 tokens 1485 -> 1510 us).
template <int M, bool REV>
__global__ void __launch_bounds__(NT) decay_pass_kernel(const DecayPass p) {
    extern __shared__ float sm[];
    const int slices = (p.dz + ZS - 1) / ZS;
    const Where w = where_of<false>(p, slices);
    check_offsets(p.seqs, p.header);
    const int dxp = (p.dx + 3) / 4 * 4, ldx = dxp + 4;
    float* xs = sm;
    float* ys = xs + kTile * ldx;
    float* zs = ys + kTile * ldx;    // [64][ZS]
    float* ps = zs + kTile * ZS;     // [64][PS]
    float* st = ps + kTile * PS;     // [dxp][ZS]
    float* pw = st + dxp * ZS;       // powers 0 .. 64 of the decay
    float* fs = pw + kTile + 4;      // [64]: factors of the tile's rows on their way into the state
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int z0 = w.slice * ZS, zn = min(ZS, p.dz - z0);
    const int64_t size = (int64_t)p.dx * p.dz;
    const float l2 = log2_decay(p.log_decay, w.h);
    const int v = p.fours ? 4 : 1;
    const Pieces qx = pieces_of(dxp / v), qz = pieces_of(ZS / v);
    for (int i = threadIdx.x; i <= kTile; i += NT) pw[i] = power(l2, i);
    grid_dep_wait();

    Walk walk(p.seqs, w.b, w.lo, w.hi, REV);
    Tile t;
    bool begun = false;
    while (walk.next(p.seqs, w.b, &t)) {
        __syncthreads();
        if (t.first || !begun) {
            const float* from = t.first ? sequence_state(p, t, w.h, w.seg) : first_state(p, w.unit, w.seg);
#pragma unroll 8
            for (int e = threadIdx.x; e < dxp * ZS; e += NT) {
                const int i = e / ZS, j = e % ZS;
                st[e] = from != nullptr && i < p.dx && j < zn ? from[state_at(p, i, z0 + j)] : 0.0f;
            }
            begun = true;
        }
        if (threadIdx.x < t.n) fs[threadIdx.x] = pw[REV ? threadIdx.x + 1 : t.n - 1 - threadIdx.x] * p.in_scale;
        const int64_t row = w.b * p.seqs.L + t.t0;
        float zero = 0.0f;  // NaN where z has a value that is not finite
        for (int a = 0; a < p.gx; ++a) {
            float o[4][4] = {};
            for (int g = 0; g < p.gy; ++g) {
                const int64_t head = w.h * p.gy + g;
                if (g == 0) load_rows(p, xs, ldx, p.x, row * p.ldx + (w.h * p.gx + a) * p.dx, p.ldx, t.n, p.dx, qx);
                if (a == 0) {
                    load_rows(p, ys, ldx, p.y, row * p.ldy + head * p.dx, p.ldy, t.n, p.dx, qx);
                    zero = 0.0f;
                    load_rows(p, zs, ZS, p.z, row * p.ldz + head * p.dz + z0, p.ldz, t.n, zn, qz, &zero);
                }
                __syncthreads();
                // the pairs of the tile: rows ty + 16 i, columns tx + 16 j; blocks that are all masked are left out
                float s[4][4] = {};
#pragma unroll 2
                for (int k = 0; k < dxp; k += 4) {
                    float4 xv[4], yv[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        xv[i] = *reinterpret_cast<const float4*>(xs + (ty + 16 * i) * ldx + k);
                        yv[i] = *reinterpret_cast<const float4*>(ys + (tx + 16 * i) * ldx + k);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (REV ? j < i : j > i) continue;
                            s[i][j] = fmaf(xv[i].x, yv[j].x, s[i][j]);
                            s[i][j] = fmaf(xv[i].y, yv[j].y, s[i][j]);
                            s[i][j] = fmaf(xv[i].z, yv[j].z, s[i][j]);
                            s[i][j] = fmaf(xv[i].w, yv[j].w, s[i][j]);
                        }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (REV ? j < i : j > i) continue;
                        const int r = ty + 16 * i, c = tx + 16 * j, dist = REV ? c - r : r - c;
                        // (a token behind the tile's last one is 0 and its power may overflow where a state grows)
                        ps[r * PS + c] = dist >= 0 && (!REV || c < t.n) ? s[i][j] * pw[dist] * p.in_scale : 0.0f;
                    }
                if (g == 0) {  // the state's part
#pragma unroll 2
                    for (int k = 0; k < dxp; k += 4) {
                        float4 xv[4], sv[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            xv[i] = *reinterpret_cast<const float4*>(xs + (ty + 16 * i) * ldx + k);
                            sv[i] = *reinterpret_cast<const float4*>(st + (k + i) * ZS + tx * 4);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float xk[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                o[i][0] = fmaf(xk[m], sv[m].x, o[i][0]);
                                o[i][1] = fmaf(xk[m], sv[m].y, o[i][1]);
                                o[i][2] = fmaf(xk[m], sv[m].z, o[i][2]);
                                o[i][3] = fmaf(xk[m], sv[m].w, o[i][3]);
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = ty + 16 * i, far = REV ? t.n - 1 - r : r + 1;
                        const float f = r < t.n ? pw[far] : 0.0f;
#pragma unroll
                        for (int c = 0; c < 4; ++c) o[i][c] *= f;
                    }
                }
                const bool finite = __syncthreads_and(zero == 0.0f);
                if (finite) {
#pragma unroll
                    for (int kb = 0; kb < 4; ++kb)
#pragma unroll 2
                        for (int k = 16 * kb; k < 16 * kb + 16; k += 4) {
                            float4 pv[4], zv[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (REV ? kb >= i : kb <= i) pv[i] = *reinterpret_cast<const float4*>(ps + (ty + 16 * i) * PS + k);
                                zv[i] = *reinterpret_cast<const float4*>(zs + (k + i) * ZS + tx * 4);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (REV ? kb < i : kb > i) continue;
                                const float pk[4] = {pv[i].x, pv[i].y, pv[i].z, pv[i].w};
#pragma unroll
                                for (int m = 0; m < 4; ++m) {
                                    o[i][0] = fmaf(pk[m], zv[m].x, o[i][0]);
                                    o[i][1] = fmaf(pk[m], zv[m].y, o[i][1]);
                                    o[i][2] = fmaf(pk[m], zv[m].z, o[i][2]);
                                    o[i][3] = fmaf(pk[m], zv[m].w, o[i][3]);
                                }
                            }
                        }
                } else {  // 0 times such a value would be NaN: masked pairs are left out one by one
#pragma unroll 1
                    for (int k = 0; k < kTile; ++k) {
                        const float4 z = *reinterpret_cast<const float4*>(zs + k * ZS + tx * 4);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (REV ? k < ty + 16 * i : k > ty + 16 * i) continue;
                            const float w = ps[(ty + 16 * i) * PS + k];
                            o[i][0] = fmaf(w, z.x, o[i][0]);
                            o[i][1] = fmaf(w, z.y, o[i][1]);
                            o[i][2] = fmaf(w, z.z, o[i][2]);
                            o[i][3] = fmaf(w, z.w, o[i][3]);
                        }
                    }
                }
                if (a == p.gx - 1) {  // every reader of the state is past the barrier above
                    const float keep = g == 0 ? pw[t.n] : 1.0f;
                    float acc[M][4][4];
#pragma unroll
                    for (int m = 0; m < M; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 4 * (ty + 16 * m) + i;
                            float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            if (r < dxp) u = *reinterpret_cast<const float4*>(st + r * ZS + tx * 4);
                            acc[m][i][0] = u.x * keep, acc[m][i][1] = u.y * keep, acc[m][i][2] = u.z * keep, acc[m][i][3] = u.w * keep;
                        }
                    add_products<M>(acc, ys, ldx, zs, fs, t.n, dxp);
#pragma unroll
                    for (int m = 0; m < M; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 4 * (ty + 16 * m) + i;
                            if (r < dxp) *reinterpret_cast<float4*>(st + r * ZS + tx * 4) = make_float4(acc[m][i][0], acc[m][i][1], acc[m][i][2], acc[m][i][3]);
                        }
                }
                __syncthreads();
            }
            const int64_t to = row * p.ldout + (w.h * p.gx + a) * p.dz + z0 + tx * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = ty + 16 * i;
#pragma unroll
                for (int c = 0; c < 4; ++c) o[i][c] *= p.out_scale;
                if (r >= t.n) continue;
                const int64_t at = to + r * p.ldout;
                if (p.fours) {
                    if (tx * 4 >= zn) continue;
                    if (p.f32) Vec<4>::st((float*)p.out + at, o[i]);
                    else Vec<4>::st((__nv_bfloat16*)p.out + at, o[i]);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (tx * 4 + c >= zn) continue;
                        if (p.f32) lz::st((float*)p.out + at + c, o[i][c]);
                        else lz::st((__nv_bfloat16*)p.out + at + c, o[i][c]);
                    }
                }
            }
        }
        if (t.last && p.fin != nullptr) {
            float* to = p.fin + (t.seq * p.Hkv + w.h) * size;
            for (int e = threadIdx.x; e < p.dx * ZS; e += NT) {
                const int i = e / ZS, j = e % ZS;
                if (j < zn) to[state_at(p, i, z0 + j)] = st[e];
            }
        }
    }
}

// States of empty sequences: what they begin with.  1024 elements to a CTA.
__global__ void __launch_bounds__(256) decay_empty_kernel(const Seqs s, const float* init, float* fin, int64_t Hkv, int64_t size) {
    const int64_t blocks = (size + 1023) / 1024, state = blockIdx.x / blocks, seq = state / Hkv;
    int64_t end;
    if (s.cu != nullptr ? s.cu[seq + 1] != s.cu[seq] : seq_tokens(s, seq, &end) != 0) return;
    const int64_t first = blockIdx.x % blocks * 1024, base = state * size;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t e = first + k * 256 + threadIdx.x;
        if (e < size) fin[base + e] = init != nullptr ? init[base + e] : 0.0f;
    }
}

// The first states of the sequences that hold the tokens behind the cuts.  1024 elements to a CTA.
__global__ void __launch_bounds__(256) decay_keep_kernel(const DecayPass p, float* kept) {
    const int64_t size = (int64_t)p.dx * p.dz, blocks = (size + 1023) / 1024;
    const int64_t state = blockIdx.x / blocks, cut = state / p.Hkv, h = state - cut * p.Hkv;
    const float* from = p.init + (seq_at(p.seqs, 0, (cut + 1) * p.seg_len).seq * p.Hkv + h) * size;
    const int64_t first = blockIdx.x % blocks * 1024;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t e = first + k * 256 + threadIdx.x;
        if (e < size) kept[state * size + e] = from[e];
    }
}

size_t ends_smem(int dx) { return sizeof(float) * (size_t)(kTile * ((dx + 3) / 4 * 4 + 4) + kTile * ZS + kTile); }
size_t pass_smem(int dx) {
    const int dxp = (dx + 3) / 4 * 4;
    return sizeof(float) * (size_t)(2 * kTile * (dxp + 4) + kTile * ZS + kTile * PS + dxp * ZS + 2 * kTile + 4);
}
constexpr size_t kMostSmem = sizeof(float) * (2 * kTile * (192 + 4) + kTile * ZS + kTile * PS + 192 * ZS + 2 * kTile + 4);
static_assert(kMostSmem <= 226 * 1024, "within a SM's shared memory");

cudaError_t run_ends(const DecayPass& p, float* recs, cudaStream_t s) {
    const unsigned grid = (unsigned)(p.units * (p.nseg - 1) * ((p.dz + ZS - 1) / ZS));
    const auto kernel = p.dx <= 64 ? decay_ends_kernel<1> : p.dx <= 128 ? decay_ends_kernel<2> : decay_ends_kernel<3>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ends_smem(192));
    if (e != cudaSuccess) return e;
    kernel<<<grid, NT, ends_smem(p.dx), s>>>(p, recs);
    return cudaGetLastError();
}

template <bool REV>
cudaError_t run_pass(const DecayPass& p, cudaStream_t s) {
    const unsigned grid = (unsigned)(p.units * p.nseg * ((p.dz + ZS - 1) / ZS));
    const auto kernel = p.dx <= 64 ? decay_pass_kernel<1, REV> : p.dx <= 128 ? decay_pass_kernel<2, REV> : decay_pass_kernel<3, REV>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostSmem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, NT, pass_smem(p.dx), s>>>(p);
    return cudaGetLastError();
}

cudaError_t run_join(const DecayPass& p, float* recs, cudaStream_t s) {
    const int64_t size = (int64_t)p.dx * p.dz;
    const cudaError_t e = launch_dependent(decay_join_kernel, dim3((unsigned)(p.units * ((size + 255) / 256))), dim3(256),
                                           sizeof(float) * p.nseg, s, p, recs);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Of two segments of a dense batch the one's end state is the other's first: nothing to join.  On the tensor
// cores two CTAs share such a segment (two segments are cut where there are CTAs for at most half the SMs).
int parts_of(const DecayArgs& a, const DecayPass& p) {
    if (p.nseg != 2 || a.seqs.cu != nullptr) return 0;
    return decay_uses_tc(a) ? 2 : 1;
}

// The states in front of the segments, [units, nseg, dk, dv], from a pass that is not transposed.  On the tensor cores
// the join of a dense batch also leaves its last states, and the pass, which then needs no third part of its products
// into the state, has none to leave (65536 tokens: 276 us, else 309).
cudaError_t segment_states(const DecayArgs& a, DecayPass* pass, float* recs, cudaStream_t s) {
    DecayPass& p = *pass;
    if (p.nseg == 1) return cudaSuccess;
    p.all_ends = decay_uses_tc(a) && a.seqs.cu == nullptr && p.parts == 0 && p.fin != nullptr;
    const cudaError_t e = decay_uses_tc(a) ? decay_tc_ends(p, recs, s) : run_ends(p, recs, s);
    if (e != cudaSuccess || p.parts > 0) return e;
    const cudaError_t j = run_join(p, recs, s);
    if (p.all_ends) p.fin = nullptr;
    return j;
}

cudaError_t outputs(const DecayArgs& a, const DecayPass& p, cudaStream_t s) {
    if (decay_uses_tc(a)) return decay_tc_pass(p, s);
    return p.rev ? run_pass<true>(p, s) : run_pass<false>(p, s);
}

cudaError_t empty_states(const DecayArgs& a, const float* init, float* fin, cudaStream_t s) {
    if (fin == nullptr || fin == init || (a.seqs.cu == nullptr && a.seqs.L > 0)) return cudaSuccess;
    decay_empty_kernel<<<(unsigned)(a.nstate * a.Hkv * ((a.dk * a.dv + 1023) / 1024)), 256, 0, s>>>(a.seqs, init, fin, a.Hkv, a.dk * a.dv);
    return cudaGetLastError();
}

size_t records(const DecayPass& p) { return p.nseg == 1 ? 0 : (size_t)(p.units * p.nseg) * p.dx * p.dz; }

// Where the last states overwrite the first ones, another segment's CTA may write one before a CTA has
// read it: such a pass reads a copy.  Only a sequence that lies across a cut is in danger, so of many packed sequences
// those at the cuts are copied (all of them, 8192 with 8 heads of 128 x 128, would take 4 GiB), else all.
bool keeps_by_cut(const DecayArgs& a, const DecayPass& p) { return a.seqs.nseq > p.nseg - 1; }
size_t kept_states(const DecayArgs& a, const DecayPass& p) {
    return (size_t)((keeps_by_cut(a, p) ? p.nseg - 1 : a.nstate) * a.Hkv * a.dk * a.dv);
}

cudaError_t own_first_states(const DecayArgs& a, DecayPass* p, float* copy, cudaStream_t s) {
    if (p->nseg == 1 || p->init == nullptr || p->init != p->fin) return cudaSuccess;
    if (keeps_by_cut(a, *p)) {
        decay_keep_kernel<<<(unsigned)((p->nseg - 1) * a.Hkv * ((a.dk * a.dv + 1023) / 1024)), 256, 0, s>>>(*p, copy);
        p->kept = copy;
        return cudaGetLastError();
    }
    const size_t bytes = sizeof(float) * (size_t)(a.nstate * a.Hkv * a.dk * a.dv);
    const cudaError_t e = cudaMemcpyAsync(copy, p->init, bytes, cudaMemcpyDeviceToDevice, s);
    p->init = copy;
    return e;
}

// Segments of whole tiles: as many as keep the CTAs, of sequences, heads and slices, within what is resident at
// a time (fp32 arithmetic: two CTAs a SM where their shared memory allows).
void cut(const DecayArgs& a, DecayPass* p) {
    const bool tensor = decay_uses_tc(a);
    const int64_t ctas = tensor ? p->units : p->units * ((a.dv + ZS - 1) / ZS), tiles = (a.seqs.L + kTile - 1) / kTile;
    const int64_t room = tensor || 2 * pass_smem((int)(a.dk > a.dv ? a.dk : a.dv)) > 226 * 1024 ? 152 : 304;
    int64_t n = room / ctas;
    n = n < tiles ? n : tiles;
    n = n < 1 ? 1 : n;
    const int64_t per = (tiles + n - 1) / n;
    p->seg_len = (per > 0 ? per : 1) * kTile;
    p->nseg = (int)(per > 0 ? (tiles + per - 1) / per : 1);
}

DecayPass base_pass(const DecayArgs& a) {
    DecayPass p{};
    p.units = a.B * a.Hkv;
    p.Hkv = a.Hkv;
    p.seqs = a.seqs;
    p.log_decay = a.log_decay;
    p.header = a.header;
    p.in_scale = p.out_scale = 1.0f;
    p.f32 = a.dtype == LIZARD_F32;
    p.fours = ((a.dk | a.dv | a.ldq | a.ldk | a.ldv | a.ldo | a.lddq | a.lddk | a.lddv) & 3) == 0;
    cut(a, &p);
    p.parts = parts_of(a, p);
    return p;
}

DecayPass output_pass(const DecayArgs& a) {
    DecayPass p = base_pass(a);
    p.x = a.q, p.y = a.k, p.z = a.v, p.out = a.o;
    p.ldx = a.ldq, p.ldy = a.ldk, p.ldz = a.ldv, p.ldout = a.ldo;
    p.dx = (int)a.dk, p.dz = (int)a.dv;
    p.gx = (int)(a.Hq / a.Hkv), p.gy = 1;
    p.out_scale = a.scale;
    p.init = a.s0;
    p.fin = a.s_out;
    return p;
}

DecayPass dq_pass(const DecayArgs& a) {
    DecayPass p = output_pass(a);
    p.x = a.d_o, p.y = a.v, p.z = a.k, p.out = a.dq;
    p.ldx = a.ldo, p.ldy = a.ldv, p.ldz = a.ldk, p.ldout = a.lddq;
    p.dx = (int)a.dv, p.dz = (int)a.dk;
    p.transposed = true;
    p.fin = nullptr;
    return p;
}

DecayPass dv_pass(const DecayArgs& a) {
    DecayPass p = base_pass(a);
    p.x = a.k, p.y = a.q, p.z = a.d_o, p.v = a.v, p.out = a.dv_;
    p.ldv = a.ldv;
    p.ldx = a.ldk, p.ldy = a.ldq, p.ldz = a.ldo, p.ldout = a.lddv;
    p.dx = (int)a.dk, p.dz = (int)a.dv;
    p.gx = 1, p.gy = (int)(a.Hq / a.Hkv);
    p.rev = true;
    p.in_scale = a.scale;
    p.init = a.ds_out;
    p.fin = a.ds0;
    return p;
}

DecayPass dk_pass(const DecayArgs& a) {
    DecayPass p = dv_pass(a);
    p.x = a.v, p.y = a.d_o, p.z = a.q, p.out = a.dk_;
    p.ldx = a.ldv, p.ldy = a.ldo, p.ldz = a.ldq, p.ldout = a.lddk;
    p.dx = (int)a.dv, p.dz = (int)a.dk;
    p.transposed = true;
    p.fin = nullptr;
    return p;
}

// --------------------------------------------------------------------------- single tokens

constexpr int SNT = 128;
constexpr int SW = 32;  // columns of the state a CTA moves on

// A CTA takes 32 columns of one state: S = e^l S + k v^T in registers and back, and q S for GH query heads
// at a time.  Bound by HBM: the state is read and written once.  128-byte rows, eight of them a thread
// in flight.
template <typename T, int V, int GH>
__global__ void __launch_bounds__(SNT) decay_step_kernel(const DecayArgs a) {
    extern __shared__ float sm[];
    constexpr int LANES = SW / V, RG = SNT / LANES, R = V == 4 ? 8 : 16;
    const int dk = (int)a.dk, dv = (int)a.dv, G = (int)(a.Hq / a.Hkv);
    float* ks = sm;            // [dk]
    float* qs = ks + dk;       // [GH][dk]
    float* part = qs + GH * dk;  // [4 warps][GH][SW]
    const int slices = (dv + SW - 1) / SW;
    const int64_t id = blockIdx.x / slices, b = id / a.Hkv, h = id - b * a.Hkv;
    const int lane = threadIdx.x % LANES, rg = threadIdx.x / LANES, warp = threadIdx.x >> 5;
    const int c0 = (int)(blockIdx.x % slices) * SW, c = c0 + lane * V;
    const bool on = c < dv;
    int64_t slot = a.slots != nullptr ? a.slots[b] : b;
    if (slot >= a.nslots) {
        if (threadIdx.x == 0) report(a.header, LIZARD_ERR_INVALID_ARG, 96);
        slot = -1;
    }
    T* out = (T*)a.o + b * a.ldo + h * G * dv;
    if (slot < 0) {
        for (int e = threadIdx.x; e < G * SW; e += SNT)
            if (c0 + e % SW < dv) lz::st(out + (int64_t)(e / SW) * dv + c0 + e % SW, 0.0f);
        return;
    }
    float* S = a.state + (slot * a.Hkv + h) * dk * dv;
    float s[R][V];
    auto fetch = [&](int r0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = r0 + r * RG;
#pragma unroll
            for (int i = 0; i < V; ++i) s[r][i] = 0.0f;
            if (on && row < dk) Vec<V>::ld(S + (int64_t)row * dv + c, s[r]);
        }
    };
    fetch(rg);  // before anything else: these loads are what the time goes to
    const float keep = power(log2_decay(a.log_decay, h), 1);
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
    if (on) Vec<V>::ld((const T*)a.v + b * a.ldv + h * dv + c, v);
    for (int i = threadIdx.x; i < dk; i += SNT) ks[i] = lz::ld((const T*)a.k + b * a.ldk + h * dk + i);
    for (int g0 = 0; g0 < G; g0 += GH) {
        const int gn = min(GH, G - g0);
        const T* q = (const T*)a.q + b * a.ldq + (h * G + g0) * dk;
        for (int i = threadIdx.x; i < GH * dk; i += SNT) qs[i] = i < gn * dk ? lz::ld(q + i) : 0.0f;
        __syncthreads();
        float acc[GH][V] = {};
        for (int r0 = rg; r0 < dk; r0 += RG * R) {
            if (g0 > 0 || r0 > rg) fetch(r0);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = r0 + r * RG;
                if (row >= dk) continue;
                if (g0 == 0) {
#pragma unroll
                    for (int i = 0; i < V; ++i) s[r][i] = fmaf(ks[row], v[i], keep * s[r][i]);
                    if (on) Vec<V>::st(S + (int64_t)row * dv + c, s[r]);
                }
#pragma unroll
                for (int g = 0; g < GH; ++g)
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[g][i] = fmaf(qs[g * dk + row], s[r][i], acc[g][i]);
            }
        }
        // the rows' sums: lanes of a warp, then warps
#pragma unroll
        for (int g = 0; g < GH; ++g)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                for (int o = LANES; o < 32; o <<= 1) acc[g][i] += __shfl_xor_sync(~0u, acc[g][i], o);
                if ((threadIdx.x & 31) < LANES) part[(warp * GH + g) * SW + lane * V + i] = acc[g][i];
            }
        __syncthreads();
        for (int e = threadIdx.x; e < gn * SW; e += SNT) {
            const int g = e / SW, col = e % SW;
            float s = 0.0f;
            for (int i = 0; i < SNT / 32; ++i) s += part[(i * GH + g) * SW + col];
            if (c0 + col < dv) lz::st(out + (int64_t)(g0 + g) * dv + c0 + col, s * a.scale);
        }
        __syncthreads();
    }
}

template <typename T, int V, int GH>
cudaError_t step_go(const DecayArgs& a, cudaStream_t s) {
    const size_t sm = sizeof(float) * (size_t)((1 + GH) * a.dk + SNT / 32 * GH * SW);
    decay_step_kernel<T, V, GH><<<(unsigned)(a.B * a.Hkv * ((a.dv + SW - 1) / SW)), SNT, sm, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t step_heads(const DecayArgs& a, cudaStream_t s) {
    const int64_t G = a.Hq / a.Hkv;
    return G == 1 ? step_go<T, V, 1>(a, s) : G == 2 ? step_go<T, V, 2>(a, s) : G <= 4 ? step_go<T, V, 4>(a, s) : step_go<T, V, 8>(a, s);
}

// Four columns at a time where rows of the state and of v keep 16 and 8 bytes.
template <typename T>
cudaError_t step_typed(const DecayArgs& a, cudaStream_t s) {
    return a.dv % 4 == 0 && a.ldv % 4 == 0 ? step_heads<T, 4>(a, s) : step_heads<T, 1>(a, s);
}

}  // namespace

// Forward: the states of its segments; backward: those of S and of dS.  Behind them, with segments, what
// own_first_states copies in calls whose last states overwrite the first ones.
size_t decay_ws_floats(const DecayArgs& a, bool bwd) {
    const DecayPass p = base_pass(a);
    return p.nseg == 1 ? 0 : (size_t)(p.units * p.nseg * (bwd ? 2 : 1) * a.dk * a.dv) + kept_states(a, p);
}

cudaError_t launch_decay_fwd(const DecayArgs& a, cudaStream_t s) {
    cudaError_t e = empty_states(a, a.s0, a.s_out, s);
    if (e != cudaSuccess || a.seqs.L == 0) return e;
    DecayPass p = output_pass(a);
    p.recs = a.ws;
    if ((e = own_first_states(a, &p, a.ws + records(p), s)) != cudaSuccess) return e;
    e = segment_states(a, &p, a.ws, s);
    return e != cudaSuccess ? e : outputs(a, p, s);
}

cudaError_t launch_decay_bwd(const DecayArgs& a, cudaStream_t s) {
    cudaError_t e = empty_states(a, a.ds_out, a.ds0, s);
    if (e != cudaSuccess || a.seqs.L == 0) return e;
    DecayPass q = dq_pass(a), v = dv_pass(a), k = dk_pass(a);
    DecayArgs f = a;  // S in front of the segments, as the forward has it
    f.s_out = nullptr;
    DecayPass o = output_pass(f);
    float* recs = a.ws + records(v);
    q.recs = a.ws;
    v.recs = k.recs = recs;
    if ((e = segment_states(a, &o, a.ws, s)) != cudaSuccess) return e;
    if ((e = outputs(a, q, s)) != cudaSuccess) return e;
    // dk reads ds_out: before dv, which may overwrite it with ds0
    if ((e = own_first_states(a, &v, recs + records(v), s)) != cudaSuccess) return e;
    if ((e = segment_states(a, &v, recs, s)) != cudaSuccess) return e;
    if (decay_uses_tc(a)) return decay_tc_grads(v, a.dk_, a.lddk, s);
    if ((e = outputs(a, k, s)) != cudaSuccess) return e;
    return outputs(a, v, s);
}

cudaError_t launch_decay_step(const DecayArgs& a, cudaStream_t s) {
    return a.dtype == LIZARD_F32 ? step_typed<float>(a, s) : step_typed<__nv_bfloat16>(a, s);
}

}  // namespace lz
