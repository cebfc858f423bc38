// Helpers of the tensor-core kernels of the linear attention with a decay for each head.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "decay.cuh"
#include "sm100.cuh"
#include "tc_util.cuh"

namespace lz {
namespace {

using namespace sm100;
using tc::kdesc;
using tc::mndesc;

constexpr int kMathWarps = 8;
constexpr int kStateWarps = 8;
constexpr int kThreads = 32 * 20;
constexpr uint32_t kBox = 8192;         // a box of 64 rows x 64 columns of bf16
constexpr uint32_t kHalf = 2 * kBox;    // from the first 64 columns of 128 rows to the next

// Waits with a limit.  When one runs out it is reported once and every role leaves.  What happens while a
// wait lasts is one function for all of them: in line, the waits would fill the instruction cache.
__device__ __noinline__ bool spin(uint64_t* bar, uint32_t parity, unsigned where, volatile int* abort, WsHeader* header) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort) return false;
        if (clock64() - t0 > tc::kTimeout) {
            if (atomicExch((int*)abort, 1) == 0) report(header, LIZARD_ERR_TIMEOUT, where);
            return false;
        }
    }
    return true;
}
struct Waiter {
    volatile int* abort;
    WsHeader* header;
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity, unsigned where) const {
        return mbar_try_wait(bar, parity) || spin(bar, parity, where, abort, header);
    }
    // by all lanes of a warp: one answer
    __device__ __forceinline__ bool all(uint64_t* bar, uint32_t parity, unsigned where) const {
        return __all_sync(~0u, (*this)(bar, parity, where));
    }
};

struct Seg {
    int64_t unit, b, h, lo, hi;
    int seg;
};
template <bool ENDS>
__device__ __forceinline__ Seg seg_of(const DecayPass& p) {
    Seg s;
    s.unit = blockIdx.x % p.units;
    s.seg = (int)(blockIdx.x / p.units);
    if (ENDS) s.seg = ending_segment(p, p.parts > 0 ? 0 : s.seg);
    s.b = s.unit / p.Hkv;
    s.h = s.unit - s.b * p.Hkv;
    s.lo = (int64_t)s.seg * p.seg_len;
    s.hi = min64(s.lo + p.seg_len, p.seqs.L);
    return s;
}

// Y~ enters the MMAs as bf16 parts, each the rounded remainder of those before: two (2^-16 of a term at most) where the
// state only meets outputs of bf16, three (fp32's 24 bits) where it leaves the call in fp32 (8192 tokens in eight
// sequences: 85 and 91 us).
inline bool three_parts(const DecayPass& p) { return p.fin != nullptr; }

// The tile's first two or all three parts from y's 64 rows, by 256 threads (token, every fourth of `pieces` pieces of
// eight columns), one part 16 KB behind another; y's second 64 columns lie `apart` bytes behind the first.
template <bool ALL, int UNROLL>
__device__ __forceinline__ void scale_rows(uint32_t ys, uint32_t apart, uint32_t kt, int pieces, int n, float f, int tid) {
    const int tok = tid & 63;
    const f2 ff = pack(f, f), minus = pack(-1.0f, -1.0f);
#pragma unroll UNROLL
    for (int c = tid >> 6; c < pieces; c += 4) {
        const uint32_t off = sw128(tok, c & 7);
        uint32_t w[4] = {0, 0, 0, 0}, hi[4], lo[4];
        if (tok < n) ld_shared_v4(ys + (c >> 3) * apart + off, w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            f2 v = mul2(pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)), ff);
            unpack(v, a, b);
            hi[i] = pack_bf16(a, b);
            v = fma2(pack(__uint_as_float(hi[i] << 16), __uint_as_float(hi[i] & 0xffff0000u)), minus, v);
            unpack(v, a, b);
            lo[i] = pack_bf16(a, b);
            if (ALL) {
                unpack(fma2(pack(__uint_as_float(lo[i] << 16), __uint_as_float(lo[i] & 0xffff0000u)), minus, v), a, b);
                w[i] = pack_bf16(a, b);
            }
        }
        st_shared_v4(kt + (c >> 3) * kBox + off, hi[0], hi[1], hi[2], hi[3]);
        st_shared_v4(kt + (c >> 3) * kBox + 2 * kBox + off, lo[0], lo[1], lo[2], lo[3]);
        if (ALL) st_shared_v4(kt + (c >> 3) * kBox + 4 * kBox + off, w[0], w[1], w[2], w[3]);
    }
}
// The third part alone, in the place of the first, whose MMAs are done.
__device__ __forceinline__ void third_of_rows(uint32_t ys, uint32_t apart, uint32_t kt, int pieces, int n, float f, int tid) {
    const int tok = tid & 63;
    const f2 ff = pack(f, f), minus = pack(-1.0f, -1.0f);
#pragma unroll 1
    for (int c = tid >> 6; c < pieces; c += 4) {
        const uint32_t off = sw128(tok, c & 7);
        uint32_t w[4] = {0, 0, 0, 0};
        if (tok < n) ld_shared_v4(ys + (c >> 3) * apart + off, w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            f2 v = mul2(pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)), ff);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                unpack(v, a, b);
                const uint32_t h = pack_bf16(a, b);
                v = fma2(pack(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u)), minus, v);
            }
            unpack(v, a, b);
            w[i] = pack_bf16(a, b);
        }
        st_shared_v4(kt + (c >> 3) * kBox + off, w[0], w[1], w[2], w[3]);
    }
}
// Rows behind a tile's last token become zeros: 0 times what lies there may be NaN.
template <int THREADS>
__device__ __forceinline__ void clear_rows(uint32_t to, uint32_t apart, int n, int tid) {
#pragma unroll 1
    for (int e = tid; e < (64 - n) * 16; e += THREADS) st_shared_v4(to + ((e >> 3) & 1) * apart + sw128(n + (e >> 4), e & 7), 0, 0, 0, 0);
}

// A value that all lanes of a warp hold, as one the compiler knows to be such: operands of an MMA that are
// known to be uniform cost a fraction of the issue time.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(~0u, v, 0); }

// An MMA by the lane for which `leader` holds, in code that the whole warp runs.
__device__ __forceinline__ void mma_bf16_one(bool leader, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"((uint32_t)leader)
        : "memory");
}
__device__ __forceinline__ void mma_bf16_ts_one(bool leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"((uint32_t)leader)
        : "memory");
}

// D += Y~^T Z over a tile's 64 tokens, `parts` of Y~'s; by a warp.  z's second 64 columns lie `apart` bytes behind the first.
template <int UNROLL>
__device__ __forceinline__ void state_mmas(bool leader, uint32_t d, uint32_t kt, const int parts, uint32_t zs, uint32_t apart, uint32_t idesc, bool fresh) {
#pragma unroll UNROLL
    for (int j = 0; j < 4 * parts; ++j)
        mma_bf16_one(leader, d, mndesc(kt + (j >> 2) * 2 * kBox + (j & 3) * 2048, kBox), mndesc(zs + (j & 3) * 2048, apart), idesc, fresh && j == 0 ? 0u : 1u);
}

// Eight values of a row times f as bf16.
__device__ __forceinline__ void st_scaled8(uint32_t to, const float* v, f2 f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        unpack(mul2(pack(v[2 * i], v[2 * i + 1]), f), a, b);
        w[i] = pack_bf16(a, b);
    }
    st_shared_v4(to, w[0], w[1], w[2], w[3]);
}

// The MMAs cut an fp32 accumulator off (towards zero) with every 16 rows that they add: a state they added to directly
// lost 3e-4 of its size in 65536 tokens without a decay.  So a chunk's products are summed from zero (D), and fp32
// instructions, which round to nearest, add them to the state: S' = e^(l n) S + D.
//
// Values that are not finite.  The products of a chunk's pairs add 0 times Z for the pairs that are masked, which is NaN
// for all tokens of the chunk where Z holds a value that is not finite.  Then D is not finite either, in every row (of such
// a value of Y: in its row).  The state's warps, which move the state on, look at D, a few columns each, and note the
// sequences; when the CTA is through, it does these again by the recurrence (walk_by_tokens).
//
// A thread of the state's warps: row `row` of S, columns [z0, z1) of its half, at `at` in TMEM; D's at `sum`.  `watch`: of
// its half's four times 16 columns of D those that the thread looks at; the rows that S has share them, and each has some.
struct StateRow {
    int in, row, z0, z1;
    uint32_t at, sum, watch;
};
__device__ __forceinline__ StateRow state_row(const DecayPass& p, uint32_t tH, uint32_t tD, int in) {
    StateRow r;
    r.in = in;
    r.row = in & 127;
    r.z0 = (in >> 7) * 64;
    r.z1 = min(r.z0 + 64, p.dz);
    r.at = tH + ((uint32_t)(in & 96) << 16);
    r.sum = r.at + tD - tH;
    const int quads = (p.dx + 31) / 32, quad = r.row >> 5;
    r.watch = 0;
    if (r.row < p.dx) {
        for (int k = quad; k < 4; k += quads) r.watch |= 1u << k;
        if (r.z0 + 16 * quad >= p.dz) r.watch |= 1u;  // (columns that there are)
    }
    return r;
}

// The sum of 16 values: not finite if one of them is not.
__device__ __forceinline__ float sum16(const float* d) {
    f2 s = pack(d[0], d[1]);
#pragma unroll
    for (int i = 2; i < 16; i += 2) s = add2(s, pack(d[i], d[i + 1]));
    return sum2(s);
}
__device__ __forceinline__ bool finite(float v) { return fabsf(v) <= 3.4028234664e38f; }
// Whether a thread's part of D is.
__device__ __forceinline__ bool chunk_finite(const StateRow& r, int nz) {
    float sum = 0.0f;
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
        if (r.z0 + 16 * k >= nz || !__any_sync(~0u, r.watch >> k & 1)) continue;
        float d[16];
        tmem_get16(r.sum + r.z0 + 16 * k, d);
        if (r.watch >> k & 1) sum += sum16(d);
    }
    return finite(sum);
}

// The sequences of a segment that hold values that are not finite, as the state's warps note them.
constexpr int kMostNoted = 64;
struct Notes {
    volatile int *found;    // the number of the sequence, counted from 1, for which a warp found some
    volatile int *entered;  // where the sequence under way enters the segment (a token, or, backwards in time, the one behind it)
    volatile int *count, *at;  // those that ended; the last of kMostNoted stands for all that follow it, too
    uint64_t* agreed;
};
// At the end of the ends-th sequence, by all state warps: whether its last state may be left.  (Not one that is done again,
// since it may overwrite the first one.)
__device__ __forceinline__ bool may_leave(const Notes& o, const Waiter& wait, const StateRow& r, int nz, int ends, bool* ok) {
    if (!chunk_finite(r, nz)) *o.found = ends;
    mbar_arrive(o.agreed);
    if (!wait.all(o.agreed, (ends & 1) ^ 1, 170)) return *ok = false;
    const bool noted = __any_sync(~0u, *o.found == ends), full = __any_sync(~0u, *o.count >= kMostNoted);
    if (noted && !full && r.in == 0) {
        o.at[*o.count] = *o.entered;
        *o.count = *o.count + 1;
    }
    return !noted && !full;
}

// 16 columns of the state behind a chunk that keeps `keep` of the state in front of it.
__device__ __forceinline__ void state_behind(const StateRow& r, int c, f2 keep, float* v) {
    float d[16];
    tmem_get16(r.at + c, v);
    tmem_get16(r.sum + c, d);
#pragma unroll
    for (int i = 0; i < 16; i += 2) unpack(fma2(pack(v[i], v[i + 1]), keep, pack(d[i], d[i + 1])), v[i], v[i + 1]);
}

// The state behind a sequence's last tile (a pass whose states are transposed leaves none).
__device__ __forceinline__ void leave_state(const DecayPass& p, const StateRow& r, int64_t h, int seq, float keep) {
    if (p.fin == nullptr) return;
    float* to = p.fin + ((seq * p.Hkv + h) * p.dx + r.row) * (int64_t)p.dz;
#pragma unroll 1
    for (int c = r.z0; c < r.z1; c += 16) {
        float v[16];
        state_behind(r, c, pack(keep, keep), v);
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            if (r.row < p.dx && c + i < r.z1) *reinterpret_cast<float4*>(to + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}

// A state from memory (null: zero), or added to what is there.
__device__ __forceinline__ void fetch_state(const DecayPass& p, const StateRow& r, const float* from, bool add) {
#pragma unroll 1
    for (int c = r.z0; c < r.z0 + 64; c += 32) {
        float v[32];
        const bool on = from != nullptr && r.row < p.dx;
        if (p.transposed) {
            const float* f = from + (int64_t)c * p.dx + r.row;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = on && c + (i & ~7) < r.z1 ? f[i * p.dx] : 0.0f;
        } else {
            const float* f = from + (int64_t)r.row * p.dz + c;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (on && c + i < r.z1) u = *reinterpret_cast<const float4*>(f + i);
                v[i] = u.x, v[i + 1] = u.y, v[i + 2] = u.z, v[i + 3] = u.w;
            }
        }
        if (add) {
            float old[32];
            tmem_get32(r.at + c, old);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] += old[i];
        }
        tmem_st32(r.at + c, v);
    }
    tmem_wait_st();
}

// The state a walk begins with: the sequence's own, or the segment's.
__device__ __forceinline__ void begin_state(const DecayPass& p, const StateRow& r, const Seg& w, const Tile& t) {
    const int64_t size = (int64_t)p.dx * p.dz;
    const float* from = t.first ? sequence_state(p, t, w.h, w.seg) : first_state(p, w.unit, w.seg);
    const int parts = t.first || p.parts < 2 ? 1 : 2;
#pragma unroll 1
    for (int k = 0; k < parts; ++k) fetch_state(p, r, k == 0 ? from : from + size, k > 0);
}

// The state in front of a chunk (fresh: as it was fetched, else behind the chunk before), and its operand copy (times
// `seen`) to shared memory.  False when what the chunk before added was not finite.
__device__ __forceinline__ bool pass_state(const StateRow& r, uint32_t st, int nz, float seen, bool fresh, float keep) {
    const f2 keep2 = pack(keep, keep), seen2 = pack(seen, seen);
    float sum = 0.0f;
    uint32_t watch = r.watch;
#pragma unroll 1
    for (int c = r.z0; c < r.z0 + 64 && c < nz; c += 16, watch >>= 1) {
        float v[16];
        tmem_get16(r.at + c, v);
        if (!fresh) {
            float d[16];
            tmem_get16(r.sum + c, d);
            if (watch & 1) sum += sum16(d);
#pragma unroll
            for (int i = 0; i < 16; i += 2) unpack(fma2(pack(v[i], v[i + 1]), keep2, pack(d[i], d[i + 1])), v[i], v[i + 1]);
            tmem_st16(r.at + c, reinterpret_cast<const uint32_t*>(v));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) st_scaled8(st + (c >> 6) * kHalf + sw128(r.row, ((c & 63) >> 3) + i), v + 8 * i, seen2);
    }
    tmem_wait_st();
    return finite(sum);
}

// The outputs of a pass's tokens from `at` (backwards in time: in front of it) to the end of their sequence, or on to that of
// the CTA's segment, by the recurrence,
//   S = e^l S + in_scale y z^T, out = out_scale x S,   backwards:  S += in_scale y z^T, out = out_scale x S, S = e^l S,
// in fp32, token by token.  S is in shared memory, 32 rows of a column to a thread of the first 512; of what has several
// heads eight are taken at a time, of eight tokens where that is all of them.  2 us a token with four heads of 128 on a
// state, 5 us for both gradients.  (Short loops and the segment handed in: what needs more registers than the roles, or
// works the segment's divisions out again, has those spill, 2 to 4 % of the ordinary call.)
constexpr uint32_t kByTokensBytes = 4 * 128 * (8 * 8 + 2 * 8 + 2 * 4 * 8 + 128);
template <bool REV>
__device__ __forceinline__ void walk_by_tokens(const DecayPass& p, const Seg w, float* sm, int64_t at, bool on_to_the_end) {
    constexpr int H = 8, W = 128, NX = REV ? 8 : 64, NY = REV ? 64 : 8, PX = REV ? 1 : H;
    float *xs = sm, *ys = xs + NX * W, *zs = ys + NY * W;       // rows of a token's head, [W] each
    float *part = zs + NY * W, *S = part + 2 * 4 * PX * W;      // [2][4][heads][W], [W][W]
    static_assert(kByTokensBytes == 4 * W * (NX + 2 * NY + 2 * 4 * PX + W), "of its arrays");
    const int tid = threadIdx.x, c = tid & 127, group = tid >> 7, r0 = 32 * group;
    const float keep = power(log2_decay(p.log_decay, w.h), 1);
    const bool on = group < 4 && c < p.dz;
    const int total = REV ? p.gy : p.gx, rows = min(p.dx, r0 + 32);  // (a multiple of eight)
    float* own = S + c;
    auto stage = [&](float* to, const void* base, int64_t row, int64_t ld, int n, int heads, int64_t head0, int width, float f) {
#pragma unroll 1
        for (int e = tid; e < n * heads * 16; e += kThreads) {  // pieces of eight values
            const int i = 8 * (e & 15), k = (e >> 4) / heads, h = (e >> 4) - k * heads;
            float v[8] = {};
            if (i < width) Vec<8>::ld((const __nv_bfloat16*)base + (row + k) * ld + (head0 + h) * width + i, v);
#pragma unroll
            for (int m = 0; m < 8; ++m) v[m] *= f;
            Vec<8>::st(to + 8 * e, v);
        }
    };
    grid_dep_wait();
    Walk walk(p.seqs, w.b, REV ? w.lo : at, REV ? at : w.hi, REV, total <= H ? H : 1);
    Tile t;
    bool begun = false, last_tile = false;
    while (!last_tile && walk.next(p.seqs, w.b, &t)) {
        last_tile = t.last && !on_to_the_end;
        const int64_t row = w.b * p.seqs.L + t.t0;
        if ((t.first || !begun) && on) {
            const float* f = t.first ? sequence_state(p, t, w.h, w.seg) : first_state(p, w.unit, w.seg);
            const bool two = !t.first && p.parts == 2;
#pragma unroll 1
            for (int r = r0; r < rows; ++r) {
                const int64_t e = p.transposed ? (int64_t)c * p.dx + r : (int64_t)r * p.dz + c;
                own[r * W] = f == nullptr ? 0.0f : two ? f[e] + f[e + (int64_t)p.dx * p.dz] : f[e];
            }
        }
        begun = true;
        for (int g0 = 0; g0 < total; g0 += H) {
            const int heads = min(H, total - g0), nx = REV ? 1 : heads, ny = REV ? heads : 1;
            const bool first = g0 == 0, last = g0 + H >= total;
            __syncthreads();
            if (!REV || first) stage(xs, p.x, row, p.ldx, t.n, nx, w.h * p.gx + (REV ? 0 : g0), p.dx, 1.0f);
            if (REV || first) {
                stage(ys, p.y, row, p.ldy, t.n, ny, w.h * p.gy + (REV ? g0 : 0), p.dx, p.in_scale);
                stage(zs, p.z, row, p.ldz, t.n, ny, w.h * p.gy + (REV ? g0 : 0), p.dz, 1.0f);
            }
            __syncthreads();
#pragma unroll 1
            for (int n = 0; n < t.n; ++n) {
                const int k = REV ? t.n - 1 - n : n;
                const float *x = xs + k * nx * W, *y = ys + k * ny * W, *z = zs + k * ny * W + c;
                float* mine = part + (n & 1) * 4 * PX * W;
                if (on) {
                    float sum[PX], zc[REV ? H : 1];
#pragma unroll
                    for (int h = 0; h < PX; ++h) sum[h] = 0.0f;
#pragma unroll
                    for (int h = 0; h < (REV ? H : 1); ++h) zc[h] = h < ny ? z[h * W] : 0.0f;
                    // only rows that are part of S: 0 times infinity would be NaN in the others
#pragma unroll 2
                    for (int r = r0; r < rows; r += 4) {
                        float s[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) s[m] = own[(r + m) * W];
                        if (REV || first) {
#pragma unroll
                            for (int h = 0; h < (REV ? H : 1); ++h) {
                                if (h >= ny) continue;
                                const float4 y4 = *reinterpret_cast<const float4*>(y + h * W + r);
                                const float f = REV ? 1.0f : keep;
                                s[0] = fmaf(y4.x, zc[h], f * s[0]), s[1] = fmaf(y4.y, zc[h], f * s[1]);
                                s[2] = fmaf(y4.z, zc[h], f * s[2]), s[3] = fmaf(y4.w, zc[h], f * s[3]);
                            }
                        }
                        if (!REV || last) {
#pragma unroll
                            for (int h = 0; h < PX; ++h) {
                                if (h >= nx) continue;
                                const float4 x4 = *reinterpret_cast<const float4*>(x + h * W + r);
                                sum[h] = fmaf(x4.w, s[3], fmaf(x4.z, s[2], fmaf(x4.y, s[1], fmaf(x4.x, s[0], sum[h]))));
                            }
                        }
                        const float f = REV && last ? keep : 1.0f;
#pragma unroll
                        for (int m = 0; m < 4; ++m) own[(r + m) * W] = f * s[m];
                    }
#pragma unroll
                    for (int h = 0; h < PX; ++h)
                        if (h < nx) mine[(group * PX + h) * W + c] = sum[h];
                }
                if (REV && !last) continue;
                __syncthreads();
#pragma unroll 1
                for (int e = tid; e < nx * W; e += kThreads) {
                    if (e % W >= p.dz) continue;
                    const float o = (mine[e] + mine[PX * W + e]) + (mine[2 * PX * W + e] + mine[3 * PX * W + e]);
                    lz::st((__nv_bfloat16*)p.out + (row + k) * p.ldout + (w.h * p.gx + (REV ? 0 : g0) + e / W) * p.dz + e % W, o * p.out_scale);
                }
            }
        }
        if (t.last && p.fin != nullptr && on) {
            float* f = p.fin + (t.seq * p.Hkv + w.h) * p.dx * p.dz + c;
#pragma unroll 1
            for (int r = r0; r < rows; ++r) f[(int64_t)r * p.dz] = own[r * W];
        }
    }
    __syncthreads();
}


// [rows, heads, width] of a tensor with token distance ld, boxes of `box_rows` x 64 columns of one head.
inline bool map_of(CUtensorMap* m, const void* ptr, int64_t rows, int64_t heads, int64_t width, int64_t ld, int box_rows = 64) {
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
    return tc::make_map(m, ptr, 3, dims, strides, box);
}

}  // namespace
}  // namespace lz
