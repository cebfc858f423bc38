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
// A thread of the state's warps: row `row` of S, columns [z0, z1) of its half, at `at` in TMEM; D's at `sum`.
struct StateRow {
    int in, row, z0, z1;
    uint32_t at, sum;
};
__device__ __forceinline__ StateRow state_row(const DecayPass& p, uint32_t tH, uint32_t tD, int in) {
    StateRow r;
    r.in = in;
    r.row = in & 127;
    r.z0 = (in >> 7) * 64;
    r.z1 = min(r.z0 + 64, p.dz);
    r.at = tH + ((uint32_t)(in & 96) << 16);
    r.sum = r.at + tD - tH;
    return r;
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
// `seen`) to shared memory.
__device__ __forceinline__ void pass_state(const StateRow& r, uint32_t st, int nz, float seen, bool fresh, float keep) {
    const f2 keep2 = pack(keep, keep), seen2 = pack(seen, seen);
#pragma unroll 1
    for (int c = r.z0; c < r.z0 + 64 && c < nz; c += 16) {
        float v[16];
        if (fresh) {
            tmem_get16(r.at + c, v);
        } else {
            state_behind(r, c, keep2, v);
            tmem_st16(r.at + c, reinterpret_cast<const uint32_t*>(v));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) st_scaled8(st + (c >> 6) * kHalf + sw128(r.row, ((c & 63) >> 3) + i), v + 8 * i, seen2);
    }
    tmem_wait_st();
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
