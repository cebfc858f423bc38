// Linear attention with a decay for each head on the tensor cores (tcgen05, TMEM and TMA, sm_103a): bf16,
// keys and values of up to 128 values.
//
// One kernel runs every pass (DecayPass: the outputs, dq, and backwards in time dv and dk).  A CTA walks a
// segment of one state head in tiles of 64 tokens.  With X up to two query heads of a tile as 128 rows, Y and
// Z the tile's 64 tokens and S the state in front of it, an item is
//   P = (X Y^T) (.) e^(l |i - j|)          [128 x 64], masked to the tokens before (rev: behind)
//   O = e^(l (i+1)) (X S) + P Z            [128 x dz]
// and a tile moves the state on:  S' = e^(l n) S + Y~^T Z,  Y~[j] = e^(l (n-1-j)) Y[j].
// Every power is of a difference of places, so all factors lie in [0, 1].
//
// Roundings: P and the operand copy of S are bf16 (a relative 2^-8 of the terms, as the output's own).  S itself
// stays in fp32 in TMEM, and Y~ goes in as a high and a low bf16 part (2^-17), since S leaves the call in fp32
// and what is rounded there would stay for the rest of the sequence.
//
// Warps: 0-7 the pairs' weights, the state part's scale and the outputs (a thread holds one row's 32 of the 64
// pairs and 64 of the 128 output columns); 8-11 the state (a row of S to a thread; Y~); 12 the copies; 13 the
// MMAs of the items; 14 those of the state.  TMEM: P and its scores two of 64 columns, O two of 128, S 128.
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
constexpr int kThreads = 32 * 15;
constexpr uint32_t kBox = 8192;  // a box of 64 rows x 64 columns of bf16

struct TcArgs {
    CUtensorMap x, y, z;
    DecayPass p;
};

// Shared memory: XST stages of XB boxes of x, YST of y and z, Y~, the state's operand copy.
template <int XST_, int XB_, int YST_, bool REV_>
struct Layout {
    static constexpr int XST = XST_, XB = XB_, YST = YST_;
    static constexpr bool REV = REV_;
    static constexpr uint32_t X = 0;
    static constexpr uint32_t YZ = XST * XB * kBox;
    static constexpr uint32_t KT = YZ + YST * 4 * kBox;  // high part, low part
    static constexpr uint32_t ST = KT + 4 * kBox;
    static constexpr uint32_t TABLE = ST + 4 * kBox;     // powers 0 .. 64, and times in_scale
    static constexpr uint32_t BARS = TABLE + 2 * 72 * 4;
    static constexpr uint32_t BYTES = BARS + 320 + 1024;
    static_assert(BYTES <= 227 * 1024, "shared memory of a CTA");
};
// forwards: tiles of two heads of x stream past one of y and z; backwards: heads of y and z past one of x
using Forwards = Layout<3, 4, 2, false>;
using Backwards = Layout<2, 2, 4, true>;

// Waits with a limit.  When one runs out it is reported once and every role leaves.
struct Waiter {
    volatile int* abort;
    WsHeader* header;
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity, unsigned where) const {
        if (mbar_try_wait(bar, parity)) return true;
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
    // by all lanes of a warp: one answer
    __device__ __forceinline__ bool all(uint64_t* bar, uint32_t parity, unsigned where) const {
        return __all_sync(~0u, (*this)(bar, parity, where));
    }
};

struct Seg {
    int64_t unit, b, h, lo, hi;
    int seg;
};
__device__ __forceinline__ Seg seg_of(const DecayPass& p) {
    Seg s;
    s.unit = blockIdx.x % p.units;
    s.seg = (int)(blockIdx.x / p.units);
    s.b = s.unit / p.Hkv;
    s.h = s.unit - s.b * p.Hkv;
    s.lo = (int64_t)s.seg * p.seg_len;
    s.hi = min64(s.lo + p.seg_len, p.seqs.L);
    return s;
}

// The tile of Y~ from y's, as high and low parts, by 128 threads (token, half of the columns); and rows of z
// behind the tile's last token become zeros: 0 times what lies there may be NaN.
__device__ __forceinline__ void scale_rows(uint32_t ys, uint32_t zs, uint32_t kt, int n, float f, int tid) {
    const int tok = tid & 63, half = tid >> 6;
    const uint32_t from = ys + half * kBox, to = kt + half * kBox;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint32_t off = sw128(tok, c);
        uint32_t w[4] = {0, 0, 0, 0}, hi[4], lo[4];
        if (tok < n) ld_shared_v4(from + off, w[0], w[1], w[2], w[3]);
        float v[8];
        tc::unpack8(w[0], w[1], w[2], w[3], v);
#pragma unroll
        for (int i = 0; i < 4; ++i) tc::split2(v[2 * i] * f, v[2 * i + 1] * f, hi[i], lo[i]);
        st_shared_v4(to + off, hi[0], hi[1], hi[2], hi[3]);
        st_shared_v4(to + 2 * kBox + off, lo[0], lo[1], lo[2], lo[3]);
        if (tok >= n) st_shared_v4(zs + half * kBox + off, 0, 0, 0, 0);
    }
}

// S += Y~^T Z over a tile's 64 tokens, both parts; one thread.
__device__ __forceinline__ void state_mmas(uint32_t d, uint32_t kt, uint32_t zs, uint32_t idesc, bool fresh) {
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        const uint64_t a = mndesc(kt + part * 2 * kBox, kBox), b = mndesc(zs, kBox);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_bf16(d, a + ((j * 2048) >> 4), b + ((j * 2048) >> 4), idesc, fresh && part == 0 && j == 0 ? 0u : 1u);
    }
}

template <typename SM>
__global__ void __launch_bounds__(kThreads, 1) decay_tc_kernel(const __grid_constant__ TcArgs g) {
    constexpr int XST = SM::XST, XB = SM::XB, YST = SM::YST;
    constexpr bool rev = SM::REV;
    extern __shared__ uint8_t smem_raw[];
    const DecayPass& p = g.p;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (base - smem_u32(smem_raw));
    float* pw = reinterpret_cast<float*>(sm + SM::TABLE);  // powers of the decay
    float* pws = pw + 72;                                  // times in_scale
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + SM::BARS);
    uint64_t *x_full = bar, *x_free = bar + 3, *yz_full = bar + 6, *yz_free = bar + 10, *zz_full = bar + 14, *s_full = bar + 18,
             *p_full = bar + 20, *xs_full = bar + 22, *pv_done = bar + 24, *o_free = bar + 26, *kt_full = bar + 28,
             *h_done = bar + 29, *st_full = bar + 30, *xs_done = bar + 31;
    uint64_t *pair = bar + 32, *drained = bar + 36;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 37);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Seg w = seg_of(p);
    check_offsets(p.seqs, p.header);
    const float l2 = log2_decay(p.log_decay, w.h);
    for (int i = tid; i <= kTile; i += kThreads) {
        pw[i] = power(l2, i);
        pws[i] = pw[i] * p.in_scale;
    }
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) {
            mbar_init(&x_full[i], 1);
            mbar_init(&x_free[i], 32 * kMathWarps);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&yz_full[i], 1);
            mbar_init(&yz_free[i], 2);
            mbar_init(&zz_full[i], 128);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 32 * kMathWarps);
            mbar_init(&xs_full[i], 1);
            mbar_init(&pv_done[i], 1);
            mbar_init(&o_free[i], 32 * kMathWarps);
        }
        mbar_init(kt_full, 128);
        mbar_init(h_done, 1);
        mbar_init(st_full, 128);
        mbar_init(xs_done, 1);
        for (int i = 0; i < 4; ++i) mbar_init(&pair[i], 64);
        mbar_init(drained, 1);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == 13) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = *tmem_slot;
    const uint32_t tS = tb, tO = tb + 128, tH = tb + 384;
    const Waiter wait{abort, p.header};
    const int nhx = (p.dx + 63) / 64, nhz = (p.dz + 63) / 64;
    const int kx = (p.dx + 15) / 16;                 // K steps over dx
    const int nz = (p.dz + 15) / 16 * 16;            // N over dz
    const int ntx = (p.gx + 1) / 2;                  // tiles of x heads
    constexpr uint32_t xhalf = (XB / 2) * kBox;      // from the first 64 columns of x to the next

    Walk walk(p.seqs, w.b, w.lo, w.hi, rev);
    Tile t;

    if (warp == 12) {
        if (lane == 0) {
            prefetch_tmap(&g.x);
            prefetch_tmap(&g.y);
            prefetch_tmap(&g.z);
            uint32_t xt = 0, yi = 0;
            bool ok = true;
            while (ok && walk.next(p.seqs, w.b, &t)) {
                const int row = (int)(w.b * p.seqs.L + t.t0);
                for (int a = 0; a < ntx && ok; ++a) {
                    for (int gh = 0; gh < p.gy && ok; ++gh) {
                        if (a == 0) {
                            const int s = yi % YST;
                            if (yi >= YST && !wait(&yz_free[s], ((yi / YST) & 1) ^ 1, 100)) {
                                ok = false;
                                break;
                            }
                            uint8_t* to = sm + SM::YZ + s * 4 * kBox;
                            mbar_arrive_expect_tx(&yz_full[s], (nhx + nhz) * kBox);
                            const int head = (int)(w.h * p.gy + gh);
                            for (int h = 0; h < nhx; ++h) tma_load_3d(to + h * kBox, &g.y, &yz_full[s], 64 * h, head, row);
                            for (int h = 0; h < nhz; ++h) tma_load_3d(to + (2 + h) * kBox, &g.z, &yz_full[s], 64 * h, head, row);
                            ++yi;
                        }
                        if (gh == 0) {
                            const int s = xt % XST, heads = p.gx - 2 * a < 2 ? 1 : 2;
                            if (xt >= XST && !wait(&x_free[s], ((xt / XST) & 1) ^ 1, 101)) {
                                ok = false;
                                break;
                            }
                            uint8_t* to = sm + SM::X + s * XB * kBox;
                            mbar_arrive_expect_tx(&x_full[s], heads * nhx * kBox);
                            for (int k = 0; k < heads; ++k)
                                for (int h = 0; h < nhx; ++h)
                                    tma_load_3d(to + h * xhalf + k * kBox, &g.x, &x_full[s], 64 * h, (int)(w.h * p.gx) + 2 * a + k, row);
                            ++xt;
                        }
                    }
                }
            }
            if (!ok) {  // let the copies under way land before the CTA leaves
                for (uint32_t q = xt > XST ? xt - XST : 0; q < xt; ++q) mbar_wait(&x_full[q % XST], (q / XST) & 1, tc::kTimeout);
                for (uint32_t q = yi > YST ? yi - YST : 0; q < yi; ++q) mbar_wait(&yz_full[q % YST], (q / YST) & 1, tc::kTimeout);
            }
        }
        __syncwarp();
    } else if (warp == 13) {
        if (lane == 0) {
            const uint32_t id_s = idesc_bf16(128, 64, false, false), id_o = idesc_bf16(128, nz, false, true);
            uint32_t it = 0, xt = 0, yi = 0, ci = 0;
            int pending = -1, pending_y = 0, pending_x = 0;
            bool pending_last = false, ok = true;
            // O += P Z of the item before
            auto values = [&]() -> bool {
                const int s = pending & 1, ys = pending_y % YST;
                if (!wait(&p_full[s], (pending >> 1) & 1, 102) || !wait(&zz_full[ys], (pending_y / YST) & 1, 103)) return false;
                tc_fence_after();
                const uint64_t b = mndesc(base + SM::YZ + (ys * 4 + 2) * kBox, kBox);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma_bf16_ts(tO + (pending_x & 1) * 128, tS + s * 64 + j * 8, b + ((j * 2048) >> 4), id_o, 1u);
                mma_commit(&pv_done[s]);
                if (pending_last) mma_commit(&yz_free[ys]);
                pending = -1;
                return true;
            };
            while (ok && walk.next(p.seqs, w.b, &t)) {
                const uint32_t y0 = yi;
                for (int a = 0; a < ntx && ok; ++a) {
                    for (int gh = 0; gh < p.gy && ok; ++gh, ++it) {
                        const int s = it & 1, xs = xt % XST;
                        const uint32_t y = y0 + gh;
                        const int ys = y % YST;
                        if (gh == 0 && !wait(&x_full[xs], (xt / XST) & 1, 104)) { ok = false; break; }
                        if (a == 0 && !wait(&yz_full[ys], (y / YST) & 1, 105)) { ok = false; break; }
                        if (it >= 2 && !wait(&pv_done[s], ((it >> 1) & 1) ^ 1, 106)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t xa = base + SM::X + xs * XB * kBox, ya = base + SM::YZ + ys * 4 * kBox;
                        for (int k = 0; k < kx; ++k) {
                            const uint32_t in = (k & 3) * 32;
                            mma_bf16(tS + s * 64, kdesc(xa + (k >> 2) * xhalf + in), kdesc(ya + (k >> 2) * kBox + in), id_s, k > 0);
                        }
                        mma_commit(&s_full[s]);
                        // what does not wait for the state of a new tile goes first
                        if (pending >= 0 && a == 0 && gh == 0 && !values()) { ok = false; break; }
                        if (gh == 0) {
                            if (xt >= 2 && !wait(&o_free[xt & 1], ((xt >> 1) & 1) ^ 1, 107)) { ok = false; break; }
                            if (a == 0 && !wait(st_full, ci & 1, 108)) { ok = false; break; }
                            tc_fence_after();
                            for (int k = 0; k < kx; ++k)
                                mma_bf16(tO + (xt & 1) * 128, kdesc(xa + (k >> 2) * xhalf + (k & 3) * 32),
                                         mndesc(base + SM::ST + k * 2048, 2 * kBox), id_o, k > 0);
                            mma_commit(&xs_full[xt & 1]);
                            if (a == ntx - 1) mma_commit(xs_done);
                        }
                        if (pending >= 0 && !values()) { ok = false; break; }
                        pending = (int)it;
                        pending_y = (int)y;
                        pending_x = (int)xt;
                        pending_last = a == ntx - 1;
                        if (gh == p.gy - 1) ++xt;
                    }
                }
                yi += p.gy;
                ++ci;
            }
            if (ok && pending >= 0) ok = values();
            if (!ok) {  // every MMA that was issued ends before the CTA leaves: they read shared memory
                mma_commit(drained);
                mbar_wait(drained, 0, tc::kTimeout);
            }
        }
        __syncwarp();
    } else if (warp == 14) {
        if (lane == 0) {
            const uint32_t id_h = idesc_bf16(128, nz, true, true);
            uint32_t yi = 0;
            bool ok = true;
            while (ok && walk.next(p.seqs, w.b, &t)) {
                for (int gh = 0; gh < p.gy; ++gh, ++yi) {
                    if (!wait(kt_full, yi & 1, 109)) { ok = false; break; }
                    tc_fence_after();
                    state_mmas(tH, base + SM::KT, base + SM::YZ + ((yi % YST) * 4 + 2) * kBox, id_h, false);
                    mma_commit(h_done);
                    mma_commit(&yz_free[yi % YST]);
                }
            }
            if (!ok && yi > 0) mbar_wait(h_done, (yi - 1) & 1, tc::kTimeout);
        }
        __syncwarp();
    } else if (warp >= 8) {
        // the state: row `row` of S
        const int row = tid - 256;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int64_t size = (int64_t)p.dx * p.dz;
        const int64_t step = p.transposed ? p.dx : 1, at = p.transposed ? row : (int64_t)row * p.dz;
        uint32_t yi = 0, ci = 0;
        bool ok = true, was_last = false;
        int64_t was_seq = 0;
        grid_dep_wait();
        // the state behind a sequence's last tile
        auto leave = [&](int64_t seq) {
            if (p.fin == nullptr) return;
            float* to = p.fin + (seq * p.Hkv + w.h) * size;
            for (int c = 0; c < p.dz; c += 32) {
                float v[32];
                tmem_ld32(tH + lanes + c, v);
                tmem_wait_ld();
                if (row < p.dx)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c + i < p.dz) to[at + (c + i) * step] = v[i];
            }
        };
        while (ok && walk.next(p.seqs, w.b, &t)) {
            if (ci > 0) {
                if (!wait.all(h_done, (yi - 1) & 1, 110) || !wait.all(xs_done, (ci - 1) & 1, 111)) { ok = false; break; }
                tc_fence_after();
                if (was_last) leave(was_seq);
            }
            const float keep = pw[t.n];
            const bool from_memory = t.first || ci == 0;
            const float* from = !from_memory ? nullptr
                                : t.first    ? (p.init == nullptr ? nullptr : p.init + (t.seq * p.Hkv + w.h) * size)
                                             : p.recs + (w.unit * p.nseg + w.seg) * size;
            for (int c = 0; c < nz; c += 32) {
                float v[32];
                if (from_memory) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = from != nullptr && row < p.dx && c + i < p.dz ? from[at + (c + i) * step] : 0.0f;
                } else {
                    tmem_ld32(tH + lanes + c, v);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int col = c + 8 * i;
                    st_shared_v4(base + SM::ST + (col >> 6) * 2 * kBox + sw128(row, (col & 63) >> 3), pack_bf16(v[8 * i], v[8 * i + 1]),
                                 pack_bf16(v[8 * i + 2], v[8 * i + 3]), pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= keep;
                tmem_st32(tH + lanes + c, v);
            }
            tmem_wait_st();
            fence_async_smem();
            tc_fence_before();
            mbar_arrive(st_full);
            for (int gh = 0; gh < p.gy; ++gh, ++yi) {
                const int ys = yi % YST;
                if (!wait.all(&yz_full[ys], (yi / YST) & 1, 112)) { ok = false; break; }
                if (gh > 0 && !wait.all(h_done, (yi - 1) & 1, 113)) { ok = false; break; }
                const int tok = row & 63, far = rev ? tok + 1 : t.n - 1 - tok;
                const uint32_t ya = base + SM::YZ + ys * 4 * kBox;
                scale_rows(ya, ya + 2 * kBox, base + SM::KT, t.n, tok < t.n ? pws[far] : 0.0f, row);
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(&zz_full[ys]);
                mbar_arrive(kt_full);
            }
            was_last = t.last;
            was_seq = t.seq;
            ++ci;
        }
        if (ok && ci > 0 && was_last && p.fin != nullptr) {
            if (wait.all(h_done, (yi - 1) & 1, 114)) {
                tc_fence_after();
                leave(was_seq);
            }
        }
    } else {
        // weights of pairs, the state part's scale, outputs: row `r` of the tile of x heads
        const int quad = warp & 3, half = warp >> 2;
        const int r = 32 * quad + lane, i = r & 63, hs = r >> 6;  // token in the tile, head of the two
        const uint32_t lanes = (uint32_t)(32 * quad) << 16;
        const int ib = quad & 1;                     // the row's block of 32 tokens; the columns' is `half`
        const bool z_on = 64 * half < p.dz;
        const int zc = z_on ? (nz - 64 * half < 64 ? nz - 64 * half : 64) : 0;  // output columns of this warp
        uint32_t it = 0, xt = 0, pairs = 0;
        bool ok = true;
        // the tile whose outputs are still to be stored
        int held = -1, held_x = 0, held_n = 0, held_heads = 0, held_a = 0;
        int64_t held_t0 = 0;
        auto store = [&]() -> bool {
            if (!wait.all(&pv_done[held & 1], (held >> 1) & 1, 115)) return false;
            tc_fence_after();
            const uint32_t stage = base + SM::X + (held_x % XST) * XB * kBox + half * xhalf;
            const bool live = hs < held_heads && z_on;  // one answer for a warp
            if (live) {
                for (int c = 0; c < zc; c += 32) {
                    float v[32];
                    tmem_ld32(tO + (held_x & 1) * 128 + lanes + 64 * half + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] *= p.out_scale;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        st_shared_v4(stage + sw128(r, (c >> 3) + k), pack_bf16(v[8 * k], v[8 * k + 1]), pack_bf16(v[8 * k + 2], v[8 * k + 3]),
                                     pack_bf16(v[8 * k + 4], v[8 * k + 5]), pack_bf16(v[8 * k + 6], v[8 * k + 7]));
                }
            }
            tc_fence_before();
            mbar_arrive(&o_free[held_x & 1]);
            __syncwarp();
            if (live) {
                const int chunk = lane & 7;
                const int64_t head = w.h * p.gx + 2 * held_a + hs;
                __nv_bfloat16* out = (__nv_bfloat16*)p.out + (w.b * p.seqs.L + held_t0) * p.ldout + head * p.dz + 64 * half + 8 * chunk;
                if (64 * half + 8 * chunk < p.dz) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int row = 4 * k + (lane >> 3), tok = (32 * quad + row) & 63;
                        uint32_t v[4];
                        ld_shared_v4(stage + sw128(32 * quad + row, chunk), v[0], v[1], v[2], v[3]);
                        if (tok < held_n) *reinterpret_cast<uint4*>(out + tok * p.ldout) = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
            fence_async_smem();
            mbar_arrive(&x_free[held_x % XST]);
            held = -1;
            return true;
        };
        while (ok && walk.next(p.seqs, w.b, &t)) {
            for (int a = 0; a < ntx && ok; ++a) {
                const int heads = p.gx - 2 * a < 2 ? 1 : 2;
                const bool live = hs < heads;
                for (int gh = 0; gh < p.gy && ok; ++gh, ++it) {
                    const int s = it & 1;
                    if (!wait.all(&s_full[s], (it >> 1) & 1, 116)) { ok = false; break; }
                    tc_fence_after();
                    if (live) {
                        const uint32_t to = tS + s * 64 + lanes + half * 16;
                        uint32_t o[16];
                        if (rev ? ib > half : ib < half) {
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = 0;
                        } else {
                            float v[32];
                            tmem_ld32(tS + s * 64 + lanes + half * 32, v);
                            tmem_wait_ld();
                            if (ib != half) {
                                // |i - j| as steps to the border between the blocks and beyond it
                                const float far = pw[rev ? 32 - (i & 31) : (i & 31) + 1];
#pragma unroll
                                for (int k = 0; k < 32; ++k) v[k] *= far * pws[rev ? k : 31 - k];
                                if (rev && t.n < kTile) {
#pragma unroll
                                    for (int k = 0; k < 32; ++k) v[k] = 32 * half + k < t.n ? v[k] : 0.0f;
                                }
                            } else {
                                const int d0 = i & 31;
#pragma unroll
                                for (int k = 0; k < 32; ++k) {
                                    const int d = rev ? k - d0 : d0 - k;
                                    v[k] = d >= 0 && 32 * half + k < t.n ? v[k] * pws[d & 63] : 0.0f;
                                }
                            }
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
                        }
                        // both halves of a row's scores are read before its weights overwrite them
                        tc_fence_before();
                        mbar_arrive(&pair[quad]);
                        if (!wait.all(&pair[quad], pairs & 1, 118)) { ok = false; break; }
                        tc_fence_after();
                        ++pairs;
                        tmem_st16(to, o);
                    }
                    if (gh == 0) {
                        if (!wait.all(&xs_full[xt & 1], (xt >> 1) & 1, 117)) { ok = false; break; }
                        tc_fence_after();
                        if (live && z_on) {
                            const float f = i < t.n ? pw[rev ? t.n - 1 - i : i + 1] : 0.0f;
                            for (int c = 0; c < zc; c += 32) {
                                float v[32];
                                tmem_ld32(tO + (xt & 1) * 128 + lanes + 64 * half + c, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 32; ++k) v[k] *= f;
                                tmem_st32(tO + (xt & 1) * 128 + lanes + 64 * half + c, v);
                            }
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(&p_full[s]);
                    if (held >= 0 && !store()) { ok = false; break; }
                    if (gh == p.gy - 1) {
                        held = (int)it;
                        held_x = (int)xt;
                        held_n = t.n;
                        held_heads = heads;
                        held_a = a;
                        held_t0 = t.t0;
                        ++xt;
                    }
                }
            }
        }
        if (ok && held >= 0) store();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tb, 512);
    }
}

// ------------------------------------------------------------------------- segments' end states

// A segment's own contribution to the state that leaves it, from all tokens that reach it, each with its
// whole power of the decay: S stays in TMEM and nothing is scaled on the way.  Two groups of four warps make
// Y~ in turn, warp 8 copies, warp 9 issues the MMAs.
constexpr int kEndsThreads = 320, kEndsStages = 4;
struct EndsSmem {
    static constexpr uint32_t YZ = 0;
    static constexpr uint32_t KT = kEndsStages * 4 * kBox;
    static constexpr uint32_t BARS = KT + 2 * 4 * kBox;
    static constexpr uint32_t BYTES = BARS + 256 + 1024;
    static_assert(BYTES <= 227 * 1024, "shared memory of a CTA");
};

template <bool rev>
__global__ void __launch_bounds__(kEndsThreads, 1) decay_tc_ends_kernel(const __grid_constant__ TcArgs g, float* recs) {
    extern __shared__ uint8_t smem_raw[];
    const DecayPass& p = g.p;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (base - smem_u32(smem_raw));
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + EndsSmem::BARS);
    uint64_t *yz_full = bar, *yz_free = bar + 4, *kt_full = bar + 8, *kt_free = bar + 10, *done = bar + 12;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 13);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Seg w = seg_of(p);
    check_offsets(p.seqs, p.header);
    const float l2 = log2_decay(p.log_decay, w.h);
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&yz_full[i], 1);
            mbar_init(&yz_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&kt_full[i], 128);
            mbar_init(&kt_free[i], 1);
        }
        mbar_init(done, 1);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(tmem_slot, 128);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dep_launch();
    const uint32_t tb = *tmem_slot;
    const Waiter wait{abort, p.header};
    const int nhx = (p.dx + 63) / 64, nhz = (p.dz + 63) / 64, nz = (p.dz + 15) / 16 * 16;
    const Reach r = reach(p.seqs, w.b, w.lo, w.hi, rev);
    const uint32_t items = (uint32_t)((r.to - r.from + kTile - 1) / kTile) * p.gy;

    if (warp == 8) {
        if (lane == 0) {
            prefetch_tmap(&g.y);
            prefetch_tmap(&g.z);
            uint32_t it = 0;
            bool ok = true;
            for (int64_t t0 = r.from; t0 < r.to && ok; t0 += kTile) {
                const int row = (int)(w.b * p.seqs.L + t0);
                for (int gh = 0; gh < p.gy; ++gh, ++it) {
                    const int s = it % kEndsStages;
                    if (it >= kEndsStages && !wait(&yz_free[s], ((it / kEndsStages) & 1) ^ 1, 120)) { ok = false; break; }
                    uint8_t* to = sm + EndsSmem::YZ + s * 4 * kBox;
                    mbar_arrive_expect_tx(&yz_full[s], (nhx + nhz) * kBox);
                    const int head = (int)(w.h * p.gy + gh);
                    for (int h = 0; h < nhx; ++h) tma_load_3d(to + h * kBox, &g.y, &yz_full[s], 64 * h, head, row);
                    for (int h = 0; h < nhz; ++h) tma_load_3d(to + (2 + h) * kBox, &g.z, &yz_full[s], 64 * h, head, row);
                }
            }
            if (!ok)
                for (uint32_t q = it > kEndsStages ? it - kEndsStages : 0; q < it; ++q)
                    mbar_wait(&yz_full[q % kEndsStages], (q / kEndsStages) & 1, tc::kTimeout);
        }
        __syncwarp();
    } else if (warp == 9) {
        if (lane == 0) {
            const uint32_t id_h = idesc_bf16(128, nz, true, true);
            uint32_t it = 0;
            for (; it < items; ++it) {
                const int k = it & 1;
                if (!wait(&kt_full[k], (it >> 1) & 1, 121)) break;
                tc_fence_after();
                state_mmas(tb, base + EndsSmem::KT + k * 4 * kBox, base + EndsSmem::YZ + ((it % kEndsStages) * 4 + 2) * kBox, id_h, it == 0);
                mma_commit(&kt_free[k]);
                mma_commit(&yz_free[it % kEndsStages]);
            }
            mma_commit(done);
            if (it < items) mbar_wait(done, 0, tc::kTimeout);
        }
        __syncwarp();
    } else {
        const int group = warp >> 2, in = tid & 127, tok = in & 63;
        uint32_t it = 0;
        bool ok = true;
        for (int64_t t0 = r.from; t0 < r.to && ok; t0 += kTile) {
            const int n = (int)min64(kTile, r.to - t0);
            for (int gh = 0; gh < p.gy; ++gh, ++it) {
                if ((int)(it & 1) != group) continue;
                const int s = it % kEndsStages;
                if (!wait.all(&yz_full[s], (it / kEndsStages) & 1, 122)) { ok = false; break; }
                if (it >= 2 && !wait.all(&kt_free[group], ((it >> 1) & 1) ^ 1, 123)) { ok = false; break; }
                const float f = tok < n ? power(l2, rev ? t0 + tok - r.from + 1 : r.to - 1 - t0 - tok) * p.in_scale : 0.0f;
                const uint32_t ya = base + EndsSmem::YZ + s * 4 * kBox;
                scale_rows(ya, ya + 2 * kBox, base + EndsSmem::KT + group * 4 * kBox, n, f, in);
                fence_async_smem();
                mbar_arrive(&kt_full[group]);
            }
        }
        if (ok && wait.all(done, 0, 124)) {
            tc_fence_after();
            const int row = 32 * (warp & 3) + lane;
            const int64_t size = (int64_t)p.dx * p.dz;
            float* to = recs + (w.unit * p.nseg + w.seg) * size + (int64_t)row * p.dz;
            const float* from = r.whole && p.init != nullptr ? p.init + (r.seq * p.Hkv + w.h) * size + (int64_t)row * p.dz : nullptr;
            const float f = from != nullptr ? power(l2, r.to - r.from) : 0.0f;
            for (int c = 64 * group; c < 64 * group + 64 && c < p.dz; c += 32) {
                float v[32];
                tmem_ld32(tb + ((uint32_t)(32 * (warp & 3)) << 16) + c, v);
                tmem_wait_ld();
                if (row < p.dx) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        if (c + k >= p.dz) continue;
                        float4 u = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                        if (from != nullptr) {
                            const float4 i = *reinterpret_cast<const float4*>(from + c + k);
                            u.x = fmaf(f, i.x, u.x), u.y = fmaf(f, i.y, u.y), u.z = fmaf(f, i.z, u.z), u.w = fmaf(f, i.w, u.w);
                        }
                        *reinterpret_cast<float4*>(to + c + k) = u;
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tb, 128);
    }
}

// [rows, heads, width] of a tensor with token distance ld, boxes of 64 rows x 64 columns of one head.
bool map_of(CUtensorMap* m, const void* ptr, int64_t rows, int64_t heads, int64_t width, int64_t ld) {
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, 1, 64};
    return tc::make_map(m, ptr, 3, dims, strides, box);
}

bool args_of(const DecayPass& p, TcArgs* a) {
    a->p = p;
    const int64_t rows = p.units / p.Hkv * p.seqs.L;
    return map_of(&a->x, p.x, rows, p.Hkv * p.gx, p.dx, p.ldx) && map_of(&a->y, p.y, rows, p.Hkv * p.gy, p.dx, p.ldy) &&
           map_of(&a->z, p.z, rows, p.Hkv * p.gy, p.dz, p.ldz);
}

template <typename SM>
cudaError_t go(const TcArgs& a, cudaStream_t s) {
    const auto kernel = decay_tc_kernel<SM>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SM::BYTES);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.p.units * a.p.nseg));
    if (a.p.nseg > 1) {  // its set-up overlaps the join of the segments
        e = launch_dependent(kernel, grid, dim3(kThreads), SM::BYTES, s, a);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    kernel<<<grid, kThreads, SM::BYTES, s>>>(a);
    return cudaGetLastError();
}

template <bool rev>
cudaError_t go_ends(const TcArgs& a, float* recs, cudaStream_t s) {
    const auto kernel = decay_tc_ends_kernel<rev>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)EndsSmem::BYTES);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(a.p.units * a.p.nseg), kEndsThreads, EndsSmem::BYTES, s>>>(a, recs);
    return cudaGetLastError();
}

}  // namespace

// bf16 of up to 128 values a head, in rows the copies can address.
bool decay_uses_tc(const DecayArgs& a) {
    const int64_t rows = a.ldq | a.ldk | a.ldv | a.ldo | a.lddq | a.lddk | a.lddv;
    return a.dtype == LIZARD_BF16 && a.dk <= 128 && a.dv <= 128 && a.dk % 8 == 0 && a.dv % 8 == 0 && rows % 8 == 0 &&
           a.B * a.seqs.L < 0x7fff0000 && a.Hq < 0x7fff0000;
}

cudaError_t decay_tc_ends(const DecayPass& p, float* recs, cudaStream_t s) {
    TcArgs a;
    if (!args_of(p, &a)) return cudaErrorInvalidValue;
    return p.rev ? go_ends<true>(a, recs, s) : go_ends<false>(a, recs, s);
}

cudaError_t decay_tc_pass(const DecayPass& p, cudaStream_t s) {
    TcArgs a;
    if (!args_of(p, &a)) return cudaErrorInvalidValue;
    return p.rev ? go<Backwards>(a, s) : go<Forwards>(a, s);
}

}  // namespace lz
