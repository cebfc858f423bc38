// Linear attention with a decay for each head on the tensor cores (tcgen05, TMEM and TMA, sm_103a): bf16,
// keys and values of up to 128 values.  Here are the passes forwards in time, of the outputs and of dq, and the
// segments' end states; dk and dv have a kernel of their own.
//
// A CTA walks a segment of one state head in chunks.  128 rows of x make an item with 64 of y and z: two query
// heads of a chunk of 64 tokens, or one head of a chunk of 128 tokens where a state has one head of x (so that the
// MMAs' 128 rows are used), with 64 of the chunk's tokens of y and z in turn.  With S the state in front of the chunk
//   P = (X Y^T) (.) e^(l (i - j)), masked to the tokens up to i,   O = e^(l (i+1)) X S + P Z
// and a chunk of n tokens moves the state on:  S' = e^(l n) S + Y~^T Z,  Y~[j] = e^(l (n-1-j)) Y[j].
//
// The decay of a pair is e^(l (i-r)) e^(l (r-j)) with r in the middle of the chunk: the second factor is a
// constant for each column of P, the first one scales the finished row of O, and the operand copy of S takes
// e^(l (r+1)).  Where all of these lie within 2^32 of 1, as they do while a token keeps 0.71 of the state (a
// half, in chunks of 64), nothing else is needed.  Heads that decay faster (or grow that much) take each pair's
// power of the difference and scale X S before P Z is added.
//
// Roundings: P and the operand copy of S are bf16 (a relative 2^-8 of the terms, as the output's own).  S itself
// stays in fp32, and Y~ goes in as two bf16 parts (2^-16), or three (2^-24) where S leaves the call: what is rounded
// there would stay for the rest of the sequence.
//
// Warps: 0-7 the pairs' weights and the outputs (a thread holds one row's 32 of 64 pairs and 64 of 128 output
// columns); 8-15 the state (half a row of S to a thread; Y~); 16 the copies; 17 the MMAs of the scores, 18 of
// the state, 19 of the outputs.  TMEM: P and its scores two of 64 columns, O 128, S 128, a chunk's part of S 128.
//
// Bound by the chain of a chunk (state out, X S, P Z, state on) and by what its warps issue in it: with 32 query heads
// on 8 of 128 the walk of 8192 tokens takes 38 us, where its bytes take 25, and that of 65536 takes 220 us, where they
// take 201.  The loops over a product's steps stay rolled: unrolled by four the longer one takes 39 us more (the code of
// seven roles shares the SM's instruction cache), and the waits' slow path is one function for the same reason.
#include "decay_tc.cuh"

namespace lz {
namespace {

struct TcArgs {
    CUtensorMap x, y, z, out;
    DecayPass p;
};

// Shared memory: XST stages of x, rows of the output on their way out, YST of y and z, Y~, the state's operand copy.
template <int XST_, int YST_>
struct Layout {
    static constexpr int XST = XST_, YST = YST_;
    static constexpr uint32_t X = 0;
    static constexpr uint32_t OUT = XST * 4 * kBox;
    static constexpr uint32_t YZ = OUT + 4 * kBox;
    static constexpr uint32_t KT = YZ + YST * 4 * kBox;  // two parts of Y~ (a third takes the first's place)
    static constexpr uint32_t ST = KT + 4 * kBox;
    static constexpr uint32_t TABLE = ST + 4 * kBox;     // powers 0 .. 128, and the columns' factors
    static constexpr uint32_t BARS = TABLE + (132 + 128) * 4;
    static constexpr uint32_t BYTES = BARS + 376 + 4 * kMostNoted + 1024;
    static_assert(BYTES <= 227 * 1024 && kByTokensBytes <= TABLE, "shared memory of a CTA");
};
// Several tiles of x for each of y and z, or one.  Then one stage of x is enough (its last reader is done long before
// the chunk is) and leaves room for a third of y and z, whose copies otherwise wait for the chunk before (16 heads of
// 64 and 128, 16384 tokens: 391 -> 371 us forwards and backwards).
using Wide = Layout<2, 2>;
using Even = Layout<1, 3>;

// three: parts of Y~ (with a stage of x less and all three at once the walk of 65536 tokens takes 36 us more).
template <typename SM, bool three>
__global__ void __launch_bounds__(kThreads, 1) decay_tc_kernel(const __grid_constant__ TcArgs g) {
    constexpr int XST = SM::XST, YST = SM::YST;
    extern __shared__ uint8_t smem_raw[];
    const DecayPass& p = g.p;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (base - smem_u32(smem_raw));
    float* pw = reinterpret_cast<float*>(sm + SM::TABLE);  // powers of the decay
    float* col = pw + 132;                                 // factors of the columns of P
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + SM::BARS);
    uint64_t *x_full = bar, *x_free = bar + 3, *yz_full = bar + 6, *yz_free = bar + 10, *zz_full = bar + 14, *s_full = bar + 18,
             *p_full = bar + 20, *xs_full = bar + 22, *pv_done = bar + 24, *o_free = bar + 26, *kt_full = bar + 28,
             *h_done = bar + 29, *st_full = bar + 30, *xs_done = bar + 31, *drained = bar + 32,
             *first_free = bar + 35, *third_full = bar + 36, *agreed = bar + 37;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 38);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    Seg* seg = reinterpret_cast<Seg*>(bar + 41);  // (for walk_by_tokens: in registers till then it makes the roles spill)
    const Notes notes{abort + 1, abort + 2, abort + 3, abort + 17, agreed};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool leader = lane == 0;
    const Seg w = seg_of<false>(p);
    check_offsets(p.seqs, p.header);
    const bool tall = p.gx == 1;                 // a tile of x: 128 tokens of a head, or 64 of two
    const int chunk = tall ? 128 : 64, mid = chunk / 2 - 1;
    const float l2 = log2_decay(p.log_decay, w.h);
    const bool slow = fabsf(l2) * (float)chunk <= 64.0f;  // factors of rows and columns (see above)
    for (int i = tid; i < 129; i += kThreads) {
        pw[i] = power(l2, i);
        if (i < 128) col[i] = power(l2, mid - i);
    }
    if (tid == 0) {
        for (int i = 0; i < XST; ++i) {
            mbar_init(&x_full[i], 1);
            mbar_init(&x_free[i], 2);  // scores and X S
        }
        for (int i = 0; i < YST; ++i) {
            mbar_init(&yz_full[i], 1);
            mbar_init(&yz_free[i], 2);
            mbar_init(&zz_full[i], 32 * kStateWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 32 * kMathWarps);
            mbar_init(&xs_full[i], 1);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(o_free, 32 * kMathWarps);
        mbar_init(kt_full, 32 * kStateWarps);
        mbar_init(h_done, 1);
        mbar_init(st_full, 32 * kStateWarps);
        mbar_init(xs_done, 1);
        mbar_init(first_free, 1);
        mbar_init(third_full, 32 * kStateWarps);
        mbar_init(agreed, 32 * kStateWarps);
        for (int i = 0; i < 3; ++i) mbar_init(&drained[i], 1);
        *abort = 0;
        *seg = w;
        *notes.found = 0;
        *notes.count = 0;
        fence_mbar_init();
    }
    if (warp == 17) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = *tmem_slot;
    const uint32_t tS = tb, tO = tb + 128, tD = tb + 256, tH = tb + 384;
    const Waiter wait{abort, p.header};
    const int nhx = (p.dx + 63) / 64, nhz = (p.dz + 63) / 64;
    const int kx = (p.dx + 15) / 16;                 // K steps over dx
    const int nz = (p.dz + 15) / 16 * 16;            // N over dz
    const int ntx = (p.gx + 1) / 2;                  // tiles of x heads

    Walk walk(p.seqs, w.b, w.lo, w.hi, false, chunk);
    Tile t;

    if (warp == 16) {
        if (lane == 0) {
            prefetch_tmap(&g.x);
            prefetch_tmap(&g.y);
            prefetch_tmap(&g.z);
            uint32_t xt = 0, yi = 0;
            bool ok = true;
            while (ok && walk.next(p.seqs, w.b, &t)) {
                const int row = (int)(w.b * p.seqs.L + t.t0);
                const int ny = t.n > 64 ? 2 : 1;
                for (int a = 0; a < ntx && ok; ++a) {
                    for (int q = 0; q < ny && ok; ++q) {
                        if (a == 0) {
                            const int s = yi % YST, head = (int)w.h, at = row + 64 * q;
                            if (yi >= YST && !wait(&yz_free[s], ((yi / YST) & 1) ^ 1, 100)) {
                                ok = false;
                                break;
                            }
                            uint8_t* to = sm + SM::YZ + s * 4 * kBox;
                            mbar_arrive_expect_tx(&yz_full[s], (nhx + nhz) * kBox);
                            for (int h = 0; h < nhx; ++h) tma_load_3d(to + h * kBox, &g.y, &yz_full[s], 64 * h, head, at);
                            for (int h = 0; h < nhz; ++h) tma_load_3d(to + (2 + h) * kBox, &g.z, &yz_full[s], 64 * h, head, at);
                            ++yi;
                        }
                        if (q == 0) {
                            const int s = xt % XST, parts = tall ? ny : p.gx - 2 * a < 2 ? 1 : 2;
                            if (xt >= XST && !wait(&x_free[s], ((xt / XST) & 1) ^ 1, 101)) {
                                ok = false;
                                break;
                            }
                            uint8_t* to = sm + SM::X + s * 4 * kBox;
                            mbar_arrive_expect_tx(&x_full[s], parts * nhx * kBox);
                            for (int k = 0; k < parts; ++k)
                                for (int h = 0; h < nhx; ++h)
                                    tma_load_3d(to + h * kHalf + k * kBox, &g.x, &x_full[s], 64 * h, (int)(w.h * p.gx) + (tall ? 0 : 2 * a + k),
                                                row + (tall ? 64 * k : 0));
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
    } else if (warp == 17) {
        // scores: X Y^T
        const uint32_t id_s = idesc_bf16(128, 64, false, false);
        uint32_t it = 0, xt = 0, yi = 0;
        bool ok = true;
        while (ok && walk.next(p.seqs, w.b, &t)) {
            const int ny = t.n > 64 ? 2 : 1;
            for (int a = 0; a < ntx && ok; ++a) {
                for (int q = 0; q < ny && ok; ++q, ++it) {
                    const int s = it & 1, xs = xt % XST;
                    const uint32_t y = yi + q;
                    const int ys = y % YST;
                    if (q == 0 && !wait.all(&x_full[xs], (xt / XST) & 1, 104)) { ok = false; break; }
                    if (a == 0 && !wait.all(&yz_full[ys], (y / YST) & 1, 105)) { ok = false; break; }
                    if (it >= 2 && !wait.all(&pv_done[s], ((it >> 1) & 1) ^ 1, 106)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t xa = uniform(base + SM::X + xs * 4 * kBox), ya = uniform(base + SM::YZ + ys * 4 * kBox), to = uniform(tS + s * 64);
#pragma unroll 1
                    for (int k = 0; k < kx; ++k)
                        mma_bf16_one(leader, to, kdesc(xa + (k >> 2) * kHalf + (k & 3) * 32), kdesc(ya + (k >> 2) * kBox + (k & 3) * 32), id_s, k > 0);
                    if (leader) {
                        mma_commit(&s_full[s]);
                        if (q == ny - 1) mma_commit(&x_free[xs]);
                    }
                    if (q == ny - 1) ++xt;
                }
            }
            yi += ny;
        }
        if (!ok) {  // every MMA that was issued ends before the CTA leaves: they read shared memory
            if (leader) mma_commit(&drained[0]);
            mbar_wait(&drained[0], 0, tc::kTimeout);
        }
    } else if (warp == 19) {
        // outputs: X S, and P Z after it in the same accumulator
        const uint32_t id_o = idesc_bf16(128, nz, false, true);
        uint32_t it = 0, xt = 0, yi = 0, ci = 0;
        bool ok = true;
        while (ok && walk.next(p.seqs, w.b, &t)) {
            const int ny = t.n > 64 ? 2 : 1;
            for (int a = 0; a < ntx && ok; ++a) {
                for (int q = 0; q < ny && ok; ++q, ++it) {
                    const int s = it & 1, xs = xt % XST;
                    const uint32_t y = yi + q;
                    const int ys = y % YST;
                    const uint32_t to = uniform(tO);
                    if (q == 0) {
                        if (!wait.all(&x_full[xs], (xt / XST) & 1, 107)) { ok = false; break; }
                        if (xt >= 1 && !wait.all(o_free, (xt & 1) ^ 1, 119)) { ok = false; break; }
                        if (a == 0 && !wait.all(st_full, ci & 1, 108)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t xa = uniform(base + SM::X + xs * 4 * kBox);
#pragma unroll 1
                        for (int k = 0; k < kx; ++k)
                            mma_bf16_one(leader, to, kdesc(xa + (k >> 2) * kHalf + (k & 3) * 32), mndesc(base + SM::ST + k * 2048, kHalf), id_o, k > 0);
                        if (leader) {
                            if (!slow) mma_commit(&xs_full[xt & 1]);
                            mma_commit(&x_free[xs]);
                            if (a == ntx - 1) mma_commit(xs_done);
                        }
                    }
                    if (!wait.all(&zz_full[ys], (y / YST) & 1, 103) || !wait.all(&p_full[s], (it >> 1) & 1, 102)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t za = uniform(base + SM::YZ + (ys * 4 + 2) * kBox), from = uniform(tS + s * 64);
                    // the weights of each 32 columns lie at the beginning of their scores
#pragma unroll 1
                    for (int j = 0; j < 4; ++j)
                        mma_bf16_ts_one(leader, to, from + (j >> 1) * 32 + (j & 1) * 8, mndesc(za + j * 2048, kBox), id_o, 1u);
                    if (leader) {
                        mma_commit(&pv_done[s]);
                        if (a == ntx - 1) mma_commit(&yz_free[ys]);
                    }
                    if (q == ny - 1) ++xt;
                }
            }
            yi += ny;
            ++ci;
        }
        if (!ok) {
            if (leader) mma_commit(&drained[1]);
            mbar_wait(&drained[1], 0, tc::kTimeout);
        }
    } else if (warp == 18) {
        const uint32_t id_h = idesc_bf16(128, nz, true, true);
        uint32_t yi = 0;
        bool ok = true;
        while (ok && walk.next(p.seqs, w.b, &t)) {
            const int ny = t.n > 64 ? 2 : 1;
            for (int q = 0; q < ny && ok; ++q, ++yi) {
                if (!wait.all(kt_full, yi & 1, 109)) { ok = false; break; }
                tc_fence_after();
                const uint32_t za = uniform(base + SM::YZ + ((yi % YST) * 4 + 2) * kBox);
                if (!three) state_mmas<1>(leader, tD, base + SM::KT, 2, za, kBox, id_h, q == 0);
                if (three) {
                    state_mmas<1>(leader, tD, base + SM::KT, 1, za, kBox, id_h, q == 0);
                    if (leader) mma_commit(first_free);
                    state_mmas<1>(leader, tD, base + SM::KT + 2 * kBox, 1, za, kBox, id_h, false);
                    if (!wait.all(third_full, yi & 1, 118)) { ok = false; break; }
                    tc_fence_after();
                    state_mmas<1>(leader, tD, base + SM::KT, 1, za, kBox, id_h, false);
                }
                if (leader) {
                    mma_commit(h_done);
                    mma_commit(&yz_free[yi % YST]);
                }
            }
        }
        if (!ok) {
            if (leader) mma_commit(&drained[2]);
            mbar_wait(&drained[2], 0, tc::kTimeout);
        }
    } else if (warp >= 8) {
        // the state: half a row of S to a thread
        const StateRow sr = state_row(p, tH, tD, tid - 32 * kMathWarps);
        float keep = 1.0f;  // of the chunk before
        uint32_t yi = 0, ci = 0;
        bool ok = true, was_last = false;
        int was_seq = 0, ends = 1;  // the sequence under way is the ends-th
        grid_dep_wait();
        while (ok && walk.next(p.seqs, w.b, &t)) {
            if (ci > 0) {
                if (!wait.all(h_done, (yi - 1) & 1, 110) || !wait.all(xs_done, (ci - 1) & 1, 111)) { ok = false; break; }
                tc_fence_after();
                if (was_last && may_leave(notes, wait, sr, nz, ends++, &ok)) leave_state(p, sr, w.h, was_seq, keep);
                if (!ok) break;
            }
            const bool fresh = t.first || ci == 0;
            if (fresh) begin_state(p, sr, w, t);
            if (!pass_state(sr, base + SM::ST, nz, slow ? pw[mid + 1] : 1.0f, fresh, keep)) *notes.found = ends;
            if (sr.in == 0) *notes.entered = max(walk.begin, walk.lo);
            keep = pw[t.n];
            fence_async_smem();
            tc_fence_before();
            mbar_arrive(st_full);
            const int ny = t.n > 64 ? 2 : 1;
            for (int q = 0; q < ny; ++q, ++yi) {
                const int ys = yi % YST, j0 = 64 * q, m = min(64, t.n - j0);
                if (!wait.all(&yz_full[ys], (yi / YST) & 1, 112)) { ok = false; break; }
                if (q > 0 && !wait.all(h_done, (yi - 1) & 1, 113)) { ok = false; break; }
                const int tok = sr.in & 63;
                const uint32_t ya = base + SM::YZ + ys * 4 * kBox;
                const float f = tok < m ? pw[t.n - 1 - j0 - tok] : 0.0f;
                if (m < 64) {
                    clear_rows<32 * kStateWarps>(ya + 2 * kBox, kBox, m, sr.in);
                    fence_async_smem();
                }
                mbar_arrive(&zz_full[ys]);
                scale_rows<false, 1>(ya, kBox, base + SM::KT, 2 * kx, m, f, sr.in);
                fence_async_smem();
                tc_fence_before();
                mbar_arrive(kt_full);
                if (three) {
                    if (!wait.all(first_free, yi & 1, 126)) { ok = false; break; }
                    third_of_rows(ya, kBox, base + SM::KT, 2 * kx, m, f, sr.in);
                    fence_async_smem();
                    tc_fence_before();
                    mbar_arrive(third_full);
                }
            }
            was_last = t.last;
            was_seq = t.seq;
            ++ci;
        }
        if (ok && ci > 0 && wait.all(h_done, (yi - 1) & 1, 114)) {
            tc_fence_after();
            if (may_leave(notes, wait, sr, nz, ends, &ok) && was_last) leave_state(p, sr, w.h, was_seq, keep);
        }
    } else {
        // weights of pairs and outputs: row `r` of the tile of x
        const int quad = warp & 3, half = warp >> 2;
        const int r = 32 * quad + lane, i = tall ? r : r & 63;  // token in the chunk
        const int tq = tall ? quad : quad & 1;                  // its block of 32 tokens
        const int slot = tall ? 0 : quad >> 1;                  // head of the two
        const uint32_t lanes = (uint32_t)(32 * quad) << 16;
        const bool z_on = 64 * half < p.dz;
        const float rowf = p.out_scale * (slow ? power(l2, i - mid) : 1.0f);
        const f2 rowf2 = pack(rowf, rowf);
        const uint32_t c0 = base + SM::TABLE + 132 * 4;
        // an item's weights; the outputs of a tile of x as soon as its products are done, since the next one's X S waits for
        // their place (65536 tokens: 284 us, 308 with the next item's weights before them)
        uint32_t it = 0, xt = 0;
        bool ok = true;
        while (ok && walk.next(p.seqs, w.b, &t)) {
            const int ny = t.n > 64 ? 2 : 1;
            for (int a = 0; a < ntx && ok; ++a, ++xt) {
                const bool live = tall ? 32 * tq < t.n : 2 * a + slot < p.gx;
                const int head = (int)(w.h * p.gx) + (tall ? 0 : 2 * a + slot);
                for (int q = 0; q < ny; ++q, ++it) {
                    const int s = it & 1, cb = 2 * q + half;  // block of the columns
                    if (!wait.all(&s_full[s], (it >> 1) & 1, 116)) { ok = false; break; }
                    tc_fence_after();
                    if (live) {
                        const uint32_t at = tS + s * 64 + lanes + half * 32;
#pragma unroll 1
                        for (int c = 0; c < 32; c += 16) {
                            uint32_t o[8];
                            if (tq < cb) {
#pragma unroll
                                for (int k = 0; k < 8; ++k) o[k] = 0;
                            } else {
                                float v[16];
                                tmem_get16(at + c, v);
                                if (slow) {
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        uint32_t f[4];
                                        ld_shared_v4(c0 + (32 * cb + c + 4 * k) * 4, f[0], f[1], f[2], f[3]);
#pragma unroll
                                        for (int m = 0; m < 2; ++m)
                                            unpack(mul2(pack(v[4 * k + 2 * m], v[4 * k + 2 * m + 1]), pack(__uint_as_float(f[2 * m]), __uint_as_float(f[2 * m + 1]))),
                                                   v[4 * k + 2 * m], v[4 * k + 2 * m + 1]);
                                    }
                                } else {
#pragma unroll
                                    for (int k = 0; k < 16; ++k) {
                                        const int d = i - 32 * cb - c - k;
                                        v[k] *= pw[d < 0 ? 0 : d];
                                    }
                                }
                                if (tq == cb) {  // tokens behind this one are left out whatever they hold
                                    const int last = lane - c;
#pragma unroll
                                    for (int k = 0; k < 16; ++k) v[k] = k <= last ? v[k] : 0.0f;
                                }
#pragma unroll
                                for (int k = 0; k < 8; ++k) o[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
                            }
                            tmem_st8(at + c / 2, o);  // over scores that this thread has read
                        }
                    }
                    if (!slow && q == 0) {  // e^(l (i+1)) X S
                        if (!wait.all(&xs_full[xt & 1], (xt >> 1) & 1, 117)) { ok = false; break; }
                        tc_fence_after();
                        if (live && z_on) {
                            const float f = i < t.n ? pw[i + 1] : 0.0f;
#pragma unroll 1
                            for (int c = 0; c < 64; c += 16) {
                                float v[16];
                                tmem_get16(tO + lanes + 64 * half + c, v);
#pragma unroll
                                for (int k = 0; k < 16; ++k) v[k] *= f;
                                tmem_st16(tO + lanes + 64 * half + c, reinterpret_cast<const uint32_t*>(v));
                            }
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(&p_full[s]);
                }
                if (!ok) break;
                const uint32_t last = it - 1;  // of the tile's items
                if (!wait.all(&pv_done[last & 1], (last >> 1) & 1, 115)) { ok = false; break; }
                tc_fence_after();
                const uint32_t stage = base + SM::OUT + half * kHalf + quad * 4096;
                const bool out_live = live && z_on;  // one answer for a warp
                if (out_live) {
                    if (lane == 0) bulk_wait_read();  // the rows before have left
                    __syncwarp();
#pragma unroll 1
                    for (int c = 0; c < 64; c += 16) {
                        float v[16];
                        tmem_get16(tO + lanes + 64 * half + c, v);
#pragma unroll
                        for (int k = 0; k < 2; ++k) st_scaled8(stage + sw128(lane, (c >> 3) + k), v + 8 * k, rowf2);
                    }
                    fence_async_smem();
                }
                tc_fence_before();
                mbar_arrive(o_free);
                __syncwarp();
                if (out_live) {
                    if (32 * tq + 32 <= t.n) {
                        if (lane == 0) {
                            tma_store_3d(&g.out, sm + SM::OUT + half * kHalf + quad * 4096, 64 * half, head, (int)(w.b * p.seqs.L) + t.t0 + 32 * tq);
                            bulk_commit();
                        }
                    } else if (32 * tq < t.n) {
                        const int c = lane & 7;
                        __nv_bfloat16* out = (__nv_bfloat16*)p.out + (w.b * p.seqs.L + t.t0) * p.ldout + (int64_t)head * p.dz + 64 * half + 8 * c;
                        if (64 * half + 8 * c < p.dz) {
#pragma unroll 1
                            for (int k = 0; k < 8; ++k) {
                                const int row = 4 * k + (lane >> 3), tok = 32 * tq + row;
                                uint32_t v[4];
                                ld_shared_v4(stage + sw128(row, c), v[0], v[1], v[2], v[3]);
                                if (tok < t.n) *reinterpret_cast<uint4*>(out + tok * p.ldout) = make_uint4(v[0], v[1], v[2], v[3]);
                            }
                        }
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(tb, 512);
    }
    if (*abort != 0) return;
    for (int i = 0; i < *notes.count; ++i) walk_by_tokens<false>(p, *seg, reinterpret_cast<float*>(sm), notes.at[i], i == kMostNoted - 1);
}

// ------------------------------------------------------------------------- segments' end states

// A segment's own contribution to the state that leaves it, from all tokens that reach it, each with its
// whole power of the decay: nothing is scaled on the way.  Two groups of eight warps make Y~ in turn, warp 16
// copies, warp 17 issues the MMAs; they sum four tiles from zero in one of two places in TMEM, and all sixteen warps
// add that to the sum in their registers (see StateRow) two places later.
constexpr int kEndsThreads = 576, kEndsStages = 4, kEndsBatch = 4;
template <bool three>
struct EndsSmem {
    static constexpr uint32_t YZ = 0;
    static constexpr uint32_t KT = kEndsStages * 4 * kBox;
    static constexpr uint32_t BARS = KT + 2 * (three ? 6 : 4) * kBox;
    static constexpr uint32_t BYTES = BARS + 256 + 1024;
    static_assert(BYTES <= 227 * 1024, "shared memory of a CTA");
};

template <bool rev, bool three>
__global__ void __launch_bounds__(kEndsThreads, 1) decay_tc_ends_kernel(const __grid_constant__ TcArgs g, float* recs) {
    using SM = EndsSmem<three>;
    constexpr uint32_t kGroup = (three ? 6 : 4) * kBox;  // a group's Y~
    extern __shared__ uint8_t smem_raw[];
    const DecayPass& p = g.p;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (base - smem_u32(smem_raw));
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + SM::BARS);
    uint64_t *yz_full = bar, *yz_free = bar + 4, *kt_full = bar + 8, *kt_free = bar + 10, *summed = bar + 12, *taken = bar + 14, *drained = bar + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 17);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Seg w = seg_of<true>(p);
    check_offsets(p.seqs, p.header);
    const float l2 = log2_decay(p.log_decay, w.h);
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&yz_full[i], 1);
            mbar_init(&yz_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&kt_full[i], 256);
            mbar_init(&kt_free[i], 1);
            mbar_init(&summed[i], 1);
            mbar_init(&taken[i], 512);
        }
        mbar_init(drained, 1);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == 17) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dep_launch();
    const uint32_t tb = *tmem_slot;
    const Waiter wait{abort, p.header};
    const int nhx = (p.dx + 63) / 64, nhz = (p.dz + 63) / 64, nz = (p.dz + 15) / 16 * 16;
    Reach r = reach(p.seqs, w.b, w.lo, w.hi, rev);
    const int64_t end = r.to, begin = r.from;  // of the tokens that reach the state
    if (p.parts == 2) {                        // this CTA's half of them
        const int64_t cut = r.from + ((r.to - r.from + 2 * kTile - 1) / (2 * kTile)) * kTile;
        if (blockIdx.x < p.units) r.to = min64(cut, end);
        else r.from = min64(cut, end), r.whole = false;
    }
    const uint32_t items = (uint32_t)((r.to - r.from + kTile - 1) / kTile) * p.gy;

    if (warp == 16) {
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
                    uint8_t* to = sm + SM::YZ + s * 4 * kBox;
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
    } else if (warp == 17) {
        const bool leader = lane == 0;
        const uint32_t id_h = idesc_bf16(128, nz, true, true);
        uint32_t it = 0;
        for (; it < items; ++it) {
            const int k = it & 1;
            const uint32_t b = it / kEndsBatch, at = it % kEndsBatch;
            if (!wait.all(&kt_full[k], (it >> 1) & 1, 121)) break;
            if (at == 0 && b >= 2 && !wait.all(&taken[b & 1], ((b >> 1) & 1) ^ 1, 125)) break;
            tc_fence_after();
            state_mmas<three ? 12 : 8>(leader, uniform(tb + (b & 1) * 128), uniform(base + SM::KT + k * kGroup), three ? 3 : 2, uniform(base + SM::YZ + ((it % kEndsStages) * 4 + 2) * kBox), kBox, id_h,
                       at == 0);
            if (leader) {
                mma_commit(&kt_free[k]);
                mma_commit(&yz_free[it % kEndsStages]);
                if (at == kEndsBatch - 1 || it == items - 1) mma_commit(&summed[b & 1]);
            }
        }
        if (it < items) {
            if (leader) mma_commit(drained);
            mbar_wait(drained, 0, tc::kTimeout);
        }
    } else {
        const int group = warp >> 3, in = tid & 255, tok = in & 63;
        const int c = 32 * (warp >> 2);  // 32 of a row's columns
        float sum[32] = {};
        uint32_t it = 0, b = 0;  // items, batches added to the sum
        auto take = [&]() {
            if (!wait.all(&summed[b & 1], (b >> 1) & 1, 124)) return false;
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
                float v[16];
                tmem_get16(tb + (b & 1) * 128 + ((uint32_t)(32 * (warp & 3)) << 16) + c + h, v);
#pragma unroll
                for (int k = 0; k < 16; ++k) sum[h + k] += v[k];
            }
            tc_fence_before();
            mbar_arrive(&taken[b & 1]);
            ++b;
            return true;
        };
        bool ok = true;
        for (int64_t t0 = r.from; t0 < r.to && ok; t0 += kTile) {
            const int n = (int)min64(kTile, r.to - t0);
            for (int gh = 0; gh < p.gy; ++gh, ++it) {
                if (it >= (b + 2) * kEndsBatch && !take()) { ok = false; break; }
                if ((int)(it & 1) != group) continue;
                const int s = it % kEndsStages;
                if (!wait.all(&yz_full[s], (it / kEndsStages) & 1, 122)) { ok = false; break; }
                if (it >= 2 && !wait.all(&kt_free[group], ((it >> 1) & 1) ^ 1, 123)) { ok = false; break; }
                const float f = tok < n ? power(l2, rev ? t0 + tok - begin + 1 : end - 1 - t0 - tok) * p.in_scale : 0.0f;
                const uint32_t ya = base + SM::YZ + s * 4 * kBox;
                if (n < 64) clear_rows<256>(ya + 2 * kBox, kBox, n, in);
                scale_rows<three, 2>(ya, kBox, base + SM::KT + group * kGroup, 2 * ((p.dx + 15) / 16), n, f, in);
                fence_async_smem();
                mbar_arrive(&kt_full[group]);
            }
        }
        while (ok && b * kEndsBatch < items) ok = take();
        if (ok) {
            const int row = 32 * (warp & 3) + lane;
            const int64_t size = (int64_t)p.dx * p.dz;
            float* to = recs + (w.unit * p.nseg + (p.parts > 0 ? (int)(blockIdx.x / p.units) : w.seg)) * size + (int64_t)row * p.dz;
            const float* from = r.whole && p.init != nullptr ? p.init + (r.seq * p.Hkv + w.h) * size + (int64_t)row * p.dz : nullptr;
            const float f = from != nullptr ? power(l2, end - begin) : 0.0f;
            if (row < p.dx) {
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    if (c + k >= p.dz) continue;
                    float4 u = make_float4(sum[k], sum[k + 1], sum[k + 2], sum[k + 3]);
                    if (from != nullptr) {
                        const float4 i = *reinterpret_cast<const float4*>(from + c + k);
                        u.x = fmaf(f, i.x, u.x), u.y = fmaf(f, i.y, u.y), u.z = fmaf(f, i.z, u.z), u.w = fmaf(f, i.w, u.w);
                    }
                    *reinterpret_cast<float4*>(to + c + k) = u;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(tb, 256);
    }
}

bool args_of(const DecayPass& p, TcArgs* a) {
    a->p = p;
    const int64_t rows = p.units / p.Hkv * p.seqs.L;
    return map_of(&a->x, p.x, rows, p.Hkv * p.gx, p.dx, p.ldx) && map_of(&a->y, p.y, rows, p.Hkv * p.gy, p.dx, p.ldy) &&
           map_of(&a->z, p.z, rows, p.Hkv * p.gy, p.dz, p.ldz) &&
           (p.out == nullptr || map_of(&a->out, p.out, rows, p.Hkv * p.gx, p.dz, p.ldout, 32));
}

template <typename SM, bool three>
cudaError_t go(const TcArgs& a, cudaStream_t s) {
    const auto kernel = decay_tc_kernel<SM, three>;
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

template <bool rev, bool three>
cudaError_t go_ends(const TcArgs& a, float* recs, cudaStream_t s) {
    using SM = EndsSmem<three>;
    const auto kernel = decay_tc_ends_kernel<rev, three>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SM::BYTES);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(a.p.units * (a.p.parts > 0 ? a.p.parts : a.p.nseg - 1 + a.p.all_ends)), kEndsThreads, SM::BYTES, s>>>(a, recs);
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
    if (three_parts(p)) return p.rev ? go_ends<true, true>(a, recs, s) : go_ends<false, true>(a, recs, s);
    return p.rev ? go_ends<true, false>(a, recs, s) : go_ends<false, false>(a, recs, s);
}

cudaError_t decay_tc_pass(const DecayPass& p, cudaStream_t s) {
    TcArgs a;
    if (!args_of(p, &a)) return cudaErrorInvalidValue;
    if (three_parts(p)) return p.gx > 1 ? go<Wide, true>(a, s) : go<Even, true>(a, s);
    return p.gx > 1 ? go<Wide, false>(a, s) : go<Even, false>(a, s);
}

}  // namespace lz
