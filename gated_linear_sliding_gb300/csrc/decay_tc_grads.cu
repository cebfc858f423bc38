// Gradients of keys and values of the linear attention with a decay for each head, on the tensor cores (tcgen05,
// TMEM and TMA, sm_103a).
//
//   dS[t] = e^l dS[t+1] + scale sum over query heads of q[t] do[t]^T,   dk[t] = dS[t] v[t],   dv[t] = dS[t]^T k[t]
// A CTA walks a segment of one state head backwards in chunks of 64 tokens.  With E the state behind a chunk as its
// last token sees it, and for two query heads at a time the 128 rows (head, i) of Q and dO,
//   P  = scale (Q K^T) (.) e^(l (i - j)),   P' = scale (dO V^T) (.) e^(l (i - j)),   masked to i >= j      [128 x 64]
//   dv^T = E^T K^T (.) e^(l (n-1-j)) + dO^T P,    dk^T = E V^T (.) e^(l (n-1-j)) + Q^T P'                 [128 x 64]
//   E' = e^l (what is before the chunk sees) = e^(l n) E + Q~^T dO,   Q~[i] = scale e^(l (i+1)) Q[i]
// Both gradients share the copies of Q, dO, K, V, the state and its updates, and both are made transposed, so that the
// MMAs' 128 rows are two heads' tokens or a head's values.  As two passes of the outputs' form (one with dS, one with
// its transpose) they took 204 us for a training step of 8 x 2048 tokens, 32 heads on 8, 128 values; together 135, of
// which their bytes take 64: bound by the chain of a chunk and by what the SM's warps issue in it.
//
// The decay of a pair is e^(l (i-r)) e^(l (r-j)), r in the middle of the chunk: a factor of the rows of P and one of the
// finished columns; heads that lose more than a half a token take each pair's power (see the outputs' kernel, also
// for the roundings).
//
// Warps: 0-7 pairs and gradients; 8-15 the state (half a row to a thread) and Q~; 16 the copies; 17 the MMAs of the
// scores, 18 those into the state, 19 those of the gradients.  TMEM: two scores of 64 columns, two gradients of 64, the
// state 128, a chunk's part of it 128.
#include "decay_tc.cuh"

namespace lz {
namespace {

struct GradArgs {
    CUtensorMap q, d_o, k, v, dk, dv;
    DecayPass p;  // the pass of dv: x = k, y = q, z = d_o
    void *dk_out, *dv_out;
    int64_t lddk, lddv;
};

// Tiles of Q and dO take turns in three places of 128 rows, or, with one query head a state, in four of 64.  With two
// items or more in a chunk the last one's dO goes where the state's operand copy was, which is read at a chunk's
// beginning and written behind its last item: three places alone had dO wait for the item before (164 us for the
// training step above).  With one query head the gradients leave through a place of their own, otherwise through that
// of P.
struct GradSmem {
    static constexpr uint32_t RING = 0;
    static constexpr uint32_t KV = 12 * kBox;         // K, V: 64 rows each
    static constexpr uint32_t OWN = RING + 8 * kBox;  // dv and dk [64 x 128] on their way out, one query head a state
    static constexpr uint32_t PP = KV + 4 * kBox;     // P, P' [128 x 64]; else dv and dk
    static constexpr uint32_t KT = PP + 4 * kBox;     // Q~: its first part, later its third; the second
    static constexpr uint32_t ST = KT + 4 * kBox;
    static constexpr uint32_t TABLE = ST + 4 * kBox;  // powers 0 .. 64, and the columns' factors
    static constexpr uint32_t BARS = TABLE + (68 + 64) * 4;
    static constexpr uint32_t BYTES = BARS + 376 + 4 * kMostNoted + 1024;
    static_assert(BYTES <= 227 * 1024 && kByTokensBytes <= TABLE, "shared memory of a CTA");
};

template <bool three>
__global__ void __launch_bounds__(kThreads, 1) decay_tc_grads_kernel(const __grid_constant__ GradArgs g) {
    using SM = GradSmem;
    extern __shared__ uint8_t smem_raw[];
    const DecayPass& p = g.p;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (base - smem_u32(smem_raw));
    float* pw = reinterpret_cast<float*>(sm + SM::TABLE);  // powers of the decay
    float* col = pw + 68;                                  // factors of the finished columns
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + SM::BARS);
    uint64_t *b_full = bar, *b_free = bar + 6, *kv_full = bar + 12, *kv_free = bar + 13, *s_full = bar + 14, *p_full = bar + 15, *pv_done = bar + 16,
             *xs_full = bar + 17, *o_free = bar + 19, *zz_full = bar + 21, *kt_full = bar + 23, *h_done = bar + 24, *st_full = bar + 25,
             *xs_done = bar + 26, *staged = bar + 27, *left = bar + 28, *late = bar + 29, *drained = bar + 30, *chunk_done = bar + 33;
    uint64_t *first_free = bar + 34, *third_full = bar + 35, *agreed = bar + 36;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 38);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    Seg* seg = reinterpret_cast<Seg*>(bar + 41);  // (for walk_by_tokens: in registers till then it makes the roles spill)
    const Notes notes{abort + 1, abort + 2, abort + 3, abort + 17, agreed};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool leader = lane == 0;
    const Seg w = seg_of<false>(p);
    check_offsets(p.seqs, p.header);
    constexpr int mid = 31;
    const float l2 = log2_decay(p.log_decay, w.h);
    const bool slow = fabsf(l2) <= 1.0f;
    for (int i = tid; i <= 64; i += kThreads) {
        pw[i] = power(l2, i);
        if (i < 64) col[i] = slow ? power(l2, mid - i) : 1.0f;
    }
    const int nhx = (p.dx + 63) / 64, nhz = (p.dz + 63) / 64;
    if (tid == 0) {
        for (int i = 0; i < 6; ++i) {
            mbar_init(&b_full[i], 1);
            mbar_init(&b_free[i], 2);  // the gradients' and the state's MMAs
        }
        mbar_init(kv_full, 1);
        mbar_init(late, 1);
        mbar_init(kv_free, 2);  // the scores and the state's parts
        mbar_init(s_full, 1);
        mbar_init(p_full, 32 * kMathWarps);
        mbar_init(pv_done, 1);
        mbar_init(chunk_done, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&xs_full[i], 1);
            mbar_init(&zz_full[i], 32 * kStateWarps);
        }
        mbar_init(o_free, 32 * kMathWarps);
        mbar_init(kt_full, 32 * kStateWarps);
        mbar_init(first_free, 1);
        mbar_init(third_full, 32 * kStateWarps);
        mbar_init(h_done, 1);
        mbar_init(st_full, 32 * kStateWarps);
        mbar_init(xs_done, 1);
        mbar_init(staged, 32 * kMathWarps);
        mbar_init(left, kMathWarps);
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
    const int kx = (p.dx + 15) / 16, kz = (p.dz + 15) / 16, nz = 16 * kz;
    const int nt = (p.gy + 1) / 2;  // items of a chunk: two query heads, or one
    const bool single = p.gy == 1;
    const uint32_t places = single ? 4 : 3, place = single ? 2 * kBox : 4 * kBox, apart = single ? kBox : kHalf;
    // of item a, whose Q is tile b of the ring: where its dO is
    auto is_late = [&](int a) { return nt > 1 && a == nt - 1; };
    auto tile = [&](uint32_t b) { return base + SM::RING + (b % places) * place; };
    auto d_o_at = [&](int a, uint32_t b) { return is_late(a) ? base + SM::ST : tile(b + 1); };

    Walk walk(p.seqs, w.b, w.lo, w.hi, true, 64);
    Tile t;

    if (warp == 16) {
        if (lane == 0) {
            prefetch_tmap(&g.q);
            prefetch_tmap(&g.d_o);
            prefetch_tmap(&g.k);
            prefetch_tmap(&g.v);
            uint32_t bi = 0, ci = 0, li = 0;
            bool ok = true;
            while (ok && walk.next(p.seqs, w.b, &t)) {
                const int row = (int)(w.b * p.seqs.L) + t.t0;
                for (int a = 0; a < nt && ok; ++a) {
                    const int heads = p.gy - 2 * a < 2 ? 1 : 2, head = (int)(w.h * p.gy) + 2 * a;
                    for (int e = 0; e < 2; ++e) {  // Q, then dO
                        const bool behind = e == 1 && is_late(a);
                        const uint32_t s = bi % places;
                        const int nh = e == 0 ? nhx : nhz;
                        if (behind ? !wait(xs_done, ci & 1, 155) : bi >= places && !wait(&b_free[s], ((bi / places) & 1) ^ 1, 130)) { ok = false; break; }
                        uint64_t* full = behind ? late : &b_full[s];
                        uint8_t* to = sm + (behind ? SM::ST : SM::RING + s * place);
                        mbar_arrive_expect_tx(full, heads * nh * kBox);
                        for (int k = 0; k < heads; ++k)
                            for (int h = 0; h < nh; ++h) tma_load_3d(to + h * apart + k * kBox, e == 0 ? &g.q : &g.d_o, full, 64 * h, head + k, row);
                        if (behind) ++li;
                        else ++bi;
                        if (a == 0 && e == 0) {  // K and V of the chunk, behind the first Q, which need not wait for their place
                            if (ci >= 1 && !wait(kv_free, (ci & 1) ^ 1, 131)) { ok = false; break; }
                            mbar_arrive_expect_tx(kv_full, (nhx + nhz) * kBox);
                            for (int h = 0; h < nhx; ++h) tma_load_3d(sm + SM::KV + h * kBox, &g.k, kv_full, 64 * h, (int)w.h, row);
                            for (int h = 0; h < nhz; ++h) tma_load_3d(sm + SM::KV + (2 + h) * kBox, &g.v, kv_full, 64 * h, (int)w.h, row);
                        }
                    }
                }
                if (ok) ++ci;
            }
            if (!ok) {  // let the copies under way land before the CTA leaves
                for (uint32_t q = bi > places ? bi - places : 0; q < bi; ++q) mbar_wait(&b_full[q % places], (q / places) & 1, tc::kTimeout);
                if (ci > 0) mbar_wait(kv_full, (ci - 1) & 1, tc::kTimeout);
                mbar_wait(kv_full, ci & 1, tc::kTimeout / 4);  // perhaps under way
                if (li > 0) mbar_wait(late, (li - 1) & 1, tc::kTimeout);
            }
        }
        __syncwarp();
    } else if (warp == 17) {
        // scores: Q K^T and dO V^T
        const uint32_t id_s = idesc_bf16(128, 64, false, false);
        uint32_t it = 0, ci = 0, q = 0;
        bool ok = true;
        while (ok && walk.next(p.seqs, w.b, &t)) {
            if (!wait.all(kv_full, ci & 1, 132)) { ok = false; break; }
            for (int a = 0; a < nt; ++a, ++it) {
                const uint32_t o = q + 1;
                if (!wait.all(&b_full[q % places], (q / places) & 1, 133) ||
                    !(is_late(a) ? wait.all(late, ci & 1, 134) : wait.all(&b_full[o % places], (o / places) & 1, 134)) ||
                    (it >= 1 && !wait.all(p_full, (it & 1) ^ 1, 135))) {  // the scores before have been read
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll 1
                for (int e = 0; e < 2; ++e) {
                    const uint32_t xa = uniform(e == 0 ? tile(q) : d_o_at(a, q)), ya = uniform(base + SM::KV + e * 2 * kBox);
#pragma unroll 1
                    for (int k = 0; k < (e == 0 ? kx : kz); ++k)
                        mma_bf16_one(leader, tS + 64 * e, kdesc(xa + (k >> 2) * apart + (k & 3) * 32), kdesc(ya + (k >> 2) * kBox + (k & 3) * 32), id_s, k > 0);
                }
                q += is_late(a) ? 1 : 2;
                if (leader) {
                    mma_commit(s_full);
                    if (a == nt - 1) mma_commit(kv_free);
                }
            }
            ++ci;
        }
        if (!ok) {  // every MMA that was issued ends before the CTA leaves: they read shared memory
            if (leader) mma_commit(&drained[0]);
            mbar_wait(&drained[0], 0, tc::kTimeout);
        }
    } else if (warp == 19) {
        // gradients, transposed: the state's parts, and the pairs' on top
        const uint32_t id_v = idesc_bf16(128, 64, true, false), id_k = idesc_bf16(128, 64, false, false), id_p = idesc_bf16(128, 64, true, true);
        uint32_t it = 0, ci = 0, q = 0;
        bool ok = true;
        while (ok && walk.next(p.seqs, w.b, &t)) {
            const uint32_t to = uniform(tO);
            if (!wait.all(kv_full, ci & 1, 136) || (ci >= 1 && !wait.all(o_free, (ci & 1) ^ 1, 137)) || !wait.all(st_full, ci & 1, 138)) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < kx; ++k)  // E^T K^T
                mma_bf16_one(leader, to, mndesc(base + SM::ST + k * 2048, kHalf), kdesc(base + SM::KV + (k >> 2) * kBox + (k & 3) * 32), id_v, k > 0);
#pragma unroll 1
            for (int k = 0; k < kz; ++k)  // E V^T
                mma_bf16_one(leader, to + 64, kdesc(base + SM::ST + (k >> 2) * kHalf + (k & 3) * 32), kdesc(base + SM::KV + (2 + (k >> 2)) * kBox + (k & 3) * 32),
                             id_k, k > 0);
            if (leader) {
                if (!slow) mma_commit(&xs_full[ci & 1]);
                mma_commit(xs_done);
                mma_commit(kv_free);
            }
            for (int a = 0; a < nt; ++a, ++it) {
                const int steps = p.gy - 2 * a < 2 ? 4 : 8;  // of 16 rows
                if (!wait.all(&zz_full[it & 1], (it >> 1) & 1, 139) || !wait.all(p_full, it & 1, 140)) { ok = false; break; }
                tc_fence_after();
#pragma unroll 1
                for (int e = 0; e < 2; ++e) {  // dO^T P, Q^T P'
                    const uint32_t xa = uniform(e == 0 ? d_o_at(a, q) : tile(q)), pa = uniform(base + SM::PP + e * 2 * kBox);
#pragma unroll 1
                    for (int k = 0; k < steps; ++k)
                        mma_bf16_one(leader, to + 64 * e, mndesc(xa + k * 2048, apart), mndesc(pa + k * 2048, kHalf), id_p, 1u);
                }
                if (leader) {
                    mma_commit(pv_done);
                    if (a == nt - 1) mma_commit(chunk_done);
                    mma_commit(&b_free[q % places]);
                    if (!is_late(a)) mma_commit(&b_free[(q + 1) % places]);
                }
                q += is_late(a) ? 1 : 2;
            }
            ++ci;
        }
        if (!ok) {
            if (leader) mma_commit(&drained[1]);
            mbar_wait(&drained[1], 0, tc::kTimeout);
        }
    } else if (warp == 18) {
        const uint32_t id_h = idesc_bf16(128, nz, true, true);
        uint32_t ui = 0, ci = 0, q = 0;
        bool ok = true;
        while (ok && walk.next(p.seqs, w.b, &t)) {
            for (int a = 0; a < nt && ok; ++a) {
                const uint32_t oa = uniform(d_o_at(a, q)), o = q + 1;
                const int heads = p.gy - 2 * a < 2 ? 1 : 2;
                if (!(is_late(a) ? wait.all(late, ci & 1, 154) : wait.all(&b_full[o % places], (o / places) & 1, 154))) { ok = false; break; }
                for (int k = 0; k < heads; ++k, ++ui) {
                    if (!wait.all(kt_full, ui & 1, 141)) { ok = false; break; }
                    tc_fence_after();
                    if (!three) state_mmas<1>(leader, tD, base + SM::KT, 2, oa + k * kBox, apart, id_h, a == 0 && k == 0);
                    if (three) {
                        state_mmas<1>(leader, tD, base + SM::KT, 1, oa + k * kBox, apart, id_h, a == 0 && k == 0);
                        if (leader) mma_commit(first_free);
                        state_mmas<1>(leader, tD, base + SM::KT + 2 * kBox, 1, oa + k * kBox, apart, id_h, false);
                        if (!wait.all(third_full, ui & 1, 158)) { ok = false; break; }
                        tc_fence_after();
                        state_mmas<1>(leader, tD, base + SM::KT, 1, oa + k * kBox, apart, id_h, false);
                    }
                    if (leader) mma_commit(h_done);
                }
                if (ok && leader) {
                    mma_commit(&b_free[q % places]);
                    if (!is_late(a)) mma_commit(&b_free[o % places]);
                }
                q += is_late(a) ? 1 : 2;
            }
            ++ci;
        }
        if (!ok) {
            if (leader) mma_commit(&drained[2]);
            mbar_wait(&drained[2], 0, tc::kTimeout);
        }
    } else if (warp >= kMathWarps) {
        // the state: half a row of E to a thread
        const StateRow sr = state_row(p, tH, tD, tid - 32 * kMathWarps);
        float keep = 1.0f;  // of the chunk before
        uint32_t it = 0, ui = 0, ci = 0, q = 0;
        bool ok = true, was_last = false;
        int was_seq = 0, ends = 1;  // the sequence under way is the ends-th
        grid_dep_wait();
        while (ok && walk.next(p.seqs, w.b, &t)) {
            if (ci > 0) {
                // (a late dO lies where the state's copy goes: the gradients' products are done with it.  A wait names
                // one of a barrier's last two phases, so these warps, which do not see every item's, have a barrier of
                // the chunks.)
                if (!wait.all(h_done, (ui - 1) & 1, 142) || !wait.all(xs_done, (ci - 1) & 1, 143) || !wait.all(chunk_done, (ci - 1) & 1, 156)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (was_last && may_leave(notes, wait, sr, nz, ends++, &ok)) leave_state(p, sr, w.h, was_seq, keep);
                if (!ok) break;
            }
            const bool fresh = t.first || ci == 0;
            if (fresh) begin_state(p, sr, w, t);
            if (!pass_state(sr, base + SM::ST, nz, slow ? power(l2, t.n - 1 - mid) : 1.0f, fresh, keep)) *notes.found = ends;
            if (sr.in == 0) *notes.entered = min(walk.end, walk.hi);
            keep = pw[t.n];
            fence_async_smem();
            tc_fence_before();
            mbar_arrive(st_full);
            for (int a = 0; a < nt && ok; ++a, ++it) {
                const uint32_t qa = tile(q), oa = d_o_at(a, q), o = q + 1;
                const int heads = p.gy - 2 * a < 2 ? 1 : 2, tok = sr.in & 63;
                if (!wait.all(&b_full[q % places], (q / places) & 1, 144)) { ok = false; break; }
                if (t.n < 64) {  // rows behind the last token are factors of the products over rows
                    if (!(is_late(a) ? wait.all(late, ci & 1, 145) : wait.all(&b_full[o % places], (o / places) & 1, 145))) { ok = false; break; }
                    for (int k = 0; k < heads; ++k) {
                        clear_rows<32 * kStateWarps>(qa + k * kBox, apart, t.n, sr.in);
                        clear_rows<32 * kStateWarps>(oa + k * kBox, apart, t.n, sr.in);
                    }
                    fence_async_smem();
                }
                mbar_arrive(&zz_full[it & 1]);
                for (int k = 0; k < heads; ++k, ++ui) {
                    // the first of a chunk: waited for before the state's copy
                    if ((a > 0 || k > 0) && !wait.all(h_done, (ui - 1) & 1, 146)) { ok = false; break; }
                    const float f = tok < t.n ? pw[tok + 1] * p.in_scale : 0.0f;
                    scale_rows<false, 1>(qa + k * kBox, apart, base + SM::KT, 2 * kx, t.n, f, sr.in);
                    fence_async_smem();
                    tc_fence_before();
                    mbar_arrive(kt_full);
                    if (three) {
                        if (!wait.all(first_free, ui & 1, 159)) { ok = false; break; }
                        third_of_rows(qa + k * kBox, apart, base + SM::KT, 2 * kx, t.n, f, sr.in);
                        fence_async_smem();
                        tc_fence_before();
                        mbar_arrive(third_full);
                    }
                }
                q += is_late(a) ? 1 : 2;
            }
            was_last = t.last;
            was_seq = t.seq;
            ++ci;
        }
        if (ok && ci > 0 && wait.all(h_done, (ui - 1) & 1, 147)) {
            tc_fence_after();
            if (may_leave(notes, wait, sr, nz, ends, &ok) && was_last) leave_state(p, sr, w.h, was_seq, keep);
        }
    } else {
        // pairs: row r = (head, token i) of an item; gradients: value r, 32 of the chunk's tokens
        const int quad = warp & 3, half = warp >> 2, r = 32 * quad + lane, i = r & 63, tq = quad & 1;
        const uint32_t lanes = (uint32_t)(32 * quad) << 16;
        const float rowf = p.in_scale * (slow ? power(l2, i - mid) : 1.0f);
        const uint32_t c0 = base + SM::TABLE + 68 * 4;
        uint32_t sw[8];  // places of a value's 16 bytes in rows of the swizzle
#pragma unroll
        for (int k = 0; k < 8; ++k) sw[k] = (((r & 63) >> 3) ^ k) << 4;
        uint32_t it = 0, ci = 0;
        const uint32_t stage = single ? SM::OWN : SM::PP;
        // this warp's part of the gradients before has left the place that is written next
        auto vacant = [&]() {
            __syncwarp();
            if (lane == 0) {
                bulk_wait_read();
                mbar_arrive(left);
            }
        };
        const uint32_t acc = tO + lanes + 32 * half;
        while (walk.next(p.seqs, w.b, &t)) {
            if (!slow) {  // e^(l (n-1-j)) on the state's parts
                if (!wait.all(&xs_full[ci & 1], (ci >> 1) & 1, 148)) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < 128; c += 16) {
                    if ((c & 63) >= 32) continue;
                    float v[16];
                    tmem_get16(acc + c, v);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const int far = t.n - 1 - 32 * half - (c & 63) - k;
                        v[k] = far >= 0 ? v[k] * pw[far] : 0.0f;
                    }
                    tmem_st16(acc + c, reinterpret_cast<const uint32_t*>(v));
                }
                tmem_wait_st();
            }
            bool ok = true;
            for (int a = 0; a < nt; ++a, ++it) {
                const bool on = 2 * a + (quad >> 1) < p.gy;
                if (!wait.all(s_full, it & 1, 149)) { ok = false; break; }
                // the place of P is free: its MMAs are done, and a chunk's gradients have left it
                if (it >= 1 && !wait.all(pv_done, (it - 1) & 1, 150)) { ok = false; break; }
                if (!single && a == 0 && ci >= 1) {
                    vacant();
                    if (!wait.all(left, (ci - 1) & 1, 151)) { ok = false; break; }
                }
                tc_fence_after();
                if (on) {
#pragma unroll 1
                    for (int c = 0; c < 128; c += 16) {  // 32 columns of P, then of P'
                        if ((c & 63) >= 32) continue;
                        const int j = 32 * half + (c & 63);
                        const uint32_t to = base + SM::PP + (c >> 6) * 2 * kBox;
                        float v[16];
                        tmem_get16(tS + lanes + 32 * half + c, v);
                        if (!slow) {
#pragma unroll
                            for (int k = 0; k < 16; ++k) v[k] *= pw[i - j - k < 0 ? 0 : i - j - k];
                        }
                        if (tq <= half || t.n < 64) {  // tokens before the column's, and behind the last one, are left out whatever they hold
                            const int last = i < t.n ? i - j : -1;
#pragma unroll
                            for (int k = 0; k < 16; ++k) v[k] = k <= last ? v[k] : 0.0f;
                        }
                        const f2 f = pack(rowf, rowf);
                        st_scaled8(to + sw128(r, (j >> 3)), v, f);
                        st_scaled8(to + sw128(r, (j >> 3) + 1), v + 8, f);
                    }
                    fence_async_smem();
                }
                tc_fence_before();
                mbar_arrive(p_full);
            }
            if (!ok) break;
            // a chunk's gradients: value r of tokens 32 half .. + 31, to rows of 128 values
            if (!wait.all(pv_done, (it - 1) & 1, 152)) break;
            if (single && ci >= 1) {
                vacant();
                if (!wait.all(left, (ci - 1) & 1, 157)) break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 128; c += 16) {
                if ((c & 63) >= 32) continue;
                const int j = 32 * half + (c & 63);
                const uint32_t to = base + stage + (c >> 6) * 2 * kBox + (r >> 6) * kBox + (r & 7) * 2 + j * 128;
                float v[16];
                tmem_get16(acc + c, v);
#pragma unroll
                for (int k = 0; k < 16; k += 4) {  // single values: 32 lanes make half a row
                    uint32_t f[4];
                    ld_shared_v4(c0 + (j + k) * 4, f[0], f[1], f[2], f[3]);
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const uint16_t h = __bfloat16_as_ushort(__float2bfloat16_rn(v[k + m] * __uint_as_float(f[m])));
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + sw[(k + m) & 7] + (k + m) * 128), "h"(h) : "memory");
                    }
                }
            }
            fence_async_smem();
            tc_fence_before();
            mbar_arrive(o_free);
            mbar_arrive(staged);
            if (!wait.all(staged, ci & 1, 153)) break;
            // a warp to each 64 values of dv and dk, or, of fewer than 64 tokens, rows by all of them
            const int row = (int)(w.b * p.seqs.L) + t.t0;
            if (t.n == 64) {
                const int e = warp >> 1, h = warp & 1;
                if (warp < 4 && h < (e == 0 ? nhz : nhx) && lane == 0) {
                    tma_store_3d(e == 0 ? &g.dv : &g.dk, sm + stage + e * 2 * kBox + h * kBox, 64 * h, (int)w.h, row);
                    bulk_commit();
                }
            } else {
#pragma unroll 1
                for (int e = 0; e < 2; ++e) {
                    const int d = e == 0 ? p.dz : p.dx;
                    const int64_t ld = e == 0 ? g.lddv : g.lddk;
                    __nv_bfloat16* out = (__nv_bfloat16*)(e == 0 ? g.dv_out : g.dk_out) + (w.b * p.seqs.L + t.t0) * ld + w.h * d;
#pragma unroll 1
                    for (int c = tid; c < t.n * 16; c += 32 * kMathWarps) {
                        const int tok = c >> 4, piece = c & 15;
                        uint32_t v[4];
                        ld_shared_v4(base + stage + e * 2 * kBox + (piece >> 3) * kBox + sw128(tok, piece & 7), v[0], v[1], v[2], v[3]);
                        if (8 * piece < d) *reinterpret_cast<uint4*>(out + tok * ld + 8 * piece) = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
            ++ci;
        }
        if (lane == 0) bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(tb, 512);
    }
    if (*abort != 0 || *notes.count == 0) return;
    DecayPass k = p;  // dk's: the same with x and y from the other side of the state.  First, since dv's may overwrite `init`.
    k.x = p.v, k.y = p.z, k.z = p.y, k.out = g.dk_out;
    k.ldx = p.ldv, k.ldy = p.ldz, k.ldz = p.ldy, k.ldout = g.lddk;
    k.dx = p.dz, k.dz = p.dx;
    k.transposed = true;
    k.fin = nullptr;
    for (int i = 0; i < *notes.count; ++i) {
        walk_by_tokens<true>(k, *seg, reinterpret_cast<float*>(sm), notes.at[i], i == kMostNoted - 1);
        walk_by_tokens<true>(p, *seg, reinterpret_cast<float*>(sm), notes.at[i], i == kMostNoted - 1);
    }
}

template <bool three>
cudaError_t go(const GradArgs& a, cudaStream_t s) {
    const auto kernel = decay_tc_grads_kernel<three>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)GradSmem::BYTES);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.p.units * a.p.nseg));
    if (a.p.nseg > 1) {  // its set-up overlaps the segments' ends
        e = launch_dependent(kernel, grid, dim3(kThreads), GradSmem::BYTES, s, a);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    kernel<<<grid, kThreads, GradSmem::BYTES, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t decay_tc_grads(const DecayPass& p, void* dk, int64_t lddk, cudaStream_t s) {
    GradArgs a;
    a.p = p;
    a.dk_out = dk;
    a.dv_out = p.out;
    a.lddk = lddk;
    a.lddv = p.ldout;
    const int64_t rows = p.units / p.Hkv * p.seqs.L;
    if (!map_of(&a.q, p.y, rows, p.Hkv * p.gy, p.dx, p.ldy) || !map_of(&a.d_o, p.z, rows, p.Hkv * p.gy, p.dz, p.ldz) ||
        !map_of(&a.k, p.x, rows, p.Hkv, p.dx, p.ldx) || !map_of(&a.v, p.v, rows, p.Hkv, p.dz, p.ldv) || !map_of(&a.dk, dk, rows, p.Hkv, p.dx, lddk) ||
        !map_of(&a.dv, p.out, rows, p.Hkv, p.dz, p.ldout))
        return cudaErrorInvalidValue;
    return three_parts(p) ? go<true>(a, s) : go<false>(a, s);
}

}  // namespace lz
