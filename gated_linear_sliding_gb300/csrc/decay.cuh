// Device helpers that the kernels of the linear attention with a decay for each head share: the walk
// over a segment's tiles and the powers of a decay.
#pragma once

#include "heads.h"

namespace lz {

constexpr int kTile = 64;  // tokens of a tile: all pairs inside it are formed

// log2 of a head's decay.  Minus infinity becomes a number whose every power but the 0th is 0 (0 times
// infinity would be NaN); NaN stays.
__device__ __forceinline__ float log2_decay(const float* log_decay, int64_t h) {
    const float l = log_decay[h] * kLog2e;
    return l < -1e4f ? -1e4f : l;
}
__device__ __forceinline__ float power(float l2, int64_t n) { return exp2f(l2 * (float)n); }

// Up to a tile's length of consecutive tokens of one sequence, in a row of the batch.
struct Tile {
    int t0, n;
    bool first, last;  // the walk enters the sequence with this tile, leaves it after it
    bool leaves;       // the sequence goes on in the walk's next segment
    int seq;
};

// The tiles of a segment [lo, hi) of row b, forwards or backwards in time.  A tile ends where its
// sequence does.  (A row has fewer than 2^31 tokens, and so has a batch sequences.)
struct Walk {
    int lo, hi, at, begin, end, seq, tile;
    bool rev;
    __device__ __forceinline__ Walk(const Seqs& s, int64_t b, int64_t lo_, int64_t hi_, bool rev_, int tile_ = kTile)
        : lo((int)lo_), hi((int)hi_), at((int)(rev_ ? hi_ : lo_)), begin(0), end(0), seq(0), tile(tile_), rev(rev_) {
        if (lo < hi) enter(s, b);
    }
    __device__ __forceinline__ void enter(const Seqs& s, int64_t b) {
        const SeqAt q = seq_at(s, b, rev ? at - 1 : at);
        begin = (int)q.begin;
        end = (int)q.end;
        seq = (int)q.seq;
    }
    __device__ __forceinline__ bool next(const Seqs& s, int64_t b, Tile* t) {
        if (rev ? at <= lo : at >= hi) return false;
        if (rev ? at <= begin : at >= end) enter(s, b);
        t->seq = seq;
        t->leaves = rev ? begin < lo : end > hi;
        if (!rev) {
            const int to = min(min(at + tile, end), hi);
            t->t0 = at;
            t->n = to - at;
            t->first = at == begin;
            t->last = to == end;
            at = to;
        } else {
            const int from = max(max(at - tile, begin), lo);
            t->t0 = from;
            t->n = at - from;
            t->first = at == end;
            t->last = from == begin;
            at = from;
        }
        return true;
    }
};

// Segments whose end state is wanted: those that another one begins with, all but the last in the order of time; or all.
__device__ __forceinline__ int ending_segment(const DecayPass& p, int i) { return p.rev && !p.all_ends ? i + 1 : i; }
__device__ __forceinline__ const float* first_state(const DecayPass& p, int64_t unit, int seg) {
    return p.recs + (unit * p.nseg + (p.parts > 0 ? 0 : seg)) * p.dx * p.dz;
}

// The state of head h that a sequence begins with, in the segment where it does (null: zero).  Only a sequence that
// goes on in another segment may have had it overwritten by then.
__device__ __forceinline__ const float* sequence_state(const DecayPass& p, const Tile& t, int64_t h, int seg) {
    if (p.init == nullptr) return nullptr;
    const int64_t size = (int64_t)p.dx * p.dz;
    if (p.kept != nullptr && t.leaves) return p.kept + ((p.rev ? seg - 1 : seg) * p.Hkv + h) * size;
    return p.init + (t.seq * p.Hkv + h) * size;
}

// The part of a segment whose tokens reach the state that leaves it: tokens [from, to), and whether
// the sequence's own first state (not the segment before) is what they begin with.
struct Reach {
    int64_t from, to, seq;
    bool whole;
};
__device__ __forceinline__ Reach reach(const Seqs& s, int64_t b, int64_t lo, int64_t hi, bool rev) {
    Reach r;
    const SeqAt q = seq_at(s, b, rev ? lo : hi - 1);
    r.seq = q.seq;
    r.from = rev ? lo : max64(q.begin, lo);
    r.to = rev ? min64(q.end, hi) : hi;
    r.whole = rev ? q.end <= hi : q.begin >= lo;
    return r;
}

}  // namespace lz
