// Host-side interface between the entry points of the query and key rotation (lizard_qk_rope_*) and
// of the linear attention with a decay for each head (lizard_decay_attn_*) and their kernels.
#pragma once

#include "selective.h"

namespace lz {

struct RopeArgs {
    int64_t B, L, Hq, Hkv;
    int64_t start;
    int64_t ldq, ldk, ldqo, ldko, lddq, lddk;
    int d, rot, axes;
    int section[4];  // pairs of each axis, as running sums
    float eps;
    int dtype, norm, neighbours;
    const void *q, *k;
    const float *w_q, *w_k, *freqs;
    const int64_t* positions;
    void *q_out, *k_out;
    // backward
    const void *dq_out, *dk_out;
    void *dq, *dk;
    float *dw_q, *dw_k;
    float* partial;  // [CTAs, 2, d]
};
cudaError_t launch_rope_fwd(const RopeArgs& a, cudaStream_t s);
int64_t rope_bwd_ctas(const RopeArgs& a);
cudaError_t launch_rope_bwd(const RopeArgs& a, cudaStream_t s);

// The arguments of a call of lizard_decay_attn_*.
struct DecayArgs {
    int64_t B, Hq, Hkv, dk, dv;
    Seqs seqs;
    int64_t nstate;  // per-sequence states: B or nseq
    int64_t ldq, ldk, ldv, ldo, lddq, lddk, lddv;
    float scale;
    int dtype;
    const void *q, *k, *v;
    const float *log_decay, *s0;
    void* o;
    float* s_out;
    // backward
    const void* d_o;
    const float* ds_out;
    void *dq, *dk_, *dv_;
    float* ds0;
    // step
    float* state;
    int64_t nslots;
    const int64_t* slots;
    WsHeader* header;
    float* ws;  // after the header
};
bool decay_uses_tc(const DecayArgs& a);
size_t decay_ws_floats(const DecayArgs& a, bool bwd);
cudaError_t launch_decay_fwd(const DecayArgs& a, cudaStream_t s);
cudaError_t launch_decay_bwd(const DecayArgs& a, cudaStream_t s);
cudaError_t launch_decay_step(const DecayArgs& a, cudaStream_t s);

// One pass of the operator and its gradients.  With x, y of `dx` and z of `dz` values a token and head,
//   out[i] = out_scale sum over heads of y, tokens j <= i (rev: j >= i) of e^{l |i - j|} in_scale (x[i].y[j]) z[j],
// the sum over earlier tokens kept as the state sum e^{l ..} in_scale y[j] z[j]^T:
//   o  = pass(q, k, v)                     from S,              l the log decay of the state head
//   dq = pass(do, v, k)                    from S^T
//   dv = pass(k, q, do) backwards in time  from dS
//   dk = pass(v, do, q) backwards in time  from dS^T
// x has gx heads and y, z have gy heads for each state head; one of the two is 1.
// Forwards the carried state is S[t] (a token sees it decayed once), backwards it is e^l dS[t + 1], what
// the token before a sequence's first one would see: ds_out enters undecayed and ds0 leaves that way.
struct DecayPass {
    const void *x, *y, *z;
    const void* v;  // the pass of dv: what the pass of dk has for x
    void* out;
    int64_t ldx, ldy, ldz, ldv, ldout;
    int dx, dz, gx, gy;
    bool rev, transposed;  // transposed: states in memory are [dz][dx]
    bool f32, fours;       // fp32 arithmetic: the type, and whether rows allow pieces of four values
    float out_scale, in_scale;
    const float *log_decay, *init;
    float* fin;
    // Where `fin` overwrites `init`, of a packed batch of many sequences: copies of the first states of the sequences
    // that lie across the cuts between segments, [nseg - 1, Hkv, dk, dv] (null: there are none, read `init`).
    const float* kept;
    // The segments' first states, [units, nseg, dk, dv]; with `parts` (two segments of a dense batch, where the
    // one's end is the other's beginning) the sum of a unit's first `parts` entries.
    const float* recs;
    bool all_ends;  // the segments' end states are wanted of the last one too: the join leaves `fin`
    int64_t units, Hkv, seg_len;
    int nseg, parts;
    Seqs seqs;
    WsHeader* header;
};
// On the tensor cores: the segments' own end states (of a pass that is not transposed), and a pass.
cudaError_t decay_tc_ends(const DecayPass& p, float* recs, cudaStream_t s);
cudaError_t decay_tc_pass(const DecayPass& p, cudaStream_t s);
// dv and dk at once, from the pass of dv.
cudaError_t decay_tc_grads(const DecayPass& p, void* dk, int64_t lddk, cudaStream_t s);

}  // namespace lz
