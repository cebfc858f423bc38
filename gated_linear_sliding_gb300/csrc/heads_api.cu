// C-ABI entry points of the query and key rotation and of the linear attention with a decay for each
// head: argument checks, sizes and dispatch.  Every check runs on the host before any launch.
#include <math.h>

#include "checks.h"
#include "heads.h"

namespace lz {
namespace {

// -------------------------------------------------------------------------------- rotation

bool rope_args(const lizard_rope_dims* d, RopeArgs* a) {
    if (d == nullptr || !dtype_ok(d->dtype)) return false;
    if (d->Hq < 1 || d->Hkv < 0 || d->Hq > kMaxExtent || d->Hkv > kMaxExtent || d->d < 1 || d->d > kMaxExtent) return false;
    if (!batch_ok(d->B, d->L, d->d, 0) || (double)d->B * (double)(d->L + 1) * (double)(d->Hq + d->Hkv) * (double)d->d > 9e15)
        return false;
    if (d->rot < 0 || d->rot > d->d || d->rot % 2 != 0 || d->axes < 1 || d->axes > 4) return false;
    if (!(d->eps >= 0.0f) || !isfinite(d->eps)) return false;
    *a = RopeArgs{};
    int64_t sum = 0;
    for (int i = 0; i < 4; ++i) {
        if (d->axes > 1 && i < d->axes) {
            if (d->section[i] < 0 || d->section[i] > d->rot) return false;
            sum += d->section[i];
        }
        a->section[i] = d->axes > 1 && i < d->axes ? (int)(sum < (1 << 30) ? sum : 1 << 30) : 1 << 30;
    }
    if (d->axes > 1 && sum != d->rot / 2) return false;
    const int64_t wq = d->Hq * d->d, wk = d->Hkv * d->d;
    if (!row_stride(d->ldq, wq, &a->ldq) || !row_stride(d->ldqo, wq, &a->ldqo) || !row_stride(d->lddq, wq, &a->lddq) ||
        !row_stride(d->ldk, wk, &a->ldk) || !row_stride(d->ldko, wk, &a->ldko) || !row_stride(d->lddk, wk, &a->lddk))
        return false;
    a->B = d->B;
    a->L = d->L;
    a->Hq = d->Hq;
    a->Hkv = d->Hkv;
    a->d = (int)d->d;  // of sizes that rope_compiled refuses nothing else is read
    a->rot = (int)d->rot;
    a->axes = (int)d->axes;
    a->start = d->start;
    a->eps = d->eps;
    a->dtype = d->dtype;
    a->norm = d->norm != 0;
    a->neighbours = d->neighbours != 0;
    return true;
}

// Heads the kernels are compiled for, counted in 32 bits (asked of the caller's sizes, which have 64).
bool rope_compiled(const lizard_rope_dims& d) { return d.d <= 512 && d.Hq + d.Hkv <= 1 << 24; }

bool rope_params(const RopeArgs& a, const float* w_q, const float* w_k, const float* freqs) {
    return (a.norm || (w_q == nullptr && w_k == nullptr)) && (w_k == nullptr || a.Hkv > 0) && (a.rot == 0 || freqs != nullptr);
}

// ---------------------------------------------------------------------------------- decays

bool decay_args(const lizard_decay_dims* d, bool step, DecayArgs* a) {
    if (d == nullptr || !dtype_ok(d->dtype)) return false;
    const int64_t L = step ? 1 : d->L, nseq = step ? 0 : d->nseq;
    if (!extent(d->Hq, 1) || !extent(d->Hkv, 1) || d->Hq % d->Hkv != 0 || !extent(d->dk, 1) || !extent(d->dv, 1)) return false;
    const int64_t wide = d->dk > d->dv ? d->dk : d->dv;
    if (!batch_ok(d->B, L, wide, nseq) || !isfinite(d->scale)) return false;
    const double rows = (double)d->B * (double)(L + 1), states = (double)(nseq > d->B ? nseq : d->B) * (double)d->Hkv;
    if (rows * (double)d->Hq * (double)wide > 9e15 || states * (double)d->dk * (double)d->dv > 9e15) return false;
    *a = DecayArgs{};
    const int64_t wq = d->Hq * d->dk, wk = d->Hkv * d->dk, wv = d->Hkv * d->dv, wo = d->Hq * d->dv;
    if (!row_stride(d->ldq, wq, &a->ldq) || !row_stride(d->ldk, wk, &a->ldk) || !row_stride(d->ldv, wv, &a->ldv) ||
        !row_stride(d->ldo, wo, &a->ldo) || !row_stride(d->lddq, wq, &a->lddq) || !row_stride(d->lddk, wk, &a->lddk) ||
        !row_stride(d->lddv, wv, &a->lddv))
        return false;
    a->B = d->B;
    a->Hq = d->Hq;
    a->Hkv = d->Hkv;
    a->dk = d->dk;
    a->dv = d->dv;
    a->scale = d->scale;
    a->dtype = d->dtype;
    a->seqs.L = L;
    a->seqs.nseq = nseq;
    a->nstate = nseq > 0 ? nseq : d->B;
    return true;
}

// Sizes the kernels are compiled for, and grids that fit.
bool decay_compiled(const DecayArgs& a) {
    return a.dk <= 192 && a.dv <= 192 && a.Hq / a.Hkv <= 1 << 16 && grid_ok((double)a.B * (double)a.Hkv * 1024.0) &&
           grid_ok((double)a.nstate * (double)a.Hkv * 64.0);
}

}  // namespace
}  // namespace lz

using namespace lz;

extern "C" {

lizard_status lizard_qk_rope_fwd(const lizard_rope_dims* dims, const void* q, const void* k,
                                 const float* w_q, const float* w_k, const float* freqs,
                                 const int64_t* positions, void* q_out, void* k_out, void* stream) {
    RopeArgs a;
    if (!rope_args(dims, &a)) return LIZARD_ERR_INVALID_ARG;
    const bool some = a.L > 0;
    if ((some && (!q || !q_out)) || (some && a.Hkv > 0 && (!k || !k_out)) || !rope_params(a, w_q, w_k, freqs) ||
        (a.axes > 1 && some && !positions))
        return LIZARD_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, w_q, w_k, freqs, q_out, k_out};
    if (!all_aligned(ptrs) || ((uintptr_t)positions & 7u) != 0) return LIZARD_ERR_INVALID_ARG;
    if (!rope_compiled(*dims)) return LIZARD_ERR_UNSUPPORTED;
    const lizard_status st = device_status();
    if (st != LIZARD_OK) return st;
    if (!some) return LIZARD_OK;
    a.q = q;
    a.k = k;
    a.w_q = w_q;
    a.w_k = w_k;
    a.freqs = freqs;
    a.positions = positions;
    a.q_out = q_out;
    a.k_out = k_out;
    return from_cuda(launch_rope_fwd(a, (cudaStream_t)stream));
}

size_t lizard_qk_rope_bwd_workspace(const lizard_rope_dims* dims) {
    RopeArgs a;
    if (!rope_args(dims, &a) || !rope_compiled(*dims)) return 0;
    return kHeaderBytes + sizeof(float) * (size_t)(rope_bwd_ctas(a) * 2 * a.d);
}

lizard_status lizard_qk_rope_bwd(const lizard_rope_dims* dims, const void* q, const void* k,
                                 const float* w_q, const float* w_k, const float* freqs,
                                 const int64_t* positions, const void* dq_out, const void* dk_out,
                                 void* dq, void* dk, float* dw_q, float* dw_k, void* workspace,
                                 size_t ws_bytes, void* stream) {
    RopeArgs a;
    if (!rope_args(dims, &a)) return LIZARD_ERR_INVALID_ARG;
    const bool some = a.L > 0;
    if ((some && (!dq_out || !dq || (a.norm && !q))) || (some && a.Hkv > 0 && (!dk_out || !dk || (a.norm && !k))) ||
        !rope_params(a, w_q, w_k, freqs) || (a.axes > 1 && some && !positions))
        return LIZARD_ERR_INVALID_ARG;
    if ((w_q == nullptr) != (dw_q == nullptr) || (w_k == nullptr) != (dw_k == nullptr)) return LIZARD_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, w_q, w_k, freqs, dq_out, dk_out, dq, dk, dw_q, dw_k, workspace};
    if (!all_aligned(ptrs) || ((uintptr_t)positions & 7u) != 0) return LIZARD_ERR_INVALID_ARG;
    if (!rope_compiled(*dims)) return LIZARD_ERR_UNSUPPORTED;
    if (workspace == nullptr || ws_bytes < lizard_qk_rope_bwd_workspace(dims)) return LIZARD_ERR_WORKSPACE;
    const lizard_status st = device_status();
    if (st != LIZARD_OK) return st;
    a.q = q;
    a.k = k;
    a.w_q = w_q;
    a.w_k = w_k;
    a.freqs = freqs;
    a.positions = positions;
    a.dq_out = dq_out;
    a.dk_out = dk_out;
    a.dq = dq;
    a.dk = dk;
    a.dw_q = dw_q;
    a.dw_k = dw_k;
    a.partial = (float*)((char*)workspace + kHeaderBytes);
    return from_cuda(launch_rope_bwd(a, (cudaStream_t)stream));
}

int lizard_decay_attn_kernel(const lizard_decay_dims* dims) {
    DecayArgs a;
    return !decay_args(dims, false, &a) || !decay_compiled(a) ? -1 : decay_uses_tc(a) ? 1 : 0;
}

size_t lizard_decay_attn_fwd_workspace(const lizard_decay_dims* dims) {
    DecayArgs a;
    if (!decay_args(dims, false, &a) || !decay_compiled(a)) return 0;
    return kHeaderBytes + sizeof(float) * decay_ws_floats(a, false);
}

lizard_status lizard_decay_attn_fwd(const lizard_decay_dims* dims, const void* q, const void* k,
                                    const void* v, const float* log_decay, const float* s0,
                                    const int64_t* cu_seqlens, void* o, float* s_out,
                                    void* workspace, size_t ws_bytes, void* stream) {
    DecayArgs a;
    if (!decay_args(dims, false, &a)) return LIZARD_ERR_INVALID_ARG;
    if (!log_decay || (a.seqs.L > 0 && (!q || !k || !v || !o)) || (a.seqs.nseq > 0 && !cu_seqlens)) return LIZARD_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, log_decay, s0, o, s_out, workspace};
    if (!all_aligned(ptrs) || ((uintptr_t)cu_seqlens & 7u) != 0) return LIZARD_ERR_INVALID_ARG;
    if (!decay_compiled(a)) return LIZARD_ERR_UNSUPPORTED;
    if (workspace == nullptr || ws_bytes < lizard_decay_attn_fwd_workspace(dims)) return LIZARD_ERR_WORKSPACE;
    const lizard_status st = device_status();
    if (st != LIZARD_OK) return st;
    a.seqs.cu = a.seqs.nseq > 0 ? cu_seqlens : nullptr;
    a.q = q;
    a.k = k;
    a.v = v;
    a.log_decay = log_decay;
    a.s0 = s0;
    a.o = o;
    a.s_out = s_out;
    a.header = (WsHeader*)workspace;
    a.ws = (float*)((char*)workspace + kHeaderBytes);
    return from_cuda(launch_decay_fwd(a, (cudaStream_t)stream));
}

size_t lizard_decay_attn_bwd_workspace(const lizard_decay_dims* dims) {
    DecayArgs a;
    if (!decay_args(dims, false, &a) || !decay_compiled(a)) return 0;
    return kHeaderBytes + sizeof(float) * decay_ws_floats(a, true);
}

lizard_status lizard_decay_attn_bwd(const lizard_decay_dims* dims, const void* q, const void* k,
                                    const void* v, const float* log_decay, const float* s0,
                                    const int64_t* cu_seqlens, const void* d_o, const float* ds_out,
                                    void* dq, void* dk, void* dv, float* ds0, void* workspace,
                                    size_t ws_bytes, void* stream) {
    DecayArgs a;
    if (!decay_args(dims, false, &a)) return LIZARD_ERR_INVALID_ARG;
    if (!log_decay || (a.seqs.L > 0 && (!q || !k || !v || !d_o || !dq || !dk || !dv)) || (a.seqs.nseq > 0 && !cu_seqlens))
        return LIZARD_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, log_decay, s0, d_o, ds_out, dq, dk, dv, ds0, workspace};
    if (!all_aligned(ptrs) || ((uintptr_t)cu_seqlens & 7u) != 0) return LIZARD_ERR_INVALID_ARG;
    if (!decay_compiled(a)) return LIZARD_ERR_UNSUPPORTED;
    if (workspace == nullptr || ws_bytes < lizard_decay_attn_bwd_workspace(dims)) return LIZARD_ERR_WORKSPACE;
    const lizard_status st = device_status();
    if (st != LIZARD_OK) return st;
    a.seqs.cu = a.seqs.nseq > 0 ? cu_seqlens : nullptr;
    a.q = q;
    a.k = k;
    a.v = v;
    a.log_decay = log_decay;
    a.s0 = s0;
    a.d_o = d_o;
    a.ds_out = ds_out;
    a.dq = dq;
    a.dk_ = dk;
    a.dv_ = dv;
    a.ds0 = ds0;
    a.header = (WsHeader*)workspace;
    a.ws = (float*)((char*)workspace + kHeaderBytes);
    return from_cuda(launch_decay_bwd(a, (cudaStream_t)stream));
}

lizard_status lizard_decay_attn_step(const lizard_decay_dims* dims, const void* q, const void* k,
                                     const void* v, const float* log_decay, float* state,
                                     int64_t nslots, const int64_t* slots, void* o,
                                     void* workspace, size_t ws_bytes, void* stream) {
    DecayArgs a;
    if (!decay_args(dims, true, &a)) return LIZARD_ERR_INVALID_ARG;
    if (!q || !k || !v || !log_decay || !state || !o) return LIZARD_ERR_INVALID_ARG;
    if (!extent(nslots, 0) || (slots == nullptr && nslots < a.B)) return LIZARD_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, log_decay, state, o};
    if (!all_aligned(ptrs) || ((uintptr_t)slots & 7u) != 0) return LIZARD_ERR_INVALID_ARG;
    if (workspace != nullptr && !aligned16(workspace)) return LIZARD_ERR_INVALID_ARG;
    if (!header_of(workspace, ws_bytes, &a.header)) return LIZARD_ERR_WORKSPACE;
    if (!decay_compiled(a)) return LIZARD_ERR_UNSUPPORTED;
    const lizard_status st = device_status();
    if (st != LIZARD_OK) return st;
    a.q = q;
    a.k = k;
    a.v = v;
    a.log_decay = log_decay;
    a.o = o;
    a.state = state;
    a.nslots = nslots;
    a.slots = slots;
    return from_cuda(launch_decay_step(a, (cudaStream_t)stream));
}

}  // extern "C"
