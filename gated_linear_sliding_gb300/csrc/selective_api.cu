// C-ABI entry points of the selective state space block: argument checks, sizes and dispatch.
// Every check runs on the host before any launch.
#include <math.h>

#include "internal.h"
#include "selective.h"

namespace lz {
namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

template <size_t n>
bool all_aligned(const void* const (&p)[n]) {
    for (const void* q : p)
        if (q != nullptr && !aligned16(q)) return false;
    return true;
}

lizard_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return LIZARD_OK;
    cudaGetLastError();
    return LIZARD_ERR_CUDA;
}

// Largest extents, so that no product of sizes below leaves 63 bits.
constexpr int64_t kMaxExtent = (int64_t)1 << 40;
bool extent(int64_t v, int64_t lo) { return v >= lo && v <= kMaxExtent; }

// A token distance: 0 selects the dense width; a row may not overlap the next.
bool row_stride(int64_t ld, int64_t width, int64_t* out) {
    *out = ld == 0 ? width : ld;
    return *out >= width && *out <= kMaxExtent;
}

// Checks an optional workspace and returns its header.
bool header_of(void* ws, size_t bytes, WsHeader** h) {
    *h = (WsHeader*)ws;
    return ws == nullptr || (aligned16(ws) && bytes >= kHeaderBytes);
}

bool batch_ok(int64_t B, int64_t L, int64_t C, int64_t nseq) {
    if (!extent(B, 1) || !extent(L, 0) || !extent(C, 1) || nseq < 0 || nseq > kMaxExtent) return false;
    if (L > 0x7fff0000) return false;  // the kernels count a row's tokens in 32 bits
    if (nseq > 0 && B != 1) return false;
    return (double)B * (double)(L > 0 ? L : 1) * (double)C < 9e15;
}

bool dtype_ok(int t) { return t == LIZARD_F32 || t == LIZARD_BF16; }

// Grids are one-dimensional and hold up to 2^31 - 1 CTAs.
bool grid_ok(double ctas) { return ctas < 2147483647.0; }

// ---------------------------------------------------------------------------- convolution

bool conv_args(const lizard_conv_dims* d, bool step, ConvArgs* a) {
    if (d == nullptr) return false;
    const int64_t L = step ? 1 : d->L, nseq = step ? 0 : d->nseq;
    if (!batch_ok(d->B, L, d->C, nseq)) return false;
    if (d->K < 1 || d->K > 8 || !dtype_ok(d->dtype)) return false;
    if (d->act != LIZARD_ACT_NONE && d->act != LIZARD_ACT_SILU) return false;
    *a = ConvArgs{};
    if (!row_stride(d->ldx, d->C, &a->ldx) || !row_stride(d->ldy, d->C, &a->ldy) ||
        !row_stride(d->lddx, d->C, &a->lddx))
        return false;
    a->B = d->B;
    a->C = d->C;
    a->K = (int)d->K;
    a->act = d->act;
    a->dtype = d->dtype;
    a->seqs.L = L;
    a->seqs.nseq = nseq;
    a->nstate = nseq > 0 ? nseq : d->B;
    return true;
}

// CTAs of 128 threads of the largest conv launch, at one channel and eight tokens a thread.
bool conv_grid_ok(const ConvArgs& a) {
    return grid_ok(((double)a.C / 32 + 1) * ((double)a.B * (double)(a.seqs.L / 8 + 1) / 4 + 1)) &&
           grid_ok((double)a.nstate * (double)a.C * a.K / 128 + 1);
}

// ------------------------------------------------------------------------------------ scan

bool scan_args(const lizard_scan_dims* d, bool step, ScanArgs* a) {
    if (d == nullptr) return false;
    const int64_t L = step ? 1 : d->L, nseq = step ? 0 : d->nseq;
    if (!batch_ok(d->B, L, d->C, nseq) || !dtype_ok(d->dtype)) return false;
    if (d->N < 1 || d->G < 1 || d->G > d->C || d->C % d->G != 0) return false;
    *a = ScanArgs{};
    const int64_t C = d->C, GN = d->G * d->N;
    if (!row_stride(d->ldx, C, &a->ldx) || !row_stride(d->lddt, C, &a->lddt) ||
        !row_stride(d->ldz, C, &a->ldz) || !row_stride(d->ldy, C, &a->ldy) ||
        !row_stride(d->ldb, GN, &a->ldb) || !row_stride(d->ldc, GN, &a->ldc) ||
        !row_stride(d->lddx, C, &a->lddx) || !row_stride(d->ldddt, C, &a->ldddt) ||
        !row_stride(d->lddz, C, &a->lddz) || !row_stride(d->lddb, GN, &a->lddb) ||
        !row_stride(d->lddc, GN, &a->lddc))
        return false;
    a->B = d->B;
    a->C = C;
    a->N = d->N;
    a->G = d->G;
    a->dtype = d->dtype;
    a->softplus = d->softplus != 0;
    a->seqs.L = L;
    a->seqs.nseq = nseq;
    a->nstate = nseq > 0 ? nseq : d->B;
    return true;
}

// Sizes the kernels are compiled for, and grids that fit.
bool scan_compiled(const ScanArgs& a) {
    return a.N <= 64 && grid_ok((double)a.B * ((double)a.seqs.L / 64 + 1) * ((double)a.C / 8 + (double)a.G + 1)) &&
           grid_ok((double)a.nstate * (double)a.C * (double)a.N / 256 + 1) &&
           grid_ok((double)a.B * (double)(a.seqs.L + 1) * (double)a.G * 2.0 * (double)a.N / 256 + 1);
}

size_t scan_states_bytes(const ScanArgs& a) {
    return sizeof(float) * (size_t)(a.B * ((a.seqs.L + 15) / 16) * a.C * a.N);
}

// ------------------------------------------------------------------------------------ norm

bool norm_args(const lizard_norm_dims* d, NormArgs* a) {
    if (d == nullptr) return false;
    if (!extent(d->T, 0) || d->D < 1 || d->groups < 1 || d->groups > d->D || d->D % d->groups != 0) return false;
    if (!dtype_ok(d->dtype) || (d->res_dtype != d->dtype && d->res_dtype != LIZARD_F32)) return false;
    if (!(d->eps_post >= 0.0f) || !(d->eps_pre >= 0.0f) || !isfinite(d->eps_post) || !isfinite(d->eps_pre)) return false;
    if (d->act != LIZARD_ACT_NONE && d->act != LIZARD_ACT_SILU && d->act != LIZARD_ACT_SIGMOID) return false;
    *a = NormArgs{};
    const int64_t D = d->D;
    if (!row_stride(d->ldo, D, &a->ldo) || !row_stride(d->ldg, D, &a->ldg) || !row_stride(d->ldr, D, &a->ldr) ||
        !row_stride(d->ldro, D, &a->ldro) || !row_stride(d->ldn, D, &a->ldn) || !row_stride(d->lddo, D, &a->lddo) ||
        !row_stride(d->lddg, D, &a->lddg) || !row_stride(d->lddr, D, &a->lddr))
        return false;
    a->T = d->T;
    a->D = D;
    a->groups = d->groups;
    a->eps_post = d->eps_post;
    a->eps_pre = d->eps_pre;
    a->dtype = d->dtype;
    a->res_dtype = d->res_dtype;
    a->act = d->act;
    a->gate_first = d->gate_first != 0;
    return true;
}

bool norm_compiled(const NormArgs& a) { return a.D <= 16384 && grid_ok((double)a.T); }

}  // namespace
}  // namespace lz

using namespace lz;

extern "C" {

lizard_status lizard_conv_fwd(const lizard_conv_dims* dims, const void* x, const float* w,
                              const float* bias, const void* state_in, const int64_t* cu_seqlens,
                              void* y, void* state_out, void* workspace, size_t ws_bytes,
                              void* stream) {
    ConvArgs a;
    if (!conv_args(dims, false, &a)) return LIZARD_ERR_INVALID_ARG;
    if (!w || (a.seqs.L > 0 && (!x || !y)) || (a.seqs.nseq > 0 && !cu_seqlens)) return LIZARD_ERR_INVALID_ARG;
    const void* ptrs[] = {x, w, bias, state_in, y, state_out};
    if (!all_aligned(ptrs) || ((uintptr_t)cu_seqlens & 7u) != 0) return LIZARD_ERR_INVALID_ARG;
    if (workspace != nullptr && !aligned16(workspace)) return LIZARD_ERR_INVALID_ARG;
    if (!header_of(workspace, ws_bytes, &a.header)) return LIZARD_ERR_WORKSPACE;
    if (!conv_grid_ok(a)) return LIZARD_ERR_UNSUPPORTED;
    const lizard_status st = device_status();
    if (st != LIZARD_OK) return st;
    a.seqs.cu = a.seqs.nseq > 0 ? cu_seqlens : nullptr;
    a.x = x;
    a.w = w;
    a.bias = bias;
    a.state_in = state_in;
    a.y = y;
    a.state_out = state_out;
    return from_cuda(launch_conv_fwd(a, (cudaStream_t)stream));
}

size_t lizard_conv_bwd_workspace(const lizard_conv_dims* dims) {
    ConvArgs a;
    if (!conv_args(dims, false, &a)) return 0;
    return kHeaderBytes + sizeof(float) * (size_t)(conv_bwd_runs(a.B, a.seqs.L, a.C) * (a.K + 1) * a.C);
}

lizard_status lizard_conv_bwd(const lizard_conv_dims* dims, const void* x, const float* w,
                              const float* bias, const void* state_in, const int64_t* cu_seqlens,
                              const void* dy, const void* dstate_out, void* dx, float* dw,
                              float* dbias, void* dstate_in, void* workspace, size_t ws_bytes,
                              void* stream) {
    ConvArgs a;
    if (!conv_args(dims, false, &a)) return LIZARD_ERR_INVALID_ARG;
    if (!w || !dw || (a.seqs.L > 0 && (!x || !dy || !dx)) || (a.seqs.nseq > 0 && !cu_seqlens)) return LIZARD_ERR_INVALID_ARG;
    if ((bias == nullptr) != (dbias == nullptr)) return LIZARD_ERR_INVALID_ARG;
    const void* ptrs[] = {x, w, bias, state_in, dy, dstate_out, dx, dw, dbias, dstate_in, workspace};
    if (!all_aligned(ptrs) || ((uintptr_t)cu_seqlens & 7u) != 0) return LIZARD_ERR_INVALID_ARG;
    if (workspace == nullptr || ws_bytes < lizard_conv_bwd_workspace(dims)) return LIZARD_ERR_WORKSPACE;
    if (!conv_grid_ok(a)) return LIZARD_ERR_UNSUPPORTED;
    const lizard_status st = device_status();
    if (st != LIZARD_OK) return st;
    a.seqs.cu = a.seqs.nseq > 0 ? cu_seqlens : nullptr;
    a.x = x;
    a.w = w;
    a.bias = bias;
    a.state_in = state_in;
    a.dy = dy;
    a.dstate_out = dstate_out;
    a.dx = dx;
    a.dw = dw;
    a.dbias = dbias;
    a.dstate_in = dstate_in;
    a.header = (WsHeader*)workspace;
    a.partial = (float*)((char*)workspace + kHeaderBytes);
    return from_cuda(launch_conv_bwd(a, (cudaStream_t)stream));
}

lizard_status lizard_conv_step(const lizard_conv_dims* dims, const void* x, const float* w,
                               const float* bias, void* state, int64_t nslots,
                               const int64_t* slots, void* y, void* workspace, size_t ws_bytes,
                               void* stream) {
    ConvArgs a;
    if (!conv_args(dims, true, &a)) return LIZARD_ERR_INVALID_ARG;
    if (!x || !w || !y || (a.K > 1 && !state)) return LIZARD_ERR_INVALID_ARG;
    if (!extent(nslots, 0) || (slots == nullptr && nslots < a.B)) return LIZARD_ERR_INVALID_ARG;
    const void* ptrs[] = {x, w, bias, state, y};
    if (!all_aligned(ptrs) || ((uintptr_t)slots & 7u) != 0) return LIZARD_ERR_INVALID_ARG;
    if (workspace != nullptr && !aligned16(workspace)) return LIZARD_ERR_INVALID_ARG;
    if (!header_of(workspace, ws_bytes, &a.header)) return LIZARD_ERR_WORKSPACE;
    if (!conv_grid_ok(a)) return LIZARD_ERR_UNSUPPORTED;
    const lizard_status st = device_status();
    if (st != LIZARD_OK) return st;
    a.x = x;
    a.w = w;
    a.bias = bias;
    a.y = y;
    a.state = state;
    a.nslots = nslots;
    a.slots = slots;
    return from_cuda(launch_conv_step(a, (cudaStream_t)stream));
}

size_t lizard_scan_fwd_workspace(const lizard_scan_dims* dims) {
    ScanArgs a;
    if (!scan_args(dims, false, &a) || !scan_compiled(a)) return 0;
    return kHeaderBytes + sizeof(float) * scan_fwd_ws_floats(a);
}

size_t lizard_scan_states_bytes(const lizard_scan_dims* dims) {
    ScanArgs a;
    return scan_args(dims, false, &a) && scan_compiled(a) ? scan_states_bytes(a) : 0;
}

lizard_status lizard_scan_fwd(const lizard_scan_dims* dims, const void* x, const void* dt,
                              const float* A, const void* Bm, const void* Cm, const float* D,
                              const void* z, const float* dt_bias, const float* h0,
                              const int64_t* cu_seqlens, void* y, float* h_out, void* states,
                              void* workspace, size_t ws_bytes, void* stream) {
    ScanArgs a;
    if (!scan_args(dims, false, &a)) return LIZARD_ERR_INVALID_ARG;
    if (!A || (a.seqs.L > 0 && (!x || !dt || !Bm || !Cm || !y)) || (a.seqs.nseq > 0 && !cu_seqlens))
        return LIZARD_ERR_INVALID_ARG;
    const void* ptrs[] = {x, dt, A, Bm, Cm, D, z, dt_bias, h0, y, h_out, states, workspace};
    if (!all_aligned(ptrs) || ((uintptr_t)cu_seqlens & 7u) != 0) return LIZARD_ERR_INVALID_ARG;
    if (!scan_compiled(a)) return LIZARD_ERR_UNSUPPORTED;
    if (workspace == nullptr || ws_bytes < lizard_scan_fwd_workspace(dims)) return LIZARD_ERR_WORKSPACE;
    const lizard_status st = device_status();
    if (st != LIZARD_OK) return st;
    a.seqs.cu = a.seqs.nseq > 0 ? cu_seqlens : nullptr;
    a.x = x;
    a.dt = dt;
    a.A = A;
    a.Bm = Bm;
    a.Cm = Cm;
    a.D = D;
    a.z = z;
    a.dt_bias = dt_bias;
    a.h0 = h0;
    a.y = y;
    a.h_out = h_out;
    a.states = (float*)states;
    a.header = (WsHeader*)workspace;
    a.ws = (float*)((char*)workspace + kHeaderBytes);
    return from_cuda(launch_scan_fwd(a, (cudaStream_t)stream));
}

size_t lizard_scan_bwd_workspace(const lizard_scan_dims* dims) {
    ScanArgs a;
    if (!scan_args(dims, false, &a) || !scan_compiled(a)) return 0;
    return kHeaderBytes + sizeof(float) * scan_bwd_ws_floats(a);
}

lizard_status lizard_scan_bwd(const lizard_scan_dims* dims, const void* x, const void* dt,
                              const float* A, const void* Bm, const void* Cm, const float* D,
                              const void* z, const float* dt_bias, const float* h0,
                              const int64_t* cu_seqlens, const void* states, const void* dy,
                              const float* dh_out, void* dx, void* ddt, void* dz, void* dBm,
                              void* dCm, float* dA, float* dD, float* ddt_bias, float* dh0,
                              void* workspace, size_t ws_bytes, void* stream) {
    ScanArgs a;
    if (!scan_args(dims, false, &a)) return LIZARD_ERR_INVALID_ARG;
    if (!A || !dA || (a.seqs.nseq > 0 && !cu_seqlens)) return LIZARD_ERR_INVALID_ARG;
    if (a.seqs.L > 0 && (!x || !dt || !Bm || !Cm || !states || !dy || !dx || !ddt || !dBm || !dCm))
        return LIZARD_ERR_INVALID_ARG;
    if ((a.seqs.L > 0 && (z == nullptr) != (dz == nullptr)) || (D == nullptr) != (dD == nullptr) ||
        (dt_bias == nullptr) != (ddt_bias == nullptr))
        return LIZARD_ERR_INVALID_ARG;
    const void* ptrs[] = {x, dt, A, Bm, Cm, D, z, dt_bias, h0, states, dy, dh_out,
                          dx, ddt, dz, dBm, dCm, dA, dD, ddt_bias, dh0, workspace};
    if (!all_aligned(ptrs) || ((uintptr_t)cu_seqlens & 7u) != 0) return LIZARD_ERR_INVALID_ARG;
    if (!scan_compiled(a)) return LIZARD_ERR_UNSUPPORTED;
    if (workspace == nullptr || ws_bytes < lizard_scan_bwd_workspace(dims)) return LIZARD_ERR_WORKSPACE;
    const lizard_status st = device_status();
    if (st != LIZARD_OK) return st;
    a.seqs.cu = a.seqs.nseq > 0 ? cu_seqlens : nullptr;
    a.x = x;
    a.dt = dt;
    a.A = A;
    a.Bm = Bm;
    a.Cm = Cm;
    a.D = D;
    a.z = z;
    a.dt_bias = dt_bias;
    a.h0 = h0;
    a.states = (float*)states;
    a.dy = dy;
    a.dh_out = dh_out;
    a.dx = dx;
    a.ddt = ddt;
    a.dz = dz;
    a.dBm = dBm;
    a.dCm = dCm;
    a.dA = dA;
    a.dD = dD;
    a.ddt_bias = ddt_bias;
    a.dh0 = dh0;
    a.header = (WsHeader*)workspace;
    a.ws = (float*)((char*)workspace + kHeaderBytes);
    return from_cuda(launch_scan_bwd(a, (cudaStream_t)stream));
}

lizard_status lizard_scan_step(const lizard_scan_dims* dims, const void* x, const void* dt,
                               const float* A, const void* Bm, const void* Cm, const float* D,
                               const void* z, const float* dt_bias, float* state, int64_t nslots,
                               const int64_t* slots, void* y, void* workspace, size_t ws_bytes,
                               void* stream) {
    ScanArgs a;
    if (!scan_args(dims, true, &a)) return LIZARD_ERR_INVALID_ARG;
    if (!x || !dt || !A || !Bm || !Cm || !state || !y) return LIZARD_ERR_INVALID_ARG;
    if (!extent(nslots, 0) || (slots == nullptr && nslots < a.B)) return LIZARD_ERR_INVALID_ARG;
    const void* ptrs[] = {x, dt, A, Bm, Cm, D, z, dt_bias, state, y};
    if (!all_aligned(ptrs) || ((uintptr_t)slots & 7u) != 0) return LIZARD_ERR_INVALID_ARG;
    if (workspace != nullptr && !aligned16(workspace)) return LIZARD_ERR_INVALID_ARG;
    if (!header_of(workspace, ws_bytes, &a.header)) return LIZARD_ERR_WORKSPACE;
    if (!scan_compiled(a)) return LIZARD_ERR_UNSUPPORTED;
    const lizard_status st = device_status();
    if (st != LIZARD_OK) return st;
    a.x = x;
    a.dt = dt;
    a.A = A;
    a.Bm = Bm;
    a.Cm = Cm;
    a.D = D;
    a.z = z;
    a.dt_bias = dt_bias;
    a.y = y;
    a.state = state;
    a.nslots = nslots;
    a.slots = slots;
    return from_cuda(launch_scan_step(a, (cudaStream_t)stream));
}

lizard_status lizard_block_norm_fwd(const lizard_norm_dims* dims, const void* o, const void* gate,
                                    const void* r, const float* w_post, const float* scale,
                                    const float* w_pre, void* r_out, void* n_out, void* stream) {
    NormArgs a;
    if (!norm_args(dims, &a)) return LIZARD_ERR_INVALID_ARG;
    if (a.T > 0 && !o) return LIZARD_ERR_INVALID_ARG;
    if ((!r_out && !n_out) || (n_out == nullptr) != (w_pre == nullptr)) return LIZARD_ERR_INVALID_ARG;
    if (gate != nullptr && a.act == LIZARD_ACT_NONE) return LIZARD_ERR_INVALID_ARG;
    const void* ptrs[] = {o, gate, r, w_post, scale, w_pre, r_out, n_out};
    if (!all_aligned(ptrs)) return LIZARD_ERR_INVALID_ARG;
    if (!norm_compiled(a)) return LIZARD_ERR_UNSUPPORTED;
    const lizard_status st = device_status();
    if (st != LIZARD_OK) return st;
    if (a.T == 0) return LIZARD_OK;
    a.o = o;
    a.gate = gate;
    a.r = r;
    a.w_post = w_post;
    a.scale = scale;
    a.w_pre = w_pre;
    a.r_out = r_out;
    a.n_out = n_out;
    return from_cuda(launch_norm_fwd(a, (cudaStream_t)stream));
}

size_t lizard_block_norm_bwd_workspace(const lizard_norm_dims* dims) {
    NormArgs a;
    if (!norm_args(dims, &a)) return 0;
    return kHeaderBytes + sizeof(float) * (size_t)(norm_bwd_ctas(a.T, a.D) * 3 * a.D);
}

lizard_status lizard_block_norm_bwd(const lizard_norm_dims* dims, const void* o, const void* gate,
                                    const void* r, const float* w_post, const float* scale,
                                    const float* w_pre, const void* dr_out, const void* dn_out,
                                    void* d_o, void* dgate, void* dr, float* dw_post,
                                    float* dscale, float* dw_pre, void* workspace,
                                    size_t ws_bytes, void* stream) {
    NormArgs a;
    if (!norm_args(dims, &a)) return LIZARD_ERR_INVALID_ARG;
    if (a.T > 0 && (!o || !d_o)) return LIZARD_ERR_INVALID_ARG;
    if (a.T > 0 && ((!dr_out && !dn_out) || (dn_out == nullptr) != (w_pre == nullptr) ||
                    (gate == nullptr) != (dgate == nullptr)))
        return LIZARD_ERR_INVALID_ARG;
    if ((w_post == nullptr) != (dw_post == nullptr) || (scale == nullptr) != (dscale == nullptr) ||
        (w_pre == nullptr) != (dw_pre == nullptr))
        return LIZARD_ERR_INVALID_ARG;
    if (gate != nullptr && a.act == LIZARD_ACT_NONE) return LIZARD_ERR_INVALID_ARG;
    const void* ptrs[] = {o, gate, r, w_post, scale, w_pre, dr_out, dn_out, d_o, dgate, dr,
                          dw_post, dscale, dw_pre, workspace};
    if (!all_aligned(ptrs)) return LIZARD_ERR_INVALID_ARG;
    if (!norm_compiled(a)) return LIZARD_ERR_UNSUPPORTED;
    if (workspace == nullptr || ws_bytes < lizard_block_norm_bwd_workspace(dims)) return LIZARD_ERR_WORKSPACE;
    const lizard_status st = device_status();
    if (st != LIZARD_OK) return st;
    a.o = o;
    a.gate = gate;
    a.r = r;
    a.w_post = w_post;
    a.scale = scale;
    a.w_pre = w_pre;
    a.dr_out = dr_out;
    a.dn_out = dn_out;
    a.d_o = d_o;
    a.dgate = dgate;
    a.dr = dr;
    a.dw_post = dw_post;
    a.dscale = dscale;
    a.dw_pre = dw_pre;
    a.partial = (float*)((char*)workspace + kHeaderBytes);
    return from_cuda(launch_norm_bwd(a, (cudaStream_t)stream));
}

}  // extern "C"
