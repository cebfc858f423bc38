// The short causal depthwise convolution (lizard_conv_*): forward, single-token step, backward.
//
//   pre[t, c] = bias[c] + sum_{j < K} w[c, j] x[t - K + 1 + j, c],   y = act(pre).
//
// Every kernel is one pass over the rows: a thread owns V neighbouring channels, walks a run of
// tokens with the last K - 1 inputs in registers, and reads each input row once (plus K - 1 rows
// of halo a run).
#include <type_traits>

#include "selective.h"

namespace lz {
namespace {

constexpr int kNT = 128;

// The K - 1 inputs before token t of its sequence, from the row or the sequence's state.
template <typename T, int K, int V>
__device__ __forceinline__ void load_window(const ConvArgs& a, const SeqAt& q, int64_t row0,
                                            int64_t t, int64_t c, float (*win)[V]) {
    const T* x = (const T*)a.x;
    const T* st = (const T*)a.state_in;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int64_t u = t - (K - 1) + j;  // token of win[j]
        if (u >= q.begin) Vec<V>::ld(x + (row0 + u) * a.ldx + c, win[j]);
        else if (st != nullptr) Vec<V>::ld(st + (q.seq * (K - 1) + (K - 1) + u - q.begin) * a.C + c, win[j]);
        else {
#pragma unroll
            for (int i = 0; i < V; ++i) win[j][i] = 0.0f;
        }
    }
}

template <int K, int V>
__device__ __forceinline__ void load_taps(const ConvArgs& a, int64_t c, float (*w)[V], float* bias) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < K; ++j) w[j][i] = a.w[(c + i) * K + j];
        bias[i] = a.bias != nullptr ? a.bias[c + i] : 0.0f;
    }
}

// The last K - 1 inputs of sequence q (of batch row b), read whole before any is written so that
// state_out may be state_in.
template <typename T, int K, int V>
__device__ __forceinline__ void write_tail(const ConvArgs& a, int64_t q, int64_t c) {
    int64_t end;
    const int64_t n = seq_tokens(a.seqs, q, &end);
    const int64_t row0 = a.seqs.cu == nullptr ? q * a.seqs.L : 0;
    const T* st = (const T*)a.state_in;
    float v[K - 1][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int64_t u = n - (K - 1) + j;  // place in the sequence
        if (u >= 0) Vec<V>::ld((const T*)a.x + (row0 + end - (K - 1) + j) * a.ldx + c, v[j]);
        else if (st != nullptr) Vec<V>::ld(st + (q * (K - 1) + (K - 1) + u) * a.C + c, v[j]);
        else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[j][i] = 0.0f;
        }
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j) Vec<V>::st((T*)a.state_out + (q * (K - 1) + j) * a.C + c, v[j]);
}

template <typename T, int K, int V>
__global__ void __launch_bounds__(kNT) conv_tail_kernel(const ConvArgs a) {
    const int64_t nv = a.C / V, id = (int64_t)blockIdx.x * kNT + threadIdx.x;
    if constexpr (K > 1) {
        if (id < a.nstate * nv) write_tail<T, K, V>(a, id / nv, id % nv * V);
    }
}

// One thread: V channels, `run` tokens of one row of the batch.  Bound by HBM: x is read and y
// written once; U rows are in flight per thread.
template <typename T, int K, int V>
__global__ void __launch_bounds__(kNT) conv_fwd_kernel(const ConvArgs a, int64_t runs, int run) {
    constexpr int U = 4;
    const bool silu = a.act == LIZARD_ACT_SILU;
    const int64_t nv = a.C / V, id = (int64_t)blockIdx.x * kNT + threadIdx.x;
    check_offsets(a.seqs, a.header);
    if (id >= a.B * runs * nv) return;
    const int64_t c = id % nv * V, rr = id / nv, b = rr / runs;
    const int64_t t0 = rr % runs * run, t1 = min64(t0 + run, a.seqs.L), row0 = b * a.seqs.L;
    float w[K][V], bias[V], win[K][V];
    load_taps<K, V>(a, c, w, bias);
    SeqAt q = seq_at(a.seqs, b, t0);
    load_window<T, K, V>(a, q, row0, t0, c, win);
    const T* x = (const T*)a.x + row0 * a.ldx + c;
    T* y = (T*)a.y + row0 * a.ldy + c;
    for (int64_t t = t0; t < t1; t += U) {
        float in[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u < t1) Vec<V>::ld(x + (t + u) * a.ldx, in[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= t1) break;
            if (t + u == q.end) {
                q = seq_at(a.seqs, b, t + u);
                load_window<T, K, V>(a, q, row0, t + u, c, win);
            }
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                win[K - 1][i] = in[u][i];
                float p = bias[i];
#pragma unroll
                for (int j = 0; j < K; ++j) p = fmaf(w[j][i], win[j][i], p);
                o[i] = silu ? p * sigm<is_fast<T>()>(p) : p;
#pragma unroll
                for (int j = 0; j + 1 < K; ++j) win[j][i] = win[j + 1][i];
            }
            Vec<V>::st(y + (t + u) * a.ldy, o);
        }
    }
}

// One token a sequence: the state's K - 1 rows are read, moved up by one and written back.
template <typename T, int K, int V>
__global__ void __launch_bounds__(kNT) conv_step_kernel(const ConvArgs a) {
    const bool silu = a.act == LIZARD_ACT_SILU;
    const int64_t nv = a.C / V, id = (int64_t)blockIdx.x * kNT + threadIdx.x;
    if (id >= a.B * nv) return;
    const int64_t c = id % nv * V, b = id / nv;
    int64_t slot = a.slots != nullptr ? a.slots[b] : b;
    T* y = (T*)a.y + b * a.ldy + c;
    float o[V];
    if (slot < 0 || slot >= a.nslots) {
        if (slot >= 0) report(a.header, LIZARD_ERR_INVALID_ARG, 33);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = 0.0f;
        Vec<V>::st(y, o);
        return;
    }
    float w[K][V], bias[V], win[K][V];
    T* st = (T*)a.state + slot * (K - 1) * a.C + c;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) Vec<V>::ld(st + j * a.C, win[j]);
    Vec<V>::ld((const T*)a.x + b * a.ldx + c, win[K - 1]);
    load_taps<K, V>(a, c, w, bias);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float p = bias[i];
#pragma unroll
        for (int j = 0; j < K; ++j) p = fmaf(w[j][i], win[j][i], p);
        o[i] = silu ? p * sigm<is_fast<T>()>(p) : p;
    }
    Vec<V>::st(y, o);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) Vec<V>::st(st + j * a.C, win[j + 1]);
}

// Backward, one thread: V channels, the tokens [t0, t1) of a run.  Walking forward, token t gives
// dp = dy act'(pre), which adds w[j] dp to the gradient of token t - K + 1 + j; acc[j] holds
// those sums, and the oldest is complete once t has been added.  The walk goes K - 1 tokens past
// the run (or to the sequence's end) to complete the run's own last tokens.  Places before a
// sequence's first token are its state, whose gradient is written by the run that holds that
// token.
template <typename T, int K, int V>
__global__ void __launch_bounds__(kNT) conv_bwd_kernel(const ConvArgs a, int64_t runs, int run) {
    constexpr int U = 4;
    const bool silu = a.act == LIZARD_ACT_SILU;
    const int64_t nv = a.C / V, id = (int64_t)blockIdx.x * kNT + threadIdx.x;
    check_offsets(a.seqs, a.header);
    if (id >= a.B * runs * nv) return;
    const int64_t c = id % nv * V, rr = id / nv, b = rr / runs;
    const int64_t t0 = rr % runs * run, t1 = min64(t0 + run, a.seqs.L), row0 = b * a.seqs.L;
    float w[K][V], bias[V], win[K][V], acc[K][V], dw[K][V], db[V];
    load_taps<K, V>(a, c, w, bias);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j) dw[j][i] = acc[j][i] = 0.0f;
    }
    const T* x = (const T*)a.x + row0 * a.ldx + c;
    const T* dy = (const T*)a.dy + row0 * a.ldy + c;
    T* dx = (T*)a.dx + row0 * a.lddx + c;
    SeqAt q = seq_at(a.seqs, b, t0);
    load_window<T, K, V>(a, q, row0, t0, c, win);
    // the gradient of token u (or of a place before the sequence's first token)
    auto put = [&](int64_t u, const float* v) {
        if (u >= q.begin) {
            if (u >= t0 && u < t1) Vec<V>::st(dx + u * a.lddx, v);
        } else if (a.dstate_in != nullptr && q.begin >= t0 && q.begin < t1) {
            Vec<V>::st((T*)a.dstate_in + (q.seq * (K - 1) + (K - 1) + u - q.begin) * a.C + c, v);
        }
    };
    int64_t t = t0;
    while (true) {
        const int64_t lim = min64(q.end, t1 + K - 1);
        for (; t < lim; t += U) {
            float in[U][V], g[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u < lim) {
                    Vec<V>::ld(x + (t + u) * a.ldx, in[u]);
                    Vec<V>::ld(dy + (t + u) * a.ldy, g[u]);
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u >= lim) break;
                const float own = t + u < t1 ? 1.0f : 0.0f;  // the halo belongs to the next run
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    win[K - 1][i] = in[u][i];
                    float dp = g[u][i];
                    if (silu) {
                        float p = bias[i];
#pragma unroll
                        for (int j = 0; j < K; ++j) p = fmaf(w[j][i], win[j][i], p);
                        dp *= dsilu(p, sigm<is_fast<T>()>(p));
                    }
                    const float od = own * dp;
                    db[i] += od;
#pragma unroll
                    for (int j = 0; j < K; ++j) {
                        dw[j][i] = fmaf(od, win[j][i], dw[j][i]);
                        acc[j][i] = fmaf(w[j][i], dp, acc[j][i]);
                    }
                }
                put(t + u - (K - 1), acc[0]);
#pragma unroll
                for (int i = 0; i < V; ++i) {
#pragma unroll
                    for (int j = 0; j + 1 < K; ++j) {
                        acc[j][i] = acc[j + 1][i];
                        win[j][i] = win[j + 1][i];
                    }
                    acc[K - 1][i] = 0.0f;
                }
            }
        }
        t = lim;
        if (t == q.end) {  // the sequence's last K - 1 places: no later token adds to them
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                if (a.dstate_out != nullptr) {
                    float d[V];
                    Vec<V>::ld((const T*)a.dstate_out + (q.seq * (K - 1) + j) * a.C + c, d);
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[j][i] += d[i];
                }
                put(t - (K - 1) + j, acc[j]);
            }
        }
        if (t >= t1) break;
        q = seq_at(a.seqs, b, t);
        load_window<T, K, V>(a, q, row0, t, c, win);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < K; ++j) acc[j][i] = 0.0f;
    }
    float* p = a.partial + rr * (K + 1) * a.C;  // [C, K], then [C]
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < K; ++j) p[(c + i) * K + j] = dw[j][i];
        p[a.C * K + c + i] = db[i];
    }
}

// Sequences without tokens pass the gradient of their state on.
template <typename T>
__global__ void __launch_bounds__(kNT) conv_bwd_empty_kernel(const ConvArgs a) {
    const int64_t w = (int64_t)(a.K - 1) * a.C, id = (int64_t)blockIdx.x * kNT + threadIdx.x;
    if (id >= a.nstate * w) return;
    int64_t end;
    if (seq_tokens(a.seqs, id / w, &end) > 0) return;
    const T* g = (const T*)a.dstate_out;
    st((T*)a.dstate_in + id, g != nullptr ? ld(g + id) : 0.0f);
}

__global__ void __launch_bounds__(256) sum_partials_kernel(const float* in, int64_t n,
                                                           int64_t stride, float* out,
                                                           int64_t count) {
    // 32 columns a CTA, eight threads a column: thread k adds partials k, k + 8, ..., then the
    // eight are added in order
    __shared__ float part[8][33];
    const int col = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + col;
    float s = 0.0f;
    if (i < count) {
#pragma unroll 4
        for (int64_t p = k; p < n; p += 8) s += in[p * stride + i];
    }
    part[k][col] = s;
    __syncthreads();
    if (k == 0 && i < count) {
#pragma unroll
        for (int j = 1; j < 8; ++j) s += part[j][col];
        out[i] = s;
    }
}

unsigned blocks_for(int64_t n) { return (unsigned)((n + kNT - 1) / kNT); }

bool rows_of(int64_t ld, int64_t width, int64_t v) { return ld % v == 0 && width % v == 0; }

// Tokens a thread walks: long runs read little halo, short ones fill the GPU (152 SMs, 2048
// threads each) on small batches.
int run_tokens(int64_t B, int64_t L, int64_t nv, int longest) {
    int run = longest;
    while (run > 8 && B * ((L + run - 1) / run) * nv < 152 * 1024) run /= 2;
    return run;
}

// Calls f.template operator()<K>() for the K of the call.
template <int K = 1, typename F>
cudaError_t with_taps(int k, F&& f) {
    if constexpr (K > 8) return cudaErrorInvalidValue;
    else return k == K ? f(std::integral_constant<int, K>()) : with_taps<K + 1>(k, f);
}

template <typename T, int V>
cudaError_t conv_fwd(const ConvArgs& a, cudaStream_t s) {
    const int64_t nv = a.C / V;
    return with_taps(a.K, [&](auto kk) {
        constexpr int K = decltype(kk)::value;
        if (a.seqs.L > 0) {
            const int run = run_tokens(a.B, a.seqs.L, nv, 32);
            const int64_t runs = (a.seqs.L + run - 1) / run;
            const unsigned g = blocks_for(a.B * runs * nv);
            conv_fwd_kernel<T, K, V><<<g, kNT, 0, s>>>(a, runs, run);
        }
        if (K > 1 && a.state_out != nullptr)
            conv_tail_kernel<T, K, V><<<blocks_for(a.nstate * nv), kNT, 0, s>>>(a);
        return cudaGetLastError();
    });
}

template <typename T, int V>
cudaError_t conv_step(const ConvArgs& a, cudaStream_t s) {
    return with_taps(a.K, [&](auto kk) {
        constexpr int K = decltype(kk)::value;
        const unsigned g = blocks_for(a.B * (a.C / V));
        conv_step_kernel<T, K, V><<<g, kNT, 0, s>>>(a);
        return cudaGetLastError();
    });
}

constexpr int kBwdRun = 64;
int bwd_run(int64_t B, int64_t L, int64_t C) { return run_tokens(B, L, (C + 3) / 4, kBwdRun); }

template <typename T, int V>
cudaError_t conv_bwd(const ConvArgs& a, cudaStream_t s) {
    const int64_t nv = a.C / V;
    const int run = bwd_run(a.B, a.seqs.L, a.C);
    const int64_t runs = (a.seqs.L + run - 1) / run;
    cudaError_t e = with_taps(a.K, [&](auto kk) {
        constexpr int K = decltype(kk)::value;
        if (runs > 0) {
            const unsigned g = blocks_for(a.B * runs * nv);
            conv_bwd_kernel<T, K, V><<<g, kNT, 0, s>>>(a, runs, run);
        }
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    if (a.dstate_in != nullptr && a.K > 1 && (a.seqs.cu != nullptr || a.seqs.L == 0)) {
        conv_bwd_empty_kernel<T><<<blocks_for(a.nstate * (a.K - 1) * a.C), kNT, 0, s>>>(a);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const int64_t n = a.B * runs, stride = (a.K + 1) * a.C;
    e = launch_sum_partials(a.partial, n, stride, a.dw, a.K * a.C, s);
    if (e == cudaSuccess && a.dbias != nullptr)
        e = launch_sum_partials(a.partial + a.K * a.C, n, stride, a.dbias, a.C, s);
    return e;
}

}  // namespace

cudaError_t launch_sum_partials(const float* in, int64_t n, int64_t stride, float* out,
                                int64_t count, cudaStream_t s) {
    sum_partials_kernel<<<(unsigned)((count + 31) / 32), 256, 0, s>>>(in, n, stride, out, count);
    return cudaGetLastError();
}

int64_t conv_bwd_runs(int64_t B, int64_t L, int64_t C) {
    const int run = bwd_run(B, L, C);
    return B * ((L + run - 1) / run);
}

cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t s) {
    if (a.dtype == LIZARD_BF16)
        return rows_of(a.ldx, a.C, 8) && a.ldy % 8 == 0 ? conv_fwd<__nv_bfloat16, 8>(a, s)
                                                        : conv_fwd<__nv_bfloat16, 1>(a, s);
    return rows_of(a.ldx, a.C, 4) && a.ldy % 4 == 0 ? conv_fwd<float, 4>(a, s) : conv_fwd<float, 1>(a, s);
}

cudaError_t launch_conv_step(const ConvArgs& a, cudaStream_t s) {
    if (a.dtype == LIZARD_BF16)
        return rows_of(a.ldx, a.C, 8) && a.ldy % 8 == 0 ? conv_step<__nv_bfloat16, 8>(a, s)
                                                        : conv_step<__nv_bfloat16, 1>(a, s);
    return rows_of(a.ldx, a.C, 4) && a.ldy % 4 == 0 ? conv_step<float, 4>(a, s) : conv_step<float, 1>(a, s);
}

cudaError_t launch_conv_bwd(const ConvArgs& a, cudaStream_t s) {
    const bool v = rows_of(a.ldx, a.C, 4) && a.ldy % 4 == 0 && a.lddx % 4 == 0;
    if (a.dtype == LIZARD_BF16) return v ? conv_bwd<__nv_bfloat16, 4>(a, s) : conv_bwd<__nv_bfloat16, 1>(a, s);
    return v ? conv_bwd<float, 4>(a, s) : conv_bwd<float, 1>(a, s);
}

}  // namespace lz
