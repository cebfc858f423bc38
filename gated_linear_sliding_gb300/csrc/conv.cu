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
constexpr int TX = 32, TY = kNT / TX;  // a CTA: TX threads along the channels, TY runs of tokens

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

// The taps of a CTA's TX V channels go through shared memory, transposed: each thread reading
// its own channels' rows of w costs more than the inputs of a run.
template <int K, int V>
struct Taps {
    float w[K][TX * V], bias[TX * V];
    __device__ __forceinline__ void fill(const ConvArgs& a, int64_t c0) {
        const int n = (int)min64(TX * V, a.C - c0);
        for (int e = threadIdx.x; e < n * K; e += kNT) w[e % K][e / K] = a.w[c0 * K + e];
        for (int e = threadIdx.x; e < n; e += kNT) bias[e] = a.bias != nullptr ? a.bias[c0 + e] : 0.0f;
        __syncthreads();
    }
};
template <int K, int V>
__device__ __forceinline__ void load_taps(const Taps<K, V>& t, int tx, float (*w)[V], float* bias) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < K; ++j) w[j][i] = t.w[j][tx * V + i];
        bias[i] = t.bias[tx * V + i];
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
// written once; the next U rows are on their way while U are computed.
template <typename T, int K, int V>
__global__ void __launch_bounds__(kNT) conv_fwd_kernel(const ConvArgs a, int64_t runs, int run, int64_t cbs) {
    constexpr int U = 8;
    const bool silu = a.act == LIZARD_ACT_SILU;
    __shared__ Taps<K, V> taps;
    const int tx = threadIdx.x % TX;
    const int64_t c0 = blockIdx.x % cbs * (TX * V), c = c0 + tx * V;
    const int64_t rr = blockIdx.x / cbs * TY + threadIdx.x / TX, b = rr / runs;
    check_offsets(a.seqs, a.header);
    taps.fill(a, c0);
    if (rr >= a.B * runs || c >= a.C) return;
    const int64_t t0 = rr % runs * run, t1 = min64(t0 + run, a.seqs.L), row0 = b * a.seqs.L;
    float w[K][V], bias[V], win[K][V];
    load_taps<K, V>(taps, tx, w, bias);
    SeqAt q = seq_at(a.seqs, b, t0);
    load_window<T, K, V>(a, q, row0, t0, c, win);
    const T* x = (const T*)a.x + (row0 + t0) * a.ldx + c;
    T* y = (T*)a.y + (row0 + t0) * a.ldy + c;
    const int n = (int)(t1 - t0);
    Pack<T, V> in[U], next[U];
    auto fetch = [&](int t) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u < n) next[u] = *reinterpret_cast<const Pack<T, V>*>(x + (int64_t)(t + u) * a.ldx);
    };
    fetch(0);
    int change = (int)min64(q.end - t0, n);  // where the next sequence begins
    for (int t = 0; t < n; t += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) in[u] = next[u];
        fetch(t + U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= n) break;
            if (t + u == change) {
                q = seq_at(a.seqs, b, t0 + t + u);
                load_window<T, K, V>(a, q, row0, t0 + t + u, c, win);
                change = (int)min64(q.end - t0, n);
            }
            float o[V];
            in[u].get(win[K - 1]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float p = bias[i];
#pragma unroll
                for (int j = 0; j < K; ++j) p = fmaf(w[j][i], win[j][i], p);
                o[i] = silu ? p * sigm<is_fast<T>()>(p) : p;
#pragma unroll
                for (int j = 0; j + 1 < K; ++j) win[j][i] = win[j + 1][i];
            }
            Vec<V>::st(y, o);
            y += a.ldy;
        }
    }
}

// One token a sequence: the state's K - 1 rows are read, moved up by one and written back.
template <typename T, int K, int V>
__global__ void __launch_bounds__(kNT) conv_step_kernel(const ConvArgs a, int64_t cbs) {
    const bool silu = a.act == LIZARD_ACT_SILU;
    __shared__ Taps<K, V> taps;
    const int tx = threadIdx.x % TX;
    const int64_t c0 = blockIdx.x % cbs * (TX * V), c = c0 + tx * V;
    const int64_t b = blockIdx.x / cbs * TY + threadIdx.x / TX;
    const bool in = b < a.B && c < a.C;
    const int64_t slot = !in ? -1 : a.slots != nullptr ? a.slots[b] : b;
    const bool live = slot >= 0 && slot < a.nslots;
    float w[K][V], bias[V], win[K][V], o[V];
    T* st = (T*)a.state + slot * (K - 1) * a.C + c;
    if (live) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) Vec<V>::ld(st + j * a.C, win[j]);
        Vec<V>::ld((const T*)a.x + b * a.ldx + c, win[K - 1]);
    }
    taps.fill(a, c0);
    if (!in) return;
    T* y = (T*)a.y + b * a.ldy + c;
    if (!live) {
        if (slot >= 0) report(a.header, LIZARD_ERR_INVALID_ARG, 33);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = 0.0f;
        Vec<V>::st(y, o);
        return;
    }
    load_taps<K, V>(taps, tx, w, bias);
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
__global__ void __launch_bounds__(kNT) conv_bwd_kernel(const ConvArgs a, int64_t runs, int run, int64_t cbs) {
    constexpr int U = 4;
    const bool silu = a.act == LIZARD_ACT_SILU;
    __shared__ Taps<K, V> taps;
    const int tx = threadIdx.x % TX;
    const int64_t c0 = blockIdx.x % cbs * (TX * V), c = c0 + tx * V;
    const int64_t rr = blockIdx.x / cbs * TY + threadIdx.x / TX, b = rr / runs;
    check_offsets(a.seqs, a.header);
    taps.fill(a, c0);
    if (rr >= a.B * runs || c >= a.C) return;
    const int64_t t0 = rr % runs * run, row0 = b * a.seqs.L;
    const int n = (int)min64(run, a.seqs.L - t0);
    float w[K][V], bias[V], win[K][V], acc[K][V], dw[K][V], db[V];
    load_taps<K, V>(taps, tx, w, bias);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j) dw[j][i] = acc[j][i] = 0.0f;
    }
    // tokens count from t0 from here on; a begin before -K and an end past n + K count as those
    const T* x = (const T*)a.x + (row0 + t0) * a.ldx + c;
    const T* dy = (const T*)a.dy + (row0 + t0) * a.ldy + c;
    T* dx = (T*)a.dx + (row0 + t0) * a.lddx + c;
    SeqAt q;
    int begin, end;
    auto enter = [&](int t) {
        q = seq_at(a.seqs, b, t0 + t);
        begin = (int)max64(q.begin - t0, -K);
        end = (int)min64(q.end - t0, n + K);
        load_window<T, K, V>(a, q, row0, t0 + t, c, win);
    };
    enter(0);
    // the gradient of token u (or of a place before the sequence's first token)
    auto put = [&](int u, const float* v) {
        if (u >= begin) {
            if (u >= 0 && u < n) Vec<V>::st(dx + u * a.lddx, v);
        } else if (a.dstate_in != nullptr && begin >= 0 && begin < n) {
            Vec<V>::st((T*)a.dstate_in + (q.seq * (K - 1) + (K - 1) + u - begin) * a.C + c, v);
        }
    };
    int t = 0;
    while (true) {
        const int lim = min(end, n + K - 1);
        Pack<T, V> in[U], g[U], nin[U], ng[U];  // the next U tokens are on their way
        auto fetch = [&](int t) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u < lim) {
                    nin[u] = *reinterpret_cast<const Pack<T, V>*>(x + (t + u) * a.ldx);
                    ng[u] = *reinterpret_cast<const Pack<T, V>*>(dy + (t + u) * a.ldy);
                }
        };
        fetch(t);
#pragma unroll 1
        for (; t < lim; t += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                in[u] = nin[u];
                g[u] = ng[u];
            }
            fetch(t + U);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u >= lim) break;
                float gy[V];
                in[u].get(win[K - 1]);
                g[u].get(gy);
                const float own = t + u < n ? 1.0f : 0.0f;  // the halo belongs to the next run
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float dp = gy[i];
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
        if (t == end) {  // the sequence's last K - 1 places: no later token adds to them
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
        if (t >= n) break;
        enter(t);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < K; ++j) acc[j][i] = 0.0f;
    }
    float* p = a.partial + rr * (K + 1) * a.C + c;  // [K + 1, C]
#pragma unroll
    for (int j = 0; j < K; ++j) Vec<V>::st(p + j * a.C, dw[j]);
    Vec<V>::st(p + K * a.C, db);
}

// dw [C, K] and dbias [C] from the runs' sums [n, K + 1, C]: 32 channels a CTA, eight threads a
// channel; thread k adds runs k, k + 8, ..., then the eight are added in order.
__global__ void __launch_bounds__(256) conv_bwd_sum_kernel(const ConvArgs a, int64_t n) {
    __shared__ float part[8][33];
    const int col = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + col, count = (a.K + 1) * a.C;
    float s = 0.0f;
    if (i < count) {
#pragma unroll 8
        for (int64_t p = k; p < n; p += 8) s += a.partial[p * count + i];
    }
    part[k][col] = s;
    __syncthreads();
    if (k != 0 || i >= count) return;
#pragma unroll
    for (int j = 1; j < 8; ++j) s += part[j][col];
    const int64_t j = i / a.C, c = i % a.C;
    if (j < a.K) a.dw[c * a.K + j] = s;
    else if (a.dbias != nullptr) a.dbias[c] = s;
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
            const int64_t cbs = (nv + TX - 1) / TX;
            conv_fwd_kernel<T, K, V><<<(unsigned)(cbs * ((a.B * runs + TY - 1) / TY)), kNT, 0, s>>>(a, runs, run, cbs);
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
        const int64_t cbs = (a.C / V + TX - 1) / TX;
        conv_step_kernel<T, K, V><<<(unsigned)(cbs * ((a.B + TY - 1) / TY)), kNT, 0, s>>>(a, cbs);
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
            const int64_t cbs = (nv + TX - 1) / TX;
            conv_bwd_kernel<T, K, V><<<(unsigned)(cbs * ((a.B * runs + TY - 1) / TY)), kNT, 0, s>>>(a, runs, run, cbs);
        }
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    if (a.dstate_in != nullptr && a.K > 1 && (a.seqs.cu != nullptr || a.seqs.L == 0)) {
        conv_bwd_empty_kernel<T><<<blocks_for(a.nstate * (a.K - 1) * a.C), kNT, 0, s>>>(a);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    conv_bwd_sum_kernel<<<(unsigned)(((a.K + 1) * a.C + 31) / 32), 256, 0, s>>>(a, a.B * runs);
    return cudaGetLastError();
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
        return rows_of(a.ldx, a.C, 4) && a.ldy % 4 == 0 ? conv_fwd<__nv_bfloat16, 4>(a, s)
                                                        : conv_fwd<__nv_bfloat16, 1>(a, s);
    return rows_of(a.ldx, a.C, 4) && a.ldy % 4 == 0 ? conv_fwd<float, 4>(a, s) : conv_fwd<float, 1>(a, s);
}

cudaError_t launch_conv_step(const ConvArgs& a, cudaStream_t s) {
    if (a.dtype == LIZARD_BF16)
        return rows_of(a.ldx, a.C, 4) && a.ldy % 4 == 0 ? conv_step<__nv_bfloat16, 4>(a, s)
                                                        : conv_step<__nv_bfloat16, 1>(a, s);
    return rows_of(a.ldx, a.C, 4) && a.ldy % 4 == 0 ? conv_step<float, 4>(a, s) : conv_step<float, 1>(a, s);
}

cudaError_t launch_conv_bwd(const ConvArgs& a, cudaStream_t s) {
    const bool v = rows_of(a.ldx, a.C, 4) && a.ldy % 4 == 0 && a.lddx % 4 == 0;
    if (a.dtype == LIZARD_BF16) return v ? conv_bwd<__nv_bfloat16, 4>(a, s) : conv_bwd<__nv_bfloat16, 1>(a, s);
    return v ? conv_bwd<float, 4>(a, s) : conv_bwd<float, 1>(a, s);
}

}  // namespace lz
