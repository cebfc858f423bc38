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

// V neighbouring channels as pairs (one channel: a pair with an idle half).
template <int V>
struct Chan {
    static constexpr int NP = (V + 1) / 2;
    static __device__ __forceinline__ void pairs(const float* f, f2* o) {
        if constexpr (V == 1) o[0] = pack(f[0], 0.0f);
        else {
#pragma unroll
            for (int i = 0; i < NP; ++i) o[i] = pack(f[2 * i], f[2 * i + 1]);
        }
    }
    template <typename T>
    static __device__ __forceinline__ void ld(const T* p, f2* o) {
        float f[V];
        Vec<V>::ld(p, f);
        pairs(f, o);
    }
    template <typename T>
    static __device__ __forceinline__ void get(const Pack<T, V>& p, f2* o) {
        float f[V];
        p.get(f);
        pairs(f, o);
    }
    template <typename T>
    static __device__ __forceinline__ void st(T* p, const f2* v) {
        float f[2 * NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) unpack(v[i], f[2 * i], f[2 * i + 1]);
        Vec<V>::st(p, f);
    }
};

// The K - 1 inputs before token t of its sequence, from the row or the sequence's state.
template <typename T, int K, int V>
__device__ __forceinline__ void load_window(const ConvArgs& a, const SeqAt& q, int64_t row0,
                                            int64_t t, int64_t c, f2 (*win)[Chan<V>::NP]) {
    const T* x = (const T*)a.x;
    const T* st = (const T*)a.state_in;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int64_t u = t - (K - 1) + j;  // token of win[j]
        if (u >= q.begin) Chan<V>::ld(x + (row0 + u) * a.ldx + c, win[j]);
        else if (st != nullptr) Chan<V>::ld(st + (q.seq * (K - 1) + (K - 1) + u - q.begin) * a.C + c, win[j]);
        else {
#pragma unroll
            for (int i = 0; i < Chan<V>::NP; ++i) win[j][i] = 0;
        }
    }
}

// The taps of a CTA's TX V channels go through shared memory, transposed: each thread reading
// its own channels' rows of w costs more than the inputs of a run.
template <int K, int V>
struct Taps {
    __align__(16) float w[K][TX * V], bias[TX * V];
    __device__ __forceinline__ void fill(const ConvArgs& a, int64_t c0) {
        const int n = (int)min64(TX * V, a.C - c0);
        for (int e = threadIdx.x; e < n * K; e += kNT) w[e % K][e / K] = a.w[c0 * K + e];
        for (int e = threadIdx.x; e < n; e += kNT) bias[e] = a.bias != nullptr ? a.bias[c0 + e] : 0.0f;
        __syncthreads();
    }
};
template <int K, int V>
__device__ __forceinline__ void load_taps(const Taps<K, V>& t, int tx, f2 (*w)[Chan<V>::NP], f2* bias) {
#pragma unroll
    for (int j = 0; j < K; ++j) Chan<V>::ld(&t.w[j][tx * V], w[j]);
    Chan<V>::ld(&t.bias[tx * V], bias);
}
// pre-activations, and act of them
template <int K, int NP>
__device__ __forceinline__ void taps_of(const f2 (*w)[NP], const f2* bias, const f2 (*win)[NP], f2* p) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        p[i] = bias[i];
#pragma unroll
        for (int j = 0; j < K; ++j) p[i] = fma2(w[j][i], win[j][i], p[i]);
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

// One thread: V channels, `run` tokens of one row of the batch.  x is read and y written once;
// bound by HBM with the instruction issue close behind (20 instructions an element).  8 x 2048 x
// 4096 bf16, K = 4: 52 us, 5.15 TB/s.  With the rows ahead in registers (104 of them, 20 warps a
// SM) 96 us: the loads in flight were too few; taps read by each thread from global memory 161 us.
template <typename T, int K, int V, bool STATES>
__global__ void __launch_bounds__(kNT) conv_fwd_kernel(const ConvArgs a, int64_t runs, int run, int64_t cbs) {
    constexpr int U = 8, S = 2;  // rows a group, groups on their way
    const bool silu = a.act == LIZARD_ACT_SILU;
    __shared__ Taps<K, V> taps;
    const int tx = threadIdx.x % TX;
    const int64_t c0 = blockIdx.x % cbs * (TX * V), c = c0 + tx * V;
    const int64_t rr = blockIdx.x / cbs * TY + threadIdx.x / TX, b = rr / runs;
    check_offsets(a.seqs, a.header);
    const bool in_range = rr < a.B * runs && c < a.C;
    const int64_t t0 = rr % runs * run, row0 = b * a.seqs.L;
    const int n = in_range ? (int)min64(run, a.seqs.L - t0) : 0;
    const T* x = (const T*)a.x + (row0 + t0) * a.ldx + c;
    T* y = (T*)a.y + (row0 + t0) * a.ldy + c;
    __shared__ Pack<T, V> rows[S][U][kNT];
    auto fetch = [&](int t) {  // the group from token t on
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u < n) copy_async<T, V>(rows[t / U % S][u][threadIdx.x].e, x + (int64_t)(t + u) * a.ldx);
        copy_commit();
    };
    constexpr int NP = Chan<V>::NP;
    f2 w[K][NP], bias[NP], win[K][NP];
    SeqAt q;
#pragma unroll
    for (int g = 0; g < S; ++g) fetch(g * U);  // on their way while the taps are
    if (in_range) {
        q = seq_at(a.seqs, b, t0);
        load_window<T, K, V>(a, q, row0, t0, c, win);
    }
    taps.fill(a, c0);
    if (!in_range) return;
    load_taps<K, V>(taps, tx, w, bias);
    // the window after a sequence's last token is what its state holds then
    auto put_state = [&]() {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) Chan<V>::st((T*)a.state_out + (q.seq * (K - 1) + j) * a.C + c, win[j]);
    };
    int change = (int)min64(q.end - t0, n);  // where the next sequence begins
    for (int t = 0; t < n; t += U) {
        copy_wait<S - 1>();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= n) break;
            if (t + u == change) {
                q = seq_at(a.seqs, b, t0 + t + u);
                load_window<T, K, V>(a, q, row0, t0 + t + u, c, win);
                change = (int)min64(q.end - t0, n);
            }
            f2 o[NP];
            Chan<V>::get(rows[t / U % S][u][threadIdx.x], win[K - 1]);
            taps_of<K, NP>(w, bias, win, o);
            if (silu) {
#pragma unroll
                for (int i = 0; i < NP; ++i) o[i] = mul2(o[i], sigm2<is_fast<T>()>(o[i]));
            }
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int j = 0; j + 1 < K; ++j) win[j][i] = win[j + 1][i];
            Chan<V>::st(y, o);
            y += a.ldy;
        }
        fetch(t + S * U);
    }
    copy_wait<0>();
    if (STATES && t0 + n == q.end) put_state();
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
    constexpr int NP = Chan<V>::NP;
    f2 w[K][NP], bias[NP], win[K][NP], o[NP];
    T* st = (T*)a.state + slot * (K - 1) * a.C + c;
    if (live) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) Chan<V>::ld(st + j * a.C, win[j]);
        Chan<V>::ld((const T*)a.x + b * a.ldx + c, win[K - 1]);
    }
    taps.fill(a, c0);
    if (!in) return;
    T* y = (T*)a.y + b * a.ldy + c;
    if (!live) {
        if (slot >= 0) report(a.header, LIZARD_ERR_INVALID_ARG, 33);
#pragma unroll
        for (int i = 0; i < NP; ++i) o[i] = 0;
        Chan<V>::st(y, o);
        return;
    }
    load_taps<K, V>(taps, tx, w, bias);
    taps_of<K, NP>(w, bias, win, o);
    if (silu) {
#pragma unroll
        for (int i = 0; i < NP; ++i) o[i] = mul2(o[i], sigm2<is_fast<T>()>(o[i]));
    }
    Chan<V>::st(y, o);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) Chan<V>::st(st + j * a.C, win[j + 1]);
}

// Backward, one thread: V channels, the tokens [t0, t1) of a run.  Walking forward, token t gives
// dp = dy act'(pre), which adds w[j] dp to the gradient of token t - K + 1 + j; acc[j] holds
// those sums, and the oldest is complete once t has been added.  The walk goes K - 1 tokens past
// the run (or to the sequence's end) to complete the run's own last tokens.  Places before a
// sequence's first token are its state, whose gradient is written by the run that holds that
// token.  8 x 2048 x 4096 bf16, K = 4: 102 us for x, dy and dx, 3.95 TB/s; 36 instructions an element
// on 122 registers (16 warps a SM) share the bound with HBM.
template <typename T, int K, int V>
__global__ void __launch_bounds__(kNT) conv_bwd_kernel(const ConvArgs a, int64_t runs, int run, int64_t cbs) {
    constexpr int U = 4, S = 2;  // rows a group, groups on their way
    const bool silu = a.act == LIZARD_ACT_SILU;
    __shared__ Taps<K, V> taps;
    const int tx = threadIdx.x % TX;
    const int64_t c0 = blockIdx.x % cbs * (TX * V), c = c0 + tx * V;
    const int64_t rr = blockIdx.x / cbs * TY + threadIdx.x / TX, b = rr / runs;
    check_offsets(a.seqs, a.header);
    const bool in_range = rr < a.B * runs && c < a.C;
    const int64_t t0 = rr % runs * run, row0 = b * a.seqs.L;
    const int n = (int)min64(run, a.seqs.L - t0);
    constexpr int NP = Chan<V>::NP;
    f2 w[K][NP], bias[NP], win[K][NP], acc[K][NP], dw[K][NP], db[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        db[i] = 0;
#pragma unroll
        for (int j = 0; j < K; ++j) dw[j][i] = acc[j][i] = 0;
    }
    // tokens count from t0 from here on; a begin before -K and an end past n + K count as those
    const T* x = (const T*)a.x + (row0 + t0) * a.ldx + c;
    const T* dy = (const T*)a.dy + (row0 + t0) * a.ldy + c;
    T* dx = (T*)a.dx + (row0 + t0) * a.lddx + c;
    SeqAt q;
    int begin = 0, end = 0, lim = 0;  // lim: end of the tokens walked of this sequence
    __shared__ Pack<T, V> rows[S][2][U][kNT];
    int groups = 0;  // fetched so far
    auto fetch = [&](int t) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u < lim) {
                copy_async<T, V>(rows[groups % S][0][u][threadIdx.x].e, x + (t + u) * a.ldx);
                copy_async<T, V>(rows[groups % S][1][u][threadIdx.x].e, dy + (t + u) * a.ldy);
            }
        copy_commit();
        ++groups;
    };
    auto enter = [&](int t) {
        q = seq_at(a.seqs, b, t0 + t);
        begin = (int)max64(q.begin - t0, -K);
        end = (int)min64(q.end - t0, n + K);
        lim = min(end, n + K - 1);
#pragma unroll
        for (int g = 0; g < S; ++g) fetch(t + g * U);
        load_window<T, K, V>(a, q, row0, t0 + t, c, win);
    };
    if (in_range) enter(0);  // on their way while the taps are
    taps.fill(a, c0);
    if (!in_range) return;
    load_taps<K, V>(taps, tx, w, bias);
    // the gradient of token u (or of a place before the sequence's first token)
    auto put = [&](int u, const f2* v) {
        if (u >= begin) {
            if (u >= 0 && u < n) Chan<V>::st(dx + u * a.lddx, v);
        } else if (a.dstate_in != nullptr && begin >= 0 && begin < n) {
            Chan<V>::st((T*)a.dstate_in + (q.seq * (K - 1) + (K - 1) + u - begin) * a.C + c, v);
        }
    };
    int t = 0;
    while (true) {
#pragma unroll 1
        for (; t < lim; t += U) {
            copy_wait<S - 1>();
            const int at = groups % S;  // the oldest group
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u >= lim) break;
                f2 dp[NP];
                Chan<V>::get(rows[at][0][u][threadIdx.x], win[K - 1]);
                Chan<V>::get(rows[at][1][u][threadIdx.x], dp);
                if (silu) {
                    f2 p[NP];
                    taps_of<K, NP>(w, bias, win, p);
#pragma unroll
                    for (int i = 0; i < NP; ++i) dp[i] = mul2(dp[i], dsilu2(p[i], sigm2<is_fast<T>()>(p[i])));
                }
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int j = 0; j < K; ++j) acc[j][i] = fma2(w[j][i], dp[i], acc[j][i]);
                if (t + u < n) {  // the halo belongs to the next run
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        db[i] = add2(db[i], dp[i]);
#pragma unroll
                        for (int j = 0; j < K; ++j) dw[j][i] = fma2(dp[i], win[j][i], dw[j][i]);
                    }
                }
                put(t + u - (K - 1), acc[0]);
#pragma unroll
                for (int i = 0; i < NP; ++i) {
#pragma unroll
                    for (int j = 0; j + 1 < K; ++j) {
                        acc[j][i] = acc[j + 1][i];
                        win[j][i] = win[j + 1][i];
                    }
                    acc[K - 1][i] = 0;
                }
            }
            fetch(t + S * U);
        }
        t = lim;
        if (t == end) {  // the sequence's last K - 1 places: no later token adds to them
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                if (a.dstate_out != nullptr) {
                    f2 d[NP];
                    Chan<V>::ld((const T*)a.dstate_out + (q.seq * (K - 1) + j) * a.C + c, d);
#pragma unroll
                    for (int i = 0; i < NP; ++i) acc[j][i] = add2(acc[j][i], d[i]);
                }
                put(t - (K - 1) + j, acc[j]);
            }
        }
        if (t >= n) break;
        copy_wait<0>();
        enter(t);
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < K; ++j) acc[j][i] = 0;
    }
    copy_wait<0>();
    float* p = a.partial + rr * (K + 1) * a.C + c;  // [K + 1, C]
#pragma unroll
    for (int j = 0; j < K; ++j) Chan<V>::st(p + j * a.C, dw[j]);
    Chan<V>::st(p + K * a.C, db);
}

// dw [C, K] and dbias [C] from the runs' sums [n, K + 1, C].
template <int KT>
__global__ void __launch_bounds__(32 * KT) conv_bwd_sum_kernel(const ConvArgs a, int64_t n) {
    const int64_t i0 = (int64_t)blockIdx.x * 32, count = (a.K + 1) * a.C;
    sum_columns<KT>(
        n, (int)min64(32, count - i0), [&](int64_t p, int i) { return a.partial[p * count + i0 + i]; },
        [&](int i, float s) {
            const int64_t j = (i0 + i) / a.C, c = (i0 + i) % a.C;
            if (j < a.K) a.dw[c * a.K + j] = s;
            else if (a.dbias != nullptr) a.dbias[c] = s;
        });
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

unsigned blocks_for(int64_t n) { return (unsigned)((n + kNT - 1) / kNT); }

bool rows_of(int64_t ld, int64_t width, int64_t v) { return ld % v == 0 && width % v == 0; }

// Tokens a thread walks: long runs read little halo and begin seldom (8 x 2048 x 4096, backward with
// its sums: 64 tokens 117 us, 128 109 us, 256 119 us), short ones fill the GPU on small batches.
constexpr int kFwdRun = 128, kBwdRun = 128;
int run_tokens(int64_t B, int64_t L, int64_t nv, int longest) {
    int run = longest;
    const int64_t warps = (nv + TX - 1) / TX;  // of a run
    while (run > 8 && B * ((L + run - 1) / run) * warps < 152 * 16) run /= 2;
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
        // The pass over the rows writes a dense batch's states too, unless they are those that its
        // other threads begin with; a packed batch's sequences may be empty, and no thread's.
        const bool states = K > 1 && a.state_out != nullptr && a.state_out != a.state_in &&
                            a.seqs.cu == nullptr && a.seqs.L > 0;
        if (a.seqs.L > 0) {
            const int run = run_tokens(a.B, a.seqs.L, nv, kFwdRun);
            const int64_t runs = (a.seqs.L + run - 1) / run;
            const int64_t cbs = (nv + TX - 1) / TX;
            const auto kernel = states ? conv_fwd_kernel<T, K, V, true> : conv_fwd_kernel<T, K, V, false>;
            kernel<<<(unsigned)(cbs * ((a.B * runs + TY - 1) / TY)), kNT, 0, s>>>(a, runs, run, cbs);
        }
        if (K > 1 && a.state_out != nullptr && !states)
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
    const unsigned g = (unsigned)(((a.K + 1) * a.C + 31) / 32);
    if (many_partials(a.B * runs, g)) conv_bwd_sum_kernel<32><<<g, 1024, 0, s>>>(a, a.B * runs);
    else conv_bwd_sum_kernel<8><<<g, 256, 0, s>>>(a, a.B * runs);
    return cudaGetLastError();
}

}  // namespace

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
