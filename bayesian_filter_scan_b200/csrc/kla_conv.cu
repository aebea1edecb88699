// kla_conv.cu -- short depthwise causal convolution with SiLU: prompts (with a
// history in and out), gradients, single tokens (sm_100a).
//   pre[t] = bias + sum_{w<W} weight[w] x[t-(W-1)+w],  out = silu(pre)
//   d[t] = dout[t] silu'(pre[t]),  dx[t] = sum_{j<W} weight[W-1-j] d[t+j],
//   dweight[w] = sum_t d[t] x[t-(W-1)+w],  dbias = sum_t d[t]
// Per channel a few products for 4 to 12 bytes: HBM binds, the two special-function
// steps of a bf16 silu next. A thread owns V contiguous channels (one 8-byte access
// where the rows allow it) and slides along a run of tokens with the last W-1 rows in
// registers, so every row is read once, but for the W-1 rows in front of each run; the
// next rows are on their way meanwhile, and a batch inside one sequence takes a path
// without its checks. Measured: 32768 packed tokens of 2048 channels in bf16 61 us (4.4
// TB/s), in fp32 97 us (5.5 TB/s); gradients of 16384 tokens 74 us (2.7 TB/s: the sums per
// tap and the halo on both sides keep the issue slots busy), in fp32 93 us (4.3 TB/s); rows
// of odd length, one element per access, take 1.5 times as long (32768 x 2047 in bf16 92
// us, gradients 193 us against 136).
#include "kla_block.cuh"

namespace kla {

namespace {

constexpr int kConvThreads = 128;
constexpr int kBwdRunMin = 16;    // tokens of one thread's shortest run, backward
constexpr int kBwdRuns = 8;       // runs per CTA
constexpr int kBwdBatch = 4;      // rows in flight per thread, backward
constexpr int kBwdLanes = 32;     // channel vectors per CTA

// The row at place p of sequence n, which starts at s0: x there, or in front of s0 the
// history's row, or 0 without one.
template <int W, int V, typename T>
__device__ __forceinline__ void row_before(const ConvArgs &g, int n, long long s0, long long p, int c,
                                           float (&v)[V]) {
    if (p >= s0) {
        load_v<V>(static_cast<const T *>(g.x) + p * g.ld_x + c, v);
    } else if (g.state0) {
        const long long r = (long long)n * (W - 1) + (W - 1) + (p - s0);
        load_v<V>(static_cast<const T *>(g.state0) + r * g.D + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
    }
}

template <int W, int V>
struct Taps {
    float w[W][V], b[V];
    __device__ __forceinline__ void load(const ConvArgs &g, int c) {
        if (W == 4 && ((uintptr_t)g.w & 15) == 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float4 t = __ldg(reinterpret_cast<const float4 *>(g.w) + c + i);
                w[0][i] = t.x; w[1 % W][i] = t.y; w[2 % W][i] = t.z; w[3 % W][i] = t.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int k = 0; k < W; ++k) w[k][i] = __ldg(g.w + (c + i) * W + k);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) b[i] = g.bias ? __ldg(g.bias + c + i) : 0.f;
    }
};

// Grid: (token blocks, then one block row per sequence for the final states, then
// blocks that clear the rows of no sequence) x channel blocks; a CTA is bx channel
// vectors x 128 / bx runs.
template <int W, int V, int BATCH, typename T>
__global__ void __launch_bounds__(kConvThreads) conv_forward_kernel(const ConvArgs g, int bx, int run, long long tok_blocks,
                                                                    long long seq_end) {
    const int cv = blockIdx.y * bx + threadIdx.x % bx, c = cv * V;
    if (blockIdx.x >= seq_end) {
        T *out = static_cast<T *>(g.out);
        const long long step = (gridDim.x - seq_end) * gridDim.y * kConvThreads, D = g.D;
        const long long from = ((blockIdx.x - seq_end) * gridDim.y + blockIdx.y) * kConvThreads + threadIdx.x;
        const long long head = min((long long)g.ax.cu[0], g.ax.ntok), tail = max(g.ax.cu[g.ax.nseq], 0);
        if (head > 0) clear(out, head * D, from, step);
        if (tail < g.ax.ntok) clear(out + tail * D, (g.ax.ntok - tail) * D, from, step);
        return;
    }
    if (c >= g.D) return;
    const T *x = static_cast<const T *>(g.x);
    if (blockIdx.x >= tok_blocks) {
        // the last W-1 inputs of one sequence
        if constexpr (W > 1) {
            const long long n = (blockIdx.x - tok_blocks) * (kConvThreads / bx) + threadIdx.x / bx;
            if (n >= g.ax.nseq) return;
            long long s0, s1;
            g.ax.range((int)n, s0, s1);
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                float v[V];
                row_before<W, V, T>(g, (int)n, s0, s1 - (W - 1) + i, c, v);
                store_v<V>(static_cast<T *>(g.final_state) + (n * (W - 1) + i) * g.D + c, v);
            }
        }
        return;
    }
    long long t = ((long long)blockIdx.x * (kConvThreads / bx) + threadIdx.x / bx) * run;
    const long long te = min(t + run, g.ax.ntok);
    if (t >= te) return;
    // a batch of rows is in flight while the one before is convolved
    Raw<V, T> in[BATCH], next[BATCH];
    auto load = [&](Raw<V, T>(&r)[BATCH], long long from) {
        const T *p = x + from * g.ld_x + c;
#pragma unroll
        for (int j = 0; j < BATCH; ++j, p += g.ld_x)
            if (from + j < te) r[j].load(p);
    };
    load(in, t);
    Pairs<V> w[W], bias, win[W];      // win: rows t-(W-1) .. t
    {
        Taps<W, V> k;
        k.load(g, c);
#pragma unroll
        for (int r = 0; r < W; ++r) w[r].set(k.w[r]);
        bias.set(k.b);
    }
    int n = -1;
    long long s0 = 0, s1 = t;  // the current stretch of tokens ends at s1
    T *out = static_cast<T *>(g.out) + t * g.D + c;
    // one token; `inside`: known to lie in the current sequence
    auto token = [&](const Raw<V, T> &r, long long tj, auto inside) {
        if (!inside.value && tj >= s1) {
            n = g.ax.find(tj);
            if (n >= 0) {
                g.ax.range(n, s0, s1);
#pragma unroll
                for (int i = 0; i < W - 1; ++i) {
                    float f[V];
                    row_before<W, V, T>(g, n, s0, tj - (W - 1) + i, c, f);
                    win[i].set(f);
                }
            } else {
                s1 = tj + 1;
            }
        }
        if (!inside.value && n < 0) return;
        float y[V];
        r.get(y);
        win[W - 1].set(y);
        Pairs<V> a = bias;
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int k = 0; k < Pairs<V>::K; ++k) a.p[k] = fma2(w[i].p[k], win[i].p[k], a.p[k]);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) win[i] = win[i + 1];
        a.get(y);
        if (g.silu)
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] *= sigmoid_for<T>(y[i]);
        store_v<V>(out, y);
    };
    for (; t < te; t += BATCH) {
        load(next, t + BATCH);
        if (n >= 0 && t + BATCH <= min(te, s1)) {
#pragma unroll
            for (int j = 0; j < BATCH; ++j, out += g.D) token(in[j], t + j, std::true_type());
        } else {
#pragma unroll
            for (int j = 0; j < BATCH; ++j, out += g.D)
                if (t + j < te) token(in[j], t + j, std::false_type());
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j) in[j] = next[j];
    }
}

// d = dout * silu'(pre) of one token
template <typename T, int W, int V>
__device__ __forceinline__ void d_pre(const ConvArgs &g, const Taps<W, V> &k, const float (&win)[W][V],
                                      const float (&dout)[V], float (&d)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        d[i] = dout[i];
        if (g.silu) {
            float a = k.b[i];
#pragma unroll
            for (int r = 0; r < W; ++r) a = fmaf(k.w[r][i], win[r][i], a);
            const float s = sigmoid_for<T>(a);
            d[i] *= s * fmaf(a, 1.f - s, 1.f);
        }
    }
}

// A CTA covers 32 channel vectors x 8 runs of tokens. A run slides over its
// tokens and the W-1 behind them (of the same sequence): dx of a token is
// complete W-1 tokens later. The runs' sums of dweight and dbias meet in shared
// memory in run order; the CTAs' sums are added by launch_colsum.
template <int W, int V, typename T>
__global__ void __launch_bounds__(kBwdLanes * kBwdRuns, V == 1 ? 3 : 2) conv_backward_kernel(const ConvArgs g, int length) {
    __shared__ float red[kBwdRuns][(W + 1) * V][kBwdLanes];
    const int lane = threadIdx.x % kBwdLanes, run = threadIdx.x / kBwdLanes;
    const int c = (blockIdx.y * kBwdLanes + lane) * V;
    const bool live = c < g.D;
    const T *x = static_cast<const T *>(g.x), *dout = static_cast<const T *>(g.dout);
    float dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) dw[w][i] = 0.f;
    }
    const long long a = ((long long)blockIdx.x * kBwdRuns + run) * length;
    const long long b = min(a + length, g.ax.ntok);
    if (live && a < b) {
        Taps<W, V> k;
        k.load(g, c);
        float win[W][V], acc[W][V];   // acc[j]: dx of token t-j so far
        int n = -1;
        long long s0 = 0, s1 = a;
        // dx of token p, complete but for the final state's share
        auto put = [&](long long p, float (&v)[V]) {
            if (W > 1 && g.dfinal && p >= s1 - (W - 1)) {
                float f[V];
                const long long r = (long long)n * (W - 1) + (W - 1) - (s1 - p);
                load_v<V>(static_cast<const T *>(g.dfinal) + r * g.D + c, f);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] += f[i];
            }
            store_v<V>(static_cast<T *>(g.dx) + p * g.D + c, v);
        };
        // a batch of rows is in flight while the one before is worked on
        const long long te = min(b + (W - 1), g.ax.ntok);
        Raw<V, T> bx[kBwdBatch], bo[kBwdBatch], nx[kBwdBatch], no[kBwdBatch];
        auto load = [&](Raw<V, T>(&rx)[kBwdBatch], Raw<V, T>(&ro)[kBwdBatch], long long from) {
#pragma unroll
            for (int j = 0; j < kBwdBatch; ++j)
                if (from + j < te) {
                    rx[j].load(x + (from + j) * g.ld_x + c);
                    ro[j].load(dout + (from + j) * g.D + c);
                }
        };
        load(bx, bo, a);
        // one token of the sequence; `inside`: neither near an end of the run nor of the sequence
        auto token = [&](const Raw<V, T> &rx, const Raw<V, T> &ro, long long t, auto inside) {
            float o[V], d[V];
            rx.get(win[W - 1]);
            ro.get(o);
            d_pre<T, W, V>(g, k, win, o, d);
#pragma unroll
            for (int q = W - 1; q > 0; --q)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[q][i] = fmaf(k.w[W - 1 - q][i], d[i], acc[q - 1][i]);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[0][i] = k.w[W - 1][i] * d[i];
            if (inside.value || t < b) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    db[i] += d[i];
#pragma unroll
                    for (int w = 0; w < W; ++w) dw[w][i] = fmaf(d[i], win[w][i], dw[w][i]);
                }
            }
#pragma unroll
            for (int r = 0; r < W - 1; ++r)
#pragma unroll
                for (int i = 0; i < V; ++i) win[r][i] = win[r + 1][i];
            if (inside.value) {
                store_v<V>(static_cast<T *>(g.dx) + (t - (W - 1)) * g.D + c, acc[W - 1]);
                return;
            }
            // token t-(W-1) is complete; at the sequence's end so are the ones behind it
            const long long lo = max(a, s0);
            if (t - (W - 1) >= lo) put(t - (W - 1), acc[W - 1]);
            if (t + 1 == s1) {
#pragma unroll
                for (int q = W - 2; q >= 0; --q)
                    if (t - q >= lo && t - q < b) put(t - q, acc[q]);
            }
        };
        bool more = true;
        for (long long t0 = a; more && t0 < te; t0 += kBwdBatch) {
            load(nx, no, t0 + kBwdBatch);
            if (n >= 0 && t0 - (W - 1) >= max(a, s0) && t0 + kBwdBatch <= b && t0 + kBwdBatch < s1) {
#pragma unroll
                for (int j = 0; j < kBwdBatch; ++j) token(bx[j], bo[j], t0 + j, std::true_type());
            } else {
#pragma unroll
                for (int j = 0; j < kBwdBatch; ++j) {
                    const long long t = t0 + j;
                    // tokens behind the run only as far as its last sequence goes
                    if (t >= te || (t >= s1 && t >= b)) more = false;
                    if (!more) continue;
                    if (t >= s1) {
                        n = g.ax.find(t);
                        if (n < 0) {
                            s1 = t + 1;
                            if (g.zero_rest) {
                                const float zero[V] = {};
                                store_v<V>(static_cast<T *>(g.dx) + t * g.D + c, zero);
                            }
                            continue;
                        }
                        g.ax.range(n, s0, s1);
#pragma unroll
                        for (int r = 0; r < W - 1; ++r) {
                            row_before<W, V, T>(g, n, s0, t - (W - 1) + r, c, win[r]);
#pragma unroll
                            for (int i = 0; i < V; ++i) acc[r][i] = 0.f;
                        }
                    }
                    if (n >= 0) token(bx[j], bo[j], t, std::false_type());
                }
            }
#pragma unroll
            for (int j = 0; j < kBwdBatch; ++j) bx[j] = nx[j], bo[j] = no[j];
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int w = 0; w < W; ++w) red[run][w * V + i][lane] = dw[w][i];
        red[run][W * V + i][lane] = db[i];
    }
    __syncthreads();
    float *part = g.part + (long long)blockIdx.x * g.D * (W + 1);
    for (int e = threadIdx.x; e < (W + 1) * V * kBwdLanes; e += kBwdLanes * kBwdRuns) {
        const int l = e % kBwdLanes, q = e / kBwdLanes, w = q / V, i = q % V;
        const int ch = (blockIdx.y * kBwdLanes + l) * V + i;
        if (ch >= g.D) continue;
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < kBwdRuns; ++r) s += red[r][q][l];
        part[w < W ? (long long)ch * W + w : (long long)g.D * W + ch] = s;
    }
}

// dstate0[n][i] = sum over tokens p <= i of weight[i-p] d[p], plus what of the
// final state was the history itself (sequences shorter than W-1).
template <int W, typename T>
__global__ void __launch_bounds__(kConvThreads) conv_dstate_kernel(const ConvArgs g) {
    if constexpr (W > 1) {
        const int c = blockIdx.y * kConvThreads + threadIdx.x;
        if (c >= g.D) return;
        const int n = blockIdx.x;
        long long s0, s1;
        g.ax.range(n, s0, s1);
        const long long len = s1 - s0;
        Taps<W, 1> k;
        k.load(g, c);
        float ds[W - 1], win[W][1];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const long long from = i - len;     // final_state[i - len] was state0[i]
            ds[i] = g.dfinal && from >= 0
                        ? to_f(static_cast<const T *>(g.dfinal)[((long long)n * (W - 1) + from) * g.D + c]) : 0.f;
            row_before<W, 1, T>(g, n, s0, s0 - (W - 1) + i, c, win[i]);
        }
#pragma unroll
        for (int p = 0; p < W - 1; ++p) {
            if (p < len) {
                float o[1], d[1];
                load_v<1>(static_cast<const T *>(g.x) + (s0 + p) * g.ld_x + c, win[W - 1]);
                load_v<1>(static_cast<const T *>(g.dout) + (s0 + p) * g.D + c, o);
                d_pre<T, W, 1>(g, k, win, o, d);
#pragma unroll
                for (int i = p; i < W - 1; ++i) ds[i] = fmaf(k.w[i - p][0], d[0], ds[i]);
#pragma unroll
                for (int r = 0; r < W - 1; ++r) win[r][0] = win[r + 1][0];
            }
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
            static_cast<T *>(g.dstate0)[((long long)n * (W - 1) + i) * g.D + c] = from_f<T>(ds[i]);
    }
}

// One token per row: the state's rows move down by one, x becomes the last. A thread
// takes the same channels of `run` rows, for which it loads the taps once.
template <int W, int V, typename T>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(const ConvArgs g, int nvec, int run) {
    const long long e = (long long)blockIdx.x * kConvThreads + threadIdx.x;
    long long n = e / nvec * run;
    const long long end = min(n + run, (long long)g.ax.nseq);
    if (n >= end) return;
    const int c = (int)(e % nvec) * V;
    Raw<V, T> in[W], next[W];
    auto load = [&](Raw<V, T>(&r)[W], long long row) {
        const T *state = static_cast<const T *>(g.final_state) + row * (W - 1) * g.D + c;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) r[i].load(state + (long long)i * g.D);
        r[W - 1].load(static_cast<const T *>(g.x) + row * g.ld_x + c);
    };
    load(in, n);
    Taps<W, V> k;
    k.load(g, c);
    for (; n < end; ++n) {
        if (n + 1 < end) load(next, n + 1);
        float a[V], f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] = k.b[i];
        T *state = static_cast<T *>(g.final_state) + n * (W - 1) * g.D + c;
#pragma unroll
        for (int r = 0; r < W; ++r) {
            in[r].get(f);
#pragma unroll
            for (int i = 0; i < V; ++i) a[i] = fmaf(k.w[r][i], f[i], a[i]);
            if (r) store_v<V>(state + (long long)(r - 1) * g.D, f);
        }
        if (g.silu)
#pragma unroll
            for (int i = 0; i < V; ++i) a[i] *= sigmoid_for<T>(a[i]);
        store_v<V>(static_cast<T *>(g.out) + n * g.D + c, a);
#pragma unroll
        for (int r = 0; r < W; ++r) in[r] = next[r];
    }
}

bool al(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Whether every row of the call's tensors starts on an `a`-byte boundary.
bool rows_aligned(const ConvArgs &g, int es, size_t a) {
    for (const void *p : {g.x, g.state0, (const void *)g.out, (const void *)g.final_state, g.dout, g.dfinal,
                          (const void *)g.dx, (const void *)g.dstate0})
        if (!al(p, a)) return false;
    return ((size_t)g.D * es) % a == 0 && ((size_t)g.ld_x * es) % a == 0;
}

template <int W, int V, int BATCH, typename T>
cudaError_t forward_t(const ConvArgs &g, int sms, cudaStream_t st) {
    const int nvec = (g.D + V - 1) / V;
    int bx = 1;
    while (bx < nvec && bx < kConvThreads) bx *= 2;
    const int runs = kConvThreads / bx;
    // long runs load the taps, the rows in front of them and their sequence's offsets less
    // often; short ones fill the SMs
    int run = 64;
    while (run > BATCH && nvec * (g.ax.ntok / run) < sms * 1024LL) run /= 2;
    const long long tok_blocks = (g.ax.ntok + (long long)runs * run - 1) / ((long long)runs * run);
    const long long seq_blocks = (W > 1 && g.final_state) ? (g.ax.nseq + runs - 1) / runs : 0;
    const long long rest_blocks = g.zero_rest && g.ax.cu ? (tok_blocks < 64 ? tok_blocks : 64) : 0;
    const long long seq_end = tok_blocks + seq_blocks, blocks = seq_end + rest_blocks;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks, (unsigned)((nvec + bx - 1) / bx));
    conv_forward_kernel<W, V, BATCH, T><<<grid, kConvThreads, 0, st>>>(g, bx, run, tok_blocks, seq_end);
    return cudaGetLastError();
}

template <int W, int V, typename T>
cudaError_t backward_t(const ConvArgs &g, int sms, int &blocks, cudaStream_t st) {
    const int nvec = (g.D + V - 1) / V, cols = (nvec + kBwdLanes - 1) / kBwdLanes;
    // the run whose waves of CTAs (three per SM of the one-element kernel, two
    // of the others, by their registers) end first; a run begins with some 24 tokens' worth of reads
    long long best = -1;
    int length = kBwdRunMin;
    for (int len : {16, 24, 32, 48, 64}) {
        const long long ctas = (g.ax.ntok + kBwdRuns * len - 1) / (kBwdRuns * len) * cols;
        const long long slots = (V == 1 ? 3LL : 2LL) * sms;
        const long long cost = (ctas + slots - 1) / slots * (len + 24);
        if (best < 0 || cost < best) best = cost, length = len;
    }
    blocks = (int)((g.ax.ntok + kBwdRuns * length - 1) / (kBwdRuns * length));
    if (blocks) {
        const dim3 grid((unsigned)blocks, (unsigned)cols);
        conv_backward_kernel<W, V, T><<<grid, kBwdLanes * kBwdRuns, 0, st>>>(g, length);
    }
    if (W > 1 && g.dstate0 && g.ax.nseq) {
        const dim3 grid((unsigned)g.ax.nseq, (unsigned)((g.D + kConvThreads - 1) / kConvThreads));
        conv_dstate_kernel<W, T><<<grid, kConvThreads, 0, st>>>(g);
    }
    return cudaGetLastError();
}

template <int W, int V, typename T>
cudaError_t step_t(const ConvArgs &g, int sms, cudaStream_t st) {
    const int nvec = (g.D + V - 1) / V;
    int run = 8;
    while (run > 1 && (long long)nvec * (g.ax.nseq / run) < sms * 256LL) run /= 2;
    const long long n = (long long)nvec * ((g.ax.nseq + run - 1) / run), blocks = (n + kConvThreads - 1) / kConvThreads;
    if (!blocks) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    conv_step_kernel<W, V, T><<<(unsigned)blocks, kConvThreads, 0, st>>>(g, nvec, run);
    return cudaGetLastError();
}

enum class Call { kForward, kBackward, kStep };

template <int W, typename T>
cudaError_t conv_w(const ConvArgs &g, Call call, int sms, int &blocks, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool vec = rows_aligned(g, sizeof(T), 8);
    // 8-byte accesses, four rows ahead: 80 registers. Chosen when 32768 tokens of 2048
    // channels took 70 us (61 now): 78 eight rows ahead, 85 and 93 with 16-byte accesses,
    // whose registers halve the warps
    if (call == Call::kForward) return vec ? forward_t<W, V / 2, 4, T>(g, sms, st) : forward_t<W, 1, 8, T>(g, sms, st);
    if (call == Call::kStep) return vec ? step_t<W, V / 2, T>(g, sms, st) : step_t<W, 1, T>(g, sms, st);
    // backward: 8-byte accesses, whose taps, windows and sums of W rows still fit in registers
    return vec ? backward_t<W, V / 2, T>(g, sms, blocks, st) : backward_t<W, 1, T>(g, sms, blocks, st);
}

template <typename T>
cudaError_t conv_t(const ConvArgs &g, Call call, int sms, int &blocks, cudaStream_t st) {
    switch (g.W) {
        case 1: return conv_w<1, T>(g, call, sms, blocks, st);
        case 2: return conv_w<2, T>(g, call, sms, blocks, st);
        case 3: return conv_w<3, T>(g, call, sms, blocks, st);
        default: return conv_w<4, T>(g, call, sms, blocks, st);
    }
}

cudaError_t conv_any(const ConvArgs &g, bool bf16, Call call, int sms, int &blocks, cudaStream_t st) {
    return bf16 ? conv_t<__nv_bfloat16>(g, call, sms, blocks, st) : conv_t<float>(g, call, sms, blocks, st);
}

}  // namespace

cudaError_t launch_conv_forward(const ConvArgs &g, bool bf16, int sms, cudaStream_t st) {
    int none = 0;
    return conv_any(g, bf16, Call::kForward, sms, none, st);
}

int conv_backward_blocks(long long ntok) {
    return (int)((ntok + kBwdRuns * kBwdRunMin - 1) / (kBwdRuns * kBwdRunMin));
}

cudaError_t launch_conv_backward(const ConvArgs &g, bool bf16, int sms, float *dweight, float *dbias, cudaStream_t st) {
    int blocks = 0;
    cudaError_t e = conv_any(g, bf16, Call::kBackward, sms, blocks, st);
    if (e != cudaSuccess) return e;
    return launch_colsum(g.part, blocks, (long long)g.D * (g.W + 1), (long long)g.D * g.W, dweight, g.D, dbias, nullptr,
                         st);
}

cudaError_t launch_conv_step(const ConvArgs &g, bool bf16, int sms, cudaStream_t st) {
    int none = 0;
    return conv_any(g, bf16, Call::kStep, sms, none, st);
}

}  // namespace kla
