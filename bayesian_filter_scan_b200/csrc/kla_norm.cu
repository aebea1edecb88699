// kla_norm.cu -- layer norm over the last axis, with the residual sum in front
// of it, and its gradients (sm_100a).
//   s = x + residual,  xh = (s - mean) rstd,  out = xh weight + bias
//   e = dout weight,  dx = rstd (e - mean(e) - xh mean(e xh)) (+ dsum)
//   dweight = sum over rows of dout xh,  dbias = sum over rows of dout
// A few operations per value: HBM binds. A row is held in registers between its
// passes (mean, then squared deviations from it, then the result), so it is read
// once; the variance is the mean of squared deviations, which loses nothing when
// the mean is large. Measured in bf16: the norm of a residual sum, 32768 rows of 2048
// (two tensors in, two out), 105 us (5.1 TB/s); 524288 rows of 128 forward 60 us (4.5
// TB/s), backward 79 us (5.1 TB/s); in fp32 212, 109 and 144 us (5.1, 4.9 and 5.6 TB/s).
// Rows that are no multiple of 16 bytes go one value per access, and a thread holds up to
// 64 of them: 128 to 255 registers, and spills from 8193 values on. A residual sum of 2^26
// values in bf16, forward and backward: rows of 2047 198 and 508 us, 4099 448 and 827, 8191
// 261 and 680, 16383 1650 and 1404, against 104 and 105 (2048), 97 and 98 (4096), 109 and
// 122 (8192), 123 and 266 (16384). fp32 rows of 16384, which spill too, 269 and 857.
#include "kla_block.cuh"

namespace kla {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWide = 512;    // backward pass of rows wider than 4096 values

// Sums over the `lanes` lanes (a power of two) and `warps` warps that share a row, the
// same values in all of them, for U rows at once. red: [U][warps of the CTA].
template <int U, int W>
__device__ __forceinline__ void row_sums(float (&v)[U], int lanes, int warps, float (&red)[U][W]) {
    for (int o = lanes >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] += __shfl_xor_sync(0xffffffffu, v[u], o);
    if (warps > 1) {
        const int warp = threadIdx.x >> 5, first = warp / warps * warps;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int u = 0; u < U; ++u) red[u][warp] = v[u];
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = 0.f;
        for (int w = 0; w < warps; ++w)
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] += red[u][first + w];
    }
}

// The fp32 weights of a thread's columns, kept for all its rows; `none` without.
template <int V, int NV>
__device__ __forceinline__ void columns(float (&v)[NV][V], const float *p, float none, int k0, int per_row, int D) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (k0 + j * per_row) * V + i;
            v[j][i] = p && c < D ? __ldg(p + c) : none;
        }
}

__device__ __forceinline__ float both(f32x2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return lo + hi;
}

// A row is spread over `lanes` lanes (warps == 1) or `warps` whole warps; a thread
// holds NV vectors of V values of it, strided so that accesses are contiguous across
// the row's threads. Persistent CTAs walk the rows and load the next one before they
// work on this one. Values behind D are zero and stay out of the squared deviations.
template <int V, int NV, typename T>
__global__ void __launch_bounds__(kNormThreads) norm_forward_kernel(const NormArgs g, int lanes, int warps) {
    __shared__ float red[2][2][1][kNormThreads / 32];
    using P = Pairs<V>;
    const int per_row = lanes * warps, slots = kNormThreads / per_row;
    const int k0 = threadIdx.x % per_row;
    const int D = g.D;
    const float inv = 1.f / (float)D;
    const long long step = (long long)gridDim.x * slots;
    long long row = (long long)blockIdx.x * slots + threadIdx.x / per_row;
    const T *x = static_cast<const T *>(g.x) + row * g.ld_x + k0 * V;
    const T *res = static_cast<const T *>(g.res) + row * g.ld_res + k0 * V;
    T *out = static_cast<T *>(g.out) + row * D + k0 * V, *sum = static_cast<T *>(g.sum) + row * D + k0 * V;
    Raw<V, T> rx[NV], rr[NV];
    auto load = [&](bool live) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (live && (k0 + j * per_row) * V < D) {
                rx[j].load(x + j * per_row * V);
                if (g.res) rr[j].load(res + j * per_row * V);
            }
    };
    load(row < g.rows);
    float wf[NV][V], bf[NV][V];
    columns<V, NV>(wf, g.w, 1.f, k0, per_row, D);
    columns<V, NV>(bf, g.b, 0.f, k0, per_row, D);
    P w[NV], b[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        w[j].set(wf[j]);
        b[j].set(bf[j]);
    }
    const long long rounds = (g.rows - (long long)blockIdx.x * slots + step - 1) / step;
    int par = 0;
    for (long long it = 0; it < rounds; ++it, row += step, par ^= 1) {
        const bool live = row < g.rows;
        P v[NV];
        f32x2 acc = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float f[V];
            rx[j].get(f);
            if (g.res) {
                // the sum is rounded to the tensors' type before it is normalised: it is the
                // stream that the next block adds to, and what the backward pass reads
                float r[V];
                rr[j].get(r);
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] += r[i];
                rr[j].round(f);
                if (g.sum && live && (k0 + j * per_row) * V < D) rr[j].store(sum + j * per_row * V);
                rr[j].get(f);
            }
            v[j].set(f);
            if (!live || (k0 + j * per_row) * V >= D)
#pragma unroll
                for (int k = 0; k < P::K; ++k) v[j].p[k] = 0;
#pragma unroll
            for (int k = 0; k < P::K; ++k) acc = add2(acc, v[j].p[k]);
        }
        x += step * g.ld_x;
        res += step * g.ld_res;
        load(row + step < g.rows);
        // the buffers alternate from round to round: a warp that is ahead writes the other ones
        float s[1] = {both(acc)};
        row_sums(s, lanes, warps, red[par][0]);
        const float mean = s[0] * inv;
        const f32x2 neg = V > 1 ? dup2(-mean) : pack2(-mean, 0.f);
        acc = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if ((k0 + j * per_row) * V < D) {
#pragma unroll
                for (int k = 0; k < P::K; ++k) {
                    const f32x2 d = add2(v[j].p[k], neg);
                    acc = fma2(d, d, acc);
                }
            }
        s[0] = both(acc);
        row_sums(s, lanes, warps, red[par][1]);
        const float rstd = rsqrtf(fmaf(s[0], inv, g.eps));
        if (live) {
            if (k0 == 0) {
                if (g.mean) g.mean[row] = mean;
                if (g.rstd) g.rstd[row] = rstd;
            }
            const f32x2 r2 = dup2(rstd);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if ((k0 + j * per_row) * V >= D) continue;
                float f[V];
                P y;
#pragma unroll
                for (int k = 0; k < P::K; ++k) y.p[k] = fma2(mul2(add2(v[j].p[k], neg), r2), w[j].p[k], b[j].p[k]);
                y.get(f);
                store_v<V>(out + j * per_row * V, f);
            }
        }
        out += step * D;
        sum += step * D;
    }
}

// The same walk; a thread keeps its columns' sums of dweight and dbias in registers.
// The CTA's rows meet in shared memory in a fixed order, the CTAs' sums in
// launch_colsum.
template <int V, int NV, int U, int THREADS, typename T>
__global__ void __launch_bounds__(THREADS) norm_backward_kernel(const NormArgs g, int lanes, int warps) {
    extern __shared__ float sm[];
    __shared__ float red[2][2 * U][THREADS / 32];
    const int per_row = lanes * warps, slots = THREADS / per_row;
    const int k0 = threadIdx.x % per_row, slot = threadIdx.x / per_row;
    const int D = g.D;
    const float inv = 1.f / (float)D;
    Raw<V, T> rx[2][U][NV], ro[2][U][NV];
    float mean[2][U], rstd[2][U];
    auto load = [&](int h, long long r0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = r0 + u * slots + slot;
            if (row >= g.rows) continue;
            mean[h][u] = g.cmean[row];
            rstd[h][u] = g.crstd[row];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (k0 + j * per_row) * V;
                if (c < D) {
                    rx[h][u][j].load(static_cast<const T *>(g.x) + row * g.ld_x + c);
                    ro[h][u][j].load(static_cast<const T *>(g.dout) + row * D + c);
                }
            }
        }
    };
    const long long step = (long long)gridDim.x * slots * U;
    long long r0 = (long long)blockIdx.x * slots * U;
    load(0, r0);
    float w[NV][V], dw[NV][V], db[NV][V];
    columns<V, NV>(w, g.w, 1.f, k0, per_row, D);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[j][i] = db[j][i] = 0.f;
    for (int par = 0; r0 < g.rows; r0 += step, par ^= 1) {
        load(1, r0 + step);
        float s[2 * U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s[2 * u] = s[2 * u + 1] = 0.f;
            if (r0 + u * slots + slot >= g.rows) continue;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if ((k0 + j * per_row) * V >= D) continue;
                float xv[V], o[V];
                rx[0][u][j].get(xv);
                ro[0][u][j].get(o);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = (xv[i] - mean[0][u]) * rstd[0][u], e = o[i] * w[j][i];
                    dw[j][i] = fmaf(o[i], xh, dw[j][i]);
                    db[j][i] += o[i];
                    s[2 * u] += e;
                    s[2 * u + 1] = fmaf(e, xh, s[2 * u + 1]);
                }
            }
        }
        // the buffers alternate from round to round: a warp that is ahead writes the other one
        row_sums(s, lanes, warps, red[par]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = r0 + u * slots + slot;
            if (row >= g.rows) continue;
            const float m0 = s[2 * u] * inv, m1 = s[2 * u + 1] * inv;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (k0 + j * per_row) * V;
                if (c >= D) continue;
                float xv[V], o[V], d[V];
                rx[0][u][j].get(xv);
                ro[0][u][j].get(o);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = (xv[i] - mean[0][u]) * rstd[0][u];
                    d[i] = (o[i] * w[j][i] - m0 - xh * m1) * rstd[0][u];
                }
                if (g.dsum) {
                    float r[V];
                    load_v<V>(static_cast<const T *>(g.dsum) + row * D + c, r);
#pragma unroll
                    for (int i = 0; i < V; ++i) d[i] += r[i];
                }
                store_v<V>(static_cast<T *>(g.dx) + row * D + c, d);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mean[0][u] = mean[1][u];
            rstd[0][u] = rstd[1][u];
#pragma unroll
            for (int j = 0; j < NV; ++j) rx[0][u][j] = rx[1][u][j], ro[0][u][j] = ro[1][u][j];
        }
    }
    if (!g.part) return;
    // [slot][2][D] in shared memory when a CTA holds several rows
    float *part = g.part + (long long)blockIdx.x * 2 * D;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (k0 + j * per_row) * V;
        if (c >= D) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (slots == 1) {
                part[c + i] = dw[j][i];
                part[D + c + i] = db[j][i];
            } else {
                sm[(slot * 2) * D + c + i] = dw[j][i];
                sm[(slot * 2 + 1) * D + c + i] = db[j][i];
            }
        }
    }
    if (slots == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * D; c += THREADS) {
        float t = 0.f;
        for (int r = 0; r < slots; ++r) t += sm[r * 2 * D + c];
        part[c] = t;
    }
}

bool al16(const void *p) { return ((uintptr_t)p & 15) == 0; }

bool rows_aligned(const NormArgs &g, int es) {
    for (const void *p : {g.x, g.res, (const void *)g.out, (const void *)g.sum, g.dout, g.dsum, (const void *)g.dx})
        if (!al16(p)) return false;
    return ((size_t)g.D * es) % 16 == 0 && ((size_t)g.ld_x * es) % 16 == 0 &&
           (!g.res || ((size_t)g.ld_res * es) % 16 == 0);
}

// How a row of nvec vectors is spread: the smallest power of two of lanes (then of
// whole warps, up to a CTA) that leaves each at most `most` vectors.
void spread(int nvec, int most, int threads, int &lanes, int &warps) {
    lanes = 1;
    warps = 1;
    while (lanes < 32 && lanes < nvec) lanes *= 2;
    while (warps < threads / 32 && (long long)lanes * warps * most < nvec) warps *= 2;
}

template <int V, int NV, typename T>
cudaError_t fwd(const NormArgs &g, int lanes, int warps, int sms, cudaStream_t st) {
    const int rows = kNormThreads / (lanes * warps);
    // four CTAs of 64 registers a thread fit on an SM (rows on 16 bytes of up to 2048 values
    // in bf16, 1024 in fp32); of the wider variants one or two, in as many more waves
    const long long blocks = (g.rows + rows - 1) / rows, most = 4LL * sms;
    norm_forward_kernel<V, NV, T><<<(unsigned)(blocks < most ? blocks : most), kNormThreads, 0, st>>>(g, lanes, warps);
    return cudaGetLastError();
}

template <int V, int NV, int U, int THREADS, typename T>
cudaError_t bwd(const NormArgs &g, int lanes, int warps, int ctas, cudaStream_t st) {
    const int slots = THREADS / (lanes * warps);
    const size_t smem = slots > 1 ? (size_t)slots * 2 * g.D * sizeof(float) : 0;
    norm_backward_kernel<V, NV, U, THREADS, T><<<ctas, THREADS, smem, st>>>(g, lanes, warps);
    return cudaGetLastError();
}

// One vector of a row per thread while a CTA's threads suffice, up to 64 values (rows of
// 16384).
template <int V, typename T>
cudaError_t fwd_v(const NormArgs &g, int sms, cudaStream_t st) {
    const int nvec = (g.D + V - 1) / V;
    int lanes, warps;
    spread(nvec, V == 1 ? 8 : 1, kNormThreads, lanes, warps);
    const int val = (nvec + lanes * warps - 1) / (lanes * warps) * V;
    if (val <= V) return fwd<V, 1, T>(g, lanes, warps, sms, st);
    if (val <= 8) return fwd<V, 8 / V, T>(g, lanes, warps, sms, st);
    if (val <= 16) return fwd<V, 16 / V, T>(g, lanes, warps, sms, st);
    if (val <= 32) return fwd<V, 32 / V, T>(g, lanes, warps, sms, st);
    return fwd<V, 64 / V, T>(g, lanes, warps, sms, st);
}

// The backward pass keeps two sums per column besides the row: one vector per thread
// while 256 threads suffice for that, up to 16 values up to 8192, 32 up to 16384.
template <int V, typename T>
cudaError_t bwd_v(const NormArgs &g, int ctas, cudaStream_t st) {
    const int nvec = (g.D + V - 1) / V;
    int lanes, warps;
    if (nvec <= kNormThreads * (16 / V)) {
        spread(nvec, V == 1 ? 4 : 1, kNormThreads, lanes, warps);
        const int val = (nvec + lanes * warps - 1) / (lanes * warps) * V;
        if (val <= V) return bwd<V, 1, 2, kNormThreads, T>(g, lanes, warps, ctas, st);
        if (V == 1 && val <= 4) return bwd<V, V == 1 ? 4 : 1, 1, kNormThreads, T>(g, lanes, warps, ctas, st);
        return bwd<V, 16 / V, 1, kNormThreads, T>(g, lanes, warps, ctas, st);
    }
    lanes = 32;
    warps = kNormWide / 32;
    if (nvec <= kNormWide * (16 / V)) return bwd<V, 16 / V, 1, kNormWide, T>(g, lanes, warps, ctas, st);
    return bwd<V, 32 / V, 1, kNormWide, T>(g, lanes, warps, ctas, st);
}

}  // namespace

cudaError_t launch_norm_forward(const NormArgs &g, bool bf16, int sms, cudaStream_t st) {
    if (g.rows == 0) return cudaSuccess;
    if (bf16)
        return rows_aligned(g, 2) ? fwd_v<8, __nv_bfloat16>(g, sms, st) : fwd_v<1, __nv_bfloat16>(g, sms, st);
    return rows_aligned(g, 4) ? fwd_v<4, float>(g, sms, st) : fwd_v<1, float>(g, sms, st);
}

int norm_backward_ctas(long long rows, int D, int sms) {
    // rows a CTA has in flight (for the vectorised form); two CTAs of 111 registers a
    // thread fit on an SM (524288 rows of 128: 80 us, 98 with three, 82 with four); of the
    // variants with 184 registers and more, or 512 threads, one
    int per = kNormThreads * 8 * 2 / (D < 8 ? 8 : D);
    if (per < 1) per = 1;
    const long long want = (rows + per - 1) / per, most = 2LL * sms;
    return (int)(want < most ? want : most);
}

cudaError_t launch_norm_backward(const NormArgs &g, bool bf16, int ctas, float *dweight, float *dbias,
                                 cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (ctas) {
        if (bf16)
            e = rows_aligned(g, 2) ? bwd_v<8, __nv_bfloat16>(g, ctas, st) : bwd_v<1, __nv_bfloat16>(g, ctas, st);
        else
            e = rows_aligned(g, 4) ? bwd_v<4, float>(g, ctas, st) : bwd_v<1, float>(g, ctas, st);
    }
    if (e != cudaSuccess || (!dweight && !dbias)) return e;
    return launch_colsum(g.part, ctas, 2LL * g.D, g.D, dweight, g.D, dbias, nullptr, st);
}

}  // namespace kla
