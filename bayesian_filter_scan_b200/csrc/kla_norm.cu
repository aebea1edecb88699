// kla_norm.cu -- layer norm over the last axis, with the residual sum in front
// of it, and its gradients (sm_100a).
//   s = x + residual,  xh = (s - mean) rstd,  out = xh weight + bias
//   e = dout weight,  dx = rstd (e - mean(e) - xh mean(e xh)) (+ dsum)
//   dweight = sum over rows of dout xh,  dbias = sum over rows of dout
// A few operations per value: HBM binds. A row is held in registers between its
// passes (mean, then squared deviations from it, then the result), so it is read
// once; the variance is the mean of squared deviations, which loses nothing when
// the mean is large.
#include "kla_block.cuh"

namespace kla {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWide = 512;    // backward pass of rows wider than 4096 values

// Sum over the `lanes` lanes (a power of two) and `warps` warps that share a
// row, the same value in all of them. red: [8] floats per slot.
__device__ __forceinline__ float row_sum(float v, int lanes, int warps, float *red) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps > 1) {
        const int warp = threadIdx.x >> 5, first = warp / warps * warps;
        if ((threadIdx.x & 31) == 0) red[warp] = v;
        __syncthreads();
        v = 0.f;
        for (int w = 0; w < warps; ++w) v += red[first + w];
    }
    return v;
}

// A row is spread over `lanes` lanes (warps == 1) or `warps` whole warps; every
// thread holds NV vectors of V values, strided so that accesses are contiguous
// across the row's threads. Values behind D count as zero in the sums.
template <int V, int NV, typename T>
__global__ void __launch_bounds__(kNormThreads) norm_forward_kernel(const NormArgs g, int lanes, int warps) {
    __shared__ float red[2][kNormThreads / 32];
    const int per_row = lanes * warps, rows = kNormThreads / per_row;
    const int k0 = threadIdx.x % per_row;
    const long long row = (long long)blockIdx.x * rows + threadIdx.x / per_row;
    const bool live = row < g.rows;
    const int D = g.D;
    const T *x = static_cast<const T *>(g.x) + row * g.ld_x;
    const T *res = static_cast<const T *>(g.res) + row * g.ld_res;
    float v[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (k0 + j * per_row) * V;
        if (live && c < D) {
            load_v<V>(x + c, v[j]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[j][i] = 0.f;
        }
    }
    if (g.res) {
        // the sum is rounded to the tensors' type before it is normalised: it is
        // the stream that the next block adds to, and what the backward pass reads
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (k0 + j * per_row) * V;
            if (live && c < D) {
                float r[V];
                load_v<V>(res + c, r);
#pragma unroll
                for (int i = 0; i < V; ++i) v[j][i] = to_f(from_f<T>(v[j][i] + r[i]));
            }
        }
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) s += v[j][i];
    const float mean = row_sum(s, lanes, warps, red[0]) / (float)D;
    s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if ((k0 + j * per_row) * V < D) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = v[j][i] - mean;
                s = fmaf(d, d, s);
            }
        }
    const float rstd = 1.f / sqrtf(row_sum(s, lanes, warps, red[1]) / (float)D + g.eps);
    if (!live) return;
    if (k0 == 0) {
        if (g.mean) g.mean[row] = mean;
        if (g.rstd) g.rstd[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (k0 + j * per_row) * V;
        if (c >= D) continue;
        if (g.sum) store_v<V>(static_cast<T *>(g.sum) + row * D + c, v[j]);
        float y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float w = g.w ? __ldg(g.w + c + i) : 1.f, b = g.b ? __ldg(g.b + c + i) : 0.f;
            y[i] = fmaf((v[j][i] - mean) * rstd, w, b);
        }
        store_v<V>(static_cast<T *>(g.out) + row * D + c, y);
    }
}

// Persistent CTAs walk the rows; a thread keeps its columns' sums of dweight and
// dbias in registers. The CTA's rows meet in shared memory in a fixed order, the
// CTAs' sums in launch_colsum.
template <int V, int NV, int THREADS, typename T>
__global__ void __launch_bounds__(THREADS) norm_backward_kernel(const NormArgs g, int lanes, int warps) {
    extern __shared__ float sm[];
    __shared__ float red[2][2][THREADS / 32];
    const int per_row = lanes * warps, rows = THREADS / per_row;
    const int k0 = threadIdx.x % per_row, slot = threadIdx.x / per_row;
    const int D = g.D;
    float dw[NV][V], db[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[j][i] = db[j][i] = 0.f;
    int par = 0;
    for (long long r0 = (long long)blockIdx.x * rows; r0 < g.rows; r0 += (long long)gridDim.x * rows, par ^= 1) {
        const long long row = r0 + slot;
        const bool live = row < g.rows;
        const T *x = static_cast<const T *>(g.x) + row * g.ld_x;
        const T *dout = static_cast<const T *>(g.dout) + row * D;
        const float mean = live ? g.cmean[row] : 0.f, rstd = live ? g.crstd[row] : 0.f;
        float xh[NV][V], e[NV][V];
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (k0 + j * per_row) * V;
            if (live && c < D) {
                load_v<V>(x + c, xh[j]);
                load_v<V>(dout + c, e[j]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) xh[j][i] = mean, e[j][i] = 0.f;
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (k0 + j * per_row) * V;
            if (c >= D) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                xh[j][i] = (xh[j][i] - mean) * rstd;
                dw[j][i] = fmaf(e[j][i], xh[j][i], dw[j][i]);
                db[j][i] += e[j][i];
                if (g.w) e[j][i] *= __ldg(g.w + c + i);
                s0 += e[j][i];
                s1 = fmaf(e[j][i], xh[j][i], s1);
            }
        }
        // the buffers alternate from row to row: a warp that is ahead writes the other pair
        s0 = row_sum(s0, lanes, warps, red[par][0]) / (float)D;
        s1 = row_sum(s1, lanes, warps, red[par][1]) / (float)D;
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (k0 + j * per_row) * V;
            if (c >= D) continue;
            float d[V];
#pragma unroll
            for (int i = 0; i < V; ++i) d[i] = (e[j][i] - s0 - xh[j][i] * s1) * rstd;
            if (g.dsum) {
                float r[V];
                load_v<V>(static_cast<const T *>(g.dsum) + row * D + c, r);
#pragma unroll
                for (int i = 0; i < V; ++i) d[i] += r[i];
            }
            store_v<V>(static_cast<T *>(g.dx) + row * D + c, d);
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
            if (rows == 1) {
                part[c + i] = dw[j][i];
                part[D + c + i] = db[j][i];
            } else {
                sm[(slot * 2) * D + c + i] = dw[j][i];
                sm[(slot * 2 + 1) * D + c + i] = db[j][i];
            }
        }
    }
    if (rows == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * D; c += THREADS) {
        float s = 0.f;
        for (int r = 0; r < rows; ++r) s += sm[r * 2 * D + c];
        part[c] = s;
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
cudaError_t fwd(const NormArgs &g, int lanes, int warps, cudaStream_t st) {
    const int rows = kNormThreads / (lanes * warps);
    const long long blocks = (g.rows + rows - 1) / rows;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    norm_forward_kernel<V, NV, T><<<(unsigned)blocks, kNormThreads, 0, st>>>(g, lanes, warps);
    return cudaGetLastError();
}

template <int V, int NV, int THREADS, typename T>
cudaError_t bwd(const NormArgs &g, int lanes, int warps, int ctas, cudaStream_t st) {
    const int rows = THREADS / (lanes * warps);
    const size_t smem = rows > 1 ? (size_t)rows * 2 * g.D * sizeof(float) : 0;
    norm_backward_kernel<V, NV, THREADS, T><<<ctas, THREADS, smem, st>>>(g, lanes, warps);
    return cudaGetLastError();
}

// A warp holds a row of up to 64 values per lane (2048); wider rows take 2, 4 or 8 warps.
template <int V, typename T>
cudaError_t fwd_v(const NormArgs &g, cudaStream_t st) {
    const int nvec = (g.D + V - 1) / V;
    int lanes, warps;
    spread(nvec, 64 / V, kNormThreads, lanes, warps);
    const int val = (nvec + lanes * warps - 1) / (lanes * warps) * V;
    if (val <= V) return fwd<V, 1, T>(g, lanes, warps, st);
    if (val <= 16) return fwd<V, 16 / V, T>(g, lanes, warps, st);
    if (val <= 32) return fwd<V, 32 / V, T>(g, lanes, warps, st);
    return fwd<V, 64 / V, T>(g, lanes, warps, st);
}

// Four arrays of a row's values live in registers (xh, e and the two sums), so a
// thread takes few of them: one vector while 256 threads suffice for that, up to
// 16 values up to 8192, 32 up to 16384.
template <int V, typename T>
cudaError_t bwd_v(const NormArgs &g, int ctas, cudaStream_t st) {
    const int nvec = (g.D + V - 1) / V;
    int lanes, warps;
    if (nvec <= kNormThreads * (16 / V)) {
        spread(nvec, V == 1 ? 4 : 1, kNormThreads, lanes, warps);
        const int val = (nvec + lanes * warps - 1) / (lanes * warps) * V;
        if (val <= V) return bwd<V, 1, kNormThreads, T>(g, lanes, warps, ctas, st);
        if (V == 1 && val <= 4) return bwd<V, V == 1 ? 4 : 1, kNormThreads, T>(g, lanes, warps, ctas, st);
        return bwd<V, 16 / V, kNormThreads, T>(g, lanes, warps, ctas, st);
    }
    lanes = 32;
    warps = kNormWide / 32;
    if (nvec <= kNormWide * (16 / V)) return bwd<V, 16 / V, kNormWide, T>(g, lanes, warps, ctas, st);
    return bwd<V, 32 / V, kNormWide, T>(g, lanes, warps, ctas, st);
}

}  // namespace

cudaError_t launch_norm_forward(const NormArgs &g, bool bf16, cudaStream_t st) {
    if (g.rows == 0) return cudaSuccess;
    if (bf16)
        return rows_aligned(g, 2) ? fwd_v<8, __nv_bfloat16>(g, st) : fwd_v<1, __nv_bfloat16>(g, st);
    return rows_aligned(g, 4) ? fwd_v<4, float>(g, st) : fwd_v<1, float>(g, st);
}

int norm_backward_ctas(long long rows, int D, int sms) {
    // rows a CTA holds at once (for the vectorised form); four CTAs per SM
    int per = kNormThreads * 8 / (D < 8 ? 8 : D);
    if (per < 1) per = 1;
    const long long want = (rows + per - 1) / per, most = 4LL * sms;
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
