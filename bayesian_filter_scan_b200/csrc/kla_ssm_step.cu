// kla_ssm_step.cu -- one token per row through the selective scan, the state
// updated in place (sm_100a). Per channel N states are read and written in fp32
// (8 N bytes) for a handful of operations: HBM binds for many rows, launch
// latency for few. `lanes` lanes (a power of two) share a channel of a row; a
// thread walks rows with the next one's reads on their way while it works on this one.
// Measured: 256 rows of 4096 channels, 16 states, 33 us (4.2 TB/s) four rows at a time,
// 48 one by one, where every lane of a channel repeats the row's step and gate (with
// nothing in L2 36, fp32 tokens 38); one row 2.5 us. Rows and channels are the grid's axes: with one axis over both, the 64-bit
// division that takes an item apart and A's reads for every row cost another 14 us.
#include "kla_block.cuh"

namespace kla {

namespace {

constexpr int kStepThreads = 128;

// 2^x of two values to 6.6e-8, without the 2e-8 to 5e-8 that the approximated power of two
// is low: a state that is stepped a thousand times would add them up. 2^f for the part f in
// [-1/2, 1/2] behind the nearest integer: a polynomial of degree 6 with p(0) = 1, fitted for
// the least relative error as softplus's is (3.0e-9 with these coefficients).
__device__ __forceinline__ void exp2_near(float &x0, float &x1) {
    if (fmaxf(fabsf(x0), fabsf(x1)) > 126.f) {
        x0 = ex2(x0);
        x1 = ex2(x1);
        return;
    }
    const f32x2 x = pack2(x0, x1), t = add2(x, dup2(12582912.f));     // 1.5 * 2^23: t's low bits are the integer
    const f32x2 f = fma2(add2(t, dup2(-12582912.f)), dup2(-1.f), x);
    f32x2 p = dup2(1.5329264e-4f);
    p = fma2(p, f, dup2(1.3390969e-3f));
    p = fma2(p, f, dup2(9.618499e-3f));
    p = fma2(p, f, dup2(5.5503596e-2f));
    p = fma2(p, f, dup2(2.4022648e-1f));
    p = fma2(p, f, dup2(6.931472e-1f));
    p = fma2(p, f, dup2(1.f));
    float t0, t1;
    unpack2(t, t0, t1);
    const f32x2 scale = pack2(__int_as_float((__float_as_int(t0) << 23) + 0x3f800000),
                              __int_as_float((__float_as_int(t1) << 23) + 0x3f800000));
    unpack2(mul2(p, scale), x0, x1);
}

// What one lane reads of a row: V states, and its scalars.
template <int V, typename T>
struct StepRow {
    Raw<V, float> h;
    Raw<V, T> b, c;
    T x, dt, z;
};

// Grid: channels x row groups; a thread keeps its channel, whose A it holds, and walks
// rows. V states at a time: 4 (rows of A and the state on 16-byte boundaries, of B and C
// on as many elements' when vec_bc) with all N states in one round of the lanes, or 1.
template <int V, typename T>
__global__ void __launch_bounds__(kStepThreads) ssm_step_kernel(const SsmArgs g, int lanes, bool vec_bc) {
    const int l = threadIdx.x % lanes, rows = g.ax.nseq;
    const int at = (int)(((long long)blockIdx.x * kStepThreads + threadIdx.x) / lanes);
    const bool live = at < g.D;        // the others keep their warp's shuffles company
    const int c = live ? at : 0, group = c / (g.D / g.G);
    auto load = [&](StepRow<V, T> &it, long long row, int n) {
        it.x = static_cast<const T *>(g.x)[row * g.ld_x + c];
        it.dt = static_cast<const T *>(g.dt)[row * g.ld_dt + c];
        if (g.z) it.z = static_cast<const T *>(g.z)[row * g.ld_z + c];
        if (n >= g.N) return;
        it.h.load(g.final_state + (row * g.D + c) * g.N + n);
        const T *B = static_cast<const T *>(g.Bm) + row * g.ld_b + (long long)group * g.N + n;
        const T *C = static_cast<const T *>(g.Cm) + row * g.ld_c + (long long)group * g.N + n;
        if (V == 1 || vec_bc) {
            it.b.load(B);
            it.c.load(C);
        } else {
            float f[V], k[V];
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = to_f(B[i]), k[i] = to_f(C[i]);
            it.b.set(f);
            it.c.set(k);
        }
    };
    StepRow<V, T> cur, next;
    int row = blockIdx.y;
    if (live) load(cur, row, l * V);
    const float bias = g.dt_bias ? g.dt_bias[c] : 0.f, skip = g.Dskip ? g.Dskip[c] : 0.f;
    float a[V];
    auto load_a = [&](int n) {
        load_v<V>(g.A + (long long)c * g.N + n, a);
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] *= kLog2e;
    };
    if (l * V < g.N) load_a(l * V);
    for (; row < rows; row += gridDim.y) {
        if (live && row + gridDim.y < rows) load(next, row + gridDim.y, l * V);
        float y = 0.f;
        if (live) {
            float del = to_f(cur.dt) + bias, spare = 0.f;
            if (g.softplus) softplus2<T>(del, spare);
            const float dx = del * to_f(cur.x);
            for (int n = l * V; n < g.N; n += lanes * V) {
                if (lanes * V < g.N) {
                    load(cur, row, n);
                    load_a(n);
                }
                float h[V], b[V], cc[V];
                cur.h.get(h);
                cur.b.get(b);
                cur.c.get(cc);
                float d[V + V % 2];
#pragma unroll
                for (int i = 0; i < V + V % 2; ++i) d[i] = i < V ? del * a[i < V ? i : 0] : 0.f;
#pragma unroll
                for (int i = 0; i < V; i += 2) exp2_near(d[i], d[i + 1]);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    h[i] = fmaf(d[i], h[i], dx * b[i]);
                    y = fmaf(cc[i], h[i], y);
                }
                store_v<V>(g.final_state + ((long long)row * g.D + c) * g.N + n, h);
            }
        }
        for (int o = lanes >> 1; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (live && l == 0) {
            float v = fmaf(skip, to_f(cur.x), y);
            if (g.z) {
                const float z = to_f(cur.z);
                v *= z * sigmoid_for<T>(z);
            }
            static_cast<T *>(g.out)[(long long)row * g.D + c] = from_f<T>(v);
        }
        cur = next;
    }
}

// Four rows at a time, for channels of four lanes or more with four states each: the
// reads of four rows are in flight together, the first four lanes of a channel each take
// one row's step, gate and output, and the sums over lanes leave each of them its row's.
template <typename T>
__global__ void __launch_bounds__(kStepThreads) ssm_step_rows_kernel(const SsmArgs g, int lanes, bool vec_bc) {
    constexpr int V = 4, R = 4;
    const int l = threadIdx.x % lanes, rows = g.ax.nseq, n = l * V;
    const int at = (int)(((long long)blockIdx.x * kStepThreads + threadIdx.x) / lanes);
    const bool live = at < g.D, states = live && n < g.N;
    const int c = live ? at : 0, group = c / (g.D / g.G);
    const float bias = g.dt_bias ? g.dt_bias[c] : 0.f, skip = g.Dskip ? g.Dskip[c] : 0.f;
    float a[V] = {0.f, 0.f, 0.f, 0.f};
    if (states) load_v<V>(g.A + (long long)c * g.N + n, a);
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] *= kLog2e;
    for (int r0 = blockIdx.y * R; r0 < rows; r0 += gridDim.y * R) {
        Raw<V, float> h[R];
        Raw<V, T> b[R], cc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!states || r0 + r >= rows) continue;
            const long long row = r0 + r;
            h[r].load(g.final_state + (row * g.D + c) * g.N + n);
            const T *B = static_cast<const T *>(g.Bm) + row * g.ld_b + (long long)group * g.N + n;
            const T *C = static_cast<const T *>(g.Cm) + row * g.ld_c + (long long)group * g.N + n;
            if (vec_bc) {
                b[r].load(B);
                cc[r].load(C);
            } else {
                float f[V], k[V];
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] = to_f(B[i]), k[i] = to_f(C[i]);
                b[r].set(f);
                cc[r].set(k);
            }
        }
        const long long own = r0 + l;
        const bool mine = live && l < R && own < rows;
        float x = 0.f, del = 0.f, z = 0.f, spare = 0.f;
        if (mine) {
            x = to_f(static_cast<const T *>(g.x)[own * g.ld_x + c]);
            del = to_f(static_cast<const T *>(g.dt)[own * g.ld_dt + c]) + bias;
            if (g.z) z = to_f(static_cast<const T *>(g.z)[own * g.ld_z + c]);
        }
        if (g.softplus) softplus2<T>(del, spare);
        const float dx = del * x;
        float y[R];
        const int first = (threadIdx.x & 31) - l;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float dr = __shfl_sync(0xffffffffu, del, first + r), xr = __shfl_sync(0xffffffffu, dx, first + r);
            y[r] = 0.f;
            if (!states || r0 + r >= rows) continue;
            float e[V], f[V], k[V], q[V];
            h[r].get(f);
            b[r].get(k);
            cc[r].get(q);
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = dr * a[i];
            exp2_near(e[0], e[1]);
            exp2_near(e[2], e[3]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                f[i] = fmaf(e[i], f[i], xr * k[i]);
                y[r] = fmaf(q[i], f[i], y[r]);
            }
            store_v<V>(g.final_state + ((long long)(r0 + r) * g.D + c) * g.N + n, f);
        }
        for (int o = lanes >> 1; o >= R; o >>= 1)
#pragma unroll
            for (int r = 0; r < R; ++r) y[r] += __shfl_xor_sync(0xffffffffu, y[r], o);
        // lane l of every four keeps row l
#pragma unroll
        for (int o = R / 2; o > 0; o >>= 1) {
            const bool up = l & o;
#pragma unroll
            for (int r = 0; r < o; ++r) {
                const float send = up ? y[r] : y[r + o], keep = up ? y[r + o] : y[r];
                y[r] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        }
        if (!mine) continue;
        float v = fmaf(skip, x, y[0]);
        if (g.z) v *= z * sigmoid_for<T>(z);
        static_cast<T *>(g.out)[own * g.D + c] = from_f<T>(v);
    }
}

template <int V, typename T>
cudaError_t step_t(const SsmArgs &g, bool vec_bc, int sms, cudaStream_t st) {
    int lanes = 1;
    while (lanes < 32 && lanes * V < g.N) lanes *= 2;
    const unsigned bx = (unsigned)(((long long)g.D * lanes + kStepThreads - 1) / kStepThreads);
    const int rows = g.ax.nseq;
    if (!rows) return cudaSuccess;
    const bool four = V == 4 && lanes >= 4 && rows >= 4;
    const int items = four ? (rows + 3) / 4 : rows;        // rows, or fours of them
    long long by = (8LL * sms + bx - 1) / bx;
    if (by > items) by = items;
    if (by > 65535) by = 65535;
    // as many items for every group, as far as they go
    by = (items + (items + by - 1) / by - 1) / ((items + by - 1) / by);
    if (four) ssm_step_rows_kernel<T><<<dim3(bx, (unsigned)by), kStepThreads, 0, st>>>(g, lanes, vec_bc);
    else ssm_step_kernel<V, T><<<dim3(bx, (unsigned)by), kStepThreads, 0, st>>>(g, lanes, vec_bc);
    return cudaGetLastError();
}

template <typename T>
cudaError_t step_any(const SsmArgs &g, int sms, cudaStream_t st) {
    auto al = [](const void *p, long long bytes, size_t a) { return (((uintptr_t)p | (size_t)bytes) & (a - 1)) == 0; };
    constexpr size_t four = 4 * sizeof(T);
    const long long es = sizeof(T);
    const bool vec = g.N % 4 == 0 && al(g.A, 0, 16) && al(g.final_state, 0, 16);
    const bool vec_bc = vec && al(g.Bm, g.ld_b * es, four) && al(g.Cm, g.ld_c * es, four);
    return vec ? step_t<4, T>(g, vec_bc, sms, st) : step_t<1, T>(g, true, sms, st);
}

}  // namespace

cudaError_t launch_ssm_step(const SsmArgs &g, bool bf16, int sms, cudaStream_t st) {
    return bf16 ? step_any<__nv_bfloat16>(g, sms, st) : step_any<float>(g, sms, st);
}

}  // namespace kla
