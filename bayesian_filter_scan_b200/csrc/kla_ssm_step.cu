// kla_ssm_step.cu -- one token per row through the selective scan, the state
// updated in place (sm_100a). Per channel N states are read and written in fp32
// (8 N bytes) for a handful of operations: HBM binds for many rows, launch
// latency for few.
#include "kla_block.cuh"

namespace kla {

namespace {

constexpr int kStepThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float softplus_f(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

// `lanes` lanes (a power of two) share a channel; each takes V states at a time.
template <int V, typename T>
__global__ void __launch_bounds__(kStepThreads) ssm_step_kernel(const SsmArgs g, int lanes, long long items) {
    const long long e = ((long long)blockIdx.x * kStepThreads + threadIdx.x) / lanes;
    const int l = threadIdx.x % lanes;
    const bool live = e < items;
    const long long row = live ? e / g.D : 0;
    const int c = live ? (int)(e - row * g.D) : 0, group = c / (g.D / g.G);
    const float x = to_f(static_cast<const T *>(g.x)[row * g.ld_x + c]);
    const float r = to_f(static_cast<const T *>(g.dt)[row * g.ld_dt + c]) + (g.dt_bias ? g.dt_bias[c] : 0.f);
    const float del = g.softplus ? softplus_f(r) : r, dx = del * x;
    const T *Bm = static_cast<const T *>(g.Bm) + row * g.ld_b + (long long)group * g.N;
    const T *Cm = static_cast<const T *>(g.Cm) + row * g.ld_c + (long long)group * g.N;
    const float *A = g.A + (long long)c * g.N;
    float *state = g.final_state + (row * g.D + c) * g.N;
    float y = 0.f;
    for (int n = l * V; n < g.N; n += lanes * V) {
        float h[V], a[V];
        load_v<V>(state + n, h);
        load_v<V>(A + n, a);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            h[i] = fmaf(exp2f(del * (a[i] * kLog2e)), h[i], dx * to_f(Bm[n + i]));
            y = fmaf(to_f(Cm[n + i]), h[i], y);
        }
        if (live) store_v<V>(state + n, h);
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (!live || l) return;
    if (g.Dskip) y = fmaf(g.Dskip[c], x, y);
    if (g.z) {
        const float zz = to_f(static_cast<const T *>(g.z)[row * g.ld_z + c]);
        y *= zz * sigmoid_f(zz);
    }
    static_cast<T *>(g.out)[row * g.D + c] = from_f<T>(y);
}

template <int V, typename T>
cudaError_t step_t(const SsmArgs &g, cudaStream_t st) {
    int lanes = 1;
    while (lanes < 8 && lanes * V < g.N) lanes *= 2;
    const long long items = (long long)g.ax.nseq * g.D, blocks = (items * lanes + kStepThreads - 1) / kStepThreads;
    if (!blocks) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    ssm_step_kernel<V, T><<<(unsigned)blocks, kStepThreads, 0, st>>>(g, lanes, items);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ssm_step(const SsmArgs &g, bool bf16, cudaStream_t st) {
    const bool vec = g.N % 4 == 0 && ((uintptr_t)g.A & 15) == 0 && ((uintptr_t)g.final_state & 15) == 0;
    if (bf16) return vec ? step_t<4, __nv_bfloat16>(g, st) : step_t<1, __nv_bfloat16>(g, st);
    return vec ? step_t<4, float>(g, st) : step_t<1, float>(g, st);
}

}  // namespace kla
