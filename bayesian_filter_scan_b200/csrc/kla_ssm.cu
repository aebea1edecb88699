// kla_ssm.cu -- selective state space scan: prompts and gradients (sm_100a).
//   delta = softplus(dt + dt_bias), a = exp(delta A)
//   h_t = a_t h_{t-1} + delta_t x_t B_t,   y_t = C_t.h_t + Dskip x_t,   out = y silu(z)
// Every (token, channel, state) costs one exponential, and the exponential unit
// (16 per clock and SM) binds: 16 states are 16 exponentials for 8 bytes of a
// bf16 token. So each decay is computed once, and what splits the time axis over
// threads may not compute it again.
//
// A CTA owns CB channels of one sequence and walks it in chunks. A warp's lanes
// are CB channels x 32/CB ranges of L tokens; a thread keeps its channel's L steps
// in registers and goes through the states. Per state: the L decays, the range's
// end state from zero and its decay product (both ends of an affine map of the
// start state); the maps of the ranges before it, joined by shuffles within the
// warp and through shared memory between warps, give the thread its true start
// state; it then replays its tokens with the same decays. The backward pass joins
// the adjoint's maps from the right in the same way.
#include "kla_block.cuh"

namespace kla {

namespace {

constexpr int kSsmWarps = 8;
constexpr int kSsmThreads = kSsmWarps * 32;
constexpr int kFwdL = 16;        // tokens per thread, forward
constexpr int kBwdL = 8;         // tokens per thread, backward
constexpr int kLdPad = 4;        // floats behind a range's tokens in shared memory: ranges on other banks
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// softplus and its slope; both in fp32 with the accurate exponential
__device__ __forceinline__ float softplus_f(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

// The shared-memory tile of B or C: [state][range][L + pad]. Its state stride is
// 4 floats off a multiple of the banks, so that a warp's writes of several states
// of a token spread over them.
template <int CB, int L>
struct Tile {
    static constexpr int kSub = 32 / CB;                    // ranges per warp
    static constexpr int kRanges = kSsmWarps * kSub;        // ranges per chunk
    static constexpr int kTok = kRanges * L;                // tokens per chunk
    static constexpr int kRow = L + kLdPad;                 // floats per range
    static constexpr int kState = kRanges * kRow + 4;       // floats per state
    static constexpr int kNB = kTok <= 256 ? 16 : 8;        // states staged at once
    static __device__ __forceinline__ int at(int n, int t) { return n * kState + (t / L) * kRow + t % L; }
};

// States [n0, n0 + kNB) of the chunk's rows of B or C into shared memory as fp32;
// zero behind the sequence's end and behind the last state.
template <int CB, int L, typename T>
__device__ __forceinline__ void stage(float *dst, const T *src, long long ld, long long t0, long long t1, int n0,
                                      int N) {
    using S = Tile<CB, L>;
    for (int e = threadIdx.x; e < S::kTok * S::kNB; e += kSsmThreads) {
        const int n = e % S::kNB, t = e / S::kNB;
        float v = 0.f;
        if (n0 + n < N && t0 + t < t1) v = to_f(src[(t0 + t) * ld + n0 + n]);
        dst[S::at(n, t)] = v;
    }
}

template <int CB, int L, int NP>
struct FwdSmem {
    static __host__ __device__ size_t bytes(int npad) {
        using S = Tile<CB, L>;
        return sizeof(float) * (2 * (size_t)S::kNB * S::kState + 2 * (size_t)npad * CB + 4 * NP * kSsmWarps * CB);
    }
};

// The unit of a CTA: sequence and channel tile; tiles do not straddle groups.
struct Unit {
    int n, tile, group, c;     // c: the thread's channel, or -1 behind the group's end
};
template <int CB>
__device__ __forceinline__ Unit unit_of(const SsmArgs &g, int lane_c) {
    const int per = g.D / g.G, tiles = (per + CB - 1) / CB;
    Unit u;
    u.n = blockIdx.x / (tiles * g.G);
    u.tile = blockIdx.x % (tiles * g.G);
    u.group = u.tile / tiles;
    const int i = (u.tile % tiles) * CB + lane_c;
    u.c = i < per ? u.group * per + i : -1;
    return u;
}

// OUT: writes out (else only states: the walk before a backward pass without
// recorded states). NP states per round share one barrier.
template <int CB, int NP, bool OUT, typename T>
__global__ void __launch_bounds__(kSsmThreads, 2) ssm_forward_kernel(const SsmArgs g) {
    constexpr int L = kFwdL;
    using S = Tile<CB, L>;
    extern __shared__ __align__(16) float sm[];
    const int npad = (g.N + NP - 1) / NP * NP;
    float *sB = sm, *sC = sB + S::kNB * S::kState;
    float *carry = sC + S::kNB * S::kState;                       // [2][npad][CB]
    float2 *exch = reinterpret_cast<float2 *>(carry + 2 * npad * CB);  // [2][NP][warps][CB]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lc = lane % CB, sub = lane / CB;
    const int range = warp * S::kSub + sub;
    const Unit u = unit_of<CB>(g, lc);
    long long s0, s1;
    g.ax.range(u.n, s0, s1);
    const bool live = u.c >= 0;
    const int c = live ? u.c : 0;
    const T *x = static_cast<const T *>(g.x) + c, *dt = static_cast<const T *>(g.dt) + c;
    const T *z = g.z ? static_cast<const T *>(g.z) + c : nullptr;
    const T *Bm = static_cast<const T *>(g.Bm) + (long long)u.group * g.N;
    const T *Cm = static_cast<const T *>(g.Cm) + (long long)u.group * g.N;
    const float bias = g.dt_bias ? g.dt_bias[c] : 0.f, skip = g.Dskip ? g.Dskip[c] : 0.f;
    const float *A = g.A + (long long)c * g.N;
    for (int e = threadIdx.x; e < npad * CB; e += kSsmThreads) {
        const int n = e % npad, j = e / npad;
        const int ch = unit_of<CB>(g, j).c;
        carry[n * CB + j] = (g.state0 && ch >= 0 && n < g.N) ? g.state0[((long long)u.n * g.D + ch) * g.N + n] : 0.f;
    }
    int par = 0, xp = 0;       // halves of carry and exch in use
    for (long long t0 = s0; t0 < s1; t0 += S::kTok, par ^= 1) {
        const long long tk = t0 + range * L;
        float del[L], dx[L], y[L], sum = 0.f;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            // tokens behind the end: step 0, so decay 1 and input 0
            del[i] = dx[i] = y[i] = 0.f;
            if (live && tk + i < s1) {
                const float r = to_f(dt[(tk + i) * g.ld_dt]) + bias;
                del[i] = g.softplus ? softplus_f(r) : r;
                dx[i] = del[i] * to_f(x[(tk + i) * g.ld_x]);
            }
            sum += del[i];
        }
        // where this range's start state is recorded, if it is
        float *ck = nullptr;
        if (g.states && live && tk < s1 && range * L % kSsmCkpt == 0)
            ck = g.states + (ssm_ckpt_base(s0, u.n) + (tk - s0) / kSsmCkpt) * g.N * g.D + c;
        for (int n0 = 0; n0 < g.N; n0 += S::kNB) {
            __syncthreads();
            stage<CB, L>(sB, Bm, g.ld_b, t0, s1, n0, g.N);
            if (OUT) stage<CB, L>(sC, Cm, g.ld_c, t0, s1, n0, g.N);
            __syncthreads();
            const int n1 = min(n0 + S::kNB, g.N);
            for (int n = n0; n < n1; n += NP, xp ^= 1) {
                float a[NP][L], P[NP], H[NP];
#pragma unroll
                for (int k = 0; k < NP; ++k) {
                    const float A2 = n + k < g.N ? A[n + k] * kLog2e : 0.f;
                    const float4 *b4 = reinterpret_cast<const float4 *>(sB + S::at(n - n0 + k, range * L));
                    float h = 0.f;
#pragma unroll
                    for (int q = 0; q < L / 4; ++q) {
                        const float4 b = b4[q];
                        const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            a[k][4 * q + i] = ex2(del[4 * q + i] * A2);
                            h = fmaf(a[k][4 * q + i], h, dx[4 * q + i] * bb[i]);
                        }
                    }
                    P[k] = ex2(sum * A2);
                    H[k] = h;
                    // inclusive join over the warp's ranges, later after earlier
#pragma unroll
                    for (int o = 1; o < S::kSub; o *= 2) {
                        const float p = __shfl_up_sync(0xffffffffu, P[k], o * CB);
                        const float hh = __shfl_up_sync(0xffffffffu, H[k], o * CB);
                        if (sub >= o) {
                            H[k] = fmaf(P[k], hh, H[k]);
                            P[k] *= p;
                        }
                    }
                    if (sub == S::kSub - 1) exch[((xp * NP + k) * kSsmWarps + warp) * CB + lc] = make_float2(P[k], H[k]);
                    // exclusive
                    P[k] = __shfl_up_sync(0xffffffffu, P[k], S::kSub > 1 ? CB : 0);
                    H[k] = __shfl_up_sync(0xffffffffu, H[k], S::kSub > 1 ? CB : 0);
                    if (sub == 0) P[k] = 1.f, H[k] = 0.f;
                }
                __syncthreads();
#pragma unroll
                for (int k = 0; k < NP; ++k) {
                    float h = carry[(par * npad + n + k) * CB + lc];
                    for (int w = 0; w < warp; ++w) {
                        const float2 e = exch[((xp * NP + k) * kSsmWarps + w) * CB + lc];
                        h = fmaf(e.x, h, e.y);
                    }
                    h = fmaf(P[k], h, H[k]);
                    if (ck && n + k < g.N) ck[(long long)(n + k) * g.D] = h;
                    const float4 *b4 = reinterpret_cast<const float4 *>(sB + S::at(n - n0 + k, range * L));
                    const float4 *c4 = reinterpret_cast<const float4 *>(sC + S::at(n - n0 + k, range * L));
#pragma unroll
                    for (int q = 0; q < L / 4; ++q) {
                        const float4 b = b4[q];
                        const float bb[4] = {b.x, b.y, b.z, b.w};
                        float cc[4] = {0.f, 0.f, 0.f, 0.f};
                        if (OUT) {
                            const float4 v = c4[q];
                            cc[0] = v.x; cc[1] = v.y; cc[2] = v.z; cc[3] = v.w;
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            h = fmaf(a[k][4 * q + i], h, dx[4 * q + i] * bb[i]);
                            if (OUT) y[4 * q + i] = fmaf(cc[i], h, y[4 * q + i]);
                        }
                    }
                    // the other half of carry: this chunk's readers may still be at theirs
                    if (range == S::kRanges - 1) carry[((par ^ 1) * npad + n + k) * CB + lc] = h;
                }
            }
        }
        if (OUT) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (!live || tk + i >= s1) continue;
                float v = fmaf(skip, to_f(x[(tk + i) * g.ld_x]), y[i]);
                if (z) {
                    const float zz = to_f(z[(tk + i) * g.ld_z]);
                    v *= zz * sigmoid_f(zz);
                }
                static_cast<T *>(g.out)[(tk + i) * g.D + c] = from_f<T>(v);
            }
        }
    }
    if (!g.final_state) return;
    __syncthreads();
    for (int e = threadIdx.x; e < npad * CB; e += kSsmThreads) {
        const int n = e % npad, j = e / npad;
        const int ch = unit_of<CB>(g, j).c;
        if (ch >= 0 && n < g.N) g.final_state[((long long)u.n * g.D + ch) * g.N + n] = carry[(par * npad + n) * CB + j];
    }
}

// Sums v[16] over the CB channel lanes of a range, by halving: after step o a lane
// holds half as many values, each the sum of twice as many lanes. Lane lc ends
// with values lc * 16/CB + j, j < 16/CB.
template <int CB>
__device__ __forceinline__ void sum_over_channels(float (&v)[16], int lc) {
    int count = 16;
#pragma unroll
    for (int o = CB / 2; o > 0; o >>= 1) {
        count >>= 1;
        const bool up = lc & o;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j < count) {
                const float send = up ? v[j] : v[j + count];
                const float keep = up ? v[j + count] : v[j];
                v[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        }
    }
}

template <int CB>
struct BwdSmem {
    static __host__ __device__ size_t bytes(int N) {
        using S = Tile<CB, kBwdL>;
        // B, C; the adjoint's carry (two halves); exchange; dA and the two channel sums per warp
        return sizeof(float) * (2 * (size_t)S::kNB * S::kState + 2 * (size_t)N * CB + 2 * 4 * kSsmWarps * CB +
                                (size_t)kSsmWarps * (N + 2) * CB);
    }
};

// Chunks from the last to the first. Per state: decays, the forward walk from the
// recorded state before the chunk, the adjoint walk dh_t = C_t g_t + a_{t+1} dh_{t+1}
// (g: the gradient at y) whose incoming value joins from the right, and the sums
// over channels of dh delta x (dB) and g h (dC), which leave as the tile's partial
// sums: a second kernel adds the tiles in a fixed order.
template <int CB, typename T>
__global__ void __launch_bounds__(kSsmThreads, 2) ssm_backward_kernel(const SsmArgs g) {
    constexpr int L = kBwdL;
    using S = Tile<CB, L>;
    static_assert(S::kTok % kSsmCkpt == 0, "chunks start at recorded states");
    extern __shared__ __align__(16) float sm[];
    float *sB = sm, *sC = sB + S::kNB * S::kState;
    float4 *exch = reinterpret_cast<float4 *>(sC + S::kNB * S::kState);    // [2][warps][CB]
    float *carry = reinterpret_cast<float *>(exch + 2 * kSsmWarps * CB);    // [2][N][CB]
    float *sA = carry + 2 * g.N * CB;                                       // [warps][N + 2][CB]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lc = lane % CB, sub = lane / CB;
    const int range = warp * S::kSub + sub;
    const Unit u = unit_of<CB>(g, lc);
    long long s0, s1;
    g.ax.range(u.n, s0, s1);
    const bool live = u.c >= 0;
    const int c = live ? u.c : 0;
    const T *x = static_cast<const T *>(g.x) + c, *dt = static_cast<const T *>(g.dt) + c;
    const T *z = g.z ? static_cast<const T *>(g.z) + c : nullptr;
    const T *dout = static_cast<const T *>(g.dout) + c;
    const T *Bm = static_cast<const T *>(g.Bm) + (long long)u.group * g.N;
    const T *Cm = static_cast<const T *>(g.Cm) + (long long)u.group * g.N;
    const float bias = g.dt_bias ? g.dt_bias[c] : 0.f, skip = g.Dskip ? g.Dskip[c] : 0.f;
    const float *A = g.A + (long long)c * g.N;
    float *part = g.part_bc + (long long)u.tile * 2 * g.N * g.ax.ntok;
    for (int e = threadIdx.x; e < g.N * CB; e += kSsmThreads) {
        const int n = e % g.N, j = e / g.N;
        const int ch = unit_of<CB>(g, j).c;
        carry[n * CB + j] = (g.dfinal && ch >= 0) ? g.dfinal[((long long)u.n * g.D + ch) * g.N + n] : 0.f;
    }
    for (int e = threadIdx.x; e < kSsmWarps * (g.N + 2) * CB; e += kSsmThreads) sA[e] = 0.f;
    float sumD = 0.f, sumT = 0.f;
    int par = 0, xp = 0;
    const long long chunks = (s1 - s0 + S::kTok - 1) / S::kTok;
    for (long long k = chunks - 1; k >= 0; --k, par ^= 1) {
        const long long t0 = s0 + k * S::kTok, tk = t0 + range * L;
        float del[L], dx[L], go[L], ddel[L], du[L], y[L], sum = 0.f;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            del[i] = dx[i] = go[i] = ddel[i] = du[i] = y[i] = 0.f;
            if (live && tk + i < s1) {
                const float r = to_f(dt[(tk + i) * g.ld_dt]) + bias;
                del[i] = g.softplus ? softplus_f(r) : r;
                dx[i] = del[i] * to_f(x[(tk + i) * g.ld_x]);
                go[i] = to_f(dout[(tk + i) * g.D]);
                if (z) {
                    const float zz = to_f(z[(tk + i) * g.ld_z]);
                    go[i] *= zz * sigmoid_f(zz);
                }
            }
            sum += del[i];
        }
        const float *ck = g.states + (ssm_ckpt_base(s0, u.n) + k * (S::kTok / kSsmCkpt)) * g.N * g.D + c;
        for (int n0 = 0; n0 < g.N; n0 += S::kNB) {
            __syncthreads();
            stage<CB, L>(sB, Bm, g.ld_b, t0, s1, n0, g.N);
            stage<CB, L>(sC, Cm, g.ld_c, t0, s1, n0, g.N);
            __syncthreads();
            const int n1 = min(n0 + S::kNB, g.N);
            for (int n = n0; n < n1; ++n, xp ^= 1) {
                const float An = A[n], A2 = An * kLog2e;
                const float start = live ? ck[(long long)n * g.D] : 0.f;
                const float *bp = sB + S::at(n - n0, range * L), *cp = sC + S::at(n - n0, range * L);
                float a[L], H = 0.f, Q = 0.f;
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    a[i] = ex2(del[i] * A2);
                    H = fmaf(a[i], H, dx[i] * bp[i]);
                }
#pragma unroll
                for (int i = L - 1; i >= 0; --i) Q = a[i] * fmaf(cp[i], go[i], Q);
                const float P = ex2(sum * A2);
                // maps of the warp's earlier ranges (forward) and later ranges (adjoint)
                float pf = P, pb = P;
#pragma unroll
                for (int o = 1; o < S::kSub; o *= 2) {
                    const float p = __shfl_up_sync(0xffffffffu, pf, o * CB), h = __shfl_up_sync(0xffffffffu, H, o * CB);
                    if (sub >= o) {
                        H = fmaf(pf, h, H);
                        pf *= p;
                    }
                    const float r = __shfl_down_sync(0xffffffffu, pb, o * CB), q = __shfl_down_sync(0xffffffffu, Q, o * CB);
                    if (sub + o < S::kSub) {
                        Q = fmaf(pb, q, Q);
                        pb *= r;
                    }
                }
                float4 *ex = exch + (xp * kSsmWarps + warp) * CB + lc;
                if (sub == S::kSub - 1) ex->x = pf, ex->y = H;
                if (sub == 0) ex->z = Q;
                if constexpr (S::kSub > 1) {
                    pf = __shfl_up_sync(0xffffffffu, pf, CB);
                    H = __shfl_up_sync(0xffffffffu, H, CB);
                    pb = __shfl_down_sync(0xffffffffu, pb, CB);
                    Q = __shfl_down_sync(0xffffffffu, Q, CB);
                }
                if (sub == 0) pf = 1.f, H = 0.f;
                if (sub == S::kSub - 1) pb = 1.f, Q = 0.f;
                __syncthreads();
                float h = start, q = carry[(par * g.N + n) * CB + lc];
                for (int w = 0; w < warp; ++w) {
                    const float4 e = exch[(xp * kSsmWarps + w) * CB + lc];
                    h = fmaf(e.x, h, e.y);
                }
                for (int w = kSsmWarps - 1; w > warp; --w) {
                    const float4 e = exch[(xp * kSsmWarps + w) * CB + lc];
                    q = fmaf(e.x, q, e.z);
                }
                h = fmaf(pf, h, H);
                q = fmaf(pb, q, Q);
                float hs[L + 1], v[16];
                hs[0] = h;
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    hs[i + 1] = fmaf(a[i], hs[i], dx[i] * bp[i]);
                    y[i] = fmaf(cp[i], hs[i + 1], y[i]);
                    v[8 + i] = go[i] * hs[i + 1];
                }
                float dA = 0.f;
#pragma unroll
                for (int i = L - 1; i >= 0; --i) {
                    const float dh = fmaf(cp[i], go[i], q);
                    v[i] = dh * dx[i];
                    du[i] = fmaf(dh, bp[i], du[i]);
                    q = a[i] * dh;
                    const float m = q * hs[i];         // dL/d(delta A)
                    ddel[i] = fmaf(m, An, ddel[i]);
                    dA = fmaf(m, del[i], dA);
                }
                if (range == 0) carry[((par ^ 1) * g.N + n) * CB + lc] = q;
#pragma unroll
                for (int o = CB; o < 32; o *= 2) dA += __shfl_xor_sync(0xffffffffu, dA, o);
                if (sub == 0) sA[(warp * (g.N + 2) + n) * CB + lc] += dA;
                // dead lanes hold zeros: their steps, inputs and gradients are zero
                sum_over_channels<CB>(v, lc);
#pragma unroll
                for (int j = 0; j < 16 / CB; ++j) {
                    const int idx = lc * (16 / CB) + j, i = idx % 8;
                    if (tk + i < s1) part[((long long)(idx / 8) * g.N + n) * g.ax.ntok + tk + i] = v[j];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (!live || tk + i >= s1) continue;
            const long long t = tk + i;
            const float r = to_f(dt[t * g.ld_dt]) + bias, xx = to_f(x[t * g.ld_x]);
            const float dd = (ddel[i] + du[i] * xx) * (g.softplus ? sigmoid_f(r) : 1.f);
            static_cast<T *>(g.dx)[t * g.D + c] = from_f<T>(fmaf(du[i], del[i], skip * go[i]));
            static_cast<T *>(g.ddt)[t * g.D + c] = from_f<T>(dd);
            sumT += dd;
            sumD = fmaf(go[i], xx, sumD);
            if (z) {
                const float zz = to_f(z[t * g.ld_z]), s = sigmoid_f(zz);
                const float full = fmaf(skip, xx, y[i]);
                static_cast<T *>(g.dz)[t * g.D + c] =
                    from_f<T>(to_f(dout[t * g.D]) * full * s * fmaf(zz, 1.f - s, 1.f));
            }
        }
    }
#pragma unroll
    for (int o = CB; o < 32; o *= 2) {
        sumD += __shfl_xor_sync(0xffffffffu, sumD, o);
        sumT += __shfl_xor_sync(0xffffffffu, sumT, o);
    }
    if (sub == 0) {
        sA[(warp * (g.N + 2) + g.N) * CB + lc] = sumD;
        sA[(warp * (g.N + 2) + g.N + 1) * CB + lc] = sumT;
    }
    __syncthreads();
    float *par_out = g.part_par + (long long)u.n * g.D * (g.N + 2);
    for (int e = threadIdx.x; e < (g.N + 2) * CB; e += kSsmThreads) {
        const int n = e % (g.N + 2), j = e / (g.N + 2);
        const int ch = unit_of<CB>(g, j).c;
        if (ch < 0) continue;
        float s = 0.f;
        for (int w = 0; w < kSsmWarps; ++w) s += sA[(w * (g.N + 2) + n) * CB + j];
        if (n < g.N) par_out[(long long)ch * g.N + n] = s;
        else par_out[(long long)g.D * n + ch] = s;
    }
    if (g.dstate0)
        for (int e = threadIdx.x; e < g.N * CB; e += kSsmThreads) {
            const int n = e % g.N, j = e / g.N;
            const int ch = unit_of<CB>(g, j).c;
            if (ch >= 0) g.dstate0[((long long)u.n * g.D + ch) * g.N + n] = carry[(par * g.N + n) * CB + j];
        }
}

// dB, dC of 32 tokens of one group: the tiles' partial sums added in tile order,
// turned through shared memory into the tensors' layout.
constexpr int kBcRows = 16;      // (which, state) rows at once
template <typename T>
__global__ void __launch_bounds__(256) ssm_bc_kernel(const SsmArgs g, int tiles) {
    __shared__ float sm[kBcRows][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = blockIdx.y;
    const long long t0 = (long long)blockIdx.x * 32, t = t0 + lane;
    const long long stride = 2LL * g.N * g.ax.ntok;
    for (int r0 = 0; r0 < 2 * g.N; r0 += kBcRows) {
        for (int r = warp; r < kBcRows && r0 + r < 2 * g.N; r += 8) {
            float s = 0.f;
            if (t < g.ax.ntok) {
                const float *p = g.part_bc + (long long)group * tiles * stride + (r0 + r) * g.ax.ntok + t;
#pragma unroll 8
                for (int k = 0; k < tiles; ++k) s += p[k * stride];
            }
            sm[r][lane] = s;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < 32 * kBcRows; e += 256) {
            const int r = e % kBcRows, i = e / kBcRows;
            const int row = r0 + r;
            if (row >= 2 * g.N || t0 + i >= g.ax.ntok) continue;
            // tokens of no sequence keep their rows
            if (g.ax.cu && (t0 + i < g.ax.cu[0] || t0 + i >= g.ax.cu[g.ax.nseq])) continue;
            T *o = static_cast<T *>(row < g.N ? g.dBm : g.dCm);
            o[((t0 + i) * g.G + group) * g.N + row % g.N] = from_f<T>(sm[r][i]);
        }
        __syncthreads();
    }
}

template <int CB, bool OUT, typename T>
cudaError_t forward_cb(const SsmArgs &g, long long units, cudaStream_t st) {
    constexpr int NP = 2;
    static PerDevice<bool> attr;
    const size_t smem = FwdSmem<CB, kFwdL, NP>::bytes((g.N + NP - 1) / NP * NP);
    auto kern = ssm_forward_kernel<CB, NP, OUT, T>;
    cudaError_t e = ensure_smem_attr(attr, kern, (int)FwdSmem<CB, kFwdL, NP>::bytes(kSsmMaxN));
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)units, kSsmThreads, smem, st>>>(g);
    return cudaGetLastError();
}

template <bool OUT, typename T>
cudaError_t forward_t(const SsmArgs &g, int sms, cudaStream_t st) {
    const int per = g.D / g.G;
    auto units = [&](int cb) { return (long long)g.ax.nseq * g.G * ((per + cb - 1) / cb); };
    if (units(4) > 0x7fffffffLL) return cudaErrorInvalidValue;
    // the widest tile whose units still give every SM two CTAs; narrower tiles
    // put more of a sequence's ranges side by side
    if (units(32) >= 2 * sms) return forward_cb<32, OUT, T>(g, units(32), st);
    if (units(16) >= 2 * sms) return forward_cb<16, OUT, T>(g, units(16), st);
    return forward_cb<8, OUT, T>(g, units(8), st);
}

constexpr int kBwdCB = 16;

template <typename T>
cudaError_t backward_t(const SsmArgs &g, cudaStream_t st) {
    static PerDevice<bool> attr;
    const int tiles = ssm_backward_tiles(g.D, g.G);
    const long long units = (long long)g.ax.nseq * tiles;
    if (units > 0x7fffffffLL) return cudaErrorInvalidValue;
    auto kern = ssm_backward_kernel<kBwdCB, T>;
    cudaError_t e = ensure_smem_attr(attr, kern, (int)BwdSmem<kBwdCB>::bytes(kSsmMaxN));
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)units, kSsmThreads, BwdSmem<kBwdCB>::bytes(g.N), st>>>(g);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (g.ax.ntok) {
        const dim3 grid((unsigned)((g.ax.ntok + 31) / 32), (unsigned)g.G);
        ssm_bc_kernel<T><<<grid, 256, 0, st>>>(g, tiles / g.G);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_ssm_forward(const SsmArgs &g, bool bf16, int sms, cudaStream_t st) {
    if (g.ax.nseq == 0) return cudaSuccess;
    if (g.out) return bf16 ? forward_t<true, __nv_bfloat16>(g, sms, st) : forward_t<true, float>(g, sms, st);
    return bf16 ? forward_t<false, __nv_bfloat16>(g, sms, st) : forward_t<false, float>(g, sms, st);
}

// Channel tiles of the backward pass over all groups.
int ssm_backward_tiles(int D, int G) { return G * ((D / G + kBwdCB - 1) / kBwdCB); }

cudaError_t launch_ssm_backward(const SsmArgs &g, bool bf16, int sms, cudaStream_t st) {
    (void)sms;
    cudaError_t e = cudaSuccess;
    if (g.ax.nseq) e = bf16 ? backward_t<__nv_bfloat16>(g, st) : backward_t<float>(g, st);
    if (e != cudaSuccess) return e;
    const long long da = (long long)g.D * g.N, cols = da + 2LL * g.D;
    return launch_colsum(g.part_par, g.ax.nseq, cols, da, g.dA, g.D, g.dDskip, g.ddt_bias, st);
}

}  // namespace kla
