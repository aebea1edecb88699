// kla_ssm.cu -- selective state space scan: prompts and gradients (sm_100a).
//   delta = softplus(dt + dt_bias), a = exp(delta A)
//   h_t = a_t h_{t-1} + delta_t x_t B_t,   y_t = C_t.h_t + Dskip x_t,   out = y silu(z)
// Every (token, channel, state) costs one exponential, and the exponential unit
// (16 per clock and SM) binds: 16 states are 16 exponentials for 8 bytes of a
// bf16 token. So each decay is computed once, and what splits the time axis over
// threads may not compute it again.
//
// Forward: the sequence is cut into tiles of 16 tokens that the warps of a CTA take
// in turn; a warp's lanes are CB channels x 32/CB states. A warp goes through the
// states of its tile, and for each needs the state at the tile's start from the
// warp that has the tile before: it comes through shared memory, one 64-bit word
// per channel and state that carries the tile's number beside the value, so no
// barrier is needed. Warps therefore follow one another at a distance of a state or
// two, all of them busy, each decay computed and used once, and nothing walked
// twice. A warp keeps steps, inputs and outputs of its tile in registers.
//
// Backward: a CTA owns 16 channels and walks chunks of 128 tokens. A thread has a
// channel and a range of 8 tokens; per state the ranges' maps of the start state
// (decay product, end state from zero) are joined within and across warps, and the
// adjoint's maps from the right in the same way; the thread then replays its tokens
// with the same decays.
#include <initializer_list>

#include "kla_block.cuh"

namespace kla {

namespace {

constexpr int kFwdL = 16;        // tokens of a tile, forward
constexpr int kFwdNB = 16;       // states whose B and C a warp stages at once
constexpr int kBwdWarps = 8;
constexpr int kBwdL = 8;         // tokens per thread, backward
constexpr int kLdPad = 4;        // floats behind a range's tokens in shared memory: ranges on other banks
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 values in one 64-bit register: one instruction for both.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ f32x2 dup2(float x) { return pack2(x, x); }

// softplus(x) = max(x, 0) + log(1 + y) of two values, y = e^-|x| in (0, 1]. log(1 + y)
// is y times a polynomial of degree 9 fitted to log(1 + y) / y on [0, 1] for the least
// relative error (5e-9; 1.5e-7 with fp32's rounding), so a small y keeps its digits,
// which the logarithm of a rounded 1 + y would not.
__device__ __forceinline__ void softplus2(float &x0, float &x1) {
    const f32x2 y = pack2(ex2(-kLog2e * fabsf(x0)), ex2(-kLog2e * fabsf(x1)));
    f32x2 p = dup2(-0.0032439809f);
    p = fma2(p, y, dup2(0.019851264f));
    p = fma2(p, y, dup2(-0.05695916f));
    p = fma2(p, y, dup2(0.10603617f));
    p = fma2(p, y, dup2(-0.1530557f));
    p = fma2(p, y, dup2(0.19675931f));
    p = fma2(p, y, dup2(-0.24954133f));
    p = fma2(p, y, dup2(0.33329964f));
    p = fma2(p, y, dup2(-0.499999f));
    p = fma2(p, y, dup2(1.f));
    float m0, m1;
    unpack2(fma2(p, y, pack2(fmaxf(x0, 0.f), fmaxf(x1, 0.f))), m0, m1);
    x0 = m0;
    x1 = m1;
}
__device__ __forceinline__ float sigmoid_a(float x) { return rcp(1.f + ex2(-kLog2e * x)); }

// How rows reach shared memory: pieces of 16 bytes (or a whole narrower row), of 4
// bytes, or single elements, by the alignment of the rows.
enum : int { kScalar = 0, kWord = 1, kWide = 2 };

template <int B>
__device__ __forceinline__ void cp_async(void *dst, const void *src) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(B) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Rows [0, rows) of `cols` elements at stride ld into dst[ROWS][WIDTH]; what lies
// outside is left as it is. In the modes of pieces cols is a whole number of them; in
// the widest, ROWS rows span less than 2^31 bytes.
template <int ROWS, int WIDTH, int THREADS, typename T>
__device__ __forceinline__ void copy_rows(T *dst, const T *src, long long ld, int rows, int cols, int mode, int tid) {
    constexpr int WB = WIDTH * (int)sizeof(T) < 16 ? WIDTH * (int)sizeof(T) : 16;
    if (mode == kWide) {
        constexpr int PE = WB / (int)sizeof(T), PR = WIDTH / PE;
#pragma unroll
        for (int e0 = 0; e0 < ROWS * PR; e0 += THREADS) {
            const int e = e0 + tid, r = e / PR, q = e % PR * PE;
            if ((ROWS * PR % THREADS == 0 || e < ROWS * PR) && r < rows && q < cols)
                cp_async<WB>(dst + r * WIDTH + q, reinterpret_cast<const char *>(src) +
                                                      (unsigned)(r * (int)ld + q) * (unsigned)sizeof(T));
        }
    } else if (mode == kWord) {
        constexpr int PE = 4 / (int)sizeof(T), PR = WIDTH / PE;
        for (int e = tid; e < ROWS * PR; e += THREADS) {
            const int r = e / PR, q = e % PR * PE;
            if (r < rows && q < cols) cp_async<4>(dst + r * WIDTH + q, src + r * ld + q);
        }
    } else {
#pragma unroll 8
        for (int e = tid; e < ROWS * WIDTH; e += THREADS) {
            const int r = e / WIDTH, q = e % WIDTH;
            if (r < rows && q < cols) dst[r * WIDTH + q] = src[r * ld + q];
        }
    }
}

// A chunk: ranges of L tokens, 32/CB per warp. B and C of a chunk stand in shared
// memory as [state][range][L + pad] fp32: a thread reads its tokens as 16-byte
// vectors, the lanes of one range the same address. The state stride is 4 floats
// off a multiple of the banks, for the writes of several states of one token.
template <int CB, int L, int WARPS>
struct Tile {
    static constexpr int kNB = CB <= 8 ? 8 : 16;            // states staged at once
    static constexpr int kSub = 32 / CB;                    // ranges per warp
    static constexpr int kRanges = WARPS * kSub;            // ranges per chunk
    static constexpr int kTok = kRanges * L;                // tokens per chunk
    static constexpr int kRow = L + kLdPad;                 // floats per range
    static constexpr int kState = kRanges * kRow + 4;       // floats per state
    static __device__ __forceinline__ int at(int n, int t) { return n * kState + (t / L) * kRow + t % L; }
};

// The unit of a CTA: sequence and channel tile; tiles do not straddle groups.
struct Unit {
    int n, tile, group, c0, live;     // c0: the tile's first channel; live: its channels
};
template <int CB>
__device__ __forceinline__ Unit unit_of(const SsmArgs &g) {
    const int per = g.D / g.G, tiles = (per + CB - 1) / CB;
    Unit u;
    u.n = blockIdx.x / (tiles * g.G);
    u.tile = blockIdx.x % (tiles * g.G);
    u.group = u.tile / tiles;
    const int i = u.tile % tiles * CB;
    u.c0 = u.group * per + i;
    u.live = min(CB, per - i);
    return u;
}

// Shared memory of the forward kernel: per warp two stages of a tile's rows (x, dt,
// z) and of a block of B and C, that block as fp32 [state][token + pad], and the
// words through which the tile before hands over its states; per CTA A * log2(e).
template <int CB, typename T>
struct FwdSmem {
    static constexpr int L = kFwdL, NB = kFwdNB, NS = 32 / CB;
    static constexpr int kRow = L + kLdPad;
    static constexpr size_t rows = 3 * (size_t)L * CB * sizeof(T);
    static constexpr size_t raw = 2 * (size_t)L * NB * sizeof(T);
    static constexpr int kC = NB * kRow + 16;       // C behind B, 16 banks on: both are written at once
    static constexpr size_t wide = (kC + (size_t)NB * kRow) * sizeof(float);
    static constexpr size_t words = 2 * (rows + raw) + wide;     // where the words start
    // states in shared memory: whole rounds of two states per lane; a state behind the
    // last has A = B = C = 0 and stays 0
    static __host__ __device__ int padded(int N) { return (N + 2 * NS - 1) / (2 * NS) * (2 * NS); }
    static __host__ __device__ size_t warp(int N) { return words + (size_t)padded(N) * CB * 8; }
    static size_t bytes(int N, int warps) { return warps * warp(N) + (size_t)padded(N) * CB * sizeof(float); }
};

constexpr int kSmemLimit = 227 * 1024;
constexpr unsigned kSpinLimit = 1u << 24;     // polls of a word before a warp gives up (about a second)

// OUT: writes out (else only states: the walk before a backward pass without
// recorded states). blockDim is (32, warps).
template <int CB, bool OUT, typename T>
__global__ void __launch_bounds__(512) ssm_forward_kernel(const SsmArgs g) {
    using M = FwdSmem<CB, T>;
    constexpr int L = M::L, NB = M::NB, NS = M::NS, LS = L / NS;   // LS: tokens of a lane outside the state loop
    constexpr int kEvery = kSsmCkpt / L;                            // tiles between recorded states
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x, warp = threadIdx.y, warps = blockDim.y, lc = lane % CB, ls = lane / CB;
    unsigned char *mine = smem + warp * M::warp(g.N);
    auto rows_at = [&](int half) { return reinterpret_cast<T *>(mine + half * M::rows); };                 // [3][L][CB]
    auto raw_at = [&](int half) { return reinterpret_cast<T *>(mine + 2 * M::rows + half * M::raw); };      // [2][L][NB]
    float *sB = reinterpret_cast<float *>(mine + 2 * (M::rows + M::raw)), *sC = sB + M::kC;                // [NB][kRow]
    auto words_of = [&](int w) {                                                                            // [N][CB]
        return reinterpret_cast<volatile unsigned long long *>(smem + w * M::warp(g.N) + M::words);
    };
    float *sA = reinterpret_cast<float *>(smem + warps * M::warp(g.N));
    const Unit u = unit_of<CB>(g);
    long long s0, s1;
    g.ax.range(u.n, s0, s1);
    const bool live = lc < u.live;
    const int c = u.c0 + (live ? lc : 0);
    const T *x = static_cast<const T *>(g.x) + s0 * g.ld_x + u.c0;
    const T *dt = static_cast<const T *>(g.dt) + s0 * g.ld_dt + u.c0;
    const T *z = g.z ? static_cast<const T *>(g.z) + s0 * g.ld_z + u.c0 : nullptr;
    const T *Bm = static_cast<const T *>(g.Bm) + s0 * g.ld_b + (long long)u.group * g.N;
    const T *Cm = static_cast<const T *>(g.Cm) + s0 * g.ld_c + (long long)u.group * g.N;
    const float bias = g.dt_bias ? g.dt_bias[c] : 0.f, skip = g.Dskip ? g.Dskip[c] : 0.f;
    const int len = (int)(s1 - s0), tiles = (int)(((long long)len + L - 1) / L);

    // copies of one step: a block of B and C, with a tile's first block its rows
    auto fetch = [&](int tile, int n0, int rh, int half) {
        const int have = min(L, len - tile * L), states = min(NB, g.N - n0);
        T *r = rows_at(rh), *b = raw_at(half);
        if (n0 == 0) {
            copy_rows<L, CB, 32>(r, x + (long long)tile * L * g.ld_x, g.ld_x, have, u.live, g.mode_x, lane);
            copy_rows<L, CB, 32>(r + L * CB, dt + (long long)tile * L * g.ld_dt, g.ld_dt, have, u.live, g.mode_x, lane);
            if (OUT && z)
                copy_rows<L, CB, 32>(r + 2 * L * CB, z + (long long)tile * L * g.ld_z, g.ld_z, have, u.live, g.mode_x, lane);
        }
        copy_rows<L, NB, 32>(b, Bm + (long long)tile * L * g.ld_b + n0, g.ld_b, have, states, g.mode_b, lane);
        if (OUT)
            copy_rows<L, NB, 32>(b + L * NB, Cm + (long long)tile * L * g.ld_c + n0, g.ld_c, have, states, g.mode_b, lane);
    };
    // The staged block of B (half the warp) and C (the other half) as fp32; zero behind
    // the sequence's end and the last state.
    auto widen = [&](const T *raw, int have, int states) {
        constexpr int V = 16 / (int)sizeof(T), PR = NB / V;
        const int t = lane % L, which = lane / L;
        float *dst = (which ? sC : sB) + t;
        const T *src = raw + which * L * NB + t * NB;
        float v[PR][V];
#pragma unroll
        for (int k = 0; k < PR; ++k) load_v<V>(src + k * V, v[k]);
        if (have < L || states < NB) {
#pragma unroll
            for (int k = 0; k < PR; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (t >= have || k * V + i >= states) v[k][i] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < PR; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) dst[(k * V + i) * M::kRow] = v[k][i];
    };

    if (warp < tiles) fetch(warp, 0, 0, 0);
    cp_async_commit();
    const int padded = M::padded(g.N);
    for (int e = warp * 32 + lane; e < padded * CB; e += warps * 32) {
        const int n = e % padded, j = e / padded;
        float a = 0.f, h = 0.f;
        if (j < u.live && n < g.N) {
            const long long at = ((long long)u.n * g.D + u.c0 + j) * g.N + n;
            a = g.A[(long long)(u.c0 + j) * g.N + n] * kLog2e;
            if (g.state0) h = g.state0[at];
            if (tiles == 0 && g.final_state) g.final_state[at] = h;
            if (tiles && g.states) g.states[(ssm_ckpt_base(s0, u.n) * g.N + n) * g.D + u.c0 + j] = h;
        }
        sA[n * CB + j] = a;
        // tile 0's words are the initial state; the others' carry no tile's number yet
        for (int w = 0; w < warps; ++w)
            words_of(w)[n * CB + j] = w ? 0xffffffff00000000ull : (unsigned long long)__float_as_uint(h);
    }
    __syncthreads();
    int rh = 0, half = 0;      // the stages of rows and of B and C in use
    for (int tile = warp; tile < tiles; tile += warps, rh ^= 1) {
        const int have = min(L, len - tile * L);
        const T *rx = rows_at(rh) + lc;
        f32x2 del[L / 2], dx[L / 2], y[L / 2];
        // where the state behind this tile is recorded: the last, or one for the backward pass
        float *rec = nullptr;
        int rec_ld = 1;
        if (tile == tiles - 1) {
            if (g.final_state) rec = g.final_state + ((long long)u.n * g.D + c) * g.N;
        } else if (g.states && tile % kEvery == kEvery - 1) {
            rec = g.states + (ssm_ckpt_base(s0, u.n) + tile / kEvery + 1) * g.N * g.D + c;
            rec_ld = g.D;
        }
        if (!live) rec = nullptr;
        for (int n0 = 0; n0 < g.N; n0 += NB, half ^= 1) {
            const int states = min(NB, g.N - n0);
            cp_async_wait();
            __syncwarp();
            widen(raw_at(half), have, states);
            if (n0 + NB < g.N) fetch(tile, n0 + NB, rh, half ^ 1);
            else if (tile + warps < tiles) fetch(tile + warps, 0, rh ^ 1, half ^ 1);
            cp_async_commit();
            if (n0 == 0) {
                // a lane's share of the tile's tokens
                float d[LS], w[LS];
#pragma unroll
                for (int i = 0; i < LS; ++i) {
                    d[i] = to_f(rx[(L + ls * LS + i) * CB]) + bias;
                    w[i] = to_f(rx[(ls * LS + i) * CB]);
                }
                if (g.softplus) {
#pragma unroll
                    for (int i = 0; i < LS; i += 2) softplus2(d[i], d[i + 1]);
                }
#pragma unroll
                for (int i = 0; i < LS; ++i) w[i] *= d[i];
                if (have < L || u.live < CB) {
                    // behind the end, and channels of no one: step 0, so decay 1 and input 0
#pragma unroll
                    for (int i = 0; i < LS; ++i)
                        if (!live || ls * LS + i >= have) d[i] = w[i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < L; i += 2) {
                    float p0 = d[i % LS], p1 = d[(i + 1) % LS], q0 = w[i % LS], q1 = w[(i + 1) % LS];
                    if constexpr (NS > 1) {
                        const int src = i / LS * CB + lc;
                        p0 = __shfl_sync(0xffffffffu, p0, src);
                        p1 = __shfl_sync(0xffffffffu, p1, src);
                        q0 = __shfl_sync(0xffffffffu, q0, src);
                        q1 = __shfl_sync(0xffffffffu, q1, src);
                    }
                    del[i / 2] = pack2(p0, p1);
                    dx[i / 2] = pack2(q0, q1);
                    y[i / 2] = 0;
                }
            }
            __syncwarp();
            // two states per round: two independent walks in flight
            const int at = (n0 + ls) * CB + lc;
            volatile unsigned long long *win = words_of(warp) + at, *wout = words_of(warp + 1 < warps ? warp + 1 : 0) + at;
            const float *pa = sA + at;
            const ulonglong2 *b4 = reinterpret_cast<const ulonglong2 *>(sB + ls * M::kRow);
            const ulonglong2 *c4 = reinterpret_cast<const ulonglong2 *>(sC + ls * M::kRow);
            constexpr int kB = NS * M::kRow / 4;      // vectors from one of the two states to the other
#pragma unroll 1
            for (int n = ls; n < states + ls; n += 2 * NS) {
                unsigned long long in0 = win[0], in1 = win[NS * CB];
                const f32x2 A0 = dup2(pa[0]), A1 = dup2(pa[NS * CB]);
                f32x2 a0[L / 2], a1[L / 2];
#pragma unroll
                for (int i = 0; i < L / 2; ++i) {
                    float e0, e1, f0, f1;
                    unpack2(mul2(del[i], A0), e0, e1);
                    unpack2(mul2(del[i], A1), f0, f1);
                    a0[i] = pack2(ex2(e0), ex2(e1));
                    a1[i] = pack2(ex2(f0), ex2(f1));
                }
                // the states before the tile, once the warp that has the tile before has left them
                for (unsigned spin = 0; !__all_sync(0xffffffffu, (unsigned)(in0 >> 32) == (unsigned)tile &&
                                                                     (unsigned)(in1 >> 32) == (unsigned)tile);) {
                    in0 = win[0];
                    in1 = win[NS * CB];
                    if (++spin > kSpinLimit) {
                        if (lane == 0) atomicOr(g.status, kStatusTimeout);
                        cp_async_wait();
                        return;
                    }
                }
                float h0 = __uint_as_float((unsigned)in0), h1 = __uint_as_float((unsigned)in1);
#pragma unroll
                for (int q = 0; q < L / 4; ++q) {
                    const ulonglong2 bv0 = b4[q], bv1 = b4[kB + q];
                    ulonglong2 cv0, cv1;
                    if (OUT) cv0 = c4[q], cv1 = c4[kB + q];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int i = 2 * q + k;
                        float e0, e1, f0, f1, u0, u1, v0, v1;
                        unpack2(mul2(dx[i], k ? bv0.y : bv0.x), u0, u1);
                        unpack2(mul2(dx[i], k ? bv1.y : bv1.x), v0, v1);
                        unpack2(a0[i], e0, e1);
                        unpack2(a1[i], f0, f1);
                        u0 = fmaf(e0, h0, u0);
                        v0 = fmaf(f0, h1, v0);
                        u1 = h0 = fmaf(e1, u0, u1);
                        v1 = h1 = fmaf(f1, v0, v1);
                        if (OUT) {
                            y[i] = fma2(k ? cv0.y : cv0.x, pack2(u0, u1), y[i]);
                            y[i] = fma2(k ? cv1.y : cv1.x, pack2(v0, v1), y[i]);
                        }
                    }
                }
                const unsigned long long tag = (unsigned long long)(unsigned)(tile + 1) << 32;
                wout[0] = tag | __float_as_uint(h0);
                wout[NS * CB] = tag | __float_as_uint(h1);
                win += 2 * NS * CB;
                wout += 2 * NS * CB;
                pa += 2 * NS * CB;
                b4 += 2 * kB;
                c4 += 2 * kB;
            }
            if (rec) {
                // what this lane has just handed over
                wout = words_of(warp + 1 < warps ? warp + 1 : 0) + at;
                for (int n = ls; n < states; n += NS, wout += NS * CB)
                    rec[(long long)(n0 + n) * rec_ld] = __uint_as_float((unsigned)*wout);
            }
            __syncwarp();
        }
        if (OUT) {
            // what the rows still hold, before anything is stored
            float xs[LS], zs[LS];
#pragma unroll
            for (int i = 0; i < LS; ++i) {
                xs[i] = to_f(rx[(ls * LS + i) * CB]);
                zs[i] = z ? to_f(rx[(2 * L + ls * LS + i) * CB]) : 0.f;
            }
            float v[L];
#pragma unroll
            for (int i = 0; i < L / 2; ++i) unpack2(y[i], v[2 * i], v[2 * i + 1]);
            // the states' lanes add up, each keeping its share of the tokens
            int count = L;
#pragma unroll
            for (int o = 16; o >= CB; o >>= 1) {
                count >>= 1;
                const bool up = lane & o;
#pragma unroll
                for (int j = 0; j < L / 2; ++j) {
                    if (j < count) {
                        const float send = up ? v[j] : v[j + count];
                        const float keep = up ? v[j + count] : v[j];
                        v[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < LS; ++i) {
                v[i] = fmaf(skip, xs[i], v[i]);
                if (z) v[i] *= zs[i] * sigmoid_a(zs[i]);
            }
            T *out = static_cast<T *>(g.out) + (s0 + tile * L + ls * LS) * g.D + c;
            const int mine_n = live ? have - ls * LS : 0;
#pragma unroll
            for (int i = 0; i < LS; ++i)
                if (i < mine_n) out[(long long)i * g.D] = from_f<T>(v[i]);
            __syncwarp();
        }
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

constexpr int kBwdThreads = kBwdWarps * 32;

// States [n0, n0 + S::kNB) of the chunk's rows of B or C into shared memory as fp32.
template <int CB, int L, typename T>
__device__ __forceinline__ void stage(float *dst, const T *src, long long ld, long long t0, long long t1, int n0,
                                      int N) {
    using S = Tile<CB, L, kBwdWarps>;
    for (int e = threadIdx.x; e < S::kTok * S::kNB; e += kBwdThreads) {
        const int n = e % S::kNB, t = e / S::kNB;
        float v = 0.f;
        if (n0 + n < N && t0 + t < t1) v = to_f(src[(t0 + t) * ld + n0 + n]);
        dst[S::at(n, t)] = v;
    }
}

template <int CB>
struct BwdSmem {
    static __host__ __device__ size_t bytes(int N) {
        using S = Tile<CB, kBwdL, kBwdWarps>;
        // B, C; the adjoint's carry (two halves); exchange; dA and the two channel sums per warp
        return sizeof(float) * (2 * (size_t)S::kNB * S::kState + 2 * (size_t)N * CB + 2 * 4 * kBwdWarps * CB +
                                (size_t)kBwdWarps * (N + 2) * CB);
    }
};

// Chunks from the last to the first. Per state: decays, the forward walk from the
// recorded state before the chunk, the adjoint walk dh_t = C_t g_t + a_{t+1} dh_{t+1}
// (g: the gradient at y) whose incoming value joins from the right, and the sums
// over channels of dh delta x (dB) and g h (dC), which leave as the tile's partial
// sums: a second kernel adds the tiles in a fixed order.
template <int CB, typename T>
__global__ void __launch_bounds__(kBwdThreads, 2) ssm_backward_kernel(const SsmArgs g) {
    constexpr int L = kBwdL;
    using S = Tile<CB, L, kBwdWarps>;
    static_assert(S::kTok % kSsmCkpt == 0, "chunks start at recorded states");
    extern __shared__ __align__(16) float sm[];
    float *sB = sm, *sC = sB + S::kNB * S::kState;
    float4 *exch = reinterpret_cast<float4 *>(sC + S::kNB * S::kState);    // [2][warps][CB]
    float *carry = reinterpret_cast<float *>(exch + 2 * kBwdWarps * CB);    // [2][N][CB]
    float *sA = carry + 2 * g.N * CB;                                       // [warps][N + 2][CB]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lc = lane % CB, sub = lane / CB;
    const int range = warp * S::kSub + sub;
    const Unit u = unit_of<CB>(g);
    long long s0, s1;
    g.ax.range(u.n, s0, s1);
    const bool live = lc < u.live;
    const int c = u.c0 + (live ? lc : 0);
    const T *x = static_cast<const T *>(g.x) + c, *dt = static_cast<const T *>(g.dt) + c;
    const T *z = g.z ? static_cast<const T *>(g.z) + c : nullptr;
    const T *dout = static_cast<const T *>(g.dout) + c;
    const T *Bm = static_cast<const T *>(g.Bm) + (long long)u.group * g.N;
    const T *Cm = static_cast<const T *>(g.Cm) + (long long)u.group * g.N;
    const float bias = g.dt_bias ? g.dt_bias[c] : 0.f, skip = g.Dskip ? g.Dskip[c] : 0.f;
    const float *A = g.A + (long long)c * g.N;
    float *part = g.part_bc + (long long)u.tile * 2 * g.N * g.ax.ntok;
    for (int e = threadIdx.x; e < g.N * CB; e += kBwdThreads) {
        const int n = e % g.N, j = e / g.N;
        const int ch = j < u.live ? u.c0 + j : -1;
        carry[n * CB + j] = (g.dfinal && ch >= 0) ? g.dfinal[((long long)u.n * g.D + ch) * g.N + n] : 0.f;
    }
    for (int e = threadIdx.x; e < kBwdWarps * (g.N + 2) * CB; e += kBwdThreads) sA[e] = 0.f;
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
                float r = to_f(dt[(tk + i) * g.ld_dt]) + bias, unused = 0.f;
                if (g.softplus) softplus2(r, unused);
                del[i] = r;
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
                float4 *ex = exch + (xp * kBwdWarps + warp) * CB + lc;
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
                    const float4 e = exch[(xp * kBwdWarps + w) * CB + lc];
                    h = fmaf(e.x, h, e.y);
                }
                for (int w = kBwdWarps - 1; w > warp; --w) {
                    const float4 e = exch[(xp * kBwdWarps + w) * CB + lc];
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
    for (int e = threadIdx.x; e < (g.N + 2) * CB; e += kBwdThreads) {
        const int n = e % (g.N + 2), j = e / (g.N + 2);
        const int ch = j < u.live ? u.c0 + j : -1;
        if (ch < 0) continue;
        float s = 0.f;
        for (int w = 0; w < kBwdWarps; ++w) s += sA[(w * (g.N + 2) + n) * CB + j];
        if (n < g.N) par_out[(long long)ch * g.N + n] = s;
        else par_out[(long long)g.D * n + ch] = s;
    }
    if (g.dstate0)
        for (int e = threadIdx.x; e < g.N * CB; e += kBwdThreads) {
            const int n = e % g.N, j = e / g.N;
            const int ch = j < u.live ? u.c0 + j : -1;
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

// The widest way rows [.][width] at stride ld of several tensors can be copied in
// pieces: 16 bytes (or `row` bytes, a narrower tile row), 4 bytes, or elements.
struct Rows {
    const void *p;
    long long ld;
};
int copy_mode(std::initializer_list<Rows> ts, long long width, size_t es, size_t row) {
    bool near = true;
    for (const Rows &t : ts) near = near && t.ld * (long long)es < (1 << 24);
    auto fits = [&](size_t a) {
        if (width * es % a) return false;
        for (const Rows &t : ts)
            if (t.p && (((uintptr_t)t.p | (size_t)t.ld * es) & (a - 1))) return false;
        return true;
    };
    return near && fits(row < 16 ? row : 16) ? kWide : fits(4) ? kWord : kScalar;
}

template <int CB, bool OUT, typename T>
cudaError_t forward_cb(SsmArgs g, long long units, int warps, cudaStream_t st) {
    static PerDevice<bool> attr;
    using M = FwdSmem<CB, T>;
    auto kern = ssm_forward_kernel<CB, OUT, T>;
    cudaError_t e = ensure_smem_attr(attr, kern, kSmemLimit);
    if (e != cudaSuccess) return e;
    while (warps > 1 && M::bytes(g.N, warps) > (size_t)kSmemLimit) --warps;
    g.mode_x = copy_mode({{g.x, g.ld_x}, {g.dt, g.ld_dt}, {g.z, g.ld_z}}, g.D / g.G, sizeof(T), CB * sizeof(T));
    g.mode_b = copy_mode({{g.Bm, g.ld_b}, {g.Cm, g.ld_c}}, g.N, sizeof(T), 16);
    kern<<<(unsigned)units, dim3(32, warps), M::bytes(g.N, warps), st>>>(g);
    return cudaGetLastError();
}

template <bool OUT, typename T>
cudaError_t forward_t(const SsmArgs &g, int sms, cudaStream_t st) {
    const int per = g.D / g.G;
    auto units = [&](int cb) { return (long long)g.ax.nseq * g.G * ((per + cb - 1) / cb); };
    if (units(8) > 0x7fffffffLL) return cudaErrorInvalidValue;
    // 16 channels per CTA, or 8 where that leaves a quarter of the SMs without one (fewer
    // channels split the same rows into more CTAs, and share what every tile costs less:
    // 8192 channels of 2048 tokens 177 us against 215, 520 channels in 12 groups 75 against
    // 49). As many warps as fill the SMs' 16: one sequence of 131072 tokens and 2048
    // channels takes 6.1, 3.6 and 2.8 ms with 4, 8 and 16 of them, 8 rows of 4096 tokens
    // 600, 586 and 671 us.
    const bool wide = 4 * units(16) >= 3LL * sms;
    const long long n = wide ? units(16) : units(8);
    int warps = n <= (wide ? sms : 2 * sms) ? 16 : 8;
    const long long most = ((g.ax.cu ? g.ax.ntok : g.ax.T) + kFwdL - 1) / kFwdL;
    while (warps > 1 && warps / 2 >= most) warps /= 2;
    return wide ? forward_cb<16, OUT, T>(g, n, warps, st) : forward_cb<8, OUT, T>(g, n, warps, st);
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
    kern<<<(unsigned)units, kBwdThreads, BwdSmem<kBwdCB>::bytes(g.N), st>>>(g);
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
