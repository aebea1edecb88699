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
// states of its tile, two per lane at a time, and for each needs the state at the
// tile's start from the warp that has the tile before: it comes through shared memory,
// one 64-bit word per channel and state that carries the tile's number beside the
// value, so no barrier is needed. Warps follow one another at a distance of a round,
// all of them busy, each decay computed and used once, and nothing walked twice. (The
// other way to split time, a range per thread whose end state from zero and decay
// product are joined by barriers before the range is walked again, took 800 us for the
// layer below and 3.3 to 5 ms for the long row.) A word is written again only after its
// reader has taken it: the warp that writes it next needs, state by state, what that
// reader hands on. A tile's steps, inputs and outputs stay in registers, as pairs of
// tokens for the packed fp32 instructions; its rows arrive by asynchronous copies while
// the tile before is worked on.
// Measured, bf16, 2048 channels, 16 states: 8 rows of 4096 tokens 550 us, one row of
// 131072 tokens 2.45 ms, 4 rows of 2048 with recorded states 174 us (259 in fp32). The exponentials
// alone are 240 us, 0.96 ms and 60 us; the exponential unit is 48 % busy, the issue
// slots 53 %: with 16 warps per SM (128 registers a thread) the dependent steps of a
// tile and the 650 instructions per tile outside its state loop (of 1480) are not
// hidden entirely.
//
// Backward: the same tiles from the last to the first, the adjoint a_{t+1} dh_{t+1}
// handed from warp to warp. The forward call records the state before every tile, so a
// warp walks its tile's states forward and then the adjoint backward with one set of
// decays. dB and dC are sums over channels: a transposing reduction over the warp's
// channels leaves each lane one token's sum, and a second kernel adds the channel tiles
// in a fixed order. Measured: 4 rows of 2048 tokens, 2048 channels, 16 states, 550 us
// (fp32 586) and 25 us for the channel tiles' sums. Eight warps per SM (255 registers) issue in
// 46 % of the slots, a quarter of the instructions are the two reductions. (Those as
// tensor-core products with ones, when this took 574 us: 531, but their tf32 operands cut
// the terms to 11 bits. Tiles of 8 tokens, which fit twice the warps: 600 us and twice the
// states.)
#include <initializer_list>

#include "kla_block.cuh"

namespace kla {

namespace {

constexpr int kTileL = 16;       // tokens of a tile
constexpr int kTileNB = 16;      // states whose B and C a warp stages at once
constexpr int kLdPad = 4;        // floats behind a state's tokens in shared memory: states on other banks

// How rows reach shared memory: pieces of 16 bytes (or a whole narrower row), of 4
// bytes, or single elements, by the alignment of the rows. Elements of bf16 have no
// asynchronous copy, so a tile waits for its rows. 4 rows of 2048 tokens, 16 states, bf16,
// forward and backward: 174 and 551 us with 2048 channels, 231 and 651 with 2046 (4 bytes),
// 334 and 895 with 2047 (elements); 8 rows of 4096 tokens forward 550 and 1250 us with 2048
// and 2047. An odd number of states does the same to B and C (17 states 381 us, 18 states
// 319). fp32 rows off 16 bytes: 2047 channels 390 and 719 us, 2048 259 and 586.
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

// A staged block of B (half the warp) and C (the other half) as fp32 [state][kRow];
// zero behind the sequence's end and the last state.
template <int NB, int ROW, typename T>
__device__ __forceinline__ void widen(float *sB, float *sC, const T *raw, int have, int states, int lane) {
    constexpr int L = kTileL, V = 16 / (int)sizeof(T), PR = NB / V;
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
        for (int i = 0; i < V; ++i) dst[(k * V + i) * ROW] = v[k][i];
}

// Adds up v over the lanes that differ in the bits FROM .. TO (powers of two, falling),
// halving the values at each: a lane ends with COUNT >> bits of them, chosen by its
// bits, the highest bit the upper half.
template <int FROM, int TO, int COUNT, int M>
__device__ __forceinline__ void reduce_halving(float (&v)[M], int lane) {
    int count = COUNT;
#pragma unroll
    for (int o = FROM; o >= TO; o >>= 1) {
        count >>= 1;
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < COUNT / 2; ++j) {
            if (j < count) {
                const float send = up ? v[j] : v[j + count];
                const float keep = up ? v[j + count] : v[j];
                v[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        }
    }
}

// The approximated power of two is low on average: by 2e-8 for exponents from -1 to -0.01
// and 5e-8 below -1 (1e-8 next to 0). A state that remembers thousands of tokens would add
// that up (a relative 2e-5 after a thousand), and an input's share in the state passes up
// to 16 of them in its own tile. So every exponent is raised by 2.5e-8, which costs nothing
// (a fused multiply-add in place of a product) and leaves a mean between -5e-9 and +1e-8
// for exponents from -1 on, those that are remembered; 2^0 stays exactly 1, which
// steps of zero need. And what a tile hands on decays by the power of two of the tile's
// whole exponent: the product of its 16 decays, which the walk applied, is taken out and
// that one put in, (2^(A sum delta) - prod a) h_start on top of the walk's end: one rounding
// in 16 tokens instead of 16, for 12 instructions of a state's 100. The states after 9001
// packed tokens are within 5.0e-7 of the 64-bit recurrence (7.0e-7 without the raised
// exponents, 3.4e-6 without either), the gradient of A of 1403 tokens of 64 states within
// 2.8e-7 (5.7e-7); 8 rows of 4096 tokens take 550 us, 520 without the tile's exponent.
constexpr float kEx2Low = 2.5e-8f;
__device__ __forceinline__ float product_of(const f32x2 (&a)[kTileL / 2]) {
    const f32x2 p = mul2(mul2(mul2(a[0], a[1]), mul2(a[2], a[3])), mul2(mul2(a[4], a[5]), mul2(a[6], a[7])));
    float lo, hi;
    unpack2(p, lo, hi);
    return lo * hi;
}
__device__ __forceinline__ float sum_of(const f32x2 (&d)[kTileL / 2]) {
    const f32x2 s = add2(add2(add2(d[0], d[1]), add2(d[2], d[3])), add2(add2(d[4], d[5]), add2(d[6], d[7])));
    float lo, hi;
    unpack2(s, lo, hi);
    return lo + hi;
}

// Shared memory of the forward kernel: per warp two stages of a tile's rows (x, dt,
// z) and of a block of B and C, that block as fp32 [state][token + pad], and the
// words through which the tile before hands over its states; per CTA A * log2(e).
template <int CB, typename T>
struct FwdSmem {
    static constexpr int L = kTileL, NB = kTileNB, NS = 32 / CB;
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

constexpr int kRestBlocks = 64;      // CTAs that clear the rows of no sequence

// Polls of a word before a warp gives up, about a second. (Read from the arguments, so that
// a test could shorten it, it cost one row of 131072 tokens 14 %: other registers.)
constexpr unsigned kSpinLimit = 1u << 24;

// OUT: writes out (else only states: the walk before a backward pass without
// recorded states). WIDE: all rows are copied in the widest pieces. blockDim is (32, warps).
// CTAs behind the units clear the rows of no sequence.
template <int CB, bool OUT, bool WIDE, typename T>
__global__ void __launch_bounds__(512) ssm_forward_kernel(const SsmArgs g, unsigned units) {
    using M = FwdSmem<CB, T>;
    constexpr int L = M::L, NB = M::NB, NS = M::NS, LS = L / NS;   // LS: tokens of a lane outside the state loop
    static_assert(L == kSsmCkpt, "every tile's start is recorded");
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x, warp = threadIdx.y, warps = blockDim.y, lc = lane % CB, ls = lane / CB;
    if (OUT && blockIdx.x >= units) {
        T *out = static_cast<T *>(g.out);
        const long long step = (long long)(gridDim.x - units) * warps * 32;
        const long long from = ((long long)(blockIdx.x - units) * warps + warp) * 32 + lane, D = g.D;
        const long long head = min((long long)g.ax.cu[0], g.ax.ntok), tail = max(g.ax.cu[g.ax.nseq], 0);
        if (head > 0) clear(out, head * D, from, step);
        if (tail < g.ax.ntok) clear(out + tail * D, (g.ax.ntok - tail) * D, from, step);
        return;
    }
    unsigned char *mine = smem + warp * M::warp(g.N);
    auto rows_at = [&](int half) { return reinterpret_cast<T *>(mine + half * M::rows); };  // [3][L][CB]
    auto raw_at = [&](int half) { return reinterpret_cast<T *>(mine + 2 * M::rows + half * M::raw); };      // [2][L][NB]
    float *sB = reinterpret_cast<float *>(mine + 2 * (M::rows + M::raw)), *sC = sB + M::kC;  // [NB][kRow]
    auto words_of = [&](int w) {  // [N][CB]
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

    const int mode_x = WIDE ? kWide : g.mode_x, mode_b = WIDE ? kWide : g.mode_b;
    // copies of one step: a block of B and C, with a tile's first block its rows
    auto fetch = [&](int tile, int n0, int rh, int half) {
        const int have = min(L, len - tile * L), states = min(NB, g.N - n0);
        const long long t = (long long)tile * L;
        T *r = rows_at(rh), *b = raw_at(half);
        if (n0 == 0) {
            copy_rows<L, CB, 32>(r, x + t * g.ld_x, g.ld_x, have, u.live, mode_x, lane);
            copy_rows<L, CB, 32>(r + L * CB, dt + t * g.ld_dt, g.ld_dt, have, u.live, mode_x, lane);
            if (OUT && z) copy_rows<L, CB, 32>(r + 2 * L * CB, z + t * g.ld_z, g.ld_z, have, u.live, mode_x, lane);
        }
        copy_rows<L, NB, 32>(b, Bm + t * g.ld_b + n0, g.ld_b, have, states, mode_b, lane);
        if (OUT) copy_rows<L, NB, 32>(b + L * NB, Cm + t * g.ld_c + n0, g.ld_c, have, states, mode_b, lane);
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
            words_of(w)[n * CB + j] = w ? 0xffffffff00000000ull : g.first_tag | __float_as_uint(h);
    }
    __syncthreads();
    int rh = 0, half = 0;      // the stages of rows and of B and C in use
    for (int tile = warp; tile < tiles; tile += warps, rh ^= 1) {
        const int have = min(L, len - tile * L);
        const T *rx = rows_at(rh) + lc;
        f32x2 del[L / 2], dx[L / 2], y[L / 2];
        float sum = 0.f;           // of the tile's steps
        // where the state behind this tile is recorded: the last one, or the next tile's start
        float *rec = nullptr;
        int rec_ld = 1;
        if (tile == tiles - 1) {
            if (g.final_state) rec = g.final_state + ((long long)u.n * g.D + c) * g.N;
        } else if (g.states) {
            rec = g.states + (ssm_ckpt_base(s0, u.n) + tile + 1) * g.N * g.D + c;
            rec_ld = g.D;
        }
        if (!live) rec = nullptr;
        for (int n0 = 0; n0 < g.N; n0 += NB, half ^= 1) {
            const int states = min(NB, g.N - n0);
            cp_async_wait();
            __syncwarp();
            widen<NB, M::kRow>(sB, sC, raw_at(half), have, states, lane);
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
                    for (int i = 0; i < LS; i += 2) softplus2<T>(d[i], d[i + 1]);
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
                sum = sum_of(del);
            }
            __syncwarp();
            // two states per round: two independent walks in flight
            const int at = (n0 + ls) * CB + lc;
            volatile unsigned long long *win = words_of(warp) + at;
            volatile unsigned long long *wout = words_of(warp + 1 < warps ? warp + 1 : 0) + at;
            const float *pa = sA + at;
            const ulonglong2 *b4 = reinterpret_cast<const ulonglong2 *>(sB + ls * M::kRow);
            const ulonglong2 *c4 = reinterpret_cast<const ulonglong2 *>(sC + ls * M::kRow);
            constexpr int kB = NS * M::kRow / 4;      // vectors from one of the two states to the other
#pragma unroll 4
            for (int n = ls; n < states + ls; n += 2 * NS) {
                unsigned long long in0 = win[0], in1 = win[NS * CB];
                const float A2_0 = pa[0], A2_1 = pa[NS * CB];
                const f32x2 A0 = dup2(A2_0), A1 = dup2(A2_1);
                f32x2 a0[L / 2], a1[L / 2];
#pragma unroll
                for (int i = 0; i < L / 2; ++i) {
                    float e0, e1, f0, f1;
                    unpack2(fma2(del[i], A0, dup2(kEx2Low)), e0, e1);
                    unpack2(fma2(del[i], A1, dup2(kEx2Low)), f0, f1);
                    a0[i] = pack2(ex2(e0), ex2(e1));
                    a1[i] = pack2(ex2(f0), ex2(f1));
                }
                const float fix0 = ex2(fmaf(sum, A2_0, kEx2Low)) - product_of(a0);
                const float fix1 = ex2(fmaf(sum, A2_1, kEx2Low)) - product_of(a1);
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
                const float first0 = __uint_as_float((unsigned)in0), first1 = __uint_as_float((unsigned)in1);
                float h0 = first0, h1 = first1;
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
                h0 = fmaf(fix0, first0, h0);
                h1 = fmaf(fix1, first1, h1);
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
            reduce_halving<16, CB, L>(v, lane);
#pragma unroll
            for (int i = 0; i < LS; ++i) {
                v[i] = fmaf(skip, xs[i], v[i]);
                if (z) v[i] *= zs[i] * sigmoid_for<T>(zs[i]);
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

// Shared memory of the backward kernel: per warp two stages of a tile's rows (x, dt,
// dout, z), of a block of B and C and of that block's start states, B and C as fp32,
// the words of the adjoint, and the sums of dA, dDskip and ddt_bias; per CTA A.
template <int CB, typename T>
struct BwdSmem {
    static constexpr int L = kTileL, NB = kTileNB, NS = 32 / CB;
    static constexpr int kRow = L + kLdPad, kC = NB * kRow + 16;
    static constexpr size_t rows = 4 * (size_t)L * CB * sizeof(T);
    static constexpr size_t raw = 2 * (size_t)L * NB * sizeof(T);
    static constexpr size_t start = (size_t)NB * CB * sizeof(float);
    static constexpr size_t wide = (kC + (size_t)NB * kRow) * sizeof(float);
    static constexpr size_t words = 2 * (rows + raw + start) + wide;
    static __host__ __device__ int padded(int N) { return (N + NS - 1) / NS * NS; }
    static __host__ __device__ size_t sums(int N) { return words + (size_t)padded(N) * CB * 8; }
    static __host__ __device__ size_t warp(int N) { return sums(N) + (size_t)(padded(N) + 2) * CB * 4; }
    static size_t bytes(int N, int warps) { return warps * warp(N) + (size_t)padded(N) * CB * sizeof(float); }
};

// GATE: z was given. blockDim is (32, warps); a warp's p-th tile from the end.
template <int CB, bool GATE, bool WIDE, typename T>
__global__ void __launch_bounds__(256) ssm_backward_kernel(const SsmArgs g) {
    using M = BwdSmem<CB, T>;
    constexpr int L = M::L, NB = M::NB, NS = M::NS, LS = L / NS;
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x, warp = threadIdx.y, warps = blockDim.y, lc = lane % CB, ls = lane / CB;
    unsigned char *mine = smem + warp * M::warp(g.N);
    auto rows_at = [&](int half) { return reinterpret_cast<T *>(mine + half * M::rows); };  // [4][L][CB]
    auto raw_at = [&](int half) { return reinterpret_cast<T *>(mine + 2 * M::rows + half * M::raw); };       // [2][L][NB]
    auto start_at = [&](int half) {  // [NB][CB]
        return reinterpret_cast<float *>(mine + 2 * (M::rows + M::raw) + half * M::start);
    };
    float *sB = reinterpret_cast<float *>(mine + 2 * (M::rows + M::raw + M::start)), *sC = sB + M::kC;       // [NB][kRow]
    auto words_of = [&](int w) {  // [N][CB]
        return reinterpret_cast<volatile unsigned long long *>(smem + w * M::warp(g.N) + M::words);
    };
    auto sums_of = [&](int w) { return reinterpret_cast<float *>(smem + w * M::warp(g.N) + M::sums(g.N)); };  // [N + 2][CB]
    float *sA = reinterpret_cast<float *>(smem + warps * M::warp(g.N));  // [N][CB]
    const Unit u = unit_of<CB>(g);
    long long s0, s1;
    g.ax.range(u.n, s0, s1);
    const bool live = lc < u.live;
    const int c = u.c0 + (live ? lc : 0);
    const T *x = static_cast<const T *>(g.x) + s0 * g.ld_x + u.c0;
    const T *dt = static_cast<const T *>(g.dt) + s0 * g.ld_dt + u.c0;
    const T *z = GATE ? static_cast<const T *>(g.z) + s0 * g.ld_z + u.c0 : nullptr;
    const T *dout = static_cast<const T *>(g.dout) + s0 * g.D + u.c0;
    const T *Bm = static_cast<const T *>(g.Bm) + s0 * g.ld_b + (long long)u.group * g.N;
    const T *Cm = static_cast<const T *>(g.Cm) + s0 * g.ld_c + (long long)u.group * g.N;
    const float *states0 = g.states + ssm_ckpt_base(s0, u.n) * g.N * g.D + u.c0;
    const float bias = g.dt_bias ? g.dt_bias[c] : 0.f, skip = g.Dskip ? g.Dskip[c] : 0.f;
    const int len = (int)(s1 - s0), tiles = (int)(((long long)len + L - 1) / L);
    float *part = g.part_bc + (long long)u.tile * 2 * g.N * g.ax.ntok;

    const int mode_x = WIDE ? kWide : g.mode_x, mode_b = WIDE ? kWide : g.mode_b, mode_s = WIDE ? kWide : g.mode_s;
    auto fetch = [&](int tile, int n0, int rh, int half) {
        const int have = min(L, len - tile * L), states = min(NB, g.N - n0);
        const long long t = (long long)tile * L;
        T *r = rows_at(rh), *b = raw_at(half);
        if (n0 == 0) {
            copy_rows<L, CB, 32>(r, x + t * g.ld_x, g.ld_x, have, u.live, mode_x, lane);
            copy_rows<L, CB, 32>(r + L * CB, dt + t * g.ld_dt, g.ld_dt, have, u.live, mode_x, lane);
            copy_rows<L, CB, 32>(r + 2 * L * CB, dout + t * g.D, g.D, have, u.live, mode_x, lane);
            if (GATE) copy_rows<L, CB, 32>(r + 3 * L * CB, z + t * g.ld_z, g.ld_z, have, u.live, mode_x, lane);
        }
        copy_rows<L, NB, 32>(b, Bm + t * g.ld_b + n0, g.ld_b, have, states, mode_b, lane);
        copy_rows<L, NB, 32>(b + L * NB, Cm + t * g.ld_c + n0, g.ld_c, have, states, mode_b, lane);
        copy_rows<NB, CB, 32>(start_at(half), states0 + ((long long)tile * g.N + n0) * g.D, g.D, states, u.live, mode_s,
                              lane);
    };

    if (warp < tiles) fetch(tiles - 1 - warp, 0, 0, 0);
    cp_async_commit();
    const int padded = M::padded(g.N);
    for (int e = warp * 32 + lane; e < padded * CB; e += warps * 32) {
        const int n = e % padded, j = e / padded;
        float a = 0.f, q = 0.f;
        if (j < u.live && n < g.N) {
            const long long at = ((long long)u.n * g.D + u.c0 + j) * g.N + n;
            a = g.A[(long long)(u.c0 + j) * g.N + n];
            if (g.dfinal) q = g.dfinal[at];
            if (tiles == 0 && g.dstate0) g.dstate0[at] = q;
        }
        sA[n * CB + j] = a;
        for (int w = 0; w < warps; ++w) {
            words_of(w)[n * CB + j] = w ? 0xffffffff00000000ull : g.first_tag | __float_as_uint(q);
            sums_of(w)[n * CB + j] = 0.f;
        }
    }
    __syncthreads();
    float sumD = 0.f, sumT = 0.f;
    int rh = 0, half = 0;
    for (int p = warp; p < tiles; p += warps, rh ^= 1) {
        const int tile = tiles - 1 - p, have = min(L, len - tile * L);
        const T *rx = rows_at(rh) + lc;
        f32x2 del[L / 2], dx[L / 2], go[L / 2], ddel[L / 2], du[L / 2], y[L / 2];
        float sum = 0.f;           // of the tile's steps
        for (int n0 = 0; n0 < g.N; n0 += NB, half ^= 1) {
            const int states = min(NB, g.N - n0);
            cp_async_wait();
            __syncwarp();
            widen<NB, M::kRow>(sB, sC, raw_at(half), have, states, lane);
            if (n0 + NB < g.N) fetch(tile, n0 + NB, rh, half ^ 1);
            else if (p + warps < tiles) fetch(tile - warps, 0, rh ^ 1, half ^ 1);
            cp_async_commit();
            if (n0 == 0) {
                // a lane's share of the tile's tokens
                float d[LS], w[LS], o[LS];
#pragma unroll
                for (int i = 0; i < LS; ++i) {
                    const int t = ls * LS + i;
                    w[i] = to_f(rx[t * CB]);
                    d[i] = to_f(rx[(L + t) * CB]) + bias;
                    o[i] = to_f(rx[(2 * L + t) * CB]);
                    if (GATE) {
                        const float zz = to_f(rx[(3 * L + t) * CB]);
                        o[i] *= zz * sigmoid_for<T>(zz);
                    }
                }
                if (g.softplus) {
#pragma unroll
                    for (int i = 0; i < LS; i += 2) softplus2<T>(d[i], d[i + 1]);
                }
#pragma unroll
                for (int i = 0; i < LS; ++i) w[i] *= d[i];
                if (have < L || u.live < CB) {
                    // behind the end, and channels of no one: step 0, so decay 1, input 0, gradient 0
#pragma unroll
                    for (int i = 0; i < LS; ++i)
                        if (!live || ls * LS + i >= have) d[i] = w[i] = o[i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < L; i += 2) {
                    const int j = i % LS, k1 = (i + 1) % LS;
                    float v[3][2] = {{d[j], d[k1]}, {w[j], w[k1]}, {o[j], o[k1]}};
                    if constexpr (NS > 1) {
#pragma unroll
                        for (int k = 0; k < 6; ++k)
                            v[k / 2][k % 2] = __shfl_sync(0xffffffffu, v[k / 2][k % 2], i / LS * CB + lc);
                    }
                    del[i / 2] = pack2(v[0][0], v[0][1]);
                    dx[i / 2] = pack2(v[1][0], v[1][1]);
                    go[i / 2] = pack2(v[2][0], v[2][1]);
                    ddel[i / 2] = du[i / 2] = y[i / 2] = 0;
                }
                sum = sum_of(del);
            }
            __syncwarp();
            const int at = (n0 + ls) * CB + lc;
            volatile unsigned long long *win = words_of(warp) + at;
            volatile unsigned long long *wout = words_of(warp + 1 < warps ? warp + 1 : 0) + at;
            const float *pa = sA + at, *ps = start_at(half) + ls * CB + lc;
            float *psum = sums_of(warp) + at;
            const ulonglong2 *b4 = reinterpret_cast<const ulonglong2 *>(sB + ls * M::kRow);
            const ulonglong2 *c4 = reinterpret_cast<const ulonglong2 *>(sC + ls * M::kRow);
#pragma unroll 1
            for (int n = ls; n < states + ls; n += NS) {
                unsigned long long in = *win;
                const float An = *pa;
                const f32x2 A22 = dup2(An * kLog2e);
                float h = live && n < states ? *ps : 0.f;
                f32x2 a[L / 2], hs[L / 2];       // decays, and the states before the tokens
                float v[L];
#pragma unroll
                for (int q4 = 0; q4 < L / 4; ++q4) {
                    const ulonglong2 bv = b4[q4], cv = c4[q4];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int i = 2 * q4 + k;
                        float e0, e1, u0, u1;
                        unpack2(fma2(del[i], A22, dup2(kEx2Low)), e0, e1);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        a[i] = pack2(e0, e1);
                        unpack2(mul2(dx[i], k ? bv.y : bv.x), u0, u1);
                        const float h0 = h, h1 = fmaf(e0, h0, u0);
                        h = fmaf(e1, h1, u1);
                        hs[i] = pack2(h0, h1);
                        const f32x2 after = pack2(h1, h);
                        if (GATE) y[i] = fma2(k ? cv.y : cv.x, after, y[i]);
                        unpack2(mul2(go[i], after), v[2 * i], v[2 * i + 1]);
                    }
                }
                // dC: lane lc ends with token lc (CB = 16), or tokens 2 lc, 2 lc + 1
                reduce_halving<CB / 2, 1, L>(v, lane);
                float *dst = part + ((long long)g.N + n0 + n) * g.ax.ntok + s0 + tile * L + lc * (L / CB);
#pragma unroll
                for (int k = 0; k < L / CB; ++k)
                    if (n < states && lc * (L / CB) + k < have) dst[k] = v[k];
                // the adjoint behind the tile, once the warp that has the tile behind has left it
                for (unsigned spin = 0; !__all_sync(0xffffffffu, (unsigned)(in >> 32) == (unsigned)p);) {
                    in = *win;
                    if (++spin > kSpinLimit) {
                        if (lane == 0) atomicOr(g.status, kStatusTimeout);
                        cp_async_wait();
                        __syncthreads();    // the one behind the tiles, where the others may stand
                        return;
                    }
                }
                const float first = __uint_as_float((unsigned)in), fix = ex2(fmaf(sum, An * kLog2e, kEx2Low)) - product_of(a);
                float q = first;
                f32x2 dA = 0;
                const f32x2 An2 = dup2(An);
#pragma unroll
                for (int q4 = L / 4 - 1; q4 >= 0; --q4) {
                    const ulonglong2 bv = b4[q4], cv = c4[q4];
#pragma unroll
                    for (int k = 1; k >= 0; --k) {
                        const int i = 2 * q4 + k;
                        float c0, c1, e0, e1;
                        unpack2(mul2(go[i], k ? cv.y : cv.x), c0, c1);
                        unpack2(a[i], e0, e1);
                        const float d1 = c1 + q, q1 = e1 * d1;
                        const float d0 = c0 + q1;
                        q = e0 * d0;
                        const f32x2 dh = pack2(d0, d1), m = mul2(pack2(q, q1), hs[i]);   // m: dL/d(delta A)
                        unpack2(mul2(dh, dx[i]), v[2 * i], v[2 * i + 1]);
                        du[i] = fma2(dh, k ? bv.y : bv.x, du[i]);
                        ddel[i] = fma2(m, An2, ddel[i]);
                        dA = fma2(m, del[i], dA);
                    }
                }
                q = fmaf(fix, first, q);
                *wout = (unsigned long long)(unsigned)(p + 1) << 32 | __float_as_uint(q);
                float a0, a1;
                unpack2(dA, a0, a1);
                *psum += a0 + a1;
                // dB, the same way
                reduce_halving<CB / 2, 1, L>(v, lane);
                dst -= (long long)g.N * g.ax.ntok;
#pragma unroll
                for (int k = 0; k < L / CB; ++k)
                    if (n < states && lc * (L / CB) + k < have) dst[k] = v[k];
                win += NS * CB;
                wout += NS * CB;
                pa += NS * CB;
                ps += NS * CB;
                psum += NS * CB;
                b4 += NS * M::kRow / 4;
                c4 += NS * M::kRow / 4;
            }
            if (tile == 0 && g.dstate0 && live) {
                wout = words_of(warp + 1 < warps ? warp + 1 : 0) + at;
                float *o = g.dstate0 + ((long long)u.n * g.D + c) * g.N + n0;
                for (int n = ls; n < states; n += NS, wout += NS * CB) o[n] = __uint_as_float((unsigned)*wout);
            }
            __syncwarp();
        }
        // what the rows still hold, before anything is stored
        float xs[LS], rs[LS], os[LS], zs[LS];
#pragma unroll
        for (int i = 0; i < LS; ++i) {
            const int t = ls * LS + i;
            xs[i] = to_f(rx[t * CB]);
            rs[i] = to_f(rx[(L + t) * CB]) + bias;
            os[i] = to_f(rx[(2 * L + t) * CB]);
            zs[i] = GATE ? to_f(rx[(3 * L + t) * CB]) : 0.f;
        }
        // the states' lanes add up, each keeping its share of the tokens
        float vu[L], vd[L], vy[L];
#pragma unroll
        for (int i = 0; i < L / 2; ++i) {
            unpack2(du[i], vu[2 * i], vu[2 * i + 1]);
            unpack2(ddel[i], vd[2 * i], vd[2 * i + 1]);
            unpack2(y[i], vy[2 * i], vy[2 * i + 1]);
        }
        reduce_halving<16, CB, L>(vu, lane);
        reduce_halving<16, CB, L>(vd, lane);
        if (GATE) reduce_halving<16, CB, L>(vy, lane);
        const long long row = (s0 + tile * L + ls * LS) * g.D + c;
        const int mine_n = live ? have - ls * LS : 0;
#pragma unroll
        for (int i = 0; i < LS; i += 2) {
            float st[2] = {rs[i], rs[i + 1]}, slope[2] = {1.f, 1.f};
            if (g.softplus) {
                f32x2 e;
                softplus2<T>(st[0], st[1], e);
                unpack2(e, slope[0], slope[1]);
                slope[0] = softplus_slope<T>(rs[i], slope[0]);
                slope[1] = softplus_slope<T>(rs[i + 1], slope[1]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int j = i + k;
                float o = os[j], dz = 0.f;
                if (GATE) {
                    const float sg = sigmoid_for<T>(zs[j]), full = fmaf(skip, xs[j], vy[j]);
                    dz = o * full * sg * fmaf(zs[j], 1.f - sg, 1.f);
                    o *= zs[j] * sg;
                }
                const float dd = fmaf(vu[j], xs[j], vd[j]) * slope[k];
                if (j < mine_n) {
                    const long long at = row + (long long)j * g.D;
                    static_cast<T *>(g.dx)[at] = from_f<T>(fmaf(vu[j], st[k], skip * o));
                    static_cast<T *>(g.ddt)[at] = from_f<T>(dd);
                    if (GATE) static_cast<T *>(g.dz)[at] = from_f<T>(dz);
                    sumT += dd;
                    sumD = fmaf(o, xs[j], sumD);
                }
            }
        }
        __syncwarp();
    }
#pragma unroll
    for (int o = 16; o >= CB; o >>= 1) {
        sumD += __shfl_xor_sync(0xffffffffu, sumD, o);
        sumT += __shfl_xor_sync(0xffffffffu, sumT, o);
    }
    if (ls == 0) {
        sums_of(warp)[padded * CB + lc] = sumD;
        sums_of(warp)[(padded + 1) * CB + lc] = sumT;
    }
    __syncthreads();
    float *out = g.part_par + (long long)u.n * g.D * (g.N + 2);
    for (int e = warp * 32 + lane; e < (g.N + 2) * CB; e += warps * 32) {
        const int n = e % (g.N + 2), j = e / (g.N + 2), at = (n < g.N ? n : padded + n - g.N) * CB + j;
        if (j >= u.live) continue;
        float s = 0.f;
        for (int w = 0; w < warps; ++w) s += sums_of(w)[at];
        if (n < g.N) out[(long long)(u.c0 + j) * g.N + n] = s;
        else out[(long long)g.D * n + u.c0 + j] = s;
    }
}

// dB, dC of 32 tokens of one group: the tiles' partial sums added in tile order and
// turned through shared memory into the tensors' layout. A warp adds one (which,
// state) row of the tokens; HBM binds (the partial sums are read once), so the loads of
// 16 tiles are in flight at a time. The rows of no sequence are cleared here, of all
// gradients of tokens.
constexpr int kBcRows = 16;      // (which, state) rows of a CTA, one per warp
template <typename T>
__global__ void __launch_bounds__(kBcRows * 32) ssm_bc_kernel(const SsmArgs g, int tiles) {
    __shared__ float sm[kBcRows][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = blockIdx.z, r0 = blockIdx.y * kBcRows;
    const long long t0 = (long long)blockIdx.x * 32, t = t0 + lane;
    const long long stride = 2LL * g.N * g.ax.ntok;
    float s = 0.f;
    if (t < g.ax.ntok && r0 + warp < 2 * g.N) {
        const float *p = g.part_bc + (long long)group * tiles * stride + (r0 + warp) * g.ax.ntok + t;
        int k = 0;
        for (; k + 16 <= tiles; k += 16) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __ldcs(p + (k + i) * stride);
#pragma unroll
            for (int i = 0; i < 16; ++i) s += v[i];
        }
        for (; k < tiles; ++k) s += __ldcs(p + k * stride);
    }
    sm[warp][lane] = s;
    __syncthreads();
    const int r = threadIdx.x % kBcRows, i = threadIdx.x / kBcRows, row = r0 + r;
    if (t0 + i >= g.ax.ntok) return;
    // tokens of no sequence have no partial sums
    const bool rest = g.ax.cu && (t0 + i < g.ax.cu[0] || t0 + i >= g.ax.cu[g.ax.nseq]);
    if (rest && !g.zero_rest) return;
    if (rest && r0 == 0) {
        const int per = g.D / g.G;
        const long long at = (t0 + i) * g.D + (long long)group * per;
        for (int c = r; c < per; c += kBcRows) {
            static_cast<T *>(g.dx)[at + c] = from_f<T>(0.f);
            static_cast<T *>(g.ddt)[at + c] = from_f<T>(0.f);
            if (g.z) static_cast<T *>(g.dz)[at + c] = from_f<T>(0.f);
        }
    }
    if (row >= 2 * g.N) return;
    T *o = static_cast<T *>(row < g.N ? g.dBm : g.dCm);
    o[((t0 + i) * g.G + group) * g.N + row % g.N] = from_f<T>(rest ? 0.f : sm[r][i]);
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
    static PerDevice<bool> attr[2];
    using M = FwdSmem<CB, T>;
    while (warps > 1 && M::bytes(g.N, warps) > (size_t)kSmemLimit) --warps;
    g.mode_x = copy_mode({{g.x, g.ld_x}, {g.dt, g.ld_dt}, {g.z, g.ld_z}}, g.D / g.G, sizeof(T), CB * sizeof(T));
    g.mode_b = copy_mode({{g.Bm, g.ld_b}, {g.Cm, g.ld_c}}, g.N, sizeof(T), 16);
    const bool wide = g.mode_x == kWide && g.mode_b == kWide;
    auto kern = wide ? ssm_forward_kernel<CB, OUT, true, T> : ssm_forward_kernel<CB, OUT, false, T>;
    const cudaError_t e = ensure_smem_attr(attr[wide], kern, kSmemLimit);
    if (e != cudaSuccess) return e;
    const unsigned rest = OUT && g.zero_rest && g.ax.cu && g.ax.ntok ? kRestBlocks : 0;
    kern<<<(unsigned)units + rest, dim3(32, warps), M::bytes(g.N, warps), st>>>(g, (unsigned)units);
    return cudaGetLastError();
}

template <bool OUT, typename T>
cudaError_t forward_t(const SsmArgs &g, int sms, cudaStream_t st) {
    const int per = g.D / g.G;
    auto units = [&](int cb) { return (long long)g.ax.nseq * g.G * ((per + cb - 1) / cb); };
    if (units(8) > 0x7fffffffLL - kRestBlocks) return cudaErrorInvalidValue;
    // 16 channels per CTA, or 8 where that leaves a quarter of the SMs without one (fewer
    // channels split the same rows into more CTAs, but share what every tile costs less:
    // with 16 and with 8 channels, 4 rows of 2048 tokens of 2048 channels took 174 and 197
    // us, 12 units of 130 channels and 64 states, of about 470 fp32 tokens, 70 and 63). As
    // many warps as fill the SMs' 16: one row of 131072 tokens of 2048 channels took 5.1,
    // 3.2 and 2.4 ms with 4, 8 and 16 of them, 8 rows of 4096 tokens 558, 547 and 585 us.
    const bool wide = 4 * units(16) >= 3LL * sms;
    const long long n = wide ? units(16) : units(8);
    // Packed sequences are uneven, and the longest is the last to end: 16 there.
    int warps = n <= (g.ax.cu ? 4 * sms : wide ? sms : 2 * sms) ? 16 : 8;
    const long long most = ((g.ax.cu ? g.ax.ntok : g.ax.T) + kTileL - 1) / kTileL;
    while (warps > 1 && warps / 2 >= most) warps /= 2;
    return wide ? forward_cb<16, OUT, T>(g, n, warps, st) : forward_cb<8, OUT, T>(g, n, warps, st);
}

template <int CB, bool GATE, typename T>
cudaError_t backward_cb(SsmArgs g, int sms, cudaStream_t st) {
    static PerDevice<bool> attr[2];
    using M = BwdSmem<CB, T>;
    const int tiles = ssm_backward_tiles(g.D, g.G, g.ax.nseq, sms);
    const long long units = (long long)g.ax.nseq * tiles;
    if (units > 0x7fffffffLL) return cudaErrorInvalidValue;
    // two CTAs of four warps fill an SM's registers (255 of a thread: the tile's six
    // arrays and a state's decays and walk stand in them; 168 cost spills and 1011 us for
    // 4 x 2048 tokens of 2048 channels against 551); eight warps where CTAs are few
    int warps = units > 2LL * sms ? 4 : 8;
    while (warps > 1 && M::bytes(g.N, warps) > (size_t)kSmemLimit) --warps;
    g.mode_x = copy_mode({{g.x, g.ld_x}, {g.dt, g.ld_dt}, {g.z, g.ld_z}, {g.dout, g.D}}, g.D / g.G, sizeof(T),
                         CB * sizeof(T));
    g.mode_b = copy_mode({{g.Bm, g.ld_b}, {g.Cm, g.ld_c}}, g.N, sizeof(T), 16);
    g.mode_s = copy_mode({{g.states, g.D}}, g.D / g.G, sizeof(float), 16);
    const bool wide = g.mode_x == kWide && g.mode_b == kWide && g.mode_s == kWide;
    auto kern = wide ? ssm_backward_kernel<CB, GATE, true, T> : ssm_backward_kernel<CB, GATE, false, T>;
    cudaError_t e = ensure_smem_attr(attr[wide], kern, kSmemLimit);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)units, dim3(32, warps), M::bytes(g.N, warps), st>>>(g);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (g.ax.ntok) {
        const unsigned rows = (2 * g.N + kBcRows - 1) / kBcRows;
        const dim3 grid((unsigned)((g.ax.ntok + 31) / 32), rows, (unsigned)g.G);
        ssm_bc_kernel<T><<<grid, kBcRows * 32, 0, st>>>(g, tiles / g.G);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Channels of a backward CTA: 16, or 8 where that leaves SMs without one.
int backward_channels(int D, int G, int nseq, int sms) {
    return (long long)nseq * G * ((D / G + 15) / 16) >= sms ? 16 : 8;
}

template <bool GATE, typename T>
cudaError_t backward_t(const SsmArgs &g, int sms, cudaStream_t st) {
    return backward_channels(g.D, g.G, g.ax.nseq, sms) == 16 ? backward_cb<16, GATE, T>(g, sms, st)
                                                             : backward_cb<8, GATE, T>(g, sms, st);
}

}  // namespace

cudaError_t launch_ssm_forward(const SsmArgs &g, bool bf16, int sms, cudaStream_t st) {
    if (g.ax.nseq == 0) return cudaSuccess;
    if (g.out) return bf16 ? forward_t<true, __nv_bfloat16>(g, sms, st) : forward_t<true, float>(g, sms, st);
    return bf16 ? forward_t<false, __nv_bfloat16>(g, sms, st) : forward_t<false, float>(g, sms, st);
}

// Channel tiles of the backward pass over all groups.
int ssm_backward_tiles(int D, int G, int nseq, int sms) {
    const int cb = backward_channels(D, G, nseq, sms);
    return G * ((D / G + cb - 1) / cb);
}

cudaError_t launch_ssm_backward(const SsmArgs &g, bool bf16, int sms, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (g.ax.nseq) {
        if (g.z) e = bf16 ? backward_t<true, __nv_bfloat16>(g, sms, st) : backward_t<true, float>(g, sms, st);
        else e = bf16 ? backward_t<false, __nv_bfloat16>(g, sms, st) : backward_t<false, float>(g, sms, st);
    }
    if (e != cudaSuccess) return e;
    const long long da = (long long)g.D * g.N, cols = da + 2LL * g.D;
    return launch_colsum(g.part_par, g.ax.nseq, cols, da, g.dA, g.D, g.dDskip, g.ddt_bias, st);
}

}  // namespace kla
