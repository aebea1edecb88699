// kla_block.cuh -- shared definitions of the recurrent block's kernels: short
// convolution, selective scan, layer norm (sm_100a).
#pragma once

#include <type_traits>

#include "kla_internal.cuh"

namespace kla {

// The sequences on the token axis: B rows of T tokens, or packed offsets.
struct SeqAxis {
    long long ntok, T;
    const int *cu;
    int nseq;

    // Tokens [s0, s1) of sequence n. Offsets are clamped to the axis, so a bad
    // offset cannot lead outside the tensors.
    __device__ __forceinline__ void range(int n, long long &s0, long long &s1) const {
        if (!cu) {
            s0 = n * T;
            s1 = s0 + T;
            return;
        }
        s0 = min(max((long long)cu[n], 0LL), ntok);
        s1 = min(max((long long)cu[n + 1], s0), ntok);
    }
    // The sequence that holds token t, or -1. Of several that start at the same
    // token the last one holds it: the others are empty.
    __device__ __forceinline__ int find(long long t) const {
        if (!cu) return (int)(t / T);
        if (t < cu[0] || t >= cu[nseq]) return -1;
        int lo = 0, hi = nseq;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= t) lo = mid; else hi = mid;
        }
        return lo;
    }
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// V contiguous values as floats: one access of V * sizeof(T) = 8 or 16 bytes, or V is 1.
template <int V, typename T>
__device__ __forceinline__ void load_v(const T *p, float (&x)[V]) {
    if constexpr (V == 1) {
        x[0] = to_f(*p);
    } else {
        constexpr int K = V * (int)sizeof(T) / 4;
        static_assert(K == 2 || K == 4, "one 8- or 16-byte access");
        uint32_t w[K];
        if constexpr (K == 4) {
            const uint4 r = *reinterpret_cast<const uint4 *>(p);
            w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
        } else {
            const uint2 r = *reinterpret_cast<const uint2 *>(p);
            w[0] = r.x; w[1] = r.y;
        }
#pragma unroll
        for (int i = 0; i < K; ++i) {
            if constexpr (sizeof(T) == 4) {
                x[i] = __uint_as_float(w[i]);
            } else {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
}

template <int V, typename T>
__device__ __forceinline__ void store_v(T *p, const float (&x)[V]) {
    if constexpr (V == 1) {
        *p = from_f<T>(x[0]);
    } else {
        constexpr int K = V * (int)sizeof(T) / 4;
        static_assert(K == 2 || K == 4, "one 8- or 16-byte access");
        uint32_t w[K];
#pragma unroll
        for (int i = 0; i < K; ++i) {
            if constexpr (sizeof(T) == 4) {
                w[i] = __float_as_uint(x[i]);
            } else {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&b);
            }
        }
        if constexpr (K == 4) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
}

// Clears n elements at p with `threads` threads, 16 bytes at a time where they go. A call:
// in line it changed the schedule of the scan's kernel around it (one row of 131072 tokens
// 2.54 ms, 2.45 with the call).
template <typename T>
__device__ __noinline__ void clear(T *p, long long n, long long tid, long long threads) {
    constexpr int V = 16 / (int)sizeof(T);
    const long long front = min(n, (long long)((16 - ((uintptr_t)p & 15)) & 15) / (int)sizeof(T));
    const long long wide = (n - front) / V, back = front + wide * V;
    for (long long e = tid; e < wide; e += threads)
        reinterpret_cast<uint4 *>(p + front)[e] = make_uint4(0, 0, 0, 0);
    for (long long e = tid; e < front + n - back; e += threads) p[e < front ? e : back + e - front] = from_f<T>(0.f);
}

// Sigmoid through the accurate exponential and an approximate quotient (2 units in
// the last place); 0 where the exponential overflows.
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + expf(-x)); }

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

// The same where the result is rounded to T: in bf16 the approximated power of two
// (2^-22) and quotient stay far below its 2^-9 and cost a third.
template <typename T>
__device__ __forceinline__ float sigmoid_for(float x) {
    if constexpr (sizeof(T) == 4) return sigmoid_f(x);
    return rcp(1.f + ex2(-kLog2e * x));
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

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 dup2(float x) { return pack2(x, x); }

// softplus(x) = max(x, 0) + log(1 + y) of two values, y = e^-|x| in (0, 1]. log(1 + y)
// is y times a polynomial of degree 9 with p(0) = 1, fitted to log(1 + y) / y on [0, 1]
// for the least relative error (iteratively reweighted least squares; each coefficient is
// rounded to fp32 before the ones behind it are fitted again). These coefficients are
// within 5.3e-9, without a side; 9.6e-8 with fp32's rounding. A small y keeps its digits
// that way, which the logarithm of a rounded 1 + y would not. T is the tensors' type: for
// bf16, whose steps are known to 2^-9, y comes from the approximated power of two, whose
// rounded exponent makes it |x| 2^-24 off (relative; 1e-6 at x = -12).
template <typename T>
__device__ __forceinline__ void softplus2(float &x0, float &x1, f32x2 &y) {
    if constexpr (sizeof(T) == 4) y = pack2(expf(-fabsf(x0)), expf(-fabsf(x1)));
    else y = pack2(ex2(-kLog2e * fabsf(x0)), ex2(-kLog2e * fabsf(x1)));
    f32x2 p = dup2(-0.0033065395f);
    p = fma2(p, y, dup2(0.020150334f));
    p = fma2(p, y, dup2(-0.057561528f));
    p = fma2(p, y, dup2(0.10670013f));
    p = fma2(p, y, dup2(-0.15349098f));
    p = fma2(p, y, dup2(0.19693193f));
    p = fma2(p, y, dup2(-0.24958156f));
    p = fma2(p, y, dup2(0.3333047f));
    p = fma2(p, y, dup2(-0.4999993f));
    p = fma2(p, y, dup2(1.f));
    float m0, m1;
    unpack2(fma2(p, y, pack2(fmaxf(x0, 0.f), fmaxf(x1, 0.f))), m0, m1);
    x0 = m0;
    x1 = m1;
}
template <typename T>
__device__ __forceinline__ void softplus2(float &x0, float &x1) {
    f32x2 y;
    softplus2<T>(x0, x1, y);
}
// The slope of softplus at x, sigmoid(x), from the y = e^-|x| that softplus2 leaves.
template <typename T>
__device__ __forceinline__ float softplus_slope(float x, float y) {
    const float n = x < 0.f ? y : 1.f;
    if constexpr (sizeof(T) == 4) return __fdividef(n, 1.f + y);
    return n * rcp(1.f + y);
}

// V floats as pairs (the last one alone when V is 1).
template <int V>
struct Pairs {
    static constexpr int K = (V + 1) / 2;
    f32x2 p[K];
    __device__ __forceinline__ void set(const float (&x)[V]) {
#pragma unroll
        for (int k = 0; k < K; ++k) p[k] = pack2(x[2 * k], V > 1 ? x[V > 1 ? 2 * k + 1 : 0] : 0.f);
    }
    __device__ __forceinline__ void get(float (&x)[V]) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float lo, hi;
            unpack2(p[k], lo, hi);
            x[2 * k] = lo;
            if (V > 1) x[V > 1 ? 2 * k + 1 : 0] = hi;
        }
    }
};
// V contiguous values as they are in memory, one access; widened when they are used.
template <int V, typename T>
struct Raw {
    static constexpr int K = V * (int)sizeof(T) / 4;      // words; 0: a single narrow element
    uint32_t w[K ? K : 1];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (K == 4) {
            const uint4 r = *reinterpret_cast<const uint4 *>(p);
            w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
        } else if constexpr (K == 2) {
            const uint2 r = *reinterpret_cast<const uint2 *>(p);
            w[0] = r.x; w[1] = r.y;
        } else if constexpr (K == 1) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
            w[0] = *reinterpret_cast<const unsigned short *>(p);
        }
    }
    // rounded to T, two values per instruction
    __device__ __forceinline__ void round(const float (&x)[V]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(x[i]);
        } else if constexpr (K == 0) {
            w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(x[0]));
        } else {
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&b);
            }
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (K == 4) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (K == 2) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else if constexpr (K == 1) *reinterpret_cast<uint32_t *>(p) = w[0];
        else *reinterpret_cast<unsigned short *>(p) = (unsigned short)w[0];
    }
    // the widened values back, exactly (they came from this type)
    __device__ __forceinline__ void set(const float (&x)[V]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(x[i]);
        } else if constexpr (K == 0) {
            w[0] = __float_as_uint(x[0]) >> 16;
        } else {
#pragma unroll
            for (int i = 0; i < K; ++i)
                w[i] = __float_as_uint(x[2 * i]) >> 16 | (__float_as_uint(x[2 * i + 1]) & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void get(float (&x)[V]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = __uint_as_float(w[i]);
        } else if constexpr (K == 0) {
            x[0] = __uint_as_float(w[0] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < K; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
};

// Sums part[rows][cols] over its rows in a fixed order: the first n0 columns go
// to out0, the next n1 to out1, the others to out2; a NULL output is skipped
// (kla_block_api.cu).
cudaError_t launch_colsum(const float *part, long long rows, long long cols, long long n0, float *out0, long long n1,
                          float *out1, float *out2, cudaStream_t st);

// Device address of the library's status word on the current device (kla_api.cu).
int *status_ptr();

// ---- launch functions behind the C ABI ------------------------------------------

struct ConvArgs {
    SeqAxis ax;
    int D, W;
    bool silu, zero_rest;
    long long ld_x;
    const void *x;
    const float *w, *bias;
    const void *state0;
    void *out, *final_state;
    // backward
    const void *dout, *dfinal;
    void *dx, *dstate0;
    float *part;       // [blocks][D*W taps, then D biases]
};
cudaError_t launch_conv_forward(const ConvArgs &, bool bf16, int sms, cudaStream_t);
int conv_backward_blocks(long long ntok);     // at most
cudaError_t launch_conv_backward(const ConvArgs &, bool bf16, int sms, float *dweight, float *dbias, cudaStream_t);
cudaError_t launch_conv_step(const ConvArgs &, bool bf16, int sms, cudaStream_t);

constexpr int kSsmCkpt = 16;      // tokens between two recorded states of a sequence
constexpr int kSsmMaxN = 128;

// Index of sequence n's first recorded state: floor(s0 / 16) + n leaves room for
// every earlier sequence's ceil(length / 16) records.
__host__ __device__ inline long long ssm_ckpt_base(long long s0, int n) { return s0 / kSsmCkpt + n; }
inline long long ssm_ckpt_count(long long ntok, int nseq) { return ntok / kSsmCkpt + nseq + 1; }

struct SsmArgs {
    SeqAxis ax;
    int D, G, N;
    bool softplus, zero_rest;
    long long ld_x, ld_dt, ld_z, ld_b, ld_c;
    const void *x, *dt, *Bm, *Cm, *z;
    const float *A, *Dskip, *dt_bias, *state0;
    void *out;
    float *final_state, *states;
    // backward
    const void *dout;
    const float *dfinal;
    void *dx, *ddt, *dBm, *dCm, *dz;
    float *dA, *dDskip, *ddt_bias, *dstate0;
    float *part_bc;    // [tiles][2][N][ntok]
    int *status;       // the library's device status word
    unsigned long long first_tag;     // the first tile's number beside its words; another one withholds them (test switch)
    int mode_x, mode_b, mode_s;  // how rows of x, dt, z (dout), of B, C, and of states are copied
    float *part_par;   // [nseq][D*N of dA, then D of dDskip, then D of ddt_bias]
};
cudaError_t launch_ssm_forward(const SsmArgs &, bool bf16, int sms, cudaStream_t);
int ssm_backward_tiles(int D, int G, int nseq, int sms);
cudaError_t launch_ssm_backward(const SsmArgs &, bool bf16, int sms, cudaStream_t);
cudaError_t launch_ssm_step(const SsmArgs &, bool bf16, int sms, cudaStream_t);

constexpr int kNormMaxD = 16384;

struct NormArgs {
    long long rows;
    int D;
    float eps;
    long long ld_x, ld_res;
    const void *x, *res;
    const float *w, *b;
    void *out, *sum;
    float *mean, *rstd;
    // backward
    const float *cmean, *crstd;
    const void *dout, *dsum;
    void *dx;
    float *part;       // [ctas][2][D]
};
cudaError_t launch_norm_forward(const NormArgs &, bool bf16, int sms, cudaStream_t);
int norm_backward_ctas(long long rows, int D, int sms);
cudaError_t launch_norm_backward(const NormArgs &, bool bf16, int ctas, float *dweight, float *dbias, cudaStream_t);

}  // namespace kla
