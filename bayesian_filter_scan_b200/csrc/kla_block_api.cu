// kla_block_api.cu -- the C ABI of the recurrent block (include/kla.h): checks of
// descriptors, pointers and overlaps, workspace layouts and launch sequences of
// the short convolution, the selective scan and layer norm; and the column sum
// that ends their gradients.
//
// Launches: every forward and step call is one kernel; kla_conv_backward two
// (three with dstate0), kla_layernorm_backward two, kla_ssm_backward three (four
// without recorded states). Nothing allocates, nothing synchronises.
#include <cstdlib>
#include <cstring>

#include "kla_block.cuh"
#include "../../include/kla.h"

namespace kla {

namespace {

// A CTA sums 32 columns: 32 row groups of strided rows, then the groups in order.
__global__ void __launch_bounds__(1024) colsum_kernel(const float *part, long long rows, long long cols, long long n0,
                                                      float *out0, long long n1, float *out1, float *out2) {
    __shared__ float sm[32][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < cols) {
#pragma unroll 4
        for (long long r = grp; r < rows; r += 32) s += part[r * cols + c];
    }
    sm[grp][lane] = s;
    __syncthreads();
    if (grp || c >= cols) return;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) s += sm[k][lane];
    if (c < n0) {
        if (out0) out0[c] = s;
    } else if (c < n0 + n1) {
        if (out1) out1[c - n0] = s;
    } else if (out2) {
        out2[c - n0 - n1] = s;
    }
}

constexpr int kMaxChannels = 1 << 20;

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

bool is_aligned(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

kla_status of_cuda(cudaError_t e) { return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA; }

int sm_count() {
    static PerDevice<int> counts;
    const int dev = current_device();
    if (dev < 0) return 148;
    int c = counts.v[dev].load(std::memory_order_acquire);
    if (!c) {
        if (cudaDeviceGetAttribute(&c, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || c <= 0) c = 148;
        counts.v[dev].store(c, std::memory_order_release);
    }
    return c;
}

// The buffers of a call: required ones present, aligned to their elements, and no
// output over an input or another output.
struct Buffers {
    struct Item { uintptr_t lo, hi; bool out; };
    Item items[24];
    int n = 0;
    bool ok = true;

    void add(const void *p, size_t bytes, size_t align, bool out, bool required) {
        if (!p) {
            if (required && bytes) ok = false;
            return;
        }
        if (!is_aligned(p, align)) ok = false;
        if (bytes) items[n++] = {(uintptr_t)p, (uintptr_t)p + bytes, out};
    }
    void in(const void *p, size_t bytes, size_t align, bool required = true) { add(p, bytes, align, false, required); }
    void out(const void *p, size_t bytes, size_t align, bool required = true) { add(p, bytes, align, true, required); }
    bool good() const {
        if (!ok) return false;
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < i; ++j)
                if ((items[i].out || items[j].out) && items[i].lo < items[j].hi && items[j].lo < items[i].hi)
                    return false;
        return true;
    }
};

// Bytes from the first to the last element of `rows` rows of `width` elements.
size_t span(long long rows, long long ld, long long width, size_t es) {
    return rows > 0 ? ((size_t)(rows - 1) * ld + width) * es : 0;
}

bool dtype_size(kla_dtype t, size_t &es) {
    if (t != KLA_BF16 && t != KLA_FP32) return false;
    es = t == KLA_BF16 ? 2 : 4;
    return true;
}

bool axis_of(int B, int T, const int *cu, int nseq, SeqAxis &ax) {
    if (B < 0 || T < 0 || (cu && nseq < 1)) return false;
    ax.ntok = (long long)B * T;
    ax.T = T;
    ax.cu = cu;
    ax.nseq = cu ? nseq : B;
    return true;
}

// 0 stands for a contiguous tensor.
bool stride_of(long long ld, long long width, long long &out) {
    out = ld ? ld : width;
    return out >= width;
}

kla_status conv_args(const kla_conv_desc *d, ConvArgs &g, size_t &es, bool step) {
    if (!d) return KLA_ERR_INVALID_ARG;
    std::memset((void *)&g, 0, sizeof(g));
    if (!axis_of(d->B, d->T, d->cu_seqlens, d->num_seqs, g.ax) || !dtype_size(d->dtype, es)) return KLA_ERR_INVALID_ARG;
    if (d->D < 1 || d->W < 1 || d->W > 4 || !stride_of(d->ld_x, d->D, g.ld_x)) return KLA_ERR_INVALID_ARG;
    if (step && (d->T != 1 || d->cu_seqlens)) return KLA_ERR_INVALID_ARG;
    if (d->D > kMaxChannels) return KLA_ERR_UNSUPPORTED;
    g.D = d->D;
    g.W = d->W;
    g.silu = d->silu != 0;
    g.zero_rest = d->zero_rest != 0;
    return KLA_OK;
}

kla_status ssm_args(const kla_ssm_desc *d, SsmArgs &g, size_t &es, bool step) {
    if (!d) return KLA_ERR_INVALID_ARG;
    std::memset((void *)&g, 0, sizeof(g));
    if (!axis_of(d->B, d->T, d->cu_seqlens, d->num_seqs, g.ax) || !dtype_size(d->dtype, es)) return KLA_ERR_INVALID_ARG;
    if (d->D < 1 || d->G < 1 || d->D % d->G || d->N < 1) return KLA_ERR_INVALID_ARG;
    const long long gn = (long long)d->G * d->N;
    if (!stride_of(d->ld_x, d->D, g.ld_x) || !stride_of(d->ld_dt, d->D, g.ld_dt) || !stride_of(d->ld_z, d->D, g.ld_z) ||
        !stride_of(d->ld_b, gn, g.ld_b) || !stride_of(d->ld_c, gn, g.ld_c))
        return KLA_ERR_INVALID_ARG;
    if (step && (d->T != 1 || d->cu_seqlens)) return KLA_ERR_INVALID_ARG;
    if (d->N > kSsmMaxN || d->D > kMaxChannels || d->G > 65535) return KLA_ERR_UNSUPPORTED;
    g.D = d->D;
    g.G = d->G;
    g.N = d->N;
    g.softplus = d->softplus != 0;
    g.zero_rest = d->zero_rest != 0;
    return KLA_OK;
}

// What the scan's kernels need where a wait runs out; the test switch lets the first one do.
bool ssm_waits(SsmArgs &g) {
    const char *s = getenv("KLA_TEST_WITHHOLD_TILES");
    g.first_tag = s && *s && *s != '0' ? 0xffffffff00000000ull : 0;
    return (g.status = status_ptr()) != nullptr;
}

size_t ssm_state_records(const SsmArgs &g) {
    return (size_t)ssm_ckpt_count(g.ax.ntok, g.ax.nseq) * g.N * g.D * sizeof(float);
}

struct SsmWorkspace { size_t bc, par, states, total; };
SsmWorkspace ssm_workspace(const SsmArgs &g, bool with_states) {
    SsmWorkspace w;
    w.bc = 0;
    w.par = align256((size_t)ssm_backward_tiles(g.D, g.G, g.ax.nseq, sm_count()) * 2 * g.N * g.ax.ntok * sizeof(float));
    w.states = w.par + align256((size_t)g.ax.nseq * g.D * (g.N + 2) * sizeof(float));
    w.total = w.states + (with_states ? 0 : align256(ssm_state_records(g)));
    return w;
}

// The inputs that every call of the scan reads.
void ssm_inputs(Buffers &b, const SsmArgs &g, size_t es) {
    const size_t d4 = (size_t)g.D * 4;
    b.in(g.x, span(g.ax.ntok, g.ld_x, g.D, es), es);
    b.in(g.dt, span(g.ax.ntok, g.ld_dt, g.D, es), es);
    b.in(g.z, span(g.ax.ntok, g.ld_z, g.D, es), es, false);
    b.in(g.Bm, span(g.ax.ntok, g.ld_b, (long long)g.G * g.N, es), es);
    b.in(g.Cm, span(g.ax.ntok, g.ld_c, (long long)g.G * g.N, es), es);
    b.in(g.A, d4 * g.N, 4);
    b.in(g.Dskip, d4, 4, false);
    b.in(g.dt_bias, d4, 4, false);
    if (g.ax.cu) b.in(g.ax.cu, 4 * ((size_t)g.ax.nseq + 1), 4);
}

kla_status norm_args(const kla_norm_desc *d, NormArgs &g, size_t &es) {
    if (!d) return KLA_ERR_INVALID_ARG;
    std::memset((void *)&g, 0, sizeof(g));
    if (d->rows < 0 || d->D < 1 || !(d->eps > 0.f) || !dtype_size(d->dtype, es)) return KLA_ERR_INVALID_ARG;
    if (!stride_of(d->ld_x, d->D, g.ld_x) || !stride_of(d->ld_residual, d->D, g.ld_res)) return KLA_ERR_INVALID_ARG;
    if (d->D > kNormMaxD) return KLA_ERR_UNSUPPORTED;
    g.rows = d->rows;
    g.D = d->D;
    g.eps = d->eps;
    return KLA_OK;
}

}  // namespace

cudaError_t launch_colsum(const float *part, long long rows, long long cols, long long n0, float *out0, long long n1,
                          float *out1, float *out2, cudaStream_t st) {
    if (cols == 0) return cudaSuccess;
    colsum_kernel<<<(unsigned)((cols + 31) / 32), 1024, 0, st>>>(part, rows, cols, n0, out0, n1, out1, out2);
    return cudaGetLastError();
}

}  // namespace kla

using namespace kla;

extern "C" {

kla_status kla_conv_forward(const kla_conv_desc *d, const void *x, const float *weight, const float *bias,
                            const void *state0, void *out, void *final_state, cudaStream_t st) {
    ConvArgs g;
    size_t es;
    kla_status s = conv_args(d, g, es, false);
    if (s != KLA_OK) return s;
    if (g.W == 1) state0 = nullptr, final_state = nullptr;
    const size_t hist = (size_t)g.ax.nseq * (g.W - 1) * g.D * es;
    Buffers b;
    b.in(x, span(g.ax.ntok, g.ld_x, g.D, es), es);
    b.in(weight, (size_t)g.D * g.W * 4, 4);
    b.in(bias, (size_t)g.D * 4, 4, false);
    b.in(state0, hist, es, false);
    if (g.ax.cu) b.in(g.ax.cu, 4 * ((size_t)g.ax.nseq + 1), 4);
    b.out(out, (size_t)g.ax.ntok * g.D * es, es);
    b.out(final_state, hist, es, false);
    if (!b.good()) return KLA_ERR_INVALID_ARG;
    g.x = x; g.w = weight; g.bias = bias; g.state0 = state0; g.out = out; g.final_state = final_state;
    return of_cuda(launch_conv_forward(g, d->dtype == KLA_BF16, sm_count(), st));
}

size_t kla_conv_backward_workspace_bytes(const kla_conv_desc *d) {
    ConvArgs g;
    size_t es;
    if (conv_args(d, g, es, false) != KLA_OK) return 0;
    return align256((size_t)conv_backward_blocks(g.ax.ntok) * g.D * (g.W + 1) * sizeof(float));
}

kla_status kla_conv_backward(const kla_conv_desc *d, const void *x, const float *weight, const float *bias,
                             const void *state0, const void *dout, const void *dfinal_state, void *dx, float *dweight,
                             float *dbias, void *dstate0, void *ws, size_t ws_bytes, cudaStream_t st) {
    ConvArgs g;
    size_t es;
    kla_status s = conv_args(d, g, es, false);
    if (s != KLA_OK) return s;
    if (g.W == 1) state0 = nullptr, dfinal_state = nullptr, dstate0 = nullptr;
    const size_t hist = (size_t)g.ax.nseq * (g.W - 1) * g.D * es, tok = (size_t)g.ax.ntok * g.D * es;
    const size_t need = kla_conv_backward_workspace_bytes(d);
    if (ws_bytes < need) return KLA_ERR_INVALID_ARG;
    Buffers b;
    b.in(x, span(g.ax.ntok, g.ld_x, g.D, es), es);
    b.in(weight, (size_t)g.D * g.W * 4, 4);
    b.in(bias, (size_t)g.D * 4, 4, false);
    b.in(state0, hist, es, false);
    b.in(dout, tok, es);
    b.in(dfinal_state, hist, es, false);
    if (g.ax.cu) b.in(g.ax.cu, 4 * ((size_t)g.ax.nseq + 1), 4);
    b.out(dx, tok, es);
    b.out(dweight, (size_t)g.D * g.W * 4, 4);
    b.out(dbias, (size_t)g.D * 4, 4, false);
    b.out(dstate0, hist, es, false);
    b.out(ws, need, 16);
    if (!b.good()) return KLA_ERR_INVALID_ARG;
    g.x = x; g.w = weight; g.bias = bias; g.state0 = state0; g.dout = dout; g.dfinal = dfinal_state;
    g.dx = dx; g.dstate0 = dstate0; g.part = (float *)ws;
    return of_cuda(launch_conv_backward(g, d->dtype == KLA_BF16, sm_count(), dweight, dbias, st));
}

kla_status kla_conv_step(const kla_conv_desc *d, const void *x, const float *weight, const float *bias, void *state,
                         void *out, cudaStream_t st) {
    ConvArgs g;
    size_t es;
    kla_status s = conv_args(d, g, es, true);
    if (s != KLA_OK) return s;
    Buffers b;
    b.in(x, span(g.ax.ntok, g.ld_x, g.D, es), es);
    b.in(weight, (size_t)g.D * g.W * 4, 4);
    b.in(bias, (size_t)g.D * 4, 4, false);
    b.out(state, (size_t)g.ax.nseq * (g.W - 1) * g.D * es, es);
    b.out(out, (size_t)g.ax.ntok * g.D * es, es);
    if (!b.good()) return KLA_ERR_INVALID_ARG;
    g.x = x; g.w = weight; g.bias = bias; g.final_state = state; g.out = out;
    return of_cuda(launch_conv_step(g, d->dtype == KLA_BF16, sm_count(), st));
}

size_t kla_ssm_states_bytes(const kla_ssm_desc *d) {
    SsmArgs g;
    size_t es;
    if (ssm_args(d, g, es, false) != KLA_OK) return 0;
    return ssm_state_records(g);
}

kla_status kla_ssm_forward(const kla_ssm_desc *d, const void *x, const void *dt, const float *A, const void *Bm,
                           const void *Cm, const float *Dskip, const void *z, const float *dt_bias,
                           const float *state0, void *out, float *final_state, float *states, cudaStream_t st) {
    SsmArgs g;
    size_t es;
    kla_status s = ssm_args(d, g, es, false);
    if (s != KLA_OK) return s;
    g.x = x; g.dt = dt; g.A = A; g.Bm = Bm; g.Cm = Cm; g.Dskip = Dskip; g.z = z; g.dt_bias = dt_bias;
    g.state0 = state0; g.out = out; g.final_state = final_state; g.states = states;
    const size_t state = (size_t)g.ax.nseq * g.D * g.N * 4;
    Buffers b;
    ssm_inputs(b, g, es);
    b.in(state0, state, 4, false);
    b.out(out, (size_t)g.ax.ntok * g.D * es, es);
    b.out(final_state, state, 4, false);
    b.out(states, ssm_state_records(g), 16, false);
    if (!b.good()) return KLA_ERR_INVALID_ARG;
    if (g.ax.ntok == 0 && !final_state) return KLA_OK;
    if (!ssm_waits(g)) return KLA_ERR_CUDA;
    return of_cuda(launch_ssm_forward(g, d->dtype == KLA_BF16, sm_count(), st));
}

size_t kla_ssm_backward_workspace_bytes(const kla_ssm_desc *d, int with_states) {
    SsmArgs g;
    size_t es;
    if (ssm_args(d, g, es, false) != KLA_OK) return 0;
    return ssm_workspace(g, with_states != 0).total;
}

kla_status kla_ssm_backward(const kla_ssm_desc *d, const void *x, const void *dt, const float *A, const void *Bm,
                            const void *Cm, const float *Dskip, const void *z, const float *dt_bias,
                            const float *state0, const float *states, const void *dout, const float *dfinal_state,
                            void *dx, void *ddt, float *dA, void *dBm, void *dCm, float *dDskip, void *dz,
                            float *ddt_bias, float *dstate0, void *ws, size_t ws_bytes, cudaStream_t st) {
    SsmArgs g;
    size_t es;
    kla_status s = ssm_args(d, g, es, false);
    if (s != KLA_OK) return s;
    if ((z == nullptr) != (dz == nullptr) && g.ax.ntok) return KLA_ERR_INVALID_ARG;
    const SsmWorkspace w = ssm_workspace(g, states != nullptr);
    if (ws_bytes < w.total) return KLA_ERR_INVALID_ARG;
    g.x = x; g.dt = dt; g.A = A; g.Bm = Bm; g.Cm = Cm; g.Dskip = Dskip; g.z = z; g.dt_bias = dt_bias;
    g.state0 = state0;
    const size_t state = (size_t)g.ax.nseq * g.D * g.N * 4, tok = (size_t)g.ax.ntok * g.D * es;
    const size_t bc = (size_t)g.ax.ntok * g.G * g.N * es, d4 = (size_t)g.D * 4;
    Buffers b;
    ssm_inputs(b, g, es);
    b.in(state0, state, 4, false);
    b.in(states, ssm_state_records(g), 16, false);
    b.in(dout, tok, es);
    b.in(dfinal_state, state, 4, false);
    b.out(dx, tok, es);
    b.out(ddt, tok, es);
    b.out(dz, tok, es, false);
    b.out(dBm, bc, es);
    b.out(dCm, bc, es);
    b.out(dA, d4 * g.N, 4);
    b.out(dDskip, d4, 4, false);
    b.out(ddt_bias, d4, 4, false);
    b.out(dstate0, state, 4, false);
    b.out(ws, w.total, 16);
    if (!b.good()) return KLA_ERR_INVALID_ARG;
    const bool bf16 = d->dtype == KLA_BF16;
    char *p = (char *)ws;
    g.part_bc = (float *)(p + w.bc);
    g.part_par = (float *)(p + w.par);
    if (!ssm_waits(g)) return KLA_ERR_CUDA;
    if (states) {
        g.states = const_cast<float *>(states);
    } else {
        // walk the states again: the forward kernel without outputs
        g.states = (float *)(p + w.states);
        if (g.ax.ntok) {
            const cudaError_t e = launch_ssm_forward(g, bf16, sm_count(), st);
            if (e != cudaSuccess) return KLA_ERR_CUDA;
        }
    }
    g.dout = dout; g.dfinal = dfinal_state;
    g.dx = dx; g.ddt = ddt; g.dz = dz; g.dBm = dBm; g.dCm = dCm;
    g.dA = dA; g.dDskip = dDskip; g.ddt_bias = ddt_bias; g.dstate0 = dstate0;
    return of_cuda(launch_ssm_backward(g, bf16, sm_count(), st));
}

kla_status kla_ssm_step(const kla_ssm_desc *d, const void *x, const void *dt, const float *A, const void *Bm,
                        const void *Cm, const float *Dskip, const void *z, const float *dt_bias, float *state,
                        void *out, cudaStream_t st) {
    SsmArgs g;
    size_t es;
    kla_status s = ssm_args(d, g, es, true);
    if (s != KLA_OK) return s;
    g.x = x; g.dt = dt; g.A = A; g.Bm = Bm; g.Cm = Cm; g.Dskip = Dskip; g.z = z; g.dt_bias = dt_bias;
    Buffers b;
    ssm_inputs(b, g, es);
    b.out(state, (size_t)g.ax.nseq * g.D * g.N * 4, 4);
    b.out(out, (size_t)g.ax.ntok * g.D * es, es);
    if (!b.good()) return KLA_ERR_INVALID_ARG;
    g.final_state = state;
    g.out = out;
    return of_cuda(launch_ssm_step(g, d->dtype == KLA_BF16, sm_count(), st));
}

kla_status kla_layernorm_forward(const kla_norm_desc *d, const void *x, const void *residual, const float *weight,
                                 const float *bias, void *out, void *sum, float *mean, float *rstd, cudaStream_t st) {
    NormArgs g;
    size_t es;
    kla_status s = norm_args(d, g, es);
    if (s != KLA_OK) return s;
    if (sum && !residual) return KLA_ERR_INVALID_ARG;
    g.x = x; g.res = residual; g.w = weight; g.b = bias; g.out = out; g.sum = sum; g.mean = mean; g.rstd = rstd;
    const size_t tok = (size_t)g.rows * g.D * es;
    // a thread reads its values of x and the residual before it writes the same
    // places, so the outputs may take the place of contiguous inputs
    const bool x_flat = g.ld_x == g.D, r_flat = g.ld_res == g.D;
    const void *over_x = x_flat && (out == x || (sum && sum == x)) ? x : nullptr;
    const void *over_r = r_flat && sum && sum == residual ? residual : nullptr;
    Buffers b;
    if (!x) return g.rows ? KLA_ERR_INVALID_ARG : KLA_OK;
    if (!over_x) b.in(x, span(g.rows, g.ld_x, g.D, es), es);
    if (!over_r) b.in(residual, span(g.rows, g.ld_res, g.D, es), es, false);
    b.in(weight, (size_t)g.D * 4, 4, false);
    b.in(bias, (size_t)g.D * 4, 4, false);
    b.out(out, tok, es);
    b.out(sum, tok, es, false);
    b.out(mean, (size_t)g.rows * 4, 4, false);
    b.out(rstd, (size_t)g.rows * 4, 4, false);
    if (!b.good()) return KLA_ERR_INVALID_ARG;
    return of_cuda(launch_norm_forward(g, d->dtype == KLA_BF16, sm_count(), st));
}

size_t kla_layernorm_backward_workspace_bytes(const kla_norm_desc *d) {
    NormArgs g;
    size_t es;
    if (norm_args(d, g, es) != KLA_OK) return 0;
    return align256((size_t)norm_backward_ctas(g.rows, g.D, sm_count()) * 2 * g.D * sizeof(float));
}

kla_status kla_layernorm_backward(const kla_norm_desc *d, const void *x, const float *weight, const float *mean,
                                  const float *rstd, const void *dout, const void *dsum, void *dx, float *dweight,
                                  float *dbias, void *ws, size_t ws_bytes, cudaStream_t st) {
    NormArgs g;
    size_t es;
    kla_status s = norm_args(d, g, es);
    if (s != KLA_OK) return s;
    const bool sums = dweight || dbias;
    const int ctas = norm_backward_ctas(g.rows, g.D, sm_count());
    const size_t need = sums ? align256((size_t)ctas * 2 * g.D * sizeof(float)) : 0;
    if (ws_bytes < need) return KLA_ERR_INVALID_ARG;
    g.x = x; g.w = weight; g.cmean = mean; g.crstd = rstd; g.dout = dout; g.dsum = dsum; g.dx = dx;
    const size_t tok = (size_t)g.rows * g.D * es, d4 = (size_t)g.D * 4;
    Buffers b;
    b.in(x, span(g.rows, g.ld_x, g.D, es), es);
    b.in(weight, d4, 4, false);
    b.in(mean, (size_t)g.rows * 4, 4);
    b.in(rstd, (size_t)g.rows * 4, 4);
    b.in(dout, tok, es);
    b.in(dsum, tok, es, false);
    b.out(dx, tok, es);
    b.out(dweight, d4, 4, false);
    b.out(dbias, d4, 4, false);
    if (sums) b.out(ws, need, 16);
    if (!b.good()) return KLA_ERR_INVALID_ARG;
    g.part = sums ? (float *)ws : nullptr;
    return of_cuda(launch_norm_backward(g, d->dtype == KLA_BF16, ctas, dweight, dbias, st));
}

}  // extern "C"
