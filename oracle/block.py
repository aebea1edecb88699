"""Plain fp64 references of the recurrent block's operators (short convolution,
selective scan, layer norm): test infrastructure, on the CPU, from the formulas,
one token after the other, with gradients by automatic differentiation.

Every function returns values and, beside each, a slack: a bound on how far a
correct fp32 evaluation may be off before its result is rounded. It is a count
of fp32 roundings times the sum of the absolute values of the terms that enter
the result, which the references get by running the same formulas on absolute
values. U is one rounding (2^-24, relative); functions of one argument (exp,
softplus, sigmoid) are within 8 U, an approximated power of two within 2^-22.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24


def spans(n_tok, cu=None, B=None, T=None):
    """[(first token, end)] of every sequence."""
    if cu is not None:
        c = [int(v) for v in cu]
        return list(zip(c, c[1:]))
    return [(i * T, (i + 1) * T) for i in range(B)]


def close(got, want, slack, what):
    """|got - want| <= half a step of got's type (relative) + slack, everywhere."""
    half = torch.finfo(got.dtype).eps / 2
    g, w = got.detach().double().cpu(), want.detach()
    assert g.shape == w.shape, (what, g.shape, w.shape)
    # rounding acts on the computed value, which is itself within slack of want
    tol = half * (w.abs() + slack) + slack + torch.finfo(torch.float32).tiny
    bad = ~((g - w).abs() <= tol)
    if bad.any():
        i = int(((g - w).abs() / tol).nan_to_num(nan=float("inf")).argmax())
        raise AssertionError("%s: %d of %d values off; worst at %d: got %.9g, want %.9g, tolerance %.3g" % (
            what, int(bad.sum()), bad.numel(), i, g.flatten()[i], w.flatten()[i], tol.flatten()[i]))


def _silu(p):
    return p * torch.sigmoid(p)


# ---- convolution ------------------------------------------------------------------

def _conv_rows(x, w, b, s0, sp, silu):
    """Output rows and final states: x [Ntok, D], w [D, W], s0 [N, W-1, D]."""
    W = w.shape[1]
    out, fin = [], []
    for n, (a, e) in enumerate(sp):
        wide = torch.cat([s0[n], x[a:e]])
        pre = b + sum(wide[i:i + e - a] * w[:, i] for i in range(W)) if e > a else x[a:e]
        out.append(_silu(pre) if silu else pre)
        fin.append(wide[wide.shape[0] - (W - 1):])
    return torch.cat(out), torch.stack(fin)


def conv(x, w, b, s0, sp, silu=True, dout=None, dfinal=None):
    """dict name -> (value, slack); the token rows are those of the sequences, in order."""
    x, w, s0 = x.double(), w.double(), s0.double()
    b = torch.zeros(x.shape[1], dtype=torch.float64) if b is None else b.double()
    W = w.shape[1]
    leaves = [t.clone().requires_grad_() for t in (x, w, b, s0)]
    out, fin = _conv_rows(*leaves, sp, silu)
    pre, _ = _conv_rows(x, w, b, s0, sp, False)
    mag, _ = _conv_rows(x.abs(), w.abs(), b.abs(), s0.abs(), sp, False)
    # W products and sums, then silu (|silu'| <= 1.1). Its value: a power of two within 4 U whose
    # exponent's product is off by |pre| log2(e) U, hence itself by |pre| U; sum, quotient, product 4 U
    act = (12 + pre.abs()) * U
    res = {"out": (out.detach(), (W + 1) * U * 1.1 * mag + (act * pre.abs() if silu else 0)), "final": (fin.detach(), 0.0)}
    if dout is None:
        return res
    rows = torch.cat([dout[a:e] for a, e in sp]).double()
    dfin = torch.zeros_like(fin) if dfinal is None else dfinal.double()
    gx, gw, gb, gs = torch.autograd.grad([out, fin], leaves, [rows, dfin], materialize_grads=True)
    tok = torch.cat([torch.arange(a, e) for a, e in sp])
    # d = dout silu'(pre): |silu''| <= 0.5 carries pre's error; the slope s (1 + pre (1 - s)) with s
    # within (8 + |pre|) U and s (1 - s) <= 1/4: within 20 U (1 + |pre|)
    s = torch.sigmoid(pre)
    slope = s * (1 + pre * (1 - s)) if silu else torch.ones_like(pre)
    derr = rows.abs() * ((0.5 * (W + 1) * U * mag + 20 * U * (1 + pre.abs())) if silu else 0 * mag)
    dabs = (rows * slope).abs()
    # sums of |terms| with |d|, and of d's errors, through the same (linear) adjoint
    labs = [t.abs().clone().requires_grad_() for t in (x, w, b, s0)]
    lin, finl = _conv_rows(*labs, sp, False)
    ax, aw, ab, as_ = torch.autograd.grad([lin, finl], labs, [dabs, dfin.abs()], retain_graph=True, materialize_grads=True)
    ex, ew, eb, es = torch.autograd.grad([lin, finl], labs, [derr, torch.zeros_like(fin)], materialize_grads=True)
    # a token's gradient adds W + 1 terms; a weight's sums run over up to 64 tokens, 8 runs,
    # then the CTAs (of 128 tokens at least) in 32 strided groups and those
    chain = 64 + 8 + 32 + -(-x.shape[0] // (128 * 32)) + 4
    res.update(dx=(gx[tok], (W + 2) * U * ax[tok] + ex[tok]), dweight=(gw, chain * U * aw + ew),
               dbias=(gb, chain * U * ab + eb), dstate0=(gs, (W + 2) * U * as_ + es))
    return res


# ---- selective scan -----------------------------------------------------------------

def _scan_rows(x, step_a, step_b, A, Bm, Cm, Dskip, gate, h0, sp):
    """out rows and final states; step_a is delta in the decay, step_b in the input."""
    D, N = A.shape
    rep = D // Bm.shape[1]
    outs, fin, pres = [], [], []
    for n, (a, e) in enumerate(sp):
        h = h0[n]
        ys = []
        for t in range(a, e):
            b, c = Bm[t].repeat_interleave(rep, 0), Cm[t].repeat_interleave(rep, 0)
            h = torch.exp(step_a[t][:, None] * A) * h + (step_b[t] * x[t])[:, None] * b
            ys.append((c * h).sum(-1) + Dskip * x[t])
        fin.append(h)
        if ys:
            y = torch.stack(ys)
            pres.append(y)
            outs.append(y * gate[a:e])
    empty = x[:0]
    return (torch.cat(outs) if outs else empty), torch.stack(fin), (torch.cat(pres) if pres else empty)


def scan(x, dt, A, Bm, Cm, sp, Dskip=None, z=None, dt_bias=None, h0=None, softplus=True, dout=None, dfinal=None):
    """dict name -> (value, slack); token rows are those of the sequences, in order."""
    d = lambda t: None if t is None else t.double()  # noqa: E731
    x, dt, A, Bm, Cm, Dskip, z, dt_bias, h0 = map(d, (x, dt, A, Bm, Cm, Dskip, z, dt_bias, h0))
    D, N = A.shape
    zero = torch.zeros(D, dtype=torch.float64)
    Dskip = zero if Dskip is None else Dskip
    bias = zero if dt_bias is None else dt_bias
    h0 = torch.zeros(len(sp), D, N, dtype=torch.float64) if h0 is None else h0
    raw = dt + bias
    step = torch.nn.functional.softplus(raw, threshold=1e4) if softplus else raw
    slope = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
    gate = torch.ones_like(x) if z is None else _silu(z)
    lx, la, lb, lA, lB, lC, lD, lg, lh = leaves = [
        t.clone().requires_grad_() for t in (x, step, step, A, Bm, Cm, Dskip, gate, h0)]
    out, fin, pre = _scan_rows(lx, la, lb, lA, lB, lC, lD, lg, lh, sp)
    absl = [t.clone().requires_grad_() for t in
            (x.abs(), step, step.abs(), A, Bm.abs(), Cm.abs(), Dskip.abs(), gate.abs(), h0.abs())]
    aout, afin, apre = _scan_rows(*absl, sp)
    longest = max([e - a for a, e in sp] + [1])
    # A decay's relative error: its power of two (2^-22), its exponent's two roundings and
    # delta's error, at an exponent of at most E where the decay still counts, and the rounding
    # of its product; a path of up to `longest` decays adds them up, twice over where the
    # ranges' maps are joined. Decays below e^-40 leave nothing that counts.
    E = float(torch.clamp(-(step[..., None] * A), 0, 40).max()) if x.shape[0] else 0.0
    k = longest * (4 + 12 * E + 4) * 2 * U + (N + 24) * U
    rows = torch.cat([torch.arange(a, e) for a, e in sp]) if sp else torch.zeros(0, dtype=torch.long)
    res = {"out": (out.detach(), (k + 16 * U) * aout.detach()), "final": (fin.detach(), k * afin.detach())}
    if dout is None:
        return res
    go = dout.double()[rows]
    gf = torch.zeros_like(fin) if dfinal is None else dfinal.double()
    gx, ga, gb, gA, gB, gC, gD, gg, gh = torch.autograd.grad([out, fin], leaves, [go, gf], materialize_grads=True)
    ax, aa, ab, aA, aB, aC, aD, ag, ah = torch.autograd.grad([aout, afin], absl, [go.abs(), gf.abs()], materialize_grads=True)
    # the adjoint's paths meet the forward's: twice the chain; the decay's gradient with |A|
    aa, flush_a, flush_A = _abs_decay_grad(absl, sp, go.abs(), gf.abs())
    k2 = 2 * k + 48 * U
    tok_sum = (x.shape[0] + 64) * U
    res.update(
        dx=(gx[rows], k2 * ax[rows]), dBm=(gB[rows], (k2 + D * U) * aB[rows]), dCm=(gC[rows], (k2 + D * U) * aC[rows]),
        dA=(gA, (k2 + tok_sum) * aA.abs() + flush_A), dD=(gD, (k2 + tok_sum) * aD),
        dstate0=(gh, k2 * ah))
    ddt = (ga + gb) * slope
    addt = (aa + ab) * slope
    eddt = k2 * addt + flush_a * slope
    res["ddt"] = (ddt[rows], eddt[rows])
    res["ddt_bias"] = (ddt[rows].sum(0), (eddt + tok_sum * addt)[rows].sum(0))
    if z is not None:
        s = torch.sigmoid(z)
        ds = s * (1 + z * (1 - s))
        amp = s * (1 + z.abs() * (1 - s))
        res["dz"] = ((gg * ds)[rows], (k + 32 * U) * (ag * amp)[rows])
    return res


def _abs_decay_grad(absl, sp, go, gf):
    """Sum over states of |A| dL/d(delta A) per token, for the absolute problem; and
    what fp32 loses of it, and of dA, by flushing: a decay below 2^-126 becomes zero,
    so the term dh a h_prev that it stands in, with h_prev and dh of any size, loses
    at most 2^-126 |dh h_prev| (times |A|, or times delta)."""
    x, sa, sb, A, Bm, Cm, Dk, gate, h0 = [t.detach() for t in absl]
    D, N = A.shape
    rep = D // Bm.shape[1]
    tiny = torch.finfo(torch.float32).tiny
    res, flush, flush_A = torch.zeros_like(sa), torch.zeros_like(sa), torch.zeros_like(A)
    row = 0
    for n, (a, e) in enumerate(sp):
        h, hs = h0[n], []
        dec = [torch.exp(sa[t][:, None] * A) for t in range(a, e)]
        for i, t in enumerate(range(a, e)):
            hs.append(h)
            h = dec[i] * h + (sb[t] * x[t])[:, None] * Bm[t].repeat_interleave(rep, 0)
        q = gf[n]
        for i in range(e - a - 1, -1, -1):
            q = q + Cm[a + i].repeat_interleave(rep, 0) * (go[row + i] * gate[a + i])[:, None]
            res[a + i] = (q * dec[i] * hs[i] * A.abs()).sum(-1)
            flush[a + i] = tiny * (q * hs[i] * A.abs()).sum(-1)
            flush_A += tiny * q * hs[i] * sa[a + i][:, None].abs()
            q = q * dec[i]
        row += e - a
    return res, flush, flush_A


# ---- layer norm -----------------------------------------------------------------------

def layernorm(x, w=None, b=None, eps=1e-5, dout=None, dsum=None):
    """dict name -> (value, slack) for x [rows, D] (the sum, where there is a residual)."""
    x = x.double()
    R, D = x.shape
    one = torch.ones(D, dtype=torch.float64)
    w = one if w is None else w.double()
    b = 0 * one if b is None else b.double()
    lx, lw, lb = [t.clone().requires_grad_() for t in (x, w, b)]
    mean = lx.mean(1, keepdim=True)
    var = ((lx - mean) ** 2).mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    xh = (lx - mean) * rstd
    out = xh * lw + lb
    # sums over a row: at most 64 values in a thread, then 5 + 8 joins
    chain = min(D, 64) + 16
    emean = chain * U * x.abs().mean(1, keepdim=True)
    r = rstd.detach()
    # the mean's error shifts every deviation and enters the variance squared
    erel = (chain + 12) * U + (emean * r) ** 2
    exh = emean * r + xh.detach().abs() * erel + 4 * U * x.abs() * r
    res = {"out": (out.detach(), exh * w.abs() + 2 * U * (xh.detach() * w).abs() + 2 * U * b.abs()),
           "mean": (mean.detach()[:, 0], emean[:, 0]), "rstd": (r[:, 0], (r * erel)[:, 0])}
    if dout is None:
        return res
    dout = dout.double()
    gx, gw, gb = torch.autograd.grad(out, (lx, lw, lb), dout)
    e = (dout * w).abs()
    xa = xh.detach().abs()
    sums = e.mean(1, keepdim=True) + xa * (e * xa).mean(1, keepdim=True)
    slack = r * ((chain + 12) * U * (e + sums) + erel * (e + sums)
                 + exh * (e * xa).mean(1, keepdim=True) + xa * (e * exh).mean(1, keepdim=True))
    if dsum is not None:
        gx = gx + dsum.double()
        slack = slack + 2 * U * dsum.double().abs()
    long = R * U + 64 * U
    res.update(dx=(gx, slack), dweight=(gw, (long * dout.abs() * xa + dout.abs() * exh).sum(0)),
               dbias=(gb, (long * dout.abs()).sum(0)))
    return res
