"""Plain fp64 references of the recurrent block's operators (short convolution,
selective scan, layer norm): test infrastructure, on the CPU, from the formulas,
one token after the other, with gradients by automatic differentiation.

Every function returns values and, beside each, a slack: a bound on how far a
correct fp32 evaluation may be off before its result is rounded. It counts fp32
roundings, each times the absolute value of the term that it rounds; the scan
carries them along its recurrence. U is one rounding (2^-24, relative);
functions of one argument (exp, softplus, sigmoid) are within 8 U, an
approximated power of two within 2^-22.
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
    rows = torch.cat([torch.arange(a, e) for a, e in sp]) if sp else torch.zeros(0, dtype=torch.long)
    go = None if dout is None else dout.double()
    gf = None if dout is None else torch.zeros_like(fin) if dfinal is None else dfinal.double()
    err = _scan_errors(x, raw, step, slope, A, Bm, Cm, Dskip, z, gate, h0, sp, softplus, go, gf)
    res = {"out": (out.detach(), err["out"][rows]), "final": (fin.detach(), err["final"])}
    if dout is None:
        return res
    gx, ga, gb, gA, gB, gC, gD, gg, gh = torch.autograd.grad([out, fin], leaves, [go[rows], gf], materialize_grads=True)
    ddt = (ga + gb) * slope
    res.update(dx=(gx[rows], err["dx"][rows]), dBm=(gB[rows], err["dBm"][rows]), dCm=(gC[rows], err["dCm"][rows]),
               dA=(gA, err["dA"]), dD=(gD, err["dD"]), dstate0=(gh, err["dstate0"]), ddt=(ddt[rows], err["ddt"][rows]),
               ddt_bias=(ddt[rows].sum(0), err["ddt_bias"]))
    if z is not None:
        s = torch.sigmoid(z)
        res["dz"] = ((gg * s * (1 + z * (1 - s)))[rows], err["dz"][rows])
    return res


def _scan_errors(x, raw, step, slope, A, Bm, Cm, Dskip, z, gate, h0, sp, softplus, go, gf):
    """dict name -> slack of ``scan``: an fp32 evaluation's errors carried along token by token, to first order (1 % on
    top for the rest) and at their worst, never with one token's or state's numbers for another's. Relative errors,
    in U:
      step      the sum with the bias is rounded once, which moves softplus by |raw| at raw < 0 (slope <= softplus) and
                by 1 above; its exponential is within 4, 1.3 |raw| for the exponent's product on top; 4 for the
                logarithm's polynomial and sums. 9 + 2.5 max(-raw, 0) in all. A plain step: 1.
      decay     the power of two 4, its raised exponent 0.3; the exponent delta A is off by the step's error, log2(e)
                and two products (2.3), and 4 more where the steps of a tile are summed up first; replacing a tile's
                product of decays takes another product per decay. 6 + |delta A| (step + 6.5). A decay below 2^-126
                may become 0.
      state     two roundings per token (the sum, a tile's correction); an input delta x B: step + 2
      gate      sigmoid 7 (an exponential 2, a sum, a quotient 4; approximated 1.3 |z| more) and two products
    A sum of n terms is off by n U of their absolute values."""
    D, N = A.shape
    G = Bm.shape[1]
    rep = D // G
    n_tok, S = x.shape[0], len(sp)
    lens = torch.tensor([e - a for a, e in sp], dtype=torch.long)
    L = int(lens.max()) if S else 0
    tiny = torch.finfo(torch.float32).tiny
    place = torch.arange(L)
    ok = place[:, None] < lens[None]                                        # [L, S]
    at = (torch.tensor([a for a, _ in sp], dtype=torch.long)[None] + place[:, None]).clamp(max=max(n_tok - 1, 0))
    zero = torch.zeros((), dtype=torch.float64)
    pick = lambda v: torch.where(ok.view(L, S, *[1] * (v.dim() - 1)), v[at] if n_tok else v.new_zeros(L, S, *v.shape[1:]), zero)  # noqa: E731

    def put(v):
        """[L, S, ...] back on the token axis."""
        res = v.new_zeros(n_tok, *v.shape[2:])
        if n_tok:
            res[at[ok]] = v[ok]
        return res

    spread = lambda v: v.repeat_interleave(rep, 2)  # noqa: E731
    X, St, Sl, Ga = pick(x), pick(step), pick(slope), pick(gate)
    B, C = pick(Bm), pick(Cm)
    e_st = pick((9 + 2.5 * (-raw).clamp(min=0)) * U) if softplus else torch.full_like(St, U)
    e_g = (9 + 1.3 * pick(z).abs()) * U if z is not None else torch.zeros_like(X)
    da = St[..., None] * A
    dec = torch.exp(da)
    e_dec = (6 + 6.5 * da.abs()) * U + da.abs() * e_st[..., None]
    u = (St * X)[..., None] * spread(B)
    live = ok[..., None, None]

    h, eh = h0, torch.zeros_like(h0)
    hs, es, prev, eprev = [], [], [], []
    for t in range(L):
        prev.append(h)
        eprev.append(eh)
        nh = dec[t] * h + u[t]
        ne = dec[t] * eh + (e_dec[t] * dec[t] + tiny) * h.abs() + 2 * U * nh.abs() + (e_st[t][..., None] + 2 * U) * u[t].abs()
        h, eh = torch.where(live[t], nh, h), torch.where(live[t], ne, eh)
        hs.append(h)
        es.append(eh)
    stack = lambda v: torch.stack(v) if L else h0.new_zeros(0, *h0.shape)  # noqa: E731
    H, E, P, EP = map(stack, (hs, es, prev, eprev))
    Cd = spread(C)
    y = (Cd * H).sum(-1) + Dskip * X
    ey = (Cd.abs() * E).sum(-1) + (N + 6) * U * (Cd * H).abs().sum(-1) + U * (Dskip * X).abs() + U * y.abs()
    slackened = lambda d: {k: 1.01 * v for k, v in d.items()}  # noqa: E731
    out = {"out": put(Ga.abs() * ey + (y * Ga).abs() * (e_g + U)), "final": eh}
    if go is None:
        return slackened(out)

    Go = pick(go)
    o, eo = Go * Ga, (Go * Ga).abs() * (e_g + U)
    q, eq = gf, torch.zeros_like(gf)
    dh, ed = [None] * L, [None] * L
    for t in range(L - 1, -1, -1):
        c = Cd[t] * o[t][..., None]
        nd = c + q
        ne = eq + Cd[t].abs() * eo[t][..., None] + 2 * U * c.abs() + U * nd.abs()
        nq = dec[t] * nd
        nqe = dec[t] * ne + (e_dec[t] * dec[t] + tiny) * nd.abs() + 2 * U * nq.abs()
        dh[t], ed[t] = nd, ne
        q, eq = torch.where(live[t], nq, q), torch.where(live[t], nqe, eq)
    DH, ED = torch.where(live, stack(dh), zero), torch.where(live, stack(ed), zero)
    Bd = spread(B)
    du = (Bd * DH).sum(-1)
    edu = (Bd.abs() * ED).sum(-1) + (N + 6) * U * (Bd * DH).abs().sum(-1)
    m = DH * dec * P                                                        # dL/d(delta A)
    em = dec * P.abs() * ED + (dec * DH).abs() * EP + m.abs() * (e_dec + 3 * U) + tiny * (DH * P).abs()
    vd = (A * m).sum(-1)
    evd = (A.abs() * em).sum(-1) + (N + 6) * U * (A * m).abs().sum(-1)
    dd = (du * X + vd) * Sl
    e_sl = pick((9 + 2.5 * raw.abs()) * U) if softplus else torch.zeros_like(Sl)
    edd = Sl * (X.abs() * edu + evd + 2 * U * ((du * X).abs() + vd.abs())) + dd.abs() * (e_sl + U)
    # sums over channels: lanes, then the channel tiles; over tokens: a thread's of every tile, warps, sequences
    over = lambda v: v.unflatten(2, (G, rep)).sum(3)  # noqa: E731
    chans, colsum = (rep / 8 + 8) * U, S / 32 + 33
    sx = (St * X)[..., None]
    tiles, toks = (L / 16 + 16 + colsum) * U, (L / 2 + 16 + colsum) * U
    out.update(
        dx=put(St * edu + (du * St).abs() * (e_st + 2 * U) + (Dskip.abs() * eo) + 2 * U * (Dskip * o).abs()),
        dBm=put(over(sx.abs() * ED + (DH * sx).abs() * (e_st[..., None] + 2 * U + chans))),
        dCm=put(over(o.abs()[..., None] * E + eo[..., None] * H.abs() + (o[..., None] * H).abs() * (U + chans))),
        dA=(St[..., None] * em + (m * St[..., None]).abs() * (e_st[..., None] + U + tiles)).sum((0, 1)),
        dD=(X.abs() * eo + (X * o).abs() * (U + toks)).sum((0, 1)),
        dstate0=eq, ddt=put(edd), ddt_bias=(edd + toks * dd.abs()).sum((0, 1)))
    if z is not None:
        Z = pick(z)
        s = torch.sigmoid(Z)
        ds = s * (1 + Z * (1 - s))
        out["dz"] = put((Go * ds).abs() * ey + (Go * y).abs() * ((18 + 3 * Z.abs()) * U * s * (1 + Z.abs()) + 3 * U * ds.abs()))
    return slackened(out)


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
