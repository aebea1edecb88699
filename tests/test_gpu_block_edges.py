"""The recurrent block where it can go wrong beside its values: padded packed axes,
accuracy of the functions of one argument, captured single tokens, waits that run
out, and the block's operators around the Kalman mixer."""
import pytest
import torch

from bayesian_filter_scan_b200 import kla
from oracle import block as ob

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture
def poisoned():
    """New tensors are filled with NaN instead of whatever was in their memory."""
    torch.use_deterministic_algorithms(True)
    was = torch.utils.deterministic.fill_uninitialized_memory
    torch.utils.deterministic.fill_uninitialized_memory = True
    yield
    torch.utils.deterministic.fill_uninitialized_memory = was
    torch.use_deterministic_algorithms(False)


# ---- padded packed axes -----------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D,G,N,cu,n", [
    (16, 1, 8, [0, 20, 53], 62), (9, 3, 5, [3, 3, 40], 57), (24, 1, 33, [5, 30, 30], 31), (40, 2, 16, [70, 75, 75], 200),
    (8, 1, 4, [6, 6], 20), (264, 1, 16, [130, 131, 400], 431)])
def test_rows_of_no_sequence_are_zero_in_new_tensors(poisoned, D, G, N, cu, n, dtype):
    g = torch.Generator().manual_seed(n)
    t = DT[dtype]
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, z, dt, dout = (r(n, D).to(t).cuda() for _ in range(4))
    Bm, Cm = (r(n, G, N).to(t).cuda() for _ in range(2))
    A, w = -torch.rand(D, N, generator=g).cuda(), r(D, 4).cuda()
    out_of = torch.ones(n, dtype=torch.bool)
    out_of[cu[0]:cu[-1]] = False
    for v in (x, z, dt, dout, Bm, Cm):      # what lies there enters nothing
        v[out_of.cuda()] = float("nan")
    kw = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    y, st = kla.ssm_forward(x, dt, A, Bm, Cm, z=z, save_states=True, **kw)
    u = kla.conv_forward(x, w, **kw)
    c = kla.conv_backward(x, w, dout, **kw)
    res = {"out": y, "u": u, "conv dx": c["dx"], "dweight": c["dweight"], "dbias": c["dbias"]}
    for gate, states in ((z, st), (None, None)):
        s = kla.ssm_backward(x, dt, A, Bm, Cm, dout, z=gate, states=states, **kw)
        res.update({"%s %d" % (k, gate is not None): v for k, v in s.items()})
    torch.cuda.synchronize()
    for k, v in res.items():
        assert torch.isfinite(v.float()).all(), k
        if v.shape[0] == n:
            assert not v.cpu()[out_of].any(), k
    # a given output keeps them
    mine = torch.full((n, D), 7.0, dtype=t, device="cuda")
    kla.ssm_forward(x, dt, A, Bm, Cm, z=z, out=mine, **kw)
    assert (mine.cpu()[out_of] == 7).all() and torch.equal(mine.cpu()[~out_of], y.cpu()[~out_of])
    mine.fill_(7.0)
    kla.conv_forward(x, w, out=mine, **kw)
    assert (mine.cpu()[out_of] == 7).all() and torch.equal(mine.cpu()[~out_of], u.cpu()[~out_of])


# ---- functions of one argument -----------------------------------------------------
# One token of one state from zero, with steps, inputs, B and C of 1, leaves exactly
# the function that is looked at in an output or a gradient.

RANGES = [(-1, 1), (-8, -1), (-30, -8), (-80, -30), (1, 20)]


def one_token(D):
    one = torch.ones(1, D, device="cuda")
    return one, torch.ones(1, 1, 1, device="cuda"), -torch.ones(D, 1, device="cuda")


def arguments(D, lo, hi):
    return (lo + (hi - lo) * torch.rand(1, D, generator=torch.Generator().manual_seed(D + hi))).cuda()


def near(got, want, bound, what):
    err = ((got.double() - want).abs() - bound).max()
    assert err <= 0, (what, float(err), float(((got.double() - want) / want).abs().max()))


@pytest.mark.parametrize("lo,hi", RANGES)
@pytest.mark.parametrize("D", [64, 4096])
def test_fp32_gate_and_slopes(D, lo, hi):
    """sigmoid: an exponential within 2 U (one unit in the last place), the sum 1 U, the quotient 4 U (two units).
    With U = 2^-24: 7 U, one more for each product behind it."""
    one, bc, A = one_token(D)
    z = arguments(D, lo, hi)
    zd = z.double()
    s = torch.sigmoid(zd)
    args = (one, one, A, bc, bc)
    out, st = kla.ssm_forward(*args, z=z, softplus=False, save_states=True)
    near(out, zd * s, 9 * ob.U * (zd * s).abs(), "gate of a prompt")
    state = torch.zeros(1, D, 1, device="cuda")
    near(kla.ssm_step(*args, state, z=z, softplus=False), zd * s, 9 * ob.U * (zd * s).abs(), "gate of a step")
    g = kla.ssm_backward(*args, one, z=z, states=st, softplus=False)
    # s (1 + z (1 - s)): 1 - s within 7 U s + U, the product with z and the sum, both factors
    near(g["dz"], s * (1 + zd * (1 - s)), 18 * ob.U * s * (1 + zd.abs()), "slope of the gate")
    near(g["dx"], zd * s, 10 * ob.U * (zd * s).abs(), "gate in the gradient of x")
    # a step dt = z through softplus: its slope is sigmoid(z)
    g = kla.ssm_backward(one, z, A, bc, bc, one)
    near(g["ddt"], s, 8 * ob.U * s, "slope of softplus")


@pytest.mark.parametrize("lo,hi", RANGES)
@pytest.mark.parametrize("D", [64, 4096])
def test_fp32_softplus(D, lo, hi):
    """The exponential within 2 U, log(1 + y) no steeper than y, its polynomial within 5.3e-9 and 2 U of rounding,
    the last sum 1 U."""
    one, bc, A = one_token(D)
    dt = arguments(D, lo, hi)
    want = torch.logaddexp(dt.double(), torch.zeros_like(dt, dtype=torch.float64))
    near(kla.ssm_forward(one, dt, A, bc, bc), want, 6 * ob.U * want, "prompt")
    near(kla.ssm_step(one, dt, A, bc, bc, torch.zeros(1, D, 1, device="cuda")), want, 6 * ob.U * want, "step")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [16, 160])
@pytest.mark.parametrize("D", [1024, 8192])
def test_decays_have_no_side(D, T, dtype):
    """States of slow decays (2^-0.1 to 2^-0.01 a token), all terms positive: the error's mean over the channels. A
    decay may be off by 1e-8 on average, so a result by that times the decays that it holds: its sensitivity to
    them, taken from the 64-bit recurrence with decays 1e-6 larger. 1e-8 more for the mean of the roundings (each
    result 1e-7 at random, a thousand channels or more)."""
    g = torch.Generator().manual_seed(T + D)
    dt = (0.02 + 0.08 * torch.rand(T, D, generator=g)).to(DT[dtype])
    A = -torch.exp(torch.linspace(-1.2, 0.0, D))[:, None] * 0.6931
    one = torch.ones(T, D, dtype=DT[dtype], device="cuda")
    bc = torch.ones(T, 1, 1, dtype=DT[dtype], device="cuda")
    args = (one, dt.cuda(), A.cuda(), bc, bc)
    out, fin, st = kla.ssm_forward(*args, softplus=False, final_state=True, save_states=True)
    grad = kla.ssm_backward(*args, one, states=st, softplus=False)

    def exact(grow):
        d, a = dt.double(), A.double().requires_grad_()
        dec = torch.exp(d * a[:, 0]) * (1 + grow)
        h, ys = torch.zeros(D, dtype=torch.float64), []
        for t in range(T):
            h = dec[t] * h + d[t]
            ys.append(h)
        dA, = torch.autograd.grad(sum(y.sum() for y in ys), a)
        return {"out": ys[-1].detach(), "final": h.detach(), "dA": dA[:, 0]}

    want, more = exact(0.0), exact(1e-6)
    got = {"final": fin[0, :, 0], "dA": grad["dA"][:, 0]}
    if dtype == "fp32":
        got["out"] = out[-1]
    for k, v in got.items():
        held = float(((more[k] - want[k]) / want[k] / 1e-6).mean())
        mean = float(((v.double().cpu() - want[k]) / want[k]).mean())
        assert held > 2 and abs(mean) <= 1e-8 * held + 1e-8, (k, mean, held)


@pytest.mark.parametrize("lo,hi", [(0, 1), (1, 10), (10, 80)])
@pytest.mark.parametrize("N", [1, 4, 16])
def test_one_decay(N, lo, hi):
    """A state of 1 after one token without input. The exponent: log2(e) in fp32 is 0.25 U off, its products with A and
    with the step round twice, so 2.25 U of |delta A|; the power of two within 4 U of a prompt, 1.2 U of a step."""
    D = 1024
    one, bc = torch.zeros(1, D, device="cuda"), torch.ones(1, 1, N, device="cuda")
    d = arguments(D, lo, hi).abs()
    A = -torch.ones(D, N, device="cuda") + 0.5 * torch.rand(D, N, generator=torch.Generator().manual_seed(N)).cuda()
    x = d.double().t() * A.double()
    want = torch.exp(x)[None]
    state = torch.ones(1, D, N, device="cuda")
    _, fin = kla.ssm_forward(one, d, A, bc, bc, state0=state, softplus=False, final_state=True)
    near(fin, want, (4 + 2.3 * x.abs()) * ob.U * want, "prompt")
    kla.ssm_step(one, d, A, bc, bc, state, softplus=False)
    near(state, want, (1.2 + 2.3 * x.abs()) * ob.U * want, "step")


# ---- waits that run out ----------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_bounded_waits_of_the_scan_report_timeout(monkeypatch, dtype):
    """With the first tile's states withheld each kernel's wait gives up, the status says so, and the context works on."""
    g = torch.Generator().manual_seed(1)
    D, N, T = 40, 16, 200
    x = torch.randn(T, D, generator=g).to(DT[dtype]).cuda()
    bc = torch.randn(T, 1, N, generator=g).to(DT[dtype]).cuda()
    A = -torch.rand(D, N, generator=g).cuda()
    args = (x, x, A, bc, bc)
    want, states = kla.ssm_forward(*args, z=x, save_states=True)
    grads = kla.ssm_backward(*args, x, z=x, states=states)
    kla.check()
    for call in (lambda: kla.ssm_forward(*args, z=x), lambda: kla.ssm_backward(*args, x, z=x, states=states),
                 lambda: kla.ssm_backward(*args, x)):
        monkeypatch.setenv("KLA_TEST_WITHHOLD_TILES", "1")
        call()
        with pytest.raises(kla.KlaError) as e:
            kla.check()
        assert e.value.status == kla.KLA_ERR_TIMEOUT
        monkeypatch.delenv("KLA_TEST_WITHHOLD_TILES")
        out = kla.ssm_forward(*args, z=x)
        again = kla.ssm_backward(*args, x, z=x, states=states)
        kla.check()
        assert torch.equal(out, want) and all(torch.equal(again[k], grads[k]) for k in grads)


# ---- single tokens in a graph -----------------------------------------------------------

@pytest.mark.parametrize("dtype,B,D,N", [("bf16", 1, 64, 16), ("fp32", 9, 40, 20), ("bf16", 70, 128, 16), ("fp32", 3, 7, 5)])
def test_captured_single_tokens_follow_eager_ones(dtype, B, D, N):
    """A decoding step's two calls, captured on another stream and replayed token by token on states that change in
    place, leave bit for bit what eager calls leave."""
    g = torch.Generator().manual_seed(B + D)
    t = DT[dtype]
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    tokens = [[v.to(t).cuda() for v in (r(B, D), r(B, D), r(B, D), r(B, 1, N), r(B, 1, N))] for _ in range(7)]
    w, b, A, Dk = r(D, 4).cuda(), r(D).cuda(), -torch.rand(D, N, generator=g).cuda(), r(D).cuda()
    hist0, state0 = r(B, 3, D).to(t).cuda(), r(B, D, N).cuda()

    def step(tok, hist, state):
        x, dt, z, Bm, Cm = tok
        return kla.ssm_step(kla.conv_step(x, w, hist, b), dt, A, Bm, Cm, state, D=Dk, z=z)

    hist, state = hist0.clone(), state0.clone()
    want = [step(tok, hist, state) for tok in tokens]
    mine, mh, ms = [v.clone() for v in tokens[0]], hist0.clone(), state0.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(mine, mh.clone(), ms.clone())
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = step(mine, mh, ms)
    torch.cuda.synchronize()
    for _ in range(2):      # the second time around from the first states again
        mh.copy_(hist0)
        ms.copy_(state0)
        for tok, exp in zip(tokens, want):
            for m, v in zip(mine, tok):
                m.copy_(v)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, exp)
        assert torch.equal(mh, hist) and torch.equal(ms, state)


# ---- around the Kalman mixer -------------------------------------------------------------

def test_convolution_and_norm_around_the_kalman_mixer():
    """q, k, v through the block's convolution, the Kalman mixer, and a norm of every head's output: forward and
    gradients against the formulas in 64 bits. The bar is that of the mixer's own gradients, 2e-3 of the largest
    value (fp32 sums along the rows); the operators around it add some hundred roundings, 2^-24 each."""
    B, T, H, dk, dv, W = 2, 45, 2, 16, 32, 4
    n = B * T
    g = torch.Generator().manual_seed(5)
    r = lambda *s, sc=1.0: sc * torch.randn(*s, generator=g)  # noqa: E731
    x = {"q": r(n, H * dk), "k": r(n, H * dk), "v": r(n, H * dv)}
    w = {"q": r(H * dk, W, sc=0.5), "k": r(H * dk, W, sc=0.5), "v": r(H * dv, W, sc=0.5)}
    bias = {k: r(v.shape[1], sc=0.1) for k, v in x.items()}
    a, qn, beta = torch.sigmoid(r(n, H, dk) + 2), 0.1 * torch.rand(n, H, dk, generator=g), torch.sigmoid(r(n, H))
    lw, lb, dout = 1 + r(dv, sc=0.1), r(dv, sc=0.1), r(n * H, dv)
    c = lambda t: t.cuda()  # noqa: E731
    kw = dict(B=B, T=T)

    conv = {k: kla.conv_forward(c(x[k]), c(w[k]), c(bias[k]), **kw) for k in x}
    heads = {k: v.view(n, H, -1) for k, v in conv.items()}
    gates = (c(a), c(qn), c(beta))
    mix = kla.forward(heads["q"], heads["k"], heads["v"], *gates, **kw)
    y, mean, rstd = kla.layernorm_forward(mix.view(n * H, dv), c(lw), c(lb), stats=True)
    ln = kla.layernorm_backward(mix.view(n * H, dv), c(dout), mean, rstd, c(lw))
    mg = kla.backward(heads["q"], heads["k"], heads["v"], *gates, ln["dx"].view(n, H, dv), **kw)
    got = {"y": y, "lw": ln["dweight"], "lb": ln["dbias"], "a": mg["da"], "beta": mg["dbeta"]}
    for k in x:
        cg = kla.conv_backward(c(x[k]), c(w[k]), mg["d" + k].view(n, -1), c(bias[k]), **kw)
        got.update({"x" + k: cg["dx"], "w" + k: cg["dweight"], "b" + k: cg["dbias"]})
    torch.cuda.synchronize()
    kla.check()

    leaf = {"lw": lw, "lb": lb, "a": a, "beta": beta, **{"x" + k: v for k, v in x.items()},
            **{"w" + k: v for k, v in w.items()}, **{"b" + k: v for k, v in bias.items()}}
    leaf = {k: v.double().requires_grad_() for k, v in leaf.items()}
    sp = ob.spans(0, B=B, T=T)
    q, k, v = (ob._conv_rows(leaf["x" + i], leaf["w" + i], leaf["b" + i],
                             torch.zeros(B, W - 1, x[i].shape[1], dtype=torch.float64), sp, True)[0].view(n, H, -1)
               for i in "qkv")
    outs, qd = [], qn.double()
    for s, e in sp:
        lam, eta = torch.ones(H, dk, dtype=torch.float64), torch.zeros(H, dk, dv, dtype=torch.float64)
        for t in range(s, e):
            den = leaf["a"][t] ** 2 + qd[t] * lam
            bk = leaf["beta"][t][:, None] * k[t]
            eta = (leaf["a"][t] / den)[..., None] * eta + bk[..., None] * v[t][:, None, :]
            lam = lam / den + bk * k[t]
            outs.append(((q[t] / lam)[..., None] * eta).sum(1))
    m = torch.stack(outs).view(n * H, dv)
    mu = m.mean(1, keepdim=True)
    want = (m - mu) * (((m - mu) ** 2).mean(1, keepdim=True) + 1e-5).rsqrt() * leaf["lw"] + leaf["lb"]
    grads = torch.autograd.grad(want, list(leaf.values()), dout.double())
    for name, exp in [("y", want.detach())] + list(zip(leaf, grads)):
        err = (got[name].double().cpu() - exp).abs().max() / exp.abs().max()
        assert err <= 2e-3, (name, float(err))
