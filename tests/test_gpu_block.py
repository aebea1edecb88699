"""The recurrent block on the GPU (short convolution, selective scan, layer norm)
against the fp64 references of oracle/block.py, whose slacks count the fp32
roundings; a result in a narrower type may be half a step of it further off."""
import pytest
import torch

from bayesian_filter_scan_b200 import kla
from oracle import block as ob

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def dev(t):
    """On the GPU with the same strides."""
    if t is None:
        return None
    base = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
    return base.copy_(t)


def rows_of(sp):
    return torch.cat([torch.arange(a, e) for a, e in sp])


def check(got, want, names, what=""):
    for name, key in names.items():
        ob.close(got[name], *want[key], what + " " + name)


def axis(lens, packed, tail=0):
    """(sequences' spans, keyword arguments, tokens); packed axes may go on behind the last sequence."""
    if not packed:
        assert len(set(lens)) == 1
        return ob.spans(0, B=len(lens), T=lens[0]), dict(B=len(lens), T=lens[0]), sum(lens)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    return ob.spans(0, cu=cu), dict(cu_seqlens=cu.cuda()), int(cu[-1]) + tail


# ---- convolution -----------------------------------------------------------------------

def conv_case(lens, packed, D, W, dtype, seed=0, strided=False, tail=0):
    g = gen(seed)
    sp, kw, n = axis(lens, packed, tail)
    wide = torch.randn(n, (2 if strided else 1) * D + (3 if strided else 0), generator=g).to(DT[dtype])
    x = wide[:, 1:D + 1] if strided else wide
    w, b = torch.randn(D, W, generator=g) / W ** 0.5, 0.1 * torch.randn(D, generator=g)
    s0 = torch.randn(len(lens), W - 1, D, generator=g).to(DT[dtype])
    dout = torch.randn(n, D, generator=g).to(DT[dtype])
    dfin = torch.randn(len(lens), W - 1, D, generator=g).to(DT[dtype])
    return sp, kw, x, w, b, s0, dout, dfin


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,packed,D,W,strided", [
    ([1], False, 8, 4, False), ([2, 2, 2], False, 64, 4, False), ([33, 33], False, 40, 3, True),
    ([16, 0, 1, 0, 47, 2, 3], True, 24, 4, False), ([300, 1, 258], True, 264, 4, False), ([70, 71], True, 9, 2, True),
    ([5, 130], True, 1, 4, False), ([64, 64], False, 128, 1, False), ([0, 0], True, 16, 4, False),
    ([700], False, 1032, 4, False)])
def test_conv(lens, packed, D, W, strided, dtype):
    sp, kw, x, w, b, s0, dout, dfin = conv_case(lens, packed, D, W, dtype, seed=len(lens) + D, strided=strided)
    for silu, bias, hist in ((True, b, s0), (False, None, None)):
        out, fin = kla.conv_forward(dev(x), w.cuda(), dev(bias), state0=dev(hist), silu=silu, final_state=True, **kw)
        g = kla.conv_backward(dev(x), w.cuda(), dev(dout), dev(bias), state0=dev(hist),
                              dfinal_state=dev(dfin) if silu else None, silu=silu, **kw)
        want = ob.conv(x, w, bias, hist if hist is not None else torch.zeros_like(s0), sp, silu, dout,
                       dfin if silu else None)
        check({"out": out, "final": fin, **g}, want,
              {k: k for k in ("out", "final", "dx", "dweight", "dbias") + (("dstate0",) if hist is not None else ())})


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("fp32", 7)])
def test_conv_split_and_steps_equal_the_whole(dtype, D):
    sp, kw, x, w, b, s0, _, _ = conv_case([50, 50, 50], False, D, 4, dtype, seed=3)
    x3 = x.view(3, 50, D)
    whole, fin = kla.conv_forward(x.cuda(), w.cuda(), b.cuda(), state0=s0.cuda(), final_state=True, **kw)
    first, mid = kla.conv_forward(x3[:, :31].reshape(-1, D).cuda(), w.cuda(), b.cuda(), state0=s0.cuda(),
                                  final_state=True, B=3, T=31)
    rest = [kla.conv_step(x3[:, t].cuda(), w.cuda(), mid, b.cuda()) for t in range(31, 50)]
    got = torch.cat([first.view(3, 31, D), torch.stack(rest, 1)], 1)
    assert torch.equal(got, whole.view(3, 50, D)) and torch.equal(mid, fin)


# ---- selective scan ----------------------------------------------------------------------

def scan_case(lens, packed, D, G, N, dtype, seed=0, strided=False, tail=0, lo=0.001, hi=0.3):
    g = gen(seed)
    t = DT[dtype]
    sp, kw, n = axis(lens, packed, tail)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    if strided:
        xz = r(n, 2 * D + 1).to(t)
        proj = r(n, 5 + 2 * G * N).to(t)
        x, z = xz[:, :D], xz[:, D + 1:]
        Bm, Cm = proj[:, 5:5 + G * N].unflatten(1, (G, N)), proj[:, 5 + G * N:].unflatten(1, (G, N))
    else:
        x, z, Bm, Cm = r(n, D).to(t), r(n, D).to(t), r(n, G, N).to(t), r(n, G, N).to(t)
    step = lo * (hi / lo) ** torch.rand(D, generator=g)
    p = dict(x=x, dt=(0.5 * r(n, D)).to(t), A=-(0.5 + torch.rand(D, N, generator=g) * N), Bm=Bm, Cm=Cm)
    o = dict(D=r(D), z=z, dt_bias=step + torch.log(-torch.expm1(-step)), state0=r(len(lens), D, N))
    return sp, kw, p, o, r(n, D).to(t), r(len(lens), D, N)


def run_scan(p, o, kw, dout, dfin, saved, softplus=True):
    P, O = {k: dev(v) for k, v in p.items()}, {k: dev(v) for k, v in o.items()}
    got = kla.ssm_forward(**P, **O, softplus=softplus, final_state=True, save_states=saved, **kw)
    g = kla.ssm_backward(P.pop("x"), P.pop("dt"), P.pop("A"), P.pop("Bm"), P.pop("Cm"), dev(dout), **O,
                         dfinal_state=dev(dfin), states=got[2] if saved else None, softplus=softplus, **kw)
    return {"out": got[0], "final": got[1], **g}


def want_scan(sp, p, o, dout, dfin, softplus=True):
    return ob.scan(**p, sp=sp, Dskip=o.get("D"), z=o.get("z"), dt_bias=o.get("dt_bias"), h0=o.get("state0"),
                   softplus=softplus, dout=dout, dfinal=dfin)


def scan_names(want):
    return {k: k for k in want}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,packed,D,G,N,strided", [
    ([1], False, 8, 1, 16, False), ([15, 15], False, 16, 1, 16, True), ([17], False, 5, 1, 1, False),
    ([128, 128], False, 24, 2, 8, False), ([129], False, 16, 1, 20, True), ([300], False, 33, 3, 5, False),
    ([1, 0, 2, 140, 0, 3], True, 18, 1, 16, False), ([257, 300], True, 20, 2, 33, True),
    ([40], False, 16, 1, 128, False), ([0, 0], True, 8, 1, 4, False), ([600], False, 8, 1, 3, False)])
def test_scan(lens, packed, D, G, N, strided, dtype):
    sp, kw, p, o, dout, dfin = scan_case(lens, packed, D, G, N, dtype, seed=D + N, strided=strided)
    want = want_scan(sp, p, o, dout, dfin)
    check(run_scan(p, o, kw, dout, dfin, saved=True), want, scan_names(want))


@pytest.mark.parametrize("B,D,T", [(40, 128, 20), (80, 128, 9), (300, 7, 130)])
def test_scan_many_units(B, D, T):
    # enough sequences that wider channel tiles are taken
    sp, kw, p, o, dout, dfin = scan_case([T] * B, False, D, 1, 4, "fp32", seed=B)
    want = want_scan(sp, p, o, dout, dfin)
    check(run_scan(p, o, kw, dout, dfin, saved=True), want, scan_names(want))


@pytest.mark.parametrize("B,D,T,N,dtype", [(160, 16, 35, 40, "bf16"), (160, 12, 18, 33, "fp32"), (120, 24, 50, 17, "bf16"),
                                           (40, 64, 33, 128, "fp32")])
def test_scan_many_units_of_many_states(B, D, T, N, dtype):
    # several blocks of states, even and odd in number, on wide channel tiles
    sp, kw, p, o, dout, dfin = scan_case([T] * B, False, D, 1, N, dtype, seed=N, strided=D == 12)
    want = want_scan(sp, p, o, dout, dfin)
    check(run_scan(p, o, kw, dout, dfin, saved=True), want, scan_names(want))


def test_scan_long_row_follows_its_parts():
    """A row of many tiles per warp equals its parts run one after the other, each from the state before it."""
    T, D, N = 9000, 40, 16
    sp, kw, p, o, dout, dfin = scan_case([T], False, D, 1, N, "fp32", seed=21)
    P, O = {k: dev(v) for k, v in p.items()}, {k: dev(v) for k, v in o.items()}
    whole, fin = kla.ssm_forward(**P, **O, final_state=True, **kw)
    state, outs = O.pop("state0"), []
    z = O.pop("z")
    for a in range(0, T, 1232):
        e = min(T, a + 1232)
        part = {k: v[a:e] if k != "A" else v for k, v in P.items()}
        out, state = kla.ssm_forward(**part, **O, z=z[a:e], state0=state, final_state=True, B=1, T=e - a)
        outs.append(out)
    # parts of whole tiles: every token takes the same steps
    assert torch.equal(torch.cat(outs), whole) and torch.equal(state, fin)


@pytest.mark.parametrize("drop", ["D", "z", "dt_bias", "state0", "all"])
def test_scan_without_optional_inputs(drop):
    sp, kw, p, o, dout, dfin = scan_case([70, 70], False, 12, 1, 6, "fp32", seed=1)
    o = {k: v for k, v in o.items() if drop not in (k, "all")}
    if "dt_bias" not in o:
        p["dt"] = p["dt"] - 2
    want = want_scan(sp, p, o, dout, None)
    check(run_scan(p, o, kw, dout, None, saved=False), want, scan_names(want))


def test_scan_plain_steps():
    # softplus off: dt is the step itself, zero among the steps
    sp, kw, p, o, dout, dfin = scan_case([90], False, 10, 1, 7, "fp32", seed=2)
    p["dt"] = (p["dt"].abs() * 0.2) * (torch.arange(90)[:, None] % 3 > 0)
    del o["dt_bias"]
    want = want_scan(sp, p, o, dout, dfin, softplus=False)
    check(run_scan(p, o, kw, dout, dfin, saved=True, softplus=False), want, scan_names(want))


@pytest.mark.parametrize("shift,scale", [(6.0, 20.0), (-12.0, 1.0), (0.0, 0.0), (100.0, 1.0)])
def test_scan_extreme_decays(shift, scale):
    # decays that underflow, steps next to zero, no decay at all, steps beyond softplus's bend
    sp, kw, p, o, dout, dfin = scan_case([200], False, 9, 1, 5, "fp32", seed=4)
    p["dt"], p["A"] = p["dt"] + shift, p["A"] * scale
    want = want_scan(sp, p, o, dout, dfin)
    got = run_scan(p, o, kw, dout, dfin, saved=True)
    assert all(torch.isfinite(v.float()).all() for v in got.values())
    check(got, want, scan_names(want))


def test_scan_states_walked_again_give_the_same_gradients():
    sp, kw, p, o, dout, dfin = scan_case([300, 131], True, 40, 1, 16, "bf16", seed=5)
    a = run_scan(p, o, kw, dout, dfin, saved=True)
    b = run_scan(p, o, kw, dout, dfin, saved=False)
    want = want_scan(sp, p, o, dout, dfin)
    check(b, want, scan_names(want))
    for k in ("dx", "dA", "dBm"):
        torch.testing.assert_close(a[k].float(), b[k].float(), rtol=2 ** -7, atol=1e-5)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows", [1, 3, 4, 7, 130])
@pytest.mark.parametrize("D,G,N,strided", [(16, 1, 16, False), (18, 2, 5, True), (8, 1, 1, False), (40, 1, 128, True),
                                           (22, 2, 32, True), (9, 3, 20, False), (5, 1, 8, False)])
def test_scan_step(D, G, N, strided, rows, dtype):
    sp, kw, p, o, _, _ = scan_case([1] * rows, False, D, G, N, dtype, seed=N, strided=strided)
    P, O = {k: dev(v) for k, v in p.items()}, {k: dev(v) for k, v in o.items()}
    state = O.pop("state0")
    out = kla.ssm_step(P["x"], P["dt"], P["A"], P["Bm"], P["Cm"], state, **O)
    want = want_scan(sp, p, o, None, None)
    check({"out": out, "final": state}, want, {"out": "out", "final": "final"})


def test_scan_prompt_then_steps_follow_the_whole():
    B, T, D, N = 3, 140, 24, 16
    sp, kw, p, o, _, _ = scan_case([T] * B, False, D, 1, N, "fp32", seed=8)
    want = want_scan(sp, p, o, None, None)
    cut = lambda t, a, e: t.view(B, T, *t.shape[1:])[:, a:e].reshape(B * (e - a), *t.shape[1:]).cuda()  # noqa: E731
    tok = {**p, "z": o["z"]}
    A, Dk, bias = p["A"].cuda(), o["D"].cuda(), o["dt_bias"].cuda()
    part = lambda a, e: {k: cut(v, a, e) for k, v in tok.items() if k != "A"}  # noqa: E731
    first, state = kla.ssm_forward(**part(0, 131), A=A, D=Dk, dt_bias=bias, state0=o["state0"].cuda(),
                                   final_state=True, B=B, T=131)
    outs = [first.view(B, 131, D)]
    for t in range(131, T):
        q = part(t, t + 1)
        outs.append(kla.ssm_step(q["x"], q["dt"], A, q["Bm"], q["Cm"], state, D=Dk, z=q["z"], dt_bias=bias)[:, None])
    check({"out": torch.cat(outs, 1).reshape(B * T, D), "final": state}, want, {"out": "out", "final": "final"})


def test_many_steps_of_a_slow_state_do_not_drift():
    """A state of constant decay and input after 4000 steps, token by token and as one prompt: its decay's
    rounding (half a unit in the last place, at random) may add up to 4000 halves at worst, its bias not."""
    n, D, N = 4000, 8, 4
    step = torch.full((1, D), 2.0 ** -10)
    A = -torch.linspace(0.25, 2.0, D * N).view(D, N)
    one, x = torch.ones(1, 1, N), torch.ones(1, D)
    dec = torch.exp(step.double().t() * A.double())
    h = 1.0 + (2.0 ** -10 / (1 - dec) - 1.0) * (1 - dec ** n)       # from 1 to the fixed point
    state = torch.ones(1, D, N, device="cuda")
    args = [t.cuda() for t in (x, step, A, one, one)]
    for _ in range(n):
        kla.ssm_step(*args, state, softplus=False)
    long = [t.cuda().expand(n, *t.shape[1:]).contiguous() if i != 2 else t.cuda() for i, t in enumerate((x, step, A, one, one))]
    _, fin = kla.ssm_forward(*long, state0=torch.ones(1, D, N, device="cuda"), softplus=False, final_state=True, B=1, T=n)
    for got in (state, fin):
        err = ((got.cpu().double()[0] - h) / h).abs().max()
        assert err <= 4000 * 2.0 ** -25, float(err)


def test_gradients_follow_differences():
    """The scan's gradients against central differences of the fp64 reference along a random direction."""
    sp, kw, p, o, dout, dfin = scan_case([60, 25], True, 14, 2, 9, "fp32", seed=11)
    got = run_scan(p, o, kw, dout, dfin, saved=True)
    g = gen(12)
    names = {"x": "dx", "dt": "ddt", "A": "dA", "Bm": "dBm", "Cm": "dCm", "D": "dD", "z": "dz", "dt_bias": "ddt_bias",
             "state0": "dstate0"}
    allp = {**p, **o}

    def loss(q):
        r = want_scan(sp, {k: q[k] for k in p}, {k: q[k] for k in o}, None, None)
        return float((r["out"][0] * dout.double()).sum() + (r["final"][0] * dfin.double()).sum())

    for k, gk in names.items():
        v = torch.randn(allp[k].shape, generator=g, dtype=torch.float64)
        eps = 2.0 ** -17
        num = [(loss({**allp, k: allp[k].double() + s * e * v}) ) for e in (eps, eps / 2) for s in (1, -1)]
        d1, d2 = (num[0] - num[1]) / (2 * eps), (num[2] - num[3]) / eps
        want = (4 * d2 - d1) / 3
        terms = got[gk].double().cpu() * v
        # fp32 gradients: 2^-14 of the terms' magnitudes covers their chains; the differences' own error is far below
        assert abs(float(terms.sum()) - want) <= 2 ** -14 * float(terms.abs().sum()) + 1e-6, k


# ---- layer norm ------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 2), (5, 5), (37, 16), (300, 31), (65, 64), (1000, 128), (9, 129),
                                    (33, 260), (20, 1000), (7, 1001), (40, 2048), (6, 2050), (5, 4096), (3, 4104),
                                    (4, 5003), (3, 8192), (2, 8200), (3, 16384), (2, 16001)])
def test_layernorm(rows, D, dtype):
    g = gen(rows + D)
    t = DT[dtype]
    x = (3 * torch.randn(rows, D, generator=g) + 5).to(t)
    res = torch.randn(rows, D, generator=g).to(t)
    w, b = torch.randn(D, generator=g), torch.randn(D, generator=g)
    dout, dsum = torch.randn(rows, D, generator=g).to(t), torch.randn(rows, D, generator=g).to(t)
    out, total, mean, rstd = kla.layernorm_forward(x.cuda(), w.cuda(), b.cuda(), residual=res.cuda(), stats=True)
    s = (x.float() + res.float()).to(t)
    assert torch.equal(total.cpu(), s)
    want = ob.layernorm(s, w, b, dout=dout, dsum=dsum)
    check({"out": out, "mean": mean, "rstd": rstd}, want, {k: k for k in ("out", "mean", "rstd")})
    got = kla.layernorm_backward(total, dout.cuda(), mean, rstd, w.cuda(), dsum=dsum.cuda())
    check(got, want, {k: k for k in ("dx", "dweight", "dbias")})
    plain = kla.layernorm_forward(x.cuda())
    check({"out": plain}, ob.layernorm(x), {"out": "out"})


def test_layernorm_strided_rows_and_in_place():
    g = gen(0)
    wide = torch.randn(50, 300, generator=g)
    for off, D in ((4, 128), (3, 101)):
        x = wide[:, off:off + D]
        got = kla.layernorm_forward(dev(wide)[:, off:off + D])
        check({"out": got}, ob.layernorm(x), {"out": "out"})
    x, res = torch.randn(40, 256, generator=g).cuda(), torch.randn(40, 256, generator=g).cuda()
    want_out, want_sum = kla.layernorm_forward(x, residual=res)
    out, total = kla.layernorm_forward(x, residual=res, out=x, sum_out=res)
    assert out.data_ptr() == x.data_ptr() and torch.equal(out, want_out) and torch.equal(res, want_sum)


def test_layernorm_large_mean_and_constant_rows():
    x = torch.full((4, 512), 1000.0)
    x[1] += torch.linspace(-1, 1, 512)
    x[2, 7] = 1001.0
    out, mean, rstd = kla.layernorm_forward(x.cuda(), stats=True)
    check({"out": out, "mean": mean, "rstd": rstd}, ob.layernorm(x), {k: k for k in ("out", "mean", "rstd")})


# ---- how the calls behave ------------------------------------------------------------------------

def test_tokens_of_no_sequence_are_left_as_they_were():
    sp, kw, p, o, dout, dfin = scan_case([20, 33], True, 16, 1, 8, "fp32", seed=1, tail=9)
    n = p["x"].shape[0]
    out = torch.full((n, 16), 7.0, device="cuda")
    P, O = {k: dev(v) for k, v in p.items()}, {k: dev(v) for k, v in o.items()}
    # what lies behind the last sequence enters nothing, whatever it is
    for k in ("x", "dt", "Bm", "Cm"):
        P[k][53:] = float("nan")
    O["z"][53:] = float("nan")
    kla.ssm_forward(**P, **O, out=out, **kw)
    assert (out[53:] == 7).all()
    want = want_scan(sp, p, o, dout, dfin)
    ob.close(out[:53], *want["out"], "out")
    d = dev(dout)
    d[53:] = float("nan")
    g = kla.ssm_backward(P["x"], P["dt"], P["A"], P["Bm"], P["Cm"], d, **O, dfinal_state=dfin.cuda(), **kw)
    for k in ("dA", "dD", "ddt_bias", "dstate0"):
        ob.close(g[k], *want[k], k)
    for k in ("dx", "ddt", "dz", "dBm", "dCm"):
        ob.close(g[k][:53], *want[k], k)
    y = torch.full((n, 16), 7.0, device="cuda")
    w = torch.randn(16, 4, generator=gen(3)).cuda()
    kla.conv_forward(P["x"], w, out=y, **kw)
    assert (y[53:] == 7).all() and torch.isfinite(y).all()
    c = kla.conv_backward(P["x"], w, d, **kw)
    assert torch.isfinite(c["dweight"]).all() and torch.isfinite(c["dbias"]).all() and torch.isfinite(c["dx"][:53]).all()


def test_offsets_behind_the_axis_end_at_it():
    sp, kw, p, o, dout, dfin = scan_case([7, 23], True, 12, 1, 6, "fp32", seed=3)
    want = run_scan(p, o, kw, dout, dfin, saved=True)
    far = dict(cu_seqlens=torch.tensor([0, 7, 400], dtype=torch.int32, device="cuda"))
    got = run_scan(p, o, far, dout, dfin, saved=True)
    assert all(torch.equal(got[k], want[k]) for k in want)
    w = torch.randn(12, 4, generator=gen(4)).cuda()
    x, d = dev(p["x"]), dev(dout)
    a, b = (kla.conv_forward(x, w, final_state=True, **k) for k in (kw, far))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = (kla.conv_backward(x, w, d, **k) for k in (kw, far))
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_identical_inputs_give_identical_bits():
    sp, kw, p, o, dout, dfin = scan_case([400, 90], True, 48, 1, 16, "bf16", seed=6)
    a, b = (run_scan(p, o, kw, dout, dfin, saved=True) for _ in range(2))
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_no_tokens_give_zero_gradients_and_pass_states():
    f = dict(device="cuda")
    x, w = torch.empty(0, 8, **f), torch.randn(8, 4, **f)
    s0, dfin = torch.randn(3, 3, 8, **f), torch.randn(3, 3, 8, **f)
    out, fin = kla.conv_forward(x, w, state0=s0, final_state=True, B=3, T=0)
    assert out.shape == (0, 8) and torch.equal(fin, s0)
    g = kla.conv_backward(x, w, x, state0=s0, dfinal_state=dfin, B=3, T=0)
    assert torch.equal(g["dstate0"], dfin) and not g["dweight"].any() and not g["dbias"].any()
    A, bc, h0 = -torch.rand(8, 4, **f), torch.empty(0, 1, 4, **f), torch.randn(3, 8, 4, **f)
    out, fin = kla.ssm_forward(x, x, A, bc, bc, state0=h0, final_state=True, B=3, T=0)
    assert torch.equal(fin, h0)
    g = kla.ssm_backward(x, x, A, bc, bc, x, state0=h0, dfinal_state=h0, B=3, T=0)
    assert torch.equal(g["dstate0"], h0) and not g["dA"].any() and not g["dD"].any()
    g = kla.layernorm_backward(x, x, torch.empty(0, **f), torch.empty(0, **f))
    assert not g["dweight"].any() and not g["dbias"].any()


def block_step(x, w, kw):
    """A pre-norm block: norm of the residual sum, input projection, convolution, the projections of dt, B and C,
    scan, output projection; and its gradients."""
    ln, total, mean, rstd = kla.layernorm_forward(x, w["lw"], w["lb"], residual=w["res"], stats=True)
    xz = ln @ w["win"]
    D = w["A"].shape[0]
    N = w["A"].shape[1]
    u = kla.conv_forward(xz[:, :D], w["cw"], w["cb"], **kw)
    proj = u @ w["wbc"]
    dt = proj[:, 2 * N:] @ w["wdt"]
    bc = lambda v: (v[:, :N].unflatten(1, (1, N)), v[:, N:2 * N].unflatten(1, (1, N)))  # noqa: E731
    Bm, Cm = bc(proj)
    more = dict(D=w["Dk"], z=xz[:, D:], dt_bias=w["bias"], **kw)
    y, st = kla.ssm_forward(u, dt, w["A"], Bm, Cm, save_states=True, **more)
    out = total + y @ w["wout"]
    dout = w["dout"]
    dy = dout @ w["wout"].t()
    g = kla.ssm_backward(u, dt, w["A"], Bm, Cm, dy, states=st, **more)
    dproj = torch.cat([g["dBm"].flatten(1), g["dCm"].flatten(1), g["ddt"] @ w["wdt"].t()], 1)
    du = g["dx"] + dproj @ w["wbc"].t()
    c = kla.conv_backward(xz[:, :D], w["cw"], du, w["cb"], **kw)
    dln = torch.cat([c["dx"], g["dz"]], 1) @ w["win"].t()
    n = kla.layernorm_backward(total, dln, mean, rstd, w["lw"], dsum=dout)
    return {"out": out, "dx": n["dx"], "dlw": n["dweight"], "dcw": c["dweight"], "dA": g["dA"], "dbias": g["ddt_bias"]}


def block_weights(n, M, D, N, R, seed=0):
    g = gen(seed)
    r = lambda *s, sc=1.0: (sc * torch.randn(*s, generator=g))  # noqa: E731
    step = 0.01 + 0.1 * torch.rand(D, generator=g)
    return r(n, M), dict(
        lw=1 + r(M, sc=0.1), lb=r(M, sc=0.1), res=r(n, M), win=r(M, 2 * D, sc=M ** -0.5), cw=r(D, 4, sc=0.5),
        cb=r(D, sc=0.1), wbc=r(D, 2 * N + R, sc=D ** -0.5), wdt=r(R, D, sc=R ** -0.5),
        A=-torch.arange(1, N + 1).float().repeat(D, 1), Dk=torch.ones(D), bias=step + torch.log(-torch.expm1(-step)),
        wout=r(D, M, sc=D ** -0.5), dout=r(n, M))


def block_reference(x, w, sp):
    """The same block in fp64 with automatic differentiation."""
    w = {k: v.double().requires_grad_(k != "dout") for k, v in w.items()}
    x = x.double().requires_grad_()
    total = x + w["res"]
    mu = total.mean(1, keepdim=True)
    ln = (total - mu) * (((total - mu) ** 2).mean(1, keepdim=True) + 1e-5).rsqrt() * w["lw"] + w["lb"]
    xz = ln @ w["win"]
    D, N = w["A"].shape
    s0 = torch.zeros(len(sp), 3, D, dtype=torch.float64)
    u, _ = ob._conv_rows(xz[:, :D], w["cw"], w["cb"], s0, sp, True)
    proj = u @ w["wbc"]
    step = torch.nn.functional.softplus(proj[:, 2 * N:] @ w["wdt"] + w["bias"])
    y, _, _ = ob._scan_rows(u, step, step, w["A"], proj[:, None, :N], proj[:, None, N:2 * N], w["Dk"],
                            ob._silu(xz[:, D:]), torch.zeros(len(sp), D, N, dtype=torch.float64), sp)
    out = total + y @ w["wout"]
    names = ("lw", "cw", "A", "bias")
    gr = torch.autograd.grad(out, [x] + [w[k] for k in names], w["dout"])
    return {"out": out.detach(), "dx": gr[0], **{"d" + k: v for k, v in zip(names, gr[1:])}}


def test_block_forward_and_gradients():
    lens = [90, 1, 47]
    sp, kw, n = axis(lens, True)
    x, w = block_weights(n, 32, 48, 8, 4)
    was = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        got = block_step(x.cuda(), {k: v.cuda() for k, v in w.items()}, kw)
    finally:
        torch.backends.cuda.matmul.allow_tf32 = was
    want = block_reference(x, w, sp)
    for k, v in want.items():
        # chains of some hundred fp32 roundings over values of this size
        err = (got[k].double().cpu() - v).abs().max() / v.abs().max()
        assert err <= 2.0 ** -24 * 512, (k, float(err))


def test_captured_and_replayed_on_another_stream():
    lens = [200, 64]
    sp, kw, n = axis(lens, True)
    x, w = block_weights(n, 32, 48, 8, 4, seed=1)
    X, W = x.cuda(), {k: v.cuda() for k, v in w.items()}
    want = block_step(X, W, kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        block_step(X, W, kw)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            got = block_step(X, W, kw)
    x2 = torch.randn(n, 32, generator=gen(9)).cuda()
    want2 = block_step(x2, W, kw)
    torch.cuda.synchronize()
    for src, exp in ((x2, want2), (x.cuda(), want), (x2, want2)):
        X.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for k in exp:
            torch.testing.assert_close(got[k], exp[k], rtol=1e-5, atol=1e-5)


def test_two_streams_at_once():
    cases = [scan_case([500, 77], True, 64, 1, 16, "bf16", seed=s) for s in (1, 2)]
    want = [run_scan(p, o, kw, dout, dfin, saved=True) for sp, kw, p, o, dout, dfin in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, (st, (sp, kw, p, o, dout, dfin)) in enumerate(zip(streams, cases)):
            with torch.cuda.stream(st):
                got[i] = run_scan(p, o, kw, dout, dfin, saved=True)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_refusals_of_the_binding():
    f = dict(device="cuda")
    x, w = torch.randn(10, 8, **f), torch.randn(8, 4, **f)
    with pytest.raises(ValueError):
        kla.conv_forward(x.t(), w)
    with pytest.raises(TypeError):
        kla.conv_forward(x.half(), w)
    with pytest.raises(ValueError):
        kla.conv_forward(x, torch.randn(8, 5, **f))
    with pytest.raises(ValueError):
        kla.conv_forward(x, w, B=3, T=3)
    with pytest.raises(ValueError):
        kla.conv_forward(x, w, state0=torch.zeros(1, 3, 9, **f))
    with pytest.raises(TypeError):
        kla.conv_forward(x, w, cu_seqlens=torch.tensor([0, 10], **f))
    with pytest.raises(ValueError):
        kla.conv_forward(x, w, cu_seqlens=torch.tensor([0, 10], dtype=torch.int32, **f), B=1, T=10)
    with pytest.raises(ValueError):
        kla.conv_forward(x.expand(10, 8)[:1].expand(10, 8), w)
    with pytest.raises(kla.KlaError):
        kla.conv_forward(x, w, out=x)
    A, bc = -torch.rand(8, 4, **f), torch.randn(10, 1, 4, **f)
    with pytest.raises(ValueError):
        kla.ssm_forward(x, x, A, torch.randn(10, 3, 4, **f), bc)
    with pytest.raises(ValueError):
        kla.ssm_forward(x, x, A.cpu(), bc, bc)
    with pytest.raises(TypeError):
        kla.ssm_forward(x, x.bfloat16(), A, bc, bc)
    with pytest.raises(kla.KlaError) as e:
        kla.ssm_forward(x, x, -torch.rand(8, 129, **f), torch.randn(10, 1, 129, **f), torch.randn(10, 1, 129, **f))
    assert e.value.status == kla.KLA_ERR_UNSUPPORTED
    with pytest.raises(kla.KlaError):
        kla.ssm_forward(x, x, A, bc, bc, out=x)
    with pytest.raises(ValueError):
        kla.ssm_backward(x, x, A, bc, bc, x, states=torch.zeros(3, **f))
    with pytest.raises(ValueError):
        kla.ssm_backward(x, x, A, bc, bc, x, workspace=torch.zeros(3, dtype=torch.uint8, **f))
    with pytest.raises(kla.KlaError):
        kla.layernorm_forward(x, eps=0.0)
    with pytest.raises(kla.KlaError):
        kla.layernorm_forward(torch.randn(2, 16385, **f))
    with pytest.raises(ValueError):
        kla.layernorm_forward(x, sum_out=torch.empty_like(x))
    torch.cuda.synchronize()
    kla.check()
