"""What the slacks of the scan's reference let through: a plain fp32 evaluation, and
neither states of 13 bits, nor results a thousandth off, nor gradients that lose a
term. On the shapes of the GPU's tests, on the CPU."""
import pytest
import torch

from oracle import block as ob

CASES = [
    ([15, 15], 16, 1, 16), ([17], 5, 1, 1), ([128, 128], 24, 2, 8), ([129], 16, 1, 20), ([300], 33, 3, 5),
    ([1, 0, 2, 140, 0, 3], 18, 1, 16), ([257, 300], 20, 2, 33), ([40], 16, 1, 128), ([600], 8, 1, 3)]


def case(lens, D, G, N):
    g = torch.Generator().manual_seed(D + N)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    n = sum(lens)
    cu = torch.tensor([0] + lens).cumsum(0)
    step = 0.001 * 300 ** torch.rand(D, generator=g)
    p = dict(x=r(n, D), dt=0.5 * r(n, D), A=-(0.5 + torch.rand(D, N, generator=g) * N), Bm=r(n, G, N), Cm=r(n, G, N),
             Dskip=r(D), z=r(n, D), dt_bias=step + torch.log(-torch.expm1(-step)), h0=r(len(lens), D, N))
    return ob.spans(0, cu=cu), p, r(n, D), r(len(lens), D, N)


def evaluate(p, sp, dout, dfin, bits=24):
    """The scan and its gradients in fp32, token by token; the state keeps `bits` bits."""
    q = {k: v.clone().requires_grad_() for k, v in p.items()}

    def cut(h):
        if bits == 24:
            return h
        m, e = torch.frexp(h.detach())
        return h + (torch.ldexp(torch.round(m * 2.0 ** bits), e - bits) - h.detach())

    raw = q["dt"] + q["dt_bias"]
    step = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    rep = p["A"].shape[0] // p["Bm"].shape[1]
    B, C = (q[k].repeat_interleave(rep, 1) for k in ("Bm", "Cm"))
    outs, fin = [], []
    for n, (a, e) in enumerate(sp):
        h = q["h0"][n]
        for t in range(a, e):
            h = cut(torch.exp(step[t][:, None] * q["A"]) * h + (step[t] * q["x"][t])[:, None] * B[t])
            y = (C[t] * h).sum(-1) + q["Dskip"] * q["x"][t]
            outs.append(y * (q["z"][t] * torch.sigmoid(q["z"][t])))
        fin.append(h)
    out, fin = torch.stack(outs), torch.stack(fin)
    names = dict(x="dx", dt="ddt", A="dA", Bm="dBm", Cm="dCm", Dskip="dD", z="dz", dt_bias="ddt_bias", h0="dstate0")
    grads = torch.autograd.grad([out, fin], [q[k] for k in names], [dout, dfin])
    return {"out": out.detach(), "final": fin.detach(), **dict(zip(names.values(), grads))}


def passes(got, want):
    try:
        ob.close(got, *want, "")
    except AssertionError:
        return False
    return True


@pytest.mark.parametrize("lens,D,G,N", CASES)
def test_slack_of_the_scan(lens, D, G, N):
    sp, p, dout, dfin = case(lens, D, G, N)
    want = ob.scan(**p, sp=sp, dout=dout, dfinal=dfin)
    got = evaluate(p, sp, dout, dfin)
    for k in want:
        assert passes(got[k], want[k]), k
        assert not passes(got[k] * 0.999, want[k]), k
    short = evaluate(p, sp, dout, dfin, bits=13)
    for k in ("out", "final", "dCm", "dA"):
        assert not passes(short[k], want[k]), k
    # half of the step's gradient lost, or the last token's share of a sum over tokens
    for k in ("ddt", "ddt_bias"):
        assert not passes(got[k] * 0.5, want[k]), k
    last = sp[-1][1] - 1
    assert not passes(got["ddt_bias"] - got["ddt"][last], want["ddt_bias"])
