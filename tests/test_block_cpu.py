"""The recurrent block without a GPU: refusals of the C entry points before any
launch, workspace sizes, and the references' gradients against differences."""
import ctypes

import pytest
import torch

from bayesian_filter_scan_b200 import build as kbuild
from bayesian_filter_scan_b200 import kla
from oracle import block as ob

BAD, UNSUP = kla.KLA_ERR_INVALID_ARG, kla.KLA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kla.lib()


def ptrs(n, gap=1 << 24):
    """Addresses far enough apart that no two tensors of these calls overlap; never used."""
    return [gap * (i + 1) for i in range(n)]


def conv_desc(**kw):
    d = dict(B=2, T=40, D=64, W=4, dtype=kla.KLA_BF16, silu=1, cu_seqlens=None, num_seqs=0, ld_x=0)
    d.update(kw)
    return kla.KlaConvDesc(*d.values())


def ssm_desc(**kw):
    d = dict(B=2, T=40, D=64, G=2, N=16, dtype=kla.KLA_BF16, softplus=1, cu_seqlens=None, num_seqs=0, ld_x=0, ld_dt=0,
             ld_z=0, ld_b=0, ld_c=0)
    d.update(kw)
    return kla.KlaSsmDesc(*d.values())


def norm_desc(**kw):
    d = dict(rows=10, D=64, dtype=kla.KLA_BF16, eps=1e-5, ld_x=0, ld_residual=0)
    d.update(kw)
    return kla.KlaNormDesc(*d.values())


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), BAD), (dict(T=-1), BAD), (dict(D=0), BAD), (dict(W=0), BAD), (dict(W=5), BAD), (dict(dtype=9), BAD),
    (dict(ld_x=63), BAD), (dict(ld_x=-64), BAD), (dict(cu_seqlens=4096, num_seqs=0), BAD), (dict(D=(1 << 20) + 1), UNSUP)])
def test_conv_descriptors_are_refused(L, bad, status):
    d = ctypes.byref(conv_desc(**bad))
    assert L.kla_conv_forward(d, *ptrs(6), None) == status
    assert L.kla_conv_backward(d, *ptrs(11), 1 << 30, None) == status
    assert L.kla_conv_backward_workspace_bytes(d) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), BAD), (dict(D=0), BAD), (dict(G=0), BAD), (dict(G=3), BAD), (dict(N=0), BAD), (dict(N=129), UNSUP),
    (dict(dtype=9), BAD), (dict(ld_x=63), BAD), (dict(ld_dt=1), BAD), (dict(ld_z=63), BAD), (dict(ld_b=31), BAD),
    (dict(ld_c=31), BAD), (dict(cu_seqlens=4096, num_seqs=0), BAD)])
def test_ssm_descriptors_are_refused(L, bad, status):
    d = ctypes.byref(ssm_desc(**bad))
    assert L.kla_ssm_forward(d, *ptrs(12), None) == status
    assert L.kla_ssm_backward(d, *ptrs(22), 1 << 30, None) == status
    assert L.kla_ssm_states_bytes(d) == 0 and L.kla_ssm_backward_workspace_bytes(d, 1) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(rows=-1), BAD), (dict(D=0), BAD), (dict(D=16385), UNSUP), (dict(eps=0.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(dtype=9), BAD), (dict(ld_x=63), BAD), (dict(ld_residual=63), BAD)])
def test_norm_descriptors_are_refused(L, bad, status):
    d = ctypes.byref(norm_desc(**bad))
    assert L.kla_layernorm_forward(d, *ptrs(8), None) == status
    assert L.kla_layernorm_backward(d, *ptrs(10), 1 << 30, None) == status


def test_missing_misaligned_and_overlapping_buffers_are_refused(L):
    fwd = lambda p, d=None: L.kla_ssm_forward(ctypes.byref(d or ssm_desc()), *p, None)  # noqa: E731
    for i in (0, 1, 2, 3, 4, 9):            # x, dt, A, Bm, Cm, out
        p = ptrs(12)
        p[i] = None
        assert fwd(p) == BAD
    for i, off in ((0, 1), (2, 2), (8, 2), (10, 1), (11, 8)):
        p = ptrs(12)
        p[i] += off
        assert fwd(p) == BAD
    p = ptrs(12)
    p[9] = p[0]                             # out over x
    assert fwd(p) == BAD
    p = ptrs(12)
    p[10] = p[8] + 16                       # final_state over state0
    assert fwd(p) == BAD
    # a workspace too small, gradients over inputs, dz without z
    need = L.kla_ssm_backward_workspace_bytes(ctypes.byref(ssm_desc()), 1)
    assert need < L.kla_ssm_backward_workspace_bytes(ctypes.byref(ssm_desc()), 0)
    bwd = lambda p, n=need: L.kla_ssm_backward(ctypes.byref(ssm_desc()), *p, n, None)  # noqa: E731
    assert bwd(ptrs(22), need - 1) == BAD
    p = ptrs(22)
    p[12] = p[0]
    assert bwd(p) == BAD
    p = ptrs(22)
    p[6] = None
    assert bwd(p) == BAD
    c = conv_desc()
    p = ptrs(6)
    p[4] = p[0] + 64
    assert L.kla_conv_forward(ctypes.byref(c), *p, None) == BAD
    need = L.kla_conv_backward_workspace_bytes(ctypes.byref(c))
    assert L.kla_conv_backward(ctypes.byref(c), *ptrs(11), need - 1, None) == BAD
    n = norm_desc()
    p = ptrs(8)
    p[1] = None                             # a sum without a residual
    assert L.kla_layernorm_forward(ctypes.byref(n), *p, None) == BAD
    p = ptrs(8)
    p[4] = p[0] + 2                         # out over x, shifted
    assert L.kla_layernorm_forward(ctypes.byref(n), *p, None) == BAD
    p = ptrs(8)
    p[4] = p[0]                             # in place, but x's rows are strided
    assert L.kla_layernorm_forward(ctypes.byref(norm_desc(ld_x=128)), *p, None) == BAD
    p = ptrs(8)
    p[4] = p[5] = p[0]                      # out and sum in one place
    assert L.kla_layernorm_forward(ctypes.byref(n), *p, None) == BAD


def test_steps_take_one_token_per_row(L):
    assert L.kla_conv_step(ctypes.byref(conv_desc(T=2)), *ptrs(5), None) == BAD
    assert L.kla_conv_step(ctypes.byref(conv_desc(T=1, cu_seqlens=4096, num_seqs=2)), *ptrs(5), None) == BAD
    assert L.kla_ssm_step(ctypes.byref(ssm_desc(T=2)), *ptrs(10), None) == BAD
    for f, d, n in ((L.kla_conv_step, conv_desc(T=1), 5), (L.kla_ssm_step, ssm_desc(T=1), 10)):
        p = ptrs(n)
        p[n - 1] = p[n - 2]                 # out over the state
        assert f(ctypes.byref(d), *p, None) == BAD
        p = ptrs(n)
        p[n - 2] = None
        assert f(ctypes.byref(d), *p, None) == BAD


def test_null_descriptors(L):
    assert L.kla_conv_forward(None, *ptrs(6), None) == BAD
    assert L.kla_ssm_forward(None, *ptrs(12), None) == BAD
    assert L.kla_layernorm_forward(None, *ptrs(8), None) == BAD
    assert L.kla_ssm_states_bytes(None) == 0 and L.kla_layernorm_backward_workspace_bytes(None) == 0


def test_state_records_cover_every_sequence():
    # record k of sequence n sits at s0 // 16 + n + k: no two sequences share one
    g = torch.Generator().manual_seed(0)
    for _ in range(200):
        lens = torch.randint(0, 400, (int(torch.randint(1, 9, (1,), generator=g)),), generator=g).tolist()
        used, s0 = set(), 0
        for n, m in enumerate(lens):
            for k in range(-(-m // 16)):
                i = s0 // 16 + n + k
                assert i not in used
                used.add(i)
            s0 += m
        assert not used or max(used) < s0 // 16 + len(lens) + 1


def test_cpu_tensors_are_refused(L):
    x, w = torch.randn(4, 8), torch.randn(8, 4)
    with pytest.raises(ValueError):
        kla.conv_forward(x, w)
    with pytest.raises(ValueError):
        kla.ssm_forward(x, x, -torch.rand(8, 4), torch.randn(4, 1, 4), torch.randn(4, 1, 4))
    with pytest.raises(ValueError):
        kla.layernorm_forward(x)


def _differences(f, t, eps=2.0 ** -14):
    """Central differences of the scalar f at every entry of t, extrapolated."""
    out = torch.zeros_like(t)
    flat, o = t.view(-1), out.view(-1)
    for i in range(flat.numel()):
        v = float(flat[i])
        d = []
        for e in (eps, eps / 2):
            flat[i] = v + e
            hi = f()
            flat[i] = v - e
            d.append((hi - f()) / (2 * e))
        flat[i] = v
        o[i] = (4 * d[1] - d[0]) / 3
    return out


def test_reference_gradients_equal_differences():
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    sp = [(0, 5), (5, 5), (5, 8)]
    x, w, b, s0 = r(8, 3), r(3, 4), r(3), r(3, 3, 3)
    do, df = r(8, 3), r(3, 3, 3)
    want = ob.conv(x, w, b, s0, sp, True, do, df)
    f = lambda: float(sum((a * c).sum() for a, c in zip(ob._conv_rows(x, w, b, s0, sp, True), (do, df))))  # noqa: E731
    for name, t in (("dx", x), ("dweight", w), ("dbias", b), ("dstate0", s0)):
        torch.testing.assert_close(want[name][0], _differences(f, t), rtol=1e-7, atol=1e-8)
    p = dict(x=r(8, 4), dt=r(8, 4), A=-r(4, 2).abs(), Bm=r(8, 2, 2), Cm=r(8, 2, 2))
    o = dict(Dskip=r(4), z=r(8, 4), dt_bias=r(4), h0=r(3, 4, 2))
    do, df = r(8, 4), r(3, 4, 2)
    want = ob.scan(**p, sp=sp, **o, dout=do, dfinal=df)

    def f():
        q = ob.scan(**p, sp=sp, **o)
        return float((q["out"][0] * do).sum() + (q["final"][0] * df).sum())

    for name, t in (("dx", p["x"]), ("ddt", p["dt"]), ("dA", p["A"]), ("dBm", p["Bm"]), ("dCm", p["Cm"]),
                    ("dD", o["Dskip"]), ("dz", o["z"]), ("ddt_bias", o["dt_bias"]), ("dstate0", o["h0"])):
        torch.testing.assert_close(want[name][0], _differences(f, t), rtol=1e-7, atol=1e-8)
    x, w, b, do = r(3, 5), r(5), r(5), r(3, 5)
    want = ob.layernorm(x, w, b, dout=do)
    f = lambda: float((ob.layernorm(x, w, b)["out"][0] * do).sum())  # noqa: E731
    for name, t in (("dx", x), ("dweight", w), ("dbias", b)):
        torch.testing.assert_close(want[name][0], _differences(f, t), rtol=1e-7, atol=1e-8)


def test_scan_reference_on_a_worked_case():
    # one channel, one state, no decay and unit steps: the state is a running sum
    x = torch.tensor([[1.0], [2.0], [4.0]])
    one = torch.ones(3, 1, 1)
    got = ob.scan(x, torch.ones(3, 1), torch.zeros(1, 1), one, one, [(0, 3)], softplus=False)
    assert got["out"][0].flatten().tolist() == [1.0, 3.0, 7.0]
    # halving each step
    A = torch.full((1, 1), -0.6931471805599453, dtype=torch.float64)
    got = ob.scan(x, torch.ones(3, 1), A, one, one, [(0, 3)], softplus=False)
    assert torch.allclose(got["out"][0].flatten(), torch.tensor([1.0, 2.5, 5.25], dtype=torch.float64))
