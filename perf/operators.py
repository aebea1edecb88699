"""The recurrent block's operators, as cases to be timed and compared.

Short causal convolution, selective state space scan (prompts, gradients,
single tokens) and layer norm (forward, gradients). With ``own`` false every
operator runs in its plain form (elementary torch operations in fp32); with
``own`` true through this package's entry points.

A case names its operator in ``op``:
  conv        prompt through the convolution, history out
  conv_train  convolution forward and gradients
  scan        prompt through the scan, state out
  scan_train  scan forward and gradients
  step        one token per row: convolution step, then scan step, states in place
  norm        layer norm of a residual sum
  norm_train  layer norm forward and gradients
Tokens of all sequences lie on one axis; ``seqs`` > 0 packs that many sequences
of uneven lengths, otherwise there are ``B`` rows of ``T`` tokens.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_CAP = 131072 * 2048 * 16      # token x channel x state of the largest listed scan


def listed():
    return [
        # a packed batch of prompts entering a 2048-channel layer, with the history kept for decoding
        {"name": "conv_packed", "op": "conv", "B": 1, "T": 32768, "seqs": 9, "D": 2048, "W": 4, "dtype": "bf16"},
        # a training microbatch of odd sizes: no row starts on a vector boundary
        {"name": "conv_train_odd", "op": "conv_train", "B": 3, "T": 1777, "seqs": 0, "D": 1001, "W": 4, "dtype": "bf16"},
        # a short prompt of one user: latency
        {"name": "scan_short", "op": "scan", "B": 1, "T": 48, "seqs": 0, "D": 512, "G": 1, "N": 16, "gate": True,
         "dtype": "bf16"},
        # the 1.3B-class layer of this repository's workloads: 8 rows of 4096 tokens
        {"name": "scan_layer", "op": "scan", "B": 8, "T": 4096, "seqs": 0, "D": 2048, "G": 1, "N": 16, "gate": True,
         "dtype": "bf16"},
        # one 128k-token document
        {"name": "scan_long", "op": "scan", "B": 1, "T": 131072, "seqs": 0, "D": 2048, "G": 1, "N": 16, "gate": True,
         "dtype": "bf16"},
        # packed prompts in fp32, two groups of B and C, a state size that is no power of two
        {"name": "scan_packed_fp32", "op": "scan", "B": 1, "T": 9001, "seqs": 7, "D": 1030, "G": 2, "N": 24,
         "gate": False, "dtype": "fp32"},
        # a training microbatch of the 2048-channel layer
        {"name": "scan_train", "op": "scan_train", "B": 4, "T": 2048, "seqs": 0, "D": 2048, "G": 1, "N": 16,
         "gate": True, "dtype": "bf16"},
        # training in fp32 with four groups, a wide state and ragged packed sequences
        {"name": "scan_train_groups", "op": "scan_train", "B": 1, "T": 1403, "seqs": 3, "D": 520, "G": 4, "N": 64,
         "gate": True, "dtype": "fp32"},
        # decoding for one user
        {"name": "step_one", "op": "step", "B": 1, "D": 2048, "W": 4, "G": 1, "N": 16, "dtype": "bf16"},
        # decoding for a full batch in a wide layer
        {"name": "step_batch", "op": "step", "B": 256, "D": 4096, "W": 4, "G": 1, "N": 16, "dtype": "bf16"},
        # the norm before a layer, with the residual sum, over a long prefill
        {"name": "norm_residual", "op": "norm", "rows": 32768, "D": 2048, "dtype": "bf16"},
        # training: the norm of every head's output (8 x 4096 tokens, 16 heads of 128)
        {"name": "norm_train_heads", "op": "norm_train", "rows": 524288, "D": 128, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_train", "scan", "scan", "scan_train", "scan_train", "step", "norm", "norm_train"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op in ("norm", "norm_train"):
        c["D"] = _log(rng, 16, 8192)
        c["rows"] = _log(rng, 1, max(2, min(1 << 20, (1 << 26) // c["D"])))
        return c
    if op == "step":
        c.update(B=_log(rng, 1, 256), D=_log(rng, 64, 4096), W=rng.choice([2, 3, 4]), G=1, N=rng.choice([8, 16, 32, 64]))
        if rng.random() < 0.3:
            c["G"] = 2
            c["D"] += c["D"] % 2
        return c
    c["B"], c["seqs"] = rng.choice([(1, 0), (2, 0), (4, 0), (1, rng.randint(2, 12))])
    c["T"] = max(c["seqs"], _log(rng, 16, 16384))
    c["D"] = _log(rng, 64, 4096)
    if op in ("conv", "conv_train"):
        c["W"] = rng.choice([2, 3, 4])
        return c
    c["G"] = rng.choice([1, 1, 2])
    c["D"] += c["D"] % c["G"]
    c["N"] = rng.choice([8, 16, 16, 20, 32, 64])
    c["gate"] = rng.random() < 0.7
    cap = _CAP // (32 if op == "scan_train" else 8)
    c["T"] = max(c["seqs"], 1, min(c["T"], cap // (c["B"] * c["D"] * c["N"])))
    return c


# ---- inputs -----------------------------------------------------------------

def _lengths(c, g):
    """Lengths of the packed sequences: uneven, at least one token each."""
    n, total = c["seqs"], c["T"]
    w = torch.rand(n, generator=g) + 0.05
    cuts = torch.cumsum(w / w.sum() * (total - n), 0).floor().to(torch.int64) + torch.arange(1, n + 1)
    cuts[-1] = total
    return torch.cat([torch.zeros(1, dtype=torch.int64), cuts])


def _offsets(c, seed):
    if c.get("seqs"):
        return _lengths(c, torch.Generator().manual_seed(seed)).tolist()
    return [i * c["T"] for i in range(c["B"] + 1)]


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DT[c["dtype"]]
    f32 = dict(generator=g, device=dev)
    s = {"c": c}

    def normal(*shape, scale=1.0, mean=0.0):
        return torch.randn(*shape, **f32).mul_(scale).add_(mean)

    if c["op"] in ("norm", "norm_train"):
        R, D = c["rows"], c["D"]
        s["x"] = normal(R, D, mean=0.3).to(dt)
        s["w"], s["b"] = normal(D, scale=0.1, mean=1.0), normal(D, scale=0.1)
        if c["op"] == "norm":
            s["res"] = normal(R, D, scale=2.0).to(dt)
        else:
            s["dout"] = normal(R, D).to(dt)
        return s

    D = c["D"]
    if c["op"] == "step":
        Ntok = c["B"]
    else:
        s["off"] = _offsets(c, seed)
        Ntok = s["off"][-1]
        lens = [b - a for a, b in zip(s["off"], s["off"][1:])]
        s["maxlen"] = max(lens)
        if c["seqs"]:
            s["cu"] = torch.tensor(s["off"], dtype=torch.int32, device=dev)
        start = torch.tensor(s["off"][:-1], device=dev)
        length = torch.tensor(lens, device=dev)
        seq = torch.repeat_interleave(torch.arange(len(lens), device=dev), length)
        # where every token stands: its sequence, its position there, its sequence's length and the sequences' starts
        s["seq"], s["pos"], s["len"] = seq, torch.arange(Ntok, device=dev) - start[seq], length[seq]
        s["start"], s["last"] = start, start + length - 1
    if c["op"] in ("conv", "conv_train", "step"):
        # the layer's input projection gives x and z side by side
        s["xz"] = normal(Ntok, 2 * D).to(dt)
        s["x"] = s["xz"][:, :D]
        s["w"] = normal(D, c["W"], scale=1.0 / math.sqrt(c["W"]))
        s["bias"] = normal(D, scale=0.1)
        if c["op"] == "conv_train":
            s["dout"] = normal(Ntok, D).to(dt)
        if c["op"] == "step":
            s["hist"] = normal(Ntok, c["W"] - 1, D).to(dt)
    if c["op"] in ("scan", "scan_train", "step"):
        G, N = c["G"], c["N"]
        if c["op"] != "step":
            s["x"] = torch.nn.functional.silu(normal(Ntok, D)).to(dt)
            if c["gate"]:
                s["z"] = normal(Ntok, 2 * D).to(dt)[:, D:]
        else:
            s["z"] = s["xz"][:, D:]
        # steps between 0.001 and 0.1 around which dt moves; decays -1..-N with some spread
        step = torch.exp(torch.rand(D, **f32) * math.log(100.0) + math.log(0.001))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["dt"] = normal(Ntok, D, scale=0.5).to(dt)
        s["A"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32) * torch.exp(normal(D, N, scale=0.1))
        # B and C are columns of one projection, behind the low-rank part of dt
        R = max(1, D // 16)
        proj = normal(Ntok, R + 2 * G * N).to(dt)
        s["Bm"] = proj[:, R:R + G * N].unflatten(1, (G, N))
        s["Cm"] = proj[:, R + G * N:].unflatten(1, (G, N))
        s["Dskip"] = normal(D, scale=0.1, mean=1.0)
        if c["op"] == "step":
            s["h"] = normal(Ntok, D, N)
        elif c["op"] == "scan" and c["seqs"]:
            s["h0"] = normal(c["seqs"], D, N)    # prompts that continue earlier ones
        if c["op"] == "scan_train":
            s["dout"] = normal(Ntok, D).to(dt)
    return s


# ---- plain forms (fp32, elementary operations) ---------------------------------

def _silu(x):
    return x / (1 + torch.exp(-x))


def _dsilu(x):
    g = 1 / (1 + torch.exp(-x))
    return g * (1 + x * (1 - g))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _back(v, pos, k):
    """v of the token k places earlier in the same sequence, 0 before its start."""
    if k == 0:
        return v
    out = torch.zeros_like(v)
    out[k:] = v[:-k]
    return out * (pos >= k)[:, None]


def _ahead(v, left, k):
    """v of the token k places later in the same sequence, 0 behind its end (left: tokens behind this one)."""
    if k == 0:
        return v
    out = torch.zeros_like(v)
    out[:-k] = v[k:]
    return out * (left >= k)[:, None]


def _conv_pre(s):
    W, x = s["c"]["W"], s["x"].float()
    return sum(_back(x, s["pos"], j) * s["w"][:, W - 1 - j] for j in range(W)) + s["bias"]


def _conv_plain(s):
    c, dt = s["c"], s["x"].dtype
    y = _silu(_conv_pre(s)).to(dt)
    # the last W-1 inputs of every sequence, zeros where it is shorter
    p = s["last"][:, None] - torch.arange(c["W"] - 2, -1, -1, device=y.device)
    hist = torch.where((p >= s["start"][:, None])[..., None], s["x"][p.clamp(min=0)], torch.zeros((), dtype=dt, device=y.device))
    return {"out": y, "hist": hist}


def _conv_train_plain(s):
    W, dt, pre = s["c"]["W"], s["x"].dtype, _conv_pre(s)
    x, d = s["x"].float(), s["dout"].float() * _dsilu(pre)
    left = s["len"] - 1 - s["pos"]
    dx = sum(_ahead(d, left, j) * s["w"][:, W - 1 - j] for j in range(W))
    dw = torch.stack([(d * _back(x, s["pos"], W - 1 - i)).sum(0) for i in range(W)], 1)
    return {"out": _silu(pre).to(dt), "dx": dx.to(dt), "dweight": dw, "dbias": d.sum(0)}


def _scan_in_place(a, b, longest, reverse=False):
    """b becomes h with h_t = a_t h_{t-1} + b_t (reverse: h_{t+1}) along the first axis, by doubling; a is used up."""
    k = 1
    while k < longest:
        cur, old = (slice(None, -k), slice(k, None)) if reverse else (slice(k, None), slice(None, -k))
        t = a[cur] * b[old]
        b[cur] += t
        t = a[cur] * a[old]
        a[cur] = t
        del t
        k *= 2
    return b


def _per_channel(v, D):
    """[Ntok, G, N] as [Ntok, D, N]: every channel sees its group's row (a view)."""
    n, G, N = v.shape
    return v.float()[:, :, None, :].expand(n, G, D // G, N).reshape(n, D, N) if G > 1 else v.float().expand(n, D, N)


def _scan_plain(s, keep=False):
    c, D, dt = s["c"], s["c"]["D"], s["x"].dtype
    x, step = s["x"].float(), _softplus(s["dt"].float() + s["dt_bias"])
    a = torch.exp(step[:, :, None] * s["A"])
    kept = a.clone() if keep else None
    b = (step * x)[:, :, None] * _per_channel(s["Bm"], D)
    if "h0" in s:
        b[s["start"]] += a[s["start"]] * s["h0"]
    a[s["start"]] = 0
    h = _scan_in_place(a, b, s["maxlen"])
    del a
    y = (h * _per_channel(s["Cm"], D)).sum(-1) + s["Dskip"] * x
    out = (y * _silu(s["z"].float()) if "z" in s else y).to(dt)
    return (out, y, h, kept, x, step) if keep else {"out": out, "state": h[s["last"]]}


def _scan_train_plain(s):
    c, D, dt = s["c"], s["c"]["D"], s["x"].dtype
    G, N = c["G"], c["N"]
    out, y, h, a, x, step = _scan_plain(s, keep=True)
    res = {"out": out}
    dy = s["dout"].float()
    if "z" in s:
        z = s["z"].float()
        res["dz"] = (dy * y * _dsilu(z)).to(dt)
        dy = dy * _silu(z)
    res["dD"] = (dy * x).sum(0)
    group = lambda v: v.unflatten(1, (G, D // G)).sum(2).to(dt)  # noqa: E731
    res["dCm"] = group(dy[:, :, None] * h)
    # dL/dh_t = C_t dy_t + a_{t+1} dL/dh_{t+1}
    d = dy[:, :, None] * _per_channel(s["Cm"], D)
    nxt = torch.zeros_like(a)
    nxt[:-1] = a[1:]
    nxt[s["last"]] = 0
    d = _scan_in_place(nxt, d, s["maxlen"], reverse=True)
    del nxt
    res["dBm"] = group(d * (step * x)[:, :, None])
    du = (d * _per_channel(s["Bm"], D)).sum(-1)
    res["dx"] = (du * step + s["Dskip"] * dy).to(dt)
    prev = torch.zeros_like(h)
    prev[1:] = h[:-1]
    prev[s["start"]] = 0
    g = d * a * prev            # dL/d(step A)
    res["dA"] = (g * step[:, :, None]).sum(0)
    ddt = ((g * s["A"]).sum(-1) + du * x) / (1 + torch.exp(-(s["dt"].float() + s["dt_bias"])))
    res["ddt"], res["ddt_bias"] = ddt.to(dt), ddt.sum(0)
    return res


def _step_plain(s):
    c, dt, D = s["c"], s["x"].dtype, s["c"]["D"]
    win = torch.cat([s["hist"], s["x"][:, None]], 1)
    u = _silu((win.float() * s["w"].t()).sum(1) + s["bias"]).to(dt)
    s["hist"].copy_(win[:, 1:])
    x, step = u.float(), _softplus(s["dt"].float() + s["dt_bias"])
    s["h"].mul_(torch.exp(step[:, :, None] * s["A"])).add_((step * x)[:, :, None] * _per_channel(s["Bm"], D))
    y = (s["h"] * _per_channel(s["Cm"], D)).sum(-1) + s["Dskip"] * x
    return {"u": u, "out": (y * _silu(s["z"].float())).to(dt), "hist": s["hist"], "state": s["h"]}


_EPS = 1e-5


def _norm_plain(s):
    dt = s["x"].dtype
    if "res" in s:
        # the sum is kept in the tensors' type and that is what is normalised
        total = (s["x"].float() + s["res"].float()).to(dt)
    else:
        total = s["x"]
    v = total.float()
    mean = v.mean(1, keepdim=True)
    v = v - mean
    rstd = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + _EPS)
    xh = v * rstd
    return total, (xh * s["w"] + s["b"]).to(dt), xh, rstd


def _norm_train_plain(s):
    dt = s["x"].dtype
    _, out, xh, rstd = _norm_plain(s)
    d = s["dout"].float()
    e = d * s["w"]
    dx = (e - e.mean(1, keepdim=True) - xh * (e * xh).mean(1, keepdim=True)) * rstd
    return {"out": out, "dx": dx.to(dt), "dweight": (d * xh).sum(0), "dbias": d.sum(0)}


# ---- the package's entry points ---------------------------------------------------

def _axis(s):
    return {"cu_seqlens": s["cu"]} if "cu" in s else {"B": s["c"]["B"], "T": s["c"]["T"]}


def _run_own(s):
    from bayesian_filter_scan_b200 import kla
    op = s["c"]["op"]
    if op == "conv":
        out, hist = kla.conv_forward(s["x"], s["w"], s["bias"], final_state=True, **_axis(s))
        return {"out": out, "hist": hist}
    if op == "conv_train":
        out = kla.conv_forward(s["x"], s["w"], s["bias"], **_axis(s))
        g = kla.conv_backward(s["x"], s["w"], s["dout"], s["bias"], **_axis(s))
        return {"out": out, "dx": g["dx"], "dweight": g["dweight"], "dbias": g["dbias"]}
    if op == "scan":
        out, state = kla.ssm_forward(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["Dskip"], z=s.get("z"),
                                     dt_bias=s["dt_bias"], state0=s.get("h0"), final_state=True, **_axis(s))
        return {"out": out, "state": state}
    if op == "scan_train":
        more = dict(D=s["Dskip"], z=s.get("z"), dt_bias=s["dt_bias"], **_axis(s))
        out, states = kla.ssm_forward(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], save_states=True, **more)
        g = kla.ssm_backward(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dout"], states=states, **more)
        res = {k: g[k] for k in ("dx", "ddt", "dA", "dBm", "dCm", "dD", "ddt_bias")}
        if "z" in s:
            res["dz"] = g["dz"]
        return {"out": out, **res}
    if op == "step":
        u = kla.conv_step(s["x"], s["w"], s["hist"], s["bias"])
        out = kla.ssm_step(u, s["dt"], s["A"], s["Bm"], s["Cm"], s["h"], D=s["Dskip"], z=s["z"], dt_bias=s["dt_bias"])
        return {"u": u, "out": out, "hist": s["hist"], "state": s["h"]}
    if op == "norm":
        out, total = kla.layernorm_forward(s["x"], s["w"], s["b"], residual=s["res"], eps=_EPS)
        return {"out": out, "sum": total}
    out, mean, rstd = kla.layernorm_forward(s["x"], s["w"], s["b"], eps=_EPS, stats=True)
    g = kla.layernorm_backward(s["x"], s["dout"], mean, rstd, s["w"])
    return {"out": out, "dx": g["dx"], "dweight": g["dweight"], "dbias": g["dbias"]}


def run(state):
    if own:
        return _run_own(state)
    op = state["c"]["op"]
    if op == "norm":
        total, out, _, _ = _norm_plain(state)
        return {"out": out, "sum": total}
    return {"conv": _conv_plain, "conv_train": _conv_train_plain, "scan": _scan_plain,
            "scan_train": _scan_train_plain, "step": _step_plain, "norm_train": _norm_train_plain}[op](state)


def work(case):
    c, es = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] in ("norm", "norm_train"):
        n = c["rows"] * c["D"]
        # residual form: two tensors in, two out; training: x in and out, then x and dout in, dx out (x once)
        return {"bytes": n * es * 4 + 8 * c["D"], "flops": n * (9 if c["op"] == "norm" else 22)}
    D = c["D"]
    ntok = c["B"] if c["op"] == "step" else c["T"] if c["seqs"] else c["B"] * c["T"]
    nseq = c["B"] if c["op"] == "step" else c["seqs"] or c["B"]
    n = ntok * D
    if c["op"] in ("conv", "conv_train"):
        W = c["W"]
        if c["op"] == "conv":
            return {"bytes": 2 * es * n + es * nseq * (W - 1) * D + 4 * D * (W + 1), "flops": n * (2 * W + 5)}
        return {"bytes": 4 * es * n + 8 * D * (W + 1), "flops": n * (6 * W + 15)}
    N, G = c["N"], c["G"]
    bc, par = 2 * ntok * G * N * es, 4 * D * (N + 2)
    if c["op"] == "step":
        W = c["W"]
        return {"bytes": es * n * (5 + 2 * (W - 1)) + 8 * n * N + bc + par + 4 * D * (W + 1), "flops": n * (7 * N + 2 * W + 20)}
    z = 1 if c["gate"] else 0
    if c["op"] == "scan":
        return {"bytes": (3 + z) * es * n + bc + par + 4 * nseq * D * N * (2 if c["seqs"] else 1), "flops": n * (7 * N + 10)}
    # x, dt, z, dout in; out, dx, ddt, dz out; B, C in and their gradients out
    return {"bytes": (6 + 2 * z) * es * n + 2 * bc + 2 * par, "flops": n * (27 * N + 30)}


# ---- 64 bits, from the definitions -------------------------------------------------

def _grid(s):
    """Tokens as [sequence, place]: flat indices (clipped) and which places hold a token."""
    off = torch.tensor(s["off"], device="cuda")
    place = torch.arange(s["maxlen"], device="cuda")
    here = place[None] < (off[1:] - off[:-1])[:, None]
    return (off[:-1, None] + place).clamp(max=s["off"][-1] - 1), here


def _exact_conv(s):
    c, W = s["c"], s["c"]["W"]
    at, here = _grid(s)
    x = torch.where(here[..., None], s["x"][at].double(), 0.0)
    n, T, D = x.shape
    wide = torch.cat([torch.zeros(n, W - 1, D, device="cuda", dtype=torch.float64), x], 1)
    w = s["w"].double()
    pre = s["bias"].double() + sum(wide[:, i:i + T] * w[:, i] for i in range(W))
    sg = torch.sigmoid(pre)
    flat = lambda v: v[here]  # noqa: E731
    if c["op"] == "conv":
        lens = here.sum(1)
        hist = torch.stack([wide[i, int(m):int(m) + W - 1] for i, m in enumerate(lens.tolist())])
        return {"out": flat(pre * sg), "hist": hist}
    dout = torch.where(here[..., None], s["dout"][at].double(), 0.0)
    d = dout * (sg + pre * sg * (1 - sg))
    dwide = torch.zeros_like(wide)
    for i in range(W):
        dwide[:, i:i + T] += d * w[:, i]
    dw = torch.stack([(d * wide[:, i:i + T]).sum((0, 1)) for i in range(W)], 1)
    return {"out": flat(pre * sg), "dx": flat(dwide[:, W - 1:]), "dweight": dw, "dbias": d.sum((0, 1))}


def _exact_scan(s):
    """Token by token in blocks of places: decays and inputs of a block at once, the recurrence one place at a time."""
    c, D, G, N = s["c"], s["c"]["D"], s["c"]["G"], s["c"]["N"]
    at, here = _grid(s)
    n, T = at.shape
    A, train = s["A"].double(), c["op"] == "scan_train"
    h = s["h0"].double() if "h0" in s else torch.zeros(n, D, N, device="cuda", dtype=torch.float64)
    spread = lambda v: v.double().repeat_interleave(D // G, dim=2)  # noqa: E731
    block = T if train else max(1, min(T, (1 << 27) // (n * D * N)))
    out = torch.empty(s["off"][-1], D, device="cuda", dtype=torch.float64)
    for lo in range(0, T, block):
        hi = min(T, lo + block)
        i, ok = at[:, lo:hi].t(), here[:, lo:hi].t()
        x = s["x"][i].double()
        raw = s["dt"][i].double() + s["dt_bias"].double()
        step = torch.where(raw > 30, raw, torch.log1p(torch.exp(raw.clamp(max=30))))
        a = torch.exp(step[..., None] * A)
        a[~ok] = 1.0
        b = (step * x)[..., None] * spread(s["Bm"][i])
        b[~ok] = 0.0
        hs = torch.empty_like(a)
        for t in range(hi - lo):
            h = torch.addcmul(b[t], a[t], h, out=hs[t])
        h = h.clone()
        C = spread(s["Cm"][i])
        y = torch.einsum("tndk,tndk->tnd", hs, C) + s["Dskip"].double() * x
        gate = 1.0
        if "z" in s:
            z = s["z"][i].double()
            sz = torch.sigmoid(z)
            gate = z * sz
        out[i[ok]] = (y * gate)[ok]
        if not train:
            del a, b, hs, C
    if not train:
        return {"out": out, "state": h}
    res = {"out": out}
    flat = lambda v: torch.empty((s["off"][-1],) + v.shape[2:], device="cuda", dtype=torch.float64).index_copy_(0, i[ok], v[ok])  # noqa: E731
    go = torch.where(ok[..., None], s["dout"][i].double(), 0.0)
    if "z" in s:
        res["dz"] = flat(go * y * (sz + z * sz * (1 - sz)))
        go = go * gate
    gh = go[..., None] * C
    for t in range(T - 2, -1, -1):
        gh[t].addcmul_(a[t + 1], gh[t + 1])
    gh[~ok] = 0.0
    before = torch.cat([torch.zeros_like(hs[:1]), hs[:-1]], 0)
    per_group = lambda v: v.unflatten(2, (G, D // G)).sum(3)  # noqa: E731
    res["dCm"], res["dBm"] = flat(per_group(go[..., None] * hs)), flat(per_group(gh * (step * x)[..., None]))
    del C, hs
    gu = torch.einsum("tndk,tndk->tnd", gh, spread(s["Bm"][i]))
    ga = gh * before * a
    gdt = (torch.einsum("tndk,dk->tnd", ga, A) + gu * x) * torch.sigmoid(raw)
    res["dx"] = flat(gu * step + go * s["Dskip"].double())
    res["ddt"], res["ddt_bias"] = flat(gdt), torch.where(ok[..., None], gdt, 0.0).sum((0, 1))
    res["dD"] = (go * x).sum((0, 1))
    res["dA"] = torch.einsum("tndk,tnd->dk", ga, step)
    return res


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("conv", "conv_train"):
        return _exact_conv(s)
    if op in ("scan", "scan_train"):
        return _exact_scan(s)
    if op == "step":
        D, G = case["D"], case["G"]
        w, x = s["w"].double(), torch.cat([s["hist"], s["x"][:, None]], 1).double()
        pre = torch.einsum("nwd,dw->nd", x, w) + s["bias"].double()
        u = pre * torch.sigmoid(pre)
        # the scan's input is the convolution's result in the tensors' type
        v = u.to(_DT[case["dtype"]]).double()
        raw = s["dt"].double() + s["dt_bias"].double()
        step = torch.log1p(torch.exp(-raw.abs())) + raw.clamp(min=0)
        spread = lambda m: m.double().repeat_interleave(D // G, dim=1)  # noqa: E731
        h = s["h"].double() * torch.exp(step[..., None] * s["A"].double()) + (step * v)[..., None] * spread(s["Bm"])
        y = torch.einsum("ndk,ndk->nd", h, spread(s["Cm"])) + s["Dskip"].double() * v
        z = s["z"].double()
        return {"u": u, "out": y * z * torch.sigmoid(z), "hist": x[:, 1:], "state": h}
    x, dt = s["x"].double(), _DT[case["dtype"]]
    if op == "norm":
        x = (x + s["res"].double()).to(torch.float32).to(dt).double()
    var, mean = torch.var_mean(x, dim=1, keepdim=True, correction=0)
    r = (var + _EPS).rsqrt()
    xh, w = (x - mean) * r, s["w"].double()
    out = xh * w + s["b"].double()
    if op == "norm":
        return {"out": out, "sum": x}
    d = s["dout"].double()
    e = d * w
    D = case["D"]
    dx = r / D * (D * e - e.sum(1, keepdim=True) - xh * (e * xh).sum(1, keepdim=True))
    return {"out": out, "dx": dx, "dweight": torch.einsum("rd,rd->d", d, xh), "dbias": d.sum(0)}
