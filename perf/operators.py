"""The state-space layer's operators, as they are measured: the short causal
convolution, the selective state-space scan and the group norm, each for
prompts, for single tokens where it has that form, and in training (forward
and backward).

``run`` computes them either in plain torch arithmetic (``own`` false) or with
this package's calls (``own`` true), on the same inputs.  Sequences are packed
along one token axis; a batch of equal sequences is the case ``seqs`` > 0 with
``cut`` = 0.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------
# cases

def listed():
    return [
        # the convolution in front of a mixer of 4096 channels over the 128k-token prompt
        dict(name="conv prompt 128k", op="conv", mode="prompt", T=131072, seqs=1, cut=0, C=4096, W=4,
             bias=True, silu=True, state=False, dtype="bf16"),
        # a packed prompt batch with carried windows: odd channel count, ragged and empty sequences
        dict(name="conv prompt packed odd", op="conv", mode="prompt", T=9001, seqs=17, cut=5, C=1283, W=3,
             bias=False, silu=False, state=True, dtype="fp32"),
        # one decode step of 256 requests
        dict(name="conv step 256", op="conv", mode="step", T=256, seqs=256, cut=0, C=4096, W=4,
             bias=True, silu=True, state=True, dtype="bf16"),
        # a training step of the convolution over the batch of 4 x 4096 tokens
        dict(name="conv training 4x4096", op="conv", mode="train", T=16384, seqs=4, cut=0, C=4096, W=4,
             bias=True, silu=True, state=False, dtype="bf16"),
        # a prompt batch of 4 x 4096 tokens through a layer of 4096 channels
        dict(name="scan prompt 4x4096", op="scan", mode="prompt", T=16384, seqs=4, cut=0, D=4096, S=16, G=1,
             gate=True, state=False, dtype="bf16"),
        # few long ragged prompts of a small layer: the token axis is the only parallel one left
        dict(name="scan prompt packed fp32", op="scan", mode="prompt", T=20011, seqs=3, cut=7, D=1100, S=16, G=2,
             gate=True, state=True, dtype="fp32"),
        # one decode step of 256 requests
        dict(name="scan step 256", op="scan", mode="step", T=256, seqs=256, cut=0, D=4096, S=16, G=1,
             gate=True, state=True, dtype="bf16"),
        # one request: the latency of a single token
        dict(name="scan step 1", op="scan", mode="step", T=1, seqs=1, cut=0, D=1536, S=16, G=1,
             gate=True, state=True, dtype="fp32"),
        # a training step over 4 x 1024 tokens of a layer of 4096 channels
        dict(name="scan training 4x1024", op="scan", mode="train", T=4096, seqs=4, cut=0, D=4096, S=16, G=1,
             gate=True, state=False, dtype="bf16"),
        # fine-tuning on short packed documents: small odd layer, wider state, no gate
        dict(name="scan training packed fp32", op="scan", mode="train", T=1999, seqs=9, cut=3, D=330, S=24, G=2,
             gate=False, state=True, dtype="fp32"),
        # the mixer's output, normalised per token and head of 128 channels
        dict(name="norm heads 4x4096", op="norm", mode="prompt", T=16384, seqs=4, cut=0, C=4096, groups=32,
             per_token=True, silu=True, dtype="bf16"),
        # whole-sequence statistics over a ragged batch, training
        dict(name="norm sequences training", op="norm", mode="train", T=24007, seqs=11, cut=2, C=640, groups=32,
             per_token=False, silu=True, dtype="bf16"),
    ]


def _size(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _channels(rng, lo, hi):
    """A channel count: mostly a multiple of 64, sometimes of 8, sometimes any."""
    c = _size(rng, lo, hi)
    step = rng.choice((64, 64, 64, 8, 1))
    return max(step, c // step * step)


def draw(rng):
    op = rng.choice(("conv", "scan", "scan", "norm"))
    mode = rng.choice(("prompt", "train") if op == "norm" else ("prompt", "step", "train"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    case = dict(op=op, mode=mode, dtype=dtype)
    if op == "scan":
        S = rng.choice((4, 8, 13, 16, 16, 16, 24, 32, 64))
        # the plain form holds tokens x channels x states in memory
        most = {"prompt": 1 << 29, "step": 1 << 26, "train": 1 << 28}[mode]
        G = rng.choice((1, 1, 1, 2, 4))
        D = _channels(rng, 64, 8192) // G * G
        cap = max(1, min(65536, most // (D * S)))
        T = _size(rng, 1, min(cap, 1024)) if mode == "step" else _size(rng, min(cap, 64), cap)
        case.update(D=D, S=S, G=G, gate=rng.random() < 0.7)
    else:
        C = _channels(rng, 64, 8192)
        most = {"prompt": 1 << 27, "step": 1 << 23, "train": 1 << 25}[mode]
        cap = max(1, min(131072, most // C))
        T = _size(rng, 1, min(cap, 1024)) if mode == "step" else _size(rng, min(cap, 64), cap)
        if op == "conv":
            case.update(C=C, W=rng.choice((2, 3, 4, 4, 4)), bias=rng.random() < 0.6, silu=rng.random() < 0.7)
        else:
            g = rng.choice((1, 4, 8, 32))
            C = max(g, C // g * g)
            case.update(C=C, groups=g, per_token=rng.random() < 0.5, silu=rng.random() < 0.6)
    if mode == "step":
        case.update(T=T, seqs=T, cut=0, state=True)
        return case
    seqs = rng.randint(1, 4)
    cut = 0
    if rng.random() < 0.5:
        seqs, cut = rng.randint(2, 24), rng.randint(1, 1 << 20)
    else:
        T = max(seqs, T // seqs * seqs)
    case.update(T=T, seqs=seqs, cut=cut)
    if op != "norm":
        case.update(state=rng.random() < 0.5)
    return case


def _bounds(case):
    """Where the sequences begin and end on the packed token axis."""
    T, n = case["T"], case["seqs"]
    if not case["cut"]:
        return [T // n * i for i in range(n + 1)]
    r = random.Random(case["cut"])
    return [0] + sorted(r.randint(0, T) for _ in range(n - 1)) + [T]


def _bytes_of(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    """The bytes that have to be read and written once, and the arithmetic:
    a product, a sum and a transcendental count one each."""
    T, n, e, mode = case["T"], case["seqs"], _bytes_of(case), case["mode"]
    if case["op"] == "conv":
        C, W = case["C"], case["W"]
        act = 4 if case["silu"] else 0
        par = 4 * C * (W + (1 if case["bias"] else 0))
        window = n * (W - 1) * C * e
        by = 2 * T * C * e + par + window * ((1 if case["state"] else 0) + 1)
        fl = T * C * (2 * W + act)
        if mode == "train":
            # x and d_out in, grad_x out in 32 bits, the parameters' gradients
            by += T * C * (2 * e + 4) + 2 * par + 4 * n * (W - 1) * C * (2 if case["state"] else 1)
            fl += T * C * (6 * W + 2 * act)
        return {"bytes": by, "flops": fl}
    if case["op"] == "scan":
        D, S, G = case["D"], case["S"], case["G"]
        z = 1 if case["gate"] else 0
        par = 4 * D * (S + 2)
        st = 4 * n * D * S
        by = T * D * e * (3 + z) + 2 * T * G * S * e + par + st * ((1 if case["state"] else 0) + 1)
        fl = T * D * (7 * S + 8 + 5 * z)
        if mode == "train":
            by += T * D * (e * (3 + z) + 4 * (2 + z)) + T * G * S * (2 * e + 8) + 2 * par
            by += st * (2 if case["state"] else 1)
            fl += T * D * (20 * S + 16 + 10 * z)
        return {"bytes": by, "flops": fl}
    C, g = case["C"], case["groups"]
    samples = T if case["per_token"] else n
    act = 4 if case["silu"] else 0
    by = 2 * T * C * e + 8 * C + 8 * samples * g
    fl = T * C * (7 + act)
    if mode == "train":
        by += T * C * (2 * e + 4) + 16 * C + 8 * samples * g
        fl += T * C * (14 + 2 * act)
    return {"bytes": by, "flops": fl}


# --------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    T, n, mode = case["T"], case["seqs"], case["mode"]

    def normal(*shape, to=torch.float32, std=1.0):
        return (std * torch.randn(*shape, generator=gen, device=dev)).to(to)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(*shape, generator=gen, device=dev)

    # the batch is [B, T, ...]: packed sequences have B = 1 and their bounds
    lead = (T,) if mode == "step" else (1, T) if case["cut"] else (n, T // n)
    s = dict(case=case, cu=None)
    if mode != "step" and case["cut"]:
        s["cu"] = torch.tensor(_bounds(case), dtype=torch.int32, device=dev)
    if case["op"] == "conv":
        C, W = case["C"], case["W"]
        s["x"] = normal(*lead, C, to=dt)
        s["weight"] = normal(C, W, std=W ** -0.5)
        s["bias"] = normal(C, std=0.2) if case["bias"] else None
        s["state"] = normal(n, W - 1, C, to=dt) if case["state"] else None
        if mode == "train":
            s["d_out"] = normal(*lead, C, to=dt)
            s["d_final"] = normal(n, W - 1, C) if case["state"] else None
    elif case["op"] == "scan":
        D, S, G = case["D"], case["S"], case["G"]
        s["u"] = normal(*lead, D, to=dt)
        s["delta"] = normal(*lead, D, to=dt, std=0.5)
        # decay rates of a fresh layer, spread by training: -(1 .. S) times a factor near one
        s["A"] = -torch.arange(1, S + 1, device=dev, dtype=torch.float32) * torch.exp(normal(D, S, std=0.3))
        s["B"] = normal(*lead, G, S, to=dt)
        s["C"] = normal(*lead, G, S, to=dt)
        s["D"] = 1 + normal(D, std=0.1)
        s["z"] = normal(*lead, D, to=dt) if case["gate"] else None
        # steps between 1e-3 and 1e-1: the bias is their softplus inverse
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), D))
        s["delta_bias"] = step + torch.log(-torch.expm1(-step))
        s["state"] = normal(n, D, S) if case["state"] else None
        if mode == "train":
            s["d_out"] = normal(*lead, D, to=dt)
            s["d_final"] = normal(n, D, S) if case["state"] else None
    else:
        C = case["C"]
        # channels with means of their own, as activations have
        s["x"] = (normal(*lead, C) + normal(C)).to(dt)
        s["weight"] = 1 + normal(C, std=0.1)
        s["bias"] = normal(C, std=0.1)
        if mode == "train":
            s["d_out"] = normal(*lead, C, to=dt)
    return s


# --------------------------------------------------------------------------
# the plain form

def _silu(v):
    return v / (1 + torch.exp(-v))


def _silu_slope(v):
    g = 1 / (1 + torch.exp(-v))
    return g * (1 + v * (1 - g))


def _softplus(v):
    return v.clamp_min(0) + torch.log1p(torch.exp(-v.abs()))


class _Packed:
    """Where each token of the packed axis belongs."""

    def __init__(self, case, device):
        at = torch.tensor(_bounds(case), device=device)
        self.first, self.last = at[:-1], at[1:] - 1      # of each sequence (empty: last < first)
        self.full = (self.last >= self.first).nonzero()[:, 0]
        self.len = at[1:] - at[:-1]
        t = torch.arange(case["T"], device=device)
        self.seq = torch.searchsorted(at[1:].contiguous(), t, right=True)
        self.longest = max(b - a for a, b in zip(_bounds(case), _bounds(case)[1:]))


def _conv_stream(s, p, W):
    """x behind each sequence's window, in 32 bits: rows of the padded stream,
    and where the tokens stand in it."""
    x = s["x"].float().flatten(0, 1)
    row = torch.arange(x.shape[0], device=x.device) + (p.seq + 1) * (W - 1)
    n = p.first.numel()
    head = (p.first + torch.arange(n, device=x.device) * (W - 1))[:, None] + torch.arange(W - 1, device=x.device)
    xe = x.new_zeros(x.shape[0] + n * (W - 1), x.shape[1])
    xe[row] = x
    if s["state"] is not None:
        xe[head.flatten()] = s["state"].float().flatten(0, 1)
    # the last W - 1 rows of every sequence's stretch
    tail = (head[:, -1:] + p.len[:, None] - (W - 2)) + torch.arange(W - 1, device=x.device)
    return xe, row, head, tail


def _plain_conv(s):
    case = s["case"]
    W, dt = case["W"], s["x"].dtype
    w = s["weight"]
    if case["mode"] == "step":
        xe = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)
        v = (xe * w.t()).sum(1)
        v = v if s["bias"] is None else v + s["bias"]
        s["state"].copy_(xe[:, 1:])
        return {"out": (_silu(v) if case["silu"] else v).to(dt), "state": s["state"]}
    p = _Packed(case, s["x"].device)
    xe, row, head, tail = _conv_stream(s, p, W)
    win = xe.unfold(0, W, 1)[row - (W - 1)]                       # [T, C, W]
    v = (win * w).sum(-1)
    v = v if s["bias"] is None else v + s["bias"]
    res = {"out": (_silu(v) if case["silu"] else v).to(dt).view(s["x"].shape),
           "final_state": xe[tail].to(dt)}
    if case["mode"] == "train":
        dv = s["d_out"].float().flatten(0, 1)
        dv = dv * _silu_slope(v) if case["silu"] else dv
        dve = torch.zeros(xe.shape[0] + W - 1, xe.shape[1], device=xe.device)
        dve[row] = dv
        dxe = (dve.unfold(0, W, 1) * w.flip(1)).sum(-1)
        if s["d_final"] is not None:
            dxe.index_add_(0, tail.flatten(), s["d_final"].flatten(0, 1))
        res["dx"] = dxe[row].view(s["x"].shape)
        res["dweight"] = (win * dv[..., None]).sum(0)
        res["dbias"] = None if s["bias"] is None else dv.sum(0)
        res["dstate"] = None if s["state"] is None else dxe[head]
    return res


def _scan(a, b, longest):
    """h[t] = a[t] h[t-1] + b[t] along the first axis, by doubling: after each
    step, a and b span twice as many tokens.  a = 0 where a sequence begins."""
    span = 1
    while span < longest:
        b = torch.cat([b[:span], torch.addcmul(b[span:], a[span:], b[:-span])])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return b


def _plain_scan(s):
    case = s["case"]
    dt_out = s["u"].dtype
    D, S, G = case["D"], case["S"], case["G"]
    step = case["mode"] == "step"

    def tokens(t):
        return t.float().reshape(case["T"], *t.shape[1 if step else 2:])

    u, raw = tokens(s["u"]), tokens(s["delta"]) + s["delta_bias"]
    dt = _softplus(raw)
    A = s["A"]

    def heads(t):                                                 # [T, G, S] over the channels of its group
        return t[:, :, None, :].expand(-1, G, D // G, S).reshape(t.shape[0], D, S)

    Bm, Cm = tokens(s["B"]), tokens(s["C"])
    a = torch.exp(dt[..., None] * A)                              # [T, D, S]
    b = (dt * u)[..., None] * heads(Bm)
    z = None if s["z"] is None else tokens(s["z"])

    def output(h):
        y = (h * heads(Cm)).sum(-1) + s["D"] * u
        return y, (y if z is None else y * _silu(z)).to(dt_out).view(s["u"].shape)

    if step:
        h = torch.addcmul(b, a, s["state"])
        s["state"].copy_(h)
        return {"out": output(h)[1], "state": s["state"]}
    p = _Packed(case, u.device)
    first, last = p.first[p.full], p.last[p.full]
    h0 = torch.zeros(p.first.numel(), D, S, device=u.device) if s["state"] is None else s["state"]
    b[first] += a[first] * h0[p.full]
    cut = a.clone()
    cut[first] = 0
    h = _scan(cut, b, p.longest)
    y, out = output(h)
    final = h0.clone()
    final[p.full] = h[last]
    res = {"out": out, "final_state": final}
    if case["mode"] == "train":
        dy = tokens(s["d_out"])
        if z is not None:
            res["dz"] = (dy * y * _silu_slope(z)).view(s["u"].shape)
            dy = dy * _silu(z)
        c = dy[..., None] * heads(Cm)
        if s["d_final"] is not None:
            c[last] += s["d_final"][p.full]
        nxt = torch.cat([cut[1:], cut[:1]])                       # the decay into the next token, 0 at an end
        nxt[last] = 0
        g = _scan(nxt.flip(0), c.flip(0), p.longest).flip(0)
        before = torch.cat([h[:1], h[:-1]])
        before[first] = h0[p.full]
        ga = g * before * a
        gb = (g * heads(Bm)).sum(-1)
        ddt = (ga * A).sum(-1) + u * gb
        ddelta = ddt / (1 + torch.exp(-raw))
        res["du"] = (dt * gb + s["D"] * dy).view(s["u"].shape)
        res["ddelta"] = ddelta.view(s["u"].shape)
        res["dA"] = (ga * dt[..., None]).sum(0)
        res["dB"] = (g * (dt * u)[..., None]).view(-1, G, D // G, S).sum(2).view(s["B"].shape)
        res["dC"] = (h * dy[..., None]).view(-1, G, D // G, S).sum(2).view(s["C"].shape)
        res["dD"] = (dy * u).sum(0)
        res["ddelta_bias"] = ddelta.sum(0)
        if s["state"] is not None:
            d0 = torch.zeros_like(h0) if s["d_final"] is None else s["d_final"].clone()
            d0[p.full] = g[first] * a[first]
            res["dstate"] = d0
    return res


def _plain_norm(s):
    case, eps = s["case"], 1e-5
    g, T, C = case["groups"], case["T"], case["C"]
    x = s["x"].float().view(T, g, C // g)
    if case["per_token"]:
        mean = x.mean(-1)
        rstd = 1 / torch.sqrt((x - mean[..., None]).square().mean(-1) + eps)
        m, r = mean, rstd
    else:
        p = _Packed(case, x.device)
        n = (p.len * (C // g)).clamp_min(1)[:, None]

        def total(v):                                             # over each sequence's tokens: long sums, in 64 bits
            return torch.zeros(p.len.numel(), g, dtype=torch.float64, device=v.device).index_add_(0, p.seq, v.double().sum(-1))

        mean = (total(x) / n).float()
        m = mean[p.seq]
        rstd = (1 / torch.sqrt(total((x - m[..., None]).square()) / n + eps)).float()
        r = rstd[p.seq]
    w, b = s["weight"].view(g, -1), s["bias"].view(g, -1)
    xhat = (x - m[..., None]) * r[..., None]
    v = xhat * w + b
    res = {"out": (_silu(v) if case["silu"] else v).to(s["x"].dtype).view(s["x"].shape), "mean": mean, "rstd": rstd}
    if case["mode"] == "train":
        dv = s["d_out"].float().view(x.shape)
        dv = dv * _silu_slope(v) if case["silu"] else dv
        k = dv * w
        if case["per_token"]:
            k1, k2 = k.mean(-1), (k * xhat).mean(-1)
        else:
            k1, k2 = (total(k) / n).float()[p.seq], (total(k * xhat) / n).float()[p.seq]
        res["dx"] = (r[..., None] * (k - k1[..., None] - xhat * k2[..., None])).view(s["x"].shape)
        res["dweight"] = (dv * xhat).double().sum(0).float().view(C)
        res["dbias"] = dv.double().sum(0).float().view(C)
    return res


# --------------------------------------------------------------------------
# this package's calls

def _own_conv(s):
    import gated_delta_rule_103_b200 as kda
    case = s["case"]
    act = "silu" if case["silu"] else None
    if case["mode"] == "step":
        out = kda.short_conv_step(s["x"], s["weight"], s["state"], bias=s["bias"], activation=act)
        return {"out": out, "state": s["state"]}
    out, final = kda.short_conv_fwd(s["x"], s["weight"], bias=s["bias"], initial_state=s["state"],
                                    cu_seqlens=s["cu"], activation=act)
    res = {"out": out, "final_state": final}
    if case["mode"] == "train":
        dx, dw, db, ds = kda.short_conv_bwd(s["x"], s["weight"], s["d_out"], bias=s["bias"],
                                            initial_state=s["state"], d_final_state=s["d_final"],
                                            cu_seqlens=s["cu"], activation=act,
                                            need_initial_state_grad=s["state"] is not None)
        res.update(dx=dx, dweight=dw, dbias=db, dstate=ds)
    return res


def _own_scan(s):
    import gated_delta_rule_103_b200 as kda
    case = s["case"]
    args = (s["u"], s["delta"], s["A"], s["B"], s["C"])
    opt = dict(D=s["D"], z=s["z"], delta_bias=s["delta_bias"], softplus=True)
    if case["mode"] == "step":
        out = kda.ssm_step(*args, s["state"], **opt)
        return {"out": out, "state": s["state"]}
    out, final = kda.ssm_scan_fwd(*args, initial_state=s["state"], cu_seqlens=s["cu"], **opt)
    res = {"out": out, "final_state": final}
    if case["mode"] == "train":
        g = kda.ssm_scan_bwd(*args, s["d_out"], initial_state=s["state"], d_final_state=s["d_final"],
                             cu_seqlens=s["cu"], need_initial_state_grad=s["state"] is not None, **opt)
        names = ("du", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddelta_bias", "dstate")
        res.update({k: v for k, v in zip(names, g) if v is not None})
    return res


def _own_norm(s):
    import gated_delta_rule_103_b200 as kda
    case = s["case"]
    opt = dict(weight=s["weight"], bias=s["bias"], activation="silu" if case["silu"] else None,
               per_token=case["per_token"], cu_seqlens=s["cu"])
    out, mean, rstd = kda.group_norm_fwd(s["x"], case["groups"], eps=1e-5, **opt)
    res = {"out": out, "mean": mean, "rstd": rstd}
    if case["mode"] == "train":
        dx, dw, db = kda.group_norm_bwd(s["x"], case["groups"], s["d_out"], mean, rstd, **opt)
        res.update(dx=dx, dweight=dw, dbias=db)
    return res


def run(state):
    op = state["case"]["op"]
    if own:
        return {"conv": _own_conv, "scan": _own_scan, "norm": _own_norm}[op](state)
    return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[op](state)


# --------------------------------------------------------------------------
# the definitions, in 64 bits: token by token, sequence by sequence

def _sig64(v):
    return 1 / (1 + torch.exp(-v))


def _exact_conv(s):
    case = s["case"]
    W = case["W"]
    x, w = s["x"].double(), s["weight"].double()
    bias = 0 if s["bias"] is None else s["bias"].double()
    if case["mode"] == "step":
        st = s["state"].double()
        v = bias + x * w[:, W - 1]
        for j in range(W - 1):
            v = v + st[:, j] * w[:, j]
        return {"out": v * _sig64(v) if case["silu"] else v, "state": torch.cat([st[:, 1:], x[:, None]], 1)}
    at, C = _bounds(case), case["C"]
    train = case["mode"] == "train"
    if case["T"] * C > (1 << 28) and train:
        return None
    xs = x.reshape(-1, C)
    out, dx = torch.empty_like(xs), torch.empty_like(xs) if train else None
    fin, d0 = [], []
    dw, db = torch.zeros_like(w), torch.zeros(C, dtype=torch.float64, device=x.device)
    for i in range(case["seqs"]):
        lo, hi = at[i], at[i + 1]
        win = torch.zeros(W - 1, C, dtype=torch.float64, device=x.device) if s["state"] is None else s["state"][i].double()
        row = torch.cat([win, xs[lo:hi]])
        L = hi - lo
        v = bias + sum(row[j:j + L] * w[:, j] for j in range(W))
        out[lo:hi] = v * _sig64(v) if case["silu"] else v
        fin.append(row[L:])
        if train:
            dv = s["d_out"].reshape(-1, C)[lo:hi].double()
            if case["silu"]:
                sg = _sig64(v)
                dv = dv * (sg + v * sg * (1 - sg))
            dr = torch.zeros_like(row)
            for j in range(W):
                dr[j:j + L] += dv * w[:, j]
                dw[:, j] += (dv * row[j:j + L]).sum(0)
            db += dv.sum(0)
            if s["d_final"] is not None:
                dr[L:] += s["d_final"][i].double()
            dx[lo:hi] = dr[W - 1:]
            d0.append(dr[:W - 1])
    res = {"out": out.view(x.shape), "final_state": torch.stack(fin)}
    if train:
        res.update(dx=dx.view(x.shape), dweight=dw, dbias=None if s["bias"] is None else db,
                   dstate=None if s["state"] is None else torch.stack(d0))
    return res


def _exact_scan(s):
    case = s["case"]
    D, S, G, n = case["D"], case["S"], case["G"], case["seqs"]
    A, skip, bias = s["A"].double(), s["D"].double(), s["delta_bias"].double()
    train = case["mode"] == "train"
    at = list(range(n + 1)) if case["mode"] == "step" else _bounds(case)
    L = [b - a for a, b in zip(at, at[1:])]
    if max(L) > 70000 or (train and n * max(L) * D * S > (1 << 31)):
        return None
    lead = s["u"].shape
    u, raw = s["u"].reshape(-1, D).double(), s["delta"].reshape(-1, D).double() + bias
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    Bm, Cm = s["B"].reshape(-1, G, 1, S), s["C"].reshape(-1, G, 1, S)
    z = None if s["z"] is None else s["z"].reshape(-1, D).double()
    # longest sequence first, so that those still running are always the first ones
    order = sorted(range(n), key=lambda i: -L[i])
    start = torch.tensor([at[i] for i in order], device=u.device)
    state = torch.zeros(n, D, S, dtype=torch.float64, device=u.device) if s["state"] is None else s["state"].double()
    h = state[order].clone()
    y = torch.empty_like(u)
    kept = []
    live = [sum(1 for v in L if v > t) for t in range(max(L))]

    def wide(m, r):
        return m[r].double().expand(-1, G, D // G, S).reshape(-1, D, S)

    for t, k in enumerate(live):
        r = start[:k] + t
        if train:
            kept.append(h[:k].clone())
        h[:k] = torch.exp(dt[r][..., None] * A) * h[:k] + (dt[r] * u[r])[..., None] * wide(Bm, r)
        y[r] = torch.einsum("kds,kds->kd", h[:k], wide(Cm, r))
    y = y + skip * u
    back = torch.tensor(sorted(range(n), key=lambda i: order[i]), device=u.device)
    out = (y if z is None else y * z * _sig64(z)).view(lead)
    if case["mode"] == "step":
        return {"out": out, "state": h[back]}
    res = {"out": out, "final_state": h[back]}
    if train:
        dy = s["d_out"].reshape(-1, D).double()
        if z is not None:
            sg = _sig64(z)
            res["dz"] = (dy * y * (sg + z * sg * (1 - sg))).view(lead)
            dy = dy * z * sg
        g = torch.zeros_like(h) if s["d_final"] is None else s["d_final"].double()[order].clone()
        gb, ddt = torch.empty_like(u), torch.empty_like(u)
        dA = torch.zeros_like(A)
        dB = torch.empty(u.shape[0], G, S, dtype=torch.float64, device=u.device)
        dC = torch.empty_like(dB)
        for t in range(max(L) - 1, -1, -1):
            k = live[t]
            r = start[:k] + t
            a = torch.exp(dt[r][..., None] * A)
            ht = a * kept[t] + (dt[r] * u[r])[..., None] * wide(Bm, r)
            dC[r] = (ht * dy[r][..., None]).view(k, G, D // G, S).sum(2)
            gt = g[:k] + dy[r][..., None] * wide(Cm, r)
            dB[r] = (gt * (dt[r] * u[r])[..., None]).view(k, G, D // G, S).sum(2)
            gb[r] = (gt * wide(Bm, r)).sum(-1)
            da = gt * kept[t] * a
            ddt[r] = (da * A).sum(-1) + u[r] * gb[r]
            dA += (da * dt[r][..., None]).sum(0)
            g[:k] = gt * a
            kept[t] = None
        ddelta = ddt * _sig64(raw)
        res.update(du=(dt * gb + skip * dy).view(lead), ddelta=ddelta.view(lead), dA=dA, dB=dB.view(s["B"].shape),
                   dC=dC.view(s["C"].shape), dD=(dy * u).sum(0), ddelta_bias=ddelta.sum(0))
        if s["state"] is not None:
            res["dstate"] = g[back]
    return res


def _exact_norm(s):
    case, eps = s["case"], 1e-5
    g, T, C = case["groups"], case["T"], case["C"]
    train = case["mode"] == "train"
    w, b = s["weight"].double().view(g, -1), s["bias"].double().view(g, -1)
    if T * C > (1 << 27) and train:
        return None
    x = s["x"].reshape(T, g, C // g)
    # per token: pieces of the token axis; else one sequence at a time
    at = list(range(0, T, 8192)) + [T] if case["per_token"] else _bounds(case)
    dims = 2 if case["per_token"] else (0, 2)
    out = torch.empty(T, g, C // g, dtype=torch.float64, device=x.device)
    dx = torch.empty_like(out) if train else None
    dw, db = torch.zeros_like(w), torch.zeros_like(w)
    means, rstds = [], []
    for lo, hi in zip(at, at[1:]):
        xs = x[lo:hi].double()
        if lo == hi:
            means.append(torch.zeros(1, g, dtype=torch.float64, device=x.device))
            rstds.append(torch.full_like(means[-1], eps ** -0.5))
            continue
        var, mu = torch.var_mean(xs, dims, correction=0, keepdim=True)
        r = (var + eps).rsqrt()
        xh = (xs - mu) * r
        v = xh * w + b
        out[lo:hi] = v * _sig64(v) if case["silu"] else v
        means.append(mu[..., 0])
        rstds.append(r[..., 0])
        if train:
            dv = s["d_out"].reshape(T, g, C // g)[lo:hi].double()
            if case["silu"]:
                sg = _sig64(v)
                dv = dv * (sg + v * sg * (1 - sg))
            dw += (dv * xh).sum(0)
            db += dv.sum(0)
            k = dv * w
            dx[lo:hi] = r * (k - k.mean(dims, keepdim=True) - xh * (k * xh).mean(dims, keepdim=True))
    res = {"out": out.view(s["x"].shape), "mean": torch.cat(means), "rstd": torch.cat(rstds)}
    if train:
        res.update(dx=dx.view(s["x"].shape), dweight=dw.view(C), dbias=db.view(C))
    return res


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](s)
