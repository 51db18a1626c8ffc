"""The layer operators (short convolution, state-space scan, group norm)
against their 64-bit forms on the same inputs.

Tolerances are norm-wise.  A 16-bit output is rounded once from fp32, at most
half a step (2^-8 for bf16) of each value, so 2^-8 of the norm.  fp32 results:
a state carries the relative errors of its decays, 2^-22 (fast exponential)
plus 2^-24 for each product, over the tokens it remembers; the inputs below
keep dt |A| above 0.02 on the slowest state, some 50 tokens, so 50 (2^-22 + 2
2^-24) = 1.8e-5 covers scans, and a quarter of it the rest, whose longest
chains are plain sums.
"""
import pytest
import torch

import gated_delta_rule_103_b200 as kda
from gated_delta_rule_103_b200 import binding
import layer_reference as ref
from helpers import rel_fro

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
SCAN_TOL, TOL = 1.8e-5, 4.5e-6


def near(got, want, tol):
    if got.dtype == BF16:
        tol = tol + 2.0 ** -8
    assert tuple(got.shape) == tuple(want.shape)
    assert torch.isfinite(got).all()
    e = rel_fro(got, want)
    assert e <= tol, f"{e:.2e} > {tol:.2e}"


class Gen:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape, dtype=F32, std=1.0):
        return (std * torch.randn(*shape, generator=self.g, device="cuda")).to(dtype)

    def uniform(self, lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(*shape, generator=self.g, device="cuda")


def wide(t):
    return None if t is None else t.detach().cpu().double().requires_grad_()


def cu_of(lengths):
    return torch.tensor(ref.bounds_of(lengths), dtype=torch.int32, device="cuda")


# ---- short convolution ---------------------------------------------------------

LENGTHS = [[1], [2, 3], [0, 5, 0, 1, 130, 3, 0], [700, 65], [64, 64, 64]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C,W,silu,bias,state", [(128, 4, True, True, True), (72, 3, False, False, True),
                                                 (37, 2, True, True, False), (6, 4, True, False, True),
                                                 (1, 3, False, True, True), (1030, 4, False, True, False)])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_short_conv(dtype, C, W, silu, bias, state, lengths):
    g, T, N = Gen(C + W), sum(lengths), len(lengths)
    x = g.normal(1, T, C, dtype=dtype)
    w = g.normal(C, W, std=0.5)
    b = g.normal(C) if bias else None
    s0 = g.normal(N, W - 1, C, dtype=dtype) if state else None
    d_out, d_fin = g.normal(1, T, C, dtype=dtype), g.normal(N, W - 1, C)
    act, cu, bounds = "silu" if silu else None, cu_of(lengths), ref.bounds_of(lengths)
    out, fin = kda.short_conv_fwd(x, w, b, s0, cu, act)
    xs, ws, bs, ss = wide(x[0]), wide(w), wide(b), wide(s0)
    ss = torch.zeros(N, W - 1, C, dtype=torch.float64, requires_grad=True) if ss is None else ss
    o_ref, f_ref = ref.short_conv(xs, ws, bs, ss, bounds, silu)
    near(out[0], o_ref, TOL)
    assert torch.equal(fin.cpu().double(), f_ref.detach())       # rows are copied
    inputs = [xs, ws, ss] + ([bs] if bias else [])
    want = ref.grads_of((o_ref, f_ref), (d_out[0].cpu().double(), d_fin.cpu().double()), inputs)
    dx, dw, db, ds = kda.short_conv_bwd(x, w, d_out, b, s0, d_fin, cu, act)
    near(dx[0], want[0], TOL)
    near(dw, want[1], TOL)
    near(ds, want[2], TOL)
    if bias:
        near(db, want[3], TOL)
    else:
        assert db is None


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_short_conv_batch_in_place_and_steps(dtype):
    """A batch of equal rows; the state updated in place; steps that go on
    from a prompt give what one longer prompt gives, bit for bit."""
    g, B, T, C, W = Gen(5), 3, 41, 64, 4
    x, w, b = g.normal(B, T, C, dtype=dtype), g.normal(C, W), g.normal(C)
    s0 = g.normal(B, W - 1, C, dtype=dtype)
    out, fin = kda.short_conv_fwd(x, w, b, s0, activation="silu")
    st = s0.clone()
    o1, f1 = kda.short_conv_fwd(x[:, :30].contiguous(), w, b, st, activation="silu", final_state=st)
    assert f1.data_ptr() == st.data_ptr()
    assert torch.equal(o1, out[:, :30])
    for t in range(30, T):
        assert torch.equal(kda.short_conv_step(x[:, t].contiguous(), w, st, b, "silu"), out[:, t])
    assert torch.equal(st, fin)


# ---- state-space scan ----------------------------------------------------------

def scan_inputs(g, lead, D, S, G, dtype, gate=True, skip=True, bias=True):
    u, delta = g.normal(*lead, D, dtype=dtype), g.normal(*lead, D, dtype=dtype, std=0.5)
    A = -g.uniform(0.5, 4.0, D, S)
    B, C = g.normal(*lead, G, S, dtype=dtype), g.normal(*lead, G, S, dtype=dtype)
    opt = dict(D=g.normal(D) if skip else None, z=g.normal(*lead, D, dtype=dtype) if gate else None,
               delta_bias=g.uniform(-2.0, 0.0, D) if bias else None)
    return (u, delta, A, B, C), opt


def check_scan(lead, bounds, cu, args, opt, s0, d_out, d_fin, softplus=True):
    dtype, D = args[0].dtype, args[2].shape[0]
    out, fin = kda.ssm_scan_fwd(*args, **opt, initial_state=s0, cu_seqlens=cu, softplus=softplus)
    T = lead[0] * lead[1]
    flat = [wide(t.reshape(T, *t.shape[2:])) if i != 2 else wide(t) for i, t in enumerate(args)]
    skip, bias = wide(opt["D"]), wide(opt["delta_bias"])
    z = None if opt["z"] is None else wide(opt["z"].reshape(T, D))
    N = len(bounds) - 1
    ss = wide(s0) if s0 is not None else torch.zeros(N, *args[2].shape, dtype=torch.float64, requires_grad=True)
    o_ref, f_ref = ref.ssm_scan(*flat, skip, z, bias, ss, bounds, softplus)
    near(out.reshape(T, D), o_ref, SCAN_TOL)
    near(fin, f_ref, SCAN_TOL)
    names = ["du", "ddelta", "dA", "dB", "dC"] + [n for n, t in (("dD", skip), ("dz", z), ("dbias", bias)) if t is not None]
    want = ref.grads_of((o_ref, f_ref), (d_out.reshape(T, D).cpu().double(), None if d_fin is None else d_fin.cpu().double()),
                        flat + [t for t in (skip, z, bias) if t is not None] + [ss])
    got = kda.ssm_scan_bwd(*args, d_out, **opt, initial_state=s0, d_final_state=d_fin, cu_seqlens=cu,
                           softplus=softplus)
    for t, i in ((opt["D"], 5), (opt["z"], 6), (opt["delta_bias"], 7)):
        assert (got[i] is None) == (t is None)
    kept = [v for v in got[:8] if v is not None] + [got[8]]
    for name, v, r in zip(names + ["dstate"], kept, want):
        e = rel_fro(v.reshape(r.shape), r)
        assert torch.isfinite(v).all() and e <= SCAN_TOL, f"{name}: {e:.2e}"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,S,G", [(64, 16, 1), (40, 13, 2), (9, 3, 3), (130, 4, 1), (24, 8, 2), (20, 24, 1),
                                   (12, 64, 2), (5, 128, 1), (72, 1, 4)])
@pytest.mark.parametrize("lengths", [[1], [0, 17, 0, 1, 40, 16, 0]])
def test_ssm_scan(dtype, D, S, G, lengths):
    g, T, N = Gen(D + S), sum(lengths), len(lengths)
    args, opt = scan_inputs(g, (1, T), D, S, G, dtype)
    check_scan((1, T), ref.bounds_of(lengths), cu_of(lengths), args, opt, g.normal(N, D, S),
               g.normal(1, T, D, dtype=dtype), g.normal(N, D, S))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths", [[700], [300, 0, 1, 450, 64, 129]])
def test_ssm_scan_cut_sequences(dtype, lengths):
    """Few chains: the sequences are cut into units that run at once."""
    D, S = 36, 16
    g, T, N = Gen(9), sum(lengths), len(lengths)
    assert kda.ssm_scan_fwd_workspace_bytes(1, T, D, S, 1, N, True, dtype) > 0
    args, opt = scan_inputs(g, (1, T), D, S, 1, dtype)
    check_scan((1, T), ref.bounds_of(lengths), cu_of(lengths), args, opt, g.normal(N, D, S),
               g.normal(1, T, D, dtype=dtype), g.normal(N, D, S))


@pytest.mark.parametrize("gate,skip,bias,softplus,state", [(False, False, False, True, False),
                                                           (True, False, False, True, True),
                                                           (False, True, True, False, True)])
def test_ssm_scan_batch_and_options(gate, skip, bias, softplus, state):
    B, T, D, S = 2, 90, 32, 16
    g = Gen(17)
    args, opt = scan_inputs(g, (B, T), D, S, 1, F32, gate, skip, bias and softplus)
    if not softplus:
        args = (args[0], args[1].abs() + 0.05) + args[2:]
        opt["delta_bias"] = g.uniform(0.0, 0.1, D)
    check_scan((B, T), [0, T, 2 * T], None, args, opt, g.normal(B, D, S) if state else None,
               g.normal(B, T, D), g.normal(B, D, S) if state else None, softplus)


def test_ssm_scan_small_steps_keep_their_precision():
    """softplus far below zero: dt = e^x, relative to which log(1 + e^x) in
    fp32 would lose all digits."""
    g, T, D, S = Gen(23), 33, 16, 4
    args, opt = scan_inputs(g, (1, T), D, S, 1, F32, gate=False, skip=False)
    opt["delta_bias"] = g.uniform(-18.0, -12.0, D)
    check_scan((1, T), [0, T], None, args, opt, None, g.normal(1, T, D), None)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,D,S,G", [(1, 24, 16, 1), (7, 33, 13, 3), (300, 64, 8, 2), (2, 5, 128, 1), (3, 6, 1, 1)])
def test_ssm_step_goes_on_from_a_prompt(dtype, N, D, S, G):
    T, more = 20, 5
    g = Gen(31)
    args, opt = scan_inputs(g, (N, T + more), D, S, G, dtype)

    def part(t, a, b):
        return None if t is None else t[:, a:b].contiguous()

    def cut(a, b):
        return [part(t, a, b) if i != 2 else t for i, t in enumerate(args)], dict(opt, z=part(opt["z"], a, b))

    out, fin = kda.ssm_scan_fwd(*args, **opt, softplus=True)
    p, o = cut(0, T)
    _, st = kda.ssm_scan_fwd(*p, **o, softplus=True)
    for t in range(T, T + more):
        p, o = cut(t, t + 1)
        y = kda.ssm_step(*[v[:, 0] if i != 2 else v for i, v in enumerate(p)], st, D=o["D"], z=o["z"][:, 0],
                         delta_bias=o["delta_bias"], softplus=True)
        near(y, out[:, t].cpu().double(), SCAN_TOL + (2.0 ** -8 if dtype == BF16 else 0))
    near(st, fin.cpu().double(), SCAN_TOL)


# ---- group norm ----------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C,groups,silu,affine", [(128, 4, True, True), (40, 8, False, True), (33, 3, True, False),
                                                  (7, 7, False, True), (2400, 2, True, True), (5000, 1, False, True),
                                                  (96, 1, True, True)])
@pytest.mark.parametrize("lengths", [[1], [0, 3, 0, 200, 1, 64, 0]])
@pytest.mark.parametrize("per_token", [True, False])
def test_group_norm(dtype, C, groups, silu, affine, lengths, per_token):
    g, T = Gen(C), sum(lengths)
    x = (g.normal(1, T, C) + 3 * g.normal(C)).to(dtype)
    w, b = (1 + g.normal(C, std=0.2), g.normal(C)) if affine else (None, None)
    d_out = g.normal(1, T, C, dtype=dtype)
    act, cu = "silu" if silu else None, cu_of(lengths)
    bounds = list(range(T + 1)) if per_token else ref.bounds_of(lengths)
    out, mean, rstd = kda.group_norm_fwd(x, groups, w, b, 1e-5, act, per_token, cu)
    xs, ws, bs = wide(x[0]), wide(w), wide(b)
    o_ref, m_ref, r_ref = ref.group_norm(xs, groups, ws, bs, 1e-5, bounds, silu)
    single = C == groups and (per_token or lengths == [1])   # groups of one value: var = 0, xhat = 0
    near(out[0], o_ref, TOL)
    near(mean, m_ref, TOL)
    near(rstd, r_ref, TOL)
    dx, dw, db = kda.group_norm_bwd(x, groups, d_out, mean, rstd, w, b, act, per_token, cu)
    want = ref.grads_of((o_ref,), (d_out[0].cpu().double(),), [xs] + ([ws, bs] if affine else []))
    if single:
        # dx and dw are 0 up to the rounding of x - mean, times rstd = 1 / sqrt(eps)
        assert dx.abs().max() <= 1e-2 * rstd.max() * d_out.float().abs().max()
    else:
        near(dx[0], want[0], 4 * TOL)  # a difference of three terms of its own size
    if affine:
        if not single:
            near(dw, want[1], 2 * TOL)
        near(db, want[2], 2 * TOL)
    else:
        assert dw is None and db is None


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C,groups", [(435, 3), (501, 1), (690, 3), (514, 1), (1026, 2), (1025, 1), (2047, 1), (2050, 1), (4095, 1),
                                      (4097, 1), (8190, 1), (8188, 1), (8193, 1), (16400, 1), (8200, 1)])
def test_group_norm_rows_of_every_width(dtype, C, groups):
    """Rows that a warp, a block or neither holds, in vectors of each width."""
    test_group_norm(dtype, C, groups, True, True, [0, 3, 0, 200, 1, 64, 0], True)


def test_group_norm_far_mean():
    """A mean of 4096 standard deviations costs no more than x's own step."""
    g, T, C = Gen(3), 500, 64
    x = 4096 + g.normal(1, T, C)
    for per_token in (True, False):
        out, _, rstd = kda.group_norm_fwd(x, 4, per_token=per_token)
        bounds = list(range(T + 1)) if per_token else [0, T]
        o_ref, _, r_ref = ref.group_norm(x[0].cpu().double(), 4, None, None, 1e-5, bounds, False)
        # the mean is held in fp32: half a step of 4096 is 2^-12 of a deviation
        near(out[0], o_ref, 2.0 ** -12)
        near(rstd, r_ref, 2.0 ** -12)


# ---- all three together, and how they may be called ----------------------------

def layer(x, p, kda_call=True):
    """conv -> scan -> norm, forward, on packed sequences."""
    h, _ = kda.short_conv_fwd(x, p["w"], p["cb"], None, p["cu"], "silu")
    y, _ = kda.ssm_scan_fwd(h, p["delta"], p["A"], p["B"], p["C"], D=p["D"], z=p["z"], delta_bias=p["db"],
                            cu_seqlens=p["cu"], softplus=True)
    o, mean, rstd = kda.group_norm_fwd(y, p["groups"], p["gw"], p["gb"], per_token=True, cu_seqlens=p["cu"])
    return h, y, o, mean, rstd


def layer_params(g, lengths, D, S, G, groups, dtype):
    T = sum(lengths)
    (x, delta, A, B, C), opt = scan_inputs(g, (1, T), D, S, G, dtype)
    return x, dict(w=g.normal(D, 4, std=0.5), cb=g.normal(D, std=0.2), delta=delta, A=A, B=B, C=C, D=opt["D"],
                   z=opt["z"], db=opt["delta_bias"], cu=cu_of(lengths), groups=groups, gw=1 + g.normal(D, std=0.1),
                   gb=g.normal(D, std=0.1))


def test_layer_of_all_three_and_its_gradients():
    lengths, D, S = [37, 0, 90, 4], 48, 16
    g = Gen(77)
    x, p = layer_params(g, lengths, D, S, 2, 4, F32)
    bounds, T = ref.bounds_of(lengths), sum(lengths)
    h, y, o, mean, rstd = layer(x, p)
    leaves = {k: wide(p[k][0] if p[k].dim() > 1 and p[k].shape[0] == 1 else p[k])
              for k in ("w", "cb", "delta", "A", "B", "C", "D", "z", "db", "gw", "gb")}
    xs = wide(x[0])
    h_ref, _ = ref.short_conv(xs, leaves["w"], leaves["cb"], None, bounds, True)
    y_ref, _ = ref.ssm_scan(h_ref, leaves["delta"], leaves["A"], leaves["B"], leaves["C"], leaves["D"], leaves["z"],
                            leaves["db"], None, bounds, True)
    o_ref, _, _ = ref.group_norm(y_ref, 4, leaves["gw"], leaves["gb"], 1e-5, list(range(T + 1)), False)
    # a head of small variance enlarges what the scan's rounding left: 1 / sqrt(var) of a few
    near(o[0], o_ref, 4 * SCAN_TOL)
    d_o = g.normal(1, T, D)
    dy, dgw, dgb = kda.group_norm_bwd(y, 4, d_o, mean, rstd, p["gw"], p["gb"], per_token=True, cu_seqlens=p["cu"])
    dh, ddelta, dA, dB, dC, dD, dz, ddb, _ = kda.ssm_scan_bwd(
        h, p["delta"], p["A"], p["B"], p["C"], dy, D=p["D"], z=p["z"], delta_bias=p["db"], cu_seqlens=p["cu"],
        softplus=True)
    dx, dw, dcb, _ = kda.short_conv_bwd(x, p["w"], dh, p["cb"], None, None, p["cu"], "silu")
    got = [dx, dw, dcb, ddelta, dA, dB, dC, dD, dz, ddb, dgw, dgb]
    names = ["w", "cb", "delta", "A", "B", "C", "D", "z", "db", "gw", "gb"]
    want = ref.grads_of((o_ref,), (d_o[0].cpu().double(),), [xs] + [leaves[n] for n in names])
    for name, a, b in zip(["x"] + names, got, want):
        e = rel_fro(a.reshape(b.shape), b)
        assert e <= 8 * SCAN_TOL, f"d{name}: {e:.2e}"


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_results_do_not_change_from_run_to_run(dtype):
    g = Gen(12)
    lengths, D, S = [500, 3, 0, 260], 96, 16
    x, p = layer_params(g, lengths, D, S, 1, 8, dtype)
    d = g.normal(1, sum(lengths), D, dtype=dtype)

    def run():
        h, y, o, mean, rstd = layer(x, p)
        a = kda.group_norm_bwd(y, 8, d, mean, rstd, p["gw"], p["gb"], cu_seqlens=p["cu"], per_token=True)
        b = kda.ssm_scan_bwd(h, p["delta"], p["A"], p["B"], p["C"], d, D=p["D"], z=p["z"], delta_bias=p["db"],
                             cu_seqlens=p["cu"], softplus=True)
        c = kda.short_conv_bwd(x, p["w"], d, p["cb"], None, None, p["cu"], "silu")
        return [h, y, o, mean, rstd, *a, *b, *c]

    first = run()
    for _ in range(2):
        torch.empty(64 << 20, dtype=torch.uint8, device="cuda").fill_(255)  # other contents for what is allocated next
        for u, v in zip(first, run()):
            assert torch.equal(u, v)


def test_rows_of_no_sequence_stay_as_they_were():
    """A packed call whose sequences end before the last row."""
    g, T, D, S, used = Gen(4), 100, 32, 16, 71
    x, p = layer_params(g, [T], D, S, 1, 4, F32)
    cu = cu_of([40, 31])
    for t in (x, p["delta"], p["z"], p["B"], p["C"]):
        t[:, used:] = float("nan")

    def filled(*shape):
        return torch.full(shape, 7.0, device="cuda")

    out = filled(1, T, D)
    kda.short_conv_fwd(x, p["w"], p["cb"], None, cu, "silu", out=out)
    assert torch.isfinite(out).all() and (out[:, used:] == 7).all()
    args = (x, p["delta"], p["A"], p["B"], p["C"])
    opt = dict(D=p["D"], z=p["z"], delta_bias=p["db"], cu_seqlens=cu, softplus=True)
    kda.ssm_scan_fwd(*args, **opt, out=out)
    assert torch.isfinite(out).all() and (out[:, used:] == 7).all()
    d = g.normal(1, T, D)
    d[:, used:] = float("nan")
    grads = [filled(1, T, D), filled(1, T, D), filled(D, S), filled(1, T, 1, S), filled(1, T, 1, S), filled(D),
             filled(1, T, D), filled(D), filled(2, D, S)]
    kda.ssm_scan_bwd(*args, d, **opt, grads=grads)
    for t in grads:
        assert torch.isfinite(t).all()
    for i in (0, 1, 3, 4, 6):
        assert (grads[i][:, used:] == 7).all()
    grads = [filled(1, T, D), filled(D, 4), filled(D), filled(2, 3, D)]
    kda.short_conv_bwd(x, p["w"], d, p["cb"], None, None, cu, "silu", grads=grads)
    for t in grads:
        assert torch.isfinite(t).all()
    assert (grads[0][:, used:] == 7).all()
    out, mean, rstd = kda.group_norm_fwd(x, 4, p["gw"], p["gb"], cu_seqlens=cu, out=filled(1, T, D))
    assert torch.isfinite(out).all() and (out[:, used:] == 7).all()
    grads = [filled(1, T, D), filled(D), filled(D)]
    kda.group_norm_bwd(x, 4, d, mean, rstd, p["gw"], p["gb"], cu_seqlens=cu, grads=grads)
    for t in grads:
        assert torch.isfinite(t).all()
    assert (grads[0][:, used:] == 7).all()


def test_empty_calls():
    D, S = 16, 4
    z = torch.zeros(2, 0, D, device="cuda")
    bc = torch.zeros(2, 0, 1, S, device="cuda")
    A, w = -torch.ones(D, S, device="cuda"), torch.ones(D, 3, device="cuda")
    s0, c0 = torch.randn(2, D, S, device="cuda"), torch.randn(2, 2, D, device="cuda")
    out, fin = kda.ssm_scan_fwd(z, z, A, bc, bc, initial_state=s0)
    assert out.numel() == 0 and torch.equal(fin, s0)
    g = kda.ssm_scan_bwd(z, z, A, bc, bc, z, D=torch.ones(D, device="cuda"), d_final_state=s0)
    assert (g[2] == 0).all() and (g[5] == 0).all() and torch.equal(g[8], s0)
    out, fin = kda.short_conv_fwd(z, w, initial_state=c0)
    assert torch.equal(fin, c0)
    g = kda.short_conv_bwd(z, w, z, bias=torch.ones(D, device="cuda"), d_final_state=c0)
    assert (g[1] == 0).all() and (g[2] == 0).all() and torch.equal(g[3], c0)
    _, mean, rstd = kda.group_norm_fwd(z, 4, eps=0.25)
    assert (mean == 0).all() and (rstd == 2).all()
    g = kda.group_norm_bwd(z, 4, z, mean, rstd, torch.ones(D, device="cuda"))
    assert (g[1] == 0).all()
    out, mean, rstd = kda.group_norm_fwd(z, 4, per_token=True)
    assert mean.numel() == 0
    g = kda.group_norm_bwd(z, 4, z, mean, rstd, torch.ones(D, device="cuda"), per_token=True)
    assert (g[1] == 0).all()
    n = torch.zeros(0, D, device="cuda")
    assert kda.short_conv_step(n, w, torch.zeros(0, 2, D, device="cuda")).numel() == 0
    nb = torch.zeros(0, 1, S, device="cuda")
    assert kda.ssm_step(n, n, A, nb, nb, torch.zeros(0, D, S, device="cuda")).numel() == 0


def test_other_streams_and_graphs():
    """The same results on a side stream (given, and current), from two calls
    in flight at once, and from a captured graph replayed on new inputs."""
    g = Gen(41)
    lengths, D, S = [300, 200], 64, 16
    x, p = layer_params(g, lengths, D, S, 1, 4, BF16)
    want = layer(x, p)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    opt = dict(D=p["D"], z=p["z"], delta_bias=p["db"], cu_seqlens=p["cu"], softplus=True)
    outs = []
    for s in (a, b):
        h, _ = kda.short_conv_fwd(x, p["w"], p["cb"], None, p["cu"], "silu", stream=s)
        y, _ = kda.ssm_scan_fwd(h, p["delta"], p["A"], p["B"], p["C"], **opt, stream=s)
        o, m, r = kda.group_norm_fwd(y, 4, p["gw"], p["gb"], per_token=True, cu_seqlens=p["cu"], stream=s)
        outs.append((h, y, o, m, r))
    with torch.cuda.stream(a):
        outs.append(layer(x, p))
    torch.cuda.synchronize()
    for got in outs:
        for u, v in zip(got, want):
            assert torch.equal(u, v)

    d = g.normal(1, sum(lengths), D, dtype=BF16)

    def step():
        h, y, o, m, r = layer(x, p)
        return (o, *kda.ssm_scan_bwd(h, p["delta"], p["A"], p["B"], p["C"], d, **opt)[:8],
                *kda.group_norm_bwd(y, 4, d, m, r, p["gw"], p["gb"], cu_seqlens=p["cu"], per_token=True),
                *kda.short_conv_bwd(x, p["w"], d, p["cb"], None, None, p["cu"], "silu")[:3])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (1, 2):
        x.copy_(Gen(seed).normal(1, sum(lengths), D, dtype=BF16))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        for u, v in zip(got, step()):
            assert torch.equal(u, v)


def test_refusals_on_device():
    g = Gen(2)
    x, w = g.normal(2, 8, 16), g.normal(16, 4)
    with pytest.raises(ValueError, match="contiguous"):
        kda.short_conv_fwd(x.transpose(0, 1), w)
    with pytest.raises(TypeError):
        kda.short_conv_fwd(x, w.bfloat16())
    with pytest.raises(ValueError, match="shape"):
        kda.short_conv_fwd(x, w, initial_state=g.normal(2, 2, 16))
    with pytest.raises(binding.KDAError) as e:       # not 16-byte aligned
        flat = g.normal(2 * 8 * 16 + 1)
        kda.short_conv_fwd(flat[1:].view(2, 8, 16), w)
    assert e.value.status == binding.KDA_ERR_INVALID_ARG
    for bad in (lambda: kda.short_conv_fwd(x, w, out=x),                         # in place
                lambda: kda.short_conv_step(x[0], w, x.new_zeros(8, 3, 16), out=x[0])):
        with pytest.raises(binding.KDAError) as e:
            bad()
        assert e.value.status == binding.KDA_ERR_INVALID_ARG
    with pytest.raises(binding.KDAError) as e:
        kda.short_conv_fwd(x, g.normal(16, 5))
    assert e.value.status == binding.KDA_ERR_UNSUPPORTED
    args, opt = scan_inputs(g, (2, 8), 16, 4, 1, F32)
    with pytest.raises(binding.KDAError):
        kda.ssm_scan_fwd(*args, **opt, out=args[0])
    with pytest.raises(ValueError, match="workspace"):
        kda.ssm_scan_bwd(*args, x, **opt, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="grads"):
        kda.ssm_scan_bwd(*args, x, **opt, grads=[None] * 9)
    with pytest.raises(binding.KDAError):
        kda.group_norm_fwd(x, 4, out=x)
    with pytest.raises(binding.KDAError):
        kda.group_norm_fwd(x, 4, eps=0.0)
    torch.cuda.synchronize()
    assert binding.device_error() == binding.KDA_OK


def test_packed_call_without_sequences():
    """cu_seqlens = [0]: no sequence, no token."""
    D, S = 8, 4
    x, bc = torch.zeros(1, 0, D, device="cuda"), torch.zeros(1, 0, 1, S, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    A, w, k = -torch.ones(D, S, device="cuda"), torch.ones(D, 4, device="cuda"), torch.ones(D, device="cuda")
    out, fin = kda.ssm_scan_fwd(x, x, A, bc, bc, cu_seqlens=cu)
    assert out.shape == x.shape and fin.shape == (0, D, S)
    assert (kda.ssm_scan_bwd(x, x, A, bc, bc, x, cu_seqlens=cu)[2] == 0).all()
    out, fin = kda.short_conv_fwd(x, w, cu_seqlens=cu)
    assert fin.shape == (0, 3, D)
    assert (kda.short_conv_bwd(x, w, x, cu_seqlens=cu)[1] == 0).all()
    _, mean, rstd = kda.group_norm_fwd(x, 2, k, cu_seqlens=cu)
    assert mean.shape == (0, 2)
    assert (kda.group_norm_bwd(x, 2, x, mean, rstd, k, cu_seqlens=cu)[1] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_value_stays_in_its_sequence(bad):
    """The last token of the middle sequence is not finite: the others' rows are
    bit for bit what they are without it."""
    g = Gen(19)
    lengths, D, S = [45, 37, 50], 40, 16
    x, p = layer_params(g, lengths, D, S, 2, 4, F32)
    d = g.normal(1, sum(lengths), D)

    def run():
        h, y, o, mean, rstd = layer(x, p)
        args = (h, p["delta"], p["A"], p["B"], p["C"])
        b = kda.ssm_scan_bwd(*args, d, D=p["D"], z=p["z"], delta_bias=p["db"], cu_seqlens=p["cu"], softplus=True)
        n, m2, r2 = kda.group_norm_fwd(h, 4, p["gw"], p["gb"], cu_seqlens=p["cu"])
        c = kda.group_norm_bwd(h, 4, d, m2, r2, p["gw"], p["gb"], cu_seqlens=p["cu"])
        e = kda.short_conv_bwd(x, p["w"], d, p["cb"], None, None, p["cu"], "silu")
        return [h, y, o, b[0], b[1], b[3], b[4], b[6], n, c[0], e[0]]

    clean = run()
    x[0, 81, 7] = bad
    dirty = run()
    for u, v in zip(clean, dirty):
        assert torch.equal(u[:, :45], v[:, :45]) and torch.equal(u[:, 82:], v[:, 82:])
    # a finite state of +-inf inputs is not made NaN by the rows behind the end
    if bad == float("inf"):
        _, fin = kda.short_conv_fwd(x, p["w"], None, None, p["cu"])
        assert fin[1, 2, 7] == float("inf")
        h = p["delta"].clone()
        h[0, 81, 7] = bad
        B = p["B"].abs() + 0.1
        _, fin = kda.ssm_scan_fwd(h, p["delta"], p["A"], B, p["C"], cu_seqlens=p["cu"], delta_bias=p["db"], softplus=True)
        assert (fin[1, 7] == float("inf")).all()


def test_offsets_beyond_32_bits():
    """More than 2^31 values a tensor: the last rows are those of a call on them
    alone."""
    T, C = 1 << 20, 2176                       # 2.28e9 values, 4.6 GB in bf16
    x = torch.empty(1, T, C, dtype=BF16, device="cuda")
    for i in range(0, T, 1 << 16):
        x[0, i:i + (1 << 16)] = Gen(i).normal(1 << 16, C, dtype=BF16)
    g, tail = Gen(1), 96
    w, b = g.normal(C, 4), g.normal(C)
    out, fin = kda.short_conv_fwd(x, w, b, activation="silu")
    last = x[:, -tail - 3:].clone()
    want, _ = kda.short_conv_fwd(last, w, b, activation="silu")
    assert torch.equal(out[:, -tail:], want[:, -tail:]) and torch.equal(fin[0], x[0, -3:])
    kda.group_norm_fwd(x, 17, b, b, per_token=True, out=out)
    want, _, _ = kda.group_norm_fwd(last, 17, b, b, per_token=True)
    assert torch.equal(out[:, -tail:], want[:, -tail:])
    # a state that forgets within a few tokens: dt |A| of 8 and more
    A = torch.full((C, 4), -8.0, device="cuda")
    bc = g.normal(1, T, 1, 4, dtype=BF16)
    kda.ssm_scan_fwd(x, x, A, bc, bc, delta_bias=torch.full((C,), 8.0, device="cuda"), softplus=True, out=out)
    end = bc[:, -tail - 3:].clone()             # a view of these rows is not 16-byte aligned
    want, _ = kda.ssm_scan_fwd(last, last, A, end, end, delta_bias=torch.full((C,), 8.0, device="cuda"), softplus=True)
    near(out[0, -tail:], want[0, -tail:].cpu().double(), SCAN_TOL)


# ---- sizes that take the paths of large calls -----------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
def test_short_conv_large(dtype):
    """Long runs of tokens per thread, sequence ends inside them."""
    lengths, C, W = [9001, 1, 0, 6000, 2999], 1024, 4
    g, T, N = Gen(51), sum(lengths), len(lengths)
    x, w, b = g.normal(1, T, C, dtype=dtype), g.normal(C, W, std=0.5), g.normal(C)
    d_out, s0 = g.normal(1, T, C, dtype=dtype), g.normal(N, W - 1, C, dtype=dtype)
    cu, bounds = cu_of(lengths), ref.bounds_of(lengths)
    out, fin = kda.short_conv_fwd(x, w, b, s0, cu, "silu")
    leaves = [wide(x[0]), wide(w), wide(b), wide(s0)]
    o_ref, f_ref = ref.short_conv(*leaves, bounds, True)
    near(out[0], o_ref, TOL)
    assert torch.equal(fin.cpu().double(), f_ref.detach())
    want = ref.grads_of((o_ref,), (d_out[0].cpu().double(),), leaves)
    got = kda.short_conv_bwd(x, w, d_out, b, s0, None, cu, "silu")
    near(got[0][0], want[0], TOL)
    for u, v in zip(got[1:], want[1:]):
        near(u, v, 4 * TOL)      # sums over 18001 tokens


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_short_conv_step_large(dtype, W):
    """Two sequences a thread, the last one alone."""
    N, C = 1201, 1024
    g = Gen(52)
    x, w, b, st = g.normal(N, C, dtype=dtype), g.normal(C, W), g.normal(C), g.normal(N, W - 1, C, dtype=dtype)
    want, fin = kda.short_conv_fwd(x[:, None].contiguous(), w, b, st, activation="silu")
    assert torch.equal(kda.short_conv_step(x, w, st, b, "silu"), want[:, 0])
    assert torch.equal(st, fin)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("S,G", [(16, 2), (13, 1), (40, 1)])
def test_ssm_step_large(dtype, S, G):
    """Four sequences a thread, three for the last."""
    N, D = 4791, 64
    g = Gen(53)
    (u, d, A, B, C), opt = scan_inputs(g, (N, 1), D, S, G, dtype)
    st = g.normal(N, D, S)
    h, (dt, x) = st.double(), (torch.nn.functional.softplus(d[:, 0].double() + opt["delta_bias"]), u[:, 0].double())
    Bd, Cd = (m[:, 0].double().repeat_interleave(D // G, 1) for m in (B, C))
    h = torch.exp(dt[..., None] * A) * h + (dt * x)[..., None] * Bd
    y = (h * Cd).sum(-1) + opt["D"] * x
    z = opt["z"][:, 0].double()
    out = kda.ssm_step(u[:, 0], d[:, 0], A, B[:, 0], C[:, 0], st, D=opt["D"], z=opt["z"][:, 0],
                       delta_bias=opt["delta_bias"], softplus=True)
    near(out, (y * z * torch.sigmoid(z)).cpu(), TOL)
    near(st, h.cpu(), TOL)


@pytest.mark.parametrize("lengths", [None, [130, 40, 3, 100]])
def test_ssm_scan_many_chains(lengths):
    """Chains enough that sequences of one length stay whole, and ragged ones
    are cut at the mean."""
    D, S = 4096, 16
    g = Gen(54)
    lead = (4, 70) if lengths is None else (1, sum(lengths))
    assert (kda.ssm_scan_fwd_workspace_bytes(*lead, D, S, 1, 4, lengths is not None, BF16) == 0) == (lengths is None)
    args, opt = scan_inputs(g, lead, D, S, 1, BF16)
    bounds = ref.bounds_of(lengths or [70] * 4)
    check_scan(lead, bounds, cu_of(lengths) if lengths else None, args, opt, g.normal(4, D, S),
               g.normal(*lead, D, dtype=BF16), g.normal(4, D, S))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C,groups", [(256, 2), (72, 9), (1536, 1)])
@pytest.mark.parametrize("per_token", [True, False])
def test_group_norm_large(dtype, C, groups, per_token):
    """More rows than walkers, more tokens than a unit."""
    lengths = [7001, 0, 12000, 999]
    g, T = Gen(55), sum(lengths)
    x = (g.normal(1, T, C) + g.normal(C)).to(dtype)
    w, b, d_out = 1 + g.normal(C, std=0.2), g.normal(C), g.normal(1, T, C, dtype=dtype)
    cu = cu_of(lengths)
    out, mean, rstd = kda.group_norm_fwd(x, groups, w, b, 1e-5, "silu", per_token, cu)
    xs, ws, bs = wide(x[0]), wide(w), wide(b)
    if per_token:
        r = xs.view(T, groups, -1)
        m = r.mean(-1)
        rs = ((r - m[..., None]).square().mean(-1) + 1e-5).rsqrt()
        v = ((r - m[..., None]) * rs[..., None]).reshape(T, C) * ws + bs
        o_ref, m_ref, r_ref = v * torch.sigmoid(v), m, rs
    else:
        o_ref, m_ref, r_ref = ref.group_norm(xs, groups, ws, bs, 1e-5, ref.bounds_of(lengths), True)
    near(out[0], o_ref, TOL)
    near(mean, m_ref, 2 * TOL)   # means near zero of values near one
    near(rstd, r_ref, TOL)
    dx, dw, db = kda.group_norm_bwd(x, groups, d_out, mean, rstd, w, b, "silu", per_token, cu)
    want = ref.grads_of((o_ref,), (d_out[0].cpu().double(),), [xs, ws, bs])
    near(dx[0], want[0], 4 * TOL)
    near(dw, want[1], 4 * TOL)   # sums over 20000 tokens
    near(db, want[2], 4 * TOL)


def test_calls_with_every_buffer_given_allocate_nothing():
    """Outputs, states, gradients and workspaces of the caller: the results are
    the same, and neither the library nor the binding takes device memory."""
    g = Gen(61)
    lengths, D, S, groups = [300, 170], 96, 16, 4
    T, N = sum(lengths), len(lengths)
    x, p = layer_params(g, lengths, D, S, 2, groups, BF16)
    d = g.normal(1, T, D, dtype=BF16)
    args = (x, p["delta"], p["A"], p["B"], p["C"])
    opt = dict(D=p["D"], z=p["z"], delta_bias=p["db"], cu_seqlens=p["cu"], softplus=True)

    def f32(*shape):
        return torch.empty(shape, device="cuda")

    def space(n):
        assert n > 0
        return torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    out, conv_state, scan_state = torch.empty_like(x), torch.empty(N, 3, D, dtype=BF16, device="cuda"), f32(N, D, S)
    norm = (torch.empty_like(x), f32(N, groups), f32(N, groups))
    conv_grads = (f32(1, T, D), f32(D, 4), f32(D), f32(N, 3, D))
    scan_grads = (f32(1, T, D), f32(1, T, D), f32(D, S), f32(1, T, 2, S), f32(1, T, 2, S), f32(D), f32(1, T, D), f32(D),
                  f32(N, D, S))
    norm_grads = (f32(1, T, D), f32(D), f32(D))
    ws = [space(kda.ssm_scan_fwd_workspace_bytes(1, T, D, S, 2, N, True)),
          space(kda.ssm_scan_bwd_workspace_bytes(1, T, D, S, 2, N, True)),
          space(kda.short_conv_bwd_workspace_bytes(1, T, D, 4, N, True)),
          space(kda.group_norm_workspace_bytes(1, T, D, groups, N, True)),
          space(kda.group_norm_workspace_bytes(1, T, D, groups, N, True, backward=True))]

    def step():
        kda.short_conv_fwd(x, p["w"], p["cb"], None, p["cu"], "silu", out=out, final_state=conv_state)
        kda.short_conv_bwd(x, p["w"], d, p["cb"], None, None, p["cu"], "silu", grads=conv_grads, workspace=ws[2])
        kda.ssm_scan_fwd(*args, **opt, out=out, final_state=scan_state, workspace=ws[0])
        kda.ssm_scan_bwd(*args, d, **opt, grads=scan_grads, workspace=ws[1])
        kda.group_norm_fwd(x, groups, p["gw"], p["gb"], cu_seqlens=p["cu"], out=norm[0], mean=norm[1], rstd=norm[2],
                           workspace=ws[3])
        kda.group_norm_bwd(x, groups, d, norm[1], norm[2], p["gw"], p["gb"], cu_seqlens=p["cu"], grads=norm_grads,
                           workspace=ws[4])

    step()
    torch.cuda.synchronize()
    free, held = torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()
    for _ in range(2):
        step()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free and torch.cuda.memory_allocated() == held
    y, st = kda.ssm_scan_fwd(*args, **opt)
    assert torch.equal(out, y) and torch.equal(scan_state, st)
    for u, v in zip(scan_grads, kda.ssm_scan_bwd(*args, d, **opt)):
        assert torch.equal(u, v)
    for u, v in zip(norm_grads, kda.group_norm_bwd(x, groups, d, norm[1], norm[2], p["gw"], p["gb"], cu_seqlens=p["cu"])):
        assert torch.equal(u, v)
    for u, v in zip(conv_grads, kda.short_conv_bwd(x, p["w"], d, p["cb"], None, None, p["cu"], "silu")):
        assert torch.equal(u, v)


def test_workspaces_that_do_not_fit_are_refused():
    g = Gen(62)
    args, opt = scan_inputs(g, (1, 300), 32, 16, 1, F32)
    need = kda.ssm_scan_fwd_workspace_bytes(1, 300, 32, 16, 1, 1, False, F32)
    assert need > 0
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        kda.ssm_scan_fwd(*args, **opt, workspace=ws[:need - 1])
    with pytest.raises(binding.KDAError):             # not 256-byte aligned
        kda.ssm_scan_fwd(*args, **opt, workspace=ws[16:])
    big = torch.empty((1, 300, 32), device="cuda")
    with pytest.raises(binding.KDAError):             # the output's memory
        kda.ssm_scan_fwd(*args, **opt, out=big, workspace=torch.as_strided(
            big.view(torch.uint8), (max(need, 1),), (1,)) if need <= big.numel() * 4 else ws[16:])
    kda.ssm_scan_fwd(*args, **opt, workspace=ws)
