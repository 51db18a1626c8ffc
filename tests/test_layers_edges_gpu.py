"""The layer operators where they can go wrong: states updated in place, and
the paths and values that the tests of the usual calls do not reach.

Tolerances are those of test_layers_gpu unless a test derives its own.
"""
import pytest
import torch

import gated_delta_rule_103_b200 as kda
import layer_reference as ref
import test_layers_gpu as base

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


# ---- states in place -------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths,packed,D,S,cut", [
    ([129], False, 1536, 16, True),            # five units, the last one of one token
    ([449, 449, 449], False, 96, 13, True),
    ([300, 0, 1, 450, 64, 129], True, 40, 16, True),
    ([0, 1, 700, 33], True, 9, 3, True),
    ([70, 70, 70, 70], False, 4096, 16, False),
    ([5, 0, 17], True, 24, 128, False)])
def test_ssm_scan_state_in_place(dtype, lengths, packed, D, S, cut):
    """final_state equal to initial_state: bit for bit the results of separate
    memory, whether or not sequences are cut into units."""
    g, N, T = base.Gen(71), len(lengths), sum(lengths)
    lead = (1, T) if packed else (N, lengths[0])
    assert (kda.ssm_scan_fwd_workspace_bytes(*lead, D, S, 1, N, packed, dtype) > 0) == cut
    args, opt = base.scan_inputs(g, lead, D, S, 1, dtype)
    cu = base.cu_of(lengths) if packed else None
    s0 = g.normal(N, D, S)
    out, fin = kda.ssm_scan_fwd(*args, **opt, initial_state=s0, cu_seqlens=cu, softplus=True)
    for _ in range(3):
        st = s0.clone()
        o, f = kda.ssm_scan_fwd(*args, **opt, initial_state=st, final_state=st, cu_seqlens=cu, softplus=True)
        assert f.data_ptr() == st.data_ptr()
        assert torch.equal(o, out) and torch.equal(st, fin)


# ---- values at the ends of their range ---------------------------------------------

@pytest.mark.parametrize("lengths,cut", [([17, 0, 40, 1], False), ([700, 129], True)])
@pytest.mark.parametrize("S", [13, 16])
def test_ssm_scan_state_that_forgets_at_once(lengths, cut, S):
    """A = -inf (an -exp(A_log) that overflowed): the state is what the last
    token put there.  Steps are above 0.01, so that A = -1e6 has the same decay,
    zero, in 64 bits, and finite terms in the gradients' formulas."""
    D, N, T = 24, len(lengths), sum(lengths)
    g, bounds = base.Gen(72), ref.bounds_of(lengths)
    assert not cut or kda.ssm_scan_fwd_workspace_bytes(1, T, D, S, 1, N, True, F32) > 0
    args, opt = base.scan_inputs(g, (1, T), D, S, 1, F32)
    args, cu = list(args), base.cu_of(lengths)
    at_once = g.uniform(0.0, 1.0, D, S) < 0.3
    s0, d_out, d_fin = g.normal(N, D, S), g.normal(1, T, D), g.normal(N, D, S)
    leaves = [base.wide(t[0] if i != 2 else torch.where(at_once, -1e6, t)) for i, t in enumerate(args)]
    leaves += [base.wide(opt["D"]), base.wide(opt["z"][0]), base.wide(opt["delta_bias"]), base.wide(s0)]
    assert float(torch.nn.functional.softplus(leaves[1] + leaves[7]).detach().min()) > 0.01
    o_ref, f_ref = ref.ssm_scan(*leaves[:8], leaves[8], bounds, True)
    want = ref.grads_of((o_ref, f_ref), (d_out[0].cpu().double(), d_fin.cpu().double()), leaves)
    for A in (float("-inf"), -3e38):
        args[2] = torch.where(at_once, A, args[2])
        out, fin = kda.ssm_scan_fwd(*args, **opt, initial_state=s0, cu_seqlens=cu, softplus=True)
        base.near(out[0], o_ref, base.SCAN_TOL)
        base.near(fin, f_ref, base.SCAN_TOL)
        got = kda.ssm_scan_bwd(*args, d_out, **opt, initial_state=s0, d_final_state=d_fin, cu_seqlens=cu, softplus=True)
        for v, r in zip(got, want):
            base.near(v.reshape(r.shape), r, base.SCAN_TOL)
        st = s0.clone()
        for t in range(lengths[0]) if not cut else ():
            one = [v[:, t].clone() if i != 2 else v for i, v in enumerate(args)]   # aligned, as a slice is not
            y = kda.ssm_step(*one, st[:1], D=opt["D"], z=opt["z"][:, t].clone(),
                             delta_bias=opt["delta_bias"], softplus=True)
            base.near(y[0], o_ref[t], 4 * base.SCAN_TOL)


# ---- long memories -----------------------------------------------------------------

@pytest.mark.parametrize("log_memory", [6, 7, 8, 10, 11, 12])
def test_ssm_scan_long_memory(log_memory):
    """Sequences that are not cut, of states that remember M tokens and terms of
    one sign, so that the decays' errors do not cancel.

    A decay is off by up to 2^-24 of its value in the mean square (a step just
    below one is 2^-24, and the fast 2^x is good to about that) and its mean by
    what the exponent's constant leaves: at most 1e-9 where M is above 2^9, 1e-8
    below.  A state of M tokens carries sqrt(M / 2) times the one and M times
    the other."""
    M, D, S = 1 << log_memory, 2048, 128
    T, g = 3 * M, base.Gen(81)
    assert kda.ssm_scan_fwd_workspace_bytes(1, T, D, S, 1, 1, False, F32) == 0
    dt = g.uniform(0.75, 1.25, 1, T, D) * (1.4 / M)
    A, u, B = -g.uniform(1.0, 2.0, D, S) / 1.4, 1 / dt, torch.ones(1, T, 1, S, device="cuda")
    _, fin = kda.ssm_scan_fwd(u, dt, A, B, B)
    A64, h = A.double(), torch.zeros(D, S, dtype=torch.float64, device="cuda")
    step, du = dt[0].double(), (dt[0].double() * u[0].double())
    for t in range(T):
        h = torch.exp(step[t][:, None] * A64).mul_(h).add_(du[t][:, None])
    e = float(((fin[0] - h) / h).square().mean().sqrt())
    tol = 2.0 ** -24 * (M / 2) ** 0.5 + M * (1e-9 if log_memory > 9 else 1e-8)
    assert e <= tol, f"{e:.2e} > {tol:.2e}"


def test_ssm_step_of_nothing_keeps_the_state():
    """dt = 0: a decay of one, bit for bit, for every rate."""
    g, N, D, S = base.Gen(82), 8, 512, 16
    A, st, zero = -torch.exp(g.normal(D, S, std=4.0)), g.normal(N, D, S), torch.zeros(N, D, device="cuda")
    A[:, :4] = torch.tensor([0.0, 1.0, float("-inf"), -3e38], device="cuda")
    want, B = st.clone(), g.normal(N, 1, S)
    kda.ssm_step(g.normal(N, D), zero, A, B, B, st)
    assert torch.equal(st, want)
    many = torch.zeros(N, 50, D, device="cuda")
    _, fin = kda.ssm_scan_fwd(many, many, A, B.expand(N, 50, S)[:, :, None].contiguous(),
                              B.expand(N, 50, S)[:, :, None].contiguous(), initial_state=st)
    assert torch.equal(fin, want)


# ---- the activations' functions -----------------------------------------------------

STEP = 2.0 ** -24      # half a step of fp32, relative


def exp_error(x):
    """e^x is good to 2^-22 (the fast 2^x) and |x| times the rounding of x log2 e
    (2^-24) and of the constant (0.22 2^-24): in half steps."""
    return 4 + 1.25 * x.abs()


def test_fp32_silu_and_its_slope():
    """Value by value over the whole range of e^x, through the convolution with
    weights 0 and 1.  silu = v / (1 + e^-v): what e^-v is off by, a sum (1), a
    reciprocal (2) and a product (1).  slope = s (1 + v (1 - s)): s (3 and e^-v's),
    1 - s as far off as s and rounded, times v s, and three roundings."""
    x = torch.linspace(-80, 80, 1 << 20, device="cuda").reshape(1, -1, 4).contiguous()
    w = torch.tensor([0.0, 1.0], device="cuda").expand(4, 2).contiguous()
    out, _ = kda.short_conv_fwd(x, w, activation="silu")
    v = x.double()
    s = torch.sigmoid(v)
    off = exp_error(v) * (1 - s)                       # of e^-v / (1 + e^-v)
    assert float(((out - v * s) / (v * s)).abs().div(off + 4).max()) <= STEP
    dx = kda.short_conv_bwd(x, w, torch.ones_like(x), activation="silu")[0]
    slope = s * (1 + v * (1 - s))
    assert float(((dx - slope).abs() / ((off + 6) * slope.abs() + ((off + 3) * s + 1) * v.abs() * s)).max()) <= STEP
    b = x[0, 5].clone()
    normed = kda.group_norm_fwd(x, 4, torch.zeros(4, device="cuda"), b, activation="silu", per_token=True)[0]
    want = (b.double() * torch.sigmoid(b.double())).expand_as(normed)
    assert float(((normed - want) / want).abs().max()) <= float(exp_error(b).max() + 4) * STEP


def test_fp32_softplus_keeps_its_precision_far_below_zero():
    """The step alone, as the state that a token leaves in an empty one (u = B =
    1).  What e^-|x| is off by, a sum (1), a reciprocal (2), four roundings around
    the series, 3e-9 that it leaves out."""
    D = 1 << 16
    x = torch.linspace(-80, 20, D, device="cuda").reshape(1, D)
    one, st = torch.ones_like(x), torch.zeros(1, D, 1, device="cuda")
    A, B = -torch.ones(D, 1, device="cuda"), torch.ones(1, 1, 1, device="cuda")
    kda.ssm_step(one, x, A, B, B, st, softplus=True)
    want, tol = torch.logaddexp(x.double(), torch.zeros_like(x.double())), (exp_error(x) + 8) * STEP
    assert float(((st[..., 0] - want).abs() / want / tol).max()) <= 1
    # and in a scan, whose series runs on two values at a time
    fin = kda.ssm_scan_fwd(one[None], x[None], A, B[None], B[None], softplus=True)[1]
    assert float(((fin[..., 0] - want).abs() / want / tol).max()) <= 1


# ---- sums over many tokens -----------------------------------------------------------

# A rounding to fp32 is uniform within half a step, which is 2^-25 to 2^-24 of the
# value: 0.42 2^-24 in the mean square.
ROUNDING = 0.42 * 2.0 ** -24


@pytest.mark.parametrize("T,C,groups", [(26884, 784, 8), (16384, 1024, 32), (8192, 4096, 1), (32768, 258, 2)])
def test_group_norm_parameter_sums_per_token(T, C, groups):
    """dbias is the plain sum of d_out: chains of 8 rows, then of a walker's
    rows / 8 (at most 32 where the kernels hold 444 and more), then 64 bits.  The
    n-th partial sum of random terms is sqrt(n / N) of the whole, so a chain of N
    costs sqrt(N / 2) roundings.  Twice that, for what is not in the mean."""
    g = base.Gen(91)
    x, d = g.normal(1, T, C), g.normal(1, T, C)
    w, b = torch.ones(C, device="cuda"), torch.zeros(C, device="cuda")
    _, mean, rstd = kda.group_norm_fwd(x, groups, w, b, per_token=True)
    _, dw, db = kda.group_norm_bwd(x, groups, d, mean, rstd, w, b, per_token=True)
    tol = 2 * ROUNDING * (8 / 2 + 8 / 2 + 1) ** 0.5
    d64, x64 = d[0].double(), x[0].double().view(T, groups, -1)
    assert base.rel_fro(db, d64.sum(0).cpu()) <= tol
    # dweight: xhat's own two roundings beside the mean's and rstd's, up to 2^-24 each
    xh = (x64 - x64.mean(-1, keepdim=True)) / (x64.var(-1, correction=0, keepdim=True) + 1e-5).sqrt()
    assert base.rel_fro(dw, (xh.view(T, C) * d64).sum(0).cpu()) <= tol + 2 * 2.0 ** -24


def test_group_norm_statistics_of_long_sequences():
    """rstd is rounded once where its parts are added up in 64 bits; a sequence's
    170 threads leave the mean of their sums' roundings (of squares: chains of 32
    and 16 terms, sqrt(48 / 3) each, half of it in the root).  Half as much again."""
    N, T, C, groups = 11, 2182, 640, 32
    g = base.Gen(92)
    x = g.normal(N, T, C) + g.normal(C)
    _, _, rstd = kda.group_norm_fwd(x, groups)
    want = (x.double().view(N, T, groups, -1).var((1, 3), correction=0) + 1e-5).rsqrt()
    assert base.rel_fro(rstd, want.cpu()) <= 1.5 * ROUNDING * (1 + 4 / 2 / 170 ** 0.5)


# ---- single tokens ------------------------------------------------------------------

@pytest.mark.parametrize("N", [3, 5000])
@pytest.mark.parametrize("D,S", [(65, 16), (7, 5), (300, 128), (257, 3)])
def test_ssm_step_channels_that_do_not_fill_a_block(N, D, S):
    """Threads behind the last channel: the states, channel 0's among them, and
    the outputs are those of a scan over one token."""
    if N * D * S > 1 << 25:
        N = 300
    g = base.Gen(95)
    args, opt = base.scan_inputs(g, (N, 1), D, S, 1, F32)
    st = g.normal(N, D, S)
    out, fin = kda.ssm_scan_fwd(*args, **opt, initial_state=st, softplus=True)
    one = [t[:, 0].contiguous() if i != 2 else t for i, t in enumerate(args)]
    y = kda.ssm_step(*one, st, D=opt["D"], z=opt["z"][:, 0].contiguous(), delta_bias=opt["delta_bias"], softplus=True)
    base.near(st, fin.double().cpu(), 8 * STEP)     # the same decays and terms, a product apart
    base.near(y, out[:, 0].double().cpu(), S * STEP + 8 * STEP)


@pytest.mark.parametrize("T,C", [(131072, 64), (65536, 33)])
def test_short_conv_parameter_sums(T, C):
    """dbias is the plain sum of d_out: a thread's run of up to 32 tokens, then a
    block's up to 256 runs, then 64 bits; dweight has a rounded product fused into
    the first.  A chain of N costs sqrt(N / 2) roundings, a chain over runs none
    that the run's own share does not shrink: half as much again in all."""
    g = base.Gen(96)
    x, d, w = g.normal(1, T, C), g.normal(1, T, C), g.normal(C, 4)
    _, dw, db, _ = kda.short_conv_bwd(x, w, d, bias=torch.zeros(C, device="cuda"), need_initial_state_grad=False)
    d64 = d[0].double()
    tx = 1
    while tx < min(32, -(-C // (4 if C % 4 == 0 else 1))):
        tx *= 2
    tol = 1.5 * ROUNDING * (32 / 2 + 256 // tx / 2 + 1) ** 0.5
    assert base.rel_fro(db, d64.sum(0).cpu()) <= tol
    ext = torch.nn.functional.pad(x[0].double(), (0, 0, 3, 0))
    want = torch.stack([(ext[j:j + T] * d64).sum(0) for j in range(4)], 1)
    assert base.rel_fro(dw, want.cpu()) <= tol


# ---- paths of the scan that no usual case takes ---------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("T,D,S,G", [(333, 40, 16, 2), (449, 21, 3, 1), (150, 130, 100, 1)])
def test_ssm_scan_cut_batch(dtype, state, T, D, S, G):
    """A batch of equal sequences, cut: each row's units, entry states and final
    state are its own."""
    N = 3
    assert kda.ssm_scan_fwd_workspace_bytes(N, T, D, S, G, N, False, dtype) > 0
    g = base.Gen(97)
    args, opt = base.scan_inputs(g, (N, T), D, S, G, dtype)
    base.check_scan((N, T), [T * i for i in range(N + 1)], None, args, opt, g.normal(N, D, S) if state else None,
                    g.normal(N, T, D, dtype=dtype), g.normal(N, D, S) if state else None)


@pytest.mark.parametrize("S", [3, 16, 100])
def test_ssm_scan_steps_of_nothing_behind_a_token(S):
    """A token of any size, then dt = 0: the state and what is read from it stay,
    bit for bit, through the rest of its tile and the next ones; so do adjoints
    on their way back."""
    g, T, D = base.Gen(98), 37, 64
    A, B, C = -g.uniform(0.001, 4.0, D, S), g.normal(1, T, 1, S), g.normal(1, 1, 1, S).expand(1, T, 1, S).contiguous()
    u, dt, s0 = g.normal(1, T, D), torch.zeros(1, T, D, device="cuda"), g.normal(1, D, S)
    dt[:, 0] = g.uniform(0.001, 2.0, D)
    out, fin = kda.ssm_scan_fwd(u, dt, A, B, C, initial_state=s0)
    one, first = kda.ssm_scan_fwd(u[:, :1].clone(), dt[:, :1].clone(), A, B[:, :1].clone(), C[:, :1].clone(),
                                  initial_state=s0)
    assert torch.equal(fin, first)
    assert torch.equal(out, one.expand(1, T, D))
    d_fin = g.normal(1, D, S)
    ds = kda.ssm_scan_bwd(u, dt, A, B, C, torch.zeros_like(u), initial_state=s0, d_final_state=d_fin)[8]
    ds1 = kda.ssm_scan_bwd(u[:, :1].clone(), dt[:, :1].clone(), A, B[:, :1].clone(), C[:, :1].clone(),
                           torch.zeros(1, 1, D, device="cuda"), initial_state=s0, d_final_state=d_fin)[8]
    assert torch.equal(ds, ds1)
