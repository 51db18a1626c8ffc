"""Plain 64-bit forms of the layer operators, token by token, on torch tensors
(differentiable), for the tests.  ``bounds`` lists where the packed sequences
begin and end."""
import torch


def bounds_of(lengths):
    b = [0]
    for n in lengths:
        b.append(b[-1] + n)
    return b


def short_conv(x, weight, bias, state, bounds, silu):
    """x [T,C], weight [C,W], state [N,W-1,C] or None -> (out, final state)."""
    W = weight.shape[1]
    outs, fins = [], []
    for n in range(len(bounds) - 1):
        rows = x[bounds[n]:bounds[n + 1]]
        head = x.new_zeros(W - 1, x.shape[1]) if state is None else state[n]
        ext = torch.cat([head, rows])
        L = rows.shape[0]
        v = sum(ext[j:j + L] * weight[:, j] for j in range(W))
        v = v if bias is None else v + bias
        outs.append(v * torch.sigmoid(v) if silu else v)
        fins.append(ext[L:])
    return torch.cat(outs), torch.stack(fins)


def ssm_scan(u, delta, A, B, C, skip, z, delta_bias, state, bounds, softplus):
    """u, delta, z [T,D], A [D,S], B, C [T,G,S], state [N,D,S] or None."""
    D, S = A.shape
    G = B.shape[1]
    raw = delta if delta_bias is None else delta + delta_bias
    dt = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    Bd, Cd = (m.repeat_interleave(D // G, dim=1) for m in (B, C))
    ys, fins = [], []
    for n in range(len(bounds) - 1):
        h = u.new_zeros(D, S) if state is None else state[n]
        for t in range(bounds[n], bounds[n + 1]):
            h = torch.exp(dt[t][:, None] * A) * h + (dt[t] * u[t])[:, None] * Bd[t]
            ys.append((h * Cd[t]).sum(-1))
        fins.append(h)
    y = torch.stack(ys) if ys else u.new_zeros(0, D)
    if skip is not None:
        y = y + skip * u
    return (y if z is None else y * z * torch.sigmoid(z)), torch.stack(fins)


def group_norm(x, groups, weight, bias, eps, bounds, silu):
    """x [T,C]; statistics over each of ``bounds``'s stretches and each group."""
    T, C = x.shape
    outs, means, rstds = [], [], []
    for a, b in zip(bounds, bounds[1:]):
        r = x[a:b].reshape(b - a, groups, C // groups)
        if a == b:
            means.append(x.new_zeros(groups))
            rstds.append(x.new_full((groups,), eps ** -0.5))
            continue
        m = r.mean((0, 2), keepdim=True)
        rs = ((r - m).square().mean((0, 2), keepdim=True) + eps).rsqrt()
        v = ((r - m) * rs).reshape(b - a, C)
        v = v if weight is None else v * weight
        v = v if bias is None else v + bias
        outs.append(v * torch.sigmoid(v) if silu else v)
        means.append(m[0, :, 0])
        rstds.append(rs[0, :, 0])
    out = torch.cat(outs) if outs else x.new_zeros(0, C)
    return out, torch.stack(means), torch.stack(rstds)


def grads_of(outputs, adjoints, inputs):
    """Gradients of sum(output . adjoint) by the inputs (zeros where none reaches)."""
    total = sum((o * a).sum() for o, a in zip(outputs, adjoints) if a is not None)
    got = torch.autograd.grad(total, inputs, allow_unused=True)
    return [torch.zeros_like(i) if g is None else g for g, i in zip(got, inputs)]
