"""Binding of the layer operators around the recurrences (``include/kda.h``):
the short causal convolution, the selective state-space scan and the group
norm, each with its backward pass and, where it carries a state, its one-token
step.

As in ``binding.py`` this only checks and marshals arguments.  Tensors must be
contiguous CUDA tensors of the current device; per-token tensors are bfloat16
or float32, parameters, scan states, statistics and gradients float32.
Without ``stream`` the calls run on the current stream; with it, what the call
allocates belongs to that stream too.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from .binding import (KDA_DTYPE_BF16, KDA_DTYPE_F32, KDA_FLAG_PER_TOKEN, KDA_FLAG_SILU,
                      KDA_FLAG_SOFTPLUS, KDAError, load_library)

_F32, _BF16 = torch.float32, torch.bfloat16
_INT_MAX = 2 ** 31 - 1
_ACTIVATIONS = {None: 0, "silu": KDA_FLAG_SILU}


# A one-token call takes about as long to check and marshal as to run, so what
# follows does one plain attribute test after the other.

def _dtype(t: torch.Tensor, name: str) -> int:
    if t.dtype is _BF16:
        return KDA_DTYPE_BF16
    if t.dtype is _F32:
        return KDA_DTYPE_F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _take(t: Optional[torch.Tensor], name: str, shape, dtype) -> Optional[int]:
    """The checked tensor's address (None for None)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (no CPU fallback)")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _sequences(cu: Optional[torch.Tensor], B: int) -> Tuple[Optional[int], int]:
    """(address of cu_seqlens, number of sequences)."""
    if cu is None:
        return None, B
    if cu.dtype != torch.int32 or cu.dim() != 1 or cu.numel() < 1:
        raise TypeError("cu_seqlens must be a 1-D int32 tensor of N + 1 bounds")
    if B != 1:
        raise ValueError("packed sequences need a batch of 1")
    _rank(cu, "cu_seqlens", 1)
    return _take(cu, "cu_seqlens", cu.shape, torch.int32), cu.numel() - 1


def _activation(name) -> int:
    try:
        return _ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be None or 'silu', got {name!r}") from None


def _rank(t: torch.Tensor, name: str, n: int):
    shape = t.shape
    if len(shape) != n:
        raise ValueError(f"{name} must have {n} dimensions, got {len(shape)}")
    for size in shape:
        if size > _INT_MAX:       # ctypes would take it modulo 2^32
            raise ValueError(f"{name} must have sizes below 2^31, got {tuple(shape)}")
    return shape


def _bytes(f, dtype, *sizes) -> int:
    """A workspace query; 0, as for every size that a call refuses, where one is
    no int of the library's."""
    if not all(-1 < n <= _INT_MAX for n in sizes):
        return 0
    dt = KDA_DTYPE_BF16 if dtype == torch.bfloat16 else KDA_DTYPE_F32
    return int(f(*sizes, dt))


class _On:
    """What a call allocates, it allocates for the stream that it runs on."""

    __slots__ = ("context",)

    def __init__(self, stream):
        self.context = None if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        if self.context is not None:
            self.context.__enter__()

    def __exit__(self, *error):
        if self.context is not None:
            self.context.__exit__(*error)


def _out(x: torch.Tensor, stream) -> torch.Tensor:
    if stream is None:
        return torch.empty_like(x)
    with _On(stream):
        return torch.empty_like(x)


def _raw(stream, t: torch.Tensor) -> int:
    """The stream's handle: the given one, or the current one of t's device
    (the library refuses tensors of another device than the current one)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else stream.cuda_stream


def _check(status: int, where: str):
    if status:
        raise KDAError(status, where)


def _given(grads, shapes):
    """Checked addresses of the caller's gradients."""
    return [_take(t, "grads", s, _F32) for t, s in zip(grads, shapes)]


def _like(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """fp32 memory of an input's shape (the quickest way to allocate it)."""
    return None if t is None else torch.empty_like(t, dtype=_F32)


def _state(given: Optional[torch.Tensor], shape, dtype, x: torch.Tensor) -> torch.Tensor:
    if given is not None:
        return torch.empty_like(given, dtype=dtype)
    return torch.empty(shape, dtype=dtype, device=x.device)


def _space(need: int, workspace: Optional[torch.Tensor], device):
    if need == 0:
        return None, 0, None
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif (not workspace.is_cuda or workspace.dtype != torch.uint8 or not workspace.is_contiguous()
          or workspace.numel() < need):
        raise ValueError(f"workspace must be a contiguous uint8 CUDA tensor of >= {need} bytes")
    return workspace.data_ptr(), workspace.numel(), workspace


# ---- short convolution -------------------------------------------------------

def short_conv_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   initial_state: Optional[torch.Tensor] = None,
                   cu_seqlens: Optional[torch.Tensor] = None, activation: Optional[str] = None,
                   output_final_state: bool = True, out: Optional[torch.Tensor] = None,
                   final_state: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Causal depthwise convolution over the last W tokens
    (``kda_short_conv_fwd``): ``v[t] = bias + sum_j weight[:, j] x[t-W+1+j]``,
    then ``activation`` (None or "silu").

    x [B,T,C] in bf16 or fp32, weight [C,W] (W = 2, 3, 4) and bias [C] fp32,
    initial_state [N,W-1,C] (x's type; the rows before each sequence, zeros
    when None), cu_seqlens [N+1] int32 (B must be 1) or None.  Returns
    ``(out, final_state)``; ``final_state`` may be passed equal to
    ``initial_state`` to update it in place.
    """
    lib = load_library()
    B, T, C = _rank(x, "x", 3)
    dt, dtype = _dtype(x, "x"), x.dtype
    W = _rank(weight, "weight", 2)[1]
    cu, N = _sequences(cu_seqlens, B)
    flags = _activation(activation)
    state = (N, W - 1, C)
    px, pw = _take(x, "x", x.shape, dtype), _take(weight, "weight", (C, W), _F32)
    pb, ps = _take(bias, "bias", (C,), _F32), _take(initial_state, "initial_state", state, dtype)
    with _On(stream):
        if out is None:
            out = torch.empty_like(x)
        if final_state is None and output_final_state:
            final_state = _state(initial_state, state, dtype, x)
        _check(lib.kda_short_conv_fwd(px, pw, pb, ps, cu, _take(out, "out", x.shape, dtype),
                                      _take(final_state, "final_state", state, dtype),
                                      B, T, C, W, N, dt, flags, _raw(stream, x)), "kda_short_conv_fwd")
    return out, final_state


def short_conv_step(x: torch.Tensor, weight: torch.Tensor, state: torch.Tensor,
                    bias: Optional[torch.Tensor] = None, activation: Optional[str] = None,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of ``short_conv_fwd`` for each of N sequences
    (``kda_short_conv_step``): x [N,C]; ``state`` [N,W-1,C] (x's type) is
    shifted in place.  Returns out [N,C]."""
    lib = load_library()
    N, C = _rank(x, "x", 2)
    dt, dtype = _dtype(x, "x"), x.dtype
    W = _rank(weight, "weight", 2)[1]
    flags = _activation(activation)
    px, pw = _take(x, "x", x.shape, dtype), _take(weight, "weight", (C, W), _F32)
    pb, ps = _take(bias, "bias", (C,), _F32), _take(state, "state", (N, W - 1, C), dtype)
    if out is not None:
        po = _take(out, "out", x.shape, dtype)
    else:
        out = _out(x, stream)
        po = out.data_ptr()
    _check(lib.kda_short_conv_step(px, pw, pb, ps, po, N, C, W, dt, flags, _raw(stream, x)),
           "kda_short_conv_step")
    return out


def short_conv_bwd_workspace_bytes(B: int, T: int, C: int, W: int, N: int, packed: bool,
                                   dtype=torch.bfloat16) -> int:
    """``kda_short_conv_bwd_workspace_bytes`` (``packed``: cu_seqlens is passed)."""
    return _bytes(load_library().kda_short_conv_bwd_workspace_bytes, dtype, B, T, C, W, N, int(packed))


def short_conv_bwd(x: torch.Tensor, weight: torch.Tensor, d_out: torch.Tensor,
                   bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                   d_final_state: Optional[torch.Tensor] = None,
                   cu_seqlens: Optional[torch.Tensor] = None, activation: Optional[str] = None,
                   need_initial_state_grad: bool = True, grads=None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward pass of ``short_conv_fwd`` (``kda_short_conv_bwd``).

    Inputs as there plus ``d_out`` (shaped and typed like x) and
    ``d_final_state`` [N,W-1,C] fp32 or None (zero).  Returns fp32 ``(dx,
    dweight, dbias, d_initial_state)``; dbias is None without a bias, the last
    is None when ``need_initial_state_grad`` is false.  ``grads``: the caller's
    four output tensors instead of new ones (a None there leaves that gradient
    out, which dx and dweight do not allow).
    """
    lib = load_library()
    B, T, C = _rank(x, "x", 3)
    dt, dtype = _dtype(x, "x"), x.dtype
    W = _rank(weight, "weight", 2)[1]
    cu, N = _sequences(cu_seqlens, B)
    flags = _activation(activation)
    state = (N, W - 1, C)
    ins = (_take(x, "x", x.shape, dtype), _take(weight, "weight", (C, W), _F32),
           _take(bias, "bias", (C,), _F32), _take(initial_state, "initial_state", state, dtype), cu,
           _take(d_out, "d_out", x.shape, dtype), _take(d_final_state, "d_final_state", state, _F32))
    shapes = ((B, T, C), (C, W), (C,), state)
    with _On(stream):
        given = grads is not None
        if not given:
            grads = (_like(x), _like(weight), _like(bias),
                     _state(initial_state, state, _F32, x) if need_initial_state_grad else None)
        dx, dw, db, ds = grads
        if dx is None or dw is None:
            raise ValueError("grads must hold dx and dweight")
        outs = _given(grads, shapes) if given else [None if t is None else t.data_ptr() for t in grads]
        ws, size, _keep = _space(
            int(lib.kda_short_conv_bwd_workspace_bytes(B, T, C, W, N, cu is not None, dt)), workspace,
            x.device)
        _check(lib.kda_short_conv_bwd(*ins, *outs, B, T, C, W, N, dt, flags, ws, size, _raw(stream, x)),
               "kda_short_conv_bwd")
    return dx, dw, db, ds


# ---- state-space scan --------------------------------------------------------

def ssm_scan_fwd_workspace_bytes(B: int, T: int, D: int, S: int, G: int, N: int, packed: bool,
                                 dtype=torch.bfloat16) -> int:
    """``kda_ssm_scan_fwd_workspace_bytes`` (0: the call needs none)."""
    return _bytes(load_library().kda_ssm_scan_fwd_workspace_bytes, dtype, B, T, D, S, G, N, int(packed))


def ssm_scan_bwd_workspace_bytes(B: int, T: int, D: int, S: int, G: int, N: int, packed: bool,
                                 dtype=torch.bfloat16) -> int:
    """``kda_ssm_scan_bwd_workspace_bytes``."""
    return _bytes(load_library().kda_ssm_scan_bwd_workspace_bytes, dtype, B, T, D, S, G, N, int(packed))


def _scan_inputs(u, delta, A, B, C, D, z, delta_bias, lead: int):
    """Addresses of the scan's inputs, checked against u's leading dimensions."""
    shape, dtype = u.shape, u.dtype
    ch = shape[-1]
    S = _rank(A, "A", 2)[1]
    bc = _rank(B, "B", lead + 2)
    G = bc[lead]
    if bc != (*shape[:lead], G, S) or G < 1 or ch % G:
        raise ValueError("B must be [..., G, S] with u's leading dimensions, A's S and G dividing the channels")
    return (_take(u, "u", shape, dtype), _take(delta, "delta", shape, dtype), _take(A, "A", (ch, S), _F32),
            _take(B, "B", bc, dtype), _take(C, "C", bc, dtype), _take(D, "D", (ch,), _F32),
            _take(z, "z", shape, dtype), _take(delta_bias, "delta_bias", (ch,), _F32)), ch, S, G


def ssm_scan_fwd(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                 D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                 delta_bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                 cu_seqlens: Optional[torch.Tensor] = None, softplus: bool = False,
                 output_final_state: bool = True, out: Optional[torch.Tensor] = None,
                 final_state: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Selective state-space scan (``kda_ssm_scan_fwd``): per channel and state
    ``h = exp(dt A) h + dt u B``, ``y = C . h + D u``, ``out = y`` or
    ``y silu(z)``, with ``dt = delta + delta_bias`` (its softplus when
    ``softplus``).

    u, delta, z [b,T,channels] and B, C [b,T,G,S] in bf16 or fp32; A
    [channels,S], D and delta_bias [channels] fp32; initial_state
    [N,channels,S] fp32 or None; cu_seqlens as for ``chunk_fwd``.  Returns
    ``(out, final_state)``; ``final_state`` may be passed equal to
    ``initial_state``.  ``workspace``: a uint8 tensor of at least
    ``ssm_scan_fwd_workspace_bytes(...)`` bytes (allocated here when None and
    needed).
    """
    lib = load_library()
    b, T, _ = _rank(u, "u", 3)
    dt = _dtype(u, "u")
    ins, ch, S, G = _scan_inputs(u, delta, A, B, C, D, z, delta_bias, 2)
    cu, N = _sequences(cu_seqlens, b)
    flags = KDA_FLAG_SOFTPLUS if softplus else 0
    state = (N, ch, S)
    ps = _take(initial_state, "initial_state", state, _F32)
    with _On(stream):
        if out is None:
            out = torch.empty_like(u)
        if final_state is None and output_final_state:
            final_state = _state(initial_state, state, _F32, u)
        ws, size, _keep = _space(
            int(lib.kda_ssm_scan_fwd_workspace_bytes(b, T, ch, S, G, N, cu is not None, dt)), workspace,
            u.device)
        _check(lib.kda_ssm_scan_fwd(*ins, ps, cu, _take(out, "out", u.shape, u.dtype),
                                    _take(final_state, "final_state", state, _F32), b, T, ch, S, G, N,
                                    dt, flags, ws, size, _raw(stream, u)), "kda_ssm_scan_fwd")
    return out, final_state


def ssm_step(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
             state: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
             delta_bias: Optional[torch.Tensor] = None, softplus: bool = False,
             out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token of ``ssm_scan_fwd`` for each of N sequences (``kda_ssm_step``):
    u, delta, z [N,channels], B, C [N,G,S]; ``state`` [N,channels,S] fp32 is
    updated in place.  Returns out [N,channels]."""
    lib = load_library()
    N, _ = _rank(u, "u", 2)
    dt = _dtype(u, "u")
    ins, ch, S, G = _scan_inputs(u, delta, A, B, C, D, z, delta_bias, 1)
    ps = _take(state, "state", (N, ch, S), _F32)
    if out is not None:
        po = _take(out, "out", u.shape, u.dtype)
    else:
        out = _out(u, stream)
        po = out.data_ptr()
    _check(lib.kda_ssm_step(*ins, ps, po, N, ch, S, G, dt, KDA_FLAG_SOFTPLUS if softplus else 0,
                            _raw(stream, u)), "kda_ssm_step")
    return out


def ssm_scan_bwd(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                 d_out: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                 delta_bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                 d_final_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                 softplus: bool = False, need_initial_state_grad: bool = True, grads=None,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward pass of ``ssm_scan_fwd`` (``kda_ssm_scan_bwd``).

    Inputs as there plus ``d_out`` (shaped and typed like u) and
    ``d_final_state`` [N,channels,S] fp32 or None (zero).  Returns fp32 ``(du,
    ddelta, dA, dB, dC, dD, dz, ddelta_bias, d_initial_state)``; dD, dz and
    ddelta_bias are None without their input, the last is None when
    ``need_initial_state_grad`` is false.  ``grads``: the caller's nine output
    tensors instead of new ones (None is allowed where this list names it).
    """
    lib = load_library()
    b, T, _ = _rank(u, "u", 3)
    dt = _dtype(u, "u")
    ins, ch, S, G = _scan_inputs(u, delta, A, B, C, D, z, delta_bias, 2)
    cu, N = _sequences(cu_seqlens, b)
    state = (N, ch, S)
    ins += (_take(initial_state, "initial_state", state, _F32), cu, _take(d_out, "d_out", u.shape, u.dtype),
            _take(d_final_state, "d_final_state", state, _F32))
    shapes = (u.shape, u.shape, A.shape, B.shape, B.shape, (ch,), u.shape, (ch,), state)
    with _On(stream):
        given = grads is not None
        if not given:
            grads = (_like(u), _like(u), _like(A), _like(B), _like(B), _like(D), _like(z),
                     _like(delta_bias),
                     _state(initial_state, state, _F32, u) if need_initial_state_grad else None)
        du, dd, dA, dB, dC, dD, dz, dbias, ds = grads
        if any(t is None for t in (du, dd, dA, dB, dC)) or (z is not None and dz is None):
            raise ValueError("grads must hold du, ddelta, dA, dB, dC and, with z, dz")
        outs = _given(grads, shapes) if given else [None if t is None else t.data_ptr() for t in grads]
        ws, size, _keep = _space(
            int(lib.kda_ssm_scan_bwd_workspace_bytes(b, T, ch, S, G, N, cu is not None, dt)), workspace,
            u.device)
        _check(lib.kda_ssm_scan_bwd(*ins, *outs, b, T, ch, S, G, N, dt, KDA_FLAG_SOFTPLUS if softplus else 0,
                                    ws, size, _raw(stream, u)), "kda_ssm_scan_bwd")
    return du, dd, dA, dB, dC, dD, dz, dbias, ds


# ---- group norm --------------------------------------------------------------

def group_norm_workspace_bytes(B: int, T: int, C: int, groups: int, N: int, packed: bool,
                               per_token: bool = False, backward: bool = False, dtype=torch.bfloat16) -> int:
    """``kda_group_norm_fwd_workspace_bytes`` (or ``_bwd_`` when ``backward``)."""
    lib = load_library()
    f = lib.kda_group_norm_bwd_workspace_bytes if backward else lib.kda_group_norm_fwd_workspace_bytes
    flags = KDA_FLAG_PER_TOKEN if per_token else 0
    return _bytes(lambda *a: f(*a, flags), dtype, B, T, C, groups, N, int(packed))


def _norm_inputs(x, groups, weight, bias, activation, per_token, cu_seqlens):
    B, T, C = _rank(x, "x", 3)
    if groups < 1 or C % groups:
        raise ValueError("groups must divide the channels")
    cu, N = _sequences(cu_seqlens, B)
    flags = _activation(activation) | (KDA_FLAG_PER_TOKEN if per_token else 0)
    ins = (_take(x, "x", x.shape, x.dtype), _take(weight, "weight", (C,), _F32),
           _take(bias, "bias", (C,), _F32), cu)
    return ins, B, T, C, N, flags, (B * T if per_token else N, groups)


def group_norm_fwd(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, eps: float = 1e-5, activation: Optional[str] = None,
                   per_token: bool = False, cu_seqlens: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
                   rstd: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Group norm, channels last (``kda_group_norm_fwd``): ``(x - mean) rstd
    weight + bias``, then ``activation`` (None or "silu"), with the statistics
    of each group's channels over a whole sequence, or over each token when
    ``per_token`` (KDA_FLAG_PER_TOKEN).

    x [B,T,C] in bf16 or fp32, weight and bias [C] fp32 or None, cu_seqlens as
    for ``chunk_fwd``.  Returns ``(out, mean, rstd)``, the last two fp32
    [samples,groups], for ``group_norm_bwd``.
    """
    lib = load_library()
    dt = _dtype(x, "x")
    ins, B, T, C, N, flags, stat = _norm_inputs(x, groups, weight, bias, activation, per_token, cu_seqlens)
    with _On(stream):
        if out is None:
            out = torch.empty_like(x)
        if mean is None:
            mean = torch.empty(stat, dtype=_F32, device=x.device)
        if rstd is None:
            rstd = torch.empty_like(mean)
        need = 0 if per_token else int(lib.kda_group_norm_fwd_workspace_bytes(
            B, T, C, groups, N, cu_seqlens is not None, dt, flags))
        ws, size, _keep = _space(need, workspace, x.device)
        _check(lib.kda_group_norm_fwd(*ins, eps, _take(out, "out", x.shape, x.dtype),
                                      _take(mean, "mean", stat, _F32), _take(rstd, "rstd", stat, _F32),
                                      B, T, C, groups, N, dt, flags, ws, size, _raw(stream, x)),
               "kda_group_norm_fwd")
    return out, mean, rstd


def group_norm_bwd(x: torch.Tensor, groups: int, d_out: torch.Tensor, mean: torch.Tensor,
                   rstd: torch.Tensor, weight: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, activation: Optional[str] = None,
                   per_token: bool = False, cu_seqlens: Optional[torch.Tensor] = None, grads=None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward pass of ``group_norm_fwd`` (``kda_group_norm_bwd``) from its
    inputs, the ``mean`` and ``rstd`` it returned and ``d_out`` (shaped and
    typed like x).  Returns fp32 ``(dx, dweight, dbias)``, the last two None
    without their input.  ``grads``: the caller's three output tensors instead
    of new ones (dweight and dbias may be None).
    """
    lib = load_library()
    dt = _dtype(x, "x")
    ins, B, T, C, N, flags, stat = _norm_inputs(x, groups, weight, bias, activation, per_token, cu_seqlens)
    ins += (_take(mean, "mean", stat, _F32), _take(rstd, "rstd", stat, _F32),
            _take(d_out, "d_out", x.shape, x.dtype))
    shapes = (x.shape, (C,), (C,))
    with _On(stream):
        given = grads is not None
        if not given:
            grads = (_like(x), _like(weight), _like(bias))
        dx, dw, db = grads
        if dx is None:
            raise ValueError("grads must hold dx")
        outs = _given(grads, shapes) if given else [None if t is None else t.data_ptr() for t in grads]
        ws, size, _keep = _space(
            int(lib.kda_group_norm_bwd_workspace_bytes(B, T, C, groups, N, cu_seqlens is not None, dt, flags)),
            workspace, x.device)
        _check(lib.kda_group_norm_bwd(*ins, *outs, B, T, C, groups, N, dt, flags, ws, size, _raw(stream, x)),
               "kda_group_norm_bwd")
    return dx, dw, db
