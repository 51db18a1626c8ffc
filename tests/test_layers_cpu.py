"""Host-side checks of the layer operators: refusals that come before any
CUDA call, workspace sizes, and the 64-bit reference forms themselves
(gradients against differences)."""
import ctypes

import pytest
import torch

import gated_delta_rule_103_b200 as kda
from gated_delta_rule_103_b200 import binding, build
import layer_reference as ref

BAD, UNSUP, OK = binding.KDA_ERR_INVALID_ARG, binding.KDA_ERR_UNSUPPORTED, binding.KDA_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def conv(lib, B=1, T=4, C=8, W=4, N=1, dt=1, flags=0, cu=None):
    return lib.kda_short_conv_fwd(None, None, None, None, cu, None, None, B, T, C, W, N, dt, flags, None)


def test_short_conv_sizes(lib):
    assert conv(lib, W=5) == UNSUP and conv(lib, W=1) == UNSUP and conv(lib, W=0) == BAD
    assert conv(lib, C=0) == BAD and conv(lib, T=-1) == BAD and conv(lib, dt=2) == BAD
    assert conv(lib, N=2) == BAD                       # N != B without cu_seqlens
    assert conv(lib, flags=16) == UNSUP and conv(lib, flags=1) == UNSUP
    assert conv(lib, B=65536, T=65536, N=65536) == UNSUP
    assert conv(lib, C=(1 << 24) + 1) == UNSUP
    assert conv(lib, B=2, N=2, cu=ctypes.c_void_p(16)) == BAD    # packed: B must be 1
    assert conv(lib, N=0, cu=ctypes.c_void_p(16)) == BAD         # tokens, and no sequence
    assert conv(lib) == BAD                            # null tensors
    assert lib.kda_short_conv_step(None, None, None, None, None, 0, 8, 4, 1, 0, None) == OK
    assert lib.kda_short_conv_step(None, None, None, None, None, 2, 8, 4, 1, 0, None) == BAD
    assert lib.kda_short_conv_step(None, None, None, None, None, 2, 8, 6, 1, 0, None) == UNSUP
    assert lib.kda_short_conv_bwd(*[None] * 11, 1, 4, 8, 5, 1, 1, 0, None, 0, None) == UNSUP
    assert lib.kda_short_conv_bwd(*[None] * 11, 1, 4, 8, 4, 1, 1, 0, None, 0, None) == BAD


def scan(lib, B=1, T=4, D=8, S=4, G=1, N=1, dt=1, flags=0, cu=None):
    return lib.kda_ssm_scan_fwd(*[None] * 9, cu, None, None, B, T, D, S, G, N, dt, flags, None, 0, None)


def test_ssm_scan_sizes(lib):
    assert scan(lib, S=129) == UNSUP and scan(lib, S=0) == BAD
    assert scan(lib, G=3) == BAD and scan(lib, G=0) == BAD
    assert scan(lib, D=0) == BAD and scan(lib, N=3) == BAD and scan(lib, dt=5) == BAD
    assert scan(lib, flags=8) == UNSUP
    assert scan(lib, N=0, cu=ctypes.c_void_p(16)) == BAD
    assert scan(lib) == BAD
    assert lib.kda_ssm_step(*[None] * 10, 0, 8, 4, 1, 1, 0, None) == OK
    assert lib.kda_ssm_step(*[None] * 10, 1, 8, 200, 1, 1, 0, None) == UNSUP
    assert lib.kda_ssm_step(*[None] * 10, 1, 8, 4, 1, 1, 0, None) == BAD
    assert lib.kda_ssm_scan_bwd(*[None] * 21, 1, 4, 8, 4, 3, 1, 1, 0, None, 0, None) == BAD
    assert lib.kda_ssm_scan_bwd(*[None] * 21, 1, 4, 8, 4, 1, 1, 1, 0, None, 0, None) == BAD


def norm(lib, eps=1e-5, B=1, T=4, C=8, G=2, N=1, dt=1, flags=0, cu=None):
    return lib.kda_group_norm_fwd(None, None, None, cu, ctypes.c_float(eps), None, None, None, B, T, C, G, N, dt,
                                  flags, None, 0, None)


def test_group_norm_sizes(lib):
    assert norm(lib, G=3) == BAD and norm(lib, G=0) == BAD and norm(lib, G=16) == BAD
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert norm(lib, eps=eps) == BAD
    assert norm(lib, flags=16) == UNSUP and norm(lib, dt=3) == BAD and norm(lib, N=2) == BAD
    assert norm(lib) == BAD
    assert lib.kda_group_norm_bwd(*[None] * 10, 1, 4, 8, 3, 1, 1, 0, None, 0, None) == BAD
    assert lib.kda_group_norm_bwd(*[None] * 10, 1, 4, 8, 2, 1, 1, 0, None, 0, None) == BAD


def test_workspace_sizes(lib):
    # sizes that a call would refuse need nothing
    assert kda.short_conv_bwd_workspace_bytes(1, 16, 8, 7, 1, False) == 0
    assert kda.ssm_scan_fwd_workspace_bytes(1, 16, 8, 300, 1, 1, False) == 0
    assert kda.ssm_scan_bwd_workspace_bytes(1, 16, 9, 4, 2, 1, False) == 0
    assert kda.group_norm_workspace_bytes(1, 16, 9, 2, 1, False) == 0
    assert kda.group_norm_workspace_bytes(1, 16, 8, 2, 2, False) == 0
    # the statistics of one token need no other's
    assert kda.group_norm_workspace_bytes(2, 100, 64, 4, 2, False, per_token=True) == 0
    assert kda.group_norm_workspace_bytes(2, 100, 64, 4, 2, False) > 0
    # many chains fill the GPU without cutting a sequence
    assert kda.ssm_scan_fwd_workspace_bytes(64, 512, 8192, 16, 1, 64, False) == 0
    assert kda.ssm_scan_fwd_workspace_bytes(1, 65536, 64, 16, 1, 1, False) > 0
    assert kda.ssm_scan_bwd_workspace_bytes(2, 64, 32, 16, 1, 2, False) > 0


def test_binding_refuses(lib):
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        kda.short_conv_fwd(x, w)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        kda.short_conv_fwd(x.half(), w)
    with pytest.raises(ValueError, match="activation"):
        kda.short_conv_fwd(x, w, activation="tanh")
    with pytest.raises(ValueError, match="dimensions"):
        kda.short_conv_fwd(x[0], w)
    with pytest.raises(ValueError, match="batch of 1"):
        kda.short_conv_fwd(torch.zeros(2, 4, 8), w, cu_seqlens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="int32"):
        kda.short_conv_fwd(x, w, cu_seqlens=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="groups"):
        kda.group_norm_fwd(x, 3)
    with pytest.raises(ValueError, match="CUDA"):
        kda.group_norm_fwd(x, 2)
    A, B = torch.zeros(8, 4), torch.zeros(1, 4, 1, 4)
    with pytest.raises(ValueError, match="CUDA"):
        kda.ssm_scan_fwd(x, x, A, B, B)
    with pytest.raises(ValueError, match="G dividing"):
        kda.ssm_scan_fwd(x, x, A, torch.zeros(1, 4, 3, 4), B)
    with pytest.raises(ValueError, match="leading"):
        kda.ssm_scan_fwd(x, x, A, torch.zeros(1, 5, 1, 4), B)
    with pytest.raises(ValueError, match="CUDA"):
        kda.ssm_step(x[0], x[0], A, B[0], B[0], torch.zeros(4, 8, 4))


def _check_differences(f, inputs):
    # A central difference over 2 eps of values up to F, each the end of some
    # 16 roundings of at most F 2^-53, is off by up to 16 F 2^-53 / eps (here F
    # is some 10^4: positive A let the states grow).
    with torch.no_grad():
        outs = f(*inputs)
    F = max(float(t.abs().max()) for t in (outs if isinstance(outs, tuple) else (outs,)))
    eps = 1e-6
    assert torch.autograd.gradcheck(f, inputs, eps=eps, atol=max(1e-7, 16 * F * 2.0 ** -53 / eps), rtol=1e-5)


def test_reference_gradients_against_differences():
    g = torch.Generator().manual_seed(3)

    def r(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64).requires_grad_()

    bounds = ref.bounds_of([3, 0, 1, 5])
    _check_differences(lambda x, w, b, s: ref.short_conv(x, w, b, s, bounds, True),
                       (r(9, 2), r(2, 4), r(2), r(4, 3, 2)))
    _check_differences(lambda u, d, A, B, C, k, z, b, s: ref.ssm_scan(u, d, A, B, C, k, z, b, s, bounds, True),
                       (r(9, 4), r(9, 4), r(4, 3), r(9, 2, 3), r(9, 2, 3), r(4), r(9, 4), r(4), r(4, 4, 3)))
    _check_differences(lambda x, w, b: ref.group_norm(x, 2, w, b, 1e-5, bounds, True)[0], (r(9, 4), r(4), r(4)))
