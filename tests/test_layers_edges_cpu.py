"""Sizes that do not fit the library's ints (no GPU needed: the refusals come
before any CUDA call)."""
import pytest
import torch

import gated_delta_rule_103_b200 as kda
from gated_delta_rule_103_b200 import build

LONG = 2 ** 32 + 4096      # as an int of 32 bits: 4096


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_tensors_longer_than_an_int():
    w, A = meta(8, 4), meta(8, 4)
    x, bc = meta(1, LONG, 8), meta(1, LONG, 1, 4)
    for call in (lambda: kda.short_conv_fwd(x, w), lambda: kda.short_conv_step(x[0], w, meta(LONG, 3, 8)),
                 lambda: kda.short_conv_bwd(x, w, x), lambda: kda.ssm_scan_fwd(x, x, A, bc, bc),
                 lambda: kda.ssm_step(x[0], x[0], A, bc[0], bc[0], meta(LONG, 8, 4)),
                 lambda: kda.ssm_scan_bwd(x, x, A, bc, bc, x), lambda: kda.group_norm_fwd(x, 2),
                 lambda: kda.group_norm_bwd(x, 2, x, meta(1, 2), meta(1, 2)),
                 lambda: kda.group_norm_fwd(meta(1, 4, LONG), 2),
                 lambda: kda.short_conv_fwd(meta(1, 4, 8), w, cu_seqlens=meta(LONG + 1, dtype=torch.int32))):
        with pytest.raises(ValueError, match=r"below 2\^31"):
            call()


def test_workspace_queries_beyond_an_int():
    for T in (LONG, -2 ** 32 + 4096):
        assert kda.short_conv_bwd_workspace_bytes(1, T, 64, 4, 1, False) == 0
        assert kda.ssm_scan_fwd_workspace_bytes(1, T, 64, 16, 1, 1, False) == 0
        assert kda.ssm_scan_bwd_workspace_bytes(1, T, 64, 16, 1, 1, False) == 0
        assert kda.group_norm_workspace_bytes(1, T, 64, 4, 1, False) == 0
        assert kda.group_norm_workspace_bytes(1, T, 64, 4, 1, False, backward=True) == 0
    assert kda.ssm_scan_fwd_workspace_bytes(1, 4096, 64, 16, 1, 1, False) > 0
    assert kda.group_norm_workspace_bytes(1, 4096, 64, 4, 1, False, backward=True) > 0


def test_which_scans_are_cut():
    """Sequences of one length stay whole from three warps an SM on (of 148: 7104
    channels of 16 states in all sequences together), ragged ones' limit is six."""
    def cut(n, T, D, packed, S=16):
        return kda.ssm_scan_fwd_workspace_bytes(1 if packed else n, n * T if packed else T, D, S, 1, n, packed) > 0

    assert cut(1, 16384, 4096, False) and not cut(2, 8192, 4096, False) and not cut(4, 4096, 4096, False)
    assert cut(6, 2000, 1024, False) and not cut(7, 2000, 1024, False)
    assert cut(1, 2000, 1024, False, 64) and not cut(2, 2000, 1024, False, 64)
    assert not cut(1, 127, 64, False) and cut(1, 128, 64, False)
    assert cut(2, 8192, 4096, True) and cut(4, 4096, 4096, True)
