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
