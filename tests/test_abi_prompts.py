"""Limits of the prompt attention's arguments, on the host: no call here touches
a GPU."""
import ctypes

import pytest


@pytest.mark.parametrize("B", [2 ** 26, 2 ** 26 + 1, 2 ** 29])
def test_more_prompts_than_are_planned_in_time_are_refused(B):
    """The planning of 2^29 sequences would outlast the waits for it."""
    import ternary_weight_ptq1_gb300 as P

    P._build.build()
    L = P.load()
    at = 16 * 1024                          # never dereferenced
    assert L.ptq_attn_prefill(at, at, at, 64, 64, 64, at, at, at, None, B, 8, 8, 1, 1, 64, 0.1, 0, P.PTQ_BF16, at,
                              ctypes.c_size_t(1 << 40), None) == 2
    assert b"B" in L.ptq_last_error()
    assert P.attn_prefill_workspace_bytes(B, 8, 2 ** 25, 1, 1, 64, P.PTQ_BF16) == 0
    assert P.attn_prefill_workspace_bytes(1, 8, 2 ** 25, 1, 1, 64, P.PTQ_BF16) > 0
