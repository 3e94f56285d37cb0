"""Sizes at the edge of what the per-channel scan, its gradient and the pool
calls accept: host arithmetic and refusals only, no kernel is launched."""
import ctypes
import itertools

import pytest

from hybrid_mamba_ssm_b200 import build as ssm_build


@pytest.fixture(scope="module")
def lib():
    ssm_build.build()
    from hybrid_mamba_ssm_b200 import ssm
    return ssm.lib


@pytest.mark.parametrize("packed", [0, 1])
def test_gradient_stays_inside_the_rows_its_workspace_holds(lib, packed):
    """One row of partial sums per CTA of a channel tile: never more than the reported size has room for, in
    particular for sequences without tokens and for lengths around a segment."""
    held = ctypes.c_int(0)
    for nseq, seqlen, dim, (N, G) in itertools.product(
            [1, 2, 3, 5, 63, 64, 65, 100, 150, 1000], [0, 1, 7, 30, 31, 32, 33, 48, 64, 100, 200, 641, 5000],
            [1, 4, 64, 130, 1002, 8192], [(1, 1), (8, 1), (16, 1), (16, 2), (64, 1), (128, 1), (256, 1)]):
        if dim % G:
            continue
        tokens = nseq * seqlen if packed else seqlen
        rows = lib.ssm_testing_selective_bwd_rows(nseq, tokens, packed, dim, N, G, ctypes.byref(held))
        assert 0 < rows <= held.value, (nseq, seqlen, dim, N, G, rows, held.value)
