"""Sizes at the edge of what the per-channel scan, its gradient and the pool
calls accept: host arithmetic and refusals only, no kernel is launched."""
import ctypes
import itertools

import pytest
import torch

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


def test_pool_calls_refuse_what_their_counters_do_not_hold(lib):
    """Slots and index lists of more than 2^30 entries: the steps of the kernels' loops would pass 2^31."""
    M, most, UNSUPPORTED = 1 << 24, 1 << 30, 2
    one = (ctypes.c_int64 * 3)(M, 1, 1)
    table, work = 1 << 44, 1 << 45                          # fake addresses: refused before anything is read
    for slots, n in ((most + 1, 4), (2 ** 31 - 1, 4), (4, most + 1), (4, 2 ** 31 - 1)):
        assert lib.ssm_pool_copy(1, one, slots, n, table, table, None, None) == UNSUPPORTED
        assert lib.ssm_pool_zero(1, one, slots, n, table, None, None) == UNSUPPORTED
        assert lib.ssm_pool_compact(1, one, slots, n, table, None, work, 1 << 40, None, None) == UNSUPPORTED
    # at the limit it is the next check that answers
    assert lib.ssm_pool_copy(1, one, most, most, table + 4, table, None, None) == 3
    assert lib.ssm_pool_compact(1, one, most, most, table, None, work, 16, None, None) == 1


def test_binding_refuses_sizes_that_do_not_fit_an_int(lib):
    """ctypes passes 2^32 + 8 as 8: such a size is named before it gets there (shapes only, nothing is allocated)."""
    from hybrid_mamba_ssm_b200 import ssm
    big = 2 ** 32 + 8
    shape = lambda *s: torch.empty(s, device="meta")  # noqa: E731
    cu = torch.zeros(2, dtype=torch.int32)
    for x, offsets in ((shape(big, 4), cu), (shape(4, big), cu), (shape(big, 1, 4), None), (shape(1, big, 4), None),
                       (shape(1, 4, big), None)):
        with pytest.raises(ValueError, match="2\\^31"):
            ssm._scan_lead(x, offsets, -1)
    x = torch.zeros(4, 8)
    for A, B in ((shape(8, big), shape(4, 1, big)), (shape(8, 2), shape(4, big, 2))):
        with pytest.raises(ValueError, match="2\\^31"):
            ssm._scan_operands((4,), 8, -1, x, x, A, B, B, None, None, None, False, None)
    for pools in (shape(big, 1), [shape(big, 4), shape(big, 2)]):
        with pytest.raises(ValueError, match="2\\^31"):
            ssm._pools(pools)
    assert ssm._pools(shape(2 ** 31 - 1, 1))[2] == 2 ** 31 - 1
