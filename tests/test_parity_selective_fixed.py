"""Gradients on fixed-length batches ([nseq, L, dim], no offsets), with
workspaces of exactly the reported size."""
import pytest
import torch

from tests.gpu_helpers import Guarded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nseq", [1, 64, 65, 100])
@pytest.mark.parametrize("dim,N", [(64, 16), (24, 4), (10, 256)])
def test_gradient_of_sequences_without_tokens(nseq, dim, N):
    """seqlen 0: the states pass through, every sum is zero, nothing is written behind the workspace."""
    from hybrid_mamba_ssm_b200 import ssm
    x, B = torch.empty(nseq, 0, dim, device="cuda"), torch.empty(nseq, 0, 1, N, device="cuda")
    A, D, bias = -torch.rand(dim, N, device="cuda"), torch.rand(dim, device="cuda"), torch.rand(dim, device="cuda")
    dhT = torch.randn(nseq, dim, N, device="cuda")
    _, _, saved = ssm.selective_scan_fwd(x, x, A, B, B, D=D, dt_bias=bias, dt_softplus=True, save_states=True)
    ws = Guarded((ssm.selective_scan_bwd_workspace_size(nseq, 0, dim, N),), torch.uint8)
    ws.t.fill_(0xff)                                       # NaN wherever a sum is read but was not written
    g = ssm.selective_scan_bwd(x, x, x, A, B, B, saved, D=D, dt_bias=bias, dt_softplus=True, dfinal_state=dhT,
                               want_dinitial=True, workspace=ws.t)
    torch.cuda.synchronize()
    ws.check("workspace")
    assert torch.equal(g.dinitial_state, dhT)
    for t in (g.dA, g.dD, g.ddt_bias):
        assert not bool(t.any())
    assert g.dx.shape == x.shape and g.dB.shape == B.shape
