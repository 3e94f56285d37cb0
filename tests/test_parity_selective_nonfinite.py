"""Values that are not finite in the per-channel scan, its gradient and decode
update: they reach what the definition lets them reach, and nothing else."""
import pytest
import torch

from tests.test_parity_selective import cu_of, operands, scan_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("dim", [64, 33])
def test_a_nan_step_size_passes_the_clamp(dim, softplus):
    """clamp(NaN) is NaN: the channel's outputs and gradients from that token on say so, the other channels do not."""
    from hybrid_mamba_ssm_b200 import ssm
    at, c = 11, 9
    p = scan_case(101, [40, 20], dim, 16, softplus=softplus, limit=(0.004, 0.08))
    args, kw = operands(p, "bf16", "f32")
    cu = cu_of(p)
    x, d, A, B, C = args
    dy = torch.randn_like(x)
    clean = ssm.selective_scan_fwd(*args, **kw, cu_seqlens=cu, save_states=True)
    gclean = ssm.selective_scan_bwd(dy, *args, clean[2], **kw, cu_seqlens=cu)
    d[at, c] = float("nan")
    y, hT, saved = ssm.selective_scan_fwd(*args, **kw, cu_seqlens=cu, save_states=True)
    rest = [i for i in range(dim) if i != c]
    assert bool(y[at:40, c].isnan().all()) and bool(hT[0, c].isnan().all())
    assert torch.equal(y[:at, c], clean[0][:at, c]) and torch.equal(y[40:], clean[0][40:])
    assert torch.equal(y[:, rest], clean[0][:, rest]) and torch.equal(hT[:, rest], clean[1][:, rest])
    g = ssm.selective_scan_bwd(dy, *args, saved, **kw, cu_seqlens=cu)
    # dx of a token before holds the gradients that came through the NaN decay; tokens behind have clean ones
    assert bool(g.dx[:at + 1, c].isnan().all()) and bool(g.ddt[:at + 1, c].isnan().all())
    assert bool(g.dA[c].isnan().all())
    assert torch.equal(g.dx[:, rest], gclean.dx[:, rest]) and torch.equal(g.dA[rest], gclean.dA[rest])
    state = torch.randn(3, dim, 16, device="cuda")
    u = ssm.selective_state_update(state, x[at - 1:at + 2], d[at - 1:at + 2], A, B[at - 1:at + 2], C[at - 1:at + 2], D=kw["D"],
                                   dt_bias=kw["dt_bias"], dt_softplus=softplus, dt_limit=p["limit"])
    assert bool(u[1, c].isnan()) and bool(state[1, c].isnan().all())
    assert bool(u[1, rest].isfinite().all()) and bool(u[[0, 2]].isfinite().all())
