"""Values that are not finite in the per-channel scan, its gradient and decode
update: they reach what the definition lets them reach, and nothing else."""
import numpy as np
import pytest
import torch

from tests import selective_ref as ref
from tests.test_parity_selective import close, cu_of, dev, operands, scan_case

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


@pytest.mark.parametrize("rate", [float("-inf"), -3e38])
@pytest.mark.parametrize("lens,dim,N", [([37, 5], 64, 16), ([33], 33, 13), ([1, 2, 3], 24, 64), ([1501], 16, 16)])
def test_a_state_that_is_forgotten_at_once(lens, dim, N, rate):
    """exp(v A) = 0 for a step size above 0 and a decay rate without bound (or one that overflows in other units):
    the state is the last token's alone, whatever length fills the last tile."""
    from hybrid_mamba_ssm_b200 import ssm
    p = scan_case(131, lens, dim, N)
    pick = np.random.default_rng(132).random(p["A"].shape) < 0.25
    p["A"][pick] = rate
    args, kw = operands(p, "bf16", "bf16")
    cu = cu_of(p)
    y, hT, saved = ssm.selective_scan_fwd(*args, **kw, initial_state=dev(p["h0"]), cu_seqlens=cu, save_states=True)
    want, wT, *_ = ref.scan(p)
    mag, mT, *_ = ref.scan(p, magnitude=True)
    assert np.isfinite(want).all() and np.isfinite(wT).all()
    close(y, want, mag, ref.scan_rounding(p), "y")
    close(hT, wT, mT, ref.scan_rounding(p), "final state")
    g = ssm.selective_scan_bwd(torch.ones_like(args[0]), *args, saved, **kw, cu_seqlens=cu, want_dinitial=True)
    q = {**p, "A": np.where(pick, -1e30, p["A"])}           # the limit: no product 0 * inf in the reference
    dy = np.ones_like(p["x"])
    zero = np.zeros_like(p["h0"])
    want, mag = ref.scan_grad(q, dy, zero), ref.scan_grad(q, dy, zero, magnitude=True)
    n = ref.scan_rounding(p)
    for t, k in [(g.dx, "dx"), (g.ddt, "ddt"), (g.dA, "dA"), (g.dB, "dB"), (g.dC, "dC"), (g.dinitial_state, "dh0")]:
        close(t, want[k], mag[k], n + (sum(lens) + dim if k in ("dA", "dB", "dC") else 0), k)
    state = dev(p["h0"])                                    # and one token
    first = [p["cu"][i] for i in range(len(lens))]
    x, d, A, B, C = args
    ssm.selective_state_update(state, x[first], d[first], A, B[first], C[first], D=kw["D"], z=kw["z"][first],
                               dt_bias=kw["dt_bias"], dt_softplus=True)
    hs = ref.scan(p)[4][first]
    close(state, hs, ref.scan(p, magnitude=True)[4][first], ref.scan_rounding(p), "state")
