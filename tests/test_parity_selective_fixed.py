"""Gradients on fixed-length batches ([nseq, L, dim], no offsets), with
workspaces of exactly the reported size."""
import numpy as np
import pytest
import torch

from tests import selective_ref as ref
from tests.gpu_helpers import Guarded
from tests.test_parity_selective import DT, F, close, dev, operands, rounder, scan_case

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


GRADS = [("dx", "dx"), ("ddt", "ddt"), ("dA", "dA"), ("dB", "dB"), ("dC", "dC"), ("dD", "dD"), ("dz", "dz"),
         ("ddt_bias", "dbias"), ("dinitial_state", "dh0")]


@pytest.mark.parametrize("dtype,dt", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("dim,N,G", [(24, 16, 1), (10, 5, 2), (6, 128, 1)])
@pytest.mark.parametrize("nseq,L", [(1, 1), (70, 1), (3, 30), (70, 30), (64, 33), (2, 200), (66, 200), (1, 700)])
def test_scan_gradient(nseq, L, dim, N, G, dtype, dt):
    """Lengths below, at and above a segment, numbers of sequences on both sides of the 64 CTAs of a tile."""
    from hybrid_mamba_ssm_b200 import ssm
    p = scan_case(141, [L] * nseq, dim, N, G, dtype, dt)
    (x, d, A, B, C), kw = operands(p, dtype, dt)
    shape = lambda t: t.view(nseq, L, *t.shape[1:])  # noqa: E731
    args = (shape(x), shape(d), A, shape(B), shape(C))
    kw["z"] = shape(kw["z"])
    rng = np.random.default_rng(142)
    dy, dhT = rounder(DT[dtype])(rng.standard_normal((nseq * L, dim))), rounder(F)(rng.standard_normal((nseq, dim, N)))
    gy, ghT = shape(dev(dy, DT[dtype])), dev(dhT)
    y, hT, saved = ssm.selective_scan_fwd(*args, **kw, initial_state=dev(p["h0"]), save_states=True)
    g = ssm.selective_scan_bwd(gy, *args, saved, **kw, dfinal_state=ghT, want_dinitial=True)
    # the caller's workspaces, exactly as large as they have to be, full of NaN
    sizes = ssm.selective_scan_workspace_size(nseq, nseq * L, dim, N, G), ssm.selective_scan_bwd_workspace_size(nseq, nseq * L, dim, N, G)
    w1, w2 = (Guarded((max(1, n),), torch.uint8) for n in sizes)
    for w in (w1, w2):
        w.t.fill_(0xff)
    y2, hT2, saved2 = ssm.selective_scan_fwd(*args, **kw, initial_state=dev(p["h0"]), save_states=True, workspace=w1.t)
    g2 = ssm.selective_scan_bwd(gy, *args, saved2, **kw, dfinal_state=ghT, want_dinitial=True, workspace=w2.t)
    torch.cuda.synchronize()
    w1.check("workspace")
    w2.check("workspace of the gradient")
    for a, b in zip((y, hT, *g), (y2, hT2, *g2)):
        assert torch.equal(a, b)
    n = ref.scan_rounding(p)
    (want, wT, *_), (mag, mT, *_) = ref.scan(p), ref.scan(p, magnitude=True)
    close(y, want, mag, n, "y")
    close(hT, wT, mT, n, "final state")
    want, mag = ref.scan_grad(p, dy, dhT), ref.scan_grad(p, dy, dhT, magnitude=True)
    for name, k in GRADS:
        many = nseq * L + dim if name in ("dA", "dB", "dC", "dD", "ddt_bias") else 0
        close(getattr(g, name), want[k], mag[k], n + many, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 4, 8])
@pytest.mark.parametrize("nseq,L,dim", [(1, 1, 64), (70, 1, 33), (5, 2, 64), (70, 3, 64), (3, 5, 33), (2, 40, 64), (3, 130, 258),
                                        (4, 0, 64)])
def test_conv_gradient(nseq, L, dim, K, dtype):
    """Sequences shorter than the window (histories that reach the final state), and longer than a tile."""
    from hybrid_mamba_ssm_b200 import ssm
    rng, r, f, t = np.random.default_rng(K + dim), rounder(DT[dtype]), rounder(F), DT[dtype]
    T = nseq * L
    p = {"x": r(rng.standard_normal((T, dim))), "weight": f(rng.standard_normal((dim, K))), "act": True,
         "bias": f(rng.standard_normal(dim)), "init": r(rng.standard_normal((nseq, dim, K - 1))), "cu": ref.offsets([L] * nseq)}
    dy, df = r(rng.standard_normal((T, dim))), r(rng.standard_normal((nseq, dim, K - 1)))
    args = (dev(dy, t).view(nseq, L, dim), dev(p["x"], t).view(nseq, L, dim), dev(p["weight"]), dev(p["bias"]))
    kw = dict(initial_state=dev(p["init"], t), dfinal_state=dev(df, t))
    got = ssm.causal_conv1d_bwd(*args, **kw)
    ws = Guarded((max(1, ssm.lib.causal_conv1d_bwd_workspace_size(T, dim, K)),), torch.uint8)
    ws.t.fill_(0xff)
    again = ssm.causal_conv1d_bwd(*args, **kw, workspace=ws.t)
    torch.cuda.synchronize()
    ws.check("workspace")
    want, mag = ref.conv_grad(p, dy, df), ref.conv_grad(p, dy, df, magnitude=True)
    # as for packed sequences: (K + 2) roundings of pre through a slope of at most 1.1, an exponential and a reciprocal
    pre = sum(np.abs(p["weight"][:, k]) for k in range(K)) * np.abs(p["x"]).max(initial=1) + np.abs(p["bias"])
    per = 32 + K + (K + 2) * float(pre.max())
    flat = ref.conv_grad({**p, "act": False}, 1.1 * dy, df, magnitude=True)
    for name, v, u, k in zip(("dx", "dweight", "dbias", "dinitial_state"), got, again, ("dx", "dw", "db", "dinit")):
        assert torch.equal(v, u), name
        close(v, want[k], np.maximum(mag[k], flat[k]), per + (T if k in ("dw", "db") else 0), name)
