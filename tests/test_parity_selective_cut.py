"""Long sequences on few channels, which the per-channel scan and its gradient
cut into segments: every number of states a lane, strided views, bf16 results,
and fp32 errors within a bound that follows the recurrence.

The bound.  With U = 2^-24, a step size v (before the transform v0) is off by
(|v0| + 8) U of itself: one rounding of raw + bias, an ulp or two of the
exponential, the polynomial, the sum.  A decay a = exp(v A) is off by 4 U
(ex2.approx: 2^-22), 0.34 U (the correction in its exponent) and |v A| times
the error of its argument (v's, and three roundings).  So the error of a state
goes e <- a e + U (5 + |v A| (|v0| + 11)) a |h| + U (|v0| + 10) |v x B| + U |h|,
and likewise backwards for its gradient: what is forgotten stops counting.  A
segment's decay comes from a sum of its step sizes, off by at most one U a
token: X e^-X <= 0.37 of (its tokens + 16) U of the state that enters, for the
cut before and, what is left of it, the ones before that (twice the first).  Sums
over n add one U a term, a gate 4 U (its exponential), 2 U (the reciprocal),
(2 |z| + 4) U (its argument and three products)."""
import ctypes

import numpy as np
import pytest
import torch

from tests import selective_ref as ref
from tests.gpu_helpers import to_np
from tests.test_parity_selective import DT, F, close, cu_of, dev, operands, rounder, scan_case

pytestmark = pytest.mark.gpu

U = ref.ULP


def segment(ssm, nseq, T, dim, N, G):
    """Tokens that a segment of the forward or the backward pass has at most: units = T // span + nseq of each."""
    row = dim * N * 4
    ws = ssm.selective_scan_workspace_size(nseq, T, dim, N, G)
    assert ws > 0
    forward = (ws - nseq * row) // (row + dim * 4) - 1       # the parts of the workspace are rounded up to 16 bytes
    backward = ssm.lib.ssm_testing_selective_bwd_rows(nseq, T, 1, dim, N, G, ctypes.byref(ctypes.c_int(0)))
    assert backward > nseq
    return T // max(1, min(forward, backward) - nseq)


def bounds(p, dy, dhT, span):
    """Largest fp32 errors of y, the final states, dx and dinitial_state, from the exact values."""
    T, dim = p["x"].shape
    A = np.abs(p["A"])
    v0 = np.abs(p["dt"] + p["bias"])
    y, hT, pre, v, hs = ref.scan(p)
    rel = v0 + 8
    z = np.zeros_like(p["x"]) if p["z"] is None else p["z"]
    gate = np.ones_like(z) if p["z"] is None else np.abs(ref.silu(z))
    gate_err = 0 * z if p["z"] is None else 10 + 2 * np.abs(z)
    B, C = (np.abs(np.repeat(p[k], dim // p[k].shape[1], axis=1)) for k in "BC")
    x, D, N = np.abs(p["x"]), np.abs(p["D"]), A.shape[1]
    dyg = np.abs(dy) * gate
    out = {k: np.zeros_like(p["x"]) for k in ("y", "dx")}
    out["hT"], out["dh0"] = np.zeros_like(hT), np.zeros_like(hT)
    for s in range(len(p["cu"]) - 1):
        lo, hi = p["cu"][s], p["cu"][s + 1]
        join = 2 * 0.37 * (min(span, hi - lo) + 16) * U
        h, e, top = np.abs(p["h0"][s]), np.zeros(A.shape), np.abs(p["h0"][s])
        for t in range(lo, hi):
            a, va = np.exp(-v[t][:, None] * A), v[t][:, None] * A
            now = np.abs(hs[t])
            e = a * e + U * ((5 + va * (rel[t][:, None] + 3)) * a * h + (rel[t][:, None] + 2) * (v[t] * x[t])[:, None] * B[t] + now)
            h, top = now, np.maximum(top, now)
            ey = ((e + join * top) * C[t]).sum(1) + U * ((N + 3) * (now * C[t]).sum(1) + 2 * D * x[t])
            out["y"][t] = ey * gate[t] + U * np.abs(pre[t]) * gate[t] * (gate_err[t] + 1)
        out["hT"][s] = e + join * top
        g, e, top = np.abs(dhT[s]), np.zeros(A.shape), np.abs(dhT[s])
        signed = dhT[s].copy()
        sdyg = dy * (1 if p["z"] is None else ref.silu(z))
        sC = np.repeat(p["C"], dim // p["C"].shape[1], axis=1)
        for t in range(hi - 1, lo - 1, -1):
            a, va = np.exp(-v[t][:, None] * A), v[t][:, None] * A
            signed = signed + sdyg[t][:, None] * sC[t]
            now = np.abs(signed)
            e = e + U * ((gate_err[t][:, None] + 2) * dyg[t][:, None] * C[t] + now)
            top = np.maximum(top, now)
            ew = ((e + join * top) * B[t]).sum(1) + U * (N + 3) * (now * B[t]).sum(1)
            out["dx"][t] = ew * v[t] + U * ((rel[t] + 2) * v[t] * (now * B[t]).sum(1) + (gate_err[t] + 3) * D * dyg[t])
            e = a * e + U * (6 + va * (rel[t][:, None] + 3)) * a * now
            signed = a * signed
        out["dh0"][s] = e + join * top
    return out


def within(got, want, bound, name):
    g = to_np(got).reshape(want.shape)
    bad = ~(np.abs(g - want) <= bound + 1e-30)
    assert not bad.any(), (name, int(bad.sum()), float((np.abs(g - want) / (bound + 1e-30)).max()))


@pytest.mark.parametrize("lens,dim,N,G", [([3000], 32, 16, 1), ([700, 0, 1800, 0, 1, 900], 16, 16, 2), ([2100], 6, 13, 2),
                                          ([1500, 800], 8, 64, 1), ([1100, 300], 5, 128, 1), ([900], 4, 256, 2)])
def test_fp32_errors_follow_the_recurrence(lens, dim, N, G):
    from hybrid_mamba_ssm_b200 import ssm
    p = scan_case(151, lens, dim, N, G, "f32", "f32")
    args, kw = operands(p, "f32", "f32")
    span = segment(ssm, len(lens), sum(lens), dim, N, G)
    rng = np.random.default_rng(152)
    dy, dhT = rounder(F)(rng.standard_normal((sum(lens), dim))), rounder(F)(rng.standard_normal((len(lens), dim, N)))
    run = dict(**kw, cu_seqlens=cu_of(p))
    y, hT, saved = ssm.selective_scan_fwd(*args, **run, initial_state=dev(p["h0"]), save_states=True)
    g = ssm.selective_scan_bwd(dev(dy), *args, saved, **run, dfinal_state=dev(dhT), want_dinitial=True)
    bound, grad = bounds(p, dy, dhT, span), ref.scan_grad(p, dy, dhT)
    want, wT, *_ = ref.scan(p)
    within(y, want, bound["y"], "y")
    within(hT, wT, bound["hT"], "final state")
    within(g.dx, grad["dx"], bound["dx"], "dx")
    within(g.dinitial_state, grad["dh0"], bound["dh0"], "dinitial_state")
    # the bound says something: far below a rounding to bf16 of the largest values
    for k, v in (("y", want), ("hT", wT), ("dx", grad["dx"]), ("dh0", grad["dh0"])):
        assert bound[k].max() < 2.0 ** -9 * np.abs(v).max() / 4, k


@pytest.mark.parametrize("dtype,dt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("lens,dim,N,G,pad", [([1500, 0, 700, 1], 8, 16, 1, 3), ([1300], 6, 16, 1, 2), ([1200, 33], 6, 5, 2, 1),
                                              ([1000, 64], 4, 32, 1, 3), ([900], 6, 64, 3, 1), ([700, 500], 4, 100, 1, 0),
                                              ([800], 4, 128, 2, 5), ([640, 100], 3, 200, 1, 1), ([600, 0, 90], 2, 256, 1, 0)])
def test_every_number_of_lanes_and_strided_rows(lens, dim, N, G, pad, dtype, dt):
    """Cut calls with 4 to 32 lanes a channel and 4 or 8 states a lane, on rows inside wider ones."""
    from hybrid_mamba_ssm_b200 import ssm
    p = scan_case(161, lens, dim, N, G, dtype, dt)
    args, kw = operands(p, dtype, dt, pad=pad)
    nseq, T = len(lens), sum(lens)
    span = segment(ssm, nseq, T, dim, N, G)
    rng = np.random.default_rng(162)
    dy, dhT = rounder(DT[dtype])(rng.standard_normal((T, dim))), rounder(F)(rng.standard_normal((nseq, dim, N)))
    run = dict(**kw, cu_seqlens=cu_of(p))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, hT, saved = ssm.selective_scan_fwd(*args, **run, initial_state=dev(p["h0"]), save_states=True, status=status)
    g = ssm.selective_scan_bwd(dev(dy, DT[dtype]), *args, saved, **run, dfinal_state=dev(dhT), want_dinitial=True, status=status)
    assert status.item() == 0 and y.dtype == DT[dtype]
    bound, grad, mag = bounds(p, dy, dhT, span), ref.scan_grad(p, dy, dhT), ref.scan_grad(p, dy, dhT, magnitude=True)
    want, wT, *_ = ref.scan(p)
    half = 2.0 ** -8 if dtype == "bf16" else 0.0            # a bf16 result: half a step of its own value, and of the bound
    within(y, want, bound["y"] * (1 + half) + half * np.abs(want), "y")
    within(hT, wT, bound["hT"], "final state")
    within(g.dx, grad["dx"], bound["dx"] * (1 + half) + half * np.abs(grad["dx"]), "dx")
    within(g.dinitial_state, grad["dh0"], bound["dh0"], "dinitial_state")
    n = ref.scan_rounding(p)
    for t, k in [(g.ddt, "ddt"), (g.dA, "dA"), (g.dB, "dB"), (g.dC, "dC"), (g.dD, "dD"), (g.dz, "dz"), (g.ddt_bias, "dbias")]:
        close(t, grad[k], mag[k], n + (T + dim if k in ("dA", "dB", "dC", "dD", "dbias") else 0), k)
