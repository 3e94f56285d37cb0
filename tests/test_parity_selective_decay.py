"""The mean error of a decay.  A state with a memory of hundreds of tokens
multiplies hundreds of decays, so their errors' mean adds up where their
scatter averages out.  ex2.approx alone is 2.0e-8 of its value low on average
between 2^-0.5 and 2^-0.003; the kernels add as much back in the exponent.
What is left has to be below half of that, 1e-8, in every path that
multiplies decays: the scan whole and cut, the gradient whole and cut, and the
decode update.

With positive inputs a state is a sum of positive terms, and d log h / d (the
relative error of every decay) is S, computed beside the states in 64 bits.
The mean of (relative error of h) / S over thousands of states whose step
sizes vary from token to token is then the mean error of a decay; rounding
errors of either sign contribute at most 2^-24 of a term a token, and average
to below 1e-9 over 4096 states (each is a sum over a hundred tokens or more)."""
import ctypes

import numpy as np
import pytest
import torch

from tests.gpu_helpers import to_np
from tests.test_parity_selective import cu_of, operands, scan_case

pytestmark = pytest.mark.gpu

T, DIM, N = 1200, 256, 16
LIMIT = 1e-8


def case(seed):
    p = scan_case(seed, [T], DIM, N, dtype="f32", dt="f32", gate=False, D=False, h0=False, softplus=False, bias=False)
    f = lambda v: v.astype(np.float32).astype(np.float64)  # noqa: E731
    rng = np.random.default_rng(seed + 1)
    for k in "xBC":
        p[k] = f(1 + np.abs(p[k]))
    # exponents v A log2 e between about 0.003 and 0.1 in the mean: a memory of 15 to 500 tokens
    p["A"] = f(-np.exp(rng.uniform(np.log(0.05), np.log(1.5), (DIM, N))))
    return p


def sensitivities(v, A, terms):
    """h and d h / d (relative error of every decay), over the rows of terms [T, dim, N]."""
    h, s = np.zeros(A.shape), np.zeros(A.shape)
    for t in range(len(terms)):
        a = np.exp(v[t][:, None] * A)
        s, h = a * (s + h), a * h + terms[t]
    return h, s


def sensitivities_backward(p):
    """The same of dh0 = a_0 (C_0 dy_0 + a_1 (C_1 dy_1 + ..)), dy = 1."""
    h, s = np.zeros(p["A"].shape), np.zeros(p["A"].shape)
    for t in range(T - 1, -1, -1):
        a = np.exp(p["dt"][t][:, None] * p["A"])
        s, h = a * (s + h + p["C"][t]), a * (h + p["C"][t])
    return h, s


def mean_error(got, h, s):
    r = (to_np(got).reshape(h.shape) - h) / s
    return float(r[s > 20 * h].mean())              # states that remember more than 20 tokens


@pytest.mark.parametrize("workspace", ["auto", None], ids=["cut", "whole"])
def test_scan_and_gradient(workspace):
    from hybrid_mamba_ssm_b200 import ssm
    p = case(171)
    args, kw = operands(p, "f32", "f32")
    run = dict(**kw, cu_seqlens=cu_of(p))
    assert ssm.selective_scan_workspace_size(1, T, DIM, N) > 0
    y, hT, saved = ssm.selective_scan_fwd(*args, **run, save_states=True, workspace=workspace)
    terms = (p["dt"] * p["x"])[:, :, None] * np.repeat(p["B"], DIM, axis=1)
    h, s = sensitivities(p["dt"], p["A"], terms)
    e = mean_error(hT, h, s)
    assert abs(e) < LIMIT, e
    if workspace is None:
        return                                      # the gradient chooses its own cuts
    g = ssm.selective_scan_bwd(torch.ones_like(args[0]), *args, saved, **run, want_dinitial=True)
    h, s = sensitivities_backward(p)
    e = mean_error(g.dinitial_state[0], h, s)
    assert abs(e) < LIMIT, e


def test_gradient_of_whole_sequences():
    """Enough sequences that none is cut."""
    from hybrid_mamba_ssm_b200 import ssm
    p = case(181)
    nseq = 100
    assert ssm.lib.ssm_testing_selective_bwd_rows(nseq, nseq * T, 1, DIM, N, 1, ctypes.byref(ctypes.c_int(0))) <= 64
    (x, d, A, B, C), kw = operands(p, "f32", "f32")
    many = lambda t: t.repeat(nseq, *[1] * (t.dim() - 1))  # noqa: E731
    args = (many(x), many(d), A, many(B), many(C))
    cu = torch.arange(nseq + 1, dtype=torch.int32, device="cuda") * T
    _, _, saved = ssm.selective_scan_fwd(*args, **kw, cu_seqlens=cu, save_states=True)
    g = ssm.selective_scan_bwd(torch.ones_like(args[0]), *args, saved, **kw, cu_seqlens=cu, want_dinitial=True)
    h, s = sensitivities_backward(p)
    for k in (0, nseq - 1):
        e = mean_error(g.dinitial_state[k], h, s)
        assert abs(e) < LIMIT, e


def test_update_token_by_token():
    from hybrid_mamba_ssm_b200 import ssm
    p = case(191)
    (x, d, A, B, C), _ = operands(p, "f32", "f32")
    state, y = torch.zeros(1, DIM, N, device="cuda"), torch.empty(1, DIM, device="cuda")
    for t in range(T):
        ssm.selective_state_update(state, x[t:t + 1], d[t:t + 1], A, B[t:t + 1], C[t:t + 1], y=y)
    terms = (p["dt"] * p["x"])[:, :, None] * np.repeat(p["B"], DIM, axis=1)
    h, s = sensitivities(p["dt"], p["A"], terms)
    e = mean_error(state[0], h, s)
    assert abs(e) < LIMIT, e
