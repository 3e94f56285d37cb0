"""The fp64 reference of the per-channel scan against results that do not come
from it (the per-head oracle, torch's autograd, differences), and the refusals
of the new entry points.  Nothing here launches a kernel."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import oracle
from hybrid_mamba_ssm_b200 import build as ssm_build
from tests import selective_ref as ref

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
F32, BF16, F16 = 0, 1, 2


# ---------------------------------------------------------------------------
# the reference
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("G", [1, 3])
def test_reference_equals_the_per_head_oracle_at_one_state(G):
    """With d_state = 1 a channel is a head of head_dim 1: the two recurrences coincide."""
    p = ref.make_scan(1, [7, 0, 12], 6, 1, G, gate=False)
    v, _ = ref.step_size(p["dt"], p["bias"], True, None)
    y, hT = oracle.scan(p["x"][:, :, None], v, p["A"][:, 0], p["B"], p["C"], p["D"], p["h0"][:, :, None],
                        cu_seqlens=np.array(p["cu"], dtype=np.int64))
    got, gT, *_ = ref.scan(p)
    np.testing.assert_allclose(got, y[:, :, 0], rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(gT, hT[:, :, 0], rtol=1e-12, atol=1e-13)


def _torch_scan(p, t):
    """The definition in torch fp64, for autograd."""
    v = t["dt"] + (0 if t["bias"] is None else t["bias"])
    if p["softplus"]:
        v = torch.nn.functional.softplus(v, threshold=700)
    if p["limit"] is not None:
        v = v.clamp(*p["limit"])
    dim = t["x"].shape[1]
    B, C = (t[k].repeat_interleave(dim // t[k].shape[1], dim=1) for k in "BC")
    ys, hTs = [], []
    for s in range(len(p["cu"]) - 1):
        h = t["h0"][s] if t["h0"] is not None else torch.zeros_like(t["A"])
        for k in range(p["cu"][s], p["cu"][s + 1]):
            h = torch.exp(v[k][:, None] * t["A"]) * h + (v[k] * t["x"][k])[:, None] * B[k]
            y = (h * C[k]).sum(1) + (0 if t["D"] is None else t["D"] * t["x"][k])
            ys.append(y if t["z"] is None else y * torch.nn.functional.silu(t["z"][k]))
        hTs.append(h)
    return torch.stack(ys), torch.stack(hTs)


@pytest.mark.parametrize("kw", [dict(), dict(gate=False, D=False, h0=False, G=2), dict(limit=(0.01, 0.05)),
                                dict(softplus=False, bias=False)])
def test_reference_gradient_equals_autograd_and_differences(kw):
    p = ref.make_scan(2, [5, 0, 1, 9], 4, 3, **kw)
    rng = np.random.default_rng(3)
    dy, dhT = rng.standard_normal(p["x"].shape), rng.standard_normal((4, 4, 3))
    names = {"x": "dx", "dt": "ddt", "A": "dA", "B": "dB", "C": "dC", "D": "dD", "z": "dz", "bias": "dbias", "h0": "dh0"}
    t = {k: None if p[k] is None else torch.tensor(p[k], dtype=torch.float64, requires_grad=True) for k in names}
    y, hT = _torch_scan(p, t)
    np.testing.assert_allclose(y.detach().numpy(), ref.scan(p)[0], rtol=1e-11, atol=1e-12)
    ((y * torch.tensor(dy)).sum() + (hT * torch.tensor(dhT)).sum()).backward()
    g = ref.scan_grad(p, dy, dhT)
    for k, n in names.items():
        if p[k] is not None:
            np.testing.assert_allclose(g[n], t[k].grad.numpy(), rtol=1e-9, atol=1e-11, err_msg=n)

    def loss(q):
        y, hT, *_ = ref.scan(q)
        return (y * dy).sum() + (hT * dhT).sum()

    for k, n in names.items():
        if p[k] is None or (k == "dt" and p["limit"] is not None):   # the clamp has a kink
            continue
        u = rng.standard_normal(p[k].shape)
        e = 1e-6
        d = (loss({**p, k: p[k] + e * u}) - loss({**p, k: p[k] - e * u})) / (2 * e)
        assert abs(d - (g[n] * u).sum()) < 1e-6 * (1 + abs(d)), n


@pytest.mark.parametrize("K,act,init", list(itertools.product([1, 2, 4], [True, False], [True, False])))
def test_conv_reference_gradient_equals_autograd(K, act, init):
    rng = np.random.default_rng(K)
    lens, dim = [5, 0, 1, 2, 8], 3
    cu = ref.offsets(lens)
    p = {"x": rng.standard_normal((cu[-1], dim)), "weight": rng.standard_normal((dim, K)), "bias": rng.standard_normal(dim),
         "act": act, "init": rng.standard_normal((5, dim, K - 1)) if init else None, "cu": cu}
    dy, dfin = rng.standard_normal(p["x"].shape), rng.standard_normal((5, dim, K - 1))
    t = {k: None if p[k] is None else torch.tensor(p[k], requires_grad=True) for k in ("x", "weight", "bias", "init")}
    loss = 0
    for s in range(5):
        front = torch.zeros(K - 1, dim, dtype=torch.float64) if t["init"] is None else t["init"][s].T
        line = torch.cat([front, t["x"][cu[s]:cu[s + 1]]])
        n = lens[s]
        pre = t["bias"] + sum(line[k:k + n] * t["weight"][:, k] for k in range(K))
        out = torch.nn.functional.silu(pre) if act else pre
        loss = loss + (out * torch.tensor(dy[cu[s]:cu[s + 1]])).sum() + (line[n:].T * torch.tensor(dfin[s])).sum()
    loss.backward()
    g = ref.conv_grad(p, dy, dfin)
    for k, n in (("x", "dx"), ("weight", "dw"), ("bias", "db"), ("init", "dinit")):
        if t[k] is not None:
            np.testing.assert_allclose(g[n], t[k].grad.numpy(), rtol=1e-10, atol=1e-12)


# ---------------------------------------------------------------------------
# refusals (fake, never-dereferenced addresses: validation rejects the call first)
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    ssm_build.build()
    from hybrid_mamba_ssm_b200 import ssm
    return ssm.lib


M = 1 << 24   # spacing of the fake buffers


def fwd(lib, nseq=2, seqlen=8, cu=None, dim=64, N=16, G=1, ind=BF16, x=M, xs=64, dtd=BF16, dt=2 * M, dts=64, A=3 * M,
        B=4 * M, Bs=16, C=5 * M, Cs=16, D=None, z=None, zs=0, h0=None, hT=6 * M, slots=0, idx=None, has=None, yd=BF16,
        y=7 * M, saved=None, ws=None, wsb=0):
    return lib.selective_scan_fwd(nseq, seqlen, cu, dim, N, G, ind, x, xs, dtd, dt, dts, A, B, Bs, C, Cs, D, z, zs, None,
                                  h0, hT, slots, idx, has, yd, y, saved, ws, wsb, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(nseq=-1), INVALID), (dict(seqlen=-1), INVALID), (dict(dim=0), INVALID), (dict(N=0), INVALID),
    (dict(G=3), INVALID), (dict(G=0), INVALID), (dict(ind=F16), INVALID), (dict(dtd=9), INVALID), (dict(yd=F16), INVALID),
    (dict(N=257), UNSUPPORTED), (dict(ind=F32, dtd=BF16), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(dt=None), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID),
    (dict(C=None), INVALID), (dict(y=None), INVALID),
    (dict(xs=63), INVALID), (dict(Bs=15), INVALID), (dict(z=8 * M, zs=10), INVALID), (dict(xs=1 << 25), UNSUPPORTED),
    (dict(x=M + 1), MISALIGNED), (dict(ind=F32, dtd=F32, x=M + 2), MISALIGNED), (dict(A=3 * M + 8), MISALIGNED),
    (dict(y=7 * M + 8), MISALIGNED), (dict(hT=6 * M + 4), MISALIGNED),
    (dict(y=M + 512), INVALID), (dict(hT=2 * M), INVALID), (dict(saved=6 * M), INVALID),
    (dict(h0=6 * M + 64), INVALID),                                   # a partial overlap of the states
    (dict(idx=9 * M, slots=0), INVALID), (dict(idx=9 * M, slots=4, hT=None), INVALID),
    (dict(nseq=0), OK), (dict(nseq=3, seqlen=0, hT=None), OK),
])
def test_scan_refusals(lib, kw, code):
    assert fwd(lib, **kw) == code


def test_scan_accepts_views_up_to_validation(lib):
    """A stride that leaves room and an address aligned to the element only are not what is refused."""
    assert fwd(lib, x=M + 2, xs=200, y=None) == INVALID               # y is
    assert fwd(lib, x=M + 2, xs=200, y=7 * M + 2) == MISALIGNED       # y is


def bwd(lib, nseq=2, seqlen=8, dim=64, N=16, G=1, ind=BF16, dtd=BF16, dy=20 * M, dys=64, x=M, saved=6 * M, dx=8 * M,
        ddt=9 * M, dA=10 * M, dB=11 * M, dC=12 * M, z=None, zs=0, dz=None, ws=13 * M, wsb=1 << 22, dhT=None, dh0=None):
    return lib.selective_scan_bwd(nseq, seqlen, None, dim, N, G, ind, dy, dys, x, 64, dtd, 2 * M, 64, 3 * M, 4 * M, 16,
                                  5 * M, 16, None, z, zs, None, saved, dhT, dx, ddt, dA, dB, dC, None, dz, None, dh0, ws,
                                  wsb, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(saved=None), INVALID), (dict(ws=None), INVALID), (dict(wsb=64), INVALID), (dict(dx=None), INVALID),
    (dict(ddt=None), INVALID), (dict(dA=None), INVALID), (dict(dB=None), INVALID), (dict(dC=None), INVALID),
    (dict(z=21 * M, zs=64), INVALID),                                 # a gate without dz
    (dict(dz=21 * M), INVALID),                                       # dz without a gate
    (dict(dy=None), INVALID), (dict(dys=3), INVALID), (dict(dx=M), INVALID), (dict(dx=8 * M + 2), MISALIGNED),
    (dict(dA=6 * M), INVALID), (dict(dh0=13 * M), INVALID), (dict(N=300), UNSUPPORTED), (dict(ind=5), INVALID),
    (dict(nseq=0), OK),
])
def test_scan_gradient_refusals(lib, kw, code):
    assert bwd(lib, **kw) == code


def upd(lib, batch=4, dim=64, N=16, G=1, state=M, slots=0, idx=None, ind=BF16, x=2 * M, xs=64, dtd=BF16, y=8 * M,
        A=4 * M):
    return lib.selective_state_update(batch, dim, N, G, state, slots, idx, ind, x, xs, dtd, 3 * M, 64, A, 5 * M, 16, 6 * M,
                                      16, None, None, 0, None, ind, y, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), INVALID), (dict(state=None), INVALID), (dict(y=None), INVALID), (dict(A=None), INVALID),
    (dict(idx=7 * M), INVALID), (dict(N=257), UNSUPPORTED), (dict(G=5), INVALID), (dict(xs=10), INVALID),
    (dict(state=M + 4), MISALIGNED), (dict(y=M), INVALID), (dict(x=M), INVALID), (dict(ind=F32), UNSUPPORTED),
    (dict(batch=0), OK),
])
def test_update_refusals(lib, kw, code):
    assert upd(lib, **kw) == code


def cbwd(lib, nseq=2, seqlen=8, dim=64, K=4, ind=BF16, dy=M, x=2 * M, w=3 * M, act=1, init=None, dfin=None, dx=5 * M,
         dw=6 * M, dinit=None, ws=8 * M, wsb=1 << 20):
    return lib.causal_conv1d_bwd(nseq, seqlen, None, dim, K, ind, dy, x, w, None, act, init, dfin, dx, dw, None, dinit, ws,
                                 wsb, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(nseq=-1), INVALID), (dict(dim=0), INVALID), (dict(K=0), INVALID), (dict(K=9), UNSUPPORTED),
    (dict(dim=1 << 24), UNSUPPORTED), (dict(ind=F16), INVALID), (dict(act=2), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(dw=None), INVALID), (dict(dx=None), INVALID), (dict(ws=None), INVALID),
    (dict(wsb=16), INVALID), (dict(dx=2 * M), INVALID), (dict(dx=M + 16), INVALID), (dict(dx=5 * M + 4), MISALIGNED),
    (dict(dinit=8 * M), INVALID),
])
def test_conv_gradient_refusals(lib, kw, code):
    assert cbwd(lib, **kw) == code


def pools(*rows):
    return (ctypes.c_int64 * (3 * len(rows)))(*[v for r in rows for v in r])


@pytest.mark.parametrize("rows,n,slots,src,dst,code", [
    ([(M, 64, 64)], 2, 0, 9 * M, 10 * M, INVALID), ([(M, 64, 32)], 2, 4, 9 * M, 10 * M, INVALID),
    ([(0, 64, 64)], 2, 4, 9 * M, 10 * M, INVALID), ([(M, 0, 64)], 2, 4, 9 * M, 10 * M, INVALID),
    ([(M, 64, 64), (M, 64, 64)], 2, 4, 9 * M, 10 * M, INVALID),       # a pool twice
    ([(M, 64, 64)], -1, 4, 9 * M, 10 * M, INVALID), ([(M, 64, 64)], 2, 4, None, 10 * M, INVALID),
    ([(M, 64, 64)], 2, 4, 9 * M + 4, 10 * M, MISALIGNED), ([(M, 64, 64)], 2, 4, M + 64, 10 * M, INVALID),
    ([(M, 64, 64)], 0, 4, None, None, OK), ([], 2, 4, 9 * M, 10 * M, OK),
])
def test_pool_refusals(lib, rows, n, slots, src, dst, code):
    assert lib.ssm_pool_copy(len(rows), pools(*rows), slots, n, src, dst, None, None) == code
    if src == 9 * M or n == 0:
        assert lib.ssm_pool_zero(len(rows), pools(*rows), slots, n, src, None, None) == code


def test_pool_compact_refusals(lib):
    one = pools((M, 64, 64))
    size = lib.ssm_pool_compact_workspace_size(8, 4)
    assert size == 4 * (8 + 2 * 4 + 1)
    assert lib.ssm_pool_compact(1, one, 8, 4, 9 * M, None, 10 * M, size - 1, None, None) == INVALID
    assert lib.ssm_pool_compact(1, one, 8, 4, None, None, 10 * M, size, None, None) == INVALID
    assert lib.ssm_pool_compact(1, one, 8, 4, 9 * M, None, None, size, None, None) == INVALID
    assert lib.ssm_pool_compact(1, one, 8, 4, 9 * M + 4, None, 10 * M, size, None, None) == MISALIGNED
    assert lib.ssm_pool_compact(1, one, 8, 4, 9 * M, 9 * M, 10 * M, size, None, None) == INVALID
    assert lib.ssm_pool_compact(1025, one, 8, 4, 9 * M, None, 10 * M, size, None, None) == UNSUPPORTED


def test_sizes(lib):
    # a row per 32 tokens and one more per sequence
    assert lib.selective_scan_saved_size(3, 100, 64, 16) == (100 // 32 + 3) * 64 * 16 * 4
    assert lib.selective_scan_saved_size(0, 100, 64, 16) == 0
    for bad in ((0, 10, 64, 16, 1), (1, 10, 64, 300, 1), (1, 10, 64, 16, 3)):
        assert lib.selective_scan_bwd_workspace_size(*bad) == 0
    assert lib.selective_scan_bwd_workspace_size(2, 10, 64, 16, 1) > 0


def test_binding_refuses_cpu_tensors():
    from hybrid_mamba_ssm_b200 import ssm
    t = torch.zeros(4, 8)
    A, B = torch.zeros(8, 2), torch.zeros(4, 1, 2)
    with pytest.raises(ValueError):
        ssm.selective_scan_fwd(t, t, A, B, B, cu_seqlens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        ssm.selective_scan_bwd(t, t, t, A, B, B, t)
    with pytest.raises(ValueError):
        ssm.selective_state_update(torch.zeros(4, 8, 2), t, t, A, B, B)
    with pytest.raises(ValueError):
        ssm.causal_conv1d_bwd(t[None], t[None], torch.zeros(8, 4))
    for f in (lambda: ssm.ssm_pool_copy(t, t[:1, 0].int(), t[:1, 0].int()), lambda: ssm.ssm_pool_zero([t], t[:1, 0].int()),
              lambda: ssm.ssm_pool_compact([t], t[:1, 0].int())):
        with pytest.raises(ValueError):
            f()
