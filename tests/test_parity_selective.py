"""The per-channel selective scan, its gradient and decode update, the conv1d
gradient and the state-pool row operations on the GPU, against the fp64
reference of tests/selective_ref.py (tolerances: derived there)."""
import numpy as np
import pytest
import torch

from tests import selective_ref as ref
from tests.gpu_helpers import Guarded, to_np

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
DT = {"bf16": BF, "f32": F}


def rounder(dtype):
    return lambda v: torch.from_numpy(np.ascontiguousarray(v)).to(dtype).double().numpy()


def dev(v, dtype=F):
    return None if v is None else torch.from_numpy(np.ascontiguousarray(v)).to(dtype).cuda()


def view_of(t, pad):
    """t as a strided view: its rows inside wider ones, `pad` elements from their start."""
    if t is None or not pad:
        return t
    wide = torch.full((t.shape[0], t[0].numel() + 2 * pad + 1), float("nan"), dtype=t.dtype, device=t.device)
    v = wide[:, pad:pad + t[0].numel()].unflatten(1, t.shape[1:])
    v.copy_(t)
    return v


def close(got, want, mag, roundings, name):
    """|got - want| within `roundings` units of 2^-24 of the magnitude sum, and half a step of a bf16 result."""
    g = to_np(got).reshape(want.shape)
    tol = roundings * ref.ULP * np.abs(mag) + 1e-30
    if got.dtype == BF:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (name, int(bad.sum()), float(np.abs(g - want)[bad].max()), np.argwhere(bad)[:3].tolist())


def scan_case(seed, lens, dim, N, G=1, dtype="bf16", dt="bf16", **kw):
    return ref.make_scan(seed, lens, dim, N, G, round_to=rounder(DT[dtype]), dt_round=rounder(DT[dt]), **kw)


def operands(p, dtype, dt, pad=0):
    t, td = DT[dtype], DT[dt]
    x, z, d = (view_of(dev(p[k], ty), pad) for k, ty in (("x", t), ("z", t), ("dt", td)))
    B, C = (view_of(dev(p[k], t), pad) for k in "BC")
    kw = dict(D=dev(p["D"]), z=z, dt_bias=dev(p["bias"]), dt_softplus=p["softplus"], dt_limit=p["limit"])
    return (x, d, dev(p["A"]), B, C), kw


def cu_of(p):
    return torch.tensor(p["cu"], dtype=torch.int32, device="cuda")


LENS = [33, 0, 1, 31, 100, 32, 5, 64]
SHAPES = [  # lens, dim, d_state, groups
    (LENS, 64, 16, 1), (LENS, 130, 16, 2), (LENS, 33, 16, 1), (LENS, 6, 13, 3), ([1], 1, 1, 1), ([70], 7, 3, 1),
    ([3, 40], 128, 4, 1), ([65, 0], 64, 8, 2), ([50], 40, 5, 1), ([50, 7], 96, 24, 1), ([50, 0, 9], 20, 32, 2),
    ([40, 3], 24, 64, 4), ([33], 12, 100, 1), ([34, 1], 10, 128, 1), ([20], 6, 200, 2), ([19, 14], 5, 256, 1),
    ([0, 0], 16, 16, 1),
]
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


def ids(s):
    return f"T{sum(s[0])}-dim{s[1]}-N{s[2]}-G{s[3]}" if isinstance(s, tuple) and len(s) == 4 else None


@pytest.mark.parametrize("dtype,dt", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_scan_packed(shape, dtype, dt):
    from hybrid_mamba_ssm_b200 import ssm
    lens, dim, N, G = shape
    p = scan_case(11, lens, dim, N, G, dtype, dt, gate=N != 24)
    args, kw = operands(p, dtype, dt, pad=3 if dim % 3 == 0 else 0)
    T = sum(lens)
    yg, hg = Guarded((T, dim), DT[dtype]), Guarded((len(lens), dim, N), F)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, hT = ssm.selective_scan_fwd(*args, **kw, initial_state=dev(p["h0"]), cu_seqlens=cu_of(p), y=yg.t, final_state=hg.t,
                                   status=status)
    torch.cuda.synchronize()
    yg.check("y")
    hg.check("final_state")
    assert status.item() == 0
    want, wT, *_ = ref.scan(p)
    mag, mT, *_ = ref.scan(p, magnitude=True)
    close(y, want, mag, ref.scan_rounding(p), "y")
    close(hT, wT, mT, ref.scan_rounding(p), "final state")


@pytest.mark.parametrize("kw", [dict(bias=False), dict(softplus=False, bias=False), dict(limit=(0.01, 0.05)),
                                dict(D=False, h0=False, gate=False)])
def test_scan_options_and_fixed_length(kw):
    from hybrid_mamba_ssm_b200 import ssm
    p = scan_case(12, [45, 45, 45], 64, 16, **kw)
    args, opt = operands(p, "bf16", "bf16")
    x, d, A, B, C = args
    shape = (3, 45)
    opt["z"] = None if opt["z"] is None else opt["z"].view(*shape, 64)
    y, hT = ssm.selective_scan_fwd(x.view(*shape, 64), d.view(*shape, 64), A, B.view(*shape, 1, 16), C.view(*shape, 1, 16),
                                   **opt, initial_state=dev(p["h0"]), y_dtype=F)
    want, wT, *_ = ref.scan(p)
    mag, mT, *_ = ref.scan(p, magnitude=True)
    assert y.shape == (3, 45, 64) and y.dtype == F
    close(y, want, mag, ref.scan_rounding(p), "y")
    close(hT, wT, mT, ref.scan_rounding(p), "final state")


@pytest.mark.parametrize("lens,dim,N,G", [([3000], 32, 16, 1), ([700, 0, 1800, 0, 1, 900], 16, 16, 1), ([2100], 6, 13, 2),
                                          ([0, 0, 2560, 0], 24, 4, 1), ([1500, 1500], 2, 64, 1)])
@pytest.mark.parametrize("inplace", [False, True])
def test_scan_cut_into_ranges(lens, dim, N, G, inplace):
    """Long streams on few channels: ranges that end inside, at and between sequences, in place on a pool."""
    from hybrid_mamba_ssm_b200 import ssm
    T = sum(lens)
    assert ssm.selective_scan_workspace_size(len(lens), T, dim, N, G) > 0
    p = scan_case(13, lens, dim, N, G, "f32", "f32")
    args, kw = operands(p, "f32", "f32")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if inplace:
        slots = list(np.random.default_rng(1).permutation(len(lens) + 2)[:len(lens)])
        pool = torch.full((len(lens) + 2, dim, N), 7.0, device="cuda")
        pool[slots] = dev(p["h0"])
        has = torch.ones(len(lens), dtype=torch.int32, device="cuda")
        has[0] = 0
        p["h0"][0] = 0
        idx = torch.tensor(slots, dtype=torch.int32, device="cuda")
        y, _ = ssm.selective_scan_fwd(*args, **kw, initial_state=pool, final_state=pool, slot_idx=idx, has_initial_state=has,
                                      cu_seqlens=cu_of(p), status=status)
        hT = pool[slots]
        rest = [i for i in range(len(lens) + 2) if i not in slots]
        assert bool((pool[rest] == 7.0).all())
    else:
        y, hT = ssm.selective_scan_fwd(*args, **kw, initial_state=dev(p["h0"]), cu_seqlens=cu_of(p), status=status)
    assert status.item() == 0
    want, wT, *_ = ref.scan(p)
    mag, mT, *_ = ref.scan(p, magnitude=True)
    close(y, want, mag, ref.scan_rounding(p), "y")
    close(hT, wT, mT, ref.scan_rounding(p), "final state")


def test_a_step_of_zero_leaves_the_state_bit_for_bit():
    """exp(0 A) is exactly 1 in every kernel, whatever is added to its argument."""
    from hybrid_mamba_ssm_b200 import ssm
    p = scan_case(14, [40], 64, 16, softplus=False, bias=False, D=False, gate=False)
    (x, d, A, B, C), _ = operands(p, "bf16", "f32")
    h0 = dev(p["h0"])
    zero = torch.zeros_like(d)
    y, hT, saved = ssm.selective_scan_fwd(x, zero, A, B, C, initial_state=h0, cu_seqlens=cu_of(p), save_states=True)
    assert torch.equal(hT, h0)
    dhT = torch.randn_like(h0)
    g = ssm.selective_scan_bwd(torch.zeros_like(x), x, zero, A, B, C, saved, dfinal_state=dhT, cu_seqlens=cu_of(p),
                               want_dinitial=True)
    assert torch.equal(g.dinitial_state, dhT)
    state = h0.clone()
    ssm.selective_state_update(state, x[:1], zero[:1], A, B[:1], C[:1])
    assert torch.equal(state, h0)


def test_scan_slots_in_place():
    from hybrid_mamba_ssm_b200 import ssm
    lens, dim, N = [20, 0, 7, 0], 64, 16
    p = scan_case(14, lens, dim, N)
    args, kw = operands(p, "bf16", "bf16")
    slots, has = [5, 1, 3, 0], [1, 0, 0, 1]
    pool0 = np.random.default_rng(2).standard_normal((7, dim, N)).astype(np.float32)
    pool = dev(pool0)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    y, got = ssm.selective_scan_fwd(*args, **kw, initial_state=pool, final_state=pool, slot_idx=i32(slots),
                                    has_initial_state=i32(has), cu_seqlens=cu_of(p))
    assert got is pool
    p["h0"] = np.stack([pool0[s].astype(np.float64) * h for s, h in zip(slots, has)])
    want, wT, *_ = ref.scan(p)
    mag, mT, *_ = ref.scan(p, magnitude=True)
    close(y, want, mag, ref.scan_rounding(p), "y")
    close(pool[slots], wT, mT, ref.scan_rounding(p), "pool rows")
    assert bool((pool[[2, 4, 6]] == dev(pool0)[[2, 4, 6]]).all())
    # an index outside the pool skips its sequence and is reported
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool, y = dev(pool0), torch.full((27, dim), 3.0, dtype=BF, device="cuda")
    ssm.selective_scan_fwd(*args, **kw, initial_state=pool, final_state=pool, slot_idx=i32([7, 1, 3, 0]), cu_seqlens=cu_of(p),
                           y=y, status=status)
    assert status.item() == ssm.SSM_ERR_DEVICE_INPUT
    assert bool((y[:20] == 3.0).all()) and not bool((y[20:] == 3.0).all())


@pytest.mark.parametrize("cu", [[0, 30, 20, 64], [3, 20, 40, 64], [0, 20, 40, 60], [0, 20, 90, 64], [0, -5, 40, 64]])
@pytest.mark.parametrize("dim", [64, 4096])
def test_scan_bad_offsets_are_reported(cu, dim):
    """Inconsistent offsets: nothing outside the buffers is touched and the status says so (with few channels the
    stream is also long enough to be cut)."""
    from hybrid_mamba_ssm_b200 import ssm
    k = 50 if dim == 64 else 1
    p = scan_case(15, [64 * k], dim, 16)
    args, kw = operands(p, "bf16", "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    yg, hg = Guarded((64 * k, dim), BF), Guarded((3, dim, 16), F)
    off = torch.tensor([v * k for v in cu], dtype=torch.int32, device="cuda")
    ssm.selective_scan_fwd(*args, **kw, cu_seqlens=off, y=yg.t, final_state=hg.t, status=status)
    torch.cuda.synchronize()
    yg.check("y")
    hg.check("final_state")
    assert status.item() == ssm.SSM_ERR_DEVICE_INPUT
    saved = torch.zeros(ssm.selective_scan_saved_size(3, 64 * k, dim, 16) // 4, device="cuda")
    status.zero_()
    ssm.selective_scan_bwd(torch.ones_like(args[0]), *args, saved, **kw, cu_seqlens=off, status=status)
    torch.cuda.synchronize()
    assert status.item() == ssm.SSM_ERR_DEVICE_INPUT


def test_scan_nonfinite_values_stay_in_their_sequence_and_channel():
    from hybrid_mamba_ssm_b200 import ssm
    p = scan_case(16, [40, 40, 40], 64, 16)
    args, kw = operands(p, "bf16", "bf16")
    clean, cT = ssm.selective_scan_fwd(*args, **kw, cu_seqlens=cu_of(p))
    x, d, A, B, C = args
    x[45, 9] = float("nan")
    d[50, 11] = float("inf")
    x[60, 13] = float("inf")
    y, hT = ssm.selective_scan_fwd(*args, **kw, cu_seqlens=cu_of(p))
    rest = [c for c in range(64) if c not in (9, 11, 13)]
    for s in (slice(0, 40), slice(80, 120)):
        assert bool((y[s] == clean[s]).all())
    assert bool((y[40:80, rest] == clean[40:80, rest]).all()) and bool((hT[1][rest] == cT[1][rest]).all())
    assert bool(y[45:80, 9].isnan().all()) and bool(hT[1, 9].isnan().all())
    assert not bool(y[60:80, 13].isfinite().any())
    assert bool((y[40:50, 11] == clean[40:50, 11]).all())


@pytest.mark.parametrize("dtype,dt", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_scan_gradient(shape, dtype, dt):
    from hybrid_mamba_ssm_b200 import ssm
    lens, dim, N, G = shape
    gate = N != 24
    p = scan_case(17, lens, dim, N, G, dtype, dt, gate=gate, limit=(0.004, 0.08) if N == 8 else None)
    args, kw = operands(p, dtype, dt, pad=3 if dim % 3 == 0 else 0)
    rng = np.random.default_rng(18)
    dy, dhT = rounder(DT[dtype])(rng.standard_normal((sum(lens), dim))), rng.standard_normal((len(lens), dim, N))
    dhT = dhT.astype(np.float32).astype(np.float64)
    y, hT, saved = ssm.selective_scan_fwd(*args, **kw, initial_state=dev(p["h0"]), cu_seqlens=cu_of(p), save_states=True)
    close(y, ref.scan(p)[0], ref.scan(p, magnitude=True)[0], ref.scan_rounding(p), "y")
    # uncut, saving the states changes nothing (cut calls agree to rounding: they join states in another order)
    uncut = dict(initial_state=dev(p["h0"]), cu_seqlens=cu_of(p), workspace=None)
    assert torch.equal(ssm.selective_scan_fwd(*args, **kw, **uncut, save_states=True)[0],
                       ssm.selective_scan_fwd(*args, **kw, **uncut)[0])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run = lambda: ssm.selective_scan_bwd(dev(dy, DT[dtype]), *args, saved, **kw, dfinal_state=dev(dhT),  # noqa: E731
                                         cu_seqlens=cu_of(p), want_dinitial=True, status=status)
    g, again = run(), run()
    assert status.item() == 0
    want, mag = ref.scan_grad(p, dy, dhT), ref.scan_grad(p, dy, dhT, magnitude=True)
    n = ref.scan_rounding(p)
    for name, t, k in [("dx", g.dx, "dx"), ("ddt", g.ddt, "ddt"), ("dA", g.dA, "dA"), ("dB", g.dB, "dB"),
                       ("dC", g.dC, "dC"), ("dD", g.dD, "dD"), ("dz", g.dz, "dz"), ("ddt_bias", g.ddt_bias, "dbias"),
                       ("dinitial_state", g.dinitial_state, "dh0")]:
        if want[k] is None:
            assert t is None
            continue
        many = sum(lens) + dim if name in ("dA", "dB", "dC", "dD", "ddt_bias") else 0
        if name in ("ddt", "ddt_bias") and p["limit"] is not None:
            v, _ = ref.step_size(p["dt"], p["bias"], True, None)   # steps within rounding of the clamp may go either way
            edge = (np.abs(v - 0.004) < 1e-8) | (np.abs(v - 0.08) < 1e-7)
            assert not edge.any()
        close(t, want[k], mag[k], n + many, name)
    for t, u in zip(g, again):
        assert t is None or bool((t == u).all())                   # sums in a fixed order: equal bits


def test_scan_gradient_many_sequences_share_a_cta():
    """More sequences than the gradient deals out (64): several per CTA, their dA, dD and bias sums added."""
    from hybrid_mamba_ssm_b200 import ssm
    lens = [int(v) for v in np.random.default_rng(4).integers(0, 9, 150)]
    p = scan_case(19, lens, 10, 5, dtype="f32", dt="f32")
    args, kw = operands(p, "f32", "f32")
    rng = np.random.default_rng(20)
    dy = rounder(F)(rng.standard_normal((sum(lens), 10)))
    *_, saved = ssm.selective_scan_fwd(*args, **kw, initial_state=dev(p["h0"]), cu_seqlens=cu_of(p), save_states=True)
    g = ssm.selective_scan_bwd(dev(dy), *args, saved, **kw, cu_seqlens=cu_of(p), want_dinitial=True)
    zero = np.zeros((150, 10, 5))
    want, mag = ref.scan_grad(p, dy, zero), ref.scan_grad(p, dy, zero, magnitude=True)
    n = ref.scan_rounding(p) + sum(lens) + 10
    for t, k in [(g.dx, "dx"), (g.dA, "dA"), (g.dB, "dB"), (g.dC, "dC"), (g.dD, "dD"), (g.ddt_bias, "dbias"),
                 (g.dinitial_state, "dh0")]:
        close(t, want[k], mag[k], n, k)


@pytest.mark.parametrize("lens,dim,N,G", [([1500, 0, 700, 1], 8, 16, 1), ([2000], 6, 5, 2), ([0, 1100, 0], 3, 64, 1),
                                          ([640, 640], 16, 4, 1)])
def test_scan_gradient_cut_into_segments(lens, dim, N, G):
    """Long sequences on few channels: states and their gradients cross the cuts between segments."""
    from hybrid_mamba_ssm_b200 import ssm
    p = scan_case(23, lens, dim, N, G, "f32", "f32")
    args, kw = operands(p, "f32", "f32")
    rng = np.random.default_rng(24)
    dy, dhT = rounder(F)(rng.standard_normal((sum(lens), dim))), rounder(F)(rng.standard_normal((len(lens), dim, N)))
    y, hT, saved = ssm.selective_scan_fwd(*args, **kw, initial_state=dev(p["h0"]), cu_seqlens=cu_of(p), save_states=True)
    g = ssm.selective_scan_bwd(dev(dy), *args, saved, **kw, dfinal_state=dev(dhT), cu_seqlens=cu_of(p), want_dinitial=True)
    want, mag = ref.scan_grad(p, dy, dhT), ref.scan_grad(p, dy, dhT, magnitude=True)
    n = ref.scan_rounding(p)
    close(y, ref.scan(p)[0], ref.scan(p, magnitude=True)[0], n, "y")
    for t, k in [(g.dx, "dx"), (g.ddt, "ddt"), (g.dA, "dA"), (g.dB, "dB"), (g.dC, "dC"), (g.dD, "dD"), (g.dz, "dz"),
                 (g.ddt_bias, "dbias"), (g.dinitial_state, "dh0")]:
        close(t, want[k], mag[k], n + (sum(lens) + dim if k in ("dA", "dB", "dC", "dD", "dbias") else 0), k)


def _parts_bytes(channels, lens, dim, N, G):
    """Workspace of whole sequences whose CTAs take `channels` channels (the parts of dB, dC, then dA, dD, the bias)."""
    up = lambda v: (v + 15) // 16 * 16  # noqa: E731
    tiles, n = -(-(dim // G) // channels), len(lens)
    return 2 * up(tiles * sum(lens) * G * N * 4) + up(n * dim * N * 4) + 2 * up(n * dim * 4)


BIG = [([int(v) for v in np.random.default_rng(8).integers(0, 9, 40)], dim, N, G)
       for dim, N, G in [(1024, 8, 1), (1030, 16, 2), (1024, 16, 2), (520, 32, 1), (264, 64, 4), (130, 128, 2)]]


@pytest.mark.parametrize("dtype,dt", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("shape", BIG + [([200], 8192, 16, 1), ([640, 100, 40], 1024, 64, 1)], ids=ids)
def test_scan_gradient_when_the_device_is_full(shape, dtype, dt):
    """Two sets of channels a warp, whole sequences and cut ones: the sums over channels and sequences of many CTAs."""
    from hybrid_mamba_ssm_b200 import ssm
    lens, dim, N, G = shape
    if len(lens) == 40:
        lanes = {8: 2, 16: 4, 32: 8, 64: 16, 128: 32}[N]
        assert ssm.selective_scan_bwd_workspace_size(40, sum(lens), dim, N, G) == _parts_bytes(256 // lanes, lens, dim, N, G)
    p = scan_case(25, lens, dim, N, G, dtype, dt)
    args, kw = operands(p, dtype, dt)
    rng = np.random.default_rng(26)
    dy, dhT = rounder(DT[dtype])(rng.standard_normal((sum(lens), dim))), rounder(F)(rng.standard_normal((len(lens), dim, N)))
    y, _, saved = ssm.selective_scan_fwd(*args, **kw, initial_state=dev(p["h0"]), cu_seqlens=cu_of(p), save_states=True)
    g = ssm.selective_scan_bwd(dev(dy, DT[dtype]), *args, saved, **kw, dfinal_state=dev(dhT), cu_seqlens=cu_of(p),
                               want_dinitial=True)
    want, mag = ref.scan_grad(p, dy, dhT), ref.scan_grad(p, dy, dhT, magnitude=True)
    n = ref.scan_rounding(p)
    for t, k in [(g.dx, "dx"), (g.ddt, "ddt"), (g.dA, "dA"), (g.dB, "dB"), (g.dC, "dC"), (g.dD, "dD"), (g.dz, "dz"),
                 (g.ddt_bias, "dbias"), (g.dinitial_state, "dh0")]:
        close(t, want[k], mag[k], n + (sum(lens) + dim if k in ("dA", "dB", "dC", "dD", "dbias") else 0), k)


@pytest.mark.parametrize("dtype,dt", TYPES)
@pytest.mark.parametrize("batch,dim,N,G", [(1, 64, 16, 1), (5, 130, 16, 2), (3, 33, 13, 1), (9, 7, 1, 1), (4, 12, 4, 3),
                                           (6, 20, 8, 1), (2, 24, 32, 2), (5, 10, 64, 1), (3, 6, 128, 1), (7, 5, 100, 1),
                                           (2, 4, 256, 2), (1, 3, 201, 1)])
def test_update(batch, dim, N, G, dtype, dt):
    from hybrid_mamba_ssm_b200 import ssm
    p = scan_case(21, [1] * batch, dim, N, G, dtype, dt, gate=N != 8)
    args, kw = operands(p, dtype, dt, pad=1 if dim % 2 else 0)
    sg, yg = Guarded((batch, dim, N), F, init=dev(p["h0"])), Guarded((batch, dim), DT[dtype])
    y = ssm.selective_state_update(sg.t, *args, **kw, y=yg.t)
    torch.cuda.synchronize()
    sg.check("state")
    yg.check("y")
    want, wT, *_ = ref.scan(p)
    mag, mT, *_ = ref.scan(p, magnitude=True)
    close(y, want, mag, ref.scan_rounding(p), "y")
    close(sg.t, wT, mT, ref.scan_rounding(p), "state")
    # the same token through the prefill call
    y2, h2 = ssm.selective_scan_fwd(*args, **kw, initial_state=dev(p["h0"]), cu_seqlens=cu_of(p))
    close(y2, want, mag, ref.scan_rounding(p), "prefill y")
    close(h2, wT, mT, ref.scan_rounding(p), "prefill state")


def test_update_slots_padding_and_bad_index():
    from hybrid_mamba_ssm_b200 import ssm
    p = scan_case(22, [1] * 6, 64, 16)
    args, kw = operands(p, "bf16", "bf16")
    pool0 = torch.randn(8, 64, 16, device="cuda")
    pool, y = pool0.clone(), torch.full((6, 64), 5.0, dtype=BF, device="cuda")
    slots = [3, -1, 0, 9, 7, -4]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.tensor(slots, dtype=torch.int32, device="cuda")
    ssm.selective_state_update(pool, *args, **kw, slot_idx=idx, y=y, status=status)
    assert status.item() == ssm.SSM_ERR_DEVICE_INPUT
    p["h0"] = np.stack([to_np(pool0[s]) if 0 <= s < 8 else np.zeros((64, 16)) for s in slots])
    want, wT, *_ = ref.scan(p)
    mag, mT, *_ = ref.scan(p, magnitude=True)
    on = [0, 2, 4]
    close(y[on], want[on], mag[on], ref.scan_rounding(p), "y")
    close(pool[[3, 0, 7]], wT[on], mT[on], ref.scan_rounding(p), "state")
    assert bool((y[[1, 3, 5]] == 5.0).all())
    left = [1, 2, 4, 5, 6]
    assert bool((pool[left] == pool0[left]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("lens,dim", [([130, 0, 1, 2, 300, 5, 3], 64), ([260], 33), ([1], 1), ([0, 0], 8), ([7, 121, 4, 250], 258)])
def test_conv_gradient(lens, dim, K, dtype):
    from hybrid_mamba_ssm_b200 import ssm
    rng = np.random.default_rng(K + dim)
    r = rounder(DT[dtype])
    f = rounder(F)
    n, T = len(lens), sum(lens)
    act, init, dfin = K != 3, dim != 33, dim % 2 == 0
    p = {"x": r(rng.standard_normal((T, dim))), "weight": f(rng.standard_normal((dim, K))), "act": act,
         "bias": f(rng.standard_normal(dim)), "init": r(rng.standard_normal((n, dim, K - 1))) if init else None,
         "cu": ref.offsets(lens)}
    dy, df = r(rng.standard_normal((T, dim))), r(rng.standard_normal((n, dim, K - 1))) if dfin else None
    t = DT[dtype]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run = lambda: ssm.causal_conv1d_bwd(dev(dy, t), dev(p["x"], t), dev(p["weight"]), dev(p["bias"]),  # noqa: E731
                                        initial_state=dev(p["init"], t), dfinal_state=dev(df, t),
                                        cu_seqlens=cu_of(p), activation="silu" if act else None, status=status)
    got, again = run(), run()
    assert status.item() == 0
    want, mag = ref.conv_grad(p, dy, df), ref.conv_grad(p, dy, df, magnitude=True)
    # pre is off by (K + 2) roundings of its magnitude, and the slope of the activation changes by at most half of
    # that; its exponential and reciprocal are off by 2^-22 each
    pre = sum(np.abs(p["weight"][:, k]) for k in range(K)) * np.abs(p["x"]).max(initial=1) + np.abs(p["bias"])
    per = 32 + K + (K + 2) * float(pre.max())
    # a gradient through a small slope: the slope's own error is absolute (it is at most 1.1), so the magnitude sums
    # take a slope of 1.1 throughout
    flat = ref.conv_grad({**p, "act": False}, 1.1 * dy, df, magnitude=True)
    for name, v, k in [("dx", got[0], "dx"), ("dweight", got[1], "dw"), ("dbias", got[2], "db"), ("dinitial", got[3], "dinit")]:
        if name == "dinitial" and not init:
            assert v is None
            continue
        many = T if name in ("dweight", "dbias") else 0
        close(v, want[k], np.maximum(mag[k], flat[k]), per + many, name)
    for a, b in zip(got, again):
        assert a is None or bool((a == b).all())


@pytest.mark.parametrize("T,dim,dtype", [(6000, 13000, "bf16"), (3000, 4097, "bf16"), (5000, 2000, "f32")])
def test_conv_gradient_of_large_inputs(T, dim, dtype):
    """Longer tiles: a few channels and all tokens against the reference (channels are independent)."""
    from hybrid_mamba_ssm_b200 import ssm
    t, K = DT[dtype], 4
    cu = [0, T // 3, T // 3 + 1, T]
    gen = torch.Generator(device="cuda").manual_seed(7)
    x, dy = (torch.randn(T, dim, generator=gen, device="cuda").to(t) for _ in range(2))
    w, b = torch.randn(dim, K, generator=gen, device="cuda") * 0.5, torch.randn(dim, generator=gen, device="cuda")
    got = ssm.causal_conv1d_bwd(dy, x, w, b, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    pick = [0, 1, 255, 256, dim // 2, dim - 2, dim - 1]
    p = {"x": to_np(x[:, pick]), "weight": to_np(w[pick]), "bias": to_np(b[pick]), "act": True, "init": None, "cu": cu}
    g = to_np(dy[:, pick])
    want, mag = ref.conv_grad(p, g, None), ref.conv_grad({**p, "act": False}, 1.1 * g, None, magnitude=True)
    pre = sum(np.abs(p["weight"][:, k]) for k in range(K)) * np.abs(p["x"]).max() + np.abs(p["bias"])
    per = 32 + K + (K + 2) * float(pre.max())          # as in test_conv_gradient
    close(got[0][:, pick], want["dx"], mag["dx"], per, "dx")
    close(got[1][pick], want["dw"], mag["dw"], per + T, "dweight")
    close(got[2][pick], want["db"], mag["db"], per + T, "dbias")


def test_conv_gradient_bad_offsets():
    from hybrid_mamba_ssm_b200 import ssm
    x = torch.randn(64, 32, device="cuda")
    for cu in ([0, 40, 20, 64], [0, 20, 90, 64], [0, -3, 40, 64], [5, 20, 40, 64], [0, 10, 20, 50]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ssm.causal_conv1d_bwd(x, x.clone(), torch.randn(32, 4, device="cuda"), status=status,
                              cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert status.item() == ssm.SSM_ERR_DEVICE_INPUT, cu


# ---------------------------------------------------------------------------
# pools
# ---------------------------------------------------------------------------
def make_pools(slots, kinds):
    g = torch.Generator(device="cuda").manual_seed(5)
    out = []
    for shape, dtype in kinds:
        t = torch.randint(0, 100, (slots, *shape), generator=g, device="cuda")
        out.append(t.to(dtype))
    return out


KINDS = [[((64, 16), F), ((64, 3), BF)], [((33,), torch.int8), ((7, 3), BF)], [((5,), F)] * 70, [((1,), torch.uint8)],
         [((16, 4), F), ((2, 3), F), ((9,), F), ((3,), BF), ((11,), torch.uint8)]]


@pytest.mark.parametrize("kinds", KINDS, ids=["states", "odd", "many", "bytes", "every-width"])
@pytest.mark.parametrize("pairs", [[(0, 3), (0, 4), (1, 5)], [(0, 1), (1, 2), (2, 0), (0, 1)], [(4, 4), (-1, 2), (3, -2), (9, 0)],
                                   [(i % 4, 4 + i % 6) for i in range(40)], [(i, i + 1) for i in range(9)], []])
def test_pool_copy_is_the_loop(kinds, pairs):
    """Forks, chains, cycles, repeated destinations and padding entries: the rows after a loop over the list."""
    from hybrid_mamba_ssm_b200 import ssm
    pools = make_pools(10, kinds)
    want = [p.clone() for p in pools]
    for s, d in pairs:
        if s >= 0 and d >= 0:
            for w in want:
                w[d] = w[s].clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.tensor(pairs, dtype=torch.int32, device="cuda").reshape(-1, 2)
    ssm.ssm_pool_copy(pools, idx[:, 0].contiguous(), idx[:, 1].contiguous(), status=status)
    for p, w in zip(pools, want):
        assert bool((p == w).all())
    assert status.item() == 0


def test_pool_copy_and_zero_skip_indices_outside_the_pool():
    from hybrid_mamba_ssm_b200 import ssm
    pool = make_pools(6, [((40,), F)])[0]
    before = pool.clone()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    status = i32(0)
    ssm.ssm_pool_copy(pool, i32(6, 1, 0), i32(2, 100, 5), status=status)
    before[5] = before[0]
    assert status.item() == ssm.SSM_ERR_DEVICE_INPUT and bool((pool == before).all())
    status.zero_()
    ssm.ssm_pool_zero(pool, i32(1, -1, 6, 1, 3), status=status)
    before[[1, 3]] = 0
    assert status.item() == ssm.SSM_ERR_DEVICE_INPUT and bool((pool == before).all())


def test_pool_rows_of_a_stacked_tensor():
    """Layers interleaved in one tensor [slots, layers, ...]: a layer's pool has a row stride."""
    from hybrid_mamba_ssm_b200 import ssm
    big = make_pools(6, [((3, 20), F)])[0]
    before = big.clone()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ssm.ssm_pool_copy([big[:, 0], big[:, 2]], i32(1), i32(4))
    before[4, 0], before[4, 2] = before[1, 0], before[1, 2]
    assert bool((big == before).all())
    with pytest.raises(ValueError):
        ssm.ssm_pool_copy([big.transpose(1, 2)], i32(0), i32(1))       # rows not contiguous
    with pytest.raises(ValueError):
        ssm.ssm_pool_copy([big, big[:5, 0]], i32(0), i32(1))           # other numbers of slots


@pytest.mark.parametrize("slots,table", [(10, [7, 2, 9, 0]), (10, [0, 1, 2]), (10, [9, -1, 9, 4, -3]), (10, []), (10, [-1]),
                                         (10, list(range(10))[::-1]), (1, [0]), (2500, "random"), (2500, "top"), (10, [3, 12, 8])])
def test_pool_compact(slots, table):
    from hybrid_mamba_ssm_b200 import ssm
    rng = np.random.default_rng(6)
    if table == "random":
        table = rng.permutation(slots)[:900].tolist()
    elif table == "top":
        table = list(range(slots - 1, slots - 1000, -1))
    pools = make_pools(slots, [((8,), F), ((3,), BF)])
    want = [p.clone() for p in pools]
    live = sorted({t for t in table if 0 <= t < slots})
    n = len(live)
    to = dict(zip([t for t in live if t >= n], [i for i in range(n) if i not in set(live)]))
    for w in want:
        for a, b in to.items():
            w[b] = w[a]
    idx = torch.tensor(table, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    count = ssm.ssm_pool_compact(pools, idx, status=status)
    assert count.item() == n
    assert idx.tolist() == [to.get(t, t) for t in table]
    for p, w in zip(pools, want):
        assert bool((p == w).all())
    assert status.item() == (ssm.SSM_ERR_DEVICE_INPUT if any(t >= slots for t in table) else 0)


# ---------------------------------------------------------------------------
# together, captured, on other streams
# ---------------------------------------------------------------------------
def test_mixer_training_step():
    """conv -> scan -> gradient of both, as a training step runs them, against the chained fp64 reference."""
    from hybrid_mamba_ssm_b200 import ssm
    lens, dim, N, K = [70, 3, 41], 64, 16, 4
    p = scan_case(31, lens, dim, N, dtype="f32", dt="f32", h0=False)
    rng = np.random.default_rng(32)
    f = rounder(F)
    q = {"x": f(rng.standard_normal((sum(lens), dim))), "weight": f(0.5 * rng.standard_normal((dim, K))),
         "bias": f(0.1 * rng.standard_normal(dim)), "act": True, "init": None, "cu": p["cu"]}
    dy = f(rng.standard_normal((sum(lens), dim)))
    (_, d, A, B, C), kw = operands(p, "f32", "f32")
    cu, raw, w, b = cu_of(p), dev(q["x"]), dev(q["weight"]), dev(q["bias"])
    x = ssm.causal_conv1d_fwd(raw, w, b, cu_seqlens=cu)
    y, _, saved = ssm.selective_scan_fwd(x, d, A, B, C, **kw, cu_seqlens=cu, save_states=True)
    g = ssm.selective_scan_bwd(dev(dy), x, d, A, B, C, saved, **kw, cu_seqlens=cu)
    draw, dw, db, _ = ssm.causal_conv1d_bwd(g.dx, raw, w, b, cu_seqlens=cu)
    pre = np.stack([q["bias"] + sum((q["x"][t - K + 1 + k] if t - K + 1 + k >= lo else 0) * q["weight"][:, k] for k in range(K))
                    for lo, hi in zip(p["cu"], p["cu"][1:]) for t in range(lo, hi)])
    p["x"] = ref.silu(pre)
    zero = np.zeros((3, dim, N))
    want = ref.scan_grad(p, dy, zero)
    wc = ref.conv_grad(q, want["dx"], None)
    # the rounding of x enters all of it: relative to the largest value, a few times scan_rounding's share
    for name, t, r in [("y", y, ref.scan(p)[0]), ("dA", g.dA, want["dA"]), ("dB", g.dB, want["dB"]), ("dz", g.dz, want["dz"]),
                       ("draw", draw, wc["dx"]), ("dweight", dw, wc["dw"]), ("dbias", db, wc["db"])]:
        assert np.abs(to_np(t) - r).max() <= 4 * ref.scan_rounding(p) * ref.ULP * np.abs(r).max(), name


def test_serving_prefill_fork_decode_retire():
    """Prefill into pool rows, fork a request, decode all, free one, compact, decode on: every row as if it ran alone."""
    from hybrid_mamba_ssm_b200 import ssm
    dim, N, K, steps = 64, 16, 4, 3
    lens = [20, 9]
    rng = np.random.default_rng(41)
    f = rounder(F)
    A, D = f(-np.exp(rng.uniform(0, 2, (dim, N)))), f(rng.standard_normal(dim))
    bias, w, cb = f(rng.uniform(-5, -2, dim)), f(0.5 * rng.standard_normal((dim, K))), f(rng.standard_normal(dim))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pool, conv = torch.zeros(6, dim, N, device="cuda"), torch.zeros(6, dim, K - 1, device="cuda")
    kw = dict(D=dev(D), dt_bias=dev(bias), dt_softplus=True)

    def tokens(n):
        return [f(rng.standard_normal((n, dim))), f(0.5 * rng.standard_normal((n, dim))),
                f(rng.standard_normal((n, 1, N))), f(rng.standard_normal((n, 1, N)))]

    first = tokens(sum(lens))
    slots = i32(4, 2)
    x = ssm.causal_conv1d_fwd(dev(first[0]), dev(w), dev(cb), conv_state=conv, cu_seqlens=i32(0, 20, 29), slot_idx=slots)
    ssm.selective_scan_fwd(x, dev(first[1]), dev(A), dev(first[2]), dev(first[3]), **kw, initial_state=pool, final_state=pool,
                           slot_idx=slots, has_initial_state=i32(0, 0), cu_seqlens=i32(0, 20, 29))
    logs = [[v[a:b] for v in first] for a, b in ((0, 20), (20, 29))]       # what each request has seen
    ssm.ssm_pool_copy([pool, conv], i32(4), i32(5))                        # request 2 forks from request 0
    logs.append([v.copy() for v in logs[0]])
    table = i32(4, 2, 5)
    got = []

    def decode(rows, n):
        for _ in range(n):
            t = tokens(len(rows))
            x = ssm.causal_conv1d_update(dev(t[0]), dev(w), dev(cb), conv, slot_idx=table)
            got.append((list(rows), ssm.selective_state_update(pool, x, dev(t[1]), dev(A), dev(t[2]), dev(t[3]), **kw,
                                                               slot_idx=table),
                        [len(logs[r][0]) for r in rows]))
            for k, r in enumerate(rows):
                logs[r] = [np.concatenate([v, u[k:k + 1]]) for v, u in zip(logs[r], t)]

    decode([0, 1, 2], steps)
    ssm.ssm_pool_zero([pool, conv], i32(4))                                # request 0 ends
    table = i32(2, 5)
    count = ssm.ssm_pool_compact([pool, conv], table)
    assert count.item() == 2 and table.tolist() == [0, 1]                  # rows 2 and 5 move into 0 and 1, ascending
    decode([1, 2], steps)
    for r in (0, 1, 2):
        lx = np.concatenate([np.zeros((K - 1, dim)), logs[r][0]])
        n = len(logs[r][0])
        xin = ref.silu(cb + sum(lx[k:k + n] * w[:, k] for k in range(K)))
        p = {"x": xin, "dt": logs[r][1], "A": A, "B": logs[r][2], "C": logs[r][3], "D": D, "z": None, "h0": None, "cu": [0, n],
             "bias": bias, "softplus": True, "limit": None}
        want, wT, *_ = ref.scan(p)
        mag, mT, *_ = ref.scan(p, magnitude=True)
        lim = 2 * ref.scan_rounding(p)                                     # the conv's roundings enter through x
        for rows, y, at in got:
            if r in rows:
                k = rows.index(r)
                close(y[k], want[at[k]], mag[at[k]], lim, f"request {r} token {at[k]}")
        if r:
            close(pool[r - 1], wT[0], mT[0], lim, f"request {r} state")


def test_captured_step_replays_on_new_inputs():
    """Forward, gradient, decode, conv gradient and pool calls in one CUDA graph: a replay on new inputs equals eager
    calls, while an eager result of the same inputs is alive; two graphs with workspaces of their own do not mix."""
    from hybrid_mamba_ssm_b200 import ssm

    def make(seed):
        p = scan_case(seed, [40, 0, 33], 64, 16)
        args, kw = operands(p, "bf16", "bf16")
        long = scan_case(seed + 1, [1200], 16, 16)
        la, lk = operands(long, "bf16", "bf16")
        state = dev(np.random.default_rng(seed).standard_normal((73, 64, 16)))
        return dict(args=args, kw=kw, la=la, lk=lk, state=state, dy=torch.randn_like(args[0]), w=torch.randn(64, 4, device="cuda"),
                    cu=cu_of(p), lcu=cu_of(long), src=torch.tensor([0], dtype=torch.int32, device="cuda"),
                    dst=torch.tensor([72], dtype=torch.int32, device="cuda"))

    def step(s):
        y, hT, saved = ssm.selective_scan_fwd(*s["args"], **s["kw"], cu_seqlens=s["cu"], save_states=True)
        g = ssm.selective_scan_bwd(s["dy"], *s["args"], saved, **s["kw"], cu_seqlens=s["cu"])
        ly, lT = ssm.selective_scan_fwd(*s["la"], **s["lk"], cu_seqlens=s["lcu"])
        u = ssm.selective_state_update(s["state"][:73], *s["args"], **s["kw"])
        c = ssm.causal_conv1d_bwd(s["dy"], s["args"][0], s["w"], cu_seqlens=s["cu"])
        ssm.ssm_pool_copy(s["state"], s["src"], s["dst"])
        ssm.ssm_pool_zero(s["state"], s["src"])
        return [t for t in (y, hT, *g, ly, lT, u, *c) if t is not None] + [s["state"].clone()]

    a, b, keep = make(51), make(52), make(53)
    alive = step(make(54))
    fresh = {k: v.clone() for k, v in (("a", a["state"]), ("b", b["state"]))}
    step(a)
    torch.cuda.synchronize()
    a["state"].copy_(fresh["a"])
    graphs = []
    for s in (a, b):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
            out = step(s)
        graphs.append((graph, out))
    a["state"].copy_(fresh["a"])
    b["state"].copy_(fresh["b"])
    for _ in range(2):
        for s in (a, b):
            s["dy"].copy_(keep["dy"])
            s["state"].copy_(keep["state"])
            for t, u in zip(s["args"] + s["la"], keep["args"] + keep["la"]):
                t.copy_(u)
        for k in ("D", "z", "dt_bias"):
            for s in (a, b):
                s["kw"][k].copy_(keep["kw"][k])
                s["lk"][k].copy_(keep["lk"][k])
        for s in (a, b):
            s["w"].copy_(keep["w"])
        torch.cuda.synchronize()
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        start = keep["state"].clone()
        want = step(keep)
        keep["state"].copy_(start)
        torch.cuda.synchronize()
        for _, out in graphs:
            for t, u in zip(out, want):
                assert torch.equal(t, u)
    assert all(bool(t.float().isfinite().all()) for t in alive)


def test_side_stream_argument():
    """stream=: outputs and workspaces belong to that stream, whatever the current stream does meanwhile."""
    from hybrid_mamba_ssm_b200 import ssm
    p = scan_case(61, [1500], 16, 16)
    args, kw = operands(p, "bf16", "bf16")
    want = ssm.selective_scan_fwd(*args, **kw, cu_seqlens=cu_of(p))
    cu = cu_of(p)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for _ in range(5):
        outs.append(ssm.selective_scan_fwd(*args, **kw, cu_seqlens=cu, stream=side))
        for _ in range(4):
            torch.empty(1 << 16, device="cuda").fill_(float("nan"))        # work of the current stream on freed blocks
    torch.cuda.synchronize()
    for y, h in outs:
        assert torch.equal(y, want[0]) and torch.equal(h, want[1])


def test_offsets_beyond_32_bits():
    """A pool and rows whose element offsets pass 2^31: the last rows are the ones addressed."""
    from hybrid_mamba_ssm_b200 import ssm
    dim, N, slots = 8192, 64, 4200                                         # 2.2e9 elements, 8.8 GB
    pool = torch.zeros(slots, dim, N, device="cuda")
    p = scan_case(71, [1, 1], dim, N, h0=False)
    args, kw = operands(p, "bf16", "bf16")
    idx = torch.tensor([slots - 1, 1], dtype=torch.int32, device="cuda")
    y = ssm.selective_state_update(pool, *args, **kw, slot_idx=idx)
    want, wT, *_ = ref.scan(p)
    mag, mT, *_ = ref.scan(p, magnitude=True)
    close(y, want, mag, ref.scan_rounding(p), "y")
    close(pool[slots - 1], wT[0], mT[0], ref.scan_rounding(p), "last row")
    i32 = lambda v: torch.tensor([v], dtype=torch.int32, device="cuda")  # noqa: E731
    ssm.ssm_pool_copy(pool, i32(slots - 1), i32(slots - 3))
    assert torch.equal(pool[slots - 3], pool[slots - 1])
    ssm.ssm_pool_zero(pool, i32(slots - 1))
    assert not bool(pool[slots - 1].any()) and bool(pool[slots - 3].any())
    table = i32(slots - 3)
    assert ssm.ssm_pool_compact(pool, table).item() == 1 and table.item() == 0
    close(pool[0], wT[0], mT[0], ref.scan_rounding(p), "moved row")


def test_two_streams_at_once():
    """Calls that overlap on the GPU have outputs and workspaces of their own."""
    from hybrid_mamba_ssm_b200 import ssm
    cases = [scan_case(81 + k, [700, 300], 24, 16) for k in range(2)]
    ops = [operands(p, "bf16", "bf16") for p in cases]
    cu = cu_of(cases[0])

    def step(k):
        args, kw = ops[k]
        y, h, saved = ssm.selective_scan_fwd(*args, **kw, cu_seqlens=cu, save_states=True)
        return [y, h, *[t for t in ssm.selective_scan_bwd(args[0], *args, saved, **kw, cu_seqlens=cu) if t is not None]]

    want = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(6):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((k, step(k)))
    torch.cuda.synchronize()
    for k, out in got:
        for t, u in zip(out, want[k]):
            assert torch.equal(t, u)


def test_binding_names_what_is_wrong():
    from hybrid_mamba_ssm_b200 import ssm
    p = scan_case(91, [30], 32, 16)
    (x, d, A, B, C), kw = operands(p, "bf16", "bf16")
    cu = cu_of(p)
    f = lambda *a, **k: ssm.selective_scan_fwd(*a, **{**kw, "cu_seqlens": cu, **k})  # noqa: E731
    for bad in [(x.t(), d, A, B, C), (x, d[:10], A, B, C), (x, d, A[:, :3], B, C), (x, d, A, B[:, :, :4], C),
                (x[:, ::2], d, A, B, C), (x, d.cpu(), A, B, C)]:
        with pytest.raises(ValueError):
            f(*bad)
    for bad, k in [((x.half(), d, A, B, C), {}), ((x, d, A.double(), B, C), {}), ((x, d, A, B.float(), C), {}),
                   ((x, d, A, B, C), dict(initial_state=torch.zeros(1, 32, 16, dtype=BF, device="cuda")))]:
        with pytest.raises(TypeError):
            f(*bad, **k)
    for k in [dict(cu_seqlens=cu.cpu()), dict(slot_idx=cu[:1]), dict(workspace="no"), dict(D=kw["D"][:5]),
              dict(y=torch.empty(30, 31, dtype=BF, device="cuda")), dict(final_state=torch.zeros(2, 32, 16, device="cuda"))]:
        with pytest.raises(ValueError):
            f(x, d, A, B, C, **k)
    with pytest.raises(ssm.SSMError):                       # every token at one address
        f(x[:1].expand(30, 32), d, A, B, C)
    with pytest.raises(ssm.SSMError):                       # an output over an input
        f(x, d, A, B, C, y=x)
    with pytest.raises(ssm.SSMError):                       # fp32 activations with bf16 dt
        f(x.float(), d, A, B.float(), C.float(), z=kw["z"].float())
    saved = f(x, d, A, B, C, save_states=True)[2]
    with pytest.raises(ValueError):
        ssm.selective_scan_bwd(x, x, d, A, B, C, saved[:-1].clone(), **kw, cu_seqlens=cu)
    with pytest.raises(ValueError):
        ssm.selective_state_update(torch.zeros(30, 32, 8, device="cuda"), x, d, A, B, C)
    with pytest.raises(ValueError):
        ssm.causal_conv1d_bwd(x[:5], x, torch.zeros(32, 4, device="cuda"), cu_seqlens=cu)
    with pytest.raises(ValueError):
        ssm.causal_conv1d_bwd(x, x, torch.zeros(32, 4, device="cuda"), cu_seqlens=cu, activation="relu")
    y, _ = f(x, d, A, B, C)                                 # and the context is as it was
    assert bool(y.isfinite().all())
