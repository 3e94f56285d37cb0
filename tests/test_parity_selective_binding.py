"""The binding of the per-channel calls on the GPU: what it refuses leaves the
caller's buffers as they were, and its two layers (the C++ one for plain calls,
the Python one for the rest) give the same results."""
import pytest
import torch

from tests.test_parity_selective import cu_of, operands, scan_case

pytestmark = pytest.mark.gpu


class NoTruth:
    def __bool__(self):
        raise KeyError("no truth value")


@pytest.mark.parametrize("flag,error", [(torch.tensor([True, False]), RuntimeError), (NoTruth(), KeyError)])
def test_a_flag_without_a_truth_value_is_refused_before_the_launch(flag, error):
    from hybrid_mamba_ssm_b200 import ssm
    p = scan_case(111, [30], 32, 16)
    args, kw = operands(p, "bf16", "bf16")
    kw.pop("dt_softplus")
    pool = torch.randn(3, 32, 16, device="cuda")
    before, cu = pool.clone(), cu_of(p)
    slot = torch.tensor([1], dtype=torch.int32, device="cuda")
    x, d, A, B, C = args
    with pytest.raises(error):
        ssm.selective_state_update(pool, x[:3], d[:3], A, B[:3], C[:3], D=kw["D"], dt_bias=kw["dt_bias"], dt_softplus=flag)
    with pytest.raises(error):
        ssm.selective_scan_fwd(*args, **kw, dt_softplus=flag, initial_state=pool, final_state=pool, slot_idx=slot, cu_seqlens=cu)
    with pytest.raises(error):
        ssm.selective_scan_fwd(*args, **kw, dt_softplus=True, initial_state=pool, final_state=pool, slot_idx=slot, cu_seqlens=cu,
                               save_states=flag)
    saved = ssm.selective_scan_fwd(*args, **kw, dt_softplus=True, cu_seqlens=cu, save_states=True)[2]
    with pytest.raises(error):
        ssm.selective_scan_bwd(x, *args, saved, **kw, dt_softplus=True, cu_seqlens=cu, want_dinitial=flag)
    torch.cuda.synchronize()
    assert torch.equal(pool, before)


def bits(t):
    return t.contiguous().view({2: torch.int16, 4: torch.int32}[t.element_size()])


@pytest.mark.parametrize("packed", [True, False])
def test_both_layers_give_the_same_bits(packed, monkeypatch):
    """Every call through the C++ layer, then through Python alone: results, states and pools are equal."""
    from hybrid_mamba_ssm_b200 import ssm
    assert ssm._marshal is not ssm._NoMarshal
    p = scan_case(121, [33, 33, 33], 48, 16, 2)
    args, kw = operands(p, "bf16", "f32")
    kw["dt_limit"] = (0.001, 0.1)
    seq = dict(cu_seqlens=cu_of(p))
    if not packed:
        shape = lambda t: t.view(3, 33, *t.shape[1:])  # noqa: E731
        args = tuple(t if t is args[2] else shape(t) for t in args)
        kw["z"], seq = shape(kw["z"]), {}
    x, d, A, B, C = args
    dy, h0 = torch.randn_like(x), torch.randn(3, 48, 16, device="cuda")
    w, wb, hist = torch.randn(48, 4, device="cuda"), torch.randn(48, device="cuda"), torch.randn(3, 48, 3, device="cuda").to(x.dtype)
    start = torch.randn(6, 48, 16, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    flat = [t.reshape(-1, *t.shape[-n:]) for t, n in ((x, 1), (d, 1), (B, 2), (C, 2))]

    def all_calls():
        out = list(ssm.selective_scan_fwd(*args, **kw, **seq, initial_state=h0, save_states=True))
        out += ssm.selective_scan_bwd(dy, *args, out[2], **kw, **seq, dfinal_state=h0, want_dinitial=True)
        pool = start.clone()
        out += [ssm.selective_scan_fwd(*args, **kw, **seq, initial_state=pool, final_state=pool, slot_idx=i32(4, 0, 2),
                                       has_initial_state=i32(1, 0, 1))[0], pool.clone()]
        xs, ds, Bs, Cs = (t[:3] for t in flat)
        out.append(ssm.selective_state_update(pool, xs, ds, A, Bs, Cs, D=kw["D"], z=xs, slot_idx=i32(5, -1, 0),
                                              dt_bias=kw["dt_bias"], dt_softplus=True))
        out += ssm.causal_conv1d_bwd(dy, x, w, wb, initial_state=hist, dfinal_state=hist, **seq)
        ssm.ssm_pool_copy([pool], i32(4, 2), i32(1, 3))
        ssm.ssm_pool_zero([pool], i32(4))
        table = i32(5, 3, -1)
        out += [pool.clone(), ssm.ssm_pool_compact([pool], table), table, pool]
        return out

    fast = all_calls()
    monkeypatch.setattr(ssm, "_marshal", ssm._NoMarshal)
    for a, b in zip(fast, all_calls(), strict=True):
        assert a.shape == b.shape and a.dtype == b.dtype and torch.equal(bits(a), bits(b))
