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
