"""A NaN step size under the clamp of the fused dt transform: clamp(NaN) is NaN
in the oracle (oracle.dt_transform) and in every per-head kernel, and stays in
its sequence and head."""
import numpy as np
import pytest
import torch

import oracle
from hybrid_mamba_ssm_b200 import inputs as synth
from tests.gpu_helpers import dev_f32, dev_tensor

pytestmark = pytest.mark.gpu

LIMIT = (1e-3, 0.1)


def test_oracle_keeps_nan():
    assert np.isnan(oracle.dt_transform(np.array([np.nan, 1.0]), None, True, *LIMIT)).tolist() == [True, False]


@pytest.mark.parametrize("dtype,P,N,G,chunk", [("bf16", 64, 128, 2, 128), ("f32", 32, 64, 2, 64)])
def test_scan(dtype, P, N, G, chunk):
    from hybrid_mamba_ssm_b200 import ssm
    lens, H, at, h = [300, 77], 8, 200, 5
    inp = synth.make_scan_inputs(401, lens, H, P, N, G, dtype=dtype, init_state=True)
    raw, bias = synth.make_raw_dt(402, (sum(lens), H), H)

    def run(dt):
        pool = dev_f32(inp.h0)
        y = ssm.ssd_chunk_scan_slots(dev_tensor(inp.x), dev_f32(dt), dev_f32(inp.A), dev_tensor(inp.B), dev_tensor(inp.C),
                                     dev_f32(inp.D), pool, None, cu_seqlens=torch.from_numpy(inp.cu_seqlens).cuda(),
                                     chunk_size=chunk, y_dtype=torch.float32, dt_bias=dev_f32(bias), dt_softplus=True,
                                     dt_limit=LIMIT)
        return y, pool

    clean, cT = run(raw)
    bad = raw.copy()
    bad[at, h] = np.nan
    y, hT = run(bad)
    assert bool(y[at:300, h].isnan().all()) and bool(hT[0, h].isnan().all())
    assert torch.equal(y[300:], clean[300:]) and torch.equal(hT[1], cT[1])
    rest = [i for i in range(H) if i // 2 != h // 2]                   # heads of other pairs
    assert torch.equal(y[:, rest], clean[:, rest]) and torch.equal(hT[:, rest], cT[:, rest])


@pytest.mark.parametrize("state", [torch.float32, torch.float16])
def test_decode(state):
    from hybrid_mamba_ssm_b200 import ssm
    batch, H, P, N, G, b, h = 6, 16, 64, 128, 4, 3, 7
    A, D = synth.make_head_params(411, H)
    step = synth.make_decode_step(413, batch, H, P, N, G)
    raw, bias = synth.make_raw_dt(414, (batch, H), H)
    raw[b, h] = np.nan
    pool = dev_f32(synth.make_state(412, (batch, H, P, N))).to(state)
    y = ssm.ssm_state_update_slots(pool, None, dev_tensor(step.x), dev_f32(raw), dev_f32(A), dev_tensor(step.B),
                                   dev_tensor(step.C), dev_f32(D), y_dtype=torch.float32, dt_bias=dev_f32(bias),
                                   dt_softplus=True, dt_limit=LIMIT)
    want = torch.zeros(batch, H, dtype=torch.bool, device="cuda")
    want[b, h] = True
    assert torch.equal(y.isnan(), want[:, :, None].expand_as(y))
    assert torch.equal(pool.isnan(), want[:, :, None, None].expand_as(pool))


def test_multi():
    from hybrid_mamba_ssm_b200 import ssm
    batch, ntok, H, P, N, G, b, t, h = 3, 4, 8, 64, 128, 2, 1, 2, 5
    A, D = synth.make_head_params(421, H)
    steps = [synth.make_decode_step(423 + k, batch, H, P, N, G) for k in range(ntok)]
    raw, bias = synth.make_raw_dt(430, (batch, ntok, H), H)
    raw[b, t, h] = np.nan
    x, B, C = (torch.stack([dev_tensor(f(s)) for s in steps], dim=1).contiguous()
               for f in (lambda s: s.x, lambda s: s.B, lambda s: s.C))
    for inter in (False, True):
        state = dev_f32(synth.make_state(422, (batch, H, P, N)))
        y, _ = ssm.ssm_state_update_multi(state, x, dev_f32(raw), dev_f32(A), B, C, dev_f32(D), want_inter=inter,
                                          accept_len=torch.full((batch,), ntok, dtype=torch.int32, device="cuda"),
                                          y_dtype=torch.float32, dt_bias=dev_f32(bias), dt_softplus=True, dt_limit=LIMIT)
        want = torch.zeros(batch, ntok, H, dtype=torch.bool, device="cuda")
        want[b, t:, h] = True
        assert torch.equal(y.isnan(), want[..., None].expand_as(y))
        assert torch.equal(state.isnan(), want[:, -1, :, None, None].expand_as(state))
