"""Cases of the per-channel selective scan, its gradient, its single-token
update, the gradient of the short convolution in front of it, and the
bookkeeping of the state pools that serve them.

The operators, over a packed stream of T tokens (sequence s = tokens cu[s] ..
cu[s+1]), channel d of group g = d // (dim // groups), state index n:

    v[t,d]   = softplus(dt[t,d] + dt_bias[d])
    h[t,d,n] = exp(v[t,d] A[d,n]) h[t-1,d,n] + v[t,d] x[t,d] B[t,g,n]
    y[t,d]   = (sum_n h[t,d,n] C[t,g,n] + D[d] x[t,d]) * silu(z[t,d])

    c[t,d]   = silu(bias[d] + sum_k weight[d,k] in[t-(K-1)+k, d])

``own`` selects what ``run`` computes with: elementary torch operations, or
the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    scan = dict(op="scan", groups=1, dtype="bf16", dt="bf16", gate=True, ragged=False, pool=0)
    grad = dict(op="scan_grad", groups=1, dtype="bf16", dt="bf16", gate=True, ragged=False)
    step = dict(op="step", groups=1, dtype="bf16", dt="bf16", gate=True)
    conv = dict(op="conv_grad", dtype="bf16", width=4, ragged=False, history=False)
    return [
        # a few short prompts that join a running batch: their states are pool rows
        dict(scan, name="scan-prompts-short", nseq=3, tokens=96, dim=2048, d_state=16, ragged=True,
             pool=8),
        # a prefill batch of equal lengths
        dict(scan, name="scan-prompts-4x2048", nseq=4, tokens=8192, dim=8192, d_state=16),
        # one long prompt alone: few channels, many tokens
        dict(scan, name="scan-prompt-1x32768", nseq=1, tokens=32768, dim=2048, d_state=16),
        # a training step of a small odd-sized layer in fp32, two groups, no gate
        dict(grad, name="grad-ragged-f32", nseq=5, tokens=701, dim=1002, d_state=13, groups=2,
             dtype="f32", dt="f32", gate=False, ragged=True),
        # a training micro-batch
        dict(grad, name="grad-4x2048", nseq=4, tokens=8192, dim=8192, d_state=16),
        # packed training documents, a wide state in groups
        dict(grad, name="grad-packed-state64", nseq=6, tokens=4096, dim=2048, d_state=64, groups=4,
             dt="f32", ragged=True),
        # one user: latency
        dict(step, name="step-batch1", batch=1, slots=4, dim=2048, d_state=16),
        # a serving batch: the pool is read and written once
        dict(step, name="step-batch256", batch=256, slots=320, dim=8192, d_state=16),
        # short odd documents with carried windows, fp32
        dict(conv, name="conv-grad-ragged-f32", nseq=7, tokens=701, dim=1002, width=3, dtype="f32",
             ragged=True, history=True),
        # the convolution of a training micro-batch
        dict(conv, name="conv-grad-4x4096", nseq=4, tokens=16384, dim=10240),
        # requests fork (several continuations of one prompt): rows copied in every layer
        dict(name="pool-fork", op="pool", what="fork", layers=24, slots=48, rows=12, dim=4096,
             d_state=16, width=4),
        # requests finish: their rows are freed, the live ones move to the front
        dict(name="pool-retire", op="pool", what="retire", layers=24, slots=96, rows=40, dim=2048,
             d_state=16, width=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_grad", "scan_grad", "step", "conv_grad", "pool"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    dt = rng.choice([dtype, "f32"])
    gate = rng.random() < 0.7
    groups = rng.choice([1, 1, 2, 4])
    n = rng.choice([4, 8, 13, 16, 16, 16, 16, 24, 32, 64, 128])
    if op in ("scan", "scan_grad"):
        dim = groups * max(1, _log(rng, 64, 8192) // groups)
        tokens = min(_log(rng, 1, 32768), max(1, 2 ** 29 // (dim * n)))
        nseq = rng.randint(1, max(1, min(16, tokens)))
        ragged = rng.random() < 0.6
        if not ragged:
            tokens = nseq * max(1, tokens // nseq)
        c = dict(op=op, nseq=nseq, tokens=tokens, dim=dim, d_state=n, groups=groups, dtype=dtype, dt=dt,
                 gate=gate, ragged=ragged)
        if op == "scan":
            c["pool"] = nseq + rng.randint(0, 9) if rng.random() < 0.4 else 0
        return c
    if op == "step":
        batch = _log(rng, 1, 256)
        dim = groups * max(1, _log(rng, 64, 8192) // groups)
        batch = max(1, min(batch, 2 ** 25 // (dim * n)))
        return dict(op="step", batch=batch, slots=batch + rng.randint(0, 64), dim=dim, d_state=n, groups=groups,
                    dtype=dtype, dt=dt, gate=gate)
    if op == "conv_grad":
        dim = _log(rng, 64, 10240)
        tokens = min(_log(rng, 1, 16384), 2 ** 27 // dim)
        nseq = rng.randint(1, max(1, min(16, tokens)))
        ragged = rng.random() < 0.6
        if not ragged:
            tokens = nseq * max(1, tokens // nseq)
        return dict(op="conv_grad", nseq=nseq, tokens=tokens, dim=dim, width=rng.choice([2, 3, 4, 4, 4, 8]),
                    dtype=dtype, ragged=ragged, history=rng.random() < 0.5)
    dim = _log(rng, 64, 4096)
    rows = _log(rng, 1, 32)
    layers = max(1, min(rng.randint(1, 24), 2 ** 27 // (dim * 16 * rows)))
    return dict(op="pool", what=rng.choice(["fork", "retire"]), layers=layers, slots=3 * rows + rng.randint(0, 16),
                rows=rows, dim=dim, d_state=16, width=4)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _offsets(case, g):
    """Sequence offsets: equal lengths, or random cuts (empty sequences happen)."""
    n, total = case["nseq"], case["tokens"]
    if not case["ragged"]:
        return torch.arange(n + 1, dtype=torch.int64) * (total // n)
    cuts = torch.sort(torch.randint(0, total + 1, (n - 1,), generator=g)).values
    return torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([total])])


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    s = {"case": case}
    op = case["op"]
    if op == "pool":
        layers, slots, rows, dim = case["layers"], case["slots"], case["rows"], case["dim"]
        s["ssm"] = normal(layers, slots, dim, case["d_state"])
        s["conv"] = normal(layers, slots, dim, case["width"] - 1, dtype=torch.bfloat16)
        s["pools"] = list(s["ssm"].unbind(0)) + list(s["conv"].unbind(0))
        order = torch.randperm(slots, generator=host).to(torch.int32)
        if case["what"] == "fork":        # few parents, each with several children
            s["src"] = order[torch.randint(0, max(1, rows // 4), (rows,), generator=host)].cuda()
            s["dst"] = order[slots - rows:].cuda()
        else:                             # `rows` requests live, as many just finished
            table = order[:rows].clone()
            if rows > 2:
                table[rows // 2] = -1     # a padding row of the batch
            s["table"] = table.cuda()
            s["free"] = order[rows:2 * rows].cuda()
        return s

    dtype, dim = DTYPES[case["dtype"]], case["dim"]
    if op == "conv_grad":
        T, K = case["tokens"], case["width"]
        s["cu"] = _offsets(case, host).to(torch.int32).cuda()
        s["x"], s["dy"] = normal(T, dim, dtype=dtype), normal(T, dim, dtype=dtype)
        s["weight"], s["bias"] = normal(dim, K, scale=K ** -0.5), normal(dim, scale=0.3)
        s["history"] = normal(case["nseq"], dim, K - 1, dtype=dtype) if case["history"] else None
        return s

    N, G = case["d_state"], case["groups"]
    T = case["batch"] if op == "step" else case["tokens"]
    # x, the gate and B, C as the projections of a mixer leave them: z is the
    # second half of the input projection's rows, B and C lie behind dt's
    # low-rank part
    rank = max(1, dim // 16)
    s["x"] = normal(T, dim, dtype=dtype)
    proj = normal(T, 2 * dim, dtype=dtype)
    s["z"] = proj[:, dim:] if case["gate"] else None
    low = normal(T, rank + 2 * G * N, dtype=dtype)
    s["B"] = low[:, rank:rank + G * N].unflatten(1, (G, N))
    s["C"] = low[:, rank + G * N:].unflatten(1, (G, N))
    s["dt"] = normal(T, dim, scale=0.5, dtype=DTYPES[case["dt"]])
    # step sizes between 1e-3 and 1e-1 at dt = 0, decay rates about 1 .. N
    step = torch.exp(torch.rand(dim, generator=gen, device="cuda") * math.log(100.0) + math.log(1e-3))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(normal(dim, N, scale=0.1))
    s["D"] = 1 + normal(dim, scale=0.1)
    if op == "step":
        s["state"] = normal(case["slots"], dim, N, scale=0.1)
        slots = torch.randperm(case["slots"], generator=host)[:T].to(torch.int32)
        if T > 4:
            slots[T // 3] = -1            # a padding row of the batch
        s["slots"], s["y"] = slots.cuda(), torch.zeros(T, dim, dtype=dtype, device="cuda")
        return s
    s["cu"] = _offsets(case, host).to(torch.int32).cuda()
    if op == "scan_grad":
        s["h0"] = normal(case["nseq"], dim, N, scale=0.1)
        s["dy"] = normal(T, dim, dtype=dtype)
        s["dhT"] = normal(case["nseq"], dim, N, scale=0.1)
    elif case["pool"]:
        s["state"] = normal(case["pool"], dim, N, scale=0.1)
        s["slots"] = torch.randperm(case["pool"], generator=host)[:case["nseq"]].to(torch.int32).cuda()
        # half of the rows were claimed just now: they start from zero
        s["has"] = (torch.rand(case["nseq"], generator=host) < 0.5).to(torch.int32).cuda()
    return s


# ---------------------------------------------------------------------------
# the plain form: fp32, rounded once at the end
# ---------------------------------------------------------------------------
def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _recur(a, b):
    """h[t] = a[t] h[t-1] + b[t] along axis 0, by doubling the span of each entry."""
    span = 1
    while span < b.shape[0]:
        b = torch.cat([b[:span], b[span:] + a[span:] * b[:-span]])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return b


def _per_channel(v, dim):
    """[T, G, N] -> [T, dim, N]: each channel reads its group's row."""
    return v.float().repeat_interleave(dim // v.shape[1], dim=1)


def _states(s, h0):
    """Decays a, steps v, states h of all tokens; first and last token of the
    sequences that have any, and which those are."""
    cu = s["cu"].long()
    some = (cu[1:] > cu[:-1]).nonzero().flatten()
    first, last = cu[:-1][some], cu[1:][some] - 1
    v = _softplus(s["dt"].float() + s["dt_bias"])
    a = torch.exp(v.unsqueeze(2) * s["A"])
    b = (v * s["x"].float()).unsqueeze(2) * _per_channel(s["B"], v.shape[1])
    if h0 is not None:
        b[first] += a[first] * h0[some]
    cut = a.clone()
    cut[first] = 0
    return a, v, _recur(cut, b), first, last, some


def _scan(s):
    c = s["case"]
    dim, N = c["dim"], c["d_state"]
    h0 = torch.zeros(c["nseq"], dim, N, device="cuda")
    if c["pool"]:
        slots = s["slots"].long()
        h0 = s["state"][slots] * s["has"].float()[:, None, None]
    _, _, h, _, last, some = _states(s, h0)
    y = (h * _per_channel(s["C"], dim)).sum(2) + s["D"] * s["x"].float()
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    hT = h0
    hT[some] = h[last]
    if c["pool"]:
        s["state"][slots] = hT
        hT = s["state"]
    return y.to(s["x"].dtype), hT


def _scan_grad(s):
    c = s["case"]
    dim, N, G = c["dim"], c["d_state"], c["groups"]
    a, v, h, first, last, some = _states(s, s["h0"])
    x, dy = s["x"].float(), s["dy"].float()
    B, C = _per_channel(s["B"], dim), _per_channel(s["C"], dim)
    y, dz = (h * C).sum(2) + s["D"] * x, None
    hT = s["h0"].clone()
    hT[some] = h[last]
    if s["z"] is not None:
        z = s["z"].float()
        sig = _sigmoid(z)
        dz = (dy * y * sig * (1 + z * (1 - sig))).to(s["z"].dtype)
        dy, y = dy * z * sig, y * z * sig
    # dh[t] = C[t] dy[t] + a[t+1] dh[t+1], cut where a sequence ends
    b = C * dy.unsqueeze(2)
    b[last] += s["dhT"][some]
    cut = torch.cat([a[1:], torch.zeros_like(a[:1])])
    cut[last] = 0
    dh = _recur(cut.flip(0), b.flip(0)).flip(0)
    del b, cut, C
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = s["h0"][some]
    q = dh * a * before
    del before
    dh0 = s["dhT"].clone()
    dh0[some] = a[first] * dh[first]
    through = (dh * B).sum(2)             # d loss / d (v x)
    dv = (q * s["A"]).sum(2) + through * x
    dA = (q * v.unsqueeze(2)).sum(0)
    del q
    ddt = dv * _sigmoid(s["dt"].float() + s["dt_bias"])
    dx = through * v + dy * s["D"]
    T = x.shape[0]
    dB = (dh * (v * x).unsqueeze(2)).view(T, G, dim // G, N).sum(2)
    dC = (h * dy.unsqueeze(2)).view(T, G, dim // G, N).sum(2)
    t = s["x"].dtype
    return (y.to(t), hT, dx.to(t), ddt.to(s["dt"].dtype), dA, dB.to(t), dC.to(t), (dy * x).sum(0), dz, ddt.sum(0), dh0)


def _step(s):
    slots = s["slots"].long()
    some = (slots >= 0).nonzero().flatten()
    rows = slots[some]
    dim = s["x"].shape[1]
    x = s["x"].float()[some]
    v = _softplus(s["dt"].float()[some] + s["dt_bias"])
    h = torch.exp(v.unsqueeze(2) * s["A"]) * s["state"][rows] \
        + (v * x).unsqueeze(2) * _per_channel(s["B"][some], dim)
    y = (h * _per_channel(s["C"][some], dim)).sum(2) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()[some]
        y = y * z * _sigmoid(z)
    s["state"][rows] = h
    s["y"][some] = y.to(s["y"].dtype)
    return s["y"], s["state"]


def _conv_grad(s):
    c = s["case"]
    K, dim = c["width"], c["dim"]
    cu = s["cu"].long()
    x, w = s["x"].float(), s["weight"]
    T = x.shape[0]
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(cu[1:], t, right=True)
    # taps[k][t] = in[t - (K-1) + k]: a token of the sequence, a history entry, or zero
    j = t[:, None] - (K - 1) + torch.arange(K, device="cuda")
    inside = j >= cu[:-1][seq][:, None]
    taps = x[j.clamp(min=0)] * inside.unsqueeze(2)
    back = (j - cu[:-1][seq][:, None] + K - 1).clamp(0, max(K - 2, 0))   # history entry of tap k
    outside = (~inside).nonzero()
    r, k = outside[:, 0], outside[:, 1]
    if s["history"] is not None and K > 1:
        taps[r, k] = s["history"].float()[seq[r], :, back[r, k]]
    pre = (taps * w.t()).sum(1) + s["bias"]
    sig = _sigmoid(pre)
    dpre = s["dy"].float() * sig * (1 + pre * (1 - sig))
    dw = (taps * dpre.unsqueeze(1)).sum(0).t().contiguous()
    # token t was read through tap k by the output at t + K-1 - k of its sequence
    u = t[:, None] + (K - 1) - torch.arange(K, device="cuda")
    read = (u < cu[1:][seq][:, None]).unsqueeze(2)
    dx = (dpre[u.clamp(max=T - 1)] * read * w.t()).sum(1)
    dhist = None
    if s["history"] is not None and K > 1:
        flat = torch.zeros(c["nseq"] * (K - 1), dim, device="cuda").index_add_(
            0, seq[r] * (K - 1) + back[r, k], dpre[r] * w.t()[k])
        dhist = flat.view(c["nseq"], K - 1, dim).transpose(1, 2).contiguous().to(s["x"].dtype)
    return dx.to(s["x"].dtype), dw, dpre.sum(0), dhist


def _pool(s):
    c = s["case"]
    if c["what"] == "fork":
        src, dst = s["src"].long(), s["dst"].long()
        s["ssm"][:, dst] = s["ssm"][:, src]
        s["conv"][:, dst] = s["conv"][:, src]
        return s["ssm"], s["conv"]
    free, table = s["free"].long(), s["table"].long()
    s["ssm"][:, free] = 0
    s["conv"][:, free] = 0
    pos = torch.arange(c["slots"], device="cuda")
    live = (table[:, None] == pos).any(0)
    count = live.sum()
    src, dst = (live & (pos >= count)).nonzero().flatten(), (~live & (pos < count)).nonzero().flatten()
    s["ssm"][:, dst] = s["ssm"][:, src]
    s["conv"][:, dst] = s["conv"][:, src]
    to = pos.clone()
    to[src] = dst
    moved = torch.where(table >= 0, to[table.clamp(min=0)], table)
    return s["ssm"], s["conv"], moved.to(torch.int32), count.to(torch.int32)


# ---------------------------------------------------------------------------
# the library's entry points
# ---------------------------------------------------------------------------
def _own(s):
    from hybrid_mamba_ssm_b200 import ssm
    op = s["case"]["op"]
    if op == "scan":
        kw = dict(D=s["D"], z=s["z"], cu_seqlens=s["cu"], dt_bias=s["dt_bias"], dt_softplus=True)
        if s["case"]["pool"]:
            kw.update(initial_state=s["state"], final_state=s["state"], slot_idx=s["slots"],
                      has_initial_state=s["has"])
        return ssm.selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], **kw)
    if op == "scan_grad":
        kw = dict(D=s["D"], z=s["z"], cu_seqlens=s["cu"], dt_bias=s["dt_bias"], dt_softplus=True)
        y, hT, saved = ssm.selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"],
                                              initial_state=s["h0"], save_states=True, **kw)
        return (y, hT, *ssm.selective_scan_bwd(s["dy"], s["x"], s["dt"], s["A"], s["B"], s["C"], saved,
                                               dfinal_state=s["dhT"], want_dinitial=True, **kw))
    if op == "step":
        return ssm.selective_state_update(s["state"], s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"],
                                          z=s["z"], slot_idx=s["slots"], dt_bias=s["dt_bias"],
                                          dt_softplus=True, y=s["y"]), s["state"]
    if op == "conv_grad":
        return ssm.causal_conv1d_bwd(s["dy"], s["x"], s["weight"], s["bias"], initial_state=s["history"],
                                     cu_seqlens=s["cu"])
    if s["case"]["what"] == "fork":
        ssm.ssm_pool_copy(s["pools"], s["src"], s["dst"])
        return s["ssm"], s["conv"]
    ssm.ssm_pool_zero(s["pools"], s["free"])
    table = s["table"].clone()
    count = ssm.ssm_pool_compact(s["pools"], table)
    return s["ssm"], s["conv"], table, count


PLAIN = {"scan": _scan, "scan_grad": _scan_grad, "step": _step, "conv_grad": _conv_grad, "pool": _pool}


def run(state):
    with torch.no_grad():
        return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "pool":
        row = case["layers"] * case["dim"] * (4 * case["d_state"] + 2 * (case["width"] - 1))
        if case["what"] == "fork":        # each parent read once, each child written
            return {"bytes": float((max(1, case["rows"] // 4) + case["rows"]) * row), "flops": 0.0}
        # freed rows are written; about rows (1 - rows / slots) live ones move
        moved = case["rows"] * (1 - case["rows"] / case["slots"])
        return {"bytes": float((case["rows"] + 2 * moved) * row), "flops": 0.0}
    es = size[case["dtype"]]
    dim = case["dim"]
    if op == "conv_grad":
        T, K = case["tokens"], case["width"]
        hist = 2 * case["nseq"] * dim * (K - 1) * es if case["history"] else 0
        return {"bytes": float(3 * T * dim * es + hist + 8 * dim * (K + 1)),
                "flops": float(T * dim * (6 * K + 10))}
    N, G, ds = case["d_state"], case["groups"], size[case["dt"]]
    T = case["batch"] if op == "step" else case["tokens"]
    gate = case["gate"]
    state = 4 * dim * N
    weights = state + 8 * dim
    rows = T * dim * (es * (2 + gate) + ds) + 2 * T * G * N * es      # x, z, dt, y; B, C
    if op == "step":
        return {"bytes": float(rows + 2 * T * state + weights), "flops": float(7 * T * dim * N)}
    if op == "scan":
        return {"bytes": float(rows + case["nseq"] * state * (2 if case["pool"] else 1) + weights),
                "flops": float(7 * T * dim * N)}
    # the forward pass and the gradients, each input read once for both
    grads = T * dim * (es * (1 + gate) + ds) + 2 * T * G * N * es     # dx, dz, ddt; dB, dC
    return {"bytes": float(rows + grads + T * dim * es + 4 * case["nseq"] * state + 2 * weights),
            "flops": float(25 * T * dim * N)}


# ---------------------------------------------------------------------------
# the definition in 64 bits, one token after another
# ---------------------------------------------------------------------------
def _padded(v, cu):
    """[T, ...] -> [L, nseq, ...] in fp64: token t of every sequence in row t, zeros behind its end."""
    lens = [cu[i + 1] - cu[i] for i in range(len(cu) - 1)]
    out = torch.zeros(max(lens), len(lens), *v.shape[1:], dtype=torch.float64, device=v.device)
    for i, n in enumerate(lens):
        out[:n, i] = v[cu[i]:cu[i + 1]].double()
    return out


def _packed(v, cu):
    return torch.cat([v[:cu[i + 1] - cu[i], i] for i in range(len(cu) - 1)])


def _wide(v, dim):
    return v[..., :, None, :].expand(*v.shape[:-1], dim // v.shape[-2], v.shape[-1]).flatten(-3, -2)


def _exact_scan(s, h0, history=False):
    """Step sizes (zero behind a sequence's end, so that its state stays), y before the gate, states."""
    cu = s["cu"].tolist()
    dim = s["x"].shape[1]
    v = _padded(torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=700.0), cu)
    x, B, C, A = _padded(s["x"], cu), _padded(s["B"], cu), _padded(s["C"], cu), s["A"].double()
    h, y, hs = h0.double(), torch.zeros_like(x), []
    for t in range(x.shape[0]):
        hs += [h] if history else []
        h = torch.exp(v[t].unsqueeze(-1) * A) * h + (v[t] * x[t]).unsqueeze(-1) * _wide(B[t], dim)
        y[t] = torch.einsum("sdn,sdn->sd", h, _wide(C[t], dim)) + s["D"].double() * x[t]
    hs += [h] if history else []
    return cu, v, x, B, C, A, y, h, hs


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    dim = case["dim"]
    if op == "pool":
        pools = [s["ssm"], s["conv"]]
        if case["what"] == "fork":
            old = [p.clone() for p in pools]
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                for p, o in zip(pools, old):
                    p[:, b] = o[:, a]
            return [p.double() for p in pools]
        table = s["table"].tolist()
        for i in s["free"].tolist():
            for p in pools:
                p[:, i] = 0
        live = sorted({i for i in table if i >= 0})
        holes = [i for i in range(len(live)) if i not in live]
        to = dict(zip([i for i in live if i >= len(live)], holes))
        for a, b in to.items():
            for p in pools:
                p[:, b] = p[:, a]
        return [p.double() for p in pools] + [torch.tensor([to.get(i, i) for i in table], dtype=torch.int32),
                                              torch.tensor(len(live), dtype=torch.int32)]
    if op == "conv_grad":
        cu, K = s["cu"].tolist(), case["width"]
        hist = s["history"]
        w = s["weight"].double()
        dx, dw = torch.zeros_like(s["x"], dtype=torch.float64), torch.zeros_like(w)
        db, dh = torch.zeros(dim, dtype=torch.float64, device="cuda"), []
        for i in range(case["nseq"]):
            n = cu[i + 1] - cu[i]
            front = torch.zeros(K - 1, dim, dtype=torch.float64, device="cuda") if hist is None \
                else hist[i].double().t()
            line = torch.cat([front, s["x"][cu[i]:cu[i + 1]].double()])
            pre = s["bias"].double() + sum(line[k:k + n] * w[:, k] for k in range(K))
            sig = torch.sigmoid(pre)
            d = s["dy"][cu[i]:cu[i + 1]].double() * (sig + pre * sig * (1 - sig))
            back = torch.zeros_like(line)
            for k in range(K):
                back[k:k + n] += d * w[:, k]
                dw[:, k] += (line[k:k + n] * d).sum(0)
            db += d.sum(0)
            dx[cu[i]:cu[i + 1]] = back[K - 1:]
            dh.append(back[:K - 1].t())
        return dx, dw, db, None if hist is None else torch.stack(dh)
    if op == "step":
        h, y = s["state"].double(), s["y"].double()
        v = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=700.0)
        A = s["A"].double()
        B, C = _wide(s["B"].double(), dim), _wide(s["C"].double(), dim)
        for b, row in enumerate(s["slots"].tolist()):
            if row < 0:
                continue
            xb = s["x"][b].double()
            h[row] = torch.exp(v[b][:, None] * A) * h[row] + (v[b] * xb)[:, None] * B[b]
            y[b] = (h[row] * C[b]).sum(1) + s["D"].double() * xb
            if s["z"] is not None:
                y[b] *= torch.nn.functional.silu(s["z"][b].double())
        return y, h
    if op == "scan":
        h0 = torch.zeros(case["nseq"], dim, case["d_state"], dtype=torch.float64, device="cuda")
        if case["pool"]:
            slots = s["slots"].long()
            h0 = s["state"][slots].double()
            h0[s["has"] == 0] = 0
        cu, _, _, _, _, _, y, h, _ = _exact_scan(s, h0)
        y = _packed(y, cu)
        if s["z"] is not None:
            y = y * torch.nn.functional.silu(s["z"].double())
        if case["pool"]:
            pool = s["state"].double()
            pool[slots] = h
            h = pool
        return y, h
    cu, v, x, B, C, A, y, hT, hs = _exact_scan(s, s["h0"], history=True)
    dy, dz, out = _padded(s["dy"], cu), None, _packed(y, cu)
    if s["z"] is not None:
        z = _padded(s["z"], cu)
        sig = torch.sigmoid(z)
        dz = _packed(dy * y * (sig + z * sig * (1 - sig)), cu)
        dy = dy * z * sig
        out = _packed(y * z * sig, cu)
    g = s["dhT"].double()                 # gradient of the state behind token t
    dx, dv, dB, dC = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(B), torch.zeros_like(C)
    dA = torch.zeros_like(A)
    G = case["groups"]
    for t in range(x.shape[0] - 1, -1, -1):
        g = g + dy[t].unsqueeze(-1) * _wide(C[t], dim)
        dC[t] = torch.einsum("sgdn,sgd->sgn", hs[t + 1].unflatten(1, (G, -1)), dy[t].unflatten(1, (G, -1)))
        dB[t] = torch.einsum("sgdn,sgd->sgn", g.unflatten(1, (G, -1)), (v[t] * x[t]).unflatten(1, (G, -1)))
        into = torch.einsum("sdn,sdn->sd", g, _wide(B[t], dim))
        g = torch.exp(v[t].unsqueeze(-1) * A) * g
        q = g * hs[t]
        dA += torch.einsum("sdn,sd->dn", q, v[t])
        dv[t] = torch.einsum("sdn,dn->sd", q, A) + into * x[t]
        dx[t] = into * v[t] + dy[t] * s["D"].double()
    dD = torch.einsum("lsd,lsd->d", dy, x)
    ddt = _packed(dv, cu) * torch.sigmoid(s["dt"].double() + s["dt_bias"].double())
    return out, hT, _packed(dx, cu), ddt, dA, _packed(dB, cu), _packed(dC, cu), dD, dz, ddt.sum(0), g
