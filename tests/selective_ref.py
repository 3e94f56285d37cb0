"""fp64 reference of the per-channel selective scan, its gradient and the
conv1d gradient, written out token by token in numpy, and what the tests
share: seeded inputs and derived tolerances.

Tolerances.  An output is a sum of products; evaluated in fp32 it is off by at
most (the number of roundings on a term's way) * (the rounding) * (the sum of
the terms' magnitudes).  ``scan`` and ``scan_grad`` evaluated on magnitudes
(``magnitude`` below) give that sum.  On a term's way lie at most two decays
per token of its sequence (one forward, one backward), each an approximate
exponential (2^-22 of the value), a product in its argument and the rounding
of the step size (together below 2^-22 for arguments below 1, where a decay
matters), and one rounding each of the recurrence and of the sums over n,
channels and tokens, which the kernels add in trees and short runs.  A result
stored in bf16 adds half a bf16 step of its own value.
"""
import numpy as np

ULP = 2.0 ** -24


def silu(z):
    return z / (1 + np.exp(-z))


def silu_slope(z):
    s = 1 / (1 + np.exp(-z))
    return s * (1 + z * (1 - s))


def silu_slope_terms(z):
    """Magnitude sum of silu'(z) = s + s z (1 - s): for z < 0 the two terms have
    opposite signs and cancel at z = -1.28, where a rounding of either is as
    large as ever, so a tolerance goes by |s| + |s z (1 - s)| and not by their
    difference."""
    s = 1 / (1 + np.exp(-z))
    return s * (1 + np.abs(z) * (1 - s))


def step_size(dt, bias, softplus, limit):
    """(step, d step / d dt) of the dt transform."""
    v = dt + (0 if bias is None else bias)
    d = np.ones_like(v)
    if softplus:
        d = 1 / (1 + np.exp(-v))
        v = np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))
    if limit is not None:
        d = np.where((v < limit[0]) | (v > limit[1]), 0.0, d)
        v = np.clip(v, *limit)
    return v, d


def _wide(v, dim):
    return np.repeat(v, dim // v.shape[1], axis=1)          # [T, G, N] -> [T, dim, N]


def scan(p, magnitude=False):
    """y [T, dim] and final states [nseq, dim, N] of the inputs p (a dict: x,
    dt, A, B, C, D, z, h0, cu, bias, softplus, limit); with magnitude, of the
    inputs' magnitudes.  Also the step sizes and the states behind every token."""
    m = np.abs if magnitude else (lambda v: v)
    dim = p["x"].shape[1]
    v, _ = step_size(p["dt"], p["bias"], p["softplus"], p["limit"])
    x, B, C = m(p["x"]), _wide(m(p["B"]), dim), _wide(m(p["C"]), dim)
    y, hs = np.zeros_like(x), np.zeros((x.shape[0], *p["A"].shape))
    nseq = len(p["cu"]) - 1
    hT = np.zeros((nseq, *p["A"].shape))
    for s in range(nseq):
        h = np.zeros(p["A"].shape) if p["h0"] is None else m(p["h0"][s])
        for t in range(p["cu"][s], p["cu"][s + 1]):
            h = np.exp(v[t][:, None] * p["A"]) * h + (v[t] * x[t])[:, None] * B[t]
            hs[t] = h
            y[t] = (h * C[t]).sum(1) + (0 if p["D"] is None else m(p["D"]) * x[t])
        hT[s] = h
    out = y if p["z"] is None else y * m(silu(p["z"]))
    return out, hT, y, v, hs


def scan_grad(p, dy, dhT, magnitude=False):
    """Gradients (a dict) of sum(dy * y) + sum(dhT * final state)."""
    m = np.abs if magnitude else (lambda v: v)
    T, dim = p["x"].shape
    G, A = p["B"].shape[1], p["A"]
    _, _, y, v, hs = scan(p, magnitude)
    _, slope = step_size(p["dt"], p["bias"], p["softplus"], p["limit"])
    x, B, C = m(p["x"]), _wide(m(p["B"]), dim), _wide(m(p["C"]), dim)
    dy, D = m(dy), np.zeros(dim) if p["D"] is None else m(p["D"])
    g = {"dx": np.zeros((T, dim)), "dv": np.zeros((T, dim)), "dA": np.zeros(A.shape),
         "dB": np.zeros((T, G, A.shape[1])), "dC": np.zeros((T, G, A.shape[1]))}
    g["dz"] = None
    if p["z"] is not None:
        g["dz"] = dy * y * (silu_slope_terms if magnitude else silu_slope)(p["z"])
        dy = dy * m(silu(p["z"]))
    nseq = len(p["cu"]) - 1
    g["dh0"] = np.zeros((nseq, *A.shape))
    for s in range(nseq):
        dh = m(dhT[s]).copy()
        for t in range(p["cu"][s + 1] - 1, p["cu"][s] - 1, -1):
            before = hs[t - 1] if t > p["cu"][s] else \
                (np.zeros(A.shape) if p["h0"] is None else m(p["h0"][s]))
            dh = dh + dy[t][:, None] * C[t]
            g["dC"][t] = (hs[t] * dy[t][:, None]).reshape(G, dim // G, -1).sum(1)
            g["dB"][t] = (dh * (v[t] * x[t])[:, None]).reshape(G, dim // G, -1).sum(1)
            w = (dh * B[t]).sum(1)
            dh = np.exp(v[t][:, None] * A) * dh
            q = dh * before
            g["dA"] += q * v[t][:, None]
            g["dv"][t] = (q * m(A)).sum(1) + w * x[t]
            g["dx"][t] = w * v[t] + D * dy[t]
        g["dh0"][s] = dh
    g["ddt"] = g.pop("dv") * slope
    g["dbias"] = g["ddt"].sum(0)
    g["dD"] = (dy * x).sum(0)
    return g


def scan_rounding(p):
    """Roundings on the way of one term, in units of 2^-24 of the magnitude sum."""
    longest = max((p["cu"][i + 1] - p["cu"][i] for i in range(len(p["cu"]) - 1)), default=0)
    return 2 * longest * (4 + 4 + 2) + p["A"].shape[1] + 32 + 64


def conv_grad(p, dy, dfinal, magnitude=False):
    """Gradients of the causal conv1d (p: x, weight, bias, act, init, cu)."""
    m = np.abs if magnitude else (lambda v: v)
    w, K = m(p["weight"]), p["weight"].shape[1]
    dim, nseq = p["x"].shape[1], len(p["cu"]) - 1
    g = {"dx": np.zeros_like(p["x"]), "dw": np.zeros_like(w), "db": np.zeros(dim),
         "dinit": np.zeros((nseq, dim, K - 1))}
    for s in range(nseq):
        a, b = p["cu"][s], p["cu"][s + 1]
        front = np.zeros((K - 1, dim)) if p["init"] is None else p["init"][s].T
        line = np.concatenate([front, p["x"][a:b]])
        n = b - a
        d = m(dy[a:b])
        if p["act"]:
            pre = (0 if p["bias"] is None else p["bias"]) + sum(line[k:k + n] * p["weight"][:, k] for k in range(K))
            d = d * m(silu_slope(pre))
        back = np.zeros_like(line)
        for k in range(K):
            back[k:k + n] += d * w[:, k]
            g["dw"][:, k] += (m(line[k:k + n]) * d).sum(0)
        if dfinal is not None and K > 1:
            back[n:] += m(dfinal[s]).T
        g["db"] += d.sum(0)
        g["dx"][a:b] = back[K - 1:]
        g["dinit"][s] = back[:K - 1].T
    return g


def offsets(lens):
    return [0, *np.cumsum(lens).tolist()]


def make_scan(seed, lens, dim, N, G=1, gate=True, D=True, h0=True, bias=True, softplus=True, limit=None,
              round_to=None, dt_round=None):
    """Seeded inputs; round_to / dt_round (functions) give the stored values of x, B, C, z / dt."""
    rng = np.random.default_rng(seed)
    T = int(sum(lens))
    r = round_to or (lambda v: v.astype(np.float32).astype(np.float64))
    rd = dt_round or (lambda v: v.astype(np.float32).astype(np.float64))
    f = lambda v: v.astype(np.float32).astype(np.float64)  # noqa: E731
    dt = 0.5 * rng.standard_normal((T, dim))
    if not softplus:
        dt = np.exp(dt - 3.0)
    return {"x": r(rng.standard_normal((T, dim))), "dt": rd(dt),
            "A": f(-np.exp(rng.uniform(-1, np.log(max(N, 3)), (dim, N)))),
            "B": r(rng.standard_normal((T, G, N))), "C": r(rng.standard_normal((T, G, N))),
            "D": f(rng.standard_normal(dim)) if D else None, "z": r(rng.standard_normal((T, dim))) if gate else None,
            "h0": f(0.3 * rng.standard_normal((len(lens), dim, N))) if h0 else None, "cu": offsets(lens),
            "bias": f(rng.uniform(-6, -2, dim)) if bias else None, "softplus": softplus, "limit": limit}
