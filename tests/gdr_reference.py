"""Plain 64-bit reference of the gated delta rule, of drafted windows and of
draft verification, with the inputs of their tests (NumPy only).

Error bounds (2-norms over the keys of one state column).  A token's step is
S' = alpha S + beta kh (v - alpha kh^T S)^T with |kh| <= 1, beta <= 1 and
alpha <= 1, so it never enlarges an error that S already carries: the errors
of the steps add up.  One step makes, in fp32 with half a unit eps = 2^-24,
  - the reduction kh^T S: at most ~20 roundings deep (a chain of 16 FMAs in a
    lane, then a tree over lanes), norms and gate factors a few units each;
  - the write and the (deferred) decay: three roundings of S, one hardware
    reciprocal, exp, sigmoid and rsqrt of a few units each.
Everything is relative to m = max over the request's tokens of
|S column| + |v|.  STEP = 32 units per token covers both:
  |dS column| <= STEP n eps m,   |do| <= scale (STEP (n + 1) eps m)
for a state (output) after n tokens, as |qh| <= scale.  Rounding an output or a
pool to bf16 adds half a step, 2^-8 of the value.
"""
from __future__ import annotations

import numpy as np

EPS = 2.0 ** -24
STEP = 32.0
BF16 = 2.0 ** -8


def to_bf16(x):
    """fp32 -> the nearest bf16 value (ties to even), as fp32."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).reshape(np.shape(x))


class Tokens:
    """Packed q, k, v, gate and beta of T tokens (fp32 arrays of exact values)."""

    def __init__(self, rng, T, H, HV, dk, dv, channel, bf16, beta_shift=0.0):
        def normal(*shape):
            return rng.standard_normal(shape, dtype=np.float32)
        self.q, self.k, self.v = normal(T, H, dk), normal(T, H, dk), normal(T, HV, dv)
        if bf16:
            self.q, self.k, self.v = to_bf16(self.q), to_bf16(self.k), to_bf16(self.v)
        self.gate = normal(T, HV, dk) if channel else normal(T, HV)
        self.beta = normal(T, HV) + np.float32(beta_shift)


class Params:
    """What a layer keeps: gate parameters and the call's scalars."""

    def __init__(self, rng, HV, dk, channel, gate_mode="softplus", lower_bound=0.0, l2_eps=1e-6, scale=None):
        self.a_log = rng.uniform(-2.0, 2.0, size=HV).astype(np.float32)
        self.dt_bias = rng.standard_normal((HV, dk) if channel else HV, dtype=np.float32)
        self.gate_mode, self.lower_bound, self.l2_eps = gate_mode, lower_bound, l2_eps
        self.scale = dk ** -0.5 if scale is None else scale
        self.channel = channel


def walk(S, tok, par, hv, rows, G):
    """State S [dk, dv] (fp64) of value head hv through `rows`: the state
    after them, the outputs, and m of the bounds above."""
    S = S.astype(np.float64)
    out, m = [], np.linalg.norm(S, axis=0)
    for t in rows:
        q, k = tok.q[t, hv // G].astype(np.float64), tok.k[t, hv // G].astype(np.float64)
        q = par.scale * q / np.sqrt(q @ q + par.l2_eps)
        k = k / np.sqrt(k @ k + par.l2_eps)
        x = np.asarray(tok.gate[t, hv], dtype=np.float64) + par.dt_bias[hv]
        amp = np.exp(np.float64(par.a_log[hv]))
        if par.gate_mode == "softplus":
            g = -amp * np.logaddexp(0.0, x)
        else:
            g = par.lower_bound / (1.0 + np.exp(-amp * x))
        beta = 1.0 / (1.0 + np.exp(-np.float64(tok.beta[t, hv])))
        v = tok.v[t, hv].astype(np.float64)
        S = np.exp(g).reshape(-1, 1) * S
        S = S + np.outer(beta * k, v - k @ S)
        out.append(q @ S)
        m = np.maximum(m, np.linalg.norm(S, axis=0) + np.abs(v))
    return S, np.array(out).reshape(len(out), S.shape[1]), m


def check_state(got, ref, m, n, bf16, what):
    """One tile's state columns after n tokens."""
    err = np.linalg.norm(got.astype(np.float64) - ref, axis=0)
    bound = STEP * max(n, 1) * EPS * m
    if bf16:
        bound = bound + BF16 * (np.linalg.norm(ref, axis=0) + bound)
    assert (err <= bound).all(), f"{what}: state off by {np.max(err / bound):.3g} of its bound"


def check_out(got, ref, m, n, scale, bf16, what):
    """One tile's outputs [n, dv]; n counts every token walked before and in it."""
    err = np.abs(got.astype(np.float64) - ref)
    bound = scale * STEP * (n + 1) * EPS * m
    if bf16:
        bound = bound + BF16 * (np.abs(ref) + bound)
    bound = np.broadcast_to(bound, err.shape)
    assert (err <= bound).all(), f"{what}: output off by {np.max(err / bound):.3g} of its bound"


def verify(target, draft, tokens, u_accept, u_sample, cu):
    """n_commit and next_token of kda_verify, in fp64."""
    def mass(row):
        row = row.astype(np.float64)
        return np.where(np.isfinite(row) & (row > 0), row, 0.0)

    V = target.shape[1]
    n_commit, next_token = [], []
    for b in range(len(cu) - 1):
        t0, t1 = int(cu[b]), int(cu[b + 1])
        if t1 == t0:
            n_commit.append(0)
            next_token.append(-1)
            continue
        kept, fell = 0, False
        for t in range(t0, t1 - 1):
            x = int(tokens[t + 1])
            q = 1.0 if draft is None else (mass(draft[t])[x] if 0 <= x < V else 0.0)
            p = mass(target[t])[x] if 0 <= x < V else 0.0
            if not np.float64(u_accept[t]) * q < p:
                fell = True
                break
            kept += 1
        r = mass(target[t0 + kept])
        if fell and draft is not None:
            r = np.maximum(r - mass(draft[t0 + kept]), 0.0)
        elif fell and 0 <= tokens[t0 + kept + 1] < V:
            r[tokens[t0 + kept + 1]] = 0.0
        cum = np.cumsum(r)
        u = np.float64(u_sample[b])
        u = u if u > 0 else 0.0
        over = np.nonzero((cum > u * cum[-1]) & (r > 0))[0]
        some = np.nonzero(r > 0)[0]
        n_commit.append(kept + 1)
        next_token.append(int(over[0]) if len(over) else (int(some[-1]) if len(some) else -1))
    return np.array(n_commit), np.array(next_token)
