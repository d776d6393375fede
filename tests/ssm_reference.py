"""Plain 64-bit reference of the selective state space scan and of the norms
around a block, with the inputs of their tests (NumPy only).

Error bounds of the scan.  Next to every value its magnitude is carried: what
it would be if nothing cancelled.  A convolved channel y = SiLU(z) has
mag(y) = |y| + 1.1 (|bias| + sum |w x|) (SiLU's slope is at most 1.1), the
state M' = a M + step mag(B) mag(x)^T, an output mag(C)^T M + |d| mag(x).  In
fp32, with eps = 2^-24 half a unit:
  - a convolution is five roundings deep, SiLU some five more units;
  - step and decay a = exp(-amp step) are off by some units of themselves and
    of amp step, and a (amp step) <= 1/e;
  - one token's update is three roundings of M, and a reduction over at most
    128 keys in a tree or a matrix instruction's chain of 32 at a time, or over
    a chunk's tokens, at most ~20 units.
Errors of earlier tokens decay with the state.  STEP = 32 units of the largest
M so far per token, as if none did:
    |dS| <= STEP n eps M,      |do| <= STEP (n + 1) eps mag(o).
Chunks: operands are sums of bf16 terms cut off by truncation.  Three terms
hold all 24 bits, and of the nine products of terms those of less than
2^-7 2^-15 relative are left out, three of them: 2^-20.4 of the magnitudes.  Two
terms hold 16 bits (2^-16 each) and leave out the product of the second ones
(2^-14): 2^-13.4.  An output passes two such products (C.B, then times x).
Rounding an output or a pool to bf16 adds half a step, 2^-8 of the value.
"""
from __future__ import annotations

import numpy as np

EPS = 2.0 ** -24
STEP = 32.0
BF16 = 2.0 ** -8
TERMS3 = 2.0 ** -20.4
TERMS2 = 2.0 ** -13.4


def to_bf16(x):
    """fp32 -> the nearest bf16 value (ties to even), as fp32."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).reshape(np.shape(x))


class Case:
    """A call's arrays (fp32 of exact values; bf16 ones already rounded)."""

    def __init__(self, seed, lens, H=1, HV=4, dk=64, dv=64, K=4, bf16=True, state_bf16=False, w_bf16=False,
                 layout="k_first", slots=None, bias=True, skip=True, extra_slots=2, decay=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.HV, self.dk, self.dv, self.K = list(lens), H, HV, dk, dv, K
        self.bf16, self.state_bf16, self.w_bf16, self.layout = bf16, state_bf16, w_bf16, layout
        B, T, C = len(lens), sum(lens), HV * dv + 2 * H * dk
        self.B, self.T, self.C = B, T, C
        N = B + extra_slots
        self.N = N

        def normal(*shape):
            return rng.standard_normal(shape, dtype=np.float32)
        act = to_bf16 if bf16 else (lambda x: x)
        wt = to_bf16 if w_bf16 else (lambda x: x)
        self.xbc = act(normal(T, C))
        self.dt = normal(T, HV)
        self.conv_w = wt((rng.random((K, C), dtype=np.float32) * 2 - 1) * np.float32(0.5))
        self.conv_b = wt((rng.random(C, dtype=np.float32) * 2 - 1) * np.float32(0.5)) if bias else None
        self.conv_win = act(normal(N, K - 1, C))
        self.a_log = np.log(1 + 15 * rng.random(HV)).astype(np.float32)
        step = np.exp(rng.random(HV) * np.log(100.0) + np.log(1e-3)) * decay
        self.dt_bias = (step + np.log(-np.expm1(-step))).astype(np.float32)
        self.d_skip = 1 + np.float32(0.1) * normal(HV) if skip else None
        pool = normal(N, HV, dk, dv) * np.float32(0.1)
        self.pool = to_bf16(pool) if state_bf16 else pool       # key-first here; laid out in tensors()
        self.slots = list(rng.permutation(N)[:B]) if slots is None else list(slots)
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)

    def tensors(self, device):
        import torch
        act = torch.bfloat16 if self.bf16 else torch.float32
        wt = torch.bfloat16 if self.w_bf16 else torch.float32

        def dev(x, dtype=torch.float32):
            return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(device).to(dtype).contiguous()
        pool = self.pool if self.layout == "k_first" else self.pool.transpose(0, 1, 3, 2)
        return dict(out=torch.full((1, self.T, self.HV, self.dv), 7.0, dtype=act, device=device),
                    xbc=dev(self.xbc[None], act), dt=dev(self.dt[None]), conv_w=dev(self.conv_w, wt),
                    conv_b=dev(self.conv_b, wt), conv_win=dev(self.conv_win), a_log=dev(self.a_log),
                    dt_bias=dev(self.dt_bias), d_skip=dev(self.d_skip), cu_seqlens=dev(self.cu, torch.int32),
                    state_pool=dev(pool, torch.bfloat16 if self.state_bf16 else torch.float32),
                    state_indices=dev(np.array(self.slots, dtype=np.int32), torch.int32))

    def walk(self, b):
        """Request b, token by token, over all heads: outputs, their magnitudes, the state, its magnitude
        (largest so far) and the window."""
        H, HV, dk, dv, K = self.H, self.HV, self.dk, self.dv, self.K
        slot = self.slots[b]
        S = self.pool[slot].astype(np.float64)
        M = np.abs(S)
        most = M.copy()
        win = self.conv_win[slot].astype(np.float64)
        w = self.conv_w.astype(np.float64)
        bias = 0.0 if self.conv_b is None else self.conv_b.astype(np.float64)
        d = np.zeros(HV) if self.d_skip is None else self.d_skip.astype(np.float64)
        amp = np.exp(self.a_log.astype(np.float64))
        outs, mags = [], []
        for t in range(self.cu[b], self.cu[b + 1]):
            seq = np.concatenate([win, self.xbc[t].astype(np.float64)[None]])
            z = bias + (seq * w).sum(0)
            y = z / (1 + np.exp(-z))
            mag = np.abs(y) + 1.1 * (np.abs(bias) + np.abs(seq * w).sum(0))
            win = seq[1:]

            def parts(v):
                x, bb, cc = np.split(v, [HV * dv, HV * dv + H * dk])
                rep = HV // H
                return (x.reshape(HV, dv), np.repeat(bb.reshape(H, dk), rep, 0), np.repeat(cc.reshape(H, dk), rep, 0))
            x, bk, ck = parts(y)
            mx, mb, mc = parts(mag)
            step = np.logaddexp(0.0, self.dt[t].astype(np.float64) + self.dt_bias)
            a = np.exp(-amp * step)[:, None, None]
            S = a * S + step[:, None, None] * bk[:, :, None] * x[:, None, :]
            M = a * M + step[:, None, None] * mb[:, :, None] * mx[:, None, :]
            most = np.maximum(most, M)
            outs.append(np.einsum("hk,hkv->hv", ck, S) + d[:, None] * x)
            mags.append(np.einsum("hk,hkv->hv", mc, most) + np.abs(d)[:, None] * mx)
        shape = (len(outs), HV, dv)
        return np.array(outs).reshape(shape), np.array(mags).reshape(shape), S, most, win

    def check(self, t, chunked):
        """Compare a call's tensors with the reference; every slot no request names is as it was."""
        import torch
        out = t["out"].float().cpu().numpy().astype(np.float64)[0]
        pool = t["state_pool"].float().cpu().numpy().astype(np.float64)
        pool = pool if self.layout == "k_first" else pool.transpose(0, 1, 3, 2)
        win = t["conv_win"].cpu().numpy()
        terms_out = (TERMS2 if self.bf16 else TERMS3) if chunked else 0.0
        terms_state = (TERMS2 if self.bf16 and self.state_bf16 else TERMS3) if chunked else 0.0
        named = set()
        for b, slot in enumerate(self.slots):
            rows = slice(self.cu[b], self.cu[b + 1])
            if slot < 0 or slot >= self.N:
                assert not out[rows].any(), f"request {b} is skipped: its rows are zero"
                continue
            n = self.lens[b]
            if n == 0:
                continue
            named.add(slot)
            o, mag, S, M, w = self.walk(b)
            k = np.arange(1, n + 1)[:, None, None]
            tol = (STEP * (k + 1) * EPS + 2 * terms_out) * mag + (BF16 * np.abs(o) if self.bf16 else 0)
            off = np.abs(out[rows] - o) - tol
            assert off.max() <= 0, f"out of request {b}: {off.max():.3g} over at {np.unravel_index(off.argmax(), off.shape)}"
            tol = (STEP * n * EPS + terms_state) * M + (BF16 * np.abs(S) if self.state_bf16 else 0)
            off = np.abs(pool[slot] - S) - tol
            assert off.max() <= 0, f"state of request {b}: {off.max():.3g} over at {np.unravel_index(off.argmax(), off.shape)}"
            assert np.array_equal(win[slot], w.astype(np.float32)), f"window of request {b}"
        for slot in set(range(self.N)) - named:
            assert np.array_equal(pool[slot], self.pool[slot].astype(np.float64)), f"state slot {slot} is no request's"
            assert np.array_equal(win[slot], self.conv_win[slot]), f"window slot {slot} is no request's"
        assert torch.isfinite(t["out"]).all() or not np.isfinite(self.xbc).all()


def sigmoid(z):
    return 1.0 / (1.0 + np.exp(-z))


def unit(x, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
