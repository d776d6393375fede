"""GPU parity of the gated delta rule where magnitudes change within a request:
one token far larger than its neighbours, a large state that a gate closes, v
that is zero for a while.  Bounds are causal here: a token's error is relative
to what its column holds by then, not to what comes later or has decayed.

A step S' = alpha S + beta kh u passes alpha of the error that S carries and,
as in tests/gdr_reference.py, adds STEP units of alpha |S| + |v|.  The decay's
exponent g = log alpha adds up to 16 units of |g| relative to alpha |S|: exp(a_log)
5 (a hardware exp of one ulp, two units, and its rounded argument), softplus up to 8
(the sum x, exp, log and reciprocal of an ulp each, two products), their product 1,
and exp's argument g log2(e) 2:
  e_i = alpha_i e_(i-1) + eps (STEP (alpha_i |S| + |v_i|) + 16 |g_i| alpha_i |S|)
  |do_i| <= scale (e_i + STEP eps (alpha_i |S| + |v_i|)).
Below fp32's normal range (2^-126) intermediates may flush to zero.  Deferred
decays hold a state 2^64 larger at most and multiply by as little again, and a
column has 128 terms: at most 2^-126 * 2^7 a step, FLOOR = 2^-117 with the
output's own terms.  kda_gdr_prefill takes |v|
over groups of tokens and, where a group has no v, what the column held in its 32
tokens so far, undecayed, as include/kda.h says; kda_gdr_decode takes the token
alone.  Column norms are at
most 2^100 here, so nothing overflows."""
import numpy as np
import pytest

from tests import gdr_reference as R
from tests.test_gpu_gdr import Batch

pytestmark = pytest.mark.gpu
FLOOR = 2.0 ** -117
NO_V = 2.0 ** -120


@pytest.fixture(scope="module")
def torch_cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_82_amd import kda
    kda.library()
    return torch


def group_max(v):
    """|v| [n, dv] -> the largest of each token's group: of every 32 tokens, 4i ..
    4i + 3 and 16 + 4i .. 16 + 4i + 3; a group of less than four goes with the one
    before."""
    n = len(v)
    top = np.empty_like(v)
    for c in range(0, n, 32):
        groups = [[t for t in range(c, min(c + 32, n)) if (t - c) % 16 // 4 == i] for i in range(4)]
        for i, g in enumerate(groups):
            if g:
                with_before = g + groups[i - 1] if i and len(g) < 4 else g
                top[g] = v[with_before].max(0)
    return top


def walk(S, tok, par, hv, rows, G, grouped):
    """State after `rows`, outputs, and their error bounds (above), in fp64."""
    rows = list(rows)
    S = S.astype(np.float64)
    e = np.zeros(S.shape[1])
    v = tok.v[rows, hv].astype(np.float64)
    top = group_max(np.abs(v)) if grouped else np.abs(v)
    out, bound = np.zeros((len(rows), S.shape[1])), np.zeros((len(rows), S.shape[1]))
    amp = np.exp(np.float64(par.a_log[hv]))
    for i, t in enumerate(rows):
        q, k = tok.q[t, hv // G].astype(np.float64), tok.k[t, hv // G].astype(np.float64)
        q = par.scale * q / np.sqrt(q @ q + par.l2_eps)
        k = k / np.sqrt(k @ k + par.l2_eps)
        x = np.float64(tok.gate[t, hv]) + par.dt_bias[hv]
        g = -amp * np.logaddexp(0.0, x) if par.gate_mode == "softplus" else par.lower_bound / (1 + np.exp(-amp * x))
        alpha, beta = np.exp(g), 1.0 / (1.0 + np.exp(-np.float64(tok.beta[t, hv])))
        if i % 32 == 0:
            so_far = np.linalg.norm(S, axis=0)
        S = alpha * S
        held = np.linalg.norm(S, axis=0)
        so_far = np.maximum(so_far, np.maximum(held, top[i]))
        if grouped:
            held = np.where(top[i] > NO_V, held, so_far)
        step = R.STEP * R.EPS * (held + top[i]) + FLOOR
        e = alpha * e + step + (16 * abs(g) * R.EPS * held if alpha > 0 else 0)
        S = S + np.outer(beta * k, v[i] - k @ S)
        out[i], bound[i] = q @ S, par.scale * (e + step)
    return S, out, e, bound


def check(torch, entry, what, lens, **kw):
    print("[case]", entry, what, lens, flush=True)
    b = Batch(torch, lens, **kw)
    d = b.device()
    b.call(entry, d)
    torch.cuda.synchronize()
    out, pool = d["out"].float().cpu().numpy()[0].astype(np.float64), b.host_pool(d).astype(np.float64)
    G = b.HV // b.H
    for r, slot in enumerate(b.slots):
        rows = range(b.cu[r], b.cu[r + 1])
        for hv in range(b.HV):
            S, ref, e, bound = walk(b.pool[slot, hv], b.tok, b.par, hv, rows, G, entry == "prefill")
            if b.qkv == "bf16":
                bound = bound + R.BF16 * (np.abs(ref) + bound)
            err = np.abs(out[list(rows), hv] - ref)
            name = f"{what} {entry} request {r} head {hv}"
            bad = ~(err <= bound)
            assert not bad.any(), (f"{name}: {bad.sum()} outputs off by up to {np.max(err[bad] / bound[bad]):.3g} of "
                                   f"their bounds, first at token, column {np.argwhere(bad)[0]}")
            if len(rows):
                err = np.linalg.norm(pool[slot, hv] - S, axis=0)
                if b.state == "bf16":
                    e = e + R.BF16 * (np.linalg.norm(S, axis=0) + e)
                assert (err <= e).all(), f"{name}: state off by {np.max(err / e):.3g} of its bound"


LENS = [70, 40, 33, 20, 7, 6, 3, 2, 1]


def scaled(t, factor):
    """Token t of each request times `factor`, in two columns of three."""
    def edit(b):
        for a, n in zip(b.cu[:-1], b.lens):
            if t < n:
                b.tok.v[a + t, :, ::3] *= np.float32(factor)
                b.tok.v[a + t, :, 1::3] *= np.float32(factor)
    return edit


@pytest.mark.parametrize("entry", ["prefill", "decode"])
@pytest.mark.parametrize("sigma", [0.0, 0.05])
@pytest.mark.parametrize("t", [0, 1, 5, 17, 31, 32, 39])
def test_one_large_token(torch_cuda, entry, sigma, t):
    for power in (10, 13, 20, 33, 100):
        check(torch_cuda, entry, f"v[{t}] * 2^{power}", LENS, H=1, HV=2, sigma=sigma, edit=scaled(t, 2.0 ** power),
              qkv="f32" if power == 20 else "bf16", layout="v_first" if t % 2 else "k_first")


@pytest.mark.parametrize("H,HV,dk,dv,qkv", [(3, 3, 128, 128, "bf16"), (9, 9, 128, 128, "f32"), (16, 32, 64, 64, "bf16"),
                                            (16, 32, 128, 128, "bf16"), (2, 4, 64, 128, "f32"), (16, 32, 32, 128, "f32"),
                                            (1, 2, 32, 32, "bf16")])
def test_one_large_token_in_every_form(torch_cuda, H, HV, dk, dv, qkv):
    check(torch_cuda, "prefill", "v[21] * 2^30", LENS, H=H, HV=HV, dk=dk, dv=dv, qkv=qkv, edit=scaled(21, 2.0 ** 30))


@pytest.mark.parametrize("entry", ["prefill", "decode"])
@pytest.mark.parametrize("gate", [7.0, 15.0, 30.0, np.inf])
@pytest.mark.parametrize("at", [0, 9, 32])
def test_large_state_that_a_gate_closes(torch_cuda, entry, gate, at):
    """A state of 2^power, open until one token's gate closes it (to e^-7, e^-15,
    e^-30 and 0): what follows is small again."""
    for power in (6, 12, 24, 60):
        def edit(b):
            b.pool[:] *= np.float32(2.0 ** power)
            b.par.a_log[:], b.par.dt_bias[:] = 0.0, 0.0
            b.tok.gate[:] = np.float32(-8)
            for a, n in zip(b.cu[:-1], b.lens):
                if at < n:
                    b.tok.gate[a + at] = np.float32(gate)
        check(torch_cuda, entry, f"S * 2^{power} closed at {at}", LENS, H=1, HV=2, edit=edit, sigma=1.0,
              qkv="f32" if power == 24 else "bf16")


@pytest.mark.parametrize("entry", ["prefill", "decode"])
@pytest.mark.parametrize("gate", [5.0, 9.0, 14.0, 40.0])
@pytest.mark.parametrize("t,at", [(4, 8), (20, 31), (28, 32), (31, 32), (10, 50)])
def test_large_token_that_a_gate_closes(torch_cuda, entry, gate, t, at):
    for power in (8, 11, 16, 40):
        big = scaled(t, 2.0 ** power)

        def edit(b):
            big(b)
            b.par.a_log[:], b.par.dt_bias[:] = 0.0, 0.0
            b.tok.gate[:] = np.float32(-8)
            for a, n in zip(b.cu[:-1], b.lens):
                if at < n:
                    b.tok.gate[a + at] = np.float32(gate)
        check(torch_cuda, entry, f"v[{t}] * 2^{power} closed at {at}", [70, 33, 12], H=1, HV=2, edit=edit)


@pytest.mark.parametrize("entry", ["prefill", "decode"])
@pytest.mark.parametrize("sigma", [0.0, 1.0])
@pytest.mark.parametrize("gate", [-8.0, 4.0])
def test_zeros_then_a_large_token(torch_cuda, entry, sigma, gate):
    """v is zero up to a large token; what the state gives before it stays exact."""
    def edit(b):
        b.par.a_log[:], b.par.dt_bias[:] = 0.0, 0.0
        b.tok.gate[:] = np.float32(gate)
        for a, n in zip(b.cu[:-1], b.lens):
            b.tok.v[a:a + n - n // 5] = 0
            b.tok.v[a + n - n // 5:a + n] *= np.float32(2.0 ** 35)
    check(torch_cuda, entry, "zeros first", LENS, H=1, HV=2, edit=edit, sigma=sigma)


@pytest.mark.parametrize("entry", ["prefill", "decode"])
@pytest.mark.parametrize("qkv,dk,dv", [("bf16", 128, 128), ("f32", 64, 128)])
def test_ordinary_tokens(torch_cuda, entry, qkv, dk, dv):
    """The causal bound on what the other tests draw."""
    for seed in range(3):
        check(torch_cuda, entry, "ordinary", LENS + [200], H=1, HV=2, dk=dk, dv=dv, qkv=qkv, seed=seed,
              sigma=[0.0, 0.05, 2.0][seed])


@pytest.mark.parametrize("entry", ["decode", "window"])
@pytest.mark.parametrize("n", [1, 5, 8, 11])
@pytest.mark.parametrize("requests", [2, 44])
def test_infinite_v_in_the_last_token(torch_cuda, entry, n, requests):
    """A last token with v = inf in one column leaves that column of the state at
    infinities of the keys' signs, token by token and several tokens at a time; all
    other columns stay exact."""
    torch = torch_cuda
    print("[case] infinite v", entry, n, requests, flush=True)
    col = 5

    def edit(b):
        tok, ends = (b.rep, [a + c - 1 for a, c in b.replay]) if entry == "window" else (b.tok, b.cu[1:] - 1)
        for t in ends:
            tok.v[t, :, col] = np.inf

    b = Batch(torch, [n] * requests, H=1, HV=2, layout="v_first", edit=edit,
              replay=[(i * n, n) for i in range(requests)] if entry == "window" else None)
    d = b.device()
    b.call(entry, d)
    torch.cuda.synchronize()
    pool = b.host_pool(d)
    tok = b.rep if entry == "window" else b.tok
    rest = np.arange(128) != col
    for r in {0, requests - 1}:
        rows = range(r * n, r * n + n)
        for hv in range(2):
            tok.v[rows[-1], hv, col] = 0
            S, _, m = R.walk(b.pool[b.slots[r], hv], tok, b.par, hv, rows, 2)
            got = pool[b.slots[r], hv]
            R.check_state(got[:, rest], S[:, rest], m[rest], n, False, f"{entry} request {r} head {hv}")
            np.testing.assert_array_equal(got[:, col], np.sign(tok.k[rows[-1], 0]) * np.inf)


@pytest.mark.parametrize("entry", ["decode", "window"])
@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["k_first", "v_first"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (32, 32), (64, 128)])
@pytest.mark.parametrize("lo,hi", [(0, 3), (3, 5), (5, 9)])
def test_many_requests_of_narrow_keys(torch_cuda, entry, state, layout, dk, dv, lo, hi):
    """The forms that large batches take at dk < 128, on both sides of the lengths at
    which they change."""
    from tests.test_gpu_gdr import run
    rng = np.random.default_rng(hi)
    HV = 1024 // (44 * (dv // 32)) + 1        # more than 512 waves
    lens = rng.integers(lo, hi + 1, size=44).tolist()
    replay = [(int(rng.integers(0, 4)), int(rng.integers(0, hi + 1))) for _ in lens]
    run(torch_cuda, entry, f"{dk}x{dv} {lo}..{hi}", lens, H=HV, HV=HV, dk=dk, dv=dv, state=state, layout=layout,
        replay=replay if entry == "window" else None, seed=lo)


@pytest.mark.parametrize("entry", ["prefill", "decode"])
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
def test_output_in_place_of_v(torch_cuda, entry, qkv):
    """out and v may be one tensor: a token's v is read before its output is written,
    also in chunks that go token by token."""
    torch = torch_cuda
    b = Batch(torch, [70, 33, 5], H=2, HV=2, qkv=qkv, edit=scaled(17, 2.0 ** 30), seed=6)
    d, e = b.device(), b.device()
    b.call(entry, d)
    e["out"] = e["v"]
    b.call(entry, e)
    torch.cuda.synchronize()
    assert torch.equal(d["out"], e["out"]) and torch.equal(d["pool"], e["pool"])


@pytest.mark.parametrize("dk,dv,qkv", [(128, 64, "f32"), (128, 128, "f32"), (128, 128, "bf16"), (64, 64, "f32")])
def test_few_last_tokens_behind_a_large_one(torch_cuda, dk, dv, qkv):
    """Small v after a large one that a gate closes, in a request's last tokens: in the
    first 16 of 32 (11, 38, 13 tokens), where the group before counts as well, and in
    the second, where these tokens' own group has four in the first."""
    def edit(b):
        b.par.a_log[:] = 0
        b.par.dt_bias[:] = 0
        b.tok.gate[:] = 0
        for a, n in zip(b.cu[:-1], b.lens):
            large, small = (n - 1) // 4 * 4 - 3, (n - 1) // 4 * 4
            b.tok.v[a + large] *= np.float32(2.0 ** 33)
            b.tok.gate[a + large + 1:a + small + 1] = 16
    lens = [23, 22, 21, 54, 87, 118, 11, 38, 67, 13]
    check(torch_cuda, "prefill", "large v in the group before the last", lens, H=1, HV=2, dk=dk, dv=dv, qkv=qkv,
          sigma=0.05, edit=edit, seed=11)
