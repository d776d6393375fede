"""GPU parity of the gated delta rule (kda_gdr_decode, kda_gdr_prefill) and of
drafted windows (kda_decode_window) against the 64-bit reference; tolerances
as derived in tests/gdr_reference.py."""
import numpy as np
import pytest

from tests import gdr_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_82_amd import kda
    kda.library()
    return torch


class Batch:
    """One drawn call: host arrays, their device copies and what they should give."""

    def __init__(self, torch, lens, H=2, HV=4, dk=128, dv=128, qkv="bf16", state="f32", layout="k_first",
                 gate_mode="softplus", lower_bound=0.0, slots=None, replay=None, channel=False, seed=0,
                 sigma=0.05, l2_eps=0.0, scale=0.0, edit=None):
        self.torch, self.lens, self.H, self.HV, self.dk, self.dv = torch, list(lens), H, HV, dk, dv
        self.qkv, self.state, self.layout, self.replay, self.channel = qkv, state, layout, replay, channel
        rng = np.random.default_rng(seed)
        B, T = len(self.lens), sum(self.lens)
        self.cu = np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int32)
        self.slots = list(range(B + 1, 1, -1)) if slots is None else list(slots)
        self.N = B + 3
        self.tok = R.Tokens(rng, T, H, HV, dk, dv, channel, qkv == "bf16")
        self.par = R.Params(rng, HV, dk, channel, gate_mode, lower_bound, l2_eps or 1e-6, scale or None)
        self.mode = dict(gate_mode=gate_mode, lower_bound=lower_bound, state_layout=layout, l2_eps=l2_eps,
                         scale=scale)
        if replay is not None:   # [(first row, tokens)] into tokens of their own
            self.rep_T = max([a + n for a, n in replay] + [0]) + 1
            self.rep = R.Tokens(rng, self.rep_T, H, HV, dk, dv, channel, qkv == "bf16")
        self.pool = (rng.standard_normal((self.N, HV, dk, dv)) * sigma).astype(np.float32)
        if state == "bf16":
            self.pool = R.to_bf16(self.pool)
        if edit is not None:
            edit(self)

    def device(self):
        torch = self.torch
        dt = torch.bfloat16 if self.qkv == "bf16" else torch.float32

        def up(x, dtype=None):
            t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
            return t if dtype is None else t.to(dtype)

        def acts(t):
            return [up(x[None], dt) for x in (t.q, t.k, t.v)] + [up(t.gate[None]), up(t.beta[None])]

        pool = self.pool if self.layout == "k_first" else np.swapaxes(self.pool, 2, 3)
        d = {}
        d["q"], d["k"], d["v"], d["gate"], d["beta"] = acts(self.tok)
        d["pool"] = up(pool, torch.bfloat16 if self.state == "bf16" else torch.float32)
        d["cu"], d["idx"] = up(self.cu), up(np.asarray(self.slots, dtype=np.int32))
        d["a_log"], d["bias"] = up(self.par.a_log), up(self.par.dt_bias)
        d["out"] = torch.full_like(d["v"], float("nan"))
        if self.replay is not None:
            _, rk, rv, rg, rb = acts(self.rep)
            d["rep"] = [rk, rv, rg, rb, up(np.asarray([a for a, _ in self.replay], dtype=np.int32)),
                        up(np.asarray([n for _, n in self.replay], dtype=np.int32))]
        return d

    def args(self, d):
        return [d[n] for n in ("out", "q", "k", "v", "gate", "beta", "a_log", "bias", "cu", "pool", "idx")]

    def call(self, entry, d):
        from gated_delta_rule_82_amd import kda
        if entry == "window":
            kda.decode_window(*self.args(d), *d["rep"], **self.mode)
        else:
            {"decode": kda.gdr_decode, "prefill": kda.gdr_prefill}[entry](*self.args(d), **self.mode)

    def host_pool(self, d):
        p = d["pool"].float().cpu().numpy()
        return p if self.layout == "k_first" else np.swapaxes(p, 2, 3)

    def check(self, entry, d, what=""):
        out, pool = d["out"].float().cpu().numpy()[0], self.host_pool(d)
        G = self.HV // self.H
        written = set()
        for b, slot in enumerate(self.slots):
            rows = range(self.cu[b], self.cu[b + 1])
            for hv in range(self.HV):
                name = f"{what} {entry} request {b} head {hv}"
                if slot < 0 or slot >= self.N:
                    assert (out[list(rows), hv] == 0).all(), name
                    continue
                S, n0 = self.pool[slot, hv], 0
                m0 = np.linalg.norm(S.astype(np.float64), axis=0)
                if entry == "window":
                    first, n0 = self.replay[b]
                    S, _, m0 = R.walk(S, self.rep, self.par, hv, range(first, first + n0), G)
                S2, ref, m = R.walk(S, self.tok, self.par, hv, rows, G)
                m = np.maximum(m, m0)
                if entry != "window":
                    S, n0, m0 = S2, len(rows), m
                n = len(rows) + (n0 if entry == "window" else 0)
                if n0:
                    R.check_state(pool[slot, hv], S, m0, n0, self.state == "bf16", name)
                    written.add((slot, hv))
                R.check_out(out[list(rows), hv], ref, m, n, self.par.scale, self.qkv == "bf16", name)
        for slot in range(self.N):
            for hv in range(self.HV):
                if (slot, hv) not in written:   # bit for bit
                    assert (pool[slot, hv] == self.pool[slot, hv]).all(), f"{what} slot {slot} head {hv} changed"


def run(torch, entry, what, lens, **kw):
    print("[case]", entry, what, lens, kw, flush=True)
    b = Batch(torch, lens, **kw)
    d = b.device()
    b.call(entry, d)
    torch.cuda.synchronize()
    b.check(entry, d, what)
    return b, d


LAYOUTS = ["k_first", "v_first"]
MIXED = [1, 3, 0, 8, 2]
REPLAYS = [(0, 2), (5, 1), (2, 0), (1, 8), (9, 3)]


@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("qkv", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (32, 32), (16, 64), (64, 16), (16, 16)])
def test_decode(torch_cuda, dk, dv, layout, qkv, state):
    run(torch_cuda, "decode", f"{dk}x{dv}", MIXED, dk=dk, dv=dv, layout=layout, qkv=qkv, state=state)


@pytest.mark.parametrize("channel", [False, True])
@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dk,dv,qkv", [(128, 128, "bf16"), (64, 128, "f32"), (128, 64, "f32"), (32, 16, "bf16"),
                                       (16, 16, "f32"), (16, 128, "bf16"), (64, 64, "bf16")])
def test_window(torch_cuda, dk, dv, qkv, layout, state, channel):
    run(torch_cuda, "window", f"{dk}x{dv}", MIXED, replay=REPLAYS, dk=dk, dv=dv, layout=layout, qkv=qkv,
        state=state, channel=channel)


# windows long enough (on average) to go several tokens at a time, with
# requests of one token, of none and of whole and broken groups of 8
LONG = [8, 33, 3, 0, 17, 9, 1, 40]
LONG_REPLAYS = [(0, 9), (3, 1), (0, 0), (2, 8), (5, 17), (1, 3), (0, 16), (4, 2)]


@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("qkv", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (32, 32), (32, 16), (64, 16), (16, 32)])
def test_long_decode(torch_cuda, dk, dv, layout, qkv, state):
    run(torch_cuda, "decode", f"long {dk}x{dv}", LONG, dk=dk, dv=dv, layout=layout, qkv=qkv, state=state)


@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("qkv", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 16), (32, 64)])
def test_long_window(torch_cuda, dk, dv, layout, qkv, state):
    run(torch_cuda, "window", f"long {dk}x{dv}", LONG, replay=LONG_REPLAYS, dk=dk, dv=dv, layout=layout, qkv=qkv,
        state=state)


@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("qkv", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 32), (32, 16)])
def test_short_window(torch_cuda, dk, dv, layout, qkv, state):
    run(torch_cuda, "window", f"short {dk}x{dv}", [1, 2, 0, 3, 1], replay=REPLAYS, dk=dk, dv=dv, layout=layout,
        qkv=qkv, state=state)


@pytest.mark.parametrize("m", range(0, 12))
def test_replay_and_window_sizes(torch_cuda, m):
    """Every number of replayed tokens with every window: those that fit go
    through the state at once (m + 2 n <= 16 rows, m + n <= 11), the others
    one after the other."""
    n = list(range(0, 9))
    for layout, state, qkv in (("v_first", "f32", "bf16"), ("k_first", "bf16", "bf16"), ("k_first", "f32", "f32")):
        run(torch_cuda, "window", f"{m} replayed", n, replay=[(i, m) for i in n], H=1, HV=2, layout=layout,
            state=state, qkv=qkv, seed=m)


@pytest.mark.parametrize("entry", ["decode", "window"])
@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("lo,hi", [(0, 2), (3, 5), (6, 9), (9, 20)])
def test_many_requests(torch_cuda, entry, state, layout, lo, hi):
    """More than half a wave per SIMD: the forms of large batches."""
    rng = np.random.default_rng(lo)
    lens = rng.integers(lo, hi + 1, size=44).tolist()
    replay = [(int(rng.integers(0, 4)), int(rng.integers(0, hi + 1))) for _ in lens]
    run(torch_cuda, entry, f"{lo}..{hi}", lens, replay=replay if entry == "window" else None, state=state,
        layout=layout, seed=lo)


@pytest.mark.parametrize("entry", ["decode", "window"])
@pytest.mark.parametrize("H,HV", [(1, 1), (3, 3), (1, 6), (5, 15)])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_heads(torch_cuda, entry, H, HV, layout):
    run(torch_cuda, entry, "heads", [2, 1], H=H, HV=HV, layout=layout, gate_mode="lower_bound", lower_bound=-5.0,
        replay=[(1, 1), (0, 3)] if entry == "window" else None)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("channel", [False, True])
def test_skipped_empty_and_clamped_requests(torch_cuda, layout, channel):
    # negative and too large indices skip; a request without tokens, one
    # without a replay, one with neither
    slots = [-1, 3, 99, 0, 1, 2]
    run(torch_cuda, "window", "skips", [2, 0, 1, 3, 0, 1], slots=slots,
        replay=[(0, 2), (2, 3), (1, 1), (0, 0), (0, 0), (4, 1)], layout=layout, channel=channel)
    if not channel:
        run(torch_cuda, "decode", "skips", [2, 0, 1, 3, 0, 1], slots=slots, layout=layout)
        run(torch_cuda, "decode", "long skips", [20, 0, 30, 35, 0, 11], slots=slots, layout=layout)
        run(torch_cuda, "window", "long skips", [20, 0, 30, 35, 0, 11], slots=slots,
            replay=[(0, 2), (2, 3), (1, 1), (0, 0), (0, 0), (4, 10)], layout=layout)


def test_replay_only_batch(torch_cuda):
    run(torch_cuda, "window", "no window at all", [0, 0], replay=[(0, 3), (3, 1)])


@pytest.mark.parametrize("entry", ["decode", "window"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("kind", ["zero qk", "strong decay", "no decay", "tiny beta", "scalars"])
def test_degenerate(torch_cuda, entry, layout, kind):
    kw, edit = {}, None
    if kind == "zero qk":
        def edit(b):
            b.tok.q[::2], b.tok.k[1::2] = 0, 0
    elif kind == "strong decay":     # the pending decay folds at once, down to exp(g) = 0
        def edit(b):
            b.tok.gate[:] += np.float32(30)
            b.tok.gate[::3] = np.float32(3e4)
            b.par.a_log[:] = 1.0
    elif kind == "no decay":
        def edit(b):
            b.tok.gate[:] = np.float32(-200)
    elif kind == "tiny beta":
        def edit(b):
            b.tok.beta[:] = np.float32(-120)
    else:
        kw = dict(l2_eps=0.5, scale=3.0)
    for lens in ([5, 1, 7], [30, 9, 12]):   # token by token, and several at a time
        run(torch_cuda, entry, kind, lens, layout=layout, edit=edit,
            replay=[(0, 4), (2, 2), (1, 0)] if entry == "window" else None, **kw)


def test_many_tokens_match_single_token_calls(torch_cuda):
    """A request's tokens in one call or one call each: the same recurrence
    (bounded by the sum of both sides' bounds; the order of work differs)."""
    torch = torch_cuda
    from gated_delta_rule_82_amd import kda
    b = Batch(torch, [6, 6], seed=5)
    one, many = b.device(), b.device()
    b.call("decode", many)
    idx = torch.tensor([0, 6], device="cuda")
    cu = torch.arange(3, dtype=torch.int32, device="cuda")
    for t in range(6):
        part = {n: one[n][:, idx + t].contiguous() for n in ("q", "k", "v", "gate", "beta", "out")}
        kda.gdr_decode(part["out"], part["q"], part["k"], part["v"], part["gate"], part["beta"], one["a_log"],
                       one["bias"], cu, one["pool"], one["idx"], **b.mode)
        one["out"][:, idx + t] = part["out"]
    torch.cuda.synchronize()
    b.check("decode", many, "one call")
    b.check("decode", one, "single tokens")


@pytest.mark.parametrize("n", [2, 16])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_window_equals_decode_of_kept_then_new(torch_cuda, layout, n):
    """decode_window = gdr_decode of the kept tokens, then of the window on a
    copy of the pool.  Both sides take the same form of the kernel (n tokens a
    request each time), so the pool is equal bit for bit."""
    torch = torch_cuda
    from gated_delta_rule_82_amd import kda
    b = Batch(torch, [n, n], replay=[(0, n), (n, n)], layout=layout, seed=3)
    d, e = b.device(), b.device()
    b.call("window", d)
    rk, rv, rg, rb, begin, count = e["rep"]
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    rk, rv, rg, rb = (x[:, :2 * n].contiguous() for x in (rk, rv, rg, rb))
    kda.gdr_decode(torch.empty_like(rv), rk, rk, rv, rg, rb, e["a_log"], e["bias"], cu, e["pool"], e["idx"], **b.mode)
    kept = e["pool"].clone()
    b.call("decode", e)
    torch.cuda.synchronize()
    assert torch.equal(d["pool"], kept)
    b.check("window", d)


@pytest.mark.parametrize("scale", [1, 6])   # token by token, and several at a time
@pytest.mark.parametrize("channel", [False, True])
def test_replay_out_of_range_stays_inside(torch_cuda, channel, scale):
    """begin is clamped to the replay's rows and count to the rows that follow."""
    torch = torch_cuda
    b = Batch(torch, [2 * scale, scale, scale], replay=[(0, 4), (1, 2), (0, 5)], channel=channel, seed=4)
    d = b.device()
    Tr = d["rep"][0].shape[1]
    d["rep"][4] = torch.tensor([-3, Tr + 5, Tr - 1], dtype=torch.int32, device="cuda")
    d["rep"][5] = torch.tensor([999, 4, 7], dtype=torch.int32, device="cuda")
    b.call("window", d)
    torch.cuda.synchronize()
    b.replay = [(0, Tr), (0, 0), (Tr - 1, 1)]
    b.check("window", d)
    d = b.device()
    d["rep"][5] = torch.tensor([-1, -2 ** 31, 0], dtype=torch.int32, device="cuda")
    b.call("window", d)
    torch.cuda.synchronize()
    b.replay = [(0, 0)] * 3
    b.check("window", d)


@pytest.mark.parametrize("entry", ["decode", "window", "prefill"])
@pytest.mark.parametrize("scale", [1, 9])
def test_rows_behind_the_last_request_and_bad_offsets(torch_cuda, entry, scale):
    """Rows past cu_seqlens[B] keep what they held; offsets outside the
    tensors are clamped to them."""
    torch = torch_cuda
    lens = [2 * scale, 3 * scale, 4 * scale]
    b = Batch(torch, lens, replay=[(0, 1)] * 3, seed=7)
    d = b.device()
    d["cu"] = d["cu"].clone()
    d["cu"][3] = 5 * scale            # the last request has no rows, its tokens lie behind
    b.call(entry, d)
    torch.cuda.synchronize()
    assert torch.isnan(d["out"][:, 5 * scale:]).all()
    b.cu, b.lens = np.array([0, 2 * scale, 5 * scale, 5 * scale]), lens[:2] + [0]
    b.check(entry, d)
    b = Batch(torch, lens, replay=[(0, 1)] * 3, seed=7)
    d = b.device()
    d["cu"] = torch.tensor([-7, 2 * scale, 5 * scale, 10 ** 9], dtype=torch.int32, device="cuda")
    b.call(entry, d)
    torch.cuda.synchronize()
    b.check(entry, d)


@pytest.mark.parametrize("entry", ["decode", "window", "prefill"])
def test_given_stream(torch_cuda, entry):
    """On a stream given by its handle, behind that stream's own work."""
    torch = torch_cuda
    from gated_delta_rule_82_amd import kda
    b = Batch(torch, [3, 40, 7], replay=[(0, 2), (1, 3), (0, 0)], seed=8)
    d, e = b.device(), b.device()
    b.call(entry, d)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    q = e["q"].clone()
    e["q"].zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(10 ** 7)
        e["q"].copy_(q)
    call = {"decode": kda.gdr_decode, "prefill": kda.gdr_prefill, "window": kda.decode_window}[entry]
    call(*b.args(e), *(e["rep"] if entry == "window" else []), stream=side.cuda_stream, **b.mode)
    torch.cuda.synchronize()
    assert torch.equal(d["out"], e["out"]) and torch.equal(d["pool"], e["pool"])


def test_binding_refuses_what_cannot_be_passed(torch_cuda):
    torch = torch_cuda
    from gated_delta_rule_82_amd import kda
    b = Batch(torch, [2, 1])
    d = b.device()
    for name, value, error in (("q", d["q"].half(), ValueError), ("q", d["q"].transpose(1, 2), ValueError),
                               ("v", d["v"].cpu(), ValueError), ("beta", None, TypeError), ("a_log", 3.0, TypeError),
                               ("pool", d["pool"][None], ValueError), ("pool", d["pool"][:, :3], ValueError)):
        with pytest.raises(error, match="out|q|v|beta_logits|a_log|state_pool"):
            kda.gdr_decode(*b.args(dict(d, **{name: value})), **b.mode)
    with pytest.raises(kda.KdaError) as e:
        kda.gdr_decode(*b.args(dict(d, bias=d["bias"][:3].clone())), **b.mode)
    assert e.value.code == kda.KDA_ERR_SHAPE
    with pytest.raises(kda.KdaError) as e:
        kda.gdr_prefill(*b.args(d), **dict(b.mode, gate_mode="lower_bound", lower_bound=-1e39))
    assert e.value.code == kda.KDA_ERR_MODE


def test_offsets_past_32_bits(torch_cuda):
    """A pool of more than 2^31 values: the last slot's tile is found."""
    torch = torch_cuda
    from gated_delta_rule_82_amd import kda
    b = Batch(torch, [2], H=1, HV=2, slots=[0])
    d = b.device()
    N = (2 ** 31) // (2 * 128 * 128) + 9
    pool = torch.zeros((N, 2, 128, 128), dtype=torch.float32, device="cuda")
    pool[N - 1] = d["pool"][0]
    args = b.args(d)
    args[9], args[10] = pool, torch.tensor([N - 1], dtype=torch.int32, device="cuda")
    kda.gdr_decode(*args, **b.mode)
    b.call("decode", e := b.device())
    torch.cuda.synchronize()
    assert torch.equal(pool[N - 1], e["pool"][0]) and torch.equal(d["out"], e["out"])
    assert not pool[:N - 1].any()


@pytest.mark.parametrize("entry", ["decode", "window", "prefill"])
def test_two_runs_are_bit_identical(torch_cuda, entry):
    torch = torch_cuda
    b = Batch(torch, [7, 70, 1, 130], seed=9, replay=[(0, 2), (0, 3), (1, 1), (0, 0)])
    runs = []
    for _ in range(3):
        d = b.device()
        b.call(entry, d)
        runs.append((d["out"], d["pool"]))
    torch.cuda.synchronize()
    for out, pool in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(pool, runs[0][1])


# ---------------------------------------------------------------------------
# whole prompts
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("qkv", ["f32", "bf16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (32, 32), (64, 64), (32, 128), (128, 32)])
def test_prefill(torch_cuda, dk, dv, layout, qkv, state):
    run(torch_cuda, "prefill", f"{dk}x{dv}", [65, 1, 130, 0, 17], H=1, HV=2, dk=dk, dv=dv, layout=layout, qkv=qkv,
        state=state)


@pytest.mark.parametrize("qkv", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 127, 128, 129, 200])
def test_prefill_lengths(torch_cuda, n, qkv):
    run(torch_cuda, "prefill", "length", [n, 3], H=1, HV=1, qkv=qkv, layout="v_first" if n % 2 else "k_first")


@pytest.mark.parametrize("B,H,HV", [(1, 1, 1), (1, 3, 3), (3, 2, 8), (2, 16, 32), (9, 16, 16)])
def test_prefill_heads(torch_cuda, B, H, HV):
    run(torch_cuda, "prefill", "heads", [40 + 13 * b for b in range(B)], H=H, HV=HV, gate_mode="lower_bound",
        lower_bound=-5.0, layout="v_first")


@pytest.mark.parametrize("HV,dk,dv,qkv", [(16, 64, 128, "bf16"), (16, 128, 128, "f32"), (6, 128, 128, "bf16"),
                                          (3, 128, 128, "f32"), (5, 32, 64, "f32"), (16, 128, 32, "bf16")])
def test_prefill_many_tiles(torch_cuda, HV, dk, dv, qkv):
    """From some to more (request, head) tiles than compute units: each form of the workgroups."""
    run(torch_cuda, "prefill", "tiles", [66 + b for b in range(20)], H=HV, HV=HV, dk=dk, dv=dv, qkv=qkv)


def test_prefill_skips(torch_cuda):
    run(torch_cuda, "prefill", "skips", [20, 0, 70, 3, 0, 100], slots=[-1, 3, 99, 0, 1, 2])


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("qkv", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["zero qk", "strong decay", "no decay", "equal keys", "tiny beta", "large v",
                                  "small and large rows", "scalars", "zero state"])
def test_prefill_degenerate(torch_cuda, kind, qkv, layout):
    kw, edit = {}, None
    if kind == "zero qk":
        def edit(b):
            b.tok.q[::2], b.tok.k[1::2] = 0, 0
    elif kind == "strong decay":
        def edit(b):
            b.tok.gate[:] += np.float32(30)
            b.tok.gate[::7] = np.float32(3e4)
            b.par.a_log[:] = 1.0
    elif kind == "no decay":
        def edit(b):
            b.tok.gate[:] = np.float32(-200)
            b.tok.beta[:] += np.float32(4)
    elif kind == "equal keys":       # the chunk's solve at its least favourable
        def edit(b):
            b.tok.k[:] = b.tok.k[:1]
            b.tok.gate[:] = np.float32(-200)
            b.tok.beta[:] = np.float32(30)
    elif kind == "tiny beta":
        def edit(b):
            b.tok.beta[:] = np.float32(-120)
    elif kind == "large v":
        def edit(b):
            b.tok.v[:, :, ::3] *= np.float32(2.0 ** 40)
            b.pool[..., 1::3] *= np.float32(2.0 ** -40)
            b.tok.v[:, :, 1::3] *= np.float32(2.0 ** -40)
    elif kind == "small and large rows":
        def edit(b):
            s = np.float32(2.0) ** np.arange(-20, 20, 40 / b.tok.q.shape[0])[:b.tok.q.shape[0], None, None]
            b.tok.q *= s.astype(np.float32)
            b.tok.k *= s[::-1].astype(np.float32)
            if b.qkv == "bf16":
                b.tok.q, b.tok.k = R.to_bf16(b.tok.q), R.to_bf16(b.tok.k)
    elif kind == "scalars":
        kw = dict(l2_eps=0.5, scale=3.0)
    else:
        kw = dict(sigma=0.0)
    run(torch_cuda, "prefill", kind, [150, 5], H=1, HV=2, qkv=qkv, layout=layout, edit=edit, **kw)


@pytest.mark.parametrize("qkv", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
@pytest.mark.parametrize("kind", ["fresh state", "after zeros", "tiny state"])
def test_prefill_large_v_over_nothing(torch_cuda, kind, dk, dv, qkv):
    """Columns of v from 2^-60 to 2^100 over a state that is zero or far
    smaller: fresh requests, a column whose v begins after several chunks, and a
    state of size 2^-90."""
    def edit(b):
        size = np.float32(2.0) ** np.resize(np.array([0, 24, 32, 40, 64, 100, -60], dtype=np.float32), b.dv)
        b.tok.v *= size.astype(np.float32)
        if kind == "after zeros":
            b.tok.v[:70, :, ::2] = 0
        if kind == "tiny state":
            b.pool[:] *= np.float32(2.0 ** -90)
    run(torch_cuda, "prefill", kind, [150, 40, 3], H=1, HV=2, dk=dk, dv=dv, qkv=qkv, edit=edit,
        sigma=1.0 if kind == "tiny state" else 0.0)


def test_prefill_long(torch_cuda):
    run(torch_cuda, "prefill", "long", [3000], H=1, HV=1, layout="v_first")


def test_prefill_infinite_gate_input(torch_cuda):
    """raw_gate of +inf (softplus) closes the gate: alpha = 0, exactly a restart."""
    def edit(b):
        b.tok.gate[10] = b.tok.gate[70] = b.tok.gate[71] = np.float32(np.inf)
    run(torch_cuda, "prefill", "closed gate", [100], H=1, HV=1, edit=edit)
    run(torch_cuda, "decode", "closed gate", [100], H=1, HV=1, edit=edit)


@pytest.mark.parametrize("entry,channel,tokens", [("decode", False, 1), ("decode", False, 2), ("window", False, 1),
                                                  ("window", False, 2), ("window", True, 1)])
@pytest.mark.parametrize("state", ["float32", "bfloat16"])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_large_batch_equals_its_parts(torch_cuda, layout, state, entry, channel, tokens):
    """128 requests x 32 heads in one call, whose launch holds fewer waves per
    CU, give bit for bit what calls of 16 requests give: requests do not meet."""
    torch = torch_cuda
    from gated_delta_rule_82_amd import kda
    B, H, D, part = 128, 32, 128, 16
    T = B * tokens
    g = torch.Generator(device="cuda").manual_seed(3)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    gate_tail = (H, D) if channel else (H,)
    acts = [[randn(1, T, H, D, dtype=torch.bfloat16) for _ in range(3)] + [randn(1, T, *gate_tail), randn(1, T, H)]
            for _ in range(2)]
    par = [randn(H) * 0.3, randn(*gate_tail)]
    pool0 = (randn(B, H, D, D) * 0.05).to(getattr(torch, state))
    count = torch.randint(0, tokens + 1, (B,), generator=g, device="cuda", dtype=torch.int32)

    def run_groups(size):
        pool, outs = pool0.clone(), []
        for b in range(0, B, size):
            rows = slice(b * tokens, (b + size) * tokens)
            x, y = ([t[:, rows] for t in a] for a in acts)
            cu = torch.arange(0, (size + 1) * tokens, tokens, dtype=torch.int32, device="cuda")
            idx = torch.arange(b, b + size, dtype=torch.int32, device="cuda")
            out = torch.full_like(x[2], float("nan"))
            call = [out, *x, *par, cu, pool, idx]
            if entry == "window":
                kda.decode_window(*call, *y[1:], cu[:-1].clone(), count[b:b + size].clone(), state_layout=layout)
            else:
                kda.gdr_decode(*call, state_layout=layout)
            outs.append(out)
        return torch.cat(outs, 1), pool

    (o_all, s_all), (o_part, s_part) = run_groups(B), run_groups(part)
    assert torch.isfinite(o_all.float()).all()
    assert torch.equal(o_all, o_part) and torch.equal(s_all, s_part)
    assert not torch.equal(s_all, pool0)
