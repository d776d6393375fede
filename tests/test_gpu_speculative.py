"""Draft verification (kda_verify) against the 64-bit reference, and the
operators as a serving loop runs them: window, verification, next window."""
import numpy as np
import pytest

from tests import gdr_reference as R
from tests.test_gpu_gdr import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_82_amd import kda
    kda.library()
    return torch


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


class Case:
    def __init__(self, lens, V, bf16=False, draft=True, seed=0, agree=0.5, edit=None):
        rng = np.random.default_rng(seed)
        T = sum(lens)
        self.V, self.bf16 = V, bf16
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        logits = rng.standard_normal((T, V)) * 2
        self.target = softmax(logits)
        self.draft = softmax(logits + agree * rng.standard_normal((T, V))) if draft else None
        if bf16:
            self.target = R.to_bf16(self.target)
            self.draft = None if self.draft is None else R.to_bf16(self.draft)
        pick = self.target if self.draft is None else self.draft
        self.tokens = np.zeros(T, dtype=np.int32)
        for t in range(T - 1):
            cum = np.cumsum(pick[t].astype(np.float64))
            self.tokens[t + 1] = min(V - 1, np.searchsorted(cum, rng.random() * cum[-1]))
        self.u_accept = rng.random(T, dtype=np.float32)
        self.u_sample = rng.random(len(lens), dtype=np.float32)
        if edit is not None:
            edit(self)

    def device(self, torch):
        dt = torch.bfloat16 if self.bf16 else torch.float32

        def up(x, dtype=None):
            t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
            return t if dtype is None else t.to(dtype)
        B = len(self.cu) - 1
        return dict(n_commit=torch.full((B,), -7, dtype=torch.int32, device="cuda"),
                    next_token=torch.full((B,), -7, dtype=torch.int32, device="cuda"),
                    target=up(self.target, dt), draft=None if self.draft is None else up(self.draft, dt),
                    tokens=up(self.tokens), u_accept=up(self.u_accept), u_sample=up(self.u_sample), cu=up(self.cu))

    def reference(self):
        return R.verify(self.target, self.draft, self.tokens, self.u_accept, self.u_sample, self.cu)


def call(d, **kw):
    from gated_delta_rule_82_amd import kda
    kda.verify(d["n_commit"], d["next_token"], d["target"], d["draft"], d["tokens"], d["u_accept"], d["u_sample"],
               d["cu"], **kw)


def check(torch, case, d=None):
    if d is None:
        d = case.device(torch)
        call(d)
    torch.cuda.synchronize()
    n, x = case.reference()
    np.testing.assert_array_equal(d["n_commit"].cpu().numpy(), n)
    np.testing.assert_array_equal(d["next_token"].cpu().numpy(), x)
    return n, x


@pytest.mark.parametrize("V", [1, 2, 3, 7, 64, 1021, 1024, 1025, 4096, 30011])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("draft", [True, False])
def test_verify(torch_cuda, V, bf16, draft):
    print("[case] verify", V, bf16, draft, flush=True)
    for seed in range(3):
        check(torch_cuda, Case([1, 5, 0, 2, 8, 3], V, bf16, draft, seed=seed))


@pytest.mark.parametrize("lens", [[1], [0, 0, 4, 0], [130, 2], [2] * 300, [5] * 64])
def test_verify_windows(torch_cuda, lens):
    print("[case] windows", len(lens), flush=True)
    n, _ = check(torch_cuda, Case(lens, 517, seed=1, agree=0.1))
    if lens[0] == 5:
        assert len(set(n.tolist())) > 2     # some drafts stand, some fall


@pytest.mark.parametrize("draft", [True, False])
def test_verify_no_tokens_at_all(torch_cuda, draft):
    check(torch_cuda, Case([0, 0, 0], 77, draft=draft))


def test_verify_large_vocabulary(torch_cuda):
    check(torch_cuda, Case([3, 4], 300007, seed=2))


def _edit(kind):
    def edit(c):
        T, V = c.target.shape
        if kind == "all accepted":
            c.u_accept[:] = 0
        elif kind == "all rejected":
            c.u_accept[:] = 1
            c.target[np.arange(T - 1), c.tokens[1:]] = 0
        elif kind == "equal distributions":      # p = q: u < 1 accepts
            c.draft = c.target.copy()
        elif kind == "no residual":              # rejected, and nothing of p exceeds q
            c.draft = c.target.copy()
            c.u_accept[:] = 1
        elif kind == "one hot target":
            c.target[:] = 0
            c.target[np.arange(T), np.arange(T) * 5 % V] = 1
        elif kind == "nothing":                  # a target without mass
            c.target[:] = 0
        elif kind == "bad values":
            c.target[:, ::7] = np.nan
            c.target[:, 1::7] = -1
            c.target[:, 2::7] = np.inf
            c.draft[:, 3::7] = np.nan
            c.draft[:, 4::7] = -np.inf
        elif kind == "bad tokens":
            c.tokens[1::3] = V
            c.tokens[2::3] = -1
        elif kind == "bad randoms":
            c.u_accept[::2] = np.nan
            c.u_sample[:] = np.resize(np.array([np.nan, -1, 1, 2, np.inf, 0], dtype=np.float32), c.u_sample.shape)
        elif kind == "tiny":                     # subnormal mass counts
            c.target[:] = np.float32(0)
            c.target[:, 11] = np.float32(2.0 ** -126)
            c.target[:, V - 1] = np.float32(2.0 ** -126)
    return edit


@pytest.mark.parametrize("V", [40, 2051])
@pytest.mark.parametrize("kind", ["all accepted", "all rejected", "equal distributions", "no residual",
                                  "one hot target", "nothing", "bad values", "bad tokens", "bad randoms", "tiny"])
def test_verify_degenerate(torch_cuda, kind, V):
    print("[case]", kind, V, flush=True)
    check(torch_cuda, Case([4, 1, 3, 0, 6, 2], V, seed=4, edit=_edit(kind)))
    if kind not in ("equal distributions", "no residual", "bad values"):
        check(torch_cuda, Case([4, 1, 3, 0, 6, 2], V, draft=False, seed=4, edit=_edit(kind)))


@pytest.mark.parametrize("u", [1.0, 2.0 ** 60, 1.0 - 2.0 ** -24])
def test_verify_scattered_mass_and_u_of_one(torch_cuda, u):
    """Rows with a few tokens of mass far apart and of very different size, as
    top-k leaves them: u of one (or more) gives the last of them.  The running
    sums of these rows round above their total at segments without mass (found
    with a model of the lane-wise scan), which must not be picked."""
    torch = torch_cuda
    print("[case] scattered mass", u, flush=True)
    seeds = [2062, 8558, 10831, 11048, 13096, 13829, 14968, 16158, 18980, 22236, 22395, 22648, 23644, 24290, 25312]

    def edit(c):
        c.target[:] = 0
        for t, seed in enumerate(seeds):
            rng = np.random.default_rng(seed)
            n = int(rng.integers(2, 40))
            segment = np.sort(rng.choice(128, n, replace=False))
            c.target[t, segment * 1024 + 500] = np.exp(9 * rng.standard_normal(n)).astype(np.float32)
        c.u_sample[:] = np.float32(u)

    c = Case([1] * len(seeds), 128 * 1024, draft=False, edit=edit)
    _, x = check(torch, c)
    if u >= 1:
        np.testing.assert_array_equal(x, [np.nonzero(row)[0][-1] for row in c.target])


def test_verify_metadata_out_of_range_stays_inside(torch_cuda):
    """cu_seqlens that breaks its precondition is clamped to the rows there are."""
    torch = torch_cuda
    c = Case([3, 3], 100, seed=6)
    d = c.device(torch)
    d["cu"] = torch.tensor([-5, 3, 400], dtype=torch.int32, device="cuda")
    call(d)
    check(torch, c, d)


def test_verify_offsets_past_32_bits(torch_cuda):
    """Rows that begin past 2^31 values of the distributions."""
    torch = torch_cuda
    V, T = 300007, 7200     # T * V > 2^31
    c = Case([4, 3], V, draft=False, seed=8)
    d = c.device(torch)
    big = torch.zeros((T, V), dtype=torch.float32, device="cuda")
    big[T - 7:] = d["target"]
    tokens = torch.zeros(T, dtype=torch.int32, device="cuda")
    tokens[T - 7:] = d["tokens"]
    u = torch.zeros(T, device="cuda")
    u[T - 7:] = d["u_accept"]
    d.update(target=big, tokens=tokens, u_accept=u,
             cu=torch.tensor([T - 7, T - 3, T], dtype=torch.int32, device="cuda"))
    call(d)
    check(torch, c, d)


def test_verify_on_two_streams_and_given_workspace(torch_cuda):
    torch = torch_cuda
    from gated_delta_rule_82_amd import kda
    cases = [Case([5] * 40, 5003, seed=s) for s in (1, 2)]
    ds = [c.device(torch) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for d, s in zip(ds, streams):
        with torch.cuda.stream(s):
            call(d)
    ws = torch.empty(kda.verify_workspace(40, 5003), device="cuda")
    torch.cuda.synchronize()
    e = cases[0].device(torch)
    torch.cuda.synchronize()
    call(e, workspace=ws, stream=streams[0].cuda_stream)
    for c, d in zip(cases + cases[:1], ds + [e]):
        check(torch, c, d)


# ---------------------------------------------------------------------------
# the run of a serving loop
# ---------------------------------------------------------------------------

def _loop_state(torch, channel):
    B, W, V = 6, 5, 1009
    b = Batch(torch, [W] * B, H=2, HV=4, layout="v_first", channel=channel, seed=12)
    rng = np.random.default_rng(3)
    windows = [R.Tokens(rng, B * W, 2, 4, 128, 128, channel, True) for _ in range(4)]
    cases = [Case([W] * B, V, seed=20 + s, agree=0.3) for s in range(4)]
    return b, windows, cases


@pytest.mark.parametrize("channel", [False, True])
def test_speculative_loop(torch_cuda, channel):
    """window -> verify -> next window with the verdict as its replay.  After
    every step the pool holds exactly the tokens that stand."""
    torch = torch_cuda
    from gated_delta_rule_82_amd import kda
    b, windows, cases = _loop_state(torch, channel)
    B, W, HV = 6, 5, 4
    d = b.device()
    cu = d["cu"]
    prev, count = None, torch.zeros(B, dtype=torch.int32, device="cuda")
    ref = {(i, hv): (b.pool[b.slots[i], hv].astype(np.float64), 0, 0.0) for i in range(B) for hv in range(HV)}
    kept = np.zeros(B, dtype=int)
    for step in range(4):
        tok = windows[step]
        up = [torch.from_numpy(x[None]).cuda().to(torch.bfloat16) for x in (tok.q, tok.k, tok.v)]
        up += [torch.from_numpy(x[None]).cuda() for x in (tok.gate, tok.beta)]
        src = prev if prev is not None else up
        out = torch.empty_like(up[2])
        kda.decode_window(out, *up, d["a_log"], d["bias"], cu, d["pool"], d["idx"], src[1], src[2], src[3], src[4],
                          cu[:-1], count, **b.mode)
        v = cases[step].device(torch)
        call(v)
        n, _ = check(torch, cases[step], v)
        got, pool = out.float().cpu().numpy()[0], b.host_pool(d)
        for i in range(B):
            for hv in range(HV):
                S, walked, m = ref[i, hv]
                if step:
                    S, _, m1 = R.walk(S, windows[step - 1], b.par, hv, range(i * W, i * W + kept[i]), 2)
                    walked, m = walked + kept[i], np.maximum(m, m1)
                    R.check_state(pool[b.slots[i], hv], S, m, walked, False, f"step {step} request {i} head {hv}")
                ref[i, hv] = (S, walked, m)
                rows = range(i * W, i * W + W)
                _, o, m2 = R.walk(S, tok, b.par, hv, rows, 2)
                R.check_out(got[list(rows), hv], o, np.maximum(m, m2), walked + W, b.par.scale, True,
                            f"step {step} request {i} head {hv}")
        kept, count, prev = n, v["n_commit"], up


def test_captured_step_replays(torch_cuda):
    """window and verify captured as one graph, replayed between eager work:
    every replay equals the eager calls."""
    torch = torch_cuda
    from gated_delta_rule_82_amd import kda
    b, windows, cases = _loop_state(torch, False)
    d, e = b.device(), b.device()
    v, w = cases[0].device(torch), cases[0].device(torch)
    count_d = torch.full((6,), 2, dtype=torch.int32, device="cuda")
    count_e = count_d.clone()

    def step(x, y, count):
        kda.decode_window(*b.args(x), x["k"], x["v"], x["gate"], x["beta"], x["cu"][:-1], count, **b.mode)
        call(y)
        count.copy_(y["n_commit"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = b.device()
        step(warm, cases[0].device(torch), count_d.clone())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(d, v, count_d)
    torch.cuda.synchronize()
    for i in range(4):
        graph.replay()
        step(e, w, count_e)
        torch.cuda.synchronize()
        assert torch.equal(d["out"], e["out"]) and torch.equal(d["pool"], e["pool"]), i
        assert torch.equal(v["next_token"], w["next_token"]) and torch.equal(count_d, count_e), i
        (e["pool"].sum() + 1).item()


@pytest.mark.parametrize("entry", ["decode", "prefill"])
def test_captured_gdr_replays(torch_cuda, entry):
    torch = torch_cuda
    b = Batch(torch, [3, 80, 1], seed=13)
    d, e = b.device(), b.device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.call(entry, b.device())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.call(entry, d)
    torch.cuda.synchronize()
    for i in range(4):
        graph.replay()
        b.call(entry, e)
        torch.cuda.synchronize()
        assert torch.equal(d["out"], e["out"]) and torch.equal(d["pool"], e["pool"]), i
        (e["pool"].sum() + 1).item()
