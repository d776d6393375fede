"""kda_ssm_decode and kda_ssm_prefill against the 64-bit token loop (bounds in ssm_reference.py)."""
import itertools

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gated_delta_rule_82_amd import kda  # noqa: E402
from tests.ssm_reference import Case  # noqa: E402

pytestmark = pytest.mark.gpu
DEVICE = "cuda:0"
CALLS = {"decode": kda.ssm_decode, "prefill": kda.ssm_prefill}


def call(case, t, entry, **kw):
    CALLS[entry](t["out"], t["xbc"], t["dt"], t["conv_w"], t["conv_b"], t["conv_win"], t["a_log"], t["dt_bias"],
                 t["d_skip"], t["cu_seqlens"], t["state_pool"], t["state_indices"], state_layout=case.layout, **kw)


def run(case, entry, **kw):
    t = case.tensors(DEVICE)
    call(case, t, entry, **kw)
    torch.cuda.synchronize()
    case.check(t, entry == "prefill")
    return t


SIZES = list(itertools.product((32, 64, 128), (32, 64, 128)))


@pytest.mark.parametrize("layout", ["k_first", "v_first"])
@pytest.mark.parametrize("state_bf16", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("dk,dv", SIZES)
def test_decode(dk, dv, bf16, state_bf16, layout):
    run(Case(dk + dv, [1, 3, 0, 2, 8], H=2, HV=6, dk=dk, dv=dv, bf16=bf16, state_bf16=state_bf16, layout=layout),
        "decode")


@pytest.mark.parametrize("lens,dk,dv,HV,layout", [([1] * 128, 128, 64, 64, "k_first"), ([0, 2] * 128, 64, 128, 32, "v_first"),
                                                  ([3, 0, 0, 1] * 32, 128, 128, 64, "k_first")])
def test_decode_of_a_full_batch(lens, dk, dv, HV, layout):
    """As many tokens as requests and workgroups enough for the launch of full batches, one token each or not."""
    run(Case(24, lens, H=1, HV=HV, dk=dk, dv=dv, layout=layout), "decode")


@pytest.mark.parametrize("layout,state_bf16,bf16", [("k_first", False, True), ("v_first", True, True),
                                                    ("v_first", False, False), ("k_first", True, False)])
@pytest.mark.parametrize("dk,dv", SIZES)
def test_prefill(dk, dv, layout, state_bf16, bf16):
    run(Case(dk * dv, [65, 0, 1, 30, 130, 64], H=2, HV=6, dk=dk, dv=dv, bf16=bf16, state_bf16=state_bf16,
             layout=layout), "prefill")


@pytest.mark.parametrize("entry", ["decode", "prefill"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("w_bf16,bias,skip", [(False, True, False), (True, False, True), (True, True, True)])
def test_convolution_forms(entry, K, w_bf16, bias, skip):
    """Taps, and requests shorter than the window."""
    run(Case(K, [1, 2, 3, 4, 5, 70], H=1, HV=3, dk=64, dv=32, K=K, w_bf16=w_bf16, bias=bias, skip=skip), entry)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191])
def test_prefill_lengths(n):
    run(Case(n, [n, 5, n + 1], H=1, HV=2, dk=64, dv=64, bf16=False), "prefill")


@pytest.mark.parametrize("H,HV", [(1, 1), (1, 7), (3, 3), (8, 8), (2, 16), (5, 15)])
@pytest.mark.parametrize("entry", ["decode", "prefill"])
def test_groups(entry, H, HV):
    run(Case(H * HV, [3, 1, 9], H=H, HV=HV, dk=32, dv=64), entry)


@pytest.mark.parametrize("lens", [[1500], [700, 0, 257, 1, 256, 512, 900], [2049, 3, 300]])
@pytest.mark.parametrize("bf16,state_bf16,layout,dk,dv", [(True, False, "k_first", 64, 128), (True, True, "v_first", 32, 32),
                                                          (False, False, "v_first", 128, 64)])
def test_split_requests(lens, bf16, state_bf16, layout, dk, dv):
    """Few heads, long requests: segments and their join."""
    run(Case(len(lens), lens, H=1, HV=2, dk=dk, dv=dv, bf16=bf16, state_bf16=state_bf16, layout=layout), "prefill")


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("H,HV,dk,dv,bf16,state_bf16,layout", [
    (2, 6, 64, 64, False, False, "v_first"), (4, 4, 32, 128, True, False, "k_first"),
    (3, 6, 128, 32, True, True, "v_first"), (2, 2, 128, 128, False, True, "k_first")])
def test_split_requests_forms(H, HV, dk, dv, bf16, state_bf16, layout, K):
    """Segments and their join with several groups, fewer taps, slots that are skipped and no skip connection."""
    run(Case(K + H, [1100, 40, 0, 333, 65], H=H, HV=HV, dk=dk, dv=dv, K=K, bf16=bf16, state_bf16=state_bf16,
             w_bf16=bf16, layout=layout, skip=False, bias=K != 3, slots=[3, -1, 0, 6, 9]), "prefill")


@pytest.mark.parametrize("entry", ["decode", "prefill"])
@pytest.mark.parametrize("decay", [1e-4, 30.0, 300.0])
def test_decays(entry, decay):
    """States that hardly decay, and that vanish within a token; in chunks, near tokens behind a large sum of decays."""
    run(Case(3, [130, 7], H=1, HV=4, dk=64, dv=64, bf16=False, decay=decay), entry)


def test_one_token_behind_large_decays():
    """The sums of a chunk's decays run to thousands, and the last tokens' own decays are small."""
    case = Case(4, [64, 64], H=1, HV=2, dk=32, dv=32, bf16=False)
    case.dt[:40] = 60.0
    case.dt[64:100] = 200.0
    case.dt[40:64] = case.dt[100:] = -3.0
    run(case, "prefill")


@pytest.mark.parametrize("entry", ["decode", "prefill"])
def test_skipped_and_clamped(entry):
    """Negative and too large slots are skipped; other slots are left."""
    run(Case(5, [3, 70, 2, 1], H=1, HV=2, dk=32, dv=64, slots=[2, -1, 6, 0]), entry)


@pytest.mark.parametrize("entry", ["decode", "prefill"])
def test_bad_offsets_stay_inside(entry):
    """cu_seqlens outside [0, T] or falling: no access outside the tensors, and requests that are right are right."""
    case = Case(6, [4, 5, 6], H=1, HV=2, dk=32, dv=32, slots=[0, 1, 2])
    t = case.tensors(DEVICE)
    t["cu_seqlens"] = torch.tensor([-3, 4, 2, 1000], dtype=torch.int32, device=DEVICE)
    call(case, t, entry)
    torch.cuda.synchronize()
    o, mag, *_ = case.walk(0)       # rows 0 .. 3; rows 2 and 3 are the last request's (2 .. 14) too
    o, mag = o[:2], mag[:2]
    off = np.abs(t["out"][0, :2].float().cpu().numpy() - o) - 2.0 ** -8 * np.abs(o) - 2.0 ** -11 * mag
    assert off.max() <= 0, off.max()


@pytest.mark.parametrize("entry", ["decode", "prefill"])
def test_nothing_to_do(entry):
    case = Case(7, [0, 0], H=1, HV=2, dk=32, dv=32)
    run(case, entry)
    t = Case(7, [3], H=1, HV=2, dk=32, dv=32).tensors(DEVICE)
    before = {n: x.clone() for n, x in t.items()}
    t["cu_seqlens"], t["state_indices"] = t["cu_seqlens"][:1].clone(), t["state_indices"][:0].clone()
    call(case, t, entry)
    torch.cuda.synchronize()
    assert all(torch.equal(t[n], before[n]) for n in ("out", "state_pool", "conv_win"))


def test_prompt_then_tokens_equals_one_prompt():
    """A prompt and three single tokens leave what one prompt of all leaves, each within its own bounds."""
    whole = Case(8, [90, 40], H=2, HV=4, dk=64, dv=64, bf16=False, slots=[1, 3])
    t = run(whole, "prefill")
    s = whole.tensors(DEVICE)
    cut = {0: 87, 1: 37}
    starts = [int(c) for c in whole.cu]
    for part in range(4):
        rows = [list(range(starts[b], starts[b] + cut[b])) if part == 0 else [starts[b] + cut[b] + part - 1]
                for b in range(2)]
        flat = torch.tensor(sum(rows, []), device=DEVICE)
        step = dict(s, xbc=s["xbc"][:, flat].contiguous(), dt=s["dt"][:, flat].contiguous(),
                    out=torch.empty_like(s["out"][:, flat]),
                    cu_seqlens=torch.tensor([0, len(rows[0]), len(flat)], dtype=torch.int32, device=DEVICE))
        call(whole, step, "prefill" if part == 0 else "decode")
        s["out"][:, flat] = step["out"]
    torch.cuda.synchronize()
    whole.check(s, True)
    assert torch.equal(s["conv_win"], t["conv_win"])


def test_more_requests_than_xcds_and_odd_heads():
    run(Case(9, [66] * 11, H=1, HV=5, dk=32, dv=32), "prefill")


@pytest.mark.parametrize("entry", ["decode", "prefill"])
def test_on_another_stream(entry):
    case = Case(10, [5, 200], H=1, HV=4, dk=64, dv=64)
    t = case.tensors(DEVICE)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    kw = {}
    if entry == "prefill":
        kw["workspace"] = torch.empty(kda.ssm_prefill_workspace(case.T, case.B, 1, 4, 64, 64, 4), device=DEVICE)
        torch.cuda.synchronize()
    call(case, t, entry, stream=stream.cuda_stream, **kw)
    stream.synchronize()
    case.check(t, entry == "prefill")


@pytest.mark.parametrize("entry,lens", [("decode", [1, 2, 1]), ("prefill", [100, 3]), ("prefill", [800, 30])])
def test_captured(entry, lens):
    """A captured call replays on the state it finds; eager work in between."""
    case = Case(11, lens, H=1, HV=2, dk=64, dv=64)
    t, eager = case.tensors(DEVICE), case.tensors(DEVICE)
    saved = {n: t[n].clone() for n in ("state_pool", "conv_win")}
    call(case, t, entry)        # warm
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(case, t, entry)
    for n, x in saved.items():
        t[n].copy_(x)
    for replay in range(3):
        graph.replay()
        call(case, eager, entry)
        torch.cuda.synchronize()
        for n in ("out", "state_pool", "conv_win"):
            assert torch.equal(t[n], eager[n]), (replay, n)


def test_two_calls_at_once():
    """Two streams, each with tensors and a workspace of its own."""
    cases = [Case(20 + i, [300, 40], H=1, HV=4, dk=64, dv=64) for i in range(2)]
    ts = [c.tensors(DEVICE) for c in cases]
    ws = [torch.empty(kda.ssm_prefill_workspace(c.T, c.B, 1, 4, 64, 64, 4), device=DEVICE) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for c, t, w, s in zip(cases, ts, ws, streams):
        call(c, t, "prefill", workspace=w, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for c, t in zip(cases, ts):
        c.check(t, True)


@pytest.mark.parametrize("entry", ["decode", "prefill"])
def test_a_neighbour_that_is_not_finite(entry):
    """Infinities and NaN in one request's tokens, state and window reach no other request."""
    case = Case(12, [30, 33, 40], H=1, HV=2, dk=32, dv=32, bf16=False, slots=[0, 1, 2])
    t = case.tensors(DEVICE)
    t["xbc"][0, 30:63] = float("inf")
    t["xbc"][0, 40:45] = float("nan")
    t["state_pool"][1] = float("nan")
    t["conv_win"][1] = float("-inf")
    call(case, t, entry)
    torch.cuda.synchronize()
    for b in (0, 2):
        o, mag, S, M, w = case.walk(b)
        rows = slice(case.cu[b], case.cu[b + 1])
        assert (np.abs(t["out"][0, rows].cpu().numpy() - o) <= 2.0 ** -12 * mag).all()
        assert (np.abs(t["state_pool"][b].cpu().numpy() - S) <= 2.0 ** -12 * M).all()


def test_large_values_stay_finite():
    """Values near the ends of fp32 that the scan itself keeps finite."""
    case = Case(13, [70], H=1, HV=2, dk=32, dv=32, bf16=False, slots=[0], bias=False)
    x = case.HV * case.dv
    case.xbc[:, :x] *= np.float32(1e30)
    case.conv_win[:, :, :x] *= np.float32(1e30)
    case.xbc[:, x:] *= np.float32(1e3)
    case.pool *= np.float32(1e30)
    run(case, "prefill")
    run(case, "decode")


@pytest.mark.parametrize("entry", ["decode", "prefill"])
@pytest.mark.parametrize("at", [5, 20, 40])
def test_keys_of_later_tokens_stay_out(entry, at):
    """C of a token times B of a later one leaves fp32; the scan never forms that product."""
    case = Case(21, [50], H=1, HV=4, dk=32, dv=32, K=2, bf16=False, bias=False)
    keys, read = case.HV * case.dv, case.HV * case.dv + case.dk
    case.conv_w[:, keys:] = np.array([[0.0], [1.0]], dtype=np.float32)
    case.xbc[at, keys:read] = 1e25
    case.xbc[:at, read:] = 1e25
    run(case, entry)


@pytest.mark.parametrize("entry", ["decode", "prefill"])
def test_decays_of_nothing_left(entry):
    """exp(a_log) beyond fp32, and steps from none to large: factors of zero and one, nothing undefined."""
    case = Case(14, [40, 3], H=1, HV=4, dk=32, dv=32, bf16=False)
    case.a_log[:] = (100.0, -100.0, 2.0, 50.0)
    case.dt[5] = 1e4
    case.dt[9] = -1e4
    case.dt[9, 0] = case.dt[9, 3] = 0.0       # (infinity times no step has no value)
    run(case, entry)


@pytest.mark.parametrize("entry,lens", [("decode", [3, 40]), ("prefill", [3, 40]), ("prefill", [1500, 40])])
@pytest.mark.parametrize("which", ["a_log", "dt_bias"])
def test_a_head_without_a_decay(entry, lens, which):
    """NaN in a head's parameters is NaN in all its outputs and its state, and reaches no other head."""
    case = Case(22, lens, H=1, HV=4, dk=32, dv=64, bf16=False, slots=[0, 1], extra_slots=0)
    t = case.tensors(DEVICE)
    t[which][2] = float("nan")
    call(case, t, entry)
    torch.cuda.synchronize()
    assert torch.isnan(t["out"][0, :, 2]).all() and torch.isnan(t["state_pool"][:, 2]).all()
    keep = [0, 1, 3]
    for b in range(2):
        o, mag, S, M, w = case.walk(b)
        rows = slice(case.cu[b], case.cu[b + 1])
        n = np.arange(1, lens[b] + 1)[:, None, None]
        tol = (32 * (n + 1) * 2.0 ** -24 + 2 * 2.0 ** -20.4) * mag
        assert (np.abs(t["out"][0, rows].cpu().numpy() - o) <= tol)[:, keep].all()
        assert (np.abs(t["state_pool"][b].cpu().numpy() - S) <= (32 * lens[b] * 2.0 ** -24 + 2.0 ** -20.4) * M)[keep].all()
        assert np.array_equal(t["conv_win"][b].cpu().numpy(), w.astype(np.float32))


@pytest.mark.parametrize("entry", ["decode", "prefill"])
@pytest.mark.parametrize("n", [50, 1500])
@pytest.mark.parametrize("K", [2, 4])
def test_taps_of_no_token(entry, n, K):
    """A tap that would leave fp32 for a token behind the last meets nothing: there is no such token."""
    case = Case(23, [n, 3], H=1, HV=2, dk=32, dv=32, K=K, bf16=False)
    x = case.HV * case.dv
    case.conv_w[K - 2, :x] = 1e30
    case.xbc[:, :x] = 0
    case.conv_win[:, :, :x] = 0
    case.xbc[n - 1, :x] = 1e10
    run(case, entry)


@pytest.mark.parametrize("dv", [32, 64, 128])
def test_captured_fp32_of_128_keys(dv):
    """The operands that take the most LDS."""
    case = Case(15, [700, 33], H=1, HV=2, dk=128, dv=dv, bf16=False)
    t, eager = case.tensors(DEVICE), case.tensors(DEVICE)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):       # the first call of this form in the process, if run alone
        call(case, t, "prefill")
    for replay in range(3):
        graph.replay()
        call(case, eager, "prefill")
        torch.cuda.synchronize()
        if replay == 0:
            case.check(eager, True)
        for n in ("out", "state_pool", "conv_win"):
            assert torch.equal(t[n], eager[n]), (replay, n)


def test_rows_behind_the_last_request():
    """Rows of out behind cu_seqlens' end are left."""
    case = Case(16, [3, 50, 20], H=1, HV=2, dk=32, dv=32)
    for entry in CALLS:
        t = case.tensors(DEVICE)
        t["cu_seqlens"] = t["cu_seqlens"][:3].clone()
        t["state_indices"] = t["state_indices"][:2].clone()
        call(case, t, entry)
        torch.cuda.synchronize()
        assert (t["out"][0, 53:] == 7).all()
        o, mag, *_ = case.walk(1)
        off = np.abs(t["out"][0, 3:53].float().cpu().numpy() - o) - 2.0 ** -8 * np.abs(o) - 2.0 ** -11 * mag
        assert off.max() <= 0


def test_same_results_again():
    """Nothing depends on the order in which workgroups run."""
    case = Case(17, [500, 900, 10], H=2, HV=4, dk=64, dv=64)
    first = None
    for _ in range(4):
        t = case.tensors(DEVICE)
        call(case, t, "prefill")
        torch.cuda.synchronize()
        got = [t[n] for n in ("out", "state_pool", "conv_win")]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_workspace_bounds():
    """The workspace is enough and nothing outside it is written: guards on both sides stay."""
    for lens, H, HV, dk, dv in (([1000, 1, 0, 77], 1, 2, 32, 32), ([64] * 9, 3, 6, 64, 128), ([2000], 1, 1, 128, 64)):
        case = Case(18, lens, H=H, HV=HV, dk=dk, dv=dv)
        t = case.tensors(DEVICE)
        n = kda.ssm_prefill_workspace(case.T, case.B, H, HV, dk, dv, case.K)
        buf = torch.full((n + 2048,), 3.25, device=DEVICE)
        call(case, t, "prefill", workspace=buf[1024:1024 + n])
        torch.cuda.synchronize()
        case.check(t, True)
        assert (buf[:1024] == 3.25).all() and (buf[1024 + n:] == 3.25).all()


@pytest.mark.parametrize("lens", [[300, 200, 210, 190, 130], [300, 200, 210, 190, 130, 1]])
def test_workspace_where_splitting_ends(lens):
    """The largest batch of 96 heads that is split, and one request more, between guards."""
    case = Case(25, lens, H=1, HV=96, dk=32, dv=32)
    t = case.tensors(DEVICE)
    n = kda.ssm_prefill_workspace(case.T, case.B, 1, 96, 32, 32, 4)
    buf = torch.full((n + 2048,), 3.25, device=DEVICE)
    call(case, t, "prefill", workspace=buf[1024:1024 + n])
    torch.cuda.synchronize()
    case.check(t, True)
    assert (buf[:1024] == 3.25).all() and (buf[1024 + n:] == 3.25).all()


@pytest.mark.parametrize("entry", ["decode", "prefill"])
@pytest.mark.parametrize("lens", [[2, 1, 3], [700, 40, 1]])
def test_offsets_beyond_32_bits(entry, lens):
    """Tokens behind a skipped request of 2^31 values, in slots behind as many of the pool."""
    case = Case(26, lens, H=1, HV=64, dk=32, dv=128)
    t = case.tensors(DEVICE)
    rows, slots = 2 ** 31 // (case.HV * case.dv) + 1, 2 ** 31 // (case.HV * case.dk * case.dv) + 1
    big = dict(t)
    for n in ("out", "xbc", "dt"):
        big[n] = torch.empty((1, rows + case.T) + t[n].shape[2:], dtype=t[n].dtype, device=DEVICE)
        big[n][:, rows:] = t[n]
    for n in ("state_pool", "conv_win"):
        big[n] = torch.empty((slots + case.N,) + t[n].shape[1:], dtype=t[n].dtype, device=DEVICE)
        big[n][slots:] = t[n]
    skipped = torch.tensor([-1], dtype=torch.int32, device=DEVICE)
    big["state_indices"] = torch.cat([skipped, t["state_indices"] + slots])
    big["cu_seqlens"] = torch.cat([torch.zeros_like(skipped), t["cu_seqlens"] + rows])
    call(case, big, entry)
    torch.cuda.synchronize()
    assert not big["out"][0, :rows].any()
    case.check(dict(t, out=big["out"][:, rows:], state_pool=big["state_pool"][slots:], conv_win=big["conv_win"][slots:]),
               entry == "prefill")


def test_refusals():
    case = Case(19, [5], H=1, HV=2, dk=32, dv=32)
    t = case.tensors(DEVICE)
    for n, x in (("xbc", t["xbc"][..., :-1].contiguous()), ("dt", t["dt"][:, :4].contiguous()),
                 ("conv_win", t["conv_win"][:, :2].contiguous()), ("state_pool", t["state_pool"].half()),
                 ("out", t["out"].float()), ("conv_b", t["conv_b"].bfloat16())):
        for entry in CALLS:
            with pytest.raises((kda.KdaError, ValueError)):
                call(case, dict(t, **{n: x}), entry)
    for entry in CALLS:
        with pytest.raises(ValueError, match="contiguous"):
            call(case, dict(t, xbc=torch.cat([t["xbc"]] * 2, -1)[..., ::2]), entry)
    with pytest.raises(ValueError, match="workspace"):
        call(case, t, "prefill", stream=torch.cuda.current_stream().cuda_stream)
    with pytest.raises(kda.KdaError):
        call(case, t, "prefill", workspace=torch.empty(10, device=DEVICE))
