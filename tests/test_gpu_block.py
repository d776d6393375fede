"""Operators as a block uses them together: residual and norm, the recurrence, the gated norm; for a prompt and then
token by token, each stage against 64 bits on what the stage before it left, and the whole captured and replayed."""
import importlib.util

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gated_delta_rule_82_amd import kda  # noqa: E402
from tests.ssm_reference import BF16, Case, sigmoid, unit  # noqa: E402
from tests.test_gpu_norm import UNITS, check, residual_reference, wide  # noqa: E402

pytestmark = pytest.mark.gpu
DEVICE = "cuda:0"
EPS_NORM = 1e-5


class Block:
    """Residual, norm, projection (torch's), scan, gated norm over groups."""

    def __init__(self, lens, seed=0, H=2, HV=4, dk=64, dv=64, D=320):
        self.case = Case(seed, lens, H=H, HV=HV, dk=dk, dv=dv, bf16=True)
        self.t = self.case.tensors(DEVICE)
        gen = torch.Generator(device=DEVICE).manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=gen, device=DEVICE)
        T, C = self.case.T, self.case.C
        self.groups, self.inner = H, HV * dv // H
        self.hidden, self.block_out = (3 * normal(T, D)).bfloat16(), normal(T, D).bfloat16()
        self.w_norm, self.scale, self.w_gate = normal(D), normal(D), normal(H, self.inner)
        self.w_in = (normal(D, C + HV * dv) / D ** 0.5).bfloat16()
        self.w_dt = normal(D, HV) / D ** 0.5

    def run(self, t, rows, call, cu, module=kda):
        """The stages on the rows given; returns what each left."""
        hidden, block_out = self.hidden[rows].contiguous(), self.block_out[rows].contiguous()
        normed = torch.empty_like(block_out)
        module.norm_residual(hidden, normed, hidden, block_out, self.w_norm, scale=self.scale, eps=EPS_NORM)
        both = normed.float() @ self.w_in.float()
        xbc = both[:, :self.case.C].bfloat16().unsqueeze(0).contiguous()
        z = both[:, self.case.C:].bfloat16().reshape(len(rows), self.groups, self.inner).contiguous()
        dt = (normed.float() @ self.w_dt).unsqueeze(0).contiguous()
        out = torch.empty(1, len(rows), self.case.HV, self.case.dv, dtype=torch.bfloat16, device=DEVICE)
        getattr(module, call)(out, xbc, dt, t["conv_w"], t["conv_b"], t["conv_win"], t["a_log"], t["dt_bias"],
                              t["d_skip"], cu, t["state_pool"], t["state_indices"])
        gated = torch.empty_like(z)
        module.norm_gate(gated, out.view(z.shape), z, self.w_gate, activation="silu", gate_first=True, eps=EPS_NORM)
        return dict(hidden=hidden, normed=normed, xbc=xbc, dt=dt, z=z, out=out, gated=gated)

    def rows(self, parts):
        flat = torch.tensor(sum(parts, []), device=DEVICE)
        cu = torch.tensor(np.concatenate([[0], np.cumsum([len(p) for p in parts])]), dtype=torch.int32, device=DEVICE)
        return flat, cu


@pytest.mark.parametrize("lens,cut", [([40, 75], [38, 72]), ([300, 7, 64], [297, 5, 60])])
def test_prompt_and_tokens(lens, cut):
    b = Block(lens, seed=len(lens))
    case, t = b.case, b.t
    starts = [int(c) for c in case.cu[:-1]]
    xbc, dt, out = t["xbc"].clone(), t["dt"].clone(), t["out"].clone()
    longest = max(n - c for n, c in zip(lens, cut))
    for step in range(-1, longest):
        if step < 0:
            parts = [list(range(s, s + c)) for s, c in zip(starts, cut)]
        else:
            parts = [[s + c + step] if c + step < n else [] for s, c, n in zip(starts, cut, lens)]
        rows, cu = b.rows(parts)
        got = b.run(t, rows, "ssm_prefill" if step < 0 else "ssm_decode", cu)
        torch.cuda.synchronize()
        want_h, want_n, mag = residual_reference(b.hidden[rows], b.block_out[rows], b.w_norm, None, b.scale, EPS_NORM)
        check(got["hidden"], want_h, True, extra=UNITS * mag)
        r = 1.0 / np.sqrt((want_h ** 2).mean(-1, keepdims=True) + EPS_NORM)
        check(got["normed"], want_n, True, extra=2 * UNITS * mag * r * np.abs(wide(b.w_norm)))
        z = wide(got["z"])
        u = wide(got["out"]).reshape(z.shape) * z * sigmoid(z)
        check(got["gated"], unit(u, EPS_NORM) * wide(b.w_gate), True)
        xbc[:, rows], dt[:, rows], out[:, rows] = got["xbc"], got["dt"], got["out"]
    # the scan of all tokens, on what the projections gave
    case.xbc, case.dt = xbc[0].float().cpu().numpy(), dt[0].cpu().numpy()
    case.check(dict(t, out=out), True)


def test_prompt_and_tokens_of_split_requests():
    """A prompt long enough to run in segments, beside a short one and then token by token."""
    test_prompt_and_tokens([1200, 40], [1197, 38])


def test_captured_step():
    """A block's token step, captured and replayed, is the eager one, replay after replay."""
    b = Block([1, 1, 1], seed=5)
    rows, cu = b.rows([[0], [1], [2]])
    state = ("state_pool", "conv_win")
    eager = {n: (x.clone() if n in state else x) for n, x in b.t.items()}
    warm = {n: (x.clone() if n in state else x) for n, x in b.t.items()}
    b.run(warm, rows, "ssm_decode", cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.run(b.t, rows, "ssm_decode", cu)
    for replay in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = b.run(eager, rows, "ssm_decode", cu)
        torch.cuda.synchronize()
        for n in ("hidden", "normed", "out", "gated"):
            assert torch.equal(got[n], want[n]), (replay, n)
        for n in state:
            assert torch.equal(b.t[n], eager[n]), (replay, n)


def test_gated_norm_behind_the_delta_rule():
    """kda_decode's output through the gated output norm, one norm per head."""
    from tests.test_gpu_gdr import Batch
    batch = Batch(torch, [1, 1, 4], channel=True, seed=4)
    d = batch.device()
    kda.decode(*batch.args(d), **batch.mode)
    out = d["out"]
    gen = torch.Generator(device=DEVICE).manual_seed(0)
    gate = torch.randn(out.shape, generator=gen, device=DEVICE).to(out.dtype)
    w = torch.randn(out.shape[-1], generator=gen, device=DEVICE)
    want = unit(wide(out), EPS_NORM) * wide(w) * sigmoid(wide(gate))
    got = torch.empty_like(out)
    kda.norm_gate(got, out, gate, w, eps=EPS_NORM)
    torch.cuda.synchronize()
    check(got, want, out.dtype == torch.bfloat16)


@pytest.mark.parametrize("call", ["ssm_decode", "ssm_prefill"])
def test_call_path_through_ctypes(tmp_path, call):
    """Without its extension the binding gives the same, optional tensors left out or not."""
    spec = importlib.util.spec_from_file_location("kda_copy", kda.__file__)
    copy = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(copy)
    copy.BINDING_PATH = str(tmp_path / "_kda_binding.so")
    copy.library()
    got = []
    for module in (kda, copy):
        b = Block([9, 40], seed=6)
        b.t["d_skip"] = b.t["conv_b"] = None
        rows, cu = b.rows([list(range(9)), list(range(9, 49))])
        got.append((b.run(b.t, rows, call, cu, module), b.t))
        torch.cuda.synchronize()
    for n, x in got[0][0].items():
        assert torch.equal(x, got[1][0][n]), n
    for n in ("state_pool", "conv_win"):
        assert torch.equal(got[0][1][n], got[1][1][n]), n
    assert copy._native is copy._described_call
