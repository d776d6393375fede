"""The call path through ctypes gives what the one through the extension gives."""
import importlib.util

import numpy as np
import pytest

from tests.test_gpu_gdr import Batch
from tests.test_gpu_speculative import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


@pytest.fixture(scope="module")
def copy(torch_cuda, tmp_path_factory):
    from gated_delta_rule_82_amd import kda
    spec = importlib.util.spec_from_file_location("kda_copy", kda.__file__)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.BINDING_PATH = str(tmp_path_factory.mktemp("none") / "_kda_binding.so")
    module.library()
    return module


@pytest.mark.parametrize("entry", ["gdr_decode", "gdr_prefill", "decode_window", "decode", "prefill"])
def test_same_results(torch_cuda, copy, entry):
    torch = torch_cuda
    from gated_delta_rule_82_amd import kda
    channel = entry in ("decode", "prefill")
    b = Batch(torch, [3, 40], replay=[(0, 2), (1, 3)], channel=channel, seed=2)
    d, e = b.device(), b.device()
    for module, x in ((kda, d), (copy, e)):
        getattr(module, entry)(*b.args(x), *(x["rep"] if entry == "decode_window" else []), **b.mode)
    torch.cuda.synchronize()
    assert torch.equal(d["out"], e["out"]) and torch.equal(d["pool"], e["pool"])
    assert copy._native is copy._described_call


@pytest.mark.parametrize("draft", [True, False])
def test_same_verdicts(torch_cuda, copy, draft):
    torch = torch_cuda
    from gated_delta_rule_82_amd import kda
    c = Case([4, 2], 501, draft=draft, seed=3)
    got = []
    for module in (kda, copy):
        x = c.device(torch)
        module.verify(x["n_commit"], x["next_token"], x["target"], x["draft"], x["tokens"], x["u_accept"],
                      x["u_sample"], x["cu"])
        got.append((x["n_commit"].cpu().numpy(), x["next_token"].cpu().numpy()))
    for a, w in zip(*got):
        np.testing.assert_array_equal(a, w)


def test_same_conv(torch_cuda, copy):
    torch = torch_cuda
    from gated_delta_rule_82_amd import kda
    b = Batch(torch, [3, 2], channel=True, seed=4)
    g = torch.Generator(device="cuda").manual_seed(1)
    outs = []
    taps = [torch.randn((4, n * 128), generator=g, device="cuda") for n in (2, 2, 4)]
    wins = [torch.randn((b.N, 3, n * 128), generator=g, device="cuda") for n in (2, 2, 4)]
    for module in (kda, copy):
        d = b.device()
        w = [x.clone() for x in wins]
        qc, kc = (torch.empty_like(d["q"], dtype=torch.float32) for _ in range(2))
        module.decode_conv(d["out"], d["q"], d["k"], d["v"], *taps, *w, qc, kc, d["gate"], d["beta"], d["a_log"],
                           d["bias"], d["cu"], d["pool"], d["idx"], **b.mode)
        outs.append([d["out"], d["pool"], qc, kc, *w])
    torch.cuda.synchronize()
    for x, y in zip(*outs):
        assert torch.equal(x, y)


def test_same_refusals(torch_cuda, copy):
    torch = torch_cuda
    b = Batch(torch, [2, 1])
    d = b.device()
    for name, value, error in (("q", d["q"].half(), ValueError), ("v", d["v"].cpu(), ValueError),
                               ("beta", None, TypeError), ("pool", d["pool"][:, :3], ValueError)):
        with pytest.raises(error):
            copy.gdr_decode(*b.args(dict(d, **{name: value})), **b.mode)
    with pytest.raises(copy.KdaError):
        copy.gdr_decode(*b.args(dict(d, bias=d["bias"][:3].clone())), **b.mode)
