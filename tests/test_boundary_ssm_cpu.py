"""CPU tests of the argument checks of kda_ssm_decode, kda_ssm_prefill, kda_norm_residual and kda_norm_gate:
every malformed call is refused before any device work.  The data pointers are fake and never dereferenced."""
import os
import re

import pytest

from gated_delta_rule_82_amd import kda

pytestmark = pytest.mark.skipif(not os.path.exists(kda.LIB_PATH),
                                reason="libkda.so not built (run the build first)")

F32, BF16, I32 = kda.KDA_F32, kda.KDA_BF16, kda.KDA_I32


def fake(i, dtype, shape):
    return kda.raw_tensor(0x100000 * (i + 1), dtype, shape)


def changed(d, name, dtype=None, shape=None, data=None):
    t = d[name]
    return dict(d, **{name: kda.raw_tensor(t.data if data is None else data, t.dtype if dtype is None else dtype,
                                           tuple(t.shape[:t.ndim]) if shape is None else shape)})


def ssm_descriptors(B=2, T=5, H=2, HV=4, DK=64, DV=32, N=8, K=4, prefill=True, C=None):
    C = HV * DV + 2 * H * DK if C is None else C
    shapes = {
        "out": (BF16, (1, T, HV, DV)), "xbc": (BF16, (1, T, C)), "dt": (F32, (1, T, HV)), "conv_w": (F32, (K, C)),
        "conv_b": (F32, (C,)), "conv_win": (F32, (N, K - 1, C)), "a_log": (F32, (HV,)), "dt_bias": (F32, (HV,)),
        "d_skip": (F32, (HV,)), "cu_seqlens": (I32, (B + 1,)), "state_pool": (F32, (N, HV, DK, DV)),
        "state_indices": (I32, (B,)),
    }
    if prefill:
        shapes["workspace"] = (F32, (kda.ssm_prefill_workspace(T, B, H, HV, DK, DV, K),))
    return {n: fake(i, *s) for i, (n, s) in enumerate(shapes.items())}


def ssm(d, layout=kda.KDA_STATE_K_FIRST):
    return kda.call_raw_ssm([d[n] for n in kda.SSM_NAMES if n in d], layout)


@pytest.mark.parametrize("prefill", [False, True])
def test_ssm_refusals(prefill):
    d = ssm_descriptors(prefill=prefill)
    for n in d:
        if n not in ("conv_b", "d_skip"):
            assert ssm(dict(d, **{n: None})) == kda.KDA_ERR_NULL, n
        assert ssm(changed(d, n, data=0)) == kda.KDA_ERR_NULL, n
        assert ssm(changed(d, n, data=d[n].data + 4)) == kda.KDA_ERR_UNSUPPORTED, n
        assert ssm(changed(d, n, dtype=17)) == kda.KDA_ERR_DTYPE, n
        assert ssm(changed(d, n, shape=tuple(d[n].shape[:d[n].ndim - 1]) or (1, 1))) == kda.KDA_ERR_SHAPE, n
        for axis in range(d[n].ndim):
            shape = list(d[n].shape[:d[n].ndim])
            shape[axis] = -1
            assert ssm(changed(d, n, shape=shape)) == kda.KDA_ERR_SHAPE, n
    for n, dtype in (("out", F32), ("xbc", F32), ("dt", BF16), ("conv_w", BF16), ("conv_b", BF16), ("conv_win", BF16),
                     ("a_log", BF16), ("dt_bias", I32), ("d_skip", BF16), ("cu_seqlens", F32), ("state_pool", I32),
                     ("state_indices", F32)):
        assert ssm(changed(d, n, dtype=dtype)) == kda.KDA_ERR_DTYPE, n
    for n, shape in (("out", (1, 5, 3, 32)), ("out", (1, 4, 4, 32)), ("out", (2, 5, 4, 32)), ("xbc", (1, 4, 384)),
                     ("xbc", (2, 5, 384)), ("dt", (1, 4, 4)), ("dt", (1, 5, 3)), ("conv_w", (4, 383)),
                     ("conv_b", (383,)), ("conv_win", (7, 3, 384)), ("conv_win", (8, 2, 384)),
                     ("conv_win", (8, 3, 383)), ("a_log", (3,)), ("dt_bias", (5,)), ("d_skip", (1,)),
                     ("cu_seqlens", (2,)), ("state_pool", (8, 3, 64, 32)), ("state_pool", (8, 4, 64, 64)),
                     ("state_indices", (3,))):
        assert ssm(changed(d, n, shape=shape)) == kda.KDA_ERR_SHAPE, (n, shape)
    assert ssm(d, 2) == kda.KDA_ERR_MODE
    assert ssm(d, kda.KDA_STATE_V_FIRST) == kda.KDA_ERR_SHAPE
    # channels that are no whole number of groups, no group, groups that do not divide the heads
    for C in (4 * 32 + 2 * 64 - 32, 4 * 32, 4 * 32 + 64, 4 * 32 + 6 * 64, 100):
        assert ssm(ssm_descriptors(C=C, prefill=prefill)) == kda.KDA_ERR_SHAPE, C


@pytest.mark.parametrize("prefill", [False, True])
def test_ssm_sizes(prefill):
    for kw in (dict(DK=16), dict(DV=16), dict(DK=256), dict(DV=96), dict(K=1), dict(K=5), dict(T=2 ** 31 - 64),
               dict(N=2 ** 31 - 64), dict(B=2 ** 31 - 64), dict(B=2 ** 20), dict(B=2 ** 23, HV=1, H=1),
               dict(HV=2 ** 19, H=1)):
        assert ssm(ssm_descriptors(prefill=prefill, **kw)) == kda.KDA_ERR_UNSUPPORTED, kw
    # an empty batch is no error
    for kw in (dict(T=0), dict(B=0)):
        assert ssm(ssm_descriptors(prefill=prefill, **kw)) == kda.KDA_OK, kw


def test_ssm_workspace():
    d = ssm_descriptors()
    n = d["workspace"].shape[0]
    assert ssm(changed(d, "workspace", shape=(n - 1,))) == kda.KDA_ERR_SHAPE
    # the binding's formula is the header's
    header = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kda.h")).read()
    body = re.search(r"#define KDA_SSM_WORKSPACE\(([^)]*)\)(.*?)\n\n", header, re.S)
    text = re.sub(r"\(int64_t\)", "", body.group(2).replace("\\\n", " "))
    text = re.sub(r"KDA_SSM_CHUNK", str(kda.KDA_SSM_CHUNK), re.sub(r"KDA_SSM_SPLIT", str(kda.KDA_SSM_SPLIT), text))
    for sizes in ((5, 2, 2, 4, 64, 32, 4), (16384, 1, 1, 64, 128, 64, 4), (12345, 77, 8, 96, 128, 128, 2)):
        names = dict(zip([x.strip() for x in body.group(1).split(",")], sizes))
        assert eval(text.replace("/", "//"), {}, names) == kda.ssm_prefill_workspace(*sizes)
    for name in ("KDA_SSM_CHUNK", "KDA_SSM_SPLIT"):
        assert int(re.search(rf"#define {name} (\d+)", header).group(1)) == getattr(kda, name)


def test_ssm_workspace_is_bounded():
    """States of split requests: 63 MiB at most and no more than the tokens need; no smaller batch needs more."""
    def rest(T, B, H, HV, dk, dv, K):
        return (T // 32 + B) * (H * (96 * dk + 1024) + 160 * HV) + B * (K - 1) * (HV * dv + 2 * H * dk) + B * HV
    for sizes in ((256 * 700, 256, 8, 96, 128, 128, 4), (256, 256, 1, 64, 128, 64, 4), (16384, 1, 1, 32, 128, 64, 4),
                  (10 ** 6, 3, 1, 64, 128, 128, 2)):
        assert (kda.ssm_prefill_workspace(*sizes) - rest(*sizes)) * 4 <= (63 << 20) + 4 * 2 ** 12, sizes
    assert kda.ssm_prefill_workspace(117, 1, 1, 32, 128, 64, 4) * 4 < 4 << 20
    most = (5000, 9, 4, 16, 128, 128, 4)
    largest = kda.ssm_prefill_workspace(*most)
    for T in (0, 1, 63, 64, 1000, 4999):
        for B in (1, 2, 5, 9):
            for HV in (4, 8, 16):
                for d in (32, 64, 128):
                    assert kda.ssm_prefill_workspace(T, B, 4, HV, d, d, 3) <= largest


def residual_descriptors(rows=(3, 5), D=64, scale=None):
    shapes = {"hidden_out": (F32, (*rows, D)), "normed": (BF16, (*rows, D)), "hidden": (F32, (*rows, D)),
              "block_out": (BF16, (*rows, D)), "weight": (F32, (D,)), "post_weight": (F32, (D,)),
              "scale": (F32, (D if scale is None else scale,))}
    return {n: fake(i, *s) for i, (n, s) in enumerate(shapes.items())}


def residual(d, eps=0.0):
    return kda.call_raw_norm_residual(list(d.values()), eps)


def test_norm_residual_refusals():
    d = residual_descriptors()
    for n in d:
        if n not in ("post_weight", "scale"):
            assert residual(dict(d, **{n: None})) == kda.KDA_ERR_NULL, n
        assert residual(changed(d, n, data=0)) == kda.KDA_ERR_NULL, n
        assert residual(changed(d, n, dtype=I32)) == kda.KDA_ERR_DTYPE, n
        assert residual(changed(d, n, data=d[n].data + 2)) == kda.KDA_ERR_UNSUPPORTED, n
    for n in ("hidden_out", "hidden"):
        assert residual(changed(d, n, dtype=BF16)) == kda.KDA_ERR_DTYPE, n
    for n in ("normed", "block_out"):
        assert residual(changed(d, n, dtype=F32)) == kda.KDA_ERR_DTYPE, n
    for n in ("hidden_out", "normed", "hidden", "block_out"):
        for shape in ((3, 4, 64), (15, 64), (3, 5, 63), (3, -1, 64)):
            assert residual(changed(d, n, shape=shape)) == kda.KDA_ERR_SHAPE, (n, shape)
        assert residual(changed(d, n, data=d[n].data + 8)) == kda.KDA_ERR_UNSUPPORTED, n
    for n in ("weight", "post_weight", "scale"):
        for shape in ((63,), (64, 1)):
            assert residual(changed(d, n, shape=shape)) == kda.KDA_ERR_SHAPE, (n, shape)
    assert residual(residual_descriptors(scale=2)) == kda.KDA_ERR_SHAPE
    for D in (0, 16385):
        assert residual(residual_descriptors(D=D)) == kda.KDA_ERR_UNSUPPORTED
    for rows in ((2 ** 16, 2 ** 15), (2 ** 40, 2 ** 40)):
        assert residual(residual_descriptors(rows=rows)) == kda.KDA_ERR_UNSUPPORTED
    assert residual(residual_descriptors(rows=(2 ** 24,), D=4096)) == kda.KDA_ERR_UNSUPPORTED
    for eps in (-1.0, float("nan"), float("inf")):
        assert residual(d, eps) == kda.KDA_ERR_MODE
    assert residual(residual_descriptors(rows=(0, 3))) == kda.KDA_OK


def gate_descriptors(shape=(1, 5, 4, 64), weight=(4, 64)):
    shapes = {"out": (BF16, shape), "x": (BF16, shape), "gate": (BF16, shape), "weight": (F32, weight)}
    return {n: fake(i, *s) for i, (n, s) in enumerate(shapes.items())}


def gate(d, *args):
    return kda.call_raw_norm_gate(list(d.values()), *args)


def test_norm_gate_refusals():
    d = gate_descriptors()
    for n in d:
        assert gate(dict(d, **{n: None})) == kda.KDA_ERR_NULL, n
        assert gate(changed(d, n, data=0)) == kda.KDA_ERR_NULL, n
        assert gate(changed(d, n, dtype=I32)) == kda.KDA_ERR_DTYPE, n
        assert gate(changed(d, n, data=d[n].data + 2)) == kda.KDA_ERR_UNSUPPORTED, n
    for n in ("out", "x", "gate"):
        assert gate(changed(d, n, dtype=F32)) == kda.KDA_ERR_DTYPE, n
        for shape in ((1, 5, 3, 64), (5, 4, 64), (1, 5, 4, 32)):
            assert gate(changed(d, n, shape=shape)) == kda.KDA_ERR_SHAPE, (n, shape)
    for shape in ((32,), (5, 64), (4, 32), (1, 4, 64)):
        assert gate(changed(d, "weight", shape=shape)) == kda.KDA_ERR_SHAPE, shape
    assert gate(gate_descriptors((64,), (1, 64))) == kda.KDA_ERR_SHAPE
    for D in (0, 16385):
        assert gate(gate_descriptors((3, D), (D,))) == kda.KDA_ERR_UNSUPPORTED
    assert gate(gate_descriptors((2 ** 30, 64), (64,))) == kda.KDA_ERR_UNSUPPORTED
    assert gate(d, 2) == gate(d, -1) == gate(d, 0, 2) == gate(d, 1, -1) == kda.KDA_ERR_MODE
    for eps in (-1.0, float("nan"), float("inf")):
        assert gate(d, 0, 0, eps) == kda.KDA_ERR_MODE
    assert gate(gate_descriptors((0, 64), (64,))) == kda.KDA_OK


def test_binding_refusals():
    """What the binding itself refuses, without a GPU."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 3, 4)
    with pytest.raises(ValueError, match="GPU tensor"):
        kda.ssm_decode(*[x] * 12)
    with pytest.raises(ValueError, match="GPU tensor"):
        kda.ssm_prefill(*[x] * 12)
    with pytest.raises(ValueError, match="GPU tensor"):
        kda.norm_residual(*[x] * 5)
    with pytest.raises(ValueError, match="GPU tensor"):
        kda.norm_gate(*[x] * 4)
    with pytest.raises(TypeError):
        kda.norm_gate(x, None, x, x)
    with pytest.raises(KeyError):
        kda.norm_gate(x, x, x, x, activation="relu")
