"""CPU tests of the argument checks of kda_gdr_decode, kda_gdr_prefill,
kda_decode_window and kda_verify: every malformed call is refused before any
device work.  The data pointers are fake and never dereferenced."""
import os

import pytest

from gated_delta_rule_82_amd import kda

pytestmark = pytest.mark.skipif(not os.path.exists(kda.LIB_PATH),
                                reason="libkda.so not built (run the build first)")

F32, BF16, I32 = kda.KDA_F32, kda.KDA_BF16, kda.KDA_I32


def fake(i, dtype, shape):
    return kda.raw_tensor(0x100000 * (i + 1), dtype, shape)


def descriptors(B=2, T=3, H=2, HV=4, DK=128, DV=64, N=8, qkv=BF16, channel=False):
    shapes = {
        "out": (qkv, (1, T, HV, DV)), "q": (qkv, (1, T, H, DK)), "k": (qkv, (1, T, H, DK)),
        "v": (qkv, (1, T, HV, DV)), "raw_gate": (F32, (1, T, HV, DK) if channel else (1, T, HV)),
        "beta_logits": (F32, (1, T, HV)), "a_log": (F32, (HV,)),
        "dt_bias": (F32, (HV, DK) if channel else (HV,)), "cu_seqlens": (I32, (B + 1,)),
        "state_pool": (F32, (N, HV, DK, DV)), "state_indices": (I32, (B,)),
    }
    return {n: fake(i, *shapes[n]) for i, n in enumerate(kda.ARG_NAMES)}


def replay_descriptors(B=2, T=5, H=2, HV=4, DK=128, DV=64, qkv=BF16, channel=False):
    shapes = {
        "k": (qkv, (1, T, H, DK)), "v": (qkv, (1, T, HV, DV)),
        "raw_gate": (F32, (1, T, HV, DK) if channel else (1, T, HV)),
        "beta_logits": (F32, (1, T, HV)), "begin": (I32, (B,)), "count": (I32, (B,)),
    }
    return {n: fake(20 + i, *shapes[n]) for i, n in enumerate(kda.REPLAY_FIELDS)}


def gdr(d, prefill=False, **mode):
    return kda.call_raw_gdr([d[n] for n in kda.ARG_NAMES], kda.make_mode(**mode), prefill, 0)


def window(d, r, **mode):
    rep = None if r is None else kda.KdaReplay(*[r[n] for n in kda.REPLAY_FIELDS])
    return kda.call_raw_window([d[n] for n in kda.ARG_NAMES], rep, kda.make_mode(**mode), 0)


def changed(d, name, dtype=None, shape=None, data=None):
    e = dict(d)
    t = d[name]
    e[name] = kda.raw_tensor(t.data if data is None else data, t.dtype if dtype is None else dtype,
                             tuple(t.shape[:t.ndim]) if shape is None else shape)
    return e


ENTRIES = {
    "decode": lambda d, **m: gdr(d, False, **m),
    "prefill": lambda d, **m: gdr(d, True, **m),
    "window": lambda d, **m: window(d, replay_descriptors(), **m),
}


@pytest.mark.parametrize("entry", sorted(ENTRIES))
def test_nulls_dtypes_shapes_and_modes(entry):
    call = ENTRIES[entry]
    d = descriptors()
    for n in kda.ARG_NAMES:
        assert call(dict(d, **{n: None})) == kda.KDA_ERR_NULL, n
        assert call(changed(d, n, data=0)) == kda.KDA_ERR_NULL, n
    for n, dtype in (("q", F32), ("k", F32), ("out", F32), ("v", I32), ("raw_gate", BF16),
                     ("beta_logits", BF16), ("a_log", I32), ("dt_bias", BF16), ("state_pool", I32),
                     ("cu_seqlens", F32), ("state_indices", F32)):
        assert call(changed(d, n, dtype=dtype)) == kda.KDA_ERR_DTYPE, n
    for n, shape in (("q", (2, 3, 2, 128)), ("k", (1, 3, 2, 64)), ("v", (1, 4, 4, 64)),
                     ("out", (1, 3, 4, 128)), ("raw_gate", (1, 3, 2)), ("raw_gate", (1, 2, 4)),
                     ("beta_logits", (1, 3, 3)), ("a_log", (3,)), ("dt_bias", (3,)), ("dt_bias", (4, 128)),
                     ("cu_seqlens", (4,)), ("state_pool", (8, 4, 64, 128)), ("state_indices", (3,))):
        assert call(changed(d, n, shape=shape)) == kda.KDA_ERR_SHAPE, (n, shape)
    for mode in (dict(gate_mode=7), dict(gate_mode="lower_bound", lower_bound=0.5), dict(state_layout=2),
                 dict(l2_eps=-1.0), dict(scale=float("nan"))):
        assert call(d, **mode) == kda.KDA_ERR_MODE, mode
    assert call(changed(d, "state_pool", data=0x100004)) == kda.KDA_ERR_UNSUPPORTED


def test_gate_rank_says_which_gate():
    # the per-head calls refuse per-channel gates; the window takes both, but not mixed
    d = descriptors(channel=True)
    assert gdr(d) == kda.KDA_ERR_SHAPE
    assert gdr(d, True) == kda.KDA_ERR_SHAPE
    assert window(d, replay_descriptors(channel=False)) == kda.KDA_ERR_SHAPE
    assert window(descriptors(), replay_descriptors(channel=True)) == kda.KDA_ERR_SHAPE
    mixed = dict(d, dt_bias=descriptors()["dt_bias"])
    assert window(mixed, replay_descriptors(channel=True)) == kda.KDA_ERR_SHAPE


def test_nothing_to_do():
    assert gdr(descriptors(B=0, T=0)) == kda.KDA_OK
    assert gdr(descriptors(B=3, T=0)) == kda.KDA_OK
    assert gdr(descriptors(B=3, T=0), True) == kda.KDA_OK
    assert window(descriptors(B=0, T=0), replay_descriptors(B=0)) == kda.KDA_OK
    assert window(descriptors(T=0), replay_descriptors(T=0)) == kda.KDA_OK


@pytest.mark.parametrize("dk,dv", [(48, 128), (128, 96), (256, 128), (128, 8)])
def test_unsupported_head_sizes(dk, dv):
    assert gdr(descriptors(DK=dk, DV=dv)) == kda.KDA_ERR_UNSUPPORTED
    assert gdr(descriptors(DK=dk, DV=dv), True) == kda.KDA_ERR_UNSUPPORTED
    assert window(descriptors(DK=dk, DV=dv), replay_descriptors(DK=dk, DV=dv)) == kda.KDA_ERR_UNSUPPORTED


@pytest.mark.parametrize("dk,dv", [(16, 128), (128, 16)])
def test_prefill_refuses_head_size_16(dk, dv):
    assert gdr(descriptors(B=0, T=0, DK=dk, DV=dv)) == kda.KDA_OK
    assert gdr(descriptors(B=0, T=0, DK=dk, DV=dv), True) == kda.KDA_ERR_UNSUPPORTED


def test_replay_checks():
    d, r = descriptors(), replay_descriptors()
    assert window(d, None) == kda.KDA_ERR_NULL
    for n in kda.REPLAY_FIELDS:
        assert window(d, changed(r, n, data=0)) == kda.KDA_ERR_NULL, n
    for n, dtype in (("k", F32), ("v", F32), ("raw_gate", BF16), ("beta_logits", BF16), ("begin", F32),
                     ("count", F32)):
        assert window(d, changed(r, n, dtype=dtype)) == kda.KDA_ERR_DTYPE, n
    for n, shape in (("k", (1, 4, 2, 128)), ("k", (1, 5, 4, 128)), ("k", (1, 5, 2, 64)), ("v", (1, 5, 4, 128)),
                     ("v", (2, 5, 4, 64)), ("raw_gate", (1, 5, 2)), ("raw_gate", (1, 4, 4)),
                     ("beta_logits", (1, 5, 2)), ("beta_logits", (1, 6, 4)), ("begin", (3,)), ("count", (1,)),
                     ("count", (1, 2))):
        assert window(d, changed(r, n, shape=shape)) == kda.KDA_ERR_SHAPE, (n, shape)
    assert window(d, changed(r, "k", data=0x2000008)) == kda.KDA_ERR_UNSUPPORTED
    assert window(d, changed(r, "begin", data=0x2000002)) == kda.KDA_ERR_UNSUPPORTED


@pytest.mark.parametrize("B,T", [(2 ** 31, 3), (2 ** 62, 3), (2, 2 ** 31), (2, 2 ** 62)])
def test_huge_extents(B, T):
    assert gdr(descriptors(B=B, T=T)) == kda.KDA_ERR_UNSUPPORTED
    assert gdr(descriptors(B=B, T=T), True) == kda.KDA_ERR_UNSUPPORTED
    assert window(descriptors(B=B, T=3), replay_descriptors(B=B, T=T)) == kda.KDA_ERR_UNSUPPORTED


# ---------------------------------------------------------------------------
# kda_verify
# ---------------------------------------------------------------------------

def verify_descriptors(B=2, T=5, V=1000, probs=F32, draft=True, ws=None):
    shapes = {
        "n_commit": (I32, (B,)), "next_token": (I32, (B,)), "target_probs": (probs, (T, V)),
        "draft_probs": (probs, (T, V)), "tokens": (I32, (T,)), "u_accept": (F32, (T,)),
        "u_sample": (F32, (B,)), "cu_seqlens": (I32, (B + 1,)),
        "workspace": (F32, (kda.verify_workspace(B, V) if ws is None else ws,)),
    }
    d = {n: fake(i, *shapes[n]) for i, n in enumerate(kda.VERIFY_NAMES)}
    if not draft:
        d["draft_probs"] = None
    return d


def verify(d):
    return kda.call_raw_verify([d[n] for n in kda.VERIFY_NAMES], 0)


def test_verify_checks():
    d = verify_descriptors()
    for n in kda.VERIFY_NAMES:
        if n != "draft_probs":
            assert verify(dict(d, **{n: None})) == kda.KDA_ERR_NULL, n
        assert verify(changed(d, n, data=0)) == kda.KDA_ERR_NULL, n
    for n, dtype in (("n_commit", F32), ("next_token", F32), ("target_probs", BF16), ("target_probs", I32),
                     ("draft_probs", BF16), ("tokens", F32), ("u_accept", BF16), ("u_sample", I32),
                     ("cu_seqlens", F32), ("workspace", I32)):
        assert verify(changed(d, n, dtype=dtype)) == kda.KDA_ERR_DTYPE, n
    for n, shape in (("n_commit", (3,)), ("next_token", (1,)), ("target_probs", (5, 999)), ("target_probs", (5,)),
                     ("draft_probs", (4, 1000)), ("tokens", (4,)), ("u_accept", (6,)), ("u_sample", (3,)),
                     ("cu_seqlens", (2,)), ("workspace", (kda.verify_workspace(2, 1000) - 1,))):
        assert verify(changed(d, n, shape=shape)) == kda.KDA_ERR_SHAPE, n
    for n, data in (("target_probs", 0x300008), ("draft_probs", 0x300004), ("workspace", 0x300008),
                    ("tokens", 0x300002), ("u_sample", 0x300001)):
        assert verify(changed(d, n, data=data)) == kda.KDA_ERR_UNSUPPORTED, n
    empty = verify_descriptors(V=1)
    for n in ("target_probs", "draft_probs"):
        empty = changed(empty, n, shape=(5, 0))
    assert verify(empty) == kda.KDA_ERR_SHAPE
    assert verify(verify_descriptors(B=0, T=0)) == kda.KDA_OK
    assert verify(verify_descriptors(B=0, T=0, draft=False)) == kda.KDA_OK


@pytest.mark.parametrize("B,T,V", [(2 ** 31, 1, 10), (1, 2 ** 31, 10), (1, 1, 2 ** 31), (2 ** 24, 1, 2 ** 20),
                                   (2 ** 62, 1, 2 ** 62)])
def test_verify_huge_extents(B, T, V):
    assert verify(verify_descriptors(B=B, T=T, V=V, ws=16)) == kda.KDA_ERR_UNSUPPORTED


def test_verify_binding():
    torch = pytest.importorskip("torch")
    t = torch.zeros(4)
    with pytest.raises(ValueError, match="workspace"):
        kda.verify(t, t, t, None, t, t, t, t, stream=0)
    with pytest.raises(ValueError, match="target_probs"):
        kda.verify(t, t, t, None, t, t, t, t)
    p = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        kda.verify(t, t, p, None, t, t, t, t)
    for call, n in ((kda.gdr_decode, 11), (kda.gdr_prefill, 11), (kda.decode_window, 17)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call(*([t] * n))
