"""kda_norm_residual and kda_norm_gate against 64 bits.

Bounds, with eps = 2^-24 half a unit of fp32: a sum of squares over D values is
at most ~6 + 64 + 8 roundings deep whatever its order (64 values in a thread, a
tree over lanes and waves), half of which reach its root; the division, root and
products add some units, sigmoid and SiLU some five (of the hardware's exp2 and
reciprocal, plus |z| for exp's argument, times the value's own slope, below 8 in
all): 64 units of the result.  A residual sum is off by units of |h| + |s y|.
bf16 results add half a step, 2^-8 of the value.  Below 2^-126 fp32 rounds to
multiples of 2^-149: x act(gate), and x times the factor's first part, are off
by up to 2^-150 each (1e-38 times a gate of 0.01 has that much), which the
factor r (316 at eps 1e-5) and the weight enlarge: 2 * 2^-150 r |weight|.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gated_delta_rule_82_amd import kda  # noqa: E402
from tests.ssm_reference import BF16, EPS, sigmoid, unit  # noqa: E402

pytestmark = pytest.mark.gpu
DEVICE = "cuda:0"
UNITS = 64 * EPS
TYPES = {True: torch.bfloat16, False: torch.float32}
SIZES = [1, 2, 7, 8, 9, 31, 32, 63, 64, 65, 80, 127, 128, 129, 500, 512, 513, 1023, 2048, 2049, 2304, 4096, 4097, 8192,
         8200, 16383, 16384]


def draw(gen, *shape, bf16, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEVICE) * scale).to(TYPES[bf16])


def wide(t):
    return t.double().cpu().numpy()


def check(got, want, bf16, units=UNITS, extra=0.0):
    got = wide(got)
    tol = units * np.abs(want) + extra + (BF16 * np.abs(want) if bf16 else 0) + 1e-44
    off = np.abs(got - want) - tol
    assert off.max() <= 0, f"{off.max():.3g} over at {np.unravel_index(off.argmax(), off.shape)}"


def residual_reference(hidden, block_out, weight, post, scale, eps):
    h, y = wide(hidden), wide(block_out)
    if post is not None:
        y = unit(y, eps) * wide(post)
    s = 1.0 if scale is None else wide(scale)
    out = h + s * y
    return out, unit(out, eps) * wide(weight), np.abs(h) + np.abs(s * y)


def residual(rows, D, hbf16, bf16, post, scale, seed=0, in_place=False, eps=1e-5, size=1.0):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    hidden, y = draw(gen, rows, D, bf16=hbf16, scale=4 * size), draw(gen, rows, D, bf16=bf16, scale=size)
    w = draw(gen, D, bf16=False)
    p = draw(gen, D, bf16=False) if post else None
    s = {None: None, "one": draw(gen, 1, bf16=False), "channel": draw(gen, D, bf16=False)}[scale]
    want_h, want_n, mag = residual_reference(hidden, y, w, p, s, eps)
    h_out, normed = (hidden, y) if in_place else (torch.empty_like(hidden), torch.empty_like(y))
    kda.norm_residual(h_out, normed, hidden, y, w, post_weight=p, scale=s, eps=eps)
    torch.cuda.synchronize()
    check(h_out, want_h, hbf16, extra=UNITS * mag)
    r = 1.0 / np.sqrt((want_h ** 2).mean(-1, keepdims=True) + eps)
    check(normed, want_n, bf16, extra=2 * (UNITS * mag + 2.0 ** -150) * r * np.abs(wide(w)))


@pytest.mark.parametrize("D", SIZES)
def test_residual_sizes(D):
    residual(5, D, True, True, False, None, D)
    residual(3, D, False, True, True, "channel", D)


@pytest.mark.parametrize("hbf16", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("scale", [None, "one", "channel"])
def test_residual_forms(hbf16, bf16, post, scale):
    residual(33, 520, hbf16, bf16, post, scale, in_place=post)


@pytest.mark.parametrize("rows", [1, 2, 3, 255, 1025])
def test_residual_rows(rows):
    residual(rows, 72, True, True, False, None)
    residual(rows, 2560, False, False, True, "one", in_place=True)


def gate(shape, D, groups, act, first, bf16, seed=0, into=None, size=1.0, eps=1e-5):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    x, z = draw(gen, *shape, D, bf16=bf16, scale=size), draw(gen, *shape, D, bf16=bf16, scale=3.0)
    w = draw(gen, D, bf16=False) if groups is None else draw(gen, groups, D, bf16=False)
    zz = wide(z)
    a = sigmoid(zz) * (zz if act == "silu" else 1.0)
    want = unit(wide(x) * a, eps) * wide(w) if first else unit(wide(x), eps) * wide(w) * a
    u = wide(x) * a if first else wide(x)
    tiny = 2 * 2.0 ** -150 * np.abs(wide(w)) / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    out = {None: torch.empty_like(x), "x": x, "gate": z}[into]
    kda.norm_gate(out, x, z, w, activation=act, gate_first=first, eps=eps)
    torch.cuda.synchronize()
    check(out, want, bf16, extra=tiny)


@pytest.mark.parametrize("D", SIZES)
def test_gate_sizes(D):
    gate((5,), D, None, "sigmoid", False, True, D)
    gate((2, 3), D, 3, "silu", True, False, D)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("into", [None, "x", "gate"])
def test_gate_forms(act, first, bf16, into):
    gate((1, 7, 5), 128, 5, act, first, bf16, into=into)
    gate((11,), 1000, None, act, first, bf16, into=into)


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-18, 1e18, 1e25, 1e36])
def test_sums_of_squares_beyond_fp32(size):
    """Rows whose squares leave fp32, among ordinary ones."""
    for eps in (1e-5, 1e-37):
        gate((3,), 128, None, "sigmoid", False, False, size=size, eps=eps)
        gate((3,), 3000, None, "silu", True, False, size=size, eps=eps)
        residual(3, 600, False, False, False, None, size=size, eps=eps)


@pytest.mark.parametrize("value", [1.8e38, -2.5e38, 3.3e38])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("D", [1, 16, 64, 128, 130, 512, 4096, 16384])
def test_values_above_half_of_fp32(D, bf16, value):
    """A value above 2^127 alone in its row, among ordinary ones, and beside its like: the row's factor must not
    take it to infinity.  bf16 results below 2^-126 are multiples of 2^-133."""
    gen = torch.Generator(device=DEVICE).manual_seed(D)
    rows = draw(gen, 4, D, bf16=bf16)
    rows[0] = 0
    rows[0, D // 2] = rows[1, D // 3] = rows[2, 0] = value
    rows[2, D - 1] = -value
    small, w = draw(gen, 4, D, bf16=bf16), draw(gen, D, bf16=False)
    tiny = 2.0 ** -134 if bf16 else 0.0
    x = wide(rows)
    z = torch.full_like(rows, 40.0)         # sigmoid is 1
    for first in (False, True):
        out = torch.empty_like(rows)
        kda.norm_gate(out, rows, z, w, gate_first=first)
        check(out, unit(x, 1e-5) * wide(w) * sigmoid(40.0), bf16, extra=tiny)
    for hidden, block_out, post in ((rows, small, None), (small, rows, w)):
        want_h, want_n, mag = residual_reference(hidden, block_out, w, post, None, 1e-5)
        h_out, normed = torch.empty_like(hidden), torch.empty_like(block_out)
        kda.norm_residual(h_out, normed, hidden, block_out, w, post_weight=post)
        check(h_out, want_h, bf16, extra=UNITS * mag + tiny)
        r = 1.0 / np.sqrt((want_h ** 2).mean(-1, keepdims=True) + 1e-5)
        check(normed, want_n, bf16, extra=2 * (UNITS * mag + 2.0 ** -150) * r * np.abs(wide(w)) + tiny)


def test_zero_rows():
    x = torch.zeros(4, 3, 64, device=DEVICE, dtype=torch.bfloat16)
    out = torch.ones_like(x)
    kda.norm_gate(out, x, torch.ones_like(x), torch.ones(64, device=DEVICE))
    assert not out.any()
    h = torch.zeros(2, 4097, device=DEVICE)
    normed = torch.ones(2, 4097, device=DEVICE, dtype=torch.bfloat16)
    kda.norm_residual(h, normed, h, torch.zeros_like(normed), torch.ones(4097, device=DEVICE),
                      post_weight=torch.ones(4097, device=DEVICE))
    assert not h.any() and not normed.any()


def test_a_row_that_is_not_finite_stays_alone():
    gen = torch.Generator(device=DEVICE).manual_seed(1)
    x, z, w = draw(gen, 9, 64, bf16=False), draw(gen, 9, 64, bf16=False), draw(gen, 64, bf16=False)
    want = unit(wide(x), 1e-5) * wide(w) * sigmoid(wide(z))
    x[3, 5], x[6, 0] = float("nan"), float("inf")
    out = torch.empty_like(x)
    kda.norm_gate(out, x, z, w)
    keep = [0, 1, 2, 4, 5, 7, 8]
    check(out[keep], want[keep], False)
    assert torch.isnan(out[3]).all() and torch.isnan(out[6, 0]) and not out[6, 1:].any()


@pytest.mark.parametrize("shape", [(0, 64), (2, 0, 64), (64,)])
def test_rows_none_and_one(shape):
    x = torch.ones(shape, device=DEVICE)
    out = torch.empty_like(x)
    kda.norm_gate(out, x, x, torch.ones(64, device=DEVICE), eps=1e-5)
    kda.norm_residual(out, x.clone(), x, x, torch.ones(64, device=DEVICE))
    torch.cuda.synchronize()
    assert (out == 2).all()


def test_vectors_at_any_element():
    """Weights and scales that begin at any float, as parts of one buffer do."""
    gen = torch.Generator(device=DEVICE).manual_seed(2)
    buf = draw(gen, 4 * 130 + 3, bf16=False)
    w, p, s = buf[1:131], buf[132:262], buf[263:393]
    h, y = draw(gen, 6, 130, bf16=True), draw(gen, 6, 130, bf16=True)
    want_h, want_n, mag = residual_reference(h, y, w, p, s, 1e-5)
    normed = torch.empty_like(y)
    kda.norm_residual(h, normed, h, y, w, post_weight=p, scale=s)
    check(h, want_h, True, extra=UNITS * mag)
    r = 1.0 / np.sqrt((want_h ** 2).mean(-1, keepdims=True) + 1e-5)
    check(normed, want_n, True, extra=2 * UNITS * mag * r * np.abs(wide(w)))


def test_captured_and_on_another_stream():
    gen = torch.Generator(device=DEVICE).manual_seed(3)
    h, y, w = draw(gen, 10, 2304, bf16=True), draw(gen, 10, 2304, bf16=True), draw(gen, 2304, bf16=False)
    z = draw(gen, 10, 2304, bf16=True)
    h2, n1, n2, o1, o2 = h.clone(), *(torch.empty_like(y) for _ in range(4))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.norm_residual(h, n1, h, y, w)
        kda.norm_gate(o1, n1, z, w, activation="silu", gate_first=True)
    stream = torch.cuda.Stream()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        kda.norm_residual(h2, n2, h2, y, w, stream=stream.cuda_stream)
        kda.norm_gate(o2, n2, z, w, activation="silu", gate_first=True, stream=stream.cuda_stream)
        stream.synchronize()
        assert torch.equal(h, h2) and torch.equal(n1, n2) and torch.equal(o1, o2)


def test_rows_beyond_32_bits():
    """The last rows of more than 2^31 values are those of a short call."""
    D, last = 2304, 64
    rows = 2 ** 31 // D + 1 + last
    gen = torch.Generator(device=DEVICE).manual_seed(4)
    h, y = draw(gen, last, D, bf16=True), draw(gen, last, D, bf16=True)
    w = draw(gen, D, bf16=False)
    want_h, want_n, want_g = (torch.empty_like(y) for _ in range(3))
    kda.norm_residual(want_h, want_n, h, y, w)
    kda.norm_gate(want_g, y, h, w)
    long_h, long_y = (torch.empty(rows, D, dtype=torch.bfloat16, device=DEVICE) for _ in range(2))
    gated = torch.empty_like(long_y)
    long_h[-last:], long_y[-last:] = h, y
    kda.norm_gate(gated, long_y, long_h, w)
    kda.norm_residual(long_h, long_y, long_h, long_y, w)
    assert torch.equal(gated[-last:], want_g)
    assert torch.equal(long_h[-last:], want_h) and torch.equal(long_y[-last:], want_n)
