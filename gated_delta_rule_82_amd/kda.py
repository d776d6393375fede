"""Thin binding of libkda (argument marshalling only).

Every step of every operator runs in the HIP library; this module checks that
torch tensors can be passed, hands them with the current HIP stream to the
library and raises :class:`KdaError` on a nonzero status.  A small extension
(csrc/kda_binding.cpp) turns tensors into ``kda_tensor`` descriptors; where it
is not built or does not fit the torch that is installed, ctypes does the same.
The ``call_raw*`` functions call the C ABI on descriptors made here.  There is
no fallback: if the library is missing or a tensor is not on a GPU, the call
raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "lib", "libkda.so")
BINDING_PATH = os.path.join(PKG, "lib", "_kda_binding.so")   # the call path, csrc/kda_binding.cpp

# enum values of include/kda.h
KDA_OK = 0
KDA_ERR_NULL = -1
KDA_ERR_DTYPE = -2
KDA_ERR_SHAPE = -3
KDA_ERR_UNSUPPORTED = -4
KDA_ERR_MODE = -5
KDA_ERR_LAUNCH = -6
KDA_ERR_PRECONDITION = -7

KDA_F32 = 0
KDA_BF16 = 1
KDA_I32 = 2

KDA_GATE_SOFTPLUS = 0
KDA_GATE_LOWER_BOUND = 1
GATE_MODES = {"softplus": KDA_GATE_SOFTPLUS, "lower_bound": KDA_GATE_LOWER_BOUND}

KDA_STATE_K_FIRST = 0
KDA_STATE_V_FIRST = 1
STATE_LAYOUTS = {"k_first": KDA_STATE_K_FIRST, "v_first": KDA_STATE_V_FIRST}

KDA_MATMUL_SPLIT_BF16 = 0
KDA_MATMUL_F32 = 1
MATMULS = {"split_bf16": KDA_MATMUL_SPLIT_BF16, "f32": KDA_MATMUL_F32}

KDA_VERIFY_SEGMENT = 1024

KDA_SSM_CHUNK = 32
KDA_SSM_SPLIT = 1536

KDA_ACT_SIGMOID = 0
KDA_ACT_SILU = 1
ACTIVATIONS = {"sigmoid": KDA_ACT_SIGMOID, "silu": KDA_ACT_SILU}

EXPORTED_SYMBOLS = ("kda_decode", "kda_decode_conv", "kda_prefill", "kda_gdr_decode",
                    "kda_gdr_prefill", "kda_decode_window", "kda_verify", "kda_ssm_decode",
                    "kda_ssm_prefill", "kda_norm_residual", "kda_norm_gate", "kda_check_host",
                    "kda_status_string", "kda_abi_version")
CONV_FIELDS = ("x_q", "x_k", "x_v", "w_q", "w_k", "w_v", "win_q", "win_k", "win_v", "q_conv",
               "k_conv")
REPLAY_FIELDS = ("k", "v", "raw_gate", "beta_logits", "begin", "count")


class KdaTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("ndim", ctypes.c_int32), ("shape", ctypes.c_int64 * 4)]


class KdaConv(ctypes.Structure):
    _fields_ = [(n, KdaTensor) for n in CONV_FIELDS]


class KdaReplay(ctypes.Structure):
    _fields_ = [(n, KdaTensor) for n in REPLAY_FIELDS]


class KdaMode(ctypes.Structure):
    _fields_ = [("gate_mode", ctypes.c_int32), ("lower_bound", ctypes.c_float),
                ("l2_eps", ctypes.c_float), ("scale", ctypes.c_float),
                ("state_layout", ctypes.c_int32)]


class KdaError(RuntimeError):
    def __init__(self, code: int, where: str = "kda_decode"):
        self.code = code
        super().__init__(f"{where} failed with status {code}: {status_string(code)}")


class KdaLibraryMissing(RuntimeError):
    pass


_lib: Optional[ctypes.CDLL] = None
_torch = None          # set by library()
_raw_stream = None
_native = None         # the extension's call(), or the same through ctypes; set by the first call
_ENTRY = {}            # entry point -> its address


def library() -> ctypes.CDLL:
    """Load libkda.so (built in-tree by ``gated_delta_rule_82_amd.build``).

    torch is imported first so that the library binds to the HIP runtime torch
    already loaded (both carry the soname libamdhip64.so.7): one runtime, one
    set of streams."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise KdaLibraryMissing(
            f"{LIB_PATH} is not built; run `python -m gated_delta_rule_82_amd.build`")
    import torch  # (binds the process to torch's HIP runtime first)
    global _torch, _raw_stream
    _torch = torch
    # the current stream's handle without a Stream object (microseconds of a short call)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    lib = ctypes.CDLL(LIB_PATH, mode=ctypes.RTLD_LOCAL)
    T, M, stream = ctypes.POINTER(KdaTensor), ctypes.POINTER(KdaMode), ctypes.c_void_p
    lib.kda_decode.argtypes = [T] * 11 + [M, stream]
    lib.kda_decode_conv.argtypes = [T, ctypes.POINTER(KdaConv)] + [T] * 7 + [M, stream]
    lib.kda_prefill.argtypes = [T] * 11 + [M, ctypes.c_int32, stream]
    lib.kda_gdr_decode.argtypes = lib.kda_gdr_prefill.argtypes = [T] * 11 + [M, stream]
    lib.kda_decode_window.argtypes = [T] * 11 + [ctypes.POINTER(KdaReplay), M, stream]
    lib.kda_verify.argtypes = [T] * 9 + [stream]
    lib.kda_ssm_decode.argtypes = [T] * 12 + [ctypes.c_int32, stream]
    lib.kda_ssm_prefill.argtypes = [T] * 13 + [ctypes.c_int32, stream]
    lib.kda_norm_residual.argtypes = [T] * 7 + [ctypes.c_float, stream]
    lib.kda_norm_gate.argtypes = [T] * 4 + [ctypes.c_int32, ctypes.c_int32, ctypes.c_float, stream]
    for name in ("kda_decode", "kda_decode_conv", "kda_prefill", "kda_gdr_decode", "kda_gdr_prefill",
                 "kda_decode_window", "kda_verify", "kda_ssm_decode", "kda_ssm_prefill", "kda_norm_residual",
                 "kda_norm_gate"):
        getattr(lib, name).restype = ctypes.c_int
    lib.kda_check_host.argtypes = [ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32),
                                   ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]
    lib.kda_check_host.restype = ctypes.c_int
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_abi_version.argtypes = []
    lib.kda_abi_version.restype = ctypes.c_int
    _ENTRY.update({name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                   for name in EXPORTED_SYMBOLS})
    _lib = lib
    return lib


def status_string(code: int) -> str:
    try:
        return library().kda_status_string(int(code)).decode()
    except KdaLibraryMissing:
        return "libkda not built"


def make_mode(gate_mode="softplus", lower_bound=0.0, l2_eps=0.0, scale=0.0,
              state_layout="k_first") -> KdaMode:
    gm = GATE_MODES[gate_mode] if isinstance(gate_mode, str) else int(gate_mode)
    sl = STATE_LAYOUTS[state_layout] if isinstance(state_layout, str) else int(state_layout)
    return KdaMode(gm, float(lower_bound), float(l2_eps), float(scale), sl)


def raw_tensor(data_ptr: int, dtype: int, shape) -> KdaTensor:
    t = KdaTensor()
    t.data = data_ptr
    t.dtype = dtype
    t.ndim = len(shape)
    for i, s in enumerate(shape):
        t.shape[i] = int(s)
    return t


def call_raw(tensors, mode: KdaMode, stream: int = 0) -> int:
    """Call kda_decode on 11 prepared descriptors (None passes NULL); returns
    the status code without raising."""
    lib = library()
    ptrs = [ctypes.byref(t) if t is not None else None for t in tensors]
    return lib.kda_decode(*ptrs, ctypes.byref(mode) if mode is not None else None,
                          ctypes.c_void_p(stream))


def call_raw_prefill(tensors, mode: KdaMode, matmul: int = KDA_MATMUL_SPLIT_BF16,
                     stream: int = 0) -> int:
    """Call kda_prefill on 11 prepared descriptors (None passes NULL); returns
    the status code without raising."""
    lib = library()
    ptrs = [ctypes.byref(t) if t is not None else None for t in tensors]
    return lib.kda_prefill(*ptrs, ctypes.byref(mode) if mode is not None else None,
                           ctypes.c_int32(matmul), ctypes.c_void_p(stream))


def call_raw_conv(out, conv, rest, mode: KdaMode, stream: int = 0) -> int:
    """Call kda_decode_conv on prepared descriptors: ``out``, a KdaConv (or
    None), and the 7 remaining tensors (raw_gate .. state_indices)."""
    lib = library()
    ref = lambda t: ctypes.byref(t) if t is not None else None  # noqa: E731
    return lib.kda_decode_conv(ref(out), ref(conv), *[ref(t) for t in rest], ref(mode),
                               ctypes.c_void_p(stream))


def call_raw_gdr(tensors, mode: KdaMode, prefill: bool = False, stream: int = 0) -> int:
    """Call kda_gdr_decode (or kda_gdr_prefill) on 11 prepared descriptors
    (None passes NULL); returns the status code without raising."""
    lib = library()
    ref = lambda t: ctypes.byref(t) if t is not None else None  # noqa: E731
    fn = lib.kda_gdr_prefill if prefill else lib.kda_gdr_decode
    return fn(*[ref(t) for t in tensors], ref(mode), ctypes.c_void_p(stream))


def call_raw_window(tensors, replay, mode: KdaMode, stream: int = 0) -> int:
    """Call kda_decode_window on 11 prepared descriptors and a KdaReplay (None
    passes NULL); returns the status code without raising."""
    ref = lambda t: ctypes.byref(t) if t is not None else None  # noqa: E731
    return library().kda_decode_window(*[ref(t) for t in tensors], ref(replay), ref(mode),
                                       ctypes.c_void_p(stream))


def call_raw_verify(tensors, stream: int = 0) -> int:
    """Call kda_verify on 9 prepared descriptors (None passes NULL); returns
    the status code without raising."""
    ref = lambda t: ctypes.byref(t) if t is not None else None  # noqa: E731
    return library().kda_verify(*[ref(t) for t in tensors], ctypes.c_void_p(stream))


def call_raw_ssm(tensors, state_layout: int = KDA_STATE_K_FIRST, stream: int = 0) -> int:
    """Call kda_ssm_decode on 12 prepared descriptors, or kda_ssm_prefill on 13
    (None passes NULL); returns the status code without raising."""
    lib = library()
    ref = lambda t: ctypes.byref(t) if t is not None else None  # noqa: E731
    fn = lib.kda_ssm_decode if len(tensors) == 12 else lib.kda_ssm_prefill
    return fn(*[ref(t) for t in tensors], ctypes.c_int32(state_layout), ctypes.c_void_p(stream))


def call_raw_norm_residual(tensors, eps: float = 0.0, stream: int = 0) -> int:
    """Call kda_norm_residual on 7 prepared descriptors (None passes NULL);
    returns the status code without raising."""
    ref = lambda t: ctypes.byref(t) if t is not None else None  # noqa: E731
    return library().kda_norm_residual(*[ref(t) for t in tensors], ctypes.c_float(eps), ctypes.c_void_p(stream))


def call_raw_norm_gate(tensors, act: int = KDA_ACT_SIGMOID, gate_first: int = 0, eps: float = 0.0,
                       stream: int = 0) -> int:
    """Call kda_norm_gate on 4 prepared descriptors (None passes NULL); returns
    the status code without raising."""
    ref = lambda t: ctypes.byref(t) if t is not None else None  # noqa: E731
    return library().kda_norm_gate(*[ref(t) for t in tensors], ctypes.c_int32(act), ctypes.c_int32(gate_first),
                                   ctypes.c_float(eps), ctypes.c_void_p(stream))


def _descriptor(t, name):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a GPU tensor, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.dim() > 4:
        raise ValueError(f"{name}: at most 4 dimensions")
    dt = {torch.float32: KDA_F32, torch.bfloat16: KDA_BF16, torch.int32: KDA_I32}.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")
    return raw_tensor(t.data_ptr(), dt, t.shape)


ARG_NAMES = ("out", "q", "k", "v", "raw_gate", "beta_logits", "a_log", "dt_bias",
             "cu_seqlens", "state_pool", "state_indices")


# ---------------------------------------------------------------------------
# the call path
# ---------------------------------------------------------------------------

# kinds of csrc/kda_binding.cpp
(_RECURRENCE, _PREFILL, _CONV, _WINDOW, _VERIFY, _SSM_DECODE, _SSM_PREFILL, _NORM_RESIDUAL,
 _NORM_GATE) = range(9)
# tensors of a kind that may be None
_OPTIONAL = {_VERIFY: (3,), _SSM_DECODE: (4, 8), _SSM_PREFILL: (4, 8), _NORM_RESIDUAL: (5, 6)}


def _refuse(tensors, names, dev):
    """Say what is wrong with the tensors of a call that could not be passed."""
    for t, n in zip(tensors, names):
        _descriptor(t, n)
    for t, n in zip(tensors, names):
        if t.device.index != dev:
            raise ValueError(f"{n}: on {t.device}, expected cuda:{dev}")
    raise ValueError("a tensor cannot be passed to libkda")


def _device(t, name):
    """Index of the GPU that ``t`` is on."""
    try:
        dev = t.get_device()
    except AttributeError:
        dev = -1
    if dev < 0:
        _descriptor(t, name)
    return dev


def _load_native():
    """Set ``_native``: the extension's call(), which is tied to this torch's and
    this Python's ABI, or, where it is not built or does not load, its like below."""
    global _native
    _native = _described_call
    if os.path.exists(BINDING_PATH):
        try:
            spec = importlib.util.spec_from_file_location("_kda_binding", BINDING_PATH)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            _native = module.call
        except ImportError:
            pass


def _described_call(kind, entry, tensors, dev, gate_mode, lower_bound, l2_eps, scale, state_layout, matmul, stream):
    """The extension's call() on descriptors made here (some ten microseconds
    more a call): the entry point's status, or None if a tensor cannot be passed."""
    described = []
    for i, t in enumerate(tensors):
        if t is None and i in _OPTIONAL.get(kind, ()):
            described.append(None)
            continue
        try:
            d = _descriptor(t, "tensor")
        except (TypeError, ValueError):
            return None
        if t.device.index != dev:
            return None
        described.append(d)
    mode = KdaMode(gate_mode, lower_bound, l2_eps, scale, state_layout)
    where = next(n for n, address in _ENTRY.items() if address == entry)
    if kind == _CONV:
        return call_raw_conv(described[0], KdaConv(*described[1:12]), described[12:], mode, stream)
    if kind == _WINDOW:
        return call_raw_window(described[:11], KdaReplay(*described[11:]), mode, stream)
    if kind == _VERIFY:
        return call_raw_verify(described, stream)
    if kind in (_SSM_DECODE, _SSM_PREFILL):
        return call_raw_ssm(described, state_layout, stream)
    if kind == _NORM_RESIDUAL:
        return call_raw_norm_residual(described, l2_eps, stream)
    if kind == _NORM_GATE:
        return call_raw_norm_gate(described, gate_mode, matmul, l2_eps, stream)
    if kind == _PREFILL:
        return call_raw_prefill(described, mode, matmul, stream)
    if where == "kda_decode":
        return call_raw(described, mode, stream)
    return call_raw_gdr(described, mode, where == "kda_gdr_prefill", stream)


def _call(kind, where, tensors, names, dev, stream, gate_mode=0, lower_bound=0.0, l2_eps=0.0, scale=0.0,
          state_layout=0, matmul=0):
    """Call entry point ``where`` with GPU ``dev`` current, on ``stream`` or torch's current one."""
    if _torch.cuda.current_device() != dev:
        with _torch.cuda.device(dev):
            return _call(kind, where, tensors, names, dev, stream, gate_mode, lower_bound, l2_eps, scale,
                         state_layout, matmul)
    if _native is None:
        _load_native()
    gm = GATE_MODES[gate_mode] if isinstance(gate_mode, str) else int(gate_mode)
    sl = STATE_LAYOUTS[state_layout] if isinstance(state_layout, str) else int(state_layout)
    rc = _native(kind, _ENTRY[where], tensors, dev, gm, lower_bound, l2_eps, scale, sl, matmul,
                 _raw_stream(dev) if stream is None else stream)
    if rc is None:
        optional = _OPTIONAL.get(kind, ())
        given = [(t, n) for i, (t, n) in enumerate(zip(tensors, names)) if t is not None or i not in optional]
        _refuse([t for t, _ in given], [n for _, n in given], dev)
    if rc != KDA_OK:
        raise KdaError(rc, where)


def _recurrence(where, tensors, gate_mode, lower_bound, l2_eps, scale, state_layout, stream, kind=_RECURRENCE,
                matmul=0):
    """The calls that take the 11 tensors of kda_decode and a mode."""
    if _lib is None:
        library()
    _call(kind, where, tensors, ARG_NAMES, _device(tensors[1], "q"), stream, gate_mode, lower_bound, l2_eps, scale,
          state_layout, matmul)


def decode(out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool,
           state_indices, *, gate_mode="softplus", lower_bound=0.0, l2_eps=0.0, scale=0.0,
           state_layout="k_first", stream: Optional[int] = None) -> None:
    """Advance the KDA decode recurrence in place (see include/kda.h).

    Tensors are torch GPU tensors with the shapes of kda.h; ``out`` and
    ``state_pool`` are written.  ``state_pool`` is float32 or bfloat16, laid
    out [N, HV, dk, dv] ("k_first") or [N, HV, dv, dk] ("v_first").  The work
    is enqueued on ``stream`` (a raw hipStream_t handle; default: torch's
    current stream of q's device)."""
    _recurrence("kda_decode",
                (out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool, state_indices),
                gate_mode, lower_bound, l2_eps, scale, state_layout, stream)


def prefill(out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool,
            state_indices, *, gate_mode="softplus", lower_bound=0.0, l2_eps=0.0, scale=0.0,
            state_layout="k_first", matmul="split_bf16", stream: Optional[int] = None) -> None:
    """The recurrence over long requests in chunks of 16 tokens on the matrix
    cores (kda_prefill in include/kda.h): same tensors and result as
    :func:`decode`; ``matmul`` is "split_bf16" (default) or "f32"."""
    mm = MATMULS[matmul] if isinstance(matmul, str) else int(matmul)
    _recurrence("kda_prefill",
                (out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool, state_indices),
                gate_mode, lower_bound, l2_eps, scale, state_layout, stream, _PREFILL, mm)


def check_host(cu_seqlens, state_indices, T: int, n_slots: int) -> int:
    """Run kda_check_host on host int32 arrays; returns the status code."""
    import numpy as np
    cu = np.ascontiguousarray(cu_seqlens, dtype=np.int32)
    idx = np.ascontiguousarray(state_indices, dtype=np.int32)
    if cu.ndim != 1 or idx.ndim != 1 or len(cu) != len(idx) + 1:
        # kda_check_host reads B + 1 entries of cu_seqlens
        raise ValueError(f"cu_seqlens needs len(state_indices) + 1 = {len(idx) + 1} entries, "
                         f"got shape {cu.shape}")
    P = ctypes.POINTER(ctypes.c_int32)
    return library().kda_check_host(cu.ctypes.data_as(P), idx.ctypes.data_as(P),
                                    len(idx), int(T), int(n_slots))


CONV_REST = ("raw_gate", "beta_logits", "a_log", "dt_bias", "cu_seqlens", "state_pool",
             "state_indices")


def decode_conv(out, x_q, x_k, x_v, w_q, w_k, w_v, win_q, win_k, win_v, q_conv, k_conv, raw_gate,
                beta_logits, a_log, dt_bias, cu_seqlens, state_pool, state_indices, *,
                gate_mode="softplus", lower_bound=0.0, l2_eps=0.0, scale=0.0,
                state_layout="k_first", stream: Optional[int] = None) -> None:
    """The decode step with the short convolutions in front (see
    kda_decode_conv in include/kda.h): x_q, x_k [1, T, H, dk] and x_v
    [1, T, HV, dv] pre-convolution inputs; taps w_* [K, C]; windows win_*
    [N, K-1, C] (updated in place); q_conv, k_conv [1, T, H, dk] receive the
    convolved q and k (they may be x_q and x_k themselves)."""
    library()
    tensors = (out, x_q, x_k, x_v, w_q, w_k, w_v, win_q, win_k, win_v, q_conv, k_conv, raw_gate,
               beta_logits, a_log, dt_bias, cu_seqlens, state_pool, state_indices)
    _call(_CONV, "kda_decode_conv", tensors, ("out",) + CONV_FIELDS + CONV_REST, _device(out, "out"), stream,
          gate_mode, lower_bound, l2_eps, scale, state_layout)


def gdr_decode(out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool,
               state_indices, *, gate_mode="softplus", lower_bound=0.0, l2_eps=0.0, scale=0.0,
               state_layout="k_first", stream: Optional[int] = None) -> None:
    """The gated delta rule with one decay per (token, value head)
    (kda_gdr_decode in include/kda.h): as :func:`decode`, with raw_gate
    [1, T, HV] and dt_bias [HV]."""
    _recurrence("kda_gdr_decode",
                (out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool, state_indices),
                gate_mode, lower_bound, l2_eps, scale, state_layout, stream)


def gdr_prefill(out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool,
                state_indices, *, gate_mode="softplus", lower_bound=0.0, l2_eps=0.0, scale=0.0,
                state_layout="k_first", stream: Optional[int] = None) -> None:
    """:func:`gdr_decode` for whole prompts (kda_gdr_prefill in
    include/kda.h): same tensors and result."""
    _recurrence("kda_gdr_prefill",
                (out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool, state_indices),
                gate_mode, lower_bound, l2_eps, scale, state_layout, stream)


_WINDOW_NAMES = ARG_NAMES + tuple(f"replay {n}" for n in REPLAY_FIELDS)


def decode_window(out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool,
                  state_indices, replay_k, replay_v, replay_gate, replay_beta, replay_begin,
                  replay_count, *, gate_mode="softplus", lower_bound=0.0, l2_eps=0.0, scale=0.0,
                  state_layout="k_first", stream: Optional[int] = None) -> None:
    """A window of drafted tokens (kda_decode_window in include/kda.h): the
    state of request b first advances by rows replay_begin[b] ..
    + replay_count[b] of the replay tensors and is written; then the window
    runs from there, with outputs, and leaves the pool alone.  raw_gate is
    [1, T, HV, dk] with dt_bias [HV, dk], or [1, T, HV] with dt_bias [HV].

    A serving loop passes the previous call's k, v, raw_gate and beta_logits
    with its ``cu_seqlens[:-1]`` and the ``n_commit`` of :func:`verify`."""
    library()
    tensors = (out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool, state_indices,
               replay_k, replay_v, replay_gate, replay_beta, replay_begin, replay_count)
    _call(_WINDOW, "kda_decode_window", tensors, _WINDOW_NAMES, _device(q, "q"), stream, gate_mode, lower_bound,
          l2_eps, scale, state_layout)


VERIFY_NAMES = ("n_commit", "next_token", "target_probs", "draft_probs", "tokens", "u_accept",
                "u_sample", "cu_seqlens", "workspace")


def verify_workspace(B: int, V: int) -> int:
    """Floats of :func:`verify`'s workspace for B requests over V tokens."""
    return 2 * B * (V // KDA_VERIFY_SEGMENT + 2)


def verify(n_commit, next_token, target_probs, draft_probs, tokens, u_accept, u_sample, cu_seqlens,
           *, workspace=None, stream: Optional[int] = None) -> None:
    """Which drafted tokens of each request's window stand, and the token that
    follows them (kda_verify in include/kda.h): n_commit [B] and next_token
    [B] (int32) are written.  target_probs and draft_probs are [T, V]; None
    for draft_probs: the drafts were certain.  ``workspace`` (float32, at
    least ``verify_workspace(B, V)`` values) is taken from torch's allocator
    if not given; with ``stream`` given it has to be too, since that memory
    belongs to torch's current stream."""
    library()
    if workspace is None and stream is not None:
        raise ValueError("workspace: required with an explicit stream")
    if not hasattr(target_probs, "dim") or target_probs.dim() != 2:
        raise ValueError("target_probs: expected a [T, V] tensor")
    dev = _device(target_probs, "target_probs")
    if workspace is None:
        if not hasattr(n_commit, "numel"):
            _descriptor(n_commit, "n_commit")
        workspace = _torch.empty(max(1, verify_workspace(n_commit.numel(), target_probs.shape[1])),
                                 dtype=_torch.float32, device=target_probs.device)
    _call(_VERIFY, "kda_verify", (n_commit, next_token, target_probs, draft_probs, tokens, u_accept, u_sample,
                                  cu_seqlens, workspace), VERIFY_NAMES, dev, stream)


SSM_NAMES = ("out", "xbc", "dt", "conv_w", "conv_b", "conv_win", "a_log", "dt_bias", "d_skip", "cu_seqlens",
             "state_pool", "state_indices", "workspace")


def ssm_prefill_workspace(T: int, B: int, H: int, HV: int, dk: int, dv: int, K: int) -> int:
    """Floats of :func:`ssm_prefill`'s workspace (KDA_SSM_WORKSPACE)."""
    return ((T // KDA_SSM_CHUNK + B) * (H * (96 * dk + 1024) + 160 * HV) + B * (K - 1) * (HV * dv + 2 * H * dk)
            + (min(T // 64 * HV * dv, KDA_SSM_SPLIT * 64) + min(B * HV * dv, KDA_SSM_SPLIT * 20)) * dk
            + 2 * KDA_SSM_SPLIT + B * HV + 64)


def ssm_decode(out, xbc, dt, conv_w, conv_b, conv_win, a_log, dt_bias, d_skip, cu_seqlens, state_pool,
               state_indices, *, state_layout="k_first", stream: Optional[int] = None) -> None:
    """The selective state space scan of a batch's next tokens, with its short
    causal convolution (kda_ssm_decode in include/kda.h): xbc [1, T, C] holds
    the channels x | B | C before the convolution, dt [1, T, HV] the time steps
    before dt_bias; conv_w [K, C], conv_b [C] or None; conv_win [N, K-1, C] and
    state_pool are updated in place; d_skip [HV] or None."""
    library()
    tensors = (out, xbc, dt, conv_w, conv_b, conv_win, a_log, dt_bias, d_skip, cu_seqlens, state_pool, state_indices)
    _call(_SSM_DECODE, "kda_ssm_decode", tensors, SSM_NAMES, _device(xbc, "xbc"), stream, state_layout=state_layout)


def ssm_prefill(out, xbc, dt, conv_w, conv_b, conv_win, a_log, dt_bias, d_skip, cu_seqlens, state_pool,
                state_indices, *, state_layout="k_first", workspace=None, stream: Optional[int] = None) -> None:
    """:func:`ssm_decode` for whole prompts (kda_ssm_prefill in include/kda.h):
    same tensors and result.  ``workspace`` (float32, at least
    ``ssm_prefill_workspace(...)`` values) is taken from torch's allocator if
    not given; with ``stream`` given it has to be too, since that memory
    belongs to torch's current stream."""
    library()
    dev = _device(xbc, "xbc")
    if workspace is None:
        if stream is not None:
            raise ValueError("workspace: required with an explicit stream")
        for t, n, dims in ((out, "out", 4), (xbc, "xbc", 3), (dt, "dt", 3), (conv_w, "conv_w", 2),
                           (state_pool, "state_pool", 4), (state_indices, "state_indices", 1)):
            _descriptor(t, n)
            if t.dim() != dims:
                raise KdaError(KDA_ERR_SHAPE, "kda_ssm_prefill")
        T, C, HV, dv = xbc.shape[1], xbc.shape[2], dt.shape[2], out.shape[3]
        sl = STATE_LAYOUTS[state_layout] if isinstance(state_layout, str) else int(state_layout)
        dk = state_pool.shape[3 if sl == KDA_STATE_V_FIRST else 2]
        H = (C - HV * dv) // (2 * dk) if dk > 0 else 0
        if H < 1:
            raise KdaError(KDA_ERR_SHAPE, "kda_ssm_prefill")
        workspace = _torch.empty(ssm_prefill_workspace(T, state_indices.shape[0], H, HV, dk, dv, conv_w.shape[0]),
                                 dtype=_torch.float32, device=xbc.device)
    tensors = (out, xbc, dt, conv_w, conv_b, conv_win, a_log, dt_bias, d_skip, cu_seqlens, state_pool, state_indices,
               workspace)
    _call(_SSM_PREFILL, "kda_ssm_prefill", tensors, SSM_NAMES, dev, stream, state_layout=state_layout)


def norm_residual(hidden_out, normed, hidden, block_out, weight, *, post_weight=None, scale=None, eps=0.0,
                  stream: Optional[int] = None) -> None:
    """In front of a block (kda_norm_residual in include/kda.h): hidden_out =
    hidden + scale * block_out (``post_weight`` given: block_out normalised
    first), normed = RMS norm of that.  ``hidden_out`` may be ``hidden`` and
    ``normed`` may be ``block_out``; scale is [D], [1] or None."""
    library()
    _call(_NORM_RESIDUAL, "kda_norm_residual", (hidden_out, normed, hidden, block_out, weight, post_weight, scale),
          ("hidden_out", "normed", "hidden", "block_out", "weight", "post_weight", "scale"),
          _device(hidden, "hidden"), stream, l2_eps=eps)


def norm_gate(out, x, gate, weight, *, activation="sigmoid", gate_first=False, eps=0.0,
              stream: Optional[int] = None) -> None:
    """Behind a recurrence (kda_norm_gate in include/kda.h): the RMS norm of x
    over its last dimension times the activation of ``gate`` ("sigmoid" or
    "silu"); with ``gate_first`` x is gated before it is normalised.  weight is
    [D], or [R, D] with R x's second-last extent; ``out`` may be ``x`` or
    ``gate``."""
    library()
    act = ACTIVATIONS[activation] if isinstance(activation, str) else int(activation)
    _call(_NORM_GATE, "kda_norm_gate", (out, x, gate, weight), ("out", "x", "gate", "weight"), _device(x, "x"),
          stream, act, l2_eps=eps, matmul=int(gate_first))
