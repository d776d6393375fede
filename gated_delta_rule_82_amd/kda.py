"""Thin ctypes binding of libkda (argument marshalling only).

Every step of the decode and of the chunked prefill runs in the HIP library; this module turns torch
device tensors into ``kda_tensor`` descriptors, passes the current HIP stream
and raises :class:`KdaError` on a nonzero status.  There is no fallback: if
the library is missing or a tensor is not on a GPU, the call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "lib", "libkda.so")

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

EXPORTED_SYMBOLS = ("kda_decode", "kda_decode_conv", "kda_prefill", "kda_gdr_decode",
                    "kda_gdr_prefill", "kda_decode_window", "kda_verify", "kda_check_host",
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
_DTYPES = {}           # torch dtype -> kda_dtype


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
    _DTYPES.update({torch.float32: KDA_F32, torch.bfloat16: KDA_BF16, torch.int32: KDA_I32})
    # the current stream's handle without a Stream object (microseconds of a short call)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    lib = ctypes.CDLL(LIB_PATH, mode=ctypes.RTLD_LOCAL)
    # tensors and structs go by address: of a ctypes structure, or of packed
    # descriptors (see _pack)
    P = ctypes.c_void_p
    lib.kda_decode.argtypes = [P] * 13
    lib.kda_decode.restype = ctypes.c_int
    lib.kda_decode_conv.argtypes = [P] * 11
    lib.kda_decode_conv.restype = ctypes.c_int
    lib.kda_prefill.argtypes = [P] * 12 + [ctypes.c_int32, P]
    lib.kda_prefill.restype = ctypes.c_int
    for fn in (lib.kda_gdr_decode, lib.kda_gdr_prefill):
        fn.argtypes = [P] * 13
        fn.restype = ctypes.c_int
    lib.kda_decode_window.argtypes = [P] * 14
    lib.kda_decode_window.restype = ctypes.c_int
    lib.kda_verify.argtypes = [P] * 10
    lib.kda_verify.restype = ctypes.c_int
    lib.kda_check_host.argtypes = [ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32),
                                   ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]
    lib.kda_check_host.restype = ctypes.c_int
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_abi_version.argtypes = []
    lib.kda_abi_version.restype = ctypes.c_int
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
# the call path: descriptors are packed straight into one buffer per call (a
# decode step of one user takes a few microseconds on the GPU, and building
# ctypes structures for 11 tensors took 20)
# ---------------------------------------------------------------------------

_TENSOR = struct.Struct("=Qii4q")     # kda_tensor
_MODE = struct.Struct("=ifffi")       # kda_mode
assert _TENSOR.size == ctypes.sizeof(KdaTensor) and _MODE.size == ctypes.sizeof(KdaMode)
_TENSORS = {n: struct.Struct("=" + "Qii4q" * n) for n in range(1, 20)}
_BUFFERS = {n: ctypes.c_char * (n * _TENSOR.size + _MODE.size) for n in range(1, 20)}


def _refuse(tensors, names, dev):
    """Say what is wrong with the tensors of a call that _pack stopped at."""
    for t, n in zip(tensors, names):
        _descriptor(t, n)
    for t, n in zip(tensors, names):
        if t.device.index != dev:
            raise ValueError(f"{n}: on {t.device}, expected cuda:{dev}")
    raise ValueError("a tensor cannot be passed to libkda")


def _pack(tensors, names, dev):
    """kda_tensor descriptors of ``tensors``, all on GPU ``dev``, one behind
    the other, with room for a kda_mode.  Returns the buffer and its address."""
    values = []
    add = values.extend
    try:
        for t in tensors:
            shape = t.shape
            n = len(shape)
            dt = _DTYPES.get(t.dtype)
            if dt is None or n > 4 or t.get_device() != dev or not t.is_contiguous():
                _refuse(tensors, names, dev)
            if n == 4:
                add((t.data_ptr(), dt, 4, *shape))
            else:
                add((t.data_ptr(), dt, n, *shape, 0, 0, 0, 0)[:7])
    except AttributeError:
        _refuse(tensors, names, dev)
    buf = _BUFFERS[len(tensors)]()
    _TENSORS[len(tensors)].pack_into(buf, 0, *values)
    return buf, ctypes.addressof(buf)


def _device(t, name):
    """Index of the GPU that ``t`` is on."""
    if not hasattr(t, "get_device") or t.get_device() < 0:
        _descriptor(t, name)
    return t.get_device()


def _pack_mode(buf, n, gate_mode, lower_bound, l2_eps, scale, state_layout):
    """kda_mode behind n descriptors."""
    at = n * _TENSOR.size
    gm = GATE_MODES[gate_mode] if isinstance(gate_mode, str) else int(gate_mode)
    sl = STATE_LAYOUTS[state_layout] if isinstance(state_layout, str) else int(state_layout)
    try:
        _MODE.pack_into(buf, at, gm, lower_bound, l2_eps, scale, sl)
    except OverflowError:   # past fp32: infinite, as ctypes has it
        mode = make_mode(gm, lower_bound, l2_eps, scale, sl)
        ctypes.memmove(ctypes.addressof(buf) + at, ctypes.addressof(mode), _MODE.size)


def _call(fn, args, dev, stream, where, tail=()):
    """Call ``fn`` with GPU ``dev`` current, on ``stream`` or torch's current one."""
    if _torch.cuda.current_device() != dev:
        with _torch.cuda.device(dev):
            return _call(fn, args, dev, stream, where, tail)
    rc = fn(*args, *tail, _raw_stream(dev) if stream is None else stream)
    if rc != KDA_OK:
        raise KdaError(rc, where)


def _recurrence(fn, where, tensors, gate_mode, lower_bound, l2_eps, scale, state_layout, stream, tail=()):
    """The calls that take the 11 tensors of kda_decode and a mode."""
    dev = _device(tensors[1], "q")
    buf, at = _pack(tensors, ARG_NAMES, dev)
    _pack_mode(buf, 11, gate_mode, lower_bound, l2_eps, scale, state_layout)
    _call(fn, range(at, at + 12 * 48, 48), dev, stream, where, tail)


def decode(out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool,
           state_indices, *, gate_mode="softplus", lower_bound=0.0, l2_eps=0.0, scale=0.0,
           state_layout="k_first", stream: Optional[int] = None) -> None:
    """Advance the KDA decode recurrence in place (see include/kda.h).

    Tensors are torch GPU tensors with the shapes of kda.h; ``out`` and
    ``state_pool`` are written.  ``state_pool`` is float32 or bfloat16, laid
    out [N, HV, dk, dv] ("k_first") or [N, HV, dv, dk] ("v_first").  The work
    is enqueued on ``stream`` (a raw hipStream_t handle; default: torch's
    current stream of q's device)."""
    _recurrence(library().kda_decode, "kda_decode",
                (out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool, state_indices),
                gate_mode, lower_bound, l2_eps, scale, state_layout, stream)


def prefill(out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool,
            state_indices, *, gate_mode="softplus", lower_bound=0.0, l2_eps=0.0, scale=0.0,
            state_layout="k_first", matmul="split_bf16", stream: Optional[int] = None) -> None:
    """The recurrence over long requests in chunks of 16 tokens on the matrix
    cores (kda_prefill in include/kda.h): same tensors and result as
    :func:`decode`; ``matmul`` is "split_bf16" (default) or "f32"."""
    mm = MATMULS[matmul] if isinstance(matmul, str) else int(matmul)
    _recurrence(library().kda_prefill, "kda_prefill",
                (out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool, state_indices),
                gate_mode, lower_bound, l2_eps, scale, state_layout, stream, (mm,))


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
    fn = library().kda_decode_conv
    tensors = (out, x_q, x_k, x_v, w_q, w_k, w_v, win_q, win_k, win_v, q_conv, k_conv, raw_gate,
               beta_logits, a_log, dt_bias, cu_seqlens, state_pool, state_indices)
    dev = _device(out, "out")
    buf, at = _pack(tensors, ("out",) + CONV_FIELDS + CONV_REST, dev)
    _pack_mode(buf, 19, gate_mode, lower_bound, l2_eps, scale, state_layout)
    # out, the kda_conv (11 descriptors), the 7 others and the mode
    _call(fn, (at, at + 48, *range(at + 12 * 48, at + 20 * 48, 48)), dev, stream, "kda_decode_conv")


def gdr_decode(out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool,
               state_indices, *, gate_mode="softplus", lower_bound=0.0, l2_eps=0.0, scale=0.0,
               state_layout="k_first", stream: Optional[int] = None) -> None:
    """The gated delta rule with one decay per (token, value head)
    (kda_gdr_decode in include/kda.h): as :func:`decode`, with raw_gate
    [1, T, HV] and dt_bias [HV]."""
    _recurrence(library().kda_gdr_decode, "kda_gdr_decode",
                (out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool, state_indices),
                gate_mode, lower_bound, l2_eps, scale, state_layout, stream)


def gdr_prefill(out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool,
                state_indices, *, gate_mode="softplus", lower_bound=0.0, l2_eps=0.0, scale=0.0,
                state_layout="k_first", stream: Optional[int] = None) -> None:
    """:func:`gdr_decode` for whole prompts (kda_gdr_prefill in
    include/kda.h): same tensors and result."""
    _recurrence(library().kda_gdr_prefill, "kda_gdr_prefill",
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
    fn = library().kda_decode_window
    tensors = (out, q, k, v, raw_gate, beta_logits, a_log, dt_bias, cu_seqlens, state_pool, state_indices,
               replay_k, replay_v, replay_gate, replay_beta, replay_begin, replay_count)
    dev = _device(q, "q")
    buf, at = _pack(tensors, _WINDOW_NAMES, dev)
    _pack_mode(buf, 17, gate_mode, lower_bound, l2_eps, scale, state_layout)
    # 11 tensors, the kda_replay (6 descriptors) and the mode
    _call(fn, (*range(at, at + 12 * 48, 48), at + 17 * 48), dev, stream, "kda_decode_window")


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
    fn = library().kda_verify
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
    # no draft probabilities: any tensor holds their place, and NULL is passed
    tensors = (n_commit, next_token, target_probs, target_probs if draft_probs is None else draft_probs,
               tokens, u_accept, u_sample, cu_seqlens, workspace)
    buf, at = _pack(tensors, VERIFY_NAMES, dev)
    args = list(range(at, at + 9 * 48, 48))
    if draft_probs is None:
        args[3] = None
    _call(fn, args, dev, stream, "kda_verify")
