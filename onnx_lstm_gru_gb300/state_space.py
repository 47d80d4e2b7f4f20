"""The operators of selective state space and linear attention layers, on the C ABI of ``include/rk.h``.

``StateSpaceLayer`` takes torch CUDA tensors: layer normalisation, the short
causal convolution and the selective scan; queries and keys normalised and
rotated by head, and attention through a state that decays by head; each with
its gradient.  The
formulas, shapes and rules are those the header states; here only arguments
are checked and packed (by the module that ``binding/state_space_binding.cpp``
builds: a call's host time is what a single token waits for).  Row operands may be slices of wider rows, some steps
of a longer sequence or transposed views: any strides with a dense last
dimension.

Prompts and single tokens are the same calls: a step is ``seq=1`` with
``initial_state`` given and ``final_state`` asked for (or given: the same
tensor as ``initial_state`` updates it in place).
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

from . import DTYPES, RkError, load, rk_create, rk_destroy, rk_last_error, rk_launch_count, rk_status_poll, rk_tensor
from ._build import BINDING_LIB


class rk_rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("offset", ctypes.c_int64), ("length", ctypes.c_int64),
                ("pitch", ctypes.c_int64), ("outer_pitch", ctypes.c_int64)]


class rk_workspace(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("offset", ctypes.c_int64), ("length", ctypes.c_int64)]


class rk_norm_problem(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("epsilon", ctypes.c_float), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


class rk_conv_problem(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("layout", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("width", ctypes.c_int32), ("seq", ctypes.c_int64), ("batch", ctypes.c_int64),
                ("channels", ctypes.c_int64)]


class rk_scan_problem(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("layout", ctypes.c_int32), ("softplus", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("seq", ctypes.c_int64), ("batch", ctypes.c_int64),
                ("channels", ctypes.c_int64), ("state", ctypes.c_int64)]


class rk_qk_problem(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("layout", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("rotary", ctypes.c_int32), ("epsilon", ctypes.c_float),
                ("seq", ctypes.c_int64), ("batch", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("key_heads", ctypes.c_int64), ("size", ctypes.c_int64)]


class rk_attn_problem(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("layout", ctypes.c_int32), ("scale", ctypes.c_float),
                ("query_heads", ctypes.c_int32), ("key_heads", ctypes.c_int32), ("value_heads", ctypes.c_int32),
                ("seq", ctypes.c_int64), ("batch", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("key_size", ctypes.c_int64), ("value_size", ctypes.c_int64)]


# Operand lists in the C structs' order: row tensors, then the others.
_OPERANDS = {
    "norm": (("X", "Y"), ("Scale", "B", "Mean", "InvStdDev")),
    "norm_grad": (("X", "dY", "dX"), ("Scale", "Mean", "InvStdDev", "dScale", "dB")),
    "conv": (("X", "Y"), ("W", "B", "sequence_lens", "initial_state", "final_state")),
    "conv_grad": (("X", "dY", "dX"), ("W", "B", "sequence_lens", "initial_state", "d_final_state", "dW", "dB",
                                       "d_initial_state")),
    "scan": (("X", "Delta", "B", "C", "Z", "Y"),
             ("A", "D", "delta_bias", "sequence_lens", "initial_state", "final_state")),
    "scan_grad": (("X", "Delta", "B", "C", "Z", "dY", "dX", "dDelta", "dB", "dC", "dZ"),
                  ("A", "D", "delta_bias", "sequence_lens", "initial_state", "d_final_state", "dA", "dD",
                   "d_delta_bias", "d_initial_state")),
    "qk": (("Q", "K", "YQ", "YK"), ("QScale", "KScale", "Frequencies", "positions", "sequence_lens")),
    "qk_grad": (("Q", "K", "dYQ", "dYK", "dQ", "dK"),
                ("QScale", "KScale", "Frequencies", "positions", "sequence_lens", "dQScale", "dKScale")),
    "attn": (("Q", "K", "V", "Decay", "Y"), ("decay_bias", "sequence_lens", "initial_state", "final_state")),
    "attn_grad": (("Q", "K", "V", "Decay", "dY", "dQ", "dK", "dV", "dDecay"),
                  ("decay_bias", "sequence_lens", "initial_state", "d_final_state", "d_decay_bias",
                   "d_initial_state")),
}


def _operand_struct(op):
    rows, tensors = _OPERANDS[op]
    fields = [(n, rk_rows) for n in rows] + [(n, rk_tensor) for n in tensors]
    return type(f"rk_{op}_operands", (ctypes.Structure,), {"_fields_": fields})


rk_norm_operands = _operand_struct("norm")
rk_norm_grad_operands = _operand_struct("norm_grad")
rk_conv_operands = _operand_struct("conv")
rk_conv_grad_operands = _operand_struct("conv_grad")
rk_scan_operands = _operand_struct("scan")
rk_scan_grad_operands = _operand_struct("scan_grad")
rk_qk_operands = _operand_struct("qk")
rk_qk_grad_operands = _operand_struct("qk_grad")
rk_attn_operands = _operand_struct("attn")
rk_attn_grad_operands = _operand_struct("attn_grad")

_P = ctypes.c_void_p
SIGNATURES = {
    "rk_norm_grad_scratch_length": (ctypes.c_int64, [_P]),
    "rk_conv_grad_scratch_length": (ctypes.c_int64, [_P]),
    "rk_scan_scratch_length": (ctypes.c_int64, [_P]),
    "rk_scan_grad_scratch_length": (ctypes.c_int64, [_P]),
    "rk_qk_grad_scratch_length": (ctypes.c_int64, [_P]),
    "rk_attn_scratch_length": (ctypes.c_int64, [_P]),
    "rk_attn_grad_scratch_length": (ctypes.c_int64, [_P]),
    "rk_attn_grad_scratch_needed": (ctypes.c_int64, [_P, _P]),
    "rk_norm_encode": (ctypes.c_int32, [_P, _P, _P, _P]),
    "rk_norm_grad_encode": (ctypes.c_int32, [_P, _P, _P, _P, _P]),
    "rk_conv_encode": (ctypes.c_int32, [_P, _P, _P, _P]),
    "rk_conv_grad_encode": (ctypes.c_int32, [_P, _P, _P, _P, _P]),
    "rk_scan_encode": (ctypes.c_int32, [_P, _P, _P, _P, _P]),
    "rk_scan_grad_encode": (ctypes.c_int32, [_P, _P, _P, _P, _P]),
    "rk_qk_encode": (ctypes.c_int32, [_P, _P, _P, _P]),
    "rk_qk_grad_encode": (ctypes.c_int32, [_P, _P, _P, _P, _P]),
    "rk_attn_encode": (ctypes.c_int32, [_P, _P, _P, _P, _P]),
    "rk_attn_grad_encode": (ctypes.c_int32, [_P, _P, _P, _P, _P]),
}


# ---- thin wrappers with the C names (argument marshalling only) ----------------------------

def _ref(x):
    return ctypes.byref(x) if x is not None else None


def rk_norm_grad_scratch_length(problem: rk_norm_problem) -> int:
    return load().rk_norm_grad_scratch_length(_ref(problem))


def rk_conv_grad_scratch_length(problem: rk_conv_problem) -> int:
    return load().rk_conv_grad_scratch_length(_ref(problem))


def rk_scan_scratch_length(problem: rk_scan_problem) -> int:
    return load().rk_scan_scratch_length(_ref(problem))


def rk_scan_grad_scratch_length(problem: rk_scan_problem) -> int:
    return load().rk_scan_grad_scratch_length(_ref(problem))


def rk_qk_grad_scratch_length(problem: rk_qk_problem) -> int:
    return load().rk_qk_grad_scratch_length(_ref(problem))


def rk_attn_scratch_length(problem: rk_attn_problem) -> int:
    return load().rk_attn_scratch_length(_ref(problem))


def rk_attn_grad_scratch_length(problem: rk_attn_problem) -> int:
    return load().rk_attn_grad_scratch_length(_ref(problem))


def rk_attn_grad_scratch_needed(problem: rk_attn_problem, ops: rk_attn_grad_operands) -> int:
    return load().rk_attn_grad_scratch_needed(_ref(problem), _ref(ops))


def rk_norm_encode(handle, problem, ops, stream) -> int:
    return load().rk_norm_encode(handle, _ref(problem), _ref(ops), stream)


def rk_norm_grad_encode(handle, problem, ops, scratch, stream) -> int:
    return load().rk_norm_grad_encode(handle, _ref(problem), _ref(ops), _ref(scratch), stream)


def rk_conv_encode(handle, problem, ops, stream) -> int:
    return load().rk_conv_encode(handle, _ref(problem), _ref(ops), stream)


def rk_conv_grad_encode(handle, problem, ops, scratch, stream) -> int:
    return load().rk_conv_grad_encode(handle, _ref(problem), _ref(ops), _ref(scratch), stream)


def rk_scan_encode(handle, problem, ops, scratch, stream) -> int:
    return load().rk_scan_encode(handle, _ref(problem), _ref(ops), _ref(scratch), stream)


def rk_scan_grad_encode(handle, problem, ops, scratch, stream) -> int:
    return load().rk_scan_grad_encode(handle, _ref(problem), _ref(ops), _ref(scratch), stream)


def rk_qk_encode(handle, problem, ops, stream) -> int:
    return load().rk_qk_encode(handle, _ref(problem), _ref(ops), stream)


def rk_qk_grad_encode(handle, problem, ops, scratch, stream) -> int:
    return load().rk_qk_grad_encode(handle, _ref(problem), _ref(ops), _ref(scratch), stream)


def rk_attn_encode(handle, problem, ops, scratch, stream) -> int:
    return load().rk_attn_encode(handle, _ref(problem), _ref(ops), _ref(scratch), stream)


def rk_attn_grad_encode(handle, problem, ops, scratch, stream) -> int:
    return load().rk_attn_grad_encode(handle, _ref(problem), _ref(ops), _ref(scratch), stream)


# ---- problem descriptions ----------------------------------------------------------------------

@functools.lru_cache(maxsize=None)
def _binding():
    """The built module that packs operands."""
    import importlib.machinery
    import importlib.util
    import torch  # noqa: F401  (the module links against its libraries)
    if not os.path.exists(BINDING_LIB):
        raise RuntimeError(f"{BINDING_LIB} missing: run onnx_lstm_gru_gb300.build() where torch is installed")
    loader = importlib.machinery.ExtensionFileLoader("state_space_binding", BINDING_LIB)
    spec = importlib.util.spec_from_file_location("state_space_binding", BINDING_LIB, loader=loader)
    module = importlib.util.module_from_spec(spec)
    loader.exec_module(module)
    return module


class _Problem:
    """What the problems share."""

    def shapes(self) -> dict:
        return {n: s for n, (s, _) in self._operands().items()}

    def _plan(self, op):
        plans = self.__dict__.get("_plans")
        if plans is None:
            plans = self.__dict__["_plans"] = {}
        plan = plans.get(op)
        if plan is None:
            plan = plans[op] = _plan(op, self)
        return plan

    def __getstate__(self):
        # the plans belong to this process: a copy finds its own
        return {k: v for k, v in self.__dict__.items() if k != "_plans"}


# element types of operands: the problem's ("t"), float32 ("f"), int32 ("i")
@dataclass(frozen=True)
class NormProblem(_Problem):
    """Layer normalisation of ``rows`` rows of ``cols`` elements (mirrors rk_norm_problem)."""
    rows: int
    cols: int
    dtype: str = "f32"
    epsilon: float = 1e-5

    def to_c(self) -> rk_norm_problem:
        return rk_norm_problem(DTYPES[self.dtype], self.epsilon, self.rows, self.cols)

    def _operands(self):
        row, col, one = (self.rows, self.cols), (self.cols,), (self.rows,)
        return {"X": (row, "t"), "Y": (row, "t"), "dY": (row, "t"), "dX": (row, "t"),
                "Scale": (col, "t"), "B": (col, "t"), "dScale": (col, "f"), "dB": (col, "f"),
                "Mean": (one, "f"), "InvStdDev": (one, "f")}


def _row_shape(layout, seq, batch, inner):
    return (seq, batch, inner) if layout == 0 else (batch, seq, inner)


@dataclass(frozen=True)
class ConvProblem(_Problem):
    """Causal convolution (mirrors rk_conv_problem); ``activation`` is "silu" or "none"."""
    seq: int
    batch: int
    channels: int
    width: int = 4
    dtype: str = "f32"
    layout: int = 0
    activation: str = "silu"

    def to_c(self) -> rk_conv_problem:
        return rk_conv_problem(DTYPES[self.dtype], self.layout, {"none": 0, "silu": 1}[self.activation], self.width,
                               self.seq, self.batch, self.channels)

    def _operands(self):
        row = _row_shape(self.layout, self.seq, self.batch, self.channels)
        state, col = (self.batch, self.width - 1, self.channels), (self.channels,)
        taps = (self.channels, self.width)
        return {"X": (row, "t"), "Y": (row, "t"), "dY": (row, "t"), "dX": (row, "t"),
                "W": (taps, "t"), "B": (col, "t"), "dW": (taps, "f"), "dB": (col, "f"),
                "sequence_lens": ((self.batch,), "i"), "initial_state": (state, "t"), "final_state": (state, "t"),
                "d_initial_state": (state, "t"), "d_final_state": (state, "t")}


@dataclass(frozen=True)
class ScanProblem(_Problem):
    """Selective scan (mirrors rk_scan_problem)."""
    seq: int
    batch: int
    channels: int
    state: int
    groups: int = 1
    dtype: str = "f32"
    layout: int = 0
    softplus: bool = True

    def to_c(self) -> rk_scan_problem:
        return rk_scan_problem(DTYPES[self.dtype], self.layout, int(self.softplus), self.groups, self.seq, self.batch,
                               self.channels, self.state)

    def _operands(self):
        row = _row_shape(self.layout, self.seq, self.batch, self.channels)
        mix = _row_shape(self.layout, self.seq, self.batch, self.groups * self.state)
        rates, col = (self.channels, self.state), (self.channels,)
        state = (self.batch, self.channels, self.state)
        names = {n: (row, "t") for n in ("X", "Delta", "Z", "Y", "dY", "dX", "dDelta", "dZ")}
        names.update({n: (mix, "t") for n in ("B", "C", "dB", "dC")})
        names.update({n: (state, "f") for n in ("initial_state", "final_state", "d_initial_state", "d_final_state")})
        names.update({"A": (rates, "f"), "dA": (rates, "f"), "D": (col, "f"), "dD": (col, "f"),
                      "delta_bias": (col, "f"), "d_delta_bias": (col, "f"), "sequence_lens": ((self.batch,), "i")})
        return names


@dataclass(frozen=True)
class QkProblem(_Problem):
    """Queries and keys normalised and rotated by head (mirrors rk_qk_problem).  ``key_heads``: as many as ``heads``
    unless given; ``norm`` is "rms", "l2" or "none"; the first ``rotary`` elements of a head are rotated, in pairs of
    neighbours where ``interleaved``."""
    seq: int
    batch: int
    heads: int
    size: int
    key_heads: int | None = None
    rotary: int = 0
    interleaved: bool = False
    norm: str = "rms"
    epsilon: float = 1e-6
    dtype: str = "f32"
    layout: int = 0

    @property
    def _key_heads(self):
        return self.heads if self.key_heads is None else self.key_heads

    def to_c(self) -> rk_qk_problem:
        return rk_qk_problem(DTYPES[self.dtype], self.layout, {"none": 0, "rms": 1, "l2": 2}[self.norm],
                             int(self.interleaved), self.rotary, self.epsilon, self.seq, self.batch, self.heads,
                             self._key_heads, self.size)

    def _operands(self):
        q = _row_shape(self.layout, self.seq, self.batch, self.heads * self.size)
        k = _row_shape(self.layout, self.seq, self.batch, self._key_heads * self.size)
        one = (self.size,)
        names = {n: (q, "t") for n in ("Q", "YQ", "dYQ", "dQ")}
        names.update({n: (k, "t") for n in ("K", "YK", "dYK", "dK")})
        names.update({"QScale": (one, "t"), "KScale": (one, "t"), "dQScale": (one, "f"), "dKScale": (one, "f"),
                      "Frequencies": ((self.rotary // 2,), "f"),
                      "positions": (q[:2], "i"), "sequence_lens": ((self.batch,), "i")})
        return names


@dataclass(frozen=True)
class AttnProblem(_Problem):
    """Attention through a state that decays by head (mirrors rk_attn_problem).  ``query_heads``, ``key_heads``,
    ``value_heads``: as many as ``heads`` unless given; ``scale``: 1 / sqrt(key_size) unless given."""
    seq: int
    batch: int
    heads: int
    key_size: int
    value_size: int
    query_heads: int | None = None
    key_heads: int | None = None
    value_heads: int | None = None
    scale: float | None = None
    dtype: str = "f32"
    layout: int = 0

    def _shared(self):
        return [self.heads if n is None else n for n in (self.query_heads, self.key_heads, self.value_heads)]

    def to_c(self) -> rk_attn_problem:
        scale = self.scale if self.scale is not None else self.key_size ** -0.5 if self.key_size > 0 else 1.0
        # 0 heads given here are none; in the C structure 0 stands for as many as heads
        shared = [-1 if n == 0 else n for n in self._shared()]
        return rk_attn_problem(DTYPES[self.dtype], self.layout, scale, *shared, self.seq, self.batch, self.heads,
                               self.key_size, self.value_size)

    def _operands(self):
        def row(heads, size):
            return _row_shape(self.layout, self.seq, self.batch, heads * size)
        qh, kh, vh = self._shared()
        state, one = (self.batch, self.heads, self.key_size, self.value_size), (self.heads,)
        names = {n: (row(qh, self.key_size), "t") for n in ("Q", "dQ")}
        names.update({n: (row(kh, self.key_size), "t") for n in ("K", "dK")})
        names.update({n: (row(vh, self.value_size), "t") for n in ("V", "dV")})
        names.update({n: (row(self.heads, self.value_size), "t") for n in ("Y", "dY")})
        names.update({n: (row(self.heads, 1), "f") for n in ("Decay", "dDecay")})
        names.update({n: (state, "f") for n in ("initial_state", "final_state", "d_initial_state", "d_final_state")})
        names.update({"decay_bias": (one, "f"), "d_decay_bias": (one, "f"), "sequence_lens": ((self.batch,), "i")})
        return names


_REQUIRED = {
    "norm": ("X",), "norm_grad": ("X", "Mean", "InvStdDev", "dY"), "conv": ("X", "W"), "conv_grad": ("X", "W", "dY"),
    "scan": ("X", "Delta", "A", "B", "C"), "scan_grad": ("X", "Delta", "A", "B", "C", "dY"),
    "qk": ("Q", "K"), "qk_grad": ("Q", "K", "dYQ", "dYK"), "attn": ("Q", "K", "V"), "attn_grad": ("Q", "K", "V", "dY"),
}
_OUTPUTS = {
    "norm": ("Y", "Mean", "InvStdDev"), "norm_grad": ("dX", "dScale", "dB"), "conv": ("Y", "final_state"),
    "conv_grad": ("dX", "dW", "dB", "d_initial_state"), "scan": ("Y", "final_state"),
    "scan_grad": ("dX", "dDelta", "dB", "dC", "dZ", "dA", "dD", "d_delta_bias", "d_initial_state"),
    "qk": ("YQ", "YK"), "qk_grad": ("dQ", "dK", "dQScale", "dKScale"), "attn": ("Y", "final_state"),
    "attn_grad": ("dQ", "dK", "dV", "dDecay", "d_decay_bias", "d_initial_state"),
}


@functools.lru_cache(maxsize=256)
def _plan(op, problem):
    """How one operator's operands of one problem are packed (equal problems share it)."""
    codes = {"t": DTYPES[problem.dtype], "f": 0, "i": 3}
    operands = problem._operands()
    rows, tensors = _OPERANDS[op]
    entries, at = [], 0
    for names, is_rows, words in ((rows, True, 5), (tensors, False, 3)):
        for name in names:
            shape, kind = operands[name]
            entries.append((name, at, is_rows, name in _REQUIRED[op], name in _OUTPUTS[op], codes[kind], shape))
            at += words
    lib = load()
    c = problem.to_c()
    length = getattr(lib, f"rk_{op}_scratch_length", None)
    encode = ctypes.cast(getattr(lib, f"rk_{op}_encode"), ctypes.c_void_p).value
    # a problem that the entry will refuse has no scratch length: its message says why
    scratch = -1 if length is None else max(length(ctypes.byref(c)), 0)
    # less where the call wants less
    needed = getattr(lib, f"rk_{op}_scratch_needed", None)
    return _binding().Plan(encode, bytes(c), scratch, entries,
                           ctypes.cast(needed, ctypes.c_void_p).value if needed is not None else 0)


class StateSpaceLayer:
    """Owns an rk handle.  Every method enqueues one operator on the current
    torch stream (or ``stream``) and returns the outputs named in ``want``,
    allocated unless they are passed by name (an input cannot be wanted that
    was not passed).  Scratch comes from torch's allocator, so calls may run on
    any stream and be captured into a graph.  Like the recurrent layer's, the
    outputs carry no autograd history, also of tensors that require gradients:
    the gradients are methods of their own, which ``examples/state_space_layer.py``
    ties into ``torch.autograd.Function``.  A problem that is kept saves a
    decoding step the look-up of an equal one.  No CPU path exists."""

    def __init__(self, flags: int = 0):
        load()
        self.handle = rk_create(flags)

    def close(self):
        if getattr(self, "handle", None):
            rk_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def launches(self) -> int:
        return rk_launch_count(self.handle)

    def poll(self, stream=None):
        """Synchronises the stream (None: torch's current one); an RkError if a wait of the linear attention in chunks
        gave up on its device since the last poll: the outputs from before are then undefined."""
        import torch
        s = stream if stream is not None else torch.cuda.current_stream()
        with torch.cuda.device(s.device):
            st = rk_status_poll(self.handle, s.cuda_stream)
        if st != 0:
            raise RkError(st, rk_last_error(self.handle))

    def norm(self, problem: NormProblem, X, want=("Y", "Mean", "InvStdDev"), stream=None, **tensors) -> dict:
        """Y, Mean, InvStdDev from X, Scale, B."""
        return self._run("norm", NormProblem, problem, X, want, stream, tensors)

    def norm_grad(self, problem: NormProblem, X, want=("dX", "dScale", "dB"), stream=None, **tensors) -> dict:
        """dX, dScale, dB from X, Scale, Mean, InvStdDev, dY."""
        return self._run("norm_grad", NormProblem, problem, X, want, stream, tensors)

    def conv(self, problem: ConvProblem, X, want=("Y", "final_state"), stream=None, **tensors) -> dict:
        """Y, final_state from X, W, B, sequence_lens, initial_state."""
        return self._run("conv", ConvProblem, problem, X, want, stream, tensors)

    def conv_grad(self, problem: ConvProblem, X, want=("dX", "dW", "dB"), stream=None, **tensors) -> dict:
        """dX, dW, dB, d_initial_state from conv's operands, dY and d_final_state."""
        return self._run("conv_grad", ConvProblem, problem, X, want, stream, tensors)

    def scan(self, problem: ScanProblem, X, want=("Y", "final_state"), stream=None, **tensors) -> dict:
        """Y, final_state from X, Delta, A, B, C, D, Z, delta_bias, sequence_lens, initial_state."""
        return self._run("scan", ScanProblem, problem, X, want, stream, tensors)

    def scan_grad(self, problem: ScanProblem, X,
                  want=("dX", "dDelta", "dA", "dB", "dC", "dD", "d_delta_bias"), stream=None, **tensors) -> dict:
        """dX, dDelta, dA, dB, dC, dD, d_delta_bias, dZ, d_initial_state from scan's operands, dY and d_final_state."""
        return self._run("scan_grad", ScanProblem, problem, X, want, stream, tensors)

    def qk(self, problem: QkProblem, Q, want=("YQ", "YK"), stream=None, **tensors) -> dict:
        """YQ, YK from Q, K, QScale, KScale, Frequencies, positions, sequence_lens."""
        return self._run("qk", QkProblem, problem, Q, want, stream, tensors)

    def qk_grad(self, problem: QkProblem, Q, want=("dQ", "dK", "dQScale", "dKScale"), stream=None, **tensors) -> dict:
        """dQ, dK, dQScale, dKScale from qk's operands, dYQ and dYK."""
        return self._run("qk_grad", QkProblem, problem, Q, want, stream, tensors)

    def attn(self, problem: AttnProblem, Q, want=("Y", "final_state"), stream=None, **tensors) -> dict:
        """Y, final_state from Q, K, V, Decay, decay_bias, sequence_lens, initial_state."""
        return self._run("attn", AttnProblem, problem, Q, want, stream, tensors)

    def attn_grad(self, problem: AttnProblem, Q, want=("dQ", "dK", "dV"), stream=None, **tensors) -> dict:
        """dQ, dK, dV, dDecay, d_decay_bias, d_initial_state from attn's operands, dY and d_final_state."""
        return self._run("attn_grad", AttnProblem, problem, Q, want, stream, tensors)

    def _run(self, op, kind, problem, X, want, stream, tensors):
        if type(problem) is not kind:
            raise TypeError(f"{op}: expected {kind.__name__}, got {type(problem).__name__}")
        if stream is not None:
            import torch
            if stream != torch.cuda.current_stream(X.device):
                # memory made here belongs to that stream; what the caller passes is
                # kept from reuse until the stream is past this call
                with torch.cuda.stream(stream):
                    out = self._run(op, kind, problem, X, want, None, tensors)
                for t in (X, *tensors.values()):
                    if t is not None:
                        t.record_stream(stream)
                return out
        out = problem._plan(op).run(self.handle, X, want, tensors)
        if type(out) is int:
            raise RkError(out, rk_last_error(self.handle))
        return out
