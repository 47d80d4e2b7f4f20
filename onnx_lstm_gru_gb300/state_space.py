"""The operators of a selective state space layer, on the C ABI of ``include/rk.h``.

``StateSpaceLayer`` takes torch CUDA tensors: layer normalisation, the short
causal convolution and the selective scan, each with its gradient.  The
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

from . import DTYPES, RkError, load, rk_create, rk_destroy, rk_last_error, rk_launch_count, rk_tensor
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

_P = ctypes.c_void_p
SIGNATURES = {
    "rk_norm_grad_scratch_length": (ctypes.c_int64, [_P]),
    "rk_conv_grad_scratch_length": (ctypes.c_int64, [_P]),
    "rk_scan_scratch_length": (ctypes.c_int64, [_P]),
    "rk_scan_grad_scratch_length": (ctypes.c_int64, [_P]),
    "rk_norm_encode": (ctypes.c_int32, [_P, _P, _P, _P]),
    "rk_norm_grad_encode": (ctypes.c_int32, [_P, _P, _P, _P, _P]),
    "rk_conv_encode": (ctypes.c_int32, [_P, _P, _P, _P]),
    "rk_conv_grad_encode": (ctypes.c_int32, [_P, _P, _P, _P, _P]),
    "rk_scan_encode": (ctypes.c_int32, [_P, _P, _P, _P, _P]),
    "rk_scan_grad_encode": (ctypes.c_int32, [_P, _P, _P, _P, _P]),
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


_REQUIRED = {
    "norm": ("X",), "norm_grad": ("X", "Mean", "InvStdDev", "dY"), "conv": ("X", "W"), "conv_grad": ("X", "W", "dY"),
    "scan": ("X", "Delta", "A", "B", "C"), "scan_grad": ("X", "Delta", "A", "B", "C", "dY"),
}
_OUTPUTS = {
    "norm": ("Y", "Mean", "InvStdDev"), "norm_grad": ("dX", "dScale", "dB"), "conv": ("Y", "final_state"),
    "conv_grad": ("dX", "dW", "dB", "d_initial_state"), "scan": ("Y", "final_state"),
    "scan_grad": ("dX", "dDelta", "dB", "dC", "dZ", "dA", "dD", "d_delta_bias", "d_initial_state"),
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
    return _binding().Plan(encode, bytes(c), scratch, entries)


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
